"""Cases, plain forms and exact values of the operators that verify drafted
trees over a paged key/value cache:

    attend   attention of every sequence's drafted nodes over its cached
             context and its own ancestors (``tree_attention``)
    verify   accept/reject of drafted tokens against given probabilities with
             given uniforms (``spec_verify_probs``, ``spec_verify_tree``)
    slots    block tables and slot maps from request lengths (``kv_slots``)
    append   keys and values written at their slots (``kv_append``)

``own = False`` computes them with elementary torch operations, ``own = True``
calls the framework.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _sv():
    import speculative_decoding_verification_85_b200 as sv
    return sv


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token of one request: what a decode step without drafts pays (latency)
        dict(name="attend_decode_b1", op="attend", B=1, tree="chain", n_lo=1, n_hi=1, ctx_lo=777,
             ctx_hi=777, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", lse=False),
        # a serving batch with gamma = 4 chains (root + 4 drafted tokens), ragged contexts
        dict(name="attend_chain_b64", op="attend", B=64, tree="chain", n_lo=5, n_hi=5, ctx_lo=1,
             ctx_hi=8192, Hq=32, Hkv=8, D=128, page=16, dtype="bf16", lse=False),
        # wide drafted trees, eight query heads to a key head: 512 query rows per key head
        dict(name="attend_tree_b16", op="attend", B=16, tree="random", n_lo=64, n_hi=64,
             ctx_lo=2000, ctx_hi=16384, Hq=64, Hkv=8, D=128, page=64, dtype="f16", lse=False),
        # one request with a very long context and few rows: the context axis has to be split
        dict(name="attend_long_b1", op="attend", B=1, tree="random", n_lo=26, n_hi=26,
             ctx_lo=131037, ctx_hi=131037, Hq=32, Hkv=4, D=128, page=128, dtype="bf16",
             lse=False),
        # K = 4 drafts of length 5 under one root, no head sharing, an odd head width, contexts
        # from none at all
        dict(name="attend_drafts_b7", op="attend", B=7, tree="drafts", n_lo=21, n_hi=21, ctx_lo=0,
             ctx_hi=1500, Hq=12, Hkv=12, D=80, page=8, dtype="bf16", lse=True),
        # the gamma = 5 step of a batch of 16 (latency)
        dict(name="verify_chain_b16", op="verify", B=16, tree="chain", n_lo=6, n_hi=6, V=32000,
             law="rows", dtype="f32", sigma=3.0, noise=0.7),
        # the large batch: gamma = 4, 256 sequences, the largest vocabulary
        dict(name="verify_chain_b256", op="verify", B=256, tree="chain", n_lo=5, n_hi=5,
             V=151936, law="rows", dtype="f32", sigma=2.5, noise=0.5),
        # drafted trees with i.i.d. children: several residuals in turn at one node
        dict(name="verify_tree_b64", op="verify", B=64, tree="random", n_lo=17, n_hi=31,
             V=128256, law="rows", dtype="bf16", sigma=2.5, noise=1.0),
        # slots of the accepted paths of a verified step
        dict(name="slots_commit_b64", op="slots", B=64, mode="path", n=26, add_lo=1, add_hi=6,
             ctx_lo=1, ctx_hi=8192, page=16),
        # slots and block tables of a batch of prompts
        dict(name="slots_prompt_b512", op="slots", B=512, mode="rows", n=4096, add_lo=1,
             add_hi=4096, ctx_lo=0, ctx_hi=2000, page=16),
        # accepted rows of a verified step, all layers of the model at once
        dict(name="append_commit_l32", op="append", layers=32, B=64, n=5, keep_lo=1, keep_hi=5,
             Hkv=8, D=128, pages=256, page=16, dtype="bf16"),
        # one layer of a batch of prompts
        dict(name="append_prompt", op="append", layers=1, B=16, n=8191, keep_lo=8191,
             keep_hi=8191, Hkv=8, D=128, pages=9000, page=16, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "verify", "verify", "slots", "append"])
    if op == "attend":
        D = rng.choice([128, 128, 64, 8 * rng.randint(2, 16)])
        Hkv = rng.choice([1, 2, 4, 5, 8])
        G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        tree = rng.choice(["chain", "random", "drafts"])
        n = _log(rng, 1, 160)
        if tree == "drafts":
            n = 1 + 5 * max(1, n // 5)
        hi = _log(rng, 1, 100000)
        B = _log(rng, 1, 200)
        # no dearer than the largest listed case (16 x 64 x 64 rows of 9,000 tokens; 64 x 4,096
        # cached tokens of 8 heads)
        B = max(1, min(B, int(64 * 4096 * 8 * 128 / (hi * Hkv * D)),
                       int(16 * 64 * 64 * 9000 / (n * Hkv * G * hi))))
        hi = max(1, min(hi, 64 * 4096 * 8 * 128 // (B * Hkv * D),
                        16 * 64 * 64 * 9000 // (n * Hkv * G * B)))
        lo = rng.choice([0, 1, hi // 2, hi])
        return dict(op="attend", B=B, tree=tree, n_lo=n if tree != "random" else rng.randint(1, n),
                    n_hi=n, ctx_lo=lo, ctx_hi=hi, Hq=Hkv * G, Hkv=Hkv, D=D,
                    page=rng.choice([8, 16, 32, 64, 128, 256]),
                    dtype=rng.choice(["bf16", "f16"]), lse=rng.random() < 0.3)
    if op == "verify":
        tree = rng.choice(["chain", "random", "drafts"])
        n = _log(rng, 2, 64)
        if tree == "drafts":
            n = 1 + 5 * max(1, n // 5)
        V = _log(rng, 1000, 151936)
        B = max(1, min(_log(rng, 1, 256), 256 * 5 * 151936 // (n * V)))
        return dict(op="verify", B=B, tree=tree, n_lo=n if tree != "random" else rng.randint(2, n),
                    n_hi=n, V=V, law=rng.choice(["rows", "rows", "point"]),
                    dtype=rng.choice(["f32", "bf16"]), sigma=rng.choice([2.0, 2.5, 3.0]),
                    noise=rng.choice([0.5, 0.7, 1.0]))
    if op == "slots":
        B = _log(rng, 1, 512)
        if rng.random() < 0.5:
            n = _log(rng, 1, 64)
            return dict(op="slots", B=B, mode="path", n=n, add_lo=0, add_hi=min(n, 9), ctx_lo=0,
                        ctx_hi=_log(rng, 1, 20000), page=rng.choice([8, 16, 32, 64, 128]))
        n = _log(rng, 1, 4096)
        return dict(op="slots", B=B, mode="rows", n=n, add_lo=0, add_hi=n, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 4000), page=rng.choice([8, 16, 32, 64, 128]))
    layers = _log(rng, 1, 32)
    Hkv, D = rng.choice([1, 4, 8]), rng.choice([64, 80, 128])
    n = _log(rng, 1, 500)
    B = max(1, min(_log(rng, 1, 64), 16 * 8192 * 8 * 128 // (layers * n * Hkv * D)))
    page = rng.choice([8, 16, 32, 64])
    pages = B * (-(-n // page)) + 5
    return dict(op="append", layers=layers, B=B, n=n, keep_lo=0, keep_hi=n, Hkv=Hkv, D=D,
                pages=pages, page=page, dtype=rng.choice(["bf16", "f16"]))


# --------------------------------------------------------- sizes of one case
def _spread(lo, hi, B, step=0.6180339887498949):
    """B whole numbers in [lo, hi], spread evenly and in no order; the first
    is the largest."""
    return [hi - int(((b * step) % 1.0) * (hi - lo + 1)) for b in range(B)]


def _cum(xs):
    out = [0]
    for x in xs:
        out.append(out[-1] + x)
    return out


def _gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _tree(kind, n, r):
    """Parents of n nodes, node 0 the root."""
    if kind == "chain":
        return [i - 1 for i in range(n)]
    if kind == "drafts":  # chains of 5 under the root
        return [-1] + [0 if (i - 1) % 5 == 0 else i - 1 for i in range(1, n)]
    par, kids = [-1], [0]
    for i in range(1, n):  # up to 4 children, later nodes preferred: some depth, some width
        while True:
            p = max(r.randrange(i), r.randrange(i))
            if kids[p] < 4:
                break
        par.append(p)
        kids.append(0)
        kids[p] += 1
    return par


def _i32(xs):
    return torch.tensor(xs, dtype=torch.int32, device=DEV)


# --------------------------------------------------------------------- inputs
def prepare(case, seed):
    return {"attend": _prep_attend, "verify": _prep_verify, "slots": _prep_slots,
            "append": _prep_append}[case["op"]](case, seed)


def _prep_attend(c, seed):
    g, r = _gen(seed), random.Random(seed)
    dt = DTYPES[c["dtype"]]
    lens = _spread(c["ctx_lo"], c["ctx_hi"], c["B"])
    nn = _spread(c["n_lo"], c["n_hi"], c["B"])
    N, page, Hkv, D = sum(nn), c["page"], c["Hkv"], c["D"]
    need = [-(-x // page) for x in lens]
    pages = sum(need) + 3
    W = max(max(need), 1)
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((c["B"], W), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)
    st = dict(case=c, lens_list=lens, nn=nn, lens=_i32(lens), cu=_i32(_cum(nn)), table=table,
              parents=_i32([p for n in nn for p in _tree(c["tree"], n, r)]),
              k_cache=rnd(pages, page, Hkv, D), v_cache=rnd(pages, page, Hkv, D),
              q=rnd(N, c["Hq"], D), k=rnd(N, Hkv, D), v=rnd(N, Hkv, D))
    if own:
        sv = _sv()
        st["ws"] = torch.empty(sv.tree_attention_workspace_size(c["Hq"], Hkv, D),
                               dtype=torch.uint8, device=DEV)
    return st


def _prep_verify(c, seed):
    g, r = _gen(seed), random.Random(seed)
    dt, V, B = DTYPES[c["dtype"]], c["V"], c["B"]
    nn = _spread(c["n_lo"], c["n_hi"], B)
    N, cu = sum(nn), _cum(nn)
    par = [_tree(c["tree"], n, r) for n in nn]
    rows = c["law"] == "rows"
    target = torch.empty(N, V, dtype=dt, device=DEV)
    draft = torch.empty(N, V, dtype=dt, device=DEV) if rows else None
    tokens = torch.zeros(N, dtype=torch.int32, device=DEV)
    bias = -1.1 * torch.log(torch.arange(1, V + 1, device=DEV, dtype=torch.float32))
    # whole sequences, about 2**27 probabilities at a time
    per = max(1, (1 << 27) // V)
    b = 0
    while b < B:
        e = b + 1
        while e < B and cu[e + 1] - cu[b] <= per:
            e += 1
        lo, hi = cu[b], cu[e]
        z = torch.randn(hi - lo, V, generator=g, device=DEV) * c["sigma"] + bias
        target[lo:hi] = torch.softmax(z, -1).to(dt)
        z = torch.softmax(z + c["noise"] * torch.randn(hi - lo, V, generator=g, device=DEV), -1)
        z = z.to(dt)
        if rows:
            draft[lo:hi] = z
        up = torch.tensor([cu[s] - lo + max(p, 0) for s in range(b, e) for p in par[s]],
                          device=DEV)
        noise = torch.empty(hi - lo, V, device=DEV).exponential_(generator=g)
        tokens[lo:hi] = (z[up].float() / noise).argmax(-1).to(torch.int32)
        b = e
    # one chain per sequence is laid out as [B, gamma + 1, V], as the chain form takes it
    chain = c["tree"] == "chain" and c["n_lo"] == c["n_hi"] and c["n_hi"] >= 2
    st = dict(case=c, chain=chain, nn=nn, max_nodes=max(nn), depth=max(_depth(p) for p in par),
              kids=max(_kids(p) for p in par), cu=_i32(cu),
              parents=_i32([p for ps in par for p in ps]), target=target, draft=draft,
              tokens=tokens, u=torch.rand(N, generator=g, device=DEV),
              u_draw=torch.rand(B, generator=g, device=DEV))
    if chain:
        n = nn[0]
        st["target"] = target.view(B, n, V)
        st["draft"] = draft.view(B, n, V)[:, :n - 1].contiguous() if rows else None
        st["tokens"] = tokens.view(B, n)[:, 1:].contiguous()
        st["u"] = st["u"].view(B, n)[:, 1:].contiguous()
    return st


def _depth(par):
    d = []
    for p in par:
        d.append(0 if p < 0 else d[p] + 1)
    return max(d)


def _kids(par):
    k = [0] * len(par)
    for p in par:
        if p >= 0:
            k[p] += 1
    return max(k)


def _prep_slots(c, seed):
    r = random.Random(seed)
    B, page, path_mode = c["B"], c["page"], c["mode"] == "path"
    lens = _spread(c["ctx_lo"], c["ctx_hi"], B)
    r.shuffle(lens)
    add = _spread(c["add_lo"], c["add_hi"], B, 0.7548776662466927)
    r.shuffle(add)
    nn = [c["n"]] * B if path_mode else list(add)
    have = [-(-x // page) for x in lens]
    want = [-(-(x + a) // page) for x, a in zip(lens, add)]
    total = sum(want) + 7
    order = list(range(total))
    r.shuffle(order)
    width = max(1, -(-(c["ctx_hi"] + c["add_hi"]) // page))
    table, at = torch.full((B, width), -1, dtype=torch.int32), 0
    for b, h in enumerate(have):
        table[b, :h] = torch.tensor(order[at:at + h], dtype=torch.int32)
        at += h
    free = order[at:]
    path = None
    if path_mode:
        path = torch.full((B, c["n"]), -1, dtype=torch.int32)
        for b in range(B):
            path[b, :add[b]] = torch.tensor(sorted(r.sample(range(c["n"]), add[b])),
                                            dtype=torch.int32)
        path = path.to(DEV)
    pool = _i32(free + [-1] * (total - len(free)))
    return dict(case=c, rows=sum(nn), lens=_i32(lens), add=_i32(add), cu=_i32(_cum(nn)),
                table=table.to(DEV), pool=pool, count=_i32([len(free)]), path=path)


def _prep_append(c, seed):
    g, r = _gen(seed), random.Random(seed)
    dt, n, B = DTYPES[c["dtype"]], c["n"], c["B"]
    keep = _spread(c["keep_lo"], c["keep_hi"], B)
    at = torch.randperm(c["pages"] * c["page"], generator=g, device=DEV)[:n * B].to(torch.int32)
    slots = at.view(B, n).clone()
    for b, k in enumerate(keep):
        if k < n:
            drop = sorted(r.sample(range(n), n - k))
            slots[b, torch.tensor(drop, device=DEV)] = -1
    def rnd(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dt)
    lead = (c["layers"],)
    return dict(case=c, slots=slots.view(-1), k=rnd(*lead, n * B, c["Hkv"], c["D"]),
                v=rnd(*lead, n * B, c["Hkv"], c["D"]),
                k_cache=rnd(*lead, c["pages"], c["page"], c["Hkv"], c["D"]),
                v_cache=rnd(*lead, c["pages"], c["page"], c["Hkv"], c["D"]))


# ----------------------------------------------------------------------- runs
def run(st):
    op = st["case"]["op"]
    if own:
        sv = _sv()
        if op == "attend":
            out, lse = sv.tree_attention(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                                         st["table"], st["lens"], st["parents"], st["cu"],
                                         with_lse=st["case"]["lse"], workspace=st["ws"])
            return [out, lse] if st["case"]["lse"] else [out]
        if op == "verify":
            if st["chain"]:
                acc, tok = sv.spec_verify_probs(st["target"], st["draft"], st["tokens"], st["u"],
                                                st["u_draw"])
                return [acc, tok]
            acc, tok, path = sv.spec_verify_tree(st["target"], st["draft"], st["tokens"],
                                                 st["parents"], st["cu"], st["u"], st["u_draw"],
                                                 max_nodes=st["max_nodes"])
            return [acc, tok, path]
        if op == "slots":
            slots, start, lens, count = sv.kv_slots(
                st["lens"], st["add"], st["cu"], st["table"], st["pool"], st["count"],
                rows=st["rows"], page_size=st["case"]["page"], path=st["path"])
            return [slots, start, lens, count, st["table"]]
        sv.kv_append(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
        return [st["k_cache"], st["v_cache"]]
    return {"attend": _plain_attend, "verify": _plain_verify, "slots": _plain_slots,
            "append": _plain_append}[op](st)


def _plain_attend(st):
    c = st["case"]
    G, D, scale = c["Hq"] // c["Hkv"], c["D"], c["D"] ** -0.5
    outs, lses, at = [], [], 0
    for b, (L, n) in enumerate(zip(st["lens_list"], st["nn"])):
        pages = st["table"][b, :-(-L // c["page"])].long()
        q = st["q"][at:at + n].float().view(n, c["Hkv"], G, D)
        kc = st["k_cache"][pages].reshape(-1, c["Hkv"], D)[:L].float()
        vc = st["v_cache"][pages].reshape(-1, c["Hkv"], D)[:L].float()
        K = torch.cat([kc, st["k"][at:at + n].float()])
        V = torch.cat([vc, st["v"][at:at + n].float()])
        par = st["parents"][at:at + n].long()
        ids = torch.arange(n, device=DEV)
        see = ((ids[:, None] == ids[None]) | (par[:, None] == ids[None])).float()
        for _ in range(max(1, (n - 1).bit_length())):  # ancestors of ancestors
            see = (see @ see > 0).float()
        s = torch.einsum("nhgd,thd->hgnt", q, K) * scale
        s[..., L:] = s[..., L:].masked_fill(see == 0, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - m)
        z = p.sum(-1, keepdim=True)
        o = torch.einsum("hgnt,thd->nhgd", p / z, V)
        outs.append(o.reshape(n, c["Hq"], D).to(st["q"].dtype))
        lses.append((m + torch.log(z)).squeeze(-1).permute(2, 0, 1).reshape(n, c["Hq"]))
        at += n
    out = torch.cat(outs)
    return [out, torch.cat(lses)] if c["lse"] else [out]


def _plain_verify(st):
    """All sequences in step: at the current node the children in order, a
    rejected child taking the node's law to its residual
    max(p - c q, 0) / M, c <- c + M."""
    c = st["case"]
    B, V, rows = c["B"], c["V"], c["law"] == "rows"
    seq = torch.arange(B, device=DEV)
    if st["chain"]:
        n = st["nn"][0]
        N, width = B * n, n
        P = st["target"].reshape(N, V)
        tok = torch.zeros(B, n, dtype=torch.long, device=DEV)
        u = torch.zeros(B, n, dtype=torch.float64, device=DEV)
        tok[:, 1:] = st["tokens"].long()
        u[:, 1:] = st["u"].double()
        tok, u = tok.view(-1), u.view(-1)
        first = seq * n
        # node i's children law is draft row i; the last node has none
        qrow = seq[:, None] * (n - 1) + torch.arange(n, device=DEV).clamp(max=n - 2)[None]
        qrow = qrow.view(-1)
        Q = st["draft"].reshape(B * (n - 1), V) if rows else None
        up = torch.arange(N, device=DEV) - 1
        up[first] = -1
    else:
        P, Q, tok, u = st["target"], st["draft"], st["tokens"].long(), st["u"].double()
        N, width = P.shape[0], st["max_nodes"]
        first = st["cu"][:-1].long()
        qrow = torch.arange(N, device=DEV)
        owner = (torch.arange(N, device=DEV)[:, None] >= st["cu"][None, 1:].long()).sum(1)
        up = torch.where(st["parents"] < 0, -1, st["parents"].long() + first[owner])
    # rank of every node among its siblings, and the table of children by rank
    ids = torch.arange(N, device=DEV)
    run_ = torch.full((N, st["kids"]), -1, dtype=torch.long, device=DEV)
    order = torch.argsort(torch.where(up < 0, N, up), stable=True)
    sup = torch.where(up < 0, N, up)[order]
    rank = ids - torch.searchsorted(sup, sup)
    ok = sup < N
    run_.view(-1).scatter_add_(0, torch.where(ok, sup * st["kids"] + rank, 0),
                               torch.where(ok, order + 1, 0))
    cur = first.clone()
    cc = torch.zeros(B, dtype=torch.float64, device=DEV)
    M = torch.ones(B, dtype=torch.float64, device=DEV)
    gone = torch.zeros(B, V, dtype=torch.bool, device=DEV) if not rows else None
    acc = torch.zeros(B, dtype=torch.int32, device=DEV)
    out = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    path = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    done = torch.zeros(B, dtype=torch.bool, device=DEV)
    for _ in range(st["depth"]):
        moved = torch.zeros(B, dtype=torch.bool, device=DEV)
        here = cur.clone()
        for k in range(st["kids"]):
            child = run_[here, k]
            live = (child >= 0) & ~moved & ~done
            x = tok[child.clamp(min=0)]
            uu = u[child.clamp(min=0)]
            p = P[here, x].double()
            if rows:
                q = Q[qrow[here], x].double()
                hit = uu * q * M < (p - cc * q).clamp(min=0)
            else:
                p = torch.where(gone[seq, x], 0.0, p)
                hit = uu * M < p
            yes, no = live & hit, live & ~hit
            acc += yes.int()
            out[seq, (acc.long() - 1).clamp(min=0)] = torch.where(
                yes, x.int(), out[seq, (acc.long() - 1).clamp(min=0)])
            path[seq, acc.long().clamp(max=width - 1)] = torch.where(
                yes, (child - first).int(), path[seq, acc.long().clamp(max=width - 1)])
            if rows:
                c2 = cc + M
                w = P[here].double() - c2[:, None] * Q[qrow[here]].double()
                M2 = w.clamp_(min=0).sum(1)
                take = no & (M2 > 0)
                cc, M = torch.where(take, c2, cc), torch.where(take, M2, M)
                del w
            else:
                M = torch.where(no, M - p, M)
                gone[seq, x] |= no
            cur = torch.where(yes, child, cur)
            cc, M = torch.where(yes, 0.0, cc), torch.where(yes, 1.0, M)
            if not rows:
                gone &= ~yes[:, None]
            moved |= yes
        done |= ~moved
    w = P[cur].double()
    if rows:
        w = (w - cc[:, None] * Q[qrow[cur]].double()).clamp_(min=0)
    else:
        w = w.masked_fill(gone, 0.0)
    C = w.cumsum(1)
    y = (C <= (st["u_draw"].double() * C[:, -1])[:, None]).sum(1)
    out[seq, acc.long()] = y.int()
    return [acc, out] if st["chain"] else [acc, out, path]


def _plain_slots(st):
    c = st["case"]
    page, B, N = c["page"], c["B"], st["rows"]
    lens, add, table = st["lens"].long(), st["add"].long(), st["table"]
    W = table.shape[1]
    have = (lens + page - 1) // page
    need = (lens + add + page - 1) // page - have
    fits = lens + add <= W * page
    need = torch.where(fits, need, 0)
    upto = need.cumsum(0)
    ok = fits & ((need == 0) | (upto <= st["count"]))
    used = torch.where(ok, upto, 0).amax()
    col = torch.arange(W, device=DEV)[None]
    k = (upto - need)[:, None] + col - have[:, None]
    fresh = ok[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    page_of = st["pool"][(st["count"] - 1 - k).clamp(0, st["pool"].numel() - 1).long()]
    table = torch.where(fresh, page_of, table)
    row = torch.arange(N, device=DEV)
    cu = st["cu"].long()
    b = torch.searchsorted(cu, row, right=True) - 1
    i = row - cu[b]
    if st["path"] is not None:
        same = (st["path"][b] == i[:, None].int()) & (
            torch.arange(st["path"].shape[1], device=DEV)[None] < add[b][:, None])
        kept, i = same.any(1), same.int().argmax(1)
    else:
        kept = i < add[b]
    kept &= ok[b]
    pos = lens[b] + i
    slot = table[b, (pos // page).clamp(max=W - 1)].long() * page + pos % page
    slots = torch.where(kept, slot, -1).int()
    start = torch.where(ok, lens, -1).int()
    return [slots, start, torch.where(ok, lens + add, lens).int(),
            (st["count"] - used).int(), table]


def _plain_append(st):
    kc, vc = st["k_cache"], st["v_cache"]
    c = st["case"]
    tokens = c["pages"] * c["page"]
    # the source row of every slot of the cache, where there is one
    src = torch.full((tokens + 1,), -1, dtype=torch.long, device=DEV)
    at = torch.where(st["slots"] >= 0, st["slots"].long(), tokens)
    src[at] = torch.arange(st["slots"].numel(), device=DEV)
    src = src[:tokens]
    keep = (src < 0)[None, :, None, None]
    for cache, x in ((kc, st["k"]), (vc, st["v"])):
        flat = cache.view(c["layers"], tokens, c["Hkv"], c["D"])
        flat.copy_(torch.where(keep, flat, x[:, src.clamp(min=0)]))
    return [kc, vc]


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "attend":
        lens = _spread(c["ctx_lo"], c["ctx_hi"], c["B"])
        nn = _spread(c["n_lo"], c["n_hi"], c["B"])
        N = sum(nn)
        kv = sum(lens) + N
        # a node sees its context and about its depth of ancestors: counted as the context
        pairs = sum(n * (L + 1) for n, L in zip(nn, lens))
        return {"bytes": 2 * (2 * kv * c["Hkv"] + 2 * N * c["Hq"]) * c["D"],
                "flops": 4 * pairs * c["Hq"] * c["D"]}
    es = {"f32": 4, "bf16": 2, "f16": 2}[c.get("dtype", "f32")]
    if c["op"] == "verify":
        # two gathered probabilities a node; the draw reads the target row it ends at, and the
        # draft row with it where a drafted child was turned down
        nn = _spread(c["n_lo"], c["n_hi"], c["B"])
        share = 1.9 if c["law"] == "rows" else 1.0
        return {"bytes": int(share * c["B"] * c["V"] * es) + 16 * sum(nn),
                "flops": int(2 * share * c["B"] * c["V"])}
    if c["op"] == "slots":
        add = sum(_spread(c["add_lo"], c["add_hi"], c["B"], 0.7548776662466927))
        N = c["B"] * c["n"] if c["mode"] == "path" else add
        return {"bytes": 4 * N + 8 * (add // c["page"] + 1) + 20 * c["B"]
                + (4 * add if c["mode"] == "path" else 0), "flops": 2 * N}
    rows = sum(_spread(c["keep_lo"], c["keep_hi"], c["B"]))
    return {"bytes": 4 * rows * c["layers"] * c["Hkv"] * c["D"] * es + 4 * c["B"] * c["n"],
            "flops": 0}


# ---------------------------------------------------------------- exact values
def exact(case, seed):
    st = prepare(case, seed)
    return {"attend": _exact_attend, "verify": _exact_verify, "slots": _exact_slots,
            "append": _exact_append}[case["op"]](st)


def _exact_attend(st):
    """Softmax attention in 64 bits, one (sequence, key head) at a time, the
    visible nodes found by walking up from every node."""
    c = st["case"]
    G, D, page = c["Hq"] // c["Hkv"], c["D"], c["page"]
    N = st["q"].shape[0]
    out = torch.empty(N, c["Hq"], D, dtype=torch.float64, device=DEV)
    lse = torch.empty(N, c["Hq"], dtype=torch.float64, device=DEV)
    parents = st["parents"].tolist()
    at = 0
    for b, (L, n) in enumerate(zip(st["lens_list"], st["nn"])):
        hide = torch.ones(n, n, dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                hide[i, j] = False
                j = parents[at + j]
        hide = hide.to(DEV)
        pos = torch.arange(L, device=DEV)
        pg, off = st["table"][b].long()[pos // page], pos % page
        for h in range(c["Hkv"]):
            k = torch.cat([st["k_cache"][pg, off, h], st["k"][at:at + n, h]]).double()
            v = torch.cat([st["v_cache"][pg, off, h], st["v"][at:at + n, h]]).double()
            q = st["q"][at:at + n, h * G:(h + 1) * G].double()
            a = (q.reshape(n * G, D) @ k.T).view(n, G, L + n) / math.sqrt(D)
            a[:, :, L:].masked_fill_(hide[:, None, :], -math.inf)
            z = torch.logsumexp(a, -1)
            lse[at:at + n, h * G:(h + 1) * G] = z
            p = torch.exp(a - z[..., None]).view(n * G, L + n)
            out[at:at + n, h * G:(h + 1) * G] = (p @ v).view(n, G, D)
        at += n
    return [out, lse] if c["lse"] else [out]


def _exact_verify(st):
    """Sequence by sequence: the law of the next token held as a normalised
    distribution, updated at every rejection."""
    c = st["case"]
    B, V, rows = c["B"], c["V"], c["law"] == "rows"
    u, ud = st["u"].double().cpu(), st["u_draw"].double().cpu()
    cu, parents = st["cu"].tolist(), st["parents"].tolist()
    width = st["nn"][0] if st["chain"] else st["max_nodes"]
    accs, outs, paths = [], [], []
    for b in range(B):
        n = st["nn"][b]
        if st["chain"]:
            P, Q = st["target"][b], (st["draft"][b] if rows else None)
            par, tok = list(range(-1, n - 1)), [0] + st["tokens"][b].tolist()
            ub = [0.0] + u[b].tolist()
        else:
            lo, hi = cu[b], cu[b + 1]
            P, Q = st["target"][lo:hi], (st["draft"][lo:hi] if rows else None)
            par, tok, ub = parents[lo:hi], st["tokens"][lo:hi].tolist(), u[lo:hi].tolist()
        cur, walk, emitted = 0, [0], []
        while True:
            law = P[cur].double()
            mass = 1.0  # the law is law / mass; the probabilities given are taken as a law
            q = Q[cur].double() if rows and cur in par else None
            nxt = -1
            for k in (i for i in range(n) if par[i] == cur):
                x = tok[k]
                left = float(law[x]) / mass
                if ub[k] * (float(q[x]) if rows else 1.0) < left:
                    nxt = k
                    break
                if rows:
                    r = (law / mass - q).clamp(min=0)
                    if float(r.sum()) > 0:
                        law, mass = r, float(r.sum())
                else:
                    law = law.clone()
                    mass -= float(law[x])
                    law[x] = 0.0
            if nxt < 0:
                break
            cur = nxt
            walk.append(cur)
            emitted.append(tok[cur])
        s = law.cumsum(0)
        y = int((s <= float(ud[b]) * float(s[-1])).sum())
        accs.append(len(emitted))
        outs.append(emitted + [y] + [-1] * (width - len(emitted) - 1))
        paths.append(walk + [-1] * (width - len(walk)))
    res = [_i32(accs), _i32(outs)]
    return res if st["chain"] else res + [_i32(paths)]


def _exact_slots(st):
    c = st["case"]
    page = c["page"]
    lens, add, cu = st["lens"].tolist(), st["add"].tolist(), st["cu"].tolist()
    table, pool, count = st["table"].cpu().clone(), st["pool"].tolist(), st["count"].item()
    path = st["path"].tolist() if st["path"] is not None else None
    slots, start, asked, used = [-1] * st["rows"], [], 0, 0
    for b, (L, a) in enumerate(zip(lens, add)):
        have = -(-L // page)
        need = -(-(L + a) // page) - have
        if L + a > table.shape[1] * page:
            start.append(-1)
            continue
        asked += need
        if need and asked > count:
            start.append(-1)
            continue
        start.append(L)
        for k in range(need):
            table[b, have + k] = pool[count - 1 - (asked - need) - k]
        if need:
            used = asked
        row = table[b].tolist()
        for t in range(a):
            r = cu[b] + (path[b][t] if path else t)
            slots[r] = row[(L + t) // page] * page + (L + t) % page
        lens[b] = L + a
    return [_i32(slots), _i32(start), _i32(lens), _i32([count - used]), table.to(DEV)]


def _exact_append(st):
    c = st["case"]
    out = []
    s = st["slots"].long()
    rows = torch.nonzero(s >= 0)[:, 0]
    for cache, x in ((st["k_cache"], st["k"]), (st["v_cache"], st["v"])):
        new = cache.clone()
        for layer in range(c["layers"]):
            new[layer, s[rows] // c["page"], s[rows] % c["page"]] = x[layer, rows]
        out.append(new)
    return out
