"""Plain 64-bit forms of the drafted-tree operators (numpy, one sequence or
request at a time), written from their definitions; test infrastructure."""
import numpy as np


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def ints(t):
    return None if t is None else t.detach().cpu().numpy().astype(np.int64)


# ----------------------------------------------------------------- verification
def verify_one(P, Q, tokens, parents, u, ud):
    """One tree: P, Q [n, V] (Q None: point drafts).  Returns (accepted node
    indices, drawn token), or None where the data marks the sequence.  The law
    is held normalised and updated at every rejection."""
    n, V = P.shape
    if n < 1 or parents[0] != -1 or any(not 0 <= parents[i] < i for i in range(1, n)):
        return None
    if not 0 <= ud < 1:
        return None
    for i in range(1, n):
        if not 0 <= tokens[i] < V or not 0 <= u[i] < 1:
            return None
        vals = [P[parents[i], tokens[i]]] + ([Q[parents[i], tokens[i]]] if Q is not None else [])
        if not all(np.isfinite(x) and x >= 0 for x in vals):
            return None
    cur, path = 0, []
    while True:
        law, mass = P[cur].copy(), 1.0
        nxt = None
        for i in range(1, n):
            if parents[i] != cur:
                continue
            x = tokens[i]
            if u[i] * (Q[cur, x] if Q is not None else 1.0) < max(law[x], 0.0) / mass:
                nxt = i
                break
            if Q is None:
                mass -= law[x]
                law[x] = 0.0
            else:
                r = law / mass - Q[cur]
                r[r < 0] = 0.0
                if not np.isfinite(r.sum()):
                    return None
                if r.sum() > 0:
                    law, mass = r, r.sum()
        if nxt is None:
            break
        cur = nxt
        path.append(cur)
    law[law < 0] = 0.0
    with np.errstate(invalid="ignore"):
        C = np.cumsum(law)
    if not (np.isfinite(C[-1]) and C[-1] > 0):
        return None
    y = int(np.searchsorted(C, ud * C[-1], side="right"))
    return path, y


def verify_tree(P, Q, tokens, parents, cu, u, ud, width):
    """Packed trees; the arrays spec_verify_tree fills."""
    B = len(cu) - 1
    acc = np.full(B, -1)
    out, paths = np.full((B, width), -1), np.full((B, width), -1)
    for b in range(B):
        lo, hi = cu[b], cu[b + 1]
        if lo < 0 or hi > len(tokens) or hi - lo < 1 or hi - lo > min(width, 1024):
            continue
        s = slice(lo, hi)
        got = verify_one(P[s], None if Q is None else Q[s], tokens[s], parents[s], u[s], ud[b])
        if got is None:
            continue
        path, y = got
        acc[b] = len(path)
        for i, node in enumerate(path):
            out[b, i] = tokens[lo + node]
            paths[b, i + 1] = node
        out[b, len(path)] = y
        paths[b, 0] = 0
    return acc, out, paths


def verify_chain(P, Q, tokens, u, ud):
    """[B, g+1, V] chains; the arrays spec_verify_probs fills."""
    B, g1, V = P.shape
    acc, out = np.full(B, -1), np.full((B, g1), -1)
    for b in range(B):
        q = None
        if Q is not None:
            q = np.concatenate([Q[b], np.zeros((1, V))])
        got = verify_one(P[b], q, np.concatenate([[0], tokens[b]]), np.arange(-1, g1 - 1),
                         np.concatenate([[0.0], u[b]]), ud[b])
        if got is None:
            continue
        path, y = got
        acc[b] = len(path)
        out[b, :len(path)] = tokens[b][:len(path)]
        out[b, len(path)] = y
    return acc, out


# ------------------------------------------------------------------- slot maps
def kv_slots(lens, add, cu, table, pool, count, rows, page, path=None):
    """Returns (slots, start, lens, count, table, pool), all new."""
    lens, table, pool = lens.copy(), table.copy(), pool.copy()
    B, W = table.shape
    slots, start = np.full(rows, -1), np.full(B, -1)
    count = min(max(count, 0), len(pool))
    asked = popped = 0
    release = []
    for b in range(B):
        L, a, lo, hi = lens[b], add[b], cu[b], cu[b + 1]
        if not 0 <= L <= W * page or a < -1 or lo < 0 or hi > rows or hi < lo:
            continue
        have = -(-L // page)
        if a == -1:
            release.append((b, have))
            continue
        if a > hi - lo or L + a > W * page:
            continue
        keep = list(range(a))
        if path is not None:
            if a > path.shape[1]:
                continue
            keep = list(path[b, :a])
            if any(x < 0 or x >= hi - lo for x in keep) or any(
                    y <= x for x, y in zip(keep, keep[1:])):
                continue
        need = -(-(L + a) // page) - have
        asked += need
        if need and asked > count:
            continue
        for k in range(need):
            table[b, have + k] = pool[count - 1 - (asked - need + k)]
        popped = max(popped, asked if need else 0)
        start[b] = L
        lens[b] = L + a
        for t, i in enumerate(keep):
            at = int(table[b, (L + t) // page])
            slots[lo + i] = at * page + (L + t) % page if at >= 0 else -1
    top = count - popped
    for b, have in release:
        for k in range(have):
            if top < len(pool):
                pool[top] = table[b, k]
            top += 1
        lens[b] = 0
    return slots, start, lens, min(top, len(pool)), table, pool


# ------------------------------------------------------------------- attention
def attention(q, k, v, k_cache, v_cache, table, lens, parents, cu, scale):
    """(out [N, Hq, D], lse [N, Hq]); rows of no sequence are 0 / 0."""
    N, Hq, D = q.shape
    Hkv, page = k.shape[1], k_cache.shape[1]
    G = Hq // Hkv
    out, lse = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(lens)):
        t = np.arange(lens[b])
        pg = table[b][t // page]
        for i in range(cu[b], cu[b + 1]):
            seen, j = [], i - cu[b]
            while j >= 0:
                seen.append(cu[b] + j)
                j = parents[cu[b] + j]
            for h in range(Hq):
                K = np.concatenate([k_cache[pg, t % page, h // G], k[seen, h // G]])
                V = np.concatenate([v_cache[pg, t % page, h // G], v[seen, h // G]])
                s = K @ q[i, h] * scale
                m = s.max()
                p = np.exp(s - m)
                out[i, h] = (p[:, None] * V).sum(0) / p.sum()
                lse[i, h] = m + np.log(p.sum())
    return out, lse


def attention_t(q, k, v, k_cache, v_cache, table, lens, parents, cu, scale):
    """`attention` in torch float64, a sequence at a time on the tensors'
    device: (out, lse, mean absolute value under the weights)."""
    import torch
    N, Hq, D = q.shape
    Hkv, page = k.shape[1], k_cache.shape[1]
    G = Hq // Hkv
    dev = q.device
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device=dev)
    mag, lse = torch.zeros_like(out), torch.zeros(N, Hq, dtype=torch.float64, device=dev)
    cu, lens, par = cu.tolist(), lens.tolist(), parents.tolist()
    for b, L in enumerate(lens):
        lo, n = cu[b], cu[b + 1] - cu[b]
        if n <= 0:
            continue
        see = torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            j = i
            while j >= 0:
                see[i, j] = True
                j = par[lo + j]
        see = see.to(dev)
        t = torch.arange(L, device=dev)
        pg = table[b].long()[t // page]
        for h in range(Hkv):
            # what no row of the column sees is cleared; what only some see is masked
            K = torch.cat([k_cache[pg, t % page, h], k[lo:lo + n, h]]).double()
            V = torch.cat([v_cache[pg, t % page, h], v[lo:lo + n, h]]).double()
            Q = q[lo:lo + n, h * G:(h + 1) * G].double()
            s = torch.einsum("ngd,td->ngt", Q, K) * scale
            s[:, :, L:] = torch.where(see[:, None], s[:, :, L:], -torch.inf)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[..., None])
            o = torch.einsum("ngt,td->ngd", p, V.nan_to_num(0, 0, 0))
            for c in torch.nonzero(~V.isfinite().all(1))[:, 0].tolist():  # 0 * inf in masked places
                w = p[:, :, c, None] * torch.where(V[c].isfinite(), 0.0, V[c])
                seen = torch.ones(n, dtype=torch.bool, device=dev) if c < L else see[:, c - L]
                o = o + torch.where(seen[:, None, None], w, 0.0)
            r = slice(lo, lo + n), slice(h * G, (h + 1) * G)
            out[r], lse[r] = o, z
            mag[r] = torch.einsum("ngt,td->ngd", p, V.nan_to_num(0, 0, 0).abs())
    return out, lse, mag
