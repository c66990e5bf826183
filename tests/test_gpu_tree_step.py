"""The drafted-tree operators together, as a decoding loop uses them: a toy
model (random projections, one attention layer after the other) decoded with
drafted trees over a PagedCache.

Its next-token laws have to be those of the same model run plainly in 64 bits
over each sequence's whole text, its cache has to hold exactly the accepted
tokens' rows, and a captured step replays to the same result."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import tree_oracle as to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
V, D, HQ, HKV, LAYERS, B = 997, 64, 8, 2, 2, 5


class Toy:
    """Embedding -> LAYERS x (q, k, v projections, attention, residual) ->
    logits; positions enter through the tree only."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def rnd(*s):
            return torch.randn(*s, generator=g, device=DEV)

        self.emb = rnd(V, HQ * D)
        self.wq = rnd(LAYERS, HQ * D, HQ * D) / (HQ * D) ** 0.5
        self.wkv = rnd(LAYERS, 2, HQ * D, HKV * D) / (HQ * D) ** 0.5
        self.head = rnd(HQ * D, V) / (HQ * D) ** 0.5 * 2

    def nodes(self, tokens, attend):
        """tokens [N] -> probabilities [N, V] and keys, values [L, N, HKV, D]."""
        x = self.emb[tokens.long()]
        ks, vs = [], []
        for layer in range(LAYERS):
            q = (x @ self.wq[layer]).view(-1, HQ, D).bfloat16()
            k, v = ((x @ self.wkv[layer, i]).view(-1, HKV, D).bfloat16() for i in range(2))
            x = x + attend(layer, q, k, v).float().flatten(1)
            ks.append(k)
            vs.append(v)
        return torch.softmax(x @ self.head, -1), torch.stack(ks), torch.stack(vs)


def _trees(rng, b):
    par = []
    for _ in range(b):
        par.append([-1] + [int(rng.integers(max(0, i - 3), i)) for i in range(1, 9)])
    return par


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def test_decoding_loop():
    rng = np.random.default_rng(1)
    g = torch.Generator(device=DEV).manual_seed(2)
    model = Toy(3)
    cache = sv.PagedCache(LAYERS, 64, 16, HKV, D, B, 256)
    texts = [list(rng.integers(0, V, n)) for n in (1, 7, 30, 16, 47)]
    # the prompts: all but the last token of each, one chain per request
    prompt = [t[:-1] for t in texts]
    cu = _i32(np.concatenate([[0], np.cumsum([len(p) for p in prompt])]))
    par = _i32([i - 1 for p in prompt for i in range(len(p))])
    _, k, v = model.nodes(_i32([x for p in prompt for x in p]),
                          lambda layer, q, k, v: cache.attend(layer, q, k, v, par, cu)[0])
    cache.extend(k, v, cu, _i32([len(p) for p in prompt]))
    accepted = 0
    for step in range(8):
        parents = _trees(rng, B)
        n = len(parents[0])
        cu = _i32(np.arange(B + 1) * n)
        par = _i32([p for t in parents for p in t])
        draft = torch.softmax(torch.randn(B * n, V, generator=g, device=DEV), -1)
        tok = torch.empty(B * n, dtype=torch.int32, device=DEV)
        up = torch.tensor([b * n + max(p, 0) for b, t in enumerate(parents) for p in t], device=DEV)
        if step % 2:  # a draft law close to the target's, so that branches are accepted
            probe = torch.zeros(B * n, dtype=torch.int32, device=DEV)
            probe[::n] = _i32([t[-1] for t in texts])
            near, _, _ = model.nodes(probe, lambda layer, q, k, v: cache.attend(
                layer, q, k, v, par, cu)[0])
            draft = near[::n].repeat_interleave(n, 0)
        e = torch.empty(B * n, V, device=DEV).exponential_(generator=g)
        tok[:] = (draft[up] / e).argmax(-1).int()
        tok[::n] = _i32([t[-1] for t in texts])
        probs, k, v = model.nodes(tok, lambda layer, q, k, v: cache.attend(
            layer, q, k, v, par, cu)[0])
        u = torch.rand(B * n, generator=g, device=DEV)
        ud = torch.rand(B, generator=g, device=DEV)
        acc, out, path = sv.spec_verify_tree(probs, draft, tok, par, cu, u, ud, max_nodes=n)
        lens = cache.lens.clone()
        start = cache.commit(k, v, cu, acc, path)
        assert torch.equal(start, lens) and torch.equal(cache.lens, lens + acc + 1)
        # verification against the plain form on the same probabilities
        want = to.verify_tree(to.f64(probs), to.f64(draft), to.ints(tok), to.ints(par),
                              to.ints(cu), to.f64(u), to.f64(ud), n)
        for got, w in zip((acc, out, path), want):
            assert np.array_equal(got.cpu().numpy(), w)
        for b in range(B):
            # the node's law is that of its whole text, run plainly in 64 bits
            node = int(path[b, int(acc[b])])
            text = texts[b] + out[b, :int(acc[b])].tolist()
            law = _plain(model, text)
            # (q, k, v, the weights and the outputs are rounded by 2^-8 at most: a layer's
            # attention output is off by 5 * 2^-8 = 2% of itself at worst, its sum with the
            # residual by less)
            assert (probs[b * n + node].double() - law).abs().max() < 0.02 * law.max()
            texts[b] = text + [int(out[b, int(acc[b])])]
            # the cache holds the text but its last token, in order
            assert int(cache.lens[b]) == len(texts[b]) - 1
        accepted += int(acc.sum())
    assert accepted > 0
    # pages go back and are found again
    used = int((cache.block_table >= 0).sum())
    assert int(cache.free_count) == 64 - used
    cache.release(torch.tensor([True, False, True, False, True], device=DEV))
    assert cache.lens.tolist()[::2] == [0, 0, 0]
    cache.release(torch.ones(B, dtype=torch.bool, device=DEV))
    assert int(cache.free_count) == 64
    assert sorted(cache.free_pages.tolist()) == list(range(64))


def _plain(model, text):
    """The law of the token after `text`, in 64 bits, attention over it all."""
    x = model.emb[torch.tensor(text, device=DEV)].double()
    n = len(text)
    mask = torch.ones(n, n, dtype=torch.bool, device=DEV).triu(1)
    for layer in range(LAYERS):
        q = (x @ model.wq[layer].double()).view(n, HKV, HQ // HKV, D)
        k, v = ((x @ model.wkv[layer, i].double()).view(n, HKV, D) for i in range(2))
        s = torch.einsum("nhgd,thd->hgnt", q, k) * D ** -0.5
        p = torch.softmax(s.masked_fill(mask, -torch.inf), -1)
        x = x + torch.einsum("hgnt,thd->nhgd", p, v).reshape(n, -1)
    return torch.softmax(x[-1] @ model.head.double(), -1)


def test_full_cache_refuses_and_recovers():
    cache = sv.PagedCache(1, 4, 16, 1, 64, 3, 64)
    rows = [20, 40, 10]
    cu = _i32(np.concatenate([[0], np.cumsum(rows)]))
    k = torch.randn(1, 70, 1, 64, device=DEV).bfloat16()
    start = cache.extend(k, k, cu, _i32(rows))
    assert start.tolist() == [0, -1, -1] and cache.lens.tolist() == [20, 0, 0]
    cache.release(torch.tensor([True, False, False], device=DEV))
    start = cache.extend(k, k, cu, _i32([0, 40, 10]))
    assert start.tolist() == [0, 0, 0] and cache.lens.tolist() == [0, 40, 10]
    got = cache.k[0][cache.block_table[1, :3].long()].flatten(0, 1)[:40]
    assert torch.equal(got, k[0, 20:60])


def test_captured_step_replays():
    """Attention, verification, slots and append captured once; two replays
    advance the cache as two plain steps do."""
    g = torch.Generator(device=DEV).manual_seed(5)
    n, steps = 4, 2
    cu, par = _i32(np.arange(B + 1) * n), _i32([-1, 0, 0, 1] * B)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV).bfloat16()

    data = [dict(q=rnd(B * n, HQ, D), k=rnd(1, B * n, HKV, D), v=rnd(1, B * n, HKV, D),
                 p=torch.softmax(rnd(B * n, V).float(), -1), d=torch.softmax(rnd(B * n, V).float(), -1),
                 t=torch.randint(V, (B * n,), device=DEV, dtype=torch.int32, generator=g),
                 u=torch.rand(B * n, device=DEV, generator=g), w=torch.rand(B, device=DEV, generator=g))
            for _ in range(steps)]

    def fresh():
        c = sv.PagedCache(1, 40, 16, HKV, D, B, 128)
        c.extend(data[0]["k"], data[0]["v"], cu, _i32([4, 3, 2, 1, 0]))
        return c

    def step(c, x):
        out, _ = c.attend(0, x["q"], x["k"][0], x["v"][0], par, cu)
        acc, tok, path = sv.spec_verify_tree(x["p"], x["d"], x["t"], par, cu, x["u"], x["w"],
                                             max_nodes=n)
        c.commit(x["k"], x["v"], cu, acc, path)
        return out, tok

    plain, want = fresh(), []
    for x in data:
        want.append([t.clone() for t in step(plain, x)])
    cap, static = fresh(), {k: t.clone() for k, t in data[0].items()}
    snap = [t.clone() for t in (cap.k, cap.v, cap.block_table, cap.lens, cap.free_pages, cap.free_count)]
    step(cap, static)  # warm up, then back to the start
    for t, s in zip((cap.k, cap.v, cap.block_table, cap.lens, cap.free_pages, cap.free_count), snap):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = step(cap, static)
    for x, w in zip(data, want):
        for k, t in static.items():
            t.copy_(x[k])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, w))
    for a, b in ((cap.lens, plain.lens), (cap.block_table, plain.block_table), (cap.k, plain.k),
                 (cap.v, plain.v), (cap.free_count, plain.free_count)):
        assert torch.equal(a, b)
