"""tree_attention against the plain 64-bit form.

Tolerance, from the number formats: the weights and the output are rounded to
the input type once each, half a step h = eps / 2 relative (bf16 2^-8, fp16
2^-11), so an output moves by at most h (A + |o|) with A = sum p |v| / sum p;
fp32 products of D = 128 terms move a score by less than 2e-5 at these
magnitudes (128 * 2^-24 * sum |q k| scale), the exponentials by 2^-22: 1e-4 A
covers both.  lse carries the score's error and the sum's: 1e-4."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import tree_oracle as to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def tree(n, kind, rng):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "roots":
        return [-1] * n
    return [-1] + [int(rng.integers(max(0, i - 9), i)) for i in range(1, n)]


def make(lens, nodes, Hq, Hkv, D, page, dtype, kind="tree", seed=0, spare=3):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    need = [-(-x // page) for x in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(lens), max(max(need, default=0), 1)), -1)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    N = sum(nodes)

    def rnd(*s):
        return torch.randn(*s, generator=g, device=DEV).to(DT[dtype])

    return dict(q=rnd(N, Hq, D), k=rnd(N, Hkv, D), v=rnd(N, Hkv, D),
                k_cache=rnd(pages, page, Hkv, D), v_cache=rnd(pages, page, Hkv, D),
                block_table=i32(table), lens=i32(lens),
                parents=i32([p for n in nodes for p in (tree(n, kind, rng) if n else [])]),
                cu_nodes=i32(np.concatenate([[0], np.cumsum(nodes)])))


def ref(st, scale=None):
    D = st["q"].shape[-1]
    return to.attention_t(st["q"], st["k"], st["v"], st["k_cache"], st["v_cache"],
                          st["block_table"], st["lens"], st["parents"], st["cu_nodes"],
                          D ** -0.5 if scale is None else scale)


def close(out, lse, want):
    o, z, mag = want
    h = torch.finfo(out.dtype).eps / 2
    fin = o.isfinite()
    assert torch.equal(out.isnan(), o.isnan())
    same = out.double()[~fin] == o[~fin]
    assert (same | o[~fin].isnan()).all()
    err = (out.double() - o).abs()[fin]
    lim = (h * (mag + o.abs()) + 1e-4 * mag + 1e-7)[fin]
    assert (err <= lim).all(), f"worst {(err / lim).max().item():.3f} of the limit"
    if lse is not None:
        assert ((lse.double() - z).abs() <= 1e-4).all()


def check(st, **kw):
    out, lse = sv.tree_attention(**st, with_lse=True, **kw)
    torch.cuda.synchronize()
    close(out, lse, ref(st, kw.get("scale")))
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv,D,page,kind", [
    ([1], [1], 1, 1, 64, 16, "chain"),
    ([0], [1], 2, 2, 128, 8, "chain"),
    ([777], [1], 32, 8, 128, 16, "chain"),
    ([128, 127, 129, 0, 5], [5, 1, 7, 3, 0], 8, 2, 128, 16, "tree"),
    ([300, 1000, 64], [16, 33, 64], 16, 2, 128, 64, "tree"),
    ([50, 700], [40, 21], 12, 12, 80, 8, "tree"),
    ([260, 513], [130, 300], 4, 4, 64, 32, "tree"),
    ([100], [300], 16, 2, 128, 128, "chain"),
    ([1000, 3], [9, 128], 5, 1, 40, 256, "tree"),
    ([513, 90], [50, 11], 21, 3, 8, 32, "tree"),
    ([200, 300], [1, 2], 128, 1, 128, 16, "chain"),
    ([400], [3], 100, 1, 104, 384, "roots"),
    ([64, 64], [17, 129], 7, 7, 72, 8, "roots"),
])
def test_shapes(lens, nodes, Hq, Hkv, D, page, kind, dtype):
    check(make(lens, nodes, Hq, Hkv, D, page, dtype, kind, seed=len(lens) + D))


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(seed):
    rng = np.random.default_rng(100 + seed)
    B = int(rng.integers(1, 12))
    Hkv, G = int(rng.integers(1, 9)), int(rng.integers(1, 17))
    lens = [int(x) for x in (rng.random(B) ** 3 * 4000)]
    nodes = [int(rng.integers(0, 70)) for _ in range(B)]
    check(make(lens, nodes, Hkv * G, Hkv, 8 * int(rng.integers(1, 17)),
               int(rng.choice([8, 16, 32, 64, 128, 256])), str(rng.choice(["bf16", "f16"])),
               str(rng.choice(["chain", "tree"])), seed))


@pytest.mark.parametrize("nodes,Hq,Hkv", [(1, 8, 8), (26, 32, 4), (64, 16, 1), (5, 4, 1)])
def test_long_context_is_split(nodes, Hq, Hkv):
    check(make([40001], [nodes], Hq, Hkv, 128, 16, "bf16", seed=nodes))


def test_many_sequences():
    """More sequences than one round of the prefix sums takes, some empty."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(0, 200, 900)]
    nodes = [int(x) for x in rng.integers(0, 4, 900)]
    check(make(lens, nodes, 4, 2, 64, 16, "bf16", seed=5))


def test_largest_tree():
    check(make([10], [1024], 2, 1, 64, 16, "bf16", "tree", seed=6))
    check(make([200], [1024], 1, 1, 128, 16, "f16", "chain", seed=7))


def test_growing_and_extreme_scores():
    """Scores that grow along the context (the accumulator is rescaled again
    and again), that fall, that are all equal, and of one dominant key."""
    st = make([3000, 700], [9, 20], 8, 2, 128, 16, "bf16", seed=8)
    grow = torch.linspace(0.0, 6.0, st["k_cache"].shape[0], device=DEV)
    for f in (grow, grow.flip(0)):
        order = torch.empty_like(f)
        used = st["block_table"][0].long()
        order[:] = 1.0
        order[used] = f[:used.numel()]
        check(dict(st, k_cache=(st["k_cache"].float() * order[:, None, None, None]).bfloat16()))
    check(dict(st, q=torch.zeros_like(st["q"])))
    k = st["k_cache"].clone()
    k[st["block_table"][0, 100], 3] = st["q"][0, 0] * 8
    check(dict(st, k_cache=k))
    check(st, scale=2.0)
    check(st, scale=1e-3)


def test_masked_places_hold_anything():
    """Unused pages, the rest of last pages, other branches and neighbours'
    rows hold NaN and infinities: the results are those without them."""
    for dtype, kind in (("bf16", "tree"), ("f16", "roots")):
        st = make([37, 300, 0], [20, 150, 3], 8, 2, 128, 16, dtype, kind, seed=9)
        base, blse = check(st)
        bad = {k: t.clone() for k, t in st.items()}
        used = set(st["block_table"][0, :3].tolist()) | set(st["block_table"][1, :19].tolist())
        for p in range(st["k_cache"].shape[0]):
            if p not in used:
                bad["k_cache"][p], bad["v_cache"][p] = float("nan"), float("inf")
        bad["k_cache"][st["block_table"][0, 2], 5:] = float("inf")
        bad["v_cache"][st["block_table"][0, 2], 5:] = float("nan")
        bad["v_cache"][st["block_table"][1, 18], 12:] = float("-inf")
        # a node that nobody else sees: the last one of the first two sequences
        for i in (19, 169):
            bad["k"][i], bad["v"][i] = float("nan"), float("nan")
            bad["v"][i, :, ::3] = float("inf")
        out, lse = sv.tree_attention(**bad, with_lse=True)
        keep = torch.ones(173, dtype=torch.bool, device=DEV)
        keep[[19, 169]] = False
        assert torch.equal(out[keep], base[keep]) and torch.equal(lse[keep], blse[keep])
        assert out[19].isnan().all() and out[169].isnan().all()


def test_visible_infinities_reach_those_who_see_them():
    st = make([40, 300], [20, 33], 8, 2, 128, 16, "bf16", "tree", seed=10)
    st["v"][3, 0, 7] = float("inf")
    st["v"][5, 1, 9] = float("-inf")
    st["v"][21, 1, 127] = float("nan")
    st["v_cache"][st["block_table"][1, 2], 4, 0, 64] = float("inf")
    out, _ = sv.tree_attention(**st)
    close(out, None, ref(st))
    assert out[3, 0, 7] == float("inf") and out[20:, 0, 64].isinf().all()


def test_marks():
    """One bad sequence at a time gets NaN; the others keep their results."""
    st = make([300, 500, 64, 900], [5, 30, 2, 9], 8, 2, 128, 16, "bf16", "chain", seed=11)
    base, _ = check(st)

    def spoil(f, rows):
        bad = {k: t.clone() for k, t in st.items()}
        f(bad)
        out, lse = sv.tree_attention(**bad, with_lse=True)
        hit = torch.zeros(46, dtype=torch.bool, device=DEV)
        hit[rows] = True
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(out[~hit], base[~hit])

    W = st["block_table"].shape[1]
    one = slice(5, 35)
    spoil(lambda s: s["lens"][1:2].fill_(-1), one)
    spoil(lambda s: s["lens"][1:2].fill_(W * 16 + 1), one)
    for page in (-1, st["k_cache"].shape[0], 2**31 - 1, -2**31):
        spoil(lambda s, page=page: s["block_table"][1, 7:8].fill_(page), one)
        spoil(lambda s, page=page: s["block_table"][3, 56:57].fill_(page), slice(37, 46))
    # node 10 of sequence 1 and every node behind it in the chain
    for p in (10, 29, -2, 500):
        spoil(lambda s, p=p: s["parents"][15:16].fill_(p), slice(15, 35))
    # bounds that do not lie in the buffers: those rows are left alone
    bad = dict(st, cu_nodes=i32([-3, 5, 35, 37, 60]))
    out = torch.full_like(base, 7.0)
    sv.tree_attention(**bad, out=out)
    assert torch.equal(out[5:37], base[5:37])
    assert (out[:5] == 7).all() and (out[37:] == 7).all()
    # more nodes than a tree may have
    big = make([10, 20], [1025, 3], 2, 1, 64, 16, "bf16", "chain", seed=12)
    out, _ = sv.tree_attention(**big)
    assert out[:1025].isnan().all() and not out[1025:].isnan().any()


def test_rows_behind_the_last_sequence_stay():
    st = make([100, 40], [5, 9], 8, 2, 128, 16, "bf16", seed=13)
    pad = {k: torch.cat([st[k], torch.full_like(st[k][:6], float("nan"))]) for k in "qkv"}
    pad["parents"] = torch.cat([st["parents"], i32([9] * 6)])
    out = torch.full((20, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((20, 8), 4.0, device=DEV)
    sv.tree_attention(**{**st, **pad}, out=out, out_lse=lse)
    close(out[:14], lse[:14], ref(st))
    assert (out[14:] == 3).all() and (lse[14:] == 4).all()


def test_strides():
    """Fused projections, pages with the heads first, keys and values of a
    page together, a wider block table."""
    st = make([100, 333], [7, 20], 8, 2, 64, 16, "f16", seed=14)
    base, _ = check(st)
    qkv = torch.cat([st["q"].flatten(1), st["k"].flatten(1), st["v"].flatten(1)], 1)
    q, k, v = (t.unflatten(1, (-1, 64)) for t in qkv.split([512, 128, 128], 1))
    pages = st["k_cache"].shape[0]
    both = torch.empty(pages, 2, 2, 16, 64, dtype=torch.float16, device=DEV)
    both[:, 0], both[:, 1] = st["k_cache"].transpose(1, 2), st["v_cache"].transpose(1, 2)
    wide = torch.full((2, st["block_table"].shape[1] + 9), -1, dtype=torch.int32, device=DEV)
    wide[:, :-9] = st["block_table"]
    out, _ = sv.tree_attention(q, k, v, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2),
                               wide[:, :-9], st["lens"], st["parents"], st["cu_nodes"])
    assert torch.equal(out, base)


def test_workspace_streams_and_graphs():
    """A workspace of any content, reused; a side stream; two calls at once on
    two streams; a captured call replayed with other lengths; equal results
    every time."""
    size = sv.tree_attention_workspace_size(16, 2, 128)
    a = make([9000, 70], [9, 30], 16, 2, 128, 16, "bf16", seed=15)
    b = make([300, 20000], [9, 30], 16, 2, 128, 16, "bf16", seed=16)
    want = [sv.tree_attention(**st)[0] for st in (a, b)]
    close(want[0], None, ref(a))
    close(want[1], None, ref(b))
    ws = torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    for st, w in ((a, want[0]), (b, want[1]), (a, want[0])):
        assert torch.equal(sv.tree_attention(**st, workspace=ws)[0], w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [sv.tree_attention(**st, stream=s)[0] for st, s in zip((a, b), streams)]
        for s in streams:
            s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    st = {k: t.clone() for k, t in a.items()}
    if st["block_table"].shape != b["block_table"].shape:
        W = max(a["block_table"].shape[1], b["block_table"].shape[1])
        P = max(a["k_cache"].shape[0], b["k_cache"].shape[0])

        def fit(x):
            x = dict(x)
            x["block_table"] = torch.nn.functional.pad(
                x["block_table"], (0, W - x["block_table"].shape[1]), value=-1)
            for c in ("k_cache", "v_cache"):
                x[c] = torch.cat([x[c], x[c][:1].expand(P - x[c].shape[0], -1, -1, -1)])
            return x

        a, b = fit(a), fit(b)
        st = {k: t.clone() for k, t in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = sv.tree_attention(**st)
    for src, w in ((b, want[1]), (a, want[0])):
        for k, t in st.items():
            t.copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)


def test_nothing_to_do():
    st = make([10], [2], 4, 2, 64, 16, "bf16", seed=17)
    none = dict(st, q=st["q"][:0], k=st["k"][:0], v=st["v"][:0], parents=st["parents"][:0])
    out, lse = sv.tree_attention(**none, with_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out = torch.full_like(st["q"], 2.0)
    sv.tree_attention(**dict(st, cu_nodes=i32([0, 0])), out=out)
    sv.tree_attention(**dict(st, cu_nodes=i32([0]), lens=st["lens"][:0],
                             block_table=st["block_table"][:0]), out=out)
    assert (out == 2).all()


def test_pages_beyond_32_bit_offsets():
    """A cache of more than 2^31 elements, its last pages in use."""
    st = make([300], [9], 8, 2, 128, 16, "bf16", seed=18)
    pages = 2**31 // (16 * 2 * 128) + 64
    kc, vc = (torch.empty(pages, 16, 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    n = st["k_cache"].shape[0]
    kc[-n:], vc[-n:] = st["k_cache"], st["v_cache"]
    want, _ = check(st)
    out, _ = sv.tree_attention(**dict(st, k_cache=kc, v_cache=vc,
                                      block_table=st["block_table"] + (pages - n)))
    assert torch.equal(out, want)
