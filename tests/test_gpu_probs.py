"""spec_verify_probs and spec_verify_tree against the plain 64-bit form:
accept lengths, tokens and paths are equal (both sides compare and sum in
fp64; a border within 1e-15 of a given fp32 uniform does not occur in these
seeded inputs)."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import tree_oracle as to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _parents(kind, n, rng):
    if kind == "chain":
        return list(range(-1, n - 1))
    if kind == "star":
        return [-1] + [0] * (n - 1)
    return [-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, n)]


def make(B, sizes, V, dtype, kind, seed, law=True, sigma=2.0, noise=0.7):
    """Packed trees with tokens drawn from their parents' draft rows."""
    rng = np.random.default_rng(seed)
    g = torch.Generator(device=DEV).manual_seed(seed)
    nn = [sizes[b % len(sizes)] for b in range(B)]
    cu = np.concatenate([[0], np.cumsum(nn)])
    N = int(cu[-1])
    par = [p for n in nn for p in (_parents(kind, n, rng) if n else [])]
    z = torch.randn(N, V, generator=g, device=DEV) * sigma
    target = torch.softmax(z, -1).to(DT[dtype])
    draft = torch.softmax(z + noise * torch.randn(N, V, generator=g, device=DEV), -1).to(DT[dtype])
    first = np.repeat(cu[:-1], nn)
    up = torch.tensor(first + np.maximum(par, 0), device=DEV, dtype=torch.long)
    e = torch.empty(N, V, device=DEV).exponential_(generator=g)
    tokens = (draft[up].float() / e).argmax(-1).to(torch.int32)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(target=target, draft=draft if law else None, tokens=tokens,
                parents=torch.tensor(par, **i32), cu_nodes=torch.tensor(cu, **i32),
                uniforms=torch.rand(N, generator=g, device=DEV),
                draw_uniforms=torch.rand(B, generator=g, device=DEV))


def run(st, width):
    acc, tok, path = sv.spec_verify_tree(**st, max_nodes=width)
    torch.cuda.synchronize()
    return acc.cpu().numpy(), tok.cpu().numpy(), path.cpu().numpy()


def ref(st, width):
    return to.verify_tree(to.f64(st["target"]), to.f64(st["draft"]), to.ints(st["tokens"]),
                          to.ints(st["parents"]), to.ints(st["cu_nodes"]),
                          to.f64(st["uniforms"]), to.f64(st["draw_uniforms"]), width)


def check(st, width):
    got, want = run(st, width), ref(st, width)
    for g, w, name in zip(got, want, ("accept_len", "tokens", "path")):
        assert np.array_equal(g, w), name
    return want


@pytest.mark.parametrize("law", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,B,sizes,V", [
    ("chain", 5, [5], 1000), ("tree", 9, [1, 2, 13, 21], 4099), ("star", 6, [9, 3], 33),
    ("tree", 3, [40], 1), ("tree", 70, [7, 0, 3], 129), ("tree", 2, [64, 50], 32000),
    ("chain", 1, [6], 50257), ("tree", 700, [4, 5], 600)])
def test_trees(kind, B, sizes, V, dtype, law):
    check(make(B, sizes, V, dtype, kind, seed=B * 7 + V, law=law), max(sizes))


def test_several_residuals_at_one_node():
    """Sixteen children of one root, drafts far from the target: most are
    rejected, so the law goes through many residuals before the draw."""
    st = make(48, [17], 2000, "f32", "star", seed=4, noise=3.0)
    acc, _, path = check(st, 17)
    assert ((acc == 0).sum() > 5) and (path[:, 1] > 3).sum() > 5


def test_largest_tree_and_out_of_room():
    """1,024 nodes; a sequence with more nodes than max_nodes is marked."""
    check(make(2, [1024], 300, "f32", "tree", seed=8), 1024)
    acc, _, _ = check(make(4, [5, 3], 64, "f32", "tree", seed=9), 4)
    assert acc[0] == -1 and acc[1] >= 0


@pytest.mark.parametrize("dtype,law", [("f32", True), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("B,g,V", [(16, 5, 32000), (3, 1, 7), (1, 64, 1021), (260, 4, 2049)])
def test_chains(B, g, V, dtype, law):
    st = make(B, [g + 1], V, dtype, "chain", seed=V + g, law=law)
    args = dict(target=st["target"].view(B, g + 1, V),
                draft=st["draft"].view(B, g + 1, V)[:, :g].contiguous() if law else None,
                tokens=st["tokens"].view(B, g + 1)[:, 1:].contiguous(),
                uniforms=st["uniforms"].view(B, g + 1)[:, 1:].contiguous(),
                draw_uniforms=st["draw_uniforms"])
    acc, tok = sv.spec_verify_probs(**args)
    racc, rtok = to.verify_chain(to.f64(args["target"]), to.f64(args["draft"]),
                                 to.ints(args["tokens"]), to.f64(args["uniforms"]),
                                 to.f64(args["draw_uniforms"]))
    assert np.array_equal(acc.cpu().numpy(), racc) and np.array_equal(tok.cpu().numpy(), rtok)


def test_unnormalised_identical_and_greedy_rows():
    """p = q (every draft accepted), one-hot targets (greedy), rows that sum
    to something else, drafts with q(x) = 0, and uniforms at 0 and just below 1."""
    st = make(12, [6], 500, "f32", "chain", seed=3)
    st["draft"][:12] = st["target"][:12]
    st["target"][12:24] = torch.nn.functional.one_hot(
        torch.randint(500, (12,), device=DEV), 500).float()
    st["target"][24:36] *= 0.25
    st["target"][36:42] *= 3.0
    st["draft"][42:48].scatter_(1, st["tokens"][43:49].long()[:, None], 0.0)
    st["uniforms"][48:54] = 0.0
    st["uniforms"][54:] = 1 - 2.0 ** -24
    st["draw_uniforms"][:6] = 0.0
    st["draw_uniforms"][6:] = 1 - 2.0 ** -24
    acc, _, _ = check(st, 6)
    assert acc[0] == 5 and acc[1] == 5


def test_residual_without_mass_leaves_the_law():
    """q >= p everywhere: the rejected child's residual is empty, and the next
    children and the draw use p itself."""
    st = make(6, [4], 40, "f32", "star", seed=11)
    st["draft"] = st["target"] * 4
    st["uniforms"][:] = 0.9
    acc, tok, _ = check(st, 4)
    assert (acc == 0).all() and (tok[:, 0] >= 0).all()


def test_marks():
    """One bad sequence at a time; its neighbours keep their results."""
    V, n = 700, 5
    good = make(4, [n], V, "f32", "chain", seed=21)
    base = run(good, n)

    def spoil(f):
        st = {k: None if t is None else t.clone() for k, t in good.items()}
        f(st)
        got = run(st, n)
        assert got[0][1] == -1 and (got[1][1] == -1).all() and (got[2][1] == -1).all()
        for b in (0, 2, 3):
            for g, w in zip(got, base):
                assert np.array_equal(g[b], w[b])

    for value in (-1, V, 2**31 - 1):
        spoil(lambda s, value=value: s["tokens"][n + 2:n + 3].fill_(value))
    for value in (-0.5, 1.0, float("nan"), float("inf")):
        spoil(lambda s, value=value: s["uniforms"][n + 4:n + 5].fill_(value))
        spoil(lambda s, value=value: s["draw_uniforms"][1:2].fill_(value))
    for value in (3, 7, -2, -1):
        spoil(lambda s, value=value: s["parents"][n + 3:n + 4].fill_(value))
    spoil(lambda s: s["parents"][n:n + 1].fill_(0))
    x = int(good["tokens"][n + 1])
    for value in (float("nan"), float("inf"), -1.0):
        for k in ("target", "draft"):
            spoil(lambda s, value=value, k=k: s[k][n, x:x + 1].fill_(value))
    # a row that cannot be drawn from: no drafted token there, so only the draw sees it
    st = make(4, [1], V, "f32", "chain", seed=22)
    for row in (torch.zeros(V), torch.full((V,), float("nan")), torch.full((V,), float("inf"))):
        st["target"][1] = row.to(DEV)
        acc, _, _ = check(st, 1)
        assert acc[1] == -1 and (acc[[0, 2, 3]] == 0).all()
    # packed bounds outside the buffers
    st = make(4, [n], V, "f32", "chain", seed=23)
    st["cu_nodes"] = torch.tensor([-5, n, 2 * n, 3 * n, 9 * n], dtype=torch.int32, device=DEV)
    acc, _, _ = run(st, n)
    assert acc[0] == -1 and acc[3] == -1 and acc[1] >= 0 and acc[2] >= 0


def test_unaligned_rows_and_outputs_given():
    """Views whose rows start at odd addresses, and output tensors passed in."""
    st = make(3, [6], 1003, "bf16", "tree", seed=31)
    wide = torch.zeros(18 * 1003 + 3, dtype=torch.bfloat16, device=DEV)
    for off in (1, 3):
        wide[off:off + 18 * 1003] = st["target"].view(-1)
        shifted = dict(st, target=wide[off:off + 18 * 1003].view(18, 1003))
        outs = dict(out_accept_len=torch.empty(3, dtype=torch.int32, device=DEV),
                    out_tokens=torch.empty(3, 6, dtype=torch.int32, device=DEV),
                    out_path=torch.empty(3, 6, dtype=torch.int32, device=DEV))
        sv.spec_verify_tree(**shifted, max_nodes=6, **outs)
        for got, want in zip(outs.values(), ref(st, 6)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_other_stream_and_graph():
    """On a side stream, and captured once and replayed with new inputs."""
    a, b = (make(8, [9, 4], 5000, "f32", "tree", seed=s) for s in (41, 42))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    acc, tok, path = sv.spec_verify_tree(**a, max_nodes=9, stream=s)
    s.synchronize()
    for got, want in zip((acc, tok, path), ref(a, 9)):
        assert np.array_equal(got.cpu().numpy(), want)
    st = {k: t.clone() for k, t in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = sv.spec_verify_tree(**st, max_nodes=9)
    for src in (b, a):
        for k, t in st.items():
            t.copy_(src[k])
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, ref(src, 9)):
            assert np.array_equal(got.cpu().numpy(), want)


def test_no_sequences():
    st = make(1, [3], 10, "f32", "chain", seed=1)
    e = dict(st, cu_nodes=st["cu_nodes"][:1], draw_uniforms=st["draw_uniforms"][:0])
    acc, tok, path = sv.spec_verify_tree(**e, max_nodes=3)
    assert acc.shape == (0,) and tok.shape == (0, 3) and path.shape == (0, 3)


def test_rows_beyond_32_bit_offsets():
    """Probabilities of more than 2^31 elements, the last rows in use."""
    V, n = 151936, 5
    st = make(2, [n], V, "bf16", "chain", seed=51)
    rows = 2**31 // V + 2 * n + 1
    big = {}
    for k in ("target", "draft"):
        big[k] = torch.empty(rows, V, dtype=torch.bfloat16, device=DEV)
        big[k][-2 * n:] = st[k]
    for k in ("tokens", "parents", "uniforms"):
        big[k] = torch.zeros(rows, dtype=st[k].dtype, device=DEV)
        big[k][-2 * n:] = st[k]
    got = run(dict(st, **big, cu_nodes=st["cu_nodes"] + (rows - 2 * n)), n)
    for g, w in zip(got, ref(st, n)):
        assert np.array_equal(g, w)
