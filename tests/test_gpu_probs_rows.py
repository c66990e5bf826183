"""Residual sums over long slices: several rounds of two whole chunks a warp,
their hand-over to single chunks, and a ragged end, at every cluster size."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import test_gpu_probs as tp
import tree_oracle as to

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,B,sizes,V", [
    ("star", 700, [4], 30008),     # one CTA a sequence: 58.6 chunks, three rounds and a tail
    ("star", 150, [9], 40024),     # four CTAs, 20 chunks each
    ("star", 5, [17], 151936),     # eight CTAs, 38 chunks each
    ("tree", 3, [12], 100008)])
def test_rejections_over_long_rows(kind, B, sizes, V, dtype):
    """Drafts far from the target, so that most sequences reject and draw from
    a residual; equal to the 64-bit form."""
    st = tp.make(B, sizes, V, dtype, kind, seed=V % 1000 + B, noise=2.5)
    acc, _, path = tp.check(st, max(sizes))
    # a sequence that stopped at a node with children summed a residual for each
    par, cu = st["parents"].tolist(), st["cu_nodes"].tolist()
    stopped = sum(any(p == path[b, acc[b]] for p in par[cu[b]:cu[b + 1]]) for b in range(B))
    assert stopped >= B // 3


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,g,V", [(230, 2, 30008),    # one CTA a sequence
                                   (120, 1, 81928)])   # two, 81 chunks each, a ragged end
def test_rejected_chains_over_long_rows(B, g, V, dtype):
    st = tp.make(B, [g + 1], V, dtype, "chain", seed=V % 1000 + B, noise=2.5)
    args = (st["target"].view(B, g + 1, V), st["draft"].view(B, g + 1, V)[:, :g].contiguous(),
            st["tokens"].view(B, g + 1)[:, 1:].contiguous(),
            st["uniforms"].view(B, g + 1)[:, 1:].contiguous(), st["draw_uniforms"])
    acc, tok = sv.spec_verify_probs(*args)
    racc, rtok = to.verify_chain(to.f64(args[0]), to.f64(args[1]), to.ints(args[2]),
                                 to.f64(args[3]), to.f64(args[4]))
    assert np.array_equal(acc.cpu().numpy(), racc) and np.array_equal(tok.cpu().numpy(), rtok)
    assert (racc < g).sum() >= B // 3


def test_residual_sums_of_unaligned_rows_agree():
    """The same laws at rows that start on a 16-byte border and off it: the
    same tokens by both ways of reading them."""
    V = 40000
    st = tp.make(20, [6], V, "f32", "star", seed=77, noise=2.5)
    want = tp.run(st, 6)
    for k in ("target", "draft"):
        wide = torch.zeros(120 * V + 1, device="cuda:0")
        wide[1:] = st[k].view(-1)
        st[k] = wide[1:].view(120, V)
    for g, w in zip(tp.run(st, 6), want):
        assert np.array_equal(g, w)
