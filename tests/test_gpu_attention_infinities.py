"""tree_attention with infinite inputs that some nodes see and others do not."""
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import test_gpu_attention as ta

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,nodes,Hq,Hkv", [
    ([0], [300], 1, 1),            # one part a tile
    ([40], [300], 4, 2),           # two query tiles
    ([900], [1000], 2, 1),
    ([40] * 90, [300] * 90, 2, 2)  # several units a CTA
])
def test_infinite_values_in_tiles_of_different_parts(lens, nodes, Hq, Hkv, dtype):
    """Infinite values on unrelated branches, in tree tiles that may belong to
    different parts of a unit: each reaches those who see it and nobody
    else, wherever the line of tiles is cut."""
    st = ta.make(lens, nodes, Hq, Hkv, 64, 16, dtype, "roots", seed=81)
    n = nodes[0]
    for b in (0, len(lens) - 1):
        st["v"][b * n + 5, 0, 3] = float("inf")
        st["v"][b * n + 200, 0, 3] = float("-inf")
        st["v"][b * n + n - 1, 0, 60] = float("nan")
        st["parents"][b * n + 201:(b + 1) * n:50] = 200  # some see one beside themselves
        st["parents"][b * n + 6:(b + 1) * n:49] = 5
    out, lse = sv.tree_attention(**st, with_lse=True)
    want = ta.ref(st)
    assert want[0][5, 0, 3] == float("inf") and want[0][200, 0, 3] == float("-inf")
    ta.close(out, lse, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lens,nodes", [([0], [2]), ([20], [3]), ([5000], [3]), ([300] * 90, [5] * 90),
                                        ([700] * 5, [200] * 5)])
def test_rows_whose_scores_are_all_minus_infinity(lens, nodes, dtype):
    """exp(-inf) is 0 for every key: the sum is 0, its logarithm -inf, and the
    output 0 / 0, NaN; the other rows are those without it."""
    st = ta.make(lens, nodes, 8, 4, 64, 16, dtype, "chain", seed=91)
    for k in ("k", "k_cache"):
        st[k][..., 0] = -1.0
    base, blse = ta.check(st)
    bad = dict(st, q=st["q"].clone())
    hit = torch.zeros(base.shape[:2], dtype=torch.bool, device=DEV)
    hit[1, 2] = hit[-1, 5] = True
    bad["q"][..., 0][hit] = float("inf")
    out, lse = sv.tree_attention(**bad, with_lse=True)
    assert out[hit].isnan().all() and (lse[hit] == float("-inf")).all()
    assert torch.equal(out[~hit], base[~hit]) and torch.equal(lse[~hit], blse[~hit])


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("lens,nodes", [([0], [2]), ([5000], [3]), ([700] * 5, [200] * 5)])
def test_rows_with_an_infinite_or_undefined_score(lens, nodes, value):
    """A score of +inf or NaN makes its row NaN, the others stay."""
    st = ta.make(lens, nodes, 8, 4, 64, 16, "f16", "chain", seed=92)
    for k in ("k", "k_cache"):
        st[k][..., 0] = -1.0
    st["k"][0, 0, 0] = 1.0  # +inf for an infinite query of the first key head
    base, blse = ta.check(st)
    bad = dict(st, q=st["q"].clone())
    bad["q"][1, 1, 0] = value
    out, lse = sv.tree_attention(**bad, with_lse=True)
    hit = torch.zeros(base.shape[:2], dtype=torch.bool, device=DEV)
    hit[1, 1] = True
    assert out[hit].isnan().all() and lse[hit].isnan().all()
    assert torch.equal(out[~hit], base[~hit]) and torch.equal(lse[~hit], blse[~hit])
