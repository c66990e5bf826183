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
