"""tree_attention where one CTA goes through many parts: their descriptions
pass through a ring of eight places, which every warp has to have read before
its place is written again."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import test_gpu_attention as ta

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
def test_many_parts_of_one_cta(D, dtype):
    """3,600 units of one or two tiles with lengths and node counts that
    differ from one to the next (a mixed-up description would be another
    unit's): right once, and the same bits thirty times."""
    rng = np.random.default_rng(61)
    lens = [int(x) for x in rng.integers(0, 140, 450)]
    nodes = [int(x) for x in rng.integers(1, 6, 450)]
    st = ta.make(lens, nodes, 16, 8, D, 16, dtype, seed=61)
    out, lse = ta.check(st)
    for _ in range(30):
        o, z = sv.tree_attention(**st, with_lse=True)
        assert torch.equal(o, out) and torch.equal(z, lse)
