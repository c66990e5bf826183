"""PagedCache: chains, streams, and calls it refuses."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, D, LAYERS = 2, 64, 2


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rnd(*s):
    return torch.randn(*s, device=DEV).bfloat16()


def state(c):
    return [t.clone() for t in (c.lens, c.block_table, c.free_pages, c.free_count, c.k, c.v)]


def test_refused_rows_leave_the_cache_as_it_was():
    """Keys or values of another type, shape, layer count or layout than the
    cache's are refused before lengths, tables and free pages change."""
    c = sv.PagedCache(LAYERS, 20, 16, H, D, 2, 128)
    cu, add = i32([0, 20, 30]), i32([20, 10])
    k = rnd(LAYERS, 30, H, D)
    c.extend(k, k, cu, add)
    before = state(c)
    bad = [(k.half(), k.half()), (k, k.half()), (k[:1], k[:1]), (k[0], k[0]), (k[..., :32], k[..., :32]),
           (k, k[:, :, :1]), (k, k[:, :29]), (k.cpu(), k.cpu()), (k, k.cpu()),
           (k.transpose(2, 3).contiguous().transpose(2, 3), k)]
    for a, b in bad:
        with pytest.raises((ValueError, TypeError)):
            c.extend(a, b, cu, add)
        with pytest.raises((ValueError, TypeError)):
            c.commit(a, b, cu, i32([1, 1]))
    with pytest.raises(ValueError):
        c.extend(k, k, cu[:2], add)
    with pytest.raises(ValueError):
        c.extend(k, k, cu, add[:1])
    assert all(torch.equal(x, y) for x, y in zip(before, state(c)))
    start = c.extend(k, k, cu, add)
    assert start.tolist() == [20, 10] and c.lens.tolist() == [40, 20]
