"""kv_slots and kv_append against their plain forms: equal, whole."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import tree_oracle as to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def make(B, page, max_len, max_add, seed, path_width=None, spare=3, release=0.0, width=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max_len + 1, B)
    add = rng.integers(0, max_add + 1, B)
    nn = np.full(B, path_width) if path_width else add + rng.integers(0, 3, B)
    path = None
    if path_width:
        add = np.minimum(add, path_width)
        path = np.full((B, path_width), -1)
        for b in range(B):
            path[b, :add[b]] = np.sort(rng.choice(path_width, add[b], replace=False))
    add = np.where(rng.random(B) < release, -1, add)
    have = -(-lens // page)
    W = width or max(1, -(-(max_len + max_add) // page))
    order = rng.permutation(int(have.sum()) + 4000)
    table, at = np.full((B, W), -1), 0
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    free = order[at:]
    need = int((-(-(lens + np.maximum(add, 0)) // page) - have).sum())
    count = max(0, min(len(free), need + spare))
    pool = np.concatenate([free[:count], np.full(50, -7)])
    return dict(lens=lens, add=add, cu=np.concatenate([[0], np.cumsum(nn)]), table=table,
                pool=pool, count=count, rows=int(nn.sum()) + 2, page=page, path=path)


def run(st, **kw):
    table, pool = i32(st["table"]), i32(st["pool"])
    slots, start, lens, count = sv.kv_slots(
        i32(st["lens"]), i32(st["add"]), i32(st["cu"]), table, pool, i32([st["count"]]),
        rows=st["rows"], page_size=st["page"],
        path=None if st["path"] is None else i32(st["path"]), **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in (slots, start, lens)] + [count.item(), table.cpu().numpy(),
                                                             pool.cpu().numpy()]


def check(st):
    want = to.kv_slots(st["lens"], st["add"], st["cu"], st["table"], st["pool"], st["count"],
                       st["rows"], st["page"], st["path"])
    got = run(st)
    for g, w, name in zip(got, want, ("slots", "start", "lens", "count", "table", "pool")):
        assert np.array_equal(g, w), name
    return want


@pytest.mark.parametrize("B,page,max_len,max_add,path_width", [
    (1, 16, 0, 1, None), (7, 16, 100, 40, None), (64, 16, 500, 6, 26), (3, 1, 5, 9, None),
    (1030, 8, 60, 5, 9), (2500, 32, 90, 12, None), (40, 128, 3000, 700, None),
    (33, 24, 1000, 300, 400), (300, 16, 3, 64, 64)])
@pytest.mark.parametrize("spare,release", [(3, 0.0), (-9, 0.0), (3, 0.3), (-9, 0.3)])
def test_slots(B, page, max_len, max_add, path_width, spare, release):
    check(make(B, page, max_len, max_add, seed=B + page, path_width=path_width, spare=spare,
               release=release))


def test_short_tables_and_bad_requests():
    """Table rows too short, lengths and rows that do not exist, paths out of
    order: those requests are refused and the others served."""
    st = make(60, 16, 200, 50, seed=5, width=14)
    start = check(st)[1]
    assert 0 < (start < 0).sum() < 60
    st = make(12, 16, 200, 8, seed=6, path_width=10)
    st["lens"][1], st["lens"][2] = -3, 10**6
    st["add"][3], st["add"][4] = -2, 11
    st["add"][5:8] = 2
    st["path"][5, :2], st["path"][6, :2], st["path"][7, :2] = [4, 4], [3, 10], [-1, 2]
    start = check(st)[1]
    assert (start[1:8] == -1).all()
    st["cu"][-1] += 100
    st["cu"][0] = -4
    assert check(st)[1][0] == -1 and check(st)[1][-1] == -1


def test_lengths_and_count_in_place_and_idle_requests():
    st = make(20, 16, 300, 0, seed=9)
    want = check(st)
    lens, count, table, pool = (i32(st["lens"]), i32([st["count"]]), i32(st["table"]),
                                i32(st["pool"]))
    st["add"][:] = 20
    st["cu"] = np.arange(21) * 20
    st["rows"] = 400
    st["table"] = np.concatenate([st["table"], np.full((20, 3), -1)], 1)
    st["pool"] = np.arange(9000, 9100)
    st["count"] = 100
    want = to.kv_slots(st["lens"], st["add"], st["cu"], st["table"], st["pool"], 100, 400, 16)
    table, pool, count = i32(st["table"]), i32(st["pool"]), i32([100])
    slots, start, l2, c2 = sv.kv_slots(lens, i32(st["add"]), i32(st["cu"]), table, pool, count,
                                       rows=400, page_size=16, out_lens=lens,
                                       out_free_count=count)
    assert l2 is lens and c2 is count
    for g, w in zip((slots, start, lens, table), (want[0], want[1], want[2], want[4])):
        assert np.array_equal(g.cpu().numpy(), w)
    assert count.item() == want[3]


def test_strided_table_and_no_requests():
    st = make(9, 16, 100, 30, seed=12)
    big = i32(np.full((9, st["table"].shape[1] + 5), -1))
    view = big[:, :st["table"].shape[1]]
    view.copy_(i32(st["table"]))
    want = to.kv_slots(st["lens"], st["add"], st["cu"], st["table"], st["pool"], st["count"],
                       st["rows"], st["page"])
    slots, *_ = sv.kv_slots(i32(st["lens"]), i32(st["add"]), i32(st["cu"]), view, i32(st["pool"]),
                            i32([st["count"]]), rows=st["rows"], page_size=16)
    assert np.array_equal(slots.cpu().numpy(), want[0])
    assert np.array_equal(view.cpu().numpy(), want[4]) and (big[:, -5:] == -1).all()
    slots, start, lens, count = sv.kv_slots(i32([]), i32([]), i32([0]), i32(np.zeros((0, 4))),
                                            i32([1, 2]), i32([2]), rows=3, page_size=16)
    assert slots.cpu().tolist() == [-1, -1, -1] and count.item() == 2


def test_many_rows():
    """Enough rows for the launch that maps them over the whole GPU."""
    check(make(50, 16, 2000, 900, seed=13))
    check(make(500, 16, 100, 30, seed=14, path_width=40, release=0.1))


# ----------------------------------------------------------------------- append
def _caches(layers, pages, page, H, D, dt):
    shape = ((layers,) if layers else ()) + (pages, page, H, D)
    x = torch.randint(-100, 100, (2,) + shape, device=DEV)
    return x[0].to(dt), x[1].to(dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32, torch.uint8])
@pytest.mark.parametrize("layers,N,H,D,pages,page", [
    (None, 1, 1, 1, 1, 1), (None, 37, 8, 128, 9, 16), (3, 50, 2, 80, 20, 8), (2, 9, 3, 7, 5, 4),
    (5, 1000, 1, 64, 100, 16)])
def test_append(layers, N, H, D, pages, page, dt):
    rng = np.random.default_rng(N)
    slots = rng.permutation(max(pages * page, N))[:N]
    slots = np.where((rng.random(N) < 0.3) | (slots >= pages * page), -1, slots)
    if N > 5:
        slots[:3] = [-5, pages * page, 2**31 - 1]
    kc, vc = _caches(layers, pages, page, H, D, dt)
    wk, wv = kc.clone(), vc.clone()
    lead = (layers,) if layers else ()
    k, v = (torch.randint(-100, 100, lead + (N, H, D), device=DEV).to(dt) for _ in range(2))
    for i, s in enumerate(slots):
        if 0 <= s < pages * page:
            for w, x in ((wk, k), (wv, v)):
                w[..., s // page, s % page, :, :] = x[..., i, :, :]
    sv.kv_append(k, v, i32(slots), kc, vc)
    assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_append_strided():
    """Keys and values out of one fused projection, the cache with its heads
    before its tokens, both caches in one tensor; odd offsets too."""
    N, H, D, pages, page = 30, 4, 64, 6, 16
    for off in (0, 1):
        qkv = torch.randn(N, 3 * H * D + 1, device=DEV).bfloat16()[:, off:off + 3 * H * D]
        k = qkv[:, H * D:2 * H * D].unflatten(1, (H, D))
        v = qkv[:, 2 * H * D:].unflatten(1, (H, D))
        both = torch.randn(pages, 2, H, page, D, device=DEV).bfloat16()
        kc, vc = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        want = both.clone()
        slots = torch.randperm(pages * page)[:N]
        for i, s in enumerate(slots.tolist()):
            want[s // page, 0, :, s % page] = k[i]
            want[s // page, 1, :, s % page] = v[i]
        sv.kv_append(k, v, slots.to(DEV, torch.int32), kc, vc)
        assert torch.equal(both, want)


def test_append_beyond_32_bit_offsets():
    """Layers of more than 2^31 elements in all; the last layer's last slots."""
    H, D, page = 2, 128, 16
    pages = 2**30 // (page * H * D) + 3
    kc, vc = (torch.zeros(2, pages, page, H, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    k, v = (torch.randint(1, 255, (2, 3, H, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    slots = [pages * page - 1, 5, pages * page - 17]
    sv.kv_append(k, v, i32(slots), kc, vc)
    for i, s in enumerate(slots):
        assert torch.equal(kc[:, s // page, s % page], k[:, i])
        assert torch.equal(vc[:, s // page, s % page], v[:, i])
    assert int((kc != 0).any(-1).sum()) == 2 * 3 * H
