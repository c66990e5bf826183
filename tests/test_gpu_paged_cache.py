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


def rows_of(c, b, n, which):
    pages = c.block_table[b, :-(-n // c.page_size)].long()
    return getattr(c, which)[:, pages].flatten(1, 2)[:, :n]


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


def test_chains_commit_without_a_path():
    """Accepted prefixes of chains, as spec_verify_probs returns them: the
    root and the first accept_len drafts join, a marked sequence stays."""
    g = torch.Generator(device=DEV).manual_seed(7)
    B, gamma, V = 6, 4, 500
    n = gamma + 1
    c = sv.PagedCache(LAYERS, 80, 8, H, D, B, 200)
    held = [3, 8, 0, 17, 5, 40]
    cu0 = i32(np.concatenate([[0], np.cumsum(held)]))
    k0, v0 = rnd(LAYERS, sum(held), H, D), rnd(LAYERS, sum(held), H, D)
    c.extend(k0, v0, cu0, i32(held))
    texts = [[(k0[:, a:b], v0[:, a:b])] for a, b in zip(cu0.tolist(), cu0.tolist()[1:])]
    cu = i32(np.arange(B + 1) * n)
    seen = set()
    for step in range(4):
        p = torch.softmax(torch.randn(B, n, V, generator=g, device=DEV), -1)
        q = torch.softmax(torch.log(p[:, :gamma]) + 0.5 * torch.randn(B, gamma, V, generator=g, device=DEV), -1)
        x = torch.multinomial(q.flatten(0, 1), 1, generator=g).view(B, gamma).int()
        u = torch.rand(B, gamma, generator=g, device=DEV)
        if step == 2:
            x[1, 0] = V  # marks sequence 1
        acc, tok = sv.spec_verify_probs(p, q, x, u, torch.rand(B, generator=g, device=DEV))
        k, v = rnd(LAYERS, B * n, H, D), rnd(LAYERS, B * n, H, D)
        start = c.commit(k, v, cu, acc)
        for b, a in enumerate(acc.tolist()):
            assert start[b].item() == held[b]
            seen.add(a)
            texts[b].append((k[:, b * n:b * n + a + 1], v[:, b * n:b * n + a + 1]))
            held[b] += a + 1
        assert c.lens.tolist() == held
    assert -1 in seen and len(seen) > 3
    for b in range(B):
        for i, which in enumerate("kv"):
            assert torch.equal(rows_of(c, b, held[b], which), torch.cat([t[i] for t in texts[b]], 1))


def test_calls_on_a_stream():
    """extend, attend, commit (with a path and without) and release on a side
    stream: what the same calls do on the current one."""
    B, n = 4, 5
    cu0, add = i32([0, 30, 31, 80, 100]), i32([30, 1, 49, 20])
    k0, v0 = rnd(LAYERS, 100, H, D), rnd(LAYERS, 100, H, D)
    cu, par = i32(np.arange(B + 1) * n), i32([-1, 0, 0, 1, 1] * B)
    q, k, v = rnd(B * n, 8, D), rnd(LAYERS, B * n, H, D), rnd(LAYERS, B * n, H, D)
    acc = i32([2, 0, -1, 1])
    path = i32([[0, 1, 3, -1, -1], [0, -1, -1, -1, -1], [-1] * 5, [0, 2, -1, -1, -1]])
    which, add2 = torch.tensor([False, True, False, True], device=DEV), i32([0, 1, 2, 3])

    def steps(c, **kw):
        got = [c.extend(k0, v0, cu0, add, **kw)]
        got.append(c.attend(1, q, k[1], v[1], par, cu, **kw)[0])
        got.append(c.commit(k, v, cu, acc, path, **kw))
        got.append(c.commit(k, v, cu, acc, **kw))
        c.release(which, **kw)
        got.append(c.extend(k0, v0, cu0, add2, **kw))
        return got

    a, b = (sv.PagedCache(LAYERS, 30, 16, H, D, B, 160) for _ in range(2))
    want = steps(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(2_000_000)  # the current stream is behind
    got = steps(b, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert all(torch.equal(x, y) for x, y in zip(state(a), state(b)))
    assert a.lens.tolist() == [30 + 3 + 3, 1, 49 + 2, 3]
