"""CPU pins of the plain forms the drafted-tree operators are tested against,
and of the closed form of repeated residuals the kernel computes with."""
import itertools

import numpy as np
import pytest

import tree_oracle as to


def _law(rng, V):
    p = rng.random(V) ** 3
    return p / p.sum()


@pytest.mark.parametrize("V,K,point", [(2, 1, False), (3, 2, False), (4, 3, False), (3, 2, True)])
def test_first_token_follows_the_target(V, K, point):
    """Enumerating the K children (drawn from q) and integrating over their
    uniforms, the token after the root follows p exactly."""
    rng = np.random.default_rng(V * 10 + K)
    p, q = _law(rng, V), _law(rng, V)
    got = np.zeros(V)
    for xs in itertools.product(range(V), repeat=K):
        weight = 1.0 if point else np.prod([q[x] for x in xs])
        if point and xs != tuple(range(K)):  # point drafts: one given choice
            continue
        alive, r = weight, p.copy()
        for x in xs:
            a = min(1.0, r[x] / (1.0 if point else q[x]))
            got[x] += alive * a
            alive *= 1 - a
            r = np.maximum(r - (np.eye(V)[x] if point else q), 0)
            if r.sum() > 0:
                r /= r.sum()
        got += alive * r
    assert np.abs(got - p).max() < 1e-12


@pytest.mark.parametrize("seed", range(5))
def test_closed_form_of_repeated_residuals(seed):
    """max(p - c_k q, 0) / M_k with c_{k+1} = c_k + M_k equals the residual
    taken and normalised k times."""
    rng = np.random.default_rng(seed)
    p, q = _law(rng, 50), _law(rng, 50)
    r, c, M = p.copy(), 0.0, 1.0
    for _ in range(4):
        r = np.maximum(r - q, 0)
        r /= r.sum()
        c, M = c + M, np.maximum(p - (c + M) * q, 0).sum()
        assert np.abs(np.maximum(p - c * q, 0) / M - r).max() < 1e-12


def test_draw_law_by_midpoints():
    """verify_one's draw: a grid of uniforms gives the law itself."""
    p = np.array([[0.1, 0.0, 0.4, 0.5]])
    n = 1000
    got = np.bincount([to.verify_one(p, None, [0], [-1], [0.0], (i + 0.5) / n)[1]
                       for i in range(n)], minlength=4) / n
    assert np.allclose(got, p[0])


def test_slots_of_a_hand_case():
    """Two requests, pages of 4: 3 + 2 tokens take one page for the second
    part, 4 + 1 a new one; a third finds none left."""
    table = np.array([[7, -1], [5, -1], [6, -1]])
    slots, start, lens, count, table, _ = to.kv_slots(
        np.array([3, 4, 4]), np.array([2, 1, 1]), np.array([0, 2, 3, 4]), table,
        np.array([1, 2]), 2, 4, 4)
    assert slots.tolist() == [31, 8, 4, -1] and start.tolist() == [3, 4, -1]
    assert lens.tolist() == [5, 5, 4] and count == 0
    assert table.tolist() == [[7, 2], [5, 1], [6, -1]]


def test_attention_of_a_hand_case():
    """Zero queries weigh everything visible alike: the mean of the context
    and the ancestors, and ln of their number."""
    k = np.zeros((3, 1, 2))
    v = np.arange(6.0).reshape(3, 1, 2)
    cache = np.full((2, 2, 1, 2), 9.0)
    out, lse = to.attention(np.zeros((3, 1, 2)), k, v, cache, cache, np.array([[1, 0]]),
                            np.array([3]), np.array([-1, 0, 0]), np.array([0, 3]), 1.0)
    assert np.allclose(out[2, 0], (3 * 9.0 + v[0, 0] + v[2, 0]) / 5)
    assert np.allclose(lse[:, 0], np.log([4, 5, 5]))


def test_vectorised_attention_equals_the_plain_one():
    import torch
    g = torch.Generator().manual_seed(3)

    def rnd(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    q, k, v = rnd(7, 4, 8), rnd(7, 2, 8), rnd(7, 2, 8)
    kc, vc = rnd(5, 4, 2, 8), rnd(5, 4, 2, 8)
    table = torch.tensor([[3, 1, 0], [4, 2, 0]])
    lens, par, cu = torch.tensor([9, 3]), torch.tensor([-1, 0, 0, 1, -1, 0, 1]), torch.tensor([0, 4, 7])
    out, lse, _ = to.attention_t(q, k, v, kc, vc, table, lens, par, cu, 0.3)
    o2, l2 = to.attention(*(t.numpy() for t in (q, k, v, kc, vc, table, lens, par, cu)), 0.3)
    assert np.abs(out.numpy() - o2).max() < 1e-12 and np.abs(lse.numpy() - l2).max() < 1e-12
