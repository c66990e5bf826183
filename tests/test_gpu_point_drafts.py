"""Point drafts whose rejections leave a law without mass: laws that do not
sum to 1 exactly (16-bit probabilities, truncated ones) come to this with
valid inputs."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NEAR1 = 1 - 2.0 ** -24


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,V", [(3, 40), (300, 5000), (2, 60001)])
def test_chain_equals_one_hot_draft_rows(B, V, dtype):
    """A drafted token of probability 1: the same tokens as with the one-hot
    draft rows written out, rows with all of their mass on the draft among
    them."""
    g = torch.Generator(device=DEV).manual_seed(V)
    gamma = 3
    target = torch.softmax(3 * torch.randn(B, gamma + 1, V, generator=g, device=DEV), -1).to(dtype)
    tokens = torch.randint(V, (B, gamma), generator=g, device=DEV, dtype=torch.int32)
    tokens[::2] = target[::2, :gamma].argmax(-1).int()
    at = torch.arange(B, device=DEV)
    for i, mass in ((1, 0.5), (0, 0.99609375)):  # the whole law: one entry below 1
        sel = at[i::3]
        target[sel, i] = 0
        target[sel, i, tokens[sel, i].long()] = mass
    u = torch.rand(B, gamma, generator=g, device=DEV)
    u[::3, 0] = NEAR1
    u[1::3, 0], u[1::3, 1] = 0.0, 0.5
    ud = torch.rand(B, generator=g, device=DEV)
    rows = torch.nn.functional.one_hot(tokens.long(), V).to(dtype)
    want = sv.spec_verify_probs(target, rows, tokens, u, ud)
    got = sv.spec_verify_probs(target, None, tokens, u, ud)
    assert (want[0] >= 0).all()
    assert (want[0][::3] == 0).all() and torch.equal(want[1][::3, 0], tokens[::3, 0])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("V", [50, 70001])
def test_tree_draws_the_entry_lost_last(V):
    """Children that cover the law's support, each turned down: the draw is of
    the entry that the law lost last (children of no weight behind it, and
    one more of a token already turned down, lose nothing)."""
    law = {7: 0.3, 11: 0.4, V - 1: 0.2}
    trees = [[7, 11, V - 1], [V - 1, 7, 11, 5], [11, V - 1, 7, 11, 9], [5, 9], [7, 11]]
    last = [V - 1, 11, 7, None, None]
    n = 6
    target = torch.zeros(len(trees) * n, V, device=DEV)
    tokens, parents, cu = [], [], [0]
    for b, kids in enumerate(trees):
        for x, p in law.items():
            target[cu[-1], x] = p
        tokens += [0] + kids
        parents += [-1] + [0] * len(kids)
        cu.append(cu[-1] + len(kids) + 1)
    N = cu[-1]
    u = torch.full((N,), NEAR1, device=DEV)
    ud = torch.full((len(trees),), 0.5, device=DEV)
    acc, tok, path = sv.spec_verify_tree(target[:N], None, i32(tokens), i32(parents), i32(cu), u, ud,
                                         max_nodes=n)
    assert acc.tolist() == [0] * len(trees)
    assert [t for t, x in zip(tok[:, 0].tolist(), last) if x is not None] == [x for x in last if x]
    # mass that is left is drawn from: 7 and 11 lost nothing of it to 5 and 9; V - 1 stays
    assert tok[3, 0].item() == 11 and tok[4, 0].item() == V - 1
    assert (tok[:, 1:] == -1).all() and (path[:, 0] == 0).all() and (path[:, 1:] == -1).all()


def test_law_without_any_mass_is_marked():
    V = 100
    target = torch.zeros(2, 3, V, device=DEV)
    target[1] = 1 / V
    acc, tok = sv.spec_verify_probs(target, None, i32([[3, 4], [3, 4]]),
                                    torch.full((2, 2), 0.5, device=DEV),
                                    torch.full((2,), 0.5, device=DEV))
    assert acc[0] == -1 and (tok[0] == -1).all() and acc[1] >= 0
