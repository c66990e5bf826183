"""tree_attention where the weights of one row span many orders of magnitude.

Tolerance, from the number formats.  Weights and output are rounded to the
input type, h = eps / 2 relative each: h (A + |o|), A = sum p |v| / sum p.  In
fp16 a weight is also rounded to a multiple of 2^-24, by 2^-25 at most, where
the row's largest is at least 2^7 (it is carried that much higher): an
absolute 2^-32 of the largest weight, 2^-32 sum |v| max p / sum p in the
output.  A score is off by D 2^-24 sum |q k| scale at most; one of the tail
and one of the dominant key together move their ratio by twice that, and the
exponentials by 2^-22 each, all relative to A.  The output itself may be an
fp16 subnormal: 2^-25."""
import pytest
import torch

import speculative_decoding_verification_85_b200 as sv
import test_gpu_attention as ta
import tree_oracle as to

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes,Hq,Hkv", [(3, 8, 4), (80, 12, 4)])
@pytest.mark.parametrize("gap", [6, 12, 15, 16, 17, 18])
def test_dominant_key_without_value(gap, nodes, Hq, Hkv, dtype):
    """The first cached token stands `gap` nats above all others and its value
    is zero, so the output is what the small weights carry.  160 or 320 units
    of 17 tiles: most lie within one CTA, as one part with that key."""
    D, B = 64, 40
    st = ta.make([2000 + 3 * b for b in range(B)], [nodes] * B, Hq, Hkv, D, 16, dtype, seed=gap)
    st["q"] *= 0.1
    st["q"][..., 0] = 8.0
    for k in ("k", "k_cache"):
        st[k] *= 0.5
        st[k][..., 0] = 0.0
    for v in ("v", "v_cache"):
        st[v] = (1.0 + 0.1 * st[v].float()).to(st[v].dtype)
    first = st["block_table"][:, 0].long()
    st["k_cache"][first, 0] = 0.0
    st["k_cache"][first, 0, :, 0] = float(gap)  # 8 gap / sqrt(64)
    st["v_cache"][first, 0] = 0.0
    out, lse = sv.tree_attention(**st, with_lse=True)
    o, z, mag = ta.ref(st)
    fmt = torch.finfo(out.dtype)
    # sum |q k| scale: gap for the dominant key; for the others below 64 x 0.1 x 0.5 x 4 x 4 / 8
    score = 2 * D * 2.0 ** -24 * max(gap, 6.4) + 2 * 2.0 ** -22
    lim = fmt.eps / 2 * (mag + o.abs()) + score * mag
    if dtype == "f16":
        # max p / sum p <= 1; sum |v| <= 2,200 tokens of at most 1.6
        lim += 2.0 ** -32 * 2200 * 1.6 + 2.0 ** -25
    err = (out.double() - o).abs()
    assert (err <= lim).all(), f"worst {(err / lim).max().item():.2f} of the limit"
    assert ((lse.double() - z).abs() <= score + 2.0 ** -20 * gap).all()


def test_weights_far_above_the_held_shift():
    """fp16 scores that grow by 5 nats a tile, just less than what makes the
    accumulator rescale, and by more: weights stay finite."""
    for step in (5.0, 5.6, 9.0):
        st = ta.make([1500, 1290], [4, 100], 8, 2, 64, 128, "f16", seed=71)
        st["q"] *= 0.1
        st["q"][..., 0] = 8.0
        for k in ("k", "k_cache"):
            st[k] *= 0.5
            st[k][..., 0] = 0.0
        for b in range(2):
            for j, page in enumerate(st["block_table"][b].tolist()):
                if page >= 0:
                    st["k_cache"][page, :, :, 0] = step * j
        out, lse = sv.tree_attention(**st, with_lse=True)
        o, z, mag = ta.ref(st)
        top = step * 12
        score = 2 * 64 * 2.0 ** -24 * (top + 6.4) + 2 * 2.0 ** -22
        lim = (2.0 ** -11 + score) * mag + 2.0 ** -11 * o.abs() + 2.0 ** -32 * 1600 * 5 + 2.0 ** -25
        err = (out.double() - o).abs()
        assert out.isfinite().all()
        assert (err <= lim).all(), f"worst {(err / lim).max().item():.2f} of the limit"
        assert ((lse.double() - z).abs() <= score + 2.0 ** -20 * top).all()
