"""Mixture-of-experts layers whose exponents lie far from the activations': the
products of small activations with large weights, of large ones with small
weights, and both kinds of blocks in one column, all with results in range.

Tolerances and the FP64 reference are those of the layer's own tests: powers of
two change no relative error as long as nothing leaves the FP32 range.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from oracle import mxfp4_ops_oracle as Q  # noqa: E402
from test_gpu_mx_moe import Case, check  # noqa: E402

pytestmark = pytest.mark.gpu


def make(xscale, lo, hi, T=6, E=5, k=2, H=1120, I=96, seed=21):
    """Gate and up exponent bytes in lo..hi, the down product's as usual. H: two whole stages and a short one."""
    case = Case(T, E, k, H, I, seed=seed, xscale=xscale)
    rng = np.random.default_rng([seed, lo, hi])
    case.e13 = rng.integers(lo, hi + 1, size=case.e13.shape).astype(np.uint8)
    return case


@pytest.mark.parametrize("xscale,lo,hi", [
    (2.0 ** -100, 236, 239),    # gate and up about 2^16: their sums without the factor 2^-114 pass 2^128
    (2.0 ** -100, 219, 222),    # about 1/2
    (2.0 ** -64, 186, 196),     # bytes on both sides of 191
    (2.0 ** 24, 58, 70),        # ... and of 64
    (2.0 ** 90, 30, 37),
    (2.0 ** 110, 0, 17),        # byte 0 among them
])
def test_exponents_against_activations(xscale, lo, hi):
    check(make(xscale, lo, hi), (xscale, lo, hi))


@pytest.mark.parametrize("where", [0, 1, 15, 17, 34])
def test_one_unusual_block(where):
    """Every block of a column usual but one, wherever the stages put it: the sums before and after it still count."""
    case = make(2.0 ** -100, 180, 184, seed=22)
    case.e13[:, where] = np.where(case.e13[:, where] % 2, 236, 182).astype(np.uint8)
    check(case, where)


@pytest.mark.parametrize("I", [288, 512])
def test_h_near_the_top_of_the_range(I):
    """h about 2^122: 32 of its products with codes add up past 2^128 before the down weights' 2^-57 brings them
    back."""
    case = make(1.0, 182, 183, H=288, I=I, seed=25)
    case.e2 = np.random.default_rng(25).integers(70, 74, size=case.e2.shape).astype(np.uint8)
    check(case, I)


def test_crowded_experts_and_long_items():
    """Groups of every size up to 8 tokens, several items per thread block, an unusual byte in some experts only."""
    case = make(2.0 ** -100, 184, 190, T=64, E=6, k=2, H=2080, I=544, seed=23)
    case.e13[1, 40] = 237
    case.e13[4, 3, ::7] = 238
    check(case)


def test_a_token_does_not_see_its_neighbours_there():
    case = make(2.0 ** -100, 188, 194, T=20, E=4, k=2, seed=24)
    dev = case.device()
    full = w4.mxfp4_moe(*dev, 2)
    for t in (0, 9, 19):
        assert torch.equal(w4.mxfp4_moe(dev[0][t:t + 1].contiguous(), *dev[1:], 2)[0], full[t])
    big = dev[0].clone()
    big[3] *= 2.0 ** 150
    again = w4.mxfp4_moe(big, *dev[1:], 2)
    keep = [t for t in range(20) if t != 3]
    assert torch.equal(again[keep], full[keep])
    assert w4.device_status() == w4.OK


@pytest.mark.parametrize("gate", [-40.0, -86.0, -88.0, -90.0, 88.0, 0.0])
def test_silu_far_from_zero(gate):
    """Every gate the same exact number, the up product large enough that silu of it matters.

    Gate and up are single exact products, so h is off by the exponential (2 units of 2^-23), the addition, the
    division (2) and two products: 2^-20 of itself; the exponential of -88 or -90 is below FP32's normal numbers, off by
    2 units of 2^-149, which gate and up multiply. It is then rounded to 11 bits; the sums over I and the choices and the routing weights add (I / 32 + 32) 2^-23, the result
    half a unit of 8 bits."""
    T, E, k, H, I = 3, 4, 2, 64, 96
    case = Case(T, E, k, H, I, seed=26)
    case.x[:] = 0
    case.x[:, 0], case.x[:, 1] = gate, 1.0
    case.router[:] = 0
    case.router[:, 1] = torch.tensor([0.5, 2.0, 1.0, 0.25])      # choices 1 and 2
    case.c13[:] = 0
    case.c13[:, 0, :I] = 2                                       # gate: 1.0 times x[0]
    case.c13[:, 1, I:] = 2 + np.arange(I) % 4                    # up: 1, 1.5, 2 or 3 times 2^100
    case.e13[:, :, :I], case.e13[:, :, I:] = 127, 227
    y, _ = case.reference()
    got = w4.mxfp4_moe(*case.device(), k, renormalize=True).double().cpu().numpy()
    _, p = Q.route(case.logits(), k, True)
    u = np.array([1.0, 1.5, 2.0, 3.0])[np.arange(I) % 4] * 2.0 ** 100
    silu = gate / (1 + np.exp(-gate))
    dh = np.abs(silu * u) * (2.0 ** -11 + 2.0 ** -20 + (I / 32 + 32) * 2.0 ** -23) + abs(gate) * 2.0 ** -148 * u
    bound = sum(p[0, j] * (dh @ np.abs(Q.values(case.c2[e], case.e2[e], 0))) for j, e in enumerate((1, 2)))
    assert np.all(np.abs(got - y) <= bound + 2.0 ** -8 * (np.abs(y) + bound) + 2.0 ** -134)
    assert (np.abs(y).max() > 0) == (gate != 0)
