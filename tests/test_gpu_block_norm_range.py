"""The step between two blocks at the ends of the FP32 range: each norm is formed in the
order it is written, x * rsqrt(mean(x^2) + eps) first and the vector after it, so no product
leaves the range that the formula's own steps stay in. Tolerances as in
test_gpu_block_norm.py."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from test_gpu_block_norm import PAIRS, close, reference  # noqa: E402

pytestmark = pytest.mark.gpu

bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
WIDE = [(bf16, bf16), (bf16, f32), (f32, f32)]   # types that reach the ends of FP32's range


def rows(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed + sum(shape)))


@pytest.mark.parametrize("dtype,res", WIDE)
@pytest.mark.parametrize("H", [256, 2608, 16384])
def test_squares_past_the_range(H, dtype, res):
    """Rows of h whose sum of squares is infinite add nothing, whatever `after` and the gate are."""
    h = rows(4, H).to(dtype)
    h[0] = torch.finfo(dtype).max * h[0].sign()
    h[1, 5] = 3e38
    h[2] = 1.5 * 2.0 ** 63     # each square is finite
    r = rows(4, H, seed=1).to(res)
    after = torch.full((H,), 1.5e10, dtype=dtype)
    weight = torch.ones(H, dtype=dtype)
    for gate in (None, torch.full((H,), 3.0, dtype=dtype)):
        new, y = w4.block_norm(r.cuda(), weight.cuda(), h.cuda(), after=after.cuda(),
                               gate=None if gate is None else gate.cuda())
        assert torch.equal(new[:3].cpu(), r[:3])
        _, want = w4.block_norm(r.cuda(), weight.cuda())
        assert torch.equal(y[:3], want[:3])
        assert bool(new[3].isfinite().all()) and not torch.equal(new[3].cpu(), r[3])
    # and rows of r' are normalised to zero
    big = (r.float() * 0 + 2.0 ** 100).to(res).cuda()
    _, y = w4.block_norm(big, torch.full((H,), 2.0 ** 60, dtype=dtype).cuda())
    assert not y.any()
    _, codes, scale = w4.block_norm(big, torch.full((H,), 2.0 ** 60, dtype=dtype).cuda(), quantize=True)
    assert not codes.any() and not scale.any()


@pytest.mark.parametrize("dtype,res", PAIRS)
def test_zero_rows_under_the_largest_weights(dtype, res):
    H = 528
    top = torch.full((H,), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    zero = torch.zeros((3, H), dtype=res, device="cuda")
    h = torch.zeros((3, H), dtype=dtype, device="cuda")
    new, y = w4.block_norm(zero, top, h, after=top)
    assert not new.any() and not y.any()
    _, codes, scale = w4.block_norm(zero, top, h, after=top, quantize=True)
    assert not codes.any() and not scale.any()


@pytest.mark.parametrize("dtype,res", WIDE)
@pytest.mark.parametrize("H", [272, 5376, 13568])
def test_large_rows_and_small_weights(H, dtype, res):
    """rsqrt * weight would be subnormal. Up to 13568 squares of 2^54 N(0, 1) sum to 2^122; of 2^60 N(0, 1), 272
    sum to 2^128, past FP32's range: those rows are normalised to zero."""
    for exponent in (54, 60):
        o = dict(residual=(rows(3, H) * 2.0 ** exponent).to(res), weight=(rows(H) * 2.0 ** -82).to(dtype))
        past = (o["residual"].double() ** 2).sum(dim=1) > 1.001 * 2.0 ** 128
        assert bool(past.all()) == (exponent == 60) or (exponent == 60 and H == 272)
        _, _, want, off = reference(o, 1.0, 1e-6)
        _, y = w4.block_norm(o["residual"].cuda(), o["weight"].cuda())
        assert not y.cpu()[past].any()
        keep = (o["residual"].double() ** 2).sum(dim=1) < 0.999 * 2.0 ** 128
        close(y.cpu()[keep], want[keep.numpy()], off[keep.numpy()], dtype)


@pytest.mark.parametrize("dtype,res", [(bf16, f32), (f32, f32)])
def test_small_rows_and_small_vectors(dtype, res):
    """h * after would be zero in FP32, and with the norm's factor is not."""
    o = dict(residual=torch.zeros((3, 2608)).to(res), h=(rows(3, 2608) * 2.0 ** -58).to(dtype),
             after=(rows(2608) * 2.0 ** -96).to(dtype), weight=None)
    want, off, _, _ = reference(o, 1.0, 2.0 ** -122)
    got = w4.block_norm(o["residual"].cuda(), None, o["h"].cuda(), after=o["after"].cuda(), eps=2.0 ** -122)
    assert bool((got != 0).any(dim=1).all())
    close(got, want, off, res)


@pytest.mark.parametrize("dtype,res", [(bf16, f32), (f32, f32)])
def test_small_rows_and_large_vectors(dtype, res):
    """h * after would be infinite, and with the norm's factor is not."""
    o = dict(residual=rows(3, 528).to(res), h=(rows(3, 528) * 2.0 ** 50).to(dtype),
             after=(rows(528) * 2.0 ** 90).to(dtype), weight=None)
    want, off, _, _ = reference(o, 1.0, 1e-6)
    got = w4.block_norm(o["residual"].cuda(), None, o["h"].cuda(), after=o["after"].cuda())
    close(got, want, off, res)
