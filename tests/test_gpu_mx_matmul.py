"""Product of two MXFP4 operands on the GPU against the FP64 oracle.

Tolerance: every product of two codes and its power-of-two scale is exact, so
the only errors are those of the FP32 accumulation and the last rounding. The
accumulator takes K / 32 block sums per element; allowing each addition an
error of 2^-22 of the running magnitude, which sum |a b| bounds, gives
|y - ref| <= (K / 32 + 8) 2^-22 sum |a b|, plus half an ulp of the output type
(2^-8 of |ref| for bf16, 2^-11 for fp16).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from oracle import mxfp4_ops_oracle as Q  # noqa: E402

pytestmark = pytest.mark.gpu

ULP = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


class Operand:
    """A random row-layout operand: uniform codes, exponent bytes in a range."""

    def __init__(self, R, K, seed, lo=118, hi=125):
        rng = np.random.default_rng(seed)
        self.codes = rng.integers(0, 16, size=(R, K)).astype(np.uint8)
        self.e = rng.integers(lo, hi + 1, size=(R, K // 32)).astype(np.uint8)
        self.R, self.K = R, K

    def device(self):
        words = torch.from_numpy(np.ascontiguousarray(Q.words(self.codes, 1)).view(np.int32)).cuda()
        return words, w4.mxfp4_tile_scales(torch.from_numpy(self.e).cuda())

    def values(self):
        return torch.from_numpy(Q.values(self.codes, self.e, 1)).cuda()


def guarded(M, N, dtype, pad=256):
    buf = torch.full((M * N + 2 * pad,), -1536.0, dtype=dtype, device="cuda")
    return buf, buf[pad:-pad].view(M, N), pad


def check(A, B, dtype, what=""):
    a, ea = A.device()
    b, eb = B.device()
    buf, y, pad = guarded(A.R, B.R, dtype)
    w4.mxfp4_matmul(a, ea, b, eb, out=y)
    again = w4.mxfp4_matmul(a, ea, b, eb, out_dtype=dtype)
    assert w4.device_status() == w4.OK
    assert torch.all(buf[:pad] == -1536.0) and torch.all(buf[-pad:] == -1536.0), "write outside the output"
    assert torch.equal(y, again), "two calls differ"
    av, bv = A.values(), B.values()
    ref = av @ bv.T
    bound = (A.K / 32 + 8) * 2.0 ** -22 * (av.abs() @ bv.abs().T) + ULP[dtype] * ref.abs()
    err = (y.double() - ref).abs()
    assert bool(torch.isfinite(y).all()), what
    assert bool((err <= bound).all()), f"{what}: worst excess {(err - bound).max():.3e}, max err {err.max():.3e}"


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("M", [1, 7, 16, 17, 32, 33, 64, 65, 128, 129, 300])
def test_few_rows(M, dtype):
    """Every row template, whole and shared tiles, tails in N and K."""
    N, K = 1048, 1120
    check(Operand(M, K, M), Operand(N, K, M + 1), dtype, M)


@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (1, 128, 64), (3, 136, 96), (16, 16, 128), (5, 264, 160), (130, 8, 224),
                                   (2, 40, 256), (1, 2048, 4128), (20, 20480, 288), (9, 43008, 512),
                                   (40, 30000, 320), (500, 4096, 160)])
def test_small_and_odd(M, N, K):
    check(Operand(M, K, 3), Operand(N, K, 4), torch.float32, (M, N, K))


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("M,N,K", [(1, 1000, 8224), (16, 2048, 5376), (17, 5376, 4128), (50, 264, 12000),
                                   (100, 1288, 9120), (200, 640, 6176)])
def test_few_tiles_of_a_long_k(M, N, K, dtype):
    """K split over the CTAs of a cluster, in equal and unequal parts, for every row template."""
    check(Operand(M, K, 16), Operand(N, K, 17), dtype, (M, N, K))


@pytest.mark.parametrize("dtype", list(ULP))
@pytest.mark.parametrize("M,N,K", [(2560, 2560, 512), (1032, 5000, 288), (513, 8008, 1056), (4100, 1288, 64),
                                   (2300, 4360, 2080)])
def test_many_tiles(M, N, K, dtype):
    """256 x 256 tiles for most CTA pairs: one and several per pair, tails in M, N and K, odd numbers of 128-row tiles."""
    check(Operand(M, K, 5), Operand(N, K, 6), dtype, (M, N, K))


@pytest.mark.parametrize("M,N,K", [(40, 520, 512), (2048, 2560, 256)])
def test_wide_exponents(M, N, K):
    """Exponent bytes over most of their range: products from 2^-107 to 2^113 in one sum."""
    check(Operand(M, K, 7, 74, 180), Operand(N, K, 8, 74, 180), torch.float32, (M, N, K))


@pytest.mark.parametrize("M,N", [(9, 264), (1290, 8448)])
def test_each_block_has_its_own_exponent(M, N):
    """One-hot rows of A pick single elements of B: exact, whatever block they are in."""
    K = 2080
    B = Operand(N, K, 9, 100, 140)
    codes = np.zeros((M, K), dtype=np.uint8)
    cols = [(37 * m + 5) % K for m in range(M)]
    codes[np.arange(M), cols] = 2                      # 1.0
    A = Operand(M, K, 10, 127, 127)
    A.codes = codes
    A.e = (127 + (np.arange(M)[:, None] + np.arange(K // 32)[None, :]) % 5).astype(np.uint8)
    y = w4.mxfp4_matmul(*A.device(), *B.device(), out_dtype=torch.float32)
    want = B.values()[:, cols].T * torch.from_numpy(np.ldexp(1.0, A.e[np.arange(M), np.array(cols) // 32].astype(int)
                                                             - 127)).cuda()[:, None]
    assert torch.equal(y.double(), want)


@pytest.mark.parametrize("M,N", [(6, 136), (700, 7696)])
def test_nan_bytes_and_zero_operands(M, N):
    K = 288
    A, B = Operand(M, K, 11), Operand(N, K, 12)
    A.e[2, 4] = 255
    B.e[N - 3, 8] = 255
    y = w4.mxfp4_matmul(*A.device(), *B.device(), out_dtype=torch.float32)
    nan = torch.isnan(y)
    assert bool(nan[2].all()) and bool(nan[:, N - 3].all())
    keep = ~(torch.arange(M) == 2).cuda()[:, None] & ~(torch.arange(N) == N - 3).cuda()[None, :]
    assert not bool(nan[keep].any())
    Z = Operand(M, K, 13)
    Z.codes[:] = 0
    assert torch.count_nonzero(w4.mxfp4_matmul(*Z.device(), *Operand(N, K, 12).device())) == 0


def test_stale_padding_rows_do_not_matter():
    """Rows past the operand's end share its last exponent tile: NaN bytes there change nothing."""
    for M, N in ((5, 200), (1000, 5000)):
        K = 160
        A, B = Operand(M, K, 14), Operand(N, K, 15)
        a, ea = A.device()
        b, eb = B.device()
        ref = w4.mxfp4_matmul(a, ea, b, eb)
        for op, t in ((A, ea), (B, eb)):
            rows = torch.arange(t.shape[0] * 128).view(t.shape[0], 1, 4, 32, 1).transpose(2, 3)
            live = (rows < op.R).expand(t.shape).cuda()
            t[~live] = 255
        assert torch.equal(w4.mxfp4_matmul(a, ea, b, eb), ref)


def test_quantise_then_multiply():
    """The layer as it is used: activations quantised per call, a weight quantised once."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((37, 672), generator=gen).to(torch.bfloat16)
    w = (torch.randn((328, 672), generator=gen) * 0.05).to(torch.bfloat16)
    b = w4.mxfp4_quantize(w.cuda(), 1)
    y = w4.mxfp4_matmul(*w4.mxfp4_quantize(x.cuda(), 1), *b, out_dtype=torch.float32)
    xv = Q.values(*Q.quantize(x.double().numpy(), 1), 1)
    wv = Q.values(*Q.quantize(w.double().numpy(), 1), 1)
    bound = (672 / 32 + 8) * 2.0 ** -22 * (np.abs(xv) @ np.abs(wv).T)
    assert np.all(np.abs(y.double().cpu().numpy() - xv @ wv.T) <= bound)


def test_workspace_reuse_and_side_stream():
    """One workspace for shapes of either size in turn, on a stream of its own, and in a CUDA graph."""
    ops = [(Operand(M, K, M), Operand(N, K, N)) for M, N, K in ((3, 2048, 2048), (70, 4104, 512), (1, 264, 96))]
    dev = [(*A.device(), *B.device()) for A, B in ops]
    ref = [w4.mxfp4_matmul(*d) for d in dev]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [w4.mxfp4_matmul(*d, stream=side) for d in dev * 2]
    torch.cuda.synchronize()
    for g, r in zip(got, ref * 2):
        assert torch.equal(g, r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [w4.mxfp4_matmul(*d) for d in dev]
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o, r)
    assert w4.device_status() == w4.OK


def test_binding_refusals():
    A, B = Operand(4, 64, 1), Operand(16, 64, 2)
    a, ea = A.device()
    b, eb = B.device()
    with pytest.raises(ValueError):
        w4.mxfp4_matmul(a, ea, b[:, :4].contiguous(), w4.mxfp4_tile_scales(
            torch.zeros((16, 1), dtype=torch.uint8, device="cuda")))
    with pytest.raises(ValueError):
        w4.mxfp4_matmul(a, ea[:, :, :16], b, eb)
    with pytest.raises(TypeError):
        w4.mxfp4_matmul(a.float(), ea, b, eb)
    with pytest.raises(TypeError):
        w4.mxfp4_matmul(a, ea, b, eb, out_dtype=torch.float64)
    with pytest.raises(ValueError):
        w4.mxfp4_matmul(a, ea, b, eb, out=torch.empty((4, 15), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(w4.W4A16Error) as err:
        w4.mxfp4_matmul(a, ea, b[:12].contiguous(), eb)                # N % 8
    assert err.value.status == w4.ERR_SHAPE
    with pytest.raises(w4.W4A16Error) as err:
        w4.mxfp4_matmul(a, ea, b, eb, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    assert err.value.status == w4.ERR_WORKSPACE
