"""The product of int8 operands against 64-bit arithmetic.

Tolerance: where every partial sum is below 2^24 the sum is exact, and
y = RN_t(RN(RN(S sa) sb)) is off by two FP32 roundings and one to the output type:
(2 * 2^-24 + eps_t / 2) |y|, a second-order term and half the smallest subnormal
besides. Larger sums are held in FP32 while they grow: at most K / 16 + 256
additions, each off by at most 2^-23 of sum |a b| (a truncated last bit).
"""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


def operands(M, N, K, seed, sigma=40.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    def codes(r):
        v = torch.randn((r, K), device="cuda", generator=gen) * sigma
        return v.round().clamp(-128, 127).to(torch.int8)
    scale = lambda r: torch.rand(r, device="cuda", generator=gen) * 2e-3 + 1e-4  # noqa: E731
    return codes(M), scale(M), codes(N), scale(N)


def check(y, a, sa, b, sb):
    M, K = a.shape
    eps = torch.finfo(y.dtype).eps / 2
    least = torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps / 2
    for n in range(0, b.shape[0], 8192):
        bd, s = b[n:n + 8192].double(), sb[n:n + 8192].double()
        S = a.double() @ bd.T                           # whole numbers below 2^53: exact
        ref = S * sa.double()[:, None] * s
        size = a.double().abs() @ bd.abs().T
        grown = torch.where(size < 2.0 ** 24, 0.0, (K / 16 + 256) * 2.0 ** -23 * size) * sa.double()[:, None] * s
        bound = (2 * 2.0 ** -24 + eps) * 1.0001 * ref.abs() + grown + least
        err = (y[:, n:n + 8192].double() - ref).abs()
        assert bool((err <= bound).all()), (err - bound).max().item()


def run(M, N, K, dtype, seed=0, sigma=40.0):
    a, sa, b, sb = operands(M, N, K, seed + M + N + K, sigma)
    buf = torch.full((M * N + 128,), -5.0, dtype=dtype, device="cuda")
    y = buf[64:64 + M * N].view(M, N)
    w4.int8_matmul(a, sa, b, sb, out=y)
    check(y, a, sa, b, sb)
    assert bool((buf[:64] == -5.0).all()) and bool((buf[-64:] == -5.0).all())
    assert w4.device_status() == w4.OK
    return a, sa, b, sb, y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65, 100, 128, 129, 192, 256, 257, 300, 513])
def test_rows(M, dtype):
    run(M, 520, 1040, dtype)


@pytest.mark.parametrize("N", [8, 16, 120, 128, 136, 264, 2600])
@pytest.mark.parametrize("M", [1, 7, 40, 150])
def test_columns(M, N):
    run(M, N, 272, torch.float32)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 112, 128, 144, 240, 256, 272, 512, 528, 2080, 8208])
@pytest.mark.parametrize("M", [1, 6, 20, 130, 300])
def test_depths(M, K):
    run(M, 264, K, torch.float32)


@pytest.mark.parametrize("M,N,K", [(1, 2048, 2048), (16, 16384, 5376), (64, 16384, 5376), (300, 2600, 2080),
                                   (128, 43008, 512), (700, 4096, 4096), (1100, 5128, 288), (2048, 8192, 1024),
                                   (5000, 264, 1040), (3, 43008, 5376), (12, 43008, 5376)])
def test_sizes(M, N, K):
    run(M, N, K, torch.bfloat16)


# On 152 SMs: 256 x 256 tiles on CTA pairs; 128-row tiles shared between CTAs; clusters of 2 to 6 CTAs per tile; eight
# rows by dot products.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(129, 20488, 1040), (257, 10248, 16), (1030, 4104, 272), (300, 16392, 144),
                                   (513, 5000, 2064), (16, 20488, 1040), (30, 43008, 272), (64, 24584, 400),
                                   (128, 20488, 656), (100, 21000, 16), (12, 6400, 5376), (40, 264, 4112),
                                   (8, 8192, 4096), (8, 8200, 8208), (6, 8192, 4096), (6, 16392, 8192), (5, 520, 1040),
                                   (7, 40, 8208), (8, 12296, 144), (16, 6152, 272), (9, 2056, 1040), (13, 264, 8208), (16, 2048, 4096)])
def test_plans(M, N, K, dtype):
    run(M, N, K, dtype)


# On 152 SMs: tiles of 32, 64 and 128 rows, several of them along M, whole and in clusters of 2 to 8.
@pytest.mark.parametrize("M,N,K", [(669, 24, 16352), (200, 2056, 2064), (3107, 40, 1008), (1097, 200, 1264), (65, 4104, 4112),
                                   (301, 2600, 2080), (257, 4096, 1040), (7201, 104, 656), (9000, 128, 272),
                                   (81, 5384, 2064), (513, 4104, 272), (12000, 104, 144), (40, 264, 8208), (129, 8, 32)])
def test_rows_per_tile(M, N, K):
    run(M, N, K, torch.bfloat16)


# A whole wave of pairs and the other columns on 128-row tiles: both write rows of the same y.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(300, 10248, 2064), (436, 10680, 4112), (900, 9224, 2064), (1030, 5128, 4112),
                                   (513, 8200, 8208)])
def test_waves_and_the_rest(M, N, K, dtype):
    run(M, N, K, dtype)


# CTA pairs with tiles of every height, part of a wave and several; columns and rows that end inside a tile.
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(420, 5944, 8208), (200, 9736, 8208), (129, 10000, 12304), (1100, 20488, 4112),
                                   (260, 6536, 8304), (2050, 2568, 8192), (8300, 2568, 5376), (300, 16392, 272), (380, 20488, 400),
                                   (640, 8200, 144), (150, 30728, 528), (225, 20008, 1040), (700, 5000, 2064), (1000, 6152, 160),
                                   (70, 17000, 1040), (100, 16392, 400), (128, 19456, 144), (4190, 424, 1040)])
def test_pair_tiles(M, N, K, dtype):
    a, sa, b, sb, y = run(M, N, K, dtype)
    for _ in range(3):
        assert torch.equal(w4.int8_matmul(a, sa, b, sb, out_dtype=dtype), y)


def test_chunks_of_many_rows():
    """More rows than are widened at a time, in both kernels that take widened rows."""
    run(8200, 1032, 144, torch.bfloat16)
    run(20000, 264, 272, torch.float32)
    run(16500, 8200, 48, torch.float16)


@pytest.mark.parametrize("M", [1, 8, 24, 100, 200, 600])
def test_every_value_and_full_size(M):
    """-128 .. 127 in both operands, then sums far past 2^24: every code of one sign and size."""
    N, K = 264, 8192
    gen = torch.Generator(device="cuda").manual_seed(M)
    a = torch.randint(-128, 128, (M, K), device="cuda", generator=gen).to(torch.int8)
    b = torch.randint(-128, 128, (N, K), device="cuda", generator=gen).to(torch.int8)
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    check(w4.int8_matmul(a, one(M), b, one(N), out_dtype=torch.float32), a, one(M), b, one(N))
    for av, bv in ((-128, -128), (127, -128), (127, 127)):
        a.fill_(av), b.fill_(bv)
        a[0, 1::2] = 0
        check(w4.int8_matmul(a, one(M), b, one(N), out_dtype=torch.float32), a, one(M), b, one(N))


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_exact_sums(M):
    """With scales of 1 and sums below 2^24 the FP32 result is the whole number itself."""
    a, _, b, _ = operands(M, 520, 1024, 5, sigma=80.0)
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = w4.int8_matmul(a, one(M), b, one(520), out_dtype=torch.float32)
    assert torch.equal(y.double(), a.double() @ b.double().T)


@pytest.mark.parametrize("M,N", [(2, 264), (7, 264), (24, 264), (60, 20488), (128, 264), (200, 264), (300, 16392)])
def test_largest_exact_sums(M, N):
    """K = 1024 codes of full size: sums up to 2^24 are whole numbers still."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    sign = lambda *s: torch.randint(0, 2, s, device="cuda", generator=gen) * 2 - 1  # noqa: E731
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    a, b = (127 * sign(M, 1024)).to(torch.int8), (127 * sign(N, 1024)).to(torch.int8)
    a[0], b[0] = 127, 127
    a[1], b[1] = -128, -128
    b[2, 1::2] = 126
    y = w4.int8_matmul(a, one(M), b, one(N), out_dtype=torch.float32)
    assert torch.equal(y.double(), a.double() @ b.double().T)
    assert y[1, 1] == 2.0 ** 24


@pytest.mark.parametrize("M", [1, 8, 40, 300])
def test_special_scales(M):
    """NaN and infinite scales stay in their row and column; a scale of zero gives zeros."""
    a, sa, b, sb = operands(M, 136, 272, 9)
    want = w4.int8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    sa, sb = sa.clone(), sb.clone()
    sa[0], sb[5] = float("nan"), float("nan")
    sb[6] = 0.0
    y = w4.int8_matmul(a, sa, b, sb, out_dtype=torch.float32)
    assert bool(y[0].isnan().all()) and bool(y[:, 5].isnan().all())
    keep = torch.ones_like(y, dtype=torch.bool)
    keep[0], keep[:, 5], keep[:, 6] = False, False, False
    assert torch.equal(y[keep], want[keep]) and bool((y[1:, 6] == 0).all())


@pytest.mark.parametrize("M", [1, 8, 40, 128, 300])
def test_repeats_bit_for_bit(M):
    """Twice the same, and a row alone or among others: its sums here are exact, so it is the same."""
    a, sa, b, sb = operands(M, 4104, 2064, 11)
    y = w4.int8_matmul(a, sa, b, sb)
    for _ in range(3):
        assert torch.equal(w4.int8_matmul(a, sa, b, sb), y)
    m = M // 2
    assert torch.equal(w4.int8_matmul(a[m:m + 1].contiguous(), sa[m:m + 1].clone(), b, sb)[0], y[m])


def test_workspace_serves_every_shape():
    """One workspace in turn for shapes of every plan, its first bytes zero again after each."""
    lib = w4.load_library()
    shapes = [(16, 16384, 512), (300, 2600, 2080), (1, 2048, 4096), (64, 4096, 5376), (100, 8200, 96), (2, 520, 64),
              (2100, 2048, 1040), (436, 10680, 4112), (128, 16384, 512), (24, 43008, 272), (16, 16384, 512)]
    need = max(lib.w4a16_int8_matmul_workspace_bytes(*s) for s in shapes)
    ws = torch.full((max(need, 4096),), 0xA5, dtype=torch.uint8, device="cuda")
    ws[:4096].zero_()
    for i, (M, N, K) in enumerate(shapes):
        a, sa, b, sb = operands(M, N, K, i)
        check(w4.int8_matmul(a, sa, b, sb, out_dtype=torch.float32, workspace=ws), a, sa, b, sb)
        assert not ws[:4096].any()
    assert w4.device_status() == w4.OK


def test_small_workspace_is_refused():
    lib = w4.load_library()
    for M, N, K in ((64, 4096, 5376), (300, 2600, 2080), (2048, 8192, 1024)):
        need = lib.w4a16_int8_matmul_workspace_bytes(M, N, K)
        if not need:
            continue
        a, sa, b, sb = operands(M, N, K, 1)
        with pytest.raises(w4.W4A16Error) as e:
            w4.int8_matmul(a, sa, b, sb, workspace=torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))
        assert e.value.status == w4.ERR_WORKSPACE


@pytest.mark.parametrize("shapes", [((64, 16384, 512), (16, 8192, 512)), ((300, 2600, 2080), (140, 2600, 512)),
                                    ((1, 2048, 2048), (8, 2048, 512)),
                                    ((436, 10680, 4112), (200, 9736, 8208))])
def test_graphs_captured_cold(shapes):
    """Two graphs of calls without a workspace, captured before any eager call, replayed in every order."""
    calls = [operands(*s, 21 + i) for i, s in enumerate(shapes)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    graphs, outs = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            outs.append(w4.int8_matmul(*c, out_dtype=torch.float32))
        graphs.append(g)
    for i in (1, 1, 0, 1, 0, 0):
        outs[i].zero_()
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        check(outs[i], *calls[i])
    assert w4.device_status() == w4.OK


def test_streams():
    """Calls on two streams at once, each with the workspace the binding keeps for its stream."""
    shapes = [(64, 8192, 1040), (300, 2600, 2080)]
    ops = [operands(*s, 31 + i) for i, s in enumerate(shapes)]
    streams = [torch.cuda.Stream() for _ in shapes]
    torch.cuda.synchronize()
    outs = [[w4.int8_matmul(*o, out_dtype=torch.float32, stream=s) for o, s in zip(ops, streams)] for _ in range(20)]
    torch.cuda.synchronize()
    for pair in outs:
        for y, o, first in zip(pair, ops, outs[0]):
            assert torch.equal(y, first)
    for y, o in zip(outs[0], ops):
        check(y, *o)


def test_past_32_bits():
    """A weight of more than 2^32 bytes and results past 2^32 elements."""
    M, N, K = 9, 300008, 16384
    gen = torch.Generator(device="cuda").manual_seed(41)
    b = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    edge = torch.randint(-127, 128, (64, K), device="cuda", generator=gen).to(torch.int8)
    b[:32], b[-32:] = edge[:32], edge[32:]
    a, sa, _, _ = operands(M, 8, K, 42)
    sb = torch.rand(N, device="cuda", generator=gen) * 1e-3
    for rows in (1, M):
        y = w4.int8_matmul(a[:rows].contiguous(), sa[:rows].clone(), b, sb, out_dtype=torch.float32)
        for part in (slice(0, 32), slice(N - 32, N)):
            check(y[:, part].contiguous(), a[:rows], sa[:rows], b[part], sb[part])
        assert not y[:, 32:-32].any()
    del b, y
    M, N, K = 32800, 131072, 16
    a, sa, b, sb = operands(M, N, K, 43)
    y = w4.int8_matmul(a, sa, b, sb)
    for part in (slice(0, 8), slice(M - 8, M)):
        check(y[part], a[part], sa[part], b, sb)
    assert w4.device_status() == w4.OK
