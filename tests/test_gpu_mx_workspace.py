"""The MXFP4 product's workspace as the header describes it: 128 KB per SM and
four tickets per 128 columns, rounded up to 256 bytes, for up to 32 rows; none
for more. One sized for the largest N serves every shape."""
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402

pytestmark = pytest.mark.gpu


def described(M, N):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return (sms << 17) + (16 * -(-N // 128) + 255) // 256 * 256 if M <= 32 else 0


@pytest.mark.parametrize("M", [1, 16, 17, 32, 33, 64, 128, 129, 300, 4096])
@pytest.mark.parametrize("N,K", [(8, 32), (2600, 2080), (43008, 5376), (1 << 20, 64)])
def test_size(M, N, K):
    assert w4.workspace_bytes(w4.OP_MXFP4_MATMUL, M, N, K, 32) == described(M, N)


def test_a_workspace_sized_from_the_text_is_taken():
    """Shapes of every plan in turn in one workspace sized for the largest N, the middle ones without any."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    lib = w4.load_library()
    ws = torch.zeros(described(1, 43008), dtype=torch.uint8, device="cuda")
    for M, N, K in ((16, 43008, 512), (300, 2600, 2080), (1, 2048, 4096), (32, 20480, 288), (70, 8200, 96),
                    (9, 20488, 1056), (2, 520, 64), (16, 43008, 512)):
        words = lambda r: torch.randint(-2 ** 31, 2 ** 31, (r, K // 8), dtype=torch.int32, device="cuda", generator=gen)
        tiles = lambda r: w4.mxfp4_tile_scales(torch.randint(118, 125, (r, K // 32), dtype=torch.uint8, device="cuda",
                                                             generator=gen))
        a, ea, b, eb = words(M), tiles(M), words(N), tiles(N)
        y = torch.empty((M, N), dtype=torch.float32, device="cuda")
        for p, n in ((ws.data_ptr(), ws.numel()),) + (((0, 0),) if M > 32 else ()):
            y.fill_(float("nan"))
            st = lib.w4a16_mxfp4_matmul(a.data_ptr(), ea.data_ptr(), b.data_ptr(), eb.data_ptr(), y.data_ptr(), M, N,
                                        K, w4.F32, p, n, torch.cuda.current_stream().cuda_stream)
            assert st == w4.OK
            av, bv = w4.mxfp4_dequant_rows(a, ea).double(), w4.mxfp4_dequant_rows(b, eb).double()
            # K / 32 block sums, each addition within 2^-22 of the running magnitude
            bound = (K / 32 + 8) * 2.0 ** -22 * (av.abs() @ bv.abs().T)
            assert bool(((y.double() - av @ bv.T).abs() <= bound).all())
    assert w4.device_status() == w4.OK
