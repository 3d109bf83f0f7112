"""The step between two blocks against 64-bit arithmetic.

Tolerance. With e = 2^-24 per FP32 rounding: a sum of squares over a row is a
chain of at most 16 fused additions per thread, 11 more additions deep over
threads, so it is off by at most 27 e, and its root by half of that; 1 / H, the mean, + eps add 3
roundings (half of them after the root), rsqrtf 4 e (2 units in the last place).
So a norm factor is off by at most 20 e, u by 23 e (three products), and r' by
24 e |scale gate u| + 2 e |r'| before it is rounded to be stored. For y the
factor's own error includes that of r': at most d = (24 ||scale gate u|| + 2 ||r'||) e
over ||r'||; y is off by (20 e + d + 3 e) |y| and the error of r' carried along,
then rounded to its type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import weight_only_int4_gb300 as w4  # noqa: E402
from oracle import int8_oracle as I8  # noqa: E402

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
bf16, f16, f32 = torch.bfloat16, torch.float16, torch.float32
PAIRS = [(bf16, bf16), (bf16, f32), (f16, f16), (f16, f32), (f32, f32)]


def inputs(T, H, dtype, res, gate, seed=0, after=True):
    gen = torch.Generator().manual_seed(seed + T * H)
    rand = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    shape = {"channel": (H,), "token": (T, 1), "element": (T, H)}.get(gate)
    return dict(residual=(3 * rand(T, H)).to(res), weight=(1 + 0.2 * rand(H)).to(dtype), h=rand(T, H).to(dtype),
                after=(1 + 0.2 * rand(H)).to(dtype) if after else None,
                gate=None if shape is None else rand(*shape).to(dtype))


def wide(t):
    return None if t is None else t.double().cpu().numpy()


def reference(o, scale, eps):
    """(r', y) and how far each may be off before its last rounding."""
    r, y = I8.block_norm(*(wide(o.get(k)) for k in ("residual", "weight", "h", "after", "gate")), scale=scale, eps=eps)
    gu = np.abs(r - wide(o["residual"]))
    dr = 24 * E * gu + 2 * E * np.abs(r)
    if y is None:
        return r, dr, None, None
    norm = np.sqrt((r * r).sum(axis=1, keepdims=True)) + 1e-300
    d = np.sqrt((dr * dr).sum(axis=1, keepdims=True)) / norm
    factor = np.abs(wide(o["weight"])) / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
    return r, dr, y, 1.01 * ((23 * E + d) * np.abs(y) + dr * factor)


def close(got, want, off, dtype):
    half = torch.finfo(dtype).eps / 2
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = np.abs(wide(got) - want)
    bound = off * (1 + half) + half * np.abs(want) + least
    assert (err <= bound).all(), (err / bound).max()


def guarded(shape, dtype):
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), 77, dtype=dtype, device="cuda")
    return buf, buf[64:64 + n].view(shape)


def on_device(o):
    return {k: None if v is None else v.cuda() for k, v in o.items()}


def check(o, dtype, res, scale=1.0, eps=1e-6):
    T, H = o["residual"].shape
    r, dr, y, dy = reference(o, scale, eps)
    dev = on_device(o)
    bufs = [guarded((T, H), res), guarded((T, H), dtype)]
    got_r, got_y = w4.block_norm(**dev, scale=scale, eps=eps, out=tuple(v for _, v in bufs))
    close(got_r, r, dr, res)
    close(got_y, y, dy, dtype)
    bufs += [guarded((T, H), res), guarded((T, H), torch.int8), guarded((T,), f32)]
    again, codes, cs = w4.block_norm(**dev, scale=scale, eps=eps, quantize=True, out=tuple(v for _, v in bufs[2:]))
    assert torch.equal(again, got_r)
    # the code is within half a step of the quotient of a y that is itself off by dy
    s = wide(cs)[:, None]
    assert (np.abs(wide(codes) * s - y) <= 0.5 * s * (1 + 4 * E) + dy + 4 * E * np.abs(y)).all()
    assert (np.abs(s[:, 0] * 127 - np.abs(y).max(axis=1)) <= dy.max(axis=1) + 2 * E * np.abs(y).max(axis=1)).all()
    if dtype == f32:   # y is returned unrounded: its codes are known bit for bit
        c, sc = I8.quantize_rows(wide(got_y))
        assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(cs.cpu().numpy(), sc)
    for b, _ in bufs:
        assert bool((b[:64] == 77).all()) and bool((b[-64:] == 77).all())


@pytest.mark.parametrize("dtype,res", PAIRS)
@pytest.mark.parametrize("T,H", [(1, 16), (2, 256), (3, 272), (1, 5376), (77, 2608), (5, 8192), (4, 8208), (3, 12288),
                                 (2, 12304), (3, 16384), (5, 1040), (2, 6128), (3, 6144), (2, 9216), (3, 9232), (2, 11008)])
def test_shapes(T, H, dtype, res):
    check(inputs(T, H, dtype, res, "channel"), dtype, res, scale=0.22)


@pytest.mark.parametrize("dtype,res", PAIRS)
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "element"])
def test_forms(gate, after, dtype, res):
    check(inputs(9, 528, dtype, res, gate, after=after), dtype, res, scale=-1.5, eps=1e-5)


@pytest.mark.parametrize("T,H", [(2, 16), (1, 32), (3, 16)])
def test_gate_shapes_of_few_tokens(T, H):
    for gate in ("channel", "token", "element"):
        check(inputs(T, H, bf16, f32, gate, seed=5), bf16, f32)


@pytest.mark.parametrize("dtype,res", PAIRS)
def test_norm_alone(dtype, res):
    """Without h: the residual comes back itself, y of it as it is."""
    o = on_device(inputs(7, 544, dtype, res, "none"))
    r, y = w4.block_norm(o["residual"], o["weight"])
    assert r is o["residual"]
    want = dict(residual=o["residual"], weight=o["weight"])
    _, _, ref, dy = reference(want, 1.0, 1e-6)
    close(y, ref, dy, dtype)
    back, codes, cs = w4.block_norm(o["residual"], o["weight"], quantize=True)
    assert back is o["residual"]
    s = wide(cs)[:, None]
    assert (np.abs(wide(codes) * s - ref) <= 0.5 * s * (1 + 4 * E) + dy + 4 * E * np.abs(ref)).all()


@pytest.mark.parametrize("dtype,res", PAIRS)
def test_residual_alone(dtype, res):
    """Without weight: r' alone, in a new tensor and in place."""
    o = inputs(7, 544, dtype, res, "token")
    o.pop("weight")
    r, dr, _, _ = reference(o, 0.5, 1e-6)
    dev = on_device(o)
    got = w4.block_norm(**dev, scale=0.5)
    close(got, r, dr, res)
    same = w4.block_norm(**dev, scale=0.5, out=dev["residual"])
    assert same is dev["residual"] and torch.equal(same, got)


@pytest.mark.parametrize("T,H", [(3, 528), (40, 16384)])
def test_in_place(T, H):
    o = on_device(inputs(T, H, bf16, f32, "element"))
    r, y = w4.block_norm(**o)
    r, y = r.clone(), y.clone()
    got = w4.block_norm(**o, out=(o["residual"], torch.empty_like(y)))
    assert got[0] is o["residual"] and torch.equal(got[0], r) and torch.equal(got[1], y)


def test_rows_are_alone():
    """A row with an infinity or a NaN, rows of zeros and very small rows; the others are as without them."""
    o = on_device(inputs(9, 528, f32, f32, "none"))
    want_r, want_y = w4.block_norm(**o)
    _, want_c, want_s = w4.block_norm(**o, quantize=True)
    o["residual"][1, 3] = float("inf")
    o["h"][2, 4] = float("nan")
    o["residual"][3], o["h"][3] = 0, 0
    o["residual"][4] *= 1e-12
    o["h"][4] *= 1e-12
    r, y = w4.block_norm(**o)
    _, c, s = w4.block_norm(**o, quantize=True)
    keep = [0, 5, 6, 7, 8]
    assert torch.equal(r[keep], want_r[keep]) and torch.equal(y[keep], want_y[keep])
    assert torch.equal(c[keep], want_c[keep]) and torch.equal(s[keep], want_s[keep])
    assert bool(y[1, 3].isnan()) and bool(y[2].isnan().all())
    assert not c[1:4].any() and bool(s[1:3].isnan().all()) and s[3] == 0 and not y[3].any()
    one = {k: v if v is None or v.dim() == 1 else v[4:5].contiguous() for k, v in o.items()}
    ref_r, dr, ref_y, dy = reference(one, 1.0, 1e-6)
    close(r[4:5], ref_r, dr, f32)
    close(y[4:5], ref_y, dy, f32)


@pytest.mark.parametrize("T", [1, 300, 5000])
def test_a_row_does_not_depend_on_the_others(T):
    o = on_device(inputs(T, 1040, bf16, bf16, "channel"))
    r, c, s = w4.block_norm(**o, quantize=True)
    t = T // 2
    one = {k: v if v is None or v.dim() == 1 else v[t:t + 1].contiguous() for k, v in o.items()}
    r1, c1, s1 = w4.block_norm(**one, quantize=True)
    assert torch.equal(r1[0], r[t]) and torch.equal(c1[0], c[t]) and s1[0] == s[t]


def test_captured():
    o = on_device(inputs(33, 2608, bf16, f32, "channel"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, c, s = w4.block_norm(**o, quantize=True)
    o["h"].mul_(2.0)
    graph.replay()
    want = w4.block_norm(**o, quantize=True)
    for got, ref in zip((r, c, s), want):
        assert torch.equal(got, ref)


def test_past_32_bits():
    T, H = 262160, 16384
    r = torch.zeros((T, H), dtype=bf16, device="cuda")
    r[-4:].normal_()
    r[:4].normal_()
    weight = torch.ones(H, dtype=bf16, device="cuda")
    _, y = w4.block_norm(r, weight)
    for part in (slice(0, 4), slice(T - 4, T)):
        _, _, ref, dy = reference(dict(residual=r[part], weight=weight), 1.0, 1e-6)
        close(y[part], ref, dy, bf16)
    assert not y[4:-4:1001].any()
