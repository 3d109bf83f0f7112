"""What is measured of the 8-bit integer linear layer and the fused block norm:
quantisation to int8, the product of int8 operands, and the step between two
blocks of a transformer (norm after, gate, residual, norm before, quantisation).

Every case exists in two forms. The plain form (`own` false) is elementary torch
arithmetic, in 32 bits, in 64 where a value next to a rounding border decides a
whole number, rounded once at the end. The framework's form (`own` true) makes
the calls a user makes of `weight_only_int4_gb300`. Both take the same state.

Formulas (one scale per row: per token of activations, per output channel of a
weight [N, K]):

    quantise   s = RN_f32(max |v| / 127), c = RN(127 v / max |v|), ties to even;
               value = c * s
    linear     y[m, n] = (sum_k c[m, k] w[n, k]) * s[m] * t[n]
    norm       u = h * rsqrt(mean(h^2) + eps) * after     (u = h without `after`)
               r' = r + scale * gate * u,  y = r' * rsqrt(mean(r'^2) + eps) * weight
    block      the norm, y quantised to int8, and the linear layer on it
"""
import math

import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
DTYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
SIZE = {BF16: 2, F16: 2, F32: 4}
EPS = 1e-6
# Largest costs a drawn case may have: elements quantised or normalised,
# multiply-adds of a linear layer.
MAX_QUANT = 43008 * 5376
MAX_LINEAR = 2048 * 43008 * 5376
MAX_NORM = 8192 * 5376


def listed():
    return [
        # one token's activations before an int8 product: a latency case
        dict(name="quant_1x5376_bf16", op="quant", rows=1, cols=5376, dtype=BF16),
        # odd row count and length, from 32-bit activations
        dict(name="quant_77x2608_f32", op="quant", rows=77, cols=2608, dtype=F32),
        # a gate_up weight at load time, one scale per output channel
        dict(name="quant_43008x5376_bf16", op="quant", rows=43008, cols=5376, dtype=BF16),
        # one token through a small layer: a latency case
        dict(name="linear_1x2048x2048_bf16", op="linear", M=1, N=2048, K=2048, dtype=BF16, out=BF16),
        # one token through the gate_up-like layer: bound by the weights' bytes
        dict(name="linear_1x43008x5376_bf16", op="linear", M=1, N=43008, K=5376, dtype=BF16, out=BF16),
        # a decode batch through a qkv-like layer
        dict(name="linear_64x16384x5376_bf16", op="linear", M=64, N=16384, K=5376, dtype=BF16, out=BF16),
        # a ragged prefill chunk: no size a multiple of a tile, 32-bit result
        dict(name="linear_300x2600x2080_f16", op="linear", M=300, N=2600, K=2080, dtype=F16, out=F32),
        # a prefill through the gate_up-like layer: bound by the tensor cores
        dict(name="linear_2048x43008x5376_bf16", op="linear", M=2048, N=43008, K=5376, dtype=BF16, out=BF16),
        # between two blocks of a decode step, on into the next int8 layer
        dict(name="block_1x5376_to_16384_bf16", op="block", T=1, H=5376, N=16384, dtype=BF16, res=F32, after=True,
             gate="none", scale=1.0),
        # odd sizes, a gate per token, a scaled residual, 32-bit residual stream
        dict(name="norm_77x2608_f16", op="norm", T=77, H=2608, dtype=F16, res=F32, after=True, gate="token",
             scale=0.22, quantize=False),
        # a prefill's step between blocks that ends in int8 activations
        dict(name="norm_2048x5376_int8", op="norm", T=2048, H=5376, dtype=BF16, res=BF16, after=False, gate="none",
             scale=1.0, quantize=True),
        # a long prefill with norms on both sides and a gate per channel
        dict(name="norm_8192x5376_bf16", op="norm", T=8192, H=5376, dtype=BF16, res=BF16, after=True, gate="channel",
             scale=1.0, quantize=False),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], uniform over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "norm", "block"])
    while True:
        if op == "quant":
            rows, cols = _log_int(rng, 1, 43008), _log_int(rng, 16, 43008, 16)
            if rows * cols <= MAX_QUANT:
                return dict(op=op, rows=rows, cols=cols, dtype=rng.choice([BF16, F16, F32]))
        elif op == "linear":
            M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 8, 43008, 8), _log_int(rng, 16, 21504, 16)
            if M * N * K <= MAX_LINEAR and N * K <= MAX_QUANT:
                return dict(op=op, M=M, N=N, K=K, dtype=rng.choice([BF16, F16, F32]),
                            out=rng.choice([BF16, F16, F32]))
        else:
            T, H = _log_int(rng, 1, 16384), _log_int(rng, 256, 16384, 16)
            if T * H > MAX_NORM:
                continue
            dtype = rng.choice([BF16, F16, F32])
            case = dict(op=op, T=T, H=H, dtype=dtype, res=rng.choice([dtype, F32]), after=rng.choice([True, False]),
                        gate=rng.choice(["none", "channel", "token", "element"]), scale=rng.choice([1.0, 0.22]))
            if op == "norm":
                return dict(case, quantize=rng.choice([True, False]))
            N = _log_int(rng, 8, 43008, 8)
            if T * H * N <= MAX_LINEAR and N * H <= MAX_QUANT:
                return dict(case, N=N)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _activations(rows, cols, dtype, gen):
    """N(0, 1) with a few channels ten times as large, as activations have them."""
    x = torch.randn((rows, cols), device="cuda", generator=gen)
    gain = torch.ones(cols, device="cuda")
    gain[torch.randint(0, cols, (max(1, cols // 128),), device="cuda", generator=gen)] = 10.0
    return (x * gain).to(DTYPES[dtype])


def _weight(N, K, gen):
    """A quantised weight: codes as N(0, 1) rows give them, scales of weights of a few hundredths."""
    w = torch.empty((N, K), dtype=torch.float16, device="cuda").normal_(0.0, 32.0, generator=gen)
    codes = w.round_().clamp_(-127, 127).to(torch.int8)
    return codes, torch.rand(N, device="cuda", generator=gen) * 6e-4 + 3e-4


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "quant":
        if case["rows"] >= 4096:
            x = torch.empty((case["rows"], case["cols"]), dtype=DTYPES[case["dtype"]], device="cuda")
            return dict(case=case, x=x.normal_(0.0, 0.02, generator=gen))
        return dict(case=case, x=_activations(case["rows"], case["cols"], case["dtype"], gen))
    if op == "linear":
        x = _activations(case["M"], case["K"], case["dtype"], gen)
        w, t = _weight(case["N"], case["K"], gen)
        return dict(case=case, x=x, w=w, t=t)
    T, H, dtype = case["T"], case["H"], DTYPES[case["dtype"]]
    vector = lambda n: (1.0 + 0.1 * torch.randn(n, device="cuda", generator=gen)).to(dtype)  # noqa: E731
    st = dict(case=case, h=_activations(T, H, case["dtype"], gen), r=2.0 * _activations(T, H, case["res"], gen),
              weight=vector(H), after=vector(H) if case["after"] else None, gate=None)
    if case["gate"] != "none":
        shape = {"channel": (H,), "token": (T, 1), "element": (T, H)}[case["gate"]]
        st["gate"] = torch.rand(shape, device="cuda", generator=gen).to(dtype)
    if op == "block":
        st["w"], st["t"] = _weight(case["N"], H, gen)
    return st


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _quantised(x):
    """Codes (as FP32 whole numbers) and FP32 scales of the rows of x."""
    amax = x.abs().amax(dim=1, keepdim=True)
    scale = amax.float() / 127.0
    codes = torch.round(x.double() * 127.0 / torch.where(amax > 0, amax, 1.0).double())
    return codes.float(), scale


def _plain_norm(st):
    case = st["case"]
    u = st["h"].float()
    if st["after"] is not None:
        u = u * torch.rsqrt((u * u).mean(dim=1, keepdim=True) + EPS) * st["after"].float()
    if st["gate"] is not None:
        u = u * st["gate"].float()
    r = st["r"].float() + case["scale"] * u
    y = r * torch.rsqrt((r * r).mean(dim=1, keepdim=True) + EPS) * st["weight"].float()
    return r.to(DTYPES[case["res"]]), y


def run(state):
    if own:
        return _run_own(state)
    case = state["case"]
    if case["op"] == "quant":
        codes, scale = _quantised(state["x"])
        return (codes * scale).to(torch.bfloat16)
    if case["op"] == "linear":
        codes, scale = _quantised(state["x"])
        y = (codes @ state["w"].float().T) * scale * state["t"]
        return y.to(DTYPES[case["out"]])
    r, y = _plain_norm(state)
    if case["op"] == "norm" and not case["quantize"]:
        return r, y.to(DTYPES[case["dtype"]])
    codes, scale = _quantised(y)
    if case["op"] == "norm":
        return r, (codes * scale).to(torch.bfloat16)
    return r, ((codes @ state["w"].float().T) * scale * state["t"]).to(torch.bfloat16)


def _run_own(state):
    import weight_only_int4_gb300 as w4
    case = state["case"]
    if case["op"] == "quant":
        # the codes and scales, read back as the values they stand for
        codes, scale = w4.int8_quantize(state["x"])
        return w4.int8_dequant(codes, scale, out_dtype=torch.bfloat16)
    if case["op"] == "linear":
        codes, scale = w4.int8_quantize(state["x"])
        return w4.int8_matmul(codes, scale, state["w"], state["t"], out_dtype=DTYPES[case["out"]])
    step = dict(after=state["after"], gate=state["gate"], scale=case["scale"], eps=EPS)
    if case["op"] == "norm" and not case["quantize"]:
        return w4.block_norm(state["r"], state["weight"], state["h"], **step)
    r, codes, scale = w4.block_norm(state["r"], state["weight"], state["h"], quantize=True, **step)
    if case["op"] == "norm":
        return r, w4.int8_dequant(codes, scale, out_dtype=torch.bfloat16)
    return r, w4.int8_matmul(codes, scale, state["w"], state["t"], out_dtype=torch.bfloat16)


# ---------------------------------------------------------------------------
# bytes and operations of one pass
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        # x in; codes, scales and the values out
        return {"bytes": n * (SIZE[case["dtype"]] + 1 + 2) + 4 * case["rows"], "flops": 3 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * SIZE[case["dtype"]] + N * K + 4 * N + M * N * SIZE[case["out"]],
                "flops": 2 * M * N * K}
    T, H, a = case["T"], case["H"], SIZE[case["dtype"]]
    vectors = H * (1 + bool(case["after"])) * a
    gate = {"none": 0, "channel": H, "token": T, "element": T * H}[case["gate"]] * a
    # h and the residual in, the residual out
    total = T * H * (a + 2 * SIZE[case["res"]]) + vectors + gate
    if case["op"] == "block":
        N = case["N"]
        return {"bytes": total + N * H + 4 * N + 2 * T * N, "flops": 2 * T * H * N}
    total += T * H * (1 + 2) + 4 * T if case["quantize"] else T * H * a
    return {"bytes": total, "flops": 10 * T * H}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_codes(v):
    """FP64 codes and scales of rows in FP64: the whole number below 127 |v| / amax, then the comparison of
    254 |v| with (2 k + 1) amax, ties to the even one. The scale is the FP32 number that is stored."""
    a = v.abs()
    amax = a.max(dim=1, keepdim=True).values
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    k = torch.floor(127.0 * a / safe)
    over = 254.0 * a - (2.0 * k + 1.0) * safe
    up = (over > 0) | ((over == 0) & (torch.remainder(k, 2.0) == 1.0))
    return torch.copysign(k + up, v), (amax / 127.0).float().double()


def _exact_product(c, s, w, t):
    y = torch.empty((c.shape[0], w.shape[0]), dtype=torch.float64, device=c.device)
    for n in range(0, w.shape[0], 4096):
        y[:, n:n + 4096] = torch.mm(c, w[n:n + 4096].double().T)
    return y * s * t.double()


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        out = torch.empty(st["x"].shape, dtype=torch.float64, device="cuda")
        for i in range(0, case["rows"], 8192):
            c, s = _exact_codes(st["x"][i:i + 8192].double())
            out[i:i + 8192] = c * s
        return out
    if case["op"] == "linear":
        c, s = _exact_codes(st["x"].double())
        return _exact_product(c, s, st["w"], st["t"])
    H = case["H"]
    u = st["h"].double()
    if case["after"]:
        u = u / torch.sqrt(torch.linalg.vector_norm(u, dim=1, keepdim=True) ** 2 / H + EPS) * st["after"].double()
    if st["gate"] is not None:
        u = st["gate"].double() * u
    r = torch.add(st["r"].double(), u, alpha=case["scale"])
    y = st["weight"].double() * r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / H + EPS)
    if case["op"] == "norm" and not case["quantize"]:
        return r, y
    c, s = _exact_codes(y)
    if case["op"] == "norm":
        return r, c * s
    return r, _exact_product(c, s, st["w"], st["t"])
