"""What is measured of the MXFP4 operators: quantisation, the product of two
quantised operands, and the mixture-of-experts layer for a few tokens.

Every case exists in two forms. The plain form (`own` false) is elementary
torch arithmetic in 32 bits, rounded once at the end. The framework's form
(`own` true) makes the calls a user makes of `weight_only_int4_gb300`. Both
take the same state.

Formulas (blocks are 32 consecutive elements along the contracted axis):

    quantise   s = max(floor(log2(max |v|)) - 2, -127),  c = E2M1(v * 2^-s),
               nearest-even, magnitudes above 6 become 6; value = c * 2^s
    linear     y = q(x) . W^T, x quantised row by row, W already quantised
    moe        p = softmax(x . R^T); the k largest (ties to the lower index),
               divided by their sum where `renorm`;
               y = sum_e p_e . ((silu(x W1_e) * (x W3_e)) W2_e)

Layouts: an int32 word holds eight consecutive codes, the first in its lowest
four bits. Codes along rows: [M, K/8], scale bytes in tiles of 128 rows x 4
blocks, [ceil(M/128), ceil(K/128), 32, 4, 4] = [row tile, block tile, row % 32,
row // 32 % 4, block % 4]. Codes along columns: [K/8, N], scale bytes [K/32, N].
"""
import math

import numpy as np
import torch

own = False

BF16, F16, F32 = "bf16", "f16", "f32"
DTYPES = {BF16: torch.bfloat16, F16: torch.float16, F32: torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# Largest costs a drawn case may have: elements quantised, multiply-adds of a
# linear layer, expert weights held by a mixture-of-experts layer.
MAX_QUANT = 5376 * 43008
MAX_LINEAR = 2048 * 43008 * 5376
MAX_MOE = 128 * 3 * 2048 * 1024


def listed():
    return [
        # one token's activations before a quantised product: a latency case
        dict(name="quant_rows_1x5376_bf16", op="quant", dim=1, rows=1, cols=5376, dtype=BF16),
        # odd row count and an odd number of blocks, from 32-bit activations
        dict(name="quant_rows_77x2592_f32", op="quant", dim=1, rows=77, cols=2592, dtype=F32),
        # a prefill's activations
        dict(name="quant_rows_2048x5376_bf16", op="quant", dim=1, rows=2048, cols=5376, dtype=BF16),
        # a gate_up weight at load time, into the layout the decode kernels read
        dict(name="quant_cols_5376x43008_bf16", op="quant", dim=0, rows=5376, cols=43008, dtype=BF16),
        # one token through a small layer: a latency case
        dict(name="linear_1x2048x2048_bf16", op="linear", M=1, N=2048, K=2048, dtype=BF16, out=BF16),
        # a decode batch through a qkv-like layer: bound by the weights' bytes
        dict(name="linear_16x16384x5376_bf16", op="linear", M=16, N=16384, K=5376, dtype=BF16, out=BF16),
        # a ragged prefill chunk: no size a multiple of a tile, 32-bit result
        dict(name="linear_300x2600x2080_f16", op="linear", M=300, N=2600, K=2080, dtype=F16, out=F32),
        # a prefill through the gate_up-like layer: bound by the tensor cores
        dict(name="linear_2048x43008x5376_bf16", op="linear", M=2048, N=43008, K=5376, dtype=BF16, out=BF16),
        # one token of a decode step, few experts
        dict(name="moe_1_e32k4_2048x1024", op="moe", T=1, E=32, k=4, H=2048, I=1024, renorm=True),
        # odd everything
        dict(name="moe_7_e9k3_544x352", op="moe", T=7, E=9, k=3, H=544, I=352, renorm=False),
        # a decode batch with wide experts
        dict(name="moe_16_e64k8_4096x1024", op="moe", T=16, E=64, k=8, H=4096, I=1024, renorm=True),
        # the largest batch: nearly every expert is chosen, several tokens each
        dict(name="moe_64_e128k8_2048x1024", op="moe", T=64, E=128, k=8, H=2048, I=1024, renorm=True),
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], uniform over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = max(lo, min(hi, int(round(v / step)) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["quant", "linear", "moe"])
    while True:
        if op == "quant":
            dim = rng.choice([0, 1])
            if dim:
                rows, cols = _log_int(rng, 1, 8192), _log_int(rng, 32, 43008, 32)
            else:
                rows, cols = _log_int(rng, 32, 21504, 32), _log_int(rng, 16, 43008, 16)
            if rows * cols <= MAX_QUANT:
                return dict(op=op, dim=dim, rows=rows, cols=cols, dtype=rng.choice([BF16, F16, F32]))
        elif op == "linear":
            M, N, K = _log_int(rng, 1, 4096), _log_int(rng, 8, 43008, 8), _log_int(rng, 32, 21504, 32)
            if M * N * K <= MAX_LINEAR and N * K <= MAX_QUANT:
                return dict(op=op, M=M, N=N, K=K, dtype=rng.choice([BF16, F16, F32]),
                            out=rng.choice([BF16, F16, F32]))
        else:
            E = _log_int(rng, 4, 128)
            T, k = _log_int(rng, 1, 64), min(E, rng.randint(1, 8))
            H, I = _log_int(rng, 256, 4096, 32), _log_int(rng, 128, 2048, 32)
            if 3 * E * H * I <= MAX_MOE and 2 * I != 3072:
                return dict(op=op, T=T, E=E, k=k, H=H, I=I, renorm=rng.choice([True, False]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _words(shape, gen):
    return torch.randint(-2 ** 31, 2 ** 31, shape, dtype=torch.int32, device="cuda", generator=gen)


def _bytes(shape, gen, lo=118, hi=121):
    """Weight scales 2^-9 .. 2^-6: weights of a few hundredths."""
    return torch.randint(lo, hi + 1, shape, dtype=torch.uint8, device="cuda", generator=gen)


def _tile_scales(e):
    """[M, K/32] scale bytes to tiles of 128 rows x 4 blocks, zero outside."""
    M, B = e.shape
    mt, bt = -(-M // 128), -(-B // 4)
    full = torch.zeros((mt * 128, bt * 4), dtype=torch.uint8, device=e.device)
    full[:M, :B] = e
    return full.view(mt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).contiguous()


def _untile_scales(tiles, M, B):
    mt, bt = tiles.shape[:2]
    return tiles.permute(0, 3, 2, 1, 4).reshape(mt * 128, bt * 4)[:M, :B]


def _activations(rows, cols, dtype, gen):
    """N(0, 1) with a few channels ten times as large, as activations have them."""
    x = torch.randn((rows, cols), device="cuda", generator=gen)
    gain = torch.ones(cols, device="cuda")
    gain[torch.randint(0, cols, (max(1, cols // 128),), device="cuda", generator=gen)] = 10.0
    return (x * gain).to(DTYPES[dtype])


def _table(dtype=torch.float32):
    """The values of the sixteen codes."""
    return torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=dtype, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "quant":
        if case["dim"]:
            x = _activations(case["rows"], case["cols"], case["dtype"], gen)
        else:
            x = torch.empty((case["rows"], case["cols"]), dtype=DTYPES[case["dtype"]], device="cuda")
            x.normal_(0.0, 0.02, generator=gen)
        return dict(case=case, x=x)
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(case=case, x=_activations(M, K, case["dtype"], gen), table=_table(), w=_words((N, K // 8), gen),
                    e=_tile_scales(_bytes((N, K // 32), gen)))
    T, E, H, I = case["T"], case["E"], case["H"], case["I"]
    x = _activations(T, H, BF16, gen)
    router = (torch.randn((E, H), device="cuda", generator=gen) / math.sqrt(H)).to(torch.bfloat16)
    return dict(case=case, x=x, router=router, table=_table(),
                w13=_words((E, H // 8, 2 * I), gen), e13=_bytes((E, H // 32, 2 * I), gen),
                w2=_words((E, I // 8, H), gen), e2=_bytes((E, I // 32, H), gen))


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _power(s):
    """FP32 2^s for whole s in [-127, 127], exactly (exp2 and pow need not be):
    the exponent field, or the subnormal 2^-127."""
    return torch.where(s < -126, 2.0 ** -127, ((s + 127) << 23).view(torch.float32))


def _quantised_values(x):
    """FP32 values of x quantised in blocks of 32 along its last axis."""
    v = x.float().reshape(*x.shape[:-1], -1, 32)
    amax = v.abs().amax(dim=-1, keepdim=True)
    s = (torch.frexp(amax).exponent - 3).clamp(min=-127)
    a = (v * _power(-s)).abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    c = torch.clamp(torch.round(a / step) * step, max=6.0)
    return (torch.copysign(c, v) * _power(s)).reshape(x.shape)


def _nibbles(words, dim):
    """Codes 0..15 of packed words, the eight of a word along `dim`."""
    sh = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    shape = list(words.shape)
    shape[dim] *= 8
    if dim == words.dim() - 1:
        return ((words.unsqueeze(-1) >> sh) & 15).reshape(shape)
    return ((words.unsqueeze(dim + 1) >> sh.view(8, 1)) & 15).reshape(shape)


def _column_weights(words, e, table):
    """FP32 [..., K, N] of codes [..., K/8, N] and scale bytes [..., K/32, N]."""
    dim = words.dim() - 2
    w = table[_nibbles(words, dim)]
    s = _power(e.int() - 127)
    return (w.reshape(*e.shape[:-1], 32, e.shape[-1]) * s.unsqueeze(-2)).reshape(w.shape)


def _row_weights(words, tiles, table):
    """FP32 [N, K] of codes [N, K/8] and tiled scale bytes."""
    n, blocks = words.shape[0], words.shape[1] // 4
    s = _power(_untile_scales(tiles, n, blocks).int() - 127)
    return (table[_nibbles(words, 1)].reshape(n, blocks, 32) * s.unsqueeze(-1)).reshape(n, blocks * 32)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _route(x, router, k, renorm):
    """Indices and weights [T, k] of the chosen experts, largest first."""
    logits = x @ router.T
    p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    p = p / p.sum(dim=1, keepdim=True)
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    chosen = torch.gather(p, 1, order)
    if renorm:
        chosen = chosen / chosen.sum(dim=1, keepdim=True)
    return order, chosen


def _plain_moe(st):
    case = st["case"]
    T, E, k, I = case["T"], case["E"], case["k"], case["I"]
    x, table = st["x"].float(), st["table"]
    idx, p = _route(x, st["router"].float(), k, case["renorm"])
    if T * k <= E:
        # few rows: one matrix-vector product for each chosen expert
        ids = idx.reshape(-1)
        rows = x.repeat_interleave(k, dim=0).unsqueeze(1)
        gu = torch.bmm(rows, _column_weights(st["w13"][ids], st["e13"][ids], table))
        h = _silu(gu[..., :I]) * gu[..., I:]
        out = torch.bmm(h, _column_weights(st["w2"][ids], st["e2"][ids], table)).reshape(T, k, -1)
        return (out * p.unsqueeze(-1)).sum(dim=1).to(torch.bfloat16)
    gate = torch.zeros((T, E), device=x.device).scatter_(1, idx, p)
    y = torch.zeros_like(x)
    for e in range(E):
        gu = x @ _column_weights(st["w13"][e], st["e13"][e], table)
        h = _silu(gu[:, :I]) * gu[:, I:]
        y += gate[:, e:e + 1] * (h @ _column_weights(st["w2"][e], st["e2"][e], table))
    return y.to(torch.bfloat16)


def run(state):
    case = state["case"]
    if own:
        return _run_own(state)
    if case["op"] == "quant":
        x = state["x"]
        if case["dim"]:
            return _quantised_values(x).to(torch.bfloat16)
        return _quantised_values(x.T.contiguous()).T.contiguous().to(torch.bfloat16)
    if case["op"] == "linear":
        w = _row_weights(state["w"], state["e"], state["table"])
        return (_quantised_values(state["x"]) @ w.T).to(DTYPES[case["out"]])
    return _plain_moe(state)


def _run_own(state):
    import weight_only_int4_gb300 as w4
    case = state["case"]
    if case["op"] == "quant":
        # the codes and scales, read back as the values they stand for
        codes, e = w4.mxfp4_quantize(state["x"], case["dim"])
        return w4.mxfp4_dequant_rows(codes, e) if case["dim"] else w4.mxfp4_dequant(codes, e)
    if case["op"] == "linear":
        a, ae = w4.mxfp4_quantize(state["x"], 1)
        return w4.mxfp4_matmul(a, ae, state["w"], state["e"], out_dtype=DTYPES[case["out"]])
    return w4.mxfp4_moe(state["x"], state["router"], state["w13"], state["e13"], state["w2"], state["e2"],
                        case["k"], renormalize=case["renorm"])


# ---------------------------------------------------------------------------
# bytes and operations of one pass
# ---------------------------------------------------------------------------
def work(case):
    size = {BF16: 2, F16: 2, F32: 4}
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        # x in; codes, scales and the values out
        return {"bytes": n * size[case["dtype"]] + n // 2 + n // 32 + 2 * n, "flops": 2 * n}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size[case["dtype"]] + N * K // 2 + N * K // 32 + M * N * size[case["out"]],
                "flops": 2 * M * N * K}
    T, E, k, H, I = case["T"], case["E"], case["k"], case["H"], case["I"]
    # experts that at least one token chooses, where all are equally likely
    active = E * (1.0 - (1.0 - k / E) ** T)
    weights = 3 * H * I
    return {"bytes": int(active * weights * (1 / 2 + 1 / 32)) + E * H * 2 + 2 * T * H * 2,
            "flops": 2 * T * k * weights + 2 * T * E * H}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_power(s):
    table = torch.from_numpy(np.ldexp(1.0, np.arange(-160, 161))).to(s.device)
    return table[s.long() + 160]


def _exact_quantised(x):
    """FP64 values of the quantised blocks: the nearest magnitude by comparing
    with the midpoints, ties to the code whose lowest bit is zero."""
    v = x.double().reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    amax = v.abs().max(dim=-1, keepdim=True).values
    bounds = torch.from_numpy(np.ldexp(1.0, np.arange(-126, 128))).to(x.device)
    # 2^(s + 2) <= amax < 2^(s + 3), found among the powers of two themselves
    s = torch.searchsorted(bounds, amax.contiguous(), right=True) - 127 - 2
    scale = _exact_power(torch.clamp(s, min=-127))
    a = v.abs() / scale
    code = torch.zeros_like(a)
    for c, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= mid) if c % 2 else (a > mid)
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)[code.long()]
    return (torch.sign(v) * mags * scale).reshape(x.shape)


def _exact_columns(words, e):
    """FP64 [K, N] of one matrix of codes [K/8, N] and bytes [K/32, N]."""
    table = _table(torch.float64)
    out = torch.empty((words.shape[0], 8, words.shape[1]), dtype=torch.float64, device=words.device)
    for j in range(8):
        out[:, j] = table[((words >> (4 * j)) & 15).long()]
    out = out.reshape(-1, words.shape[1])
    scale = _exact_power(e.int() - 127)
    return out * scale.repeat_interleave(32, dim=0)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quant":
        if case["dim"]:
            return _exact_quantised(st["x"])
        rows = []
        for c in range(0, case["cols"], 4096):
            rows.append(_exact_quantised(st["x"][:, c:c + 4096].T.contiguous()).T)
        return torch.cat(rows, dim=1).contiguous()
    if case["op"] == "linear":
        N, B = case["N"], case["K"] // 32
        x = _exact_quantised(st["x"])
        y = torch.empty((case["M"], N), dtype=torch.float64, device="cuda")
        e = _untile_scales(st["e"], N, B)
        for n in range(0, N, 4096):
            w = _exact_columns(st["w"][n:n + 4096].T.contiguous(), e[n:n + 4096].T.contiguous())
            y[:, n:n + 4096] = x @ w
        return y
    k, I = case["k"], case["I"]
    x = st["x"].double()
    logits = x @ st["router"].double().T
    order = torch.argsort(logits, dim=1, descending=True, stable=True)[:, :k].cpu().numpy()
    prob = torch.softmax(logits, dim=1).cpu().numpy()
    y = torch.zeros_like(x)
    for e in np.unique(order):
        tokens, _ = np.nonzero(order == e)
        t = torch.from_numpy(tokens).cuda()
        w = prob[tokens, e]
        if case["renorm"]:
            w = w / np.take_along_axis(prob[tokens], order[tokens], axis=1).sum(axis=1)
        gu = x[t] @ _exact_columns(st["w13"][int(e)], st["e13"][int(e)])
        g, u = gu[:, :I], gu[:, I:]
        h = g * torch.sigmoid(g) * u
        y[t] += torch.from_numpy(w).cuda().unsqueeze(1) * (h @ _exact_columns(st["w2"][int(e)], st["e2"][int(e)]))
    return y
