"""A transformer's feed-forward block in 8-bit integers, its norms and residual fused.

    n, s = q(norm(r))                       norm before, quantised to int8
    g    = (n W13^T) s t13                  gate and up, one int8 product
    h    = silu(gate) * up
    o    = (q(h) W2^T) s t2                 down
    r'   = r + scale * norm(o) * after      norm after, residual update, and the next block's norm before

Dense weights are quantised once, one scale per output channel. A pass makes five
calls: block_norm, int8_matmul, int8_quantize (after a plain silu), int8_matmul and
block_norm. Run on a GB300 after building the library:

    python examples/int8_block.py [tokens]

It prints the largest difference from the same block computed in FP32 on the
dense copies of the quantised operands.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_gb300 as w4  # noqa: E402


class Int8Block:
    def __init__(self, hidden: int, inner: int, scale: float = 0.5, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(n, k):
            return (torch.randn((n, k), device=device, generator=gen) * k ** -0.5).to(torch.bfloat16)

        def vector():
            return (1.0 + 0.1 * torch.randn(hidden, device=device, generator=gen)).to(torch.bfloat16)

        self.scale = scale
        self.w13 = w4.int8_quantize(weight(2 * inner, hidden))
        self.w2 = w4.int8_quantize(weight(hidden, inner))
        self.before, self.after, self.next = vector(), vector(), vector()

    def __call__(self, r):
        """r float32 [T, hidden] -> (r' float32, the next block's input bfloat16)."""
        _, codes, s = w4.block_norm(r, self.before, quantize=True)
        gate, up = w4.int8_matmul(codes, s, *self.w13).chunk(2, dim=1)
        h = torch.nn.functional.silu(gate) * up
        o = w4.int8_matmul(*w4.int8_quantize(h), *self.w2)
        return w4.block_norm(r, self.next, o, after=self.after, scale=self.scale)

    def dense(self, r):
        """The block in FP32 on the dense copies, rounded and quantised where the block is."""
        def norm(x, w):
            return x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + 1e-6) * w.float()

        def dense(pair):
            return w4.int8_dequant(*pair, out_dtype=torch.float32)

        n = dense(w4.int8_quantize(norm(r, self.before)))
        gate, up = (n @ dense(self.w13).T).to(torch.bfloat16).chunk(2, dim=1)
        h = torch.nn.functional.silu(gate) * up
        o = (dense(w4.int8_quantize(h)) @ dense(self.w2).T).to(torch.bfloat16).float()
        new = r + self.scale * norm(o, self.after)
        return new, norm(new, self.next)


def main(tokens: int = 8) -> float:
    block = Int8Block(hidden=2048, inner=1024)
    r = torch.randn((tokens, 2048), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    got, ref = block(r), block.dense(r)
    if w4.device_status() != w4.OK:
        raise RuntimeError("device status not OK")
    err = max(((g.float() - x).abs().max() / x.abs().max()).item() for g, x in zip(got, ref))
    print(f"{tokens} tokens: max difference {err:.2e} of the largest output")
    return err


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
