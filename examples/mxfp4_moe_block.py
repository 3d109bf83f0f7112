"""A decode step through a quantised block: projection, then mixture of experts.

    a = x + q(x) Wo^T          q(x): the activations quantised to MXFP4 row by row
    y = a + experts(a)

Dense bf16 weights are quantised once: the projection along its rows (one
output feature per row, the operand of the 4-bit product), the experts along K
(the layout the decode kernels read). Each step then makes three calls:
mxfp4_quantize, mxfp4_matmul and mxfp4_moe. Run on a GB300 after building the
library:

    python examples/mxfp4_moe_block.py [tokens]

It prints the largest difference from the same block computed in FP32 on the
dense copies of the quantised weights.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_int4_gb300 as w4  # noqa: E402


class MoeBlock:
    def __init__(self, hidden: int, inner: int, experts: int, top_k: int, seed: int = 0, device="cuda"):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape, fan_in):
            return (torch.randn(shape, device=device, generator=gen) * fan_in ** -0.5).to(torch.bfloat16)

        self.top_k = top_k
        self.router = weight(experts, hidden, fan_in=hidden)
        self.wo = w4.mxfp4_quantize(weight(hidden, hidden, fan_in=hidden), 1)
        self.w13 = w4.mxfp4_quantize(weight(experts, hidden, 2 * inner, fan_in=hidden), 0)
        self.w2 = w4.mxfp4_quantize(weight(experts, inner, hidden, fan_in=inner), 0)

    def __call__(self, x):
        a = x + w4.mxfp4_matmul(*w4.mxfp4_quantize(x, 1), *self.wo)
        return a + w4.mxfp4_moe(a, self.router, *self.w13, *self.w2, self.top_k)

    def dense(self, x):
        """The block in FP32 on the dense copies of the quantised operands, rounded to bf16 where the block
        rounds before the experts are chosen: the choice depends on the last bit."""
        q = w4.mxfp4_dequant_rows(*w4.mxfp4_quantize(x, 1)).float()
        a = (x + (q @ w4.mxfp4_dequant_rows(*self.wo).float().T).to(torch.bfloat16)).float()
        logits = a @ self.router.float().T
        top, index = logits.topk(self.top_k, dim=1)
        p = torch.softmax(top, dim=1)
        out = a.clone()
        for e in index.unique().tolist():
            tokens, slot = torch.nonzero(index == e, as_tuple=True)
            gate, up = (a[tokens] @ w4.mxfp4_dequant(self.w13[0][e], self.w13[1][e]).float()).chunk(2, dim=1)
            h = torch.nn.functional.silu(gate) * up
            out[tokens] += p[tokens, slot, None] * (h @ w4.mxfp4_dequant(self.w2[0][e], self.w2[1][e]).float())
        return out


def main(tokens: int = 8) -> float:
    block = MoeBlock(hidden=2048, inner=1024, experts=16, top_k=4)
    x = torch.randn((tokens, 2048), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x = x.to(torch.bfloat16)
    y, ref = block(x), block.dense(x)
    if w4.device_status() != w4.OK:
        raise RuntimeError("device status not OK")
    err = ((y.float() - ref).abs().max() / ref.abs().max()).item()
    print(f"{tokens} tokens: max difference {err:.2e} of the largest output")
    return err


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
