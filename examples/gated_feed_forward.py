"""A gated feed-forward block, y = (act(x Wg^T) * (x Wu^T)) Wd^T, trained and served on quantized operands.

    python examples/gated_feed_forward.py [--tokens 2048] [--hidden 1024] [--ffn 2816] [--steps 5]

Training: the forward products run on NVFP4 operands, the gradients' on MXFP8 (towards the inputs) and on
NVFP4 with the random Hadamard transform and stochastic rounding (towards the weights); both projections,
the activation and the product are one kernel, their backward pass another, and the weight gradients
are clipped to a global norm.  Serving: one token at a time from the same NVFP4 weights.  Sizes: tokens
multiples of 32, hidden and 2 ffn multiples of 512.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_nvfp4_amd as bsq  # noqa: E402

ACT = bsq.ACT_SILU
MX = bsq.FMT_MXFP8 | bsq.FMT_MX_SLAB


class GatedFeedForward:
    def __init__(self, hidden: int, ffn: int, device="cuda:0", seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        normal = lambda r, c: (torch.randn((r, c), generator=g) / c ** 0.5).to(device)   # noqa: E731
        self.w1, self.w2 = normal(2 * ffn, hidden), normal(hidden, ffn)   # [gate; up] and down, fp32 masters
        self.ffn = ffn
        self.signs = ((torch.randint(0, 2, (16,), generator=g) * 2 - 1).to(torch.int8)).to(device)
        self.quantize()

    def quantize(self):
        """The weights' NVFP4 operands: what the forward pass and the serving of tokens read."""
        self.q1, self.q2 = bsq.nvfp4_quantize(self.w1.to(torch.bfloat16)), bsq.nvfp4_quantize(self.w2.to(torch.bfloat16))

    def _w1(self):
        F, q = self.ffn, self.q1
        s = q["s_enc"][:1]
        gate = (q["row_codes"][:F], q["row_scales"][:F], s)
        return gate, (q["row_codes"][F:], q["row_scales"][F:], s)

    def _w2(self):
        return self.q2["row_codes"], self.q2["row_scales"], self.q2["s_enc"][:1]

    def forward(self, x: torch.Tensor, seed: int):
        """y [T, hidden] bf16 and what the backward pass needs."""
        cast = lambda t, stream: bsq.nvfp4_quantize_fprop_wgrad(t, bsq.SR, seed, stream, self.signs)   # noqa: E731
        qx = cast(x, 1)
        gate, up = self._w1()
        h, gate_up = bsq.blockscaled_gated_gemm(bsq.FMT_NVFP4, ACT, qx["row_codes"], qx["row_scales"], qx["s_enc"][:1],
                                                *gate, *up, save_gate_up=True)
        qh = cast(h, 3)
        y = bsq.blockscaled_gemm(bsq.FMT_NVFP4, qh["row_codes"], qh["row_scales"], qh["s_enc"][:1], *self._w2())
        return y, (qx, qh, gate_up)

    def backward(self, dy: torch.Tensor, saved, seed: int):
        """dx [T, hidden] bf16 and the fp32 gradients of w1 and w2."""
        qx, qh, gate_up = saved
        cast = lambda t, stream: bsq.nvfp4_col_mxfp8_row_quantize(t, bsq.SR, seed, stream, self.signs, mx_slab=True)   # noqa: E731
        columns = lambda q: bsq.mxfp8_requantize_nvfp4(   # noqa: E731
            q["row_codes"], q["row_scales"], q["s_enc"][:1], bsq.COL | bsq.MX_SLAB)
        wgrad = lambda a, b: bsq.blockscaled_gemm(   # noqa: E731
            bsq.FMT_NVFP4, a["col_codes"], a["col_scales"], a["s_enc"][1:], b["col_codes"], b["col_scales"],
            b["s_enc"][1:], out_dtype=torch.float32)
        qdy, w2 = cast(dy, 0), columns(self.q2)
        d_gate_up = bsq.blockscaled_gated_gemm_backward(MX, ACT, qdy["mx_row_codes"], qdy["mx_row_scales"], None,
                                                        w2["col_codes"], w2["col_scales"], None, gate_up, out=gate_up)
        qd, w1 = cast(d_gate_up, 2), columns(self.q1)
        dx = bsq.blockscaled_gemm(MX, qd["mx_row_codes"], qd["mx_row_scales"], None, w1["col_codes"], w1["col_scales"],
                                  None)
        return dx, wgrad(qd, qx), wgrad(qdy, qh)

    def step(self, grads, lr: float, max_norm: float) -> torch.Tensor:
        """One clipped step; returns the gradients' norm before clipping."""
        norm = bsq.clip_grad_norm(grads, max_norm)
        for w, g in zip((self.w1, self.w2), grads):
            w.sub_(g, alpha=lr)
        self.quantize()
        return norm

    def token(self, x: torch.Tensor) -> torch.Tensor:
        """y of a few tokens x [m, hidden], not quantized, in two kernels."""
        gate, up = self._w1()
        return bsq.nvfp4_matvec(bsq.nvfp4_gated_matvec(ACT, x, *gate, *up), *self._w2())


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--hidden", type=int, default=1024)
    p.add_argument("--ffn", type=int, default=2816)
    p.add_argument("--steps", type=int, default=5)
    a = p.parse_args()
    block, target = GatedFeedForward(a.hidden, a.ffn), GatedFeedForward(a.hidden, a.ffn, seed=1)
    g = torch.Generator().manual_seed(2)
    for i in range(a.steps):
        x = torch.randn((a.tokens, a.hidden), generator=g).to(torch.bfloat16).to("cuda:0")
        y, saved = block.forward(x, i)
        err = y.float() - target.forward(x, i)[0].float()
        _, *grads = block.backward((err / a.tokens).to(torch.bfloat16), saved, i)
        norm = block.step(grads, lr=1.0, max_norm=1.0)
        print("step %d: loss %.5f, gradient norm %.4f" % (i, float(err.square().mean()), float(norm)))
    y = block.token(x[:1])
    print("one token: y[:4] = %s" % [round(float(v), 4) for v in y[0, :4]])


if __name__ == "__main__":
    main()
