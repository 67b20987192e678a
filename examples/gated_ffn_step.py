"""Training and serving of one gated feed-forward block with FP8 operands.

A block y = (silu(x Wg^T) * (x Wu^T)) Wd^T learns a random block of its own shape:

- forward: x and the weights are quantised, both projections, the activation and the product are one
  call, whose FP8 result is the operand of the down projection;
- backward: one call turns the gradient of h into the FP8 operands of Dgrad and of both Wgrads, and
  the weight gradients accumulate in FP32;
- update: the gradients are orthogonalised by Newton-Schulz steps (momentum, then the update, as the
  Muon optimiser does), gate and up projection as a batch of two;
- serving: the trained weights, quantised once, answer single tokens.

    python examples/gated_ffn_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_amax_gb300 as fq  # noqa: E402


class GatedFFN:
    """BF16 weights Wg, Wu stacked [2F][D] and Wd [D][F], FP8 products, FP32 gradients."""

    def __init__(self, D, F, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.D, self.F = D, F
        self.w = (torch.randn(2 * F, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
        self.wd = (torch.randn(D, F, generator=g, device="cuda") / F ** 0.5).bfloat16()
        self.dw = torch.zeros(2 * F, D, device="cuda")
        self.dwd = torch.zeros(D, F, device="cuda")
        self.quantise()

    def quantise(self):
        """FP8 codes of the weights and, for Dgrad, of their transposes."""
        self.qw, self.sw, self.qwT = fq.fp8q_quant_weight(self.w, with_transpose=True)
        self.qwd, self.swd, self.qwdT = fq.fp8q_quant_weight(self.wd, with_transpose=True)

    def forward(self, x, train=False):
        self.qx, self.sx = fq.fp8q_quant_act(x)
        r = fq.fp8q_gemm_swiglu(self.qx, self.sx, self.qw, self.sw, with_h=False, with_gu=train,
                                with_codes=True)
        self.gu = r.gu
        return fq.fp8q_gemm(r.q, r.s, self.qwd, self.swd)

    def backward(self, dy):
        """Adds to dw and dwd (FP32) and returns dx."""
        qdyT, sdyT, qdy, sdy = fq.fp8q_quant_act_T(dy, with_rows=True)
        dh = fq.fp8q_gemm(qdy, sdy, self.qwdT, self.swd, bscale_kind=fq.FP8Q_BSCALE_BLOCK_T)
        g = fq.fp8q_swiglu_bwd(dh, self.gu)
        fq.fp8q_gemm_accumulate(qdyT, sdyT, g.hT, g.shT, self.dwd, bscale_kind=fq.FP8Q_BSCALE_ROW)
        qxT, sxT = fq.fp8q_requant_act_T(self.qx, self.sx)
        fq.fp8q_gemm_accumulate(g.qT, g.sT, qxT, sxT, self.dw, bscale_kind=fq.FP8Q_BSCALE_ROW)
        return fq.fp8q_gemm(g.q, g.s, self.qwT, self.sw, bscale_kind=fq.FP8Q_BSCALE_BLOCK_T)

    def update(self, lr, momentum=0.9):
        """w -= lr * orthogonalised momentum; the running sums keep `momentum` of themselves."""
        for w, dw in ((self.w.view(2, self.F, self.D), self.dw.view(2, self.F, self.D)),
                      (self.wd, self.dwd)):
            o = fq.fp8q_newton_schulz(dw, out_dtype=fq.FP8Q_OUT_FP32)
            w.copy_((w.float() - lr * o).bfloat16())
            dw.mul_(momentum)
        self.quantise()


def main(D=512, F=1024, T=2048, steps=30, lr=0.02, seed=0):
    teacher, block = GatedFFN(D, F, seed + 1), GatedFFN(D, F, seed + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for step in range(steps):
        x = torch.randn(T, D, generator=g, device="cuda").bfloat16()
        want = teacher.forward(x).float()
        diff = block.forward(x, train=True).float() - want
        losses.append(float(diff.square().mean() / want.square().mean()))
        dx = block.backward((diff / T).bfloat16())
        block.update(lr * (1 - step / steps))
        if step % 5 == 0 or step + 1 == steps:
            print(f"step {step:3d}  relative squared error {losses[-1]:.4f}  |dx| {float(dx.float().norm()):.3e}")
    # single tokens: the same rows, one at a time and together
    x = torch.randn(4, D, generator=g, device="cuda").bfloat16()
    together = block.forward(x)
    single = torch.cat([block.forward(x[i:i + 1]) for i in range(4)])
    apart = float((together.float() - single.float()).norm() / together.float().norm())
    print(f"four tokens together and one by one: {apart:.1e} apart")
    status = fq.fp8q_sync_status()
    if status:
        raise RuntimeError(f"device status {status}: {fq.status_string(status)}")
    return losses, apart


if __name__ == "__main__":
    main()
