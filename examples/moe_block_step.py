"""Training of one block of a mixture of experts: norm, router, experts, optimiser.

A pre-norm block out = x + res + sum_j weight_j * expert_j(norm(x + res)) learns a random block of its own
shape:

- forward: one call adds the residual, normalises and leaves the FP8 operand of the experts; the router's call
  turns the logits into choices, weights, the balance loss, and the order and offsets that the experts' grouped
  products take;
- backward: the experts' Dgrad in FP8, the router's and the norm's backward passes; the norm's adds the residual
  stream's own gradient;
- update: one AdamW call for the experts' FP32 master weights, with moments in 8 bits and BF16 copies that are
  quantised again, and one for the norm and the router.

    python examples/moe_block_step.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_fine_grained_amax_gb300 as fq  # noqa: E402


class Moments:
    """What AdamW keeps of a list of parameters: FP32, or 8 bits with a scale per 128 values."""

    def __init__(self, params, codes):
        dtype = torch.uint8 if codes else torch.float32
        self.m, self.v = ([torch.zeros_like(p, dtype=dtype) for p in params] for _ in range(2))
        self.ms, self.vs = ([p.new_zeros((p.numel() + 127) // 128) for p in params] if codes else None
                            for _ in range(2))

    def step(self, params, grads, copies=None, **kw):
        fq.fp8q_adamw(params, grads, self.m, self.v, m_scales=self.ms, v_scales=self.vs, copies=copies, **kw)


class MoEBlock:
    """E experts of D -> F -> D, k of them per token.  FP32 masters; BF16 copies and FP8 codes of the experts."""

    def __init__(self, D, F, E, k, seed, balance=1e-2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        randn = lambda *s, scale: torch.randn(*s, generator=g, device="cuda") * scale  # noqa: E731
        self.D, self.F, self.E, self.k, self.balance = D, F, E, k, balance
        self.norm = torch.ones(D, device="cuda")
        self.router = randn(E, D, scale=D ** -0.5)
        self.w = randn(E, 2 * F, D, scale=D ** -0.5)
        self.wd = randn(E, D, F, scale=F ** -0.5)
        self.copies = [self.w.bfloat16(), self.wd.bfloat16()]
        self.small, self.large = Moments([self.norm, self.router], False), Moments([self.w, self.wd], True)
        self.steps = 0
        self.quantise()

    def quantise(self):
        """FP8 codes of the experts' weights and of their transposes."""
        def stack(w):
            q, s, qT = zip(*(fq.fp8q_quant_weight(e, with_transpose=True) for e in w))
            s = torch.stack(s)
            return torch.stack(q), s, torch.stack(qT), s.mT.contiguous()
        self.qw, self.sw, self.qwT, self.swT = stack(self.copies[0])
        self.qwd, self.swd, self.qwdT, self.swdT = stack(self.copies[1])

    def forward(self, x, res, valid=None, closed=None):
        """x (BF16, e.g. an attention's result) and the residual stream, [T][D] -> the block's contribution in
        FP32, the new stream and the balance loss.  valid (bool [T], optional) is False for padding, closed (bool
        [T][E], optional) True where a token may not take an expert: what takes no expert contributes nothing."""
        n = self.n = fq.fp8q_rmsnorm(x, self.norm, residual=res, with_y=True, with_rstd=True)
        self.logits = n.y.float() @ self.router.t()
        if closed is not None:
            self.logits = self.logits.masked_fill(closed, float("-inf"))
        self.valid = valid
        r = self.r = fq.fp8q_route(self.logits, self.k, valid=valid)
        self.rows = r.order // self.k  # the token of each sorted row (any token behind the last choice)
        # a choice that is none (slot -1) has no row: rows behind the last choice are not written by the products,
        # so what is gathered there is replaced, not multiplied by a weight of zero
        self.none = (r.slot < 0)[..., None]
        g = fq.fp8q_grouped_gemm_swiglu(n.q[self.rows], n.s[:, self.rows].contiguous(), self.qw, self.sw, r.offs,
                                        with_h=True, with_gu=True, with_codes=True)
        self.h, self.gu = g.h, g.gu
        y = fq.fp8q_grouped_gemm(g.q, g.s, self.qwd, self.swd, r.offs)
        self.y = y[r.slot].float().masked_fill(self.none, 0.0)  # [T][k][D]
        return (self.y * r.weight[..., None]).sum(1), n.r, r.loss

    def backward(self, dout):
        """dout (FP32 [T][D]): the gradient of the contribution, and of the stream, which the block's result
        adds up.  Leaves the weights' gradients and returns that of x (and of res)."""
        n, r, T = self.n, self.r, dout.shape[0]
        # one row more than choices: -1 is that one
        dy = torch.empty(T * self.k + 1, self.D, dtype=torch.bfloat16, device="cuda")
        dy[r.slot.reshape(-1)] = (dout[:, None] * r.weight[..., None]).bfloat16().reshape(-1, self.D)
        dy = dy[:-1]
        q, s = fq.fp8q_quant_act(dy)
        dh = fq.fp8q_grouped_gemm(q, s, self.qwdT, self.swdT, r.offs)
        d = fq.fp8q_swiglu_bwd(dh, self.gu, with_d=True, with_rows=True, with_cols=False, with_h=False)
        dx = fq.fp8q_grouped_gemm(d.q, d.s, self.qwT, self.swT, r.offs)
        # the experts' weight gradients, segment by segment
        self.dw, self.dwd = torch.zeros_like(self.w), torch.zeros_like(self.wd)
        x, ends = n.y[self.rows], r.offs.tolist()
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            self.dw[e] = d.d[lo:hi].t() @ x[lo:hi]
            self.dwd[e] = dy[lo:hi].t() @ self.h[lo:hi]
        dweight = (self.y * dout[:, None]).sum(-1)
        dlogits = fq.fp8q_route_bwd(self.logits, r.idx, r.counts, r.tokens, dweight=dweight,
                                    dloss=torch.full((1,), self.balance, device="cuda"), valid=self.valid)
        self.drouter = dlogits.t() @ n.y.float()
        dnorm = dx[r.slot].float().masked_fill(self.none, 0.0).sum(1) + dlogits @ self.router
        g = fq.fp8q_rmsnorm_bwd(dnorm, n.r, n.rstd, self.norm, dres=dout, out_dtype=fq.FP8Q_OUT_FP32)
        self.dnorm = g.dw
        return g.dx

    def update(self, lr):
        self.steps += 1
        kw = dict(step=self.steps, lr=lr, betas=(0.9, 0.95))
        self.small.step([self.norm, self.router], [self.dnorm, self.drouter], **kw)
        self.large.step([self.w, self.wd], [self.dw, self.dwd], self.copies, weight_decay=0.1, **kw)
        self.quantise()


def main(D=256, F=512, E=8, k=2, T=1024, steps=30, lr=3e-3, seed=0):
    teacher, block = MoEBlock(D, F, E, k, seed + 1), MoEBlock(D, F, E, k, seed + 2)
    g = torch.Generator(device="cuda").manual_seed(seed)
    losses = []
    for step in range(steps):
        x, res = (torch.randn(T, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        want = teacher.forward(x, res)[0]
        out, _, balance = block.forward(x, res)
        diff = out - want
        losses.append(float(diff.square().mean() / want.square().mean()))
        dx = block.backward(diff / T)
        block.update(lr)
        if step % 5 == 0 or step + 1 == steps:
            print(f"step {step:3d}  relative squared error {losses[-1]:.4f}  balance {float(balance):.3f}  "
                  f"|dx| {float(dx.norm()):.3e}")
    status = fq.fp8q_sync_status()
    if status:
        raise RuntimeError(f"device status {status}: {fq.status_string(status)}")
    return losses


if __name__ == "__main__":
    main()
