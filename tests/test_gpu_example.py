"""The example's training loop follows the same loop in plain unquantised arithmetic, and its
single-token path agrees with the batched one.

The loss is the relative squared error of the block against its teacher, about 2 at the start.  E4M3
codes are 2.6 % rms off (a uniform error of half a step, 2^-4 of the value at most); three quantised
factors on each of two blocks put about 2 * 3 * 0.026^2 = 0.4 % of noise into the squared error, and
weights that follow slightly different gradients a few times that: 5 % of the loss.
"""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def plain_losses(w, wd, tw, twd, T, steps, lr, seed):
    """The example's loop in FP32 / 64 bits from the given BF16 weights."""
    F, D = wd.shape[1], wd.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    dw, dwd = torch.zeros(2 * F, D, device="cuda"), torch.zeros(D, F, device="cuda")

    def block(x, w, wd):
        gu = x @ w.float().t()
        h = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
        return gu, h, h @ wd.float().t()

    def orthogonal(m):
        x = m.double()
        tall = x.shape[0] > x.shape[1]
        x = x.t() if tall else x
        x = x / (x.norm() + 1e-7)
        for _ in range(5):
            A = x @ x.t()
            x = 3.4445 * x + (-4.7750 * A + 2.0315 * A @ A) @ x
        return (x.t() if tall else x).float()

    losses = []
    for step in range(steps):
        x = torch.randn(T, D, generator=g, device="cuda").bfloat16().float()
        want = block(x, tw, twd)[2]
        gu, h, y = block(x, w, wd)
        diff = y - want
        losses.append(float(diff.square().mean() / want.square().mean()))
        dy = diff / T
        dwd += dy.t() @ h
        dh, gate, up = dy @ wd.float(), gu[:, :F], gu[:, F:]
        s = torch.sigmoid(gate)
        d = torch.cat([dh * up * s * (1 + gate * (1 - s)), dh * gate * s], 1)
        dw += d.t() @ x
        rate = lr * (1 - step / steps)
        w = (w.float() - rate * torch.cat([orthogonal(dw[:F]), orthogonal(dw[F:])])).bfloat16()
        wd = (wd.float() - rate * orthogonal(dwd)).bfloat16()
        dw *= 0.9
        dwd *= 0.9
    return losses


def test_gated_ffn_step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    spec = importlib.util.spec_from_file_location(
        "gated_ffn_step", os.path.join(ROOT, "examples", "gated_ffn_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    D, F, T, steps, lr, seed = 256, 384, 1024, 12, 0.02, 0
    teacher, block = example.GatedFFN(D, F, seed + 1), example.GatedFFN(D, F, seed + 2)
    plain = plain_losses(block.w, block.wd, teacher.w, teacher.wd, T, steps, lr, seed)
    losses, apart = example.main(D, F, T, steps, lr, seed)
    assert plain[-1] < plain[0]
    for step, (got, want) in enumerate(zip(losses, plain)):
        assert abs(got - want) <= 0.05 * want, (step, got, want)
    # one token or four: the same kernel and the same sums
    assert apart == 0.0
