"""The diagonals of A and B stay FP32 in the Newton-Schulz kernel.

The bound comes from the iteration itself: in 64 bits, with only the kernel's FP16 roundings (X, and A
and B beside their diagonals), and once more with the diagonals rounded too.  72 x 3303 with a
decaying spectrum: 6.1e-4 and 1.5e-3 to 1.8e-3 off the exact iteration.  The kernel has to be below the
geometric mean of the two, which rounded diagonals exceed by a factor of 1.6 to 1.7 and the kernel's
own roundings undercut by the same factor (FP32 sums add 2^-24 sqrt(3303) = 3e-6).
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu
a, b, c = 3.4445, -4.7750, 2.0315


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def gradient(m, n, seed):
    g = torch.Generator().manual_seed(seed)
    r = max(1, min(m, n) // 8)
    low = (torch.randn(m, r, generator=g) * torch.arange(1, r + 1).rsqrt()) @ torch.randn(r, n, generator=g)
    return (low / low.square().mean().sqrt() + torch.randn(m, n, generator=g)) * 1e-4


def half(t):
    return (t * 256).half().double() / 256


def iterate(g, rounded, fp32_diagonals=True):
    """Five steps in 64 bits; `rounded`: with FP16 operands."""
    def split(A):
        if not (rounded and fp32_diagonals):
            return (half(A) if rounded else A), torch.zeros(A.shape[0], dtype=torch.float64)
        d = A.diagonal().float().double()
        return half(A - torch.diag(A.diagonal())), d

    x = g.double()
    x = x / (x.norm() + 1e-7)
    x = half(x) if rounded else x
    for step in range(5):
        O, d = split(x @ x.T)
        P = b * O + c * (O @ O + d[:, None] * O + O * d) + torch.diag(b * d + c * d * d)
        O, d = split(P)
        x = (a + d)[:, None] * x + O @ x
        if rounded and step < 4:
            x = half(x)
    return x


@pytest.mark.parametrize("seed", [0, 1, 2])
@pytest.mark.parametrize("tall", [False, True])
def test_diagonals_are_not_rounded(seed, tall):
    g = gradient(72, 3303, seed)
    exact = iterate(g, rounded=False)

    def off(x):
        return float((x - exact).norm() / exact.norm())

    kept, lost = off(iterate(g, True)), off(iterate(g, True, fp32_diagonals=False))
    assert lost > 2 * kept
    x = fq.fp8q_newton_schulz(g.t().contiguous().cuda() if tall else g.cuda(), out_dtype=fq.FP8Q_OUT_FP32)
    x = x.double().cpu()
    assert off(x.t() if tall else x) < (kept * lost) ** 0.5
