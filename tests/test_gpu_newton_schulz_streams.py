"""Newton-Schulz calls on several streams at once, of two priorities, beside other kernels.  The
pairs of one call wait for one another, so a call has to get all of its CTAs whatever else runs; the
waits are bounded, and a call that did not would report it."""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def test_streams_of_two_priorities_beside_other_kernels():
    shapes = [(1500, 2000), (896, 1800), (1000, 1000), (2048, 1024)]
    gs = [torch.randn(*s, generator=torch.Generator().manual_seed(i)).cuda() for i, s in enumerate(shapes)]
    a = torch.randint(0, 100, (512, 1024), dtype=torch.uint8).cuda()
    b = torch.randint(0, 100, (2048, 1024), dtype=torch.uint8).cuda()
    sa, sb = torch.rand(8, 512).cuda(), torch.rand(16, 8).cuda()
    want = [fq.fp8q_newton_schulz(g) for g in gs]
    gated, few = fq.fp8q_gemm_swiglu(a, sa, b, sb).h, fq.fp8q_gemm_swiglu(a[:9], sa[:, :9].contiguous(), b, sb).h
    src, dst = torch.ones(2, 1 << 24, device="cuda")
    sa9 = sa[:, :9].contiguous()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(priority=p) for p in (0, -1, 0, -1)]
    got, others = [[] for _ in gs], []
    B.fp8q_set_wait_timeout_ns(500_000_000)
    try:
        for _ in range(6):
            for i, s in enumerate(streams):
                with torch.cuda.stream(s):
                    got[i].append(fq.fp8q_newton_schulz(gs[i]))
                    dst.copy_(src)
                    others.append((fq.fp8q_gemm_swiglu(a, sa, b, sb).h, gated))
                    others.append((fq.fp8q_gemm_swiglu(a[:9], sa9, b, sb).h, few))
        torch.cuda.synchronize()
    finally:
        B.fp8q_set_wait_timeout_ns(0)
    assert B.fp8q_sync_status() == 0
    for i, w in enumerate(want):
        assert all(torch.equal(x, w) for x in got[i])
    assert all(torch.equal(x, w) for x, w in others)
