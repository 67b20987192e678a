"""The Newton-Schulz kernel hands tiles from warp to warp and from SM to SM through counters.  What
a counter guards is seen complete: under memory traffic from another stream, which moves the
hand-offs apart, every call still gives the bits of a quiet one."""
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


# split sums handed from pair to pair; old values and diagonals of tiles that other
# pairs wrote; many tiles per pair
@pytest.mark.parametrize("batch,m,n", [(1, 1280, 16384), (1, 1700, 2300), (16, 896, 640), (60, 300, 320)])
def test_every_call_gives_the_bits_of_a_quiet_one(batch, m, n):
    g = torch.randn(batch, m, n, generator=torch.Generator().manual_seed(m)).cuda()
    want = fq.fp8q_newton_schulz(g)
    src, dst = torch.ones(2, 1 << 26, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        with torch.cuda.stream(side):
            for _ in range(4):
                dst.copy_(src)
        got.append(fq.fp8q_newton_schulz(g))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for x in got)
