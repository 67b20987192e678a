"""fp8q_sync_status: every kernel family's failure is reported once, and the call costs little more
than the one copy to the host that it needs."""
import threading
import time

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


def codes(*shape):
    return torch.zeros(*shape, dtype=torch.uint8, device="cuda")


def bad_scales(*shape):
    return torch.full(shape, 0.3, device="cuda")  # no power of two


def few_tokens(stream):
    fq.fp8q_gemm_swiglu_pow2(codes(4, 128), bad_scales(1, 4), codes(256, 128), bad_scales(2, 1), stream=stream)


def pow2_gemm(stream):
    fq.fp8q_gemm_pow2(codes(256, 128), bad_scales(1, 256), codes(256, 128), bad_scales(2, 1), stream=stream)


def timeout(stream):
    fq.fp8q_selftest_wait_timeout(1_000_000, stream=stream)


@pytest.mark.parametrize("other", [False, True])
@pytest.mark.parametrize("fails,status", [([few_tokens], [B.FP8Q_ERR_INVALID]),
                                          ([pow2_gemm], [B.FP8Q_ERR_INVALID]),
                                          ([timeout], [B.FP8Q_ERR_TIMEOUT]),
                                          ([pow2_gemm, timeout, few_tokens], [B.FP8Q_ERR_TIMEOUT])])
def test_a_failure_is_reported_once(fails, status, other):
    stream = torch.cuda.Stream() if other else torch.cuda.current_stream()
    torch.cuda.synchronize()
    for f in fails:
        f(stream)
    torch.cuda.synchronize()
    assert [B.fp8q_sync_status(stream) for _ in range(3)] == status + [0, 0]


def test_threads_take_a_failure_once_between_them():
    streams = [torch.cuda.Stream() for _ in range(8)]
    for _ in range(20):
        pow2_gemm(torch.cuda.current_stream())
        torch.cuda.synchronize()
        got = []
        threads = [threading.Thread(target=lambda s=s: got.append(B.fp8q_sync_status(s))) for s in streams]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert sorted(got) == [0] * 7 + [B.FP8Q_ERR_INVALID]


def test_one_copy_to_the_host():
    # a value read back through torch is one copy and one wait; a copy per status
    # word would take more than four of them
    x = torch.zeros((), device="cuda")

    def least(f):
        best = float("inf")
        for _ in range(20):
            t = time.perf_counter()
            for _ in range(20):
                f()
            best = min(best, (time.perf_counter() - t) / 20)
        return best

    torch.cuda.synchronize()
    one, all_words = least(x.item), least(B.fp8q_sync_status)
    assert all_words < 3 * one, (all_words, one)
