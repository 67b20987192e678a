"""What the compiled marshalling of the gated feed-forward and Newton-Schulz calls does with its
arguments, with the caller's streams, and with the interpreter."""
import threading
import time

import numpy as np
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


def gated_operands(M=5, F=128, K=256):
    g = torch.Generator().manual_seed(3)
    a = torch.randn(M, K, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
    b = torch.randn(2 * F, K, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)
    return a.cuda(), torch.ones(K // 128, M).cuda(), b.cuda(), torch.ones(2 * F // 128, K // 128).cuda()


# ------------------------------------------------------------------ arguments
@pytest.mark.parametrize("yes,no", [(True, False), (1, 0), (np.bool_(True), np.bool_(False)), ("y", "")])
def test_flags_are_taken_by_their_truth(yes, no):
    r = fq.fp8q_gemm_swiglu(*gated_operands(), with_h=no, with_gu=yes, with_codes=yes)
    assert [t is not None for t in r] == [False, True, True, True]
    r = fq.fp8q_gemm_swiglu(*gated_operands(), with_h=yes, with_gu=no, with_codes=no)
    assert [t is not None for t in r] == [True, False, False, False]
    dh, gu = torch.ones(128, 128).bfloat16().cuda(), torch.ones(128, 256).bfloat16().cuda()
    r = fq.fp8q_swiglu_bwd(dh, gu, with_d=yes, with_rows=no, with_cols=no, with_h=yes)
    assert [t is not None for t in r] == [True, False, False, False, False, True, True]
    r = fq.fp8q_swiglu_bwd(dh, gu, with_d=no, with_rows=yes, with_cols=yes, with_h=no)
    assert [t is not None for t in r] == [False, True, True, True, True, False, False]


def test_a_flag_without_truth_raises():
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(*gated_operands(), with_gu=np.ones(2))


@pytest.mark.parametrize("far", [1 << 32, -(1 << 32), 1 << 80])
def test_numbers_past_an_int_are_refused(far):
    # the low 32 bits alone would be a valid mode, count or type
    a, sa, b, sb = gated_operands()
    dh, gu = torch.ones(128, 128).bfloat16().cuda(), torch.ones(128, 256).bfloat16().cuda()
    g = torch.ones(8, 16).cuda()
    for call in (lambda: fq.fp8q_gemm_swiglu(a, sa, b, sb, scale_mode=far),
                 lambda: fq.fp8q_swiglu_bwd(dh, gu, scale_mode=far),
                 lambda: fq.fp8q_newton_schulz(g, steps=far + 5),
                 lambda: fq.fp8q_newton_schulz(g, out_dtype=far)):
        with pytest.raises(fq.FP8QError) as err:
            call()
        assert err.value.status == B.FP8Q_ERR_INVALID


def test_out_of_memory_is_torchs_own_error():
    # a workspace of more than the card holds; g and out are views of one matrix
    g = torch.zeros(1, 4096, 4096, dtype=torch.bfloat16, device="cuda").expand(3000, -1, -1)
    need = fq.fp8q_newton_schulz_workspace_bytes(3000, 4096, 4096)
    assert need > torch.cuda.get_device_properties(0).total_memory
    with pytest.raises(torch.OutOfMemoryError):
        fq.fp8q_newton_schulz(g, out=torch.empty_like(g[:1]).expand(3000, -1, -1))
    assert torch.equal(fq.fp8q_newton_schulz(g[0]), torch.zeros_like(g[0]))


def test_every_operand_is_on_the_first_ones_device():
    # with one card, host memory is the only other place
    a, sa, b, sb = gated_operands()
    b3, sb3 = b[None], sb[None]
    offs = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    dh, gu = torch.ones(128, 128).bfloat16().cuda(), torch.ones(128, 256).bfloat16().cuda()
    g = torch.ones(8, 16).cuda()
    ws = torch.empty(fq.fp8q_newton_schulz_workspace_bytes(1, 8, 16), dtype=torch.uint8)
    for call in (lambda: fq.fp8q_gemm_swiglu(a, sa.cpu(), b, sb), lambda: fq.fp8q_gemm_swiglu(a, sa, b.cpu(), sb),
                 lambda: fq.fp8q_gemm_swiglu(a, sa, b, sb.cpu()),
                 lambda: fq.fp8q_gemm_swiglu(a, sa, b, sb, h=torch.empty(5, 128).bfloat16()),
                 lambda: fq.fp8q_grouped_gemm_swiglu(a, sa, b3.cpu(), sb3, offs),
                 lambda: fq.fp8q_grouped_gemm_swiglu(a, sa, b3, sb3.cpu(), offs),
                 lambda: fq.fp8q_grouped_gemm_swiglu(a, sa, b3, sb3, offs.cpu()),
                 lambda: fq.fp8q_swiglu_bwd(dh, gu.cpu()),
                 lambda: fq.fp8q_swiglu_bwd(dh, gu, q=torch.empty(128, 256, dtype=torch.uint8)),
                 lambda: fq.fp8q_newton_schulz(g, out=torch.empty(8, 16).bfloat16()),
                 lambda: fq.fp8q_newton_schulz(g, workspace=ws)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    assert fq.fp8q_grouped_gemm_swiglu(a, sa, b3, sb3, offs).h.shape == (5, 128)


# ------------------------------------------------------------------ streams
def home_of(t):
    """Handle of the stream that a tensor's memory was taken on."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


def other_stream():
    """A stream whose pool the allocator keeps apart from the current one's."""
    s = torch.cuda.Stream()
    assert s.cuda_stream != torch.cuda.current_stream().cuda_stream
    return s


def test_newton_schulz_scratch_is_not_given_away_while_the_call_runs():
    # the call waits on its stream behind a kernel that sleeps; the current stream
    # meanwhile takes and fills every block of the size that the scratch has
    m, n = 300, 700
    g = torch.randn(m, n, generator=torch.Generator().manual_seed(1)).cuda()
    want = fq.fp8q_newton_schulz(g)
    size = fq.fp8q_newton_schulz_workspace_bytes(1, m, n)
    side = other_stream()

    def blocks():
        return [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(8)]

    # both streams keep freed blocks of that size: no allocation below waits for the device
    with torch.cuda.stream(side):
        blocks()
        fq.fp8q_newton_schulz(g)
    blocks()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    got = fq.fp8q_newton_schulz(g, stream=side)
    held = blocks()
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the call was over before the blocks were filled"
    torch.cuda.synchronize()
    assert B.fp8q_sync_status() == 0
    assert torch.equal(got, want)
    assert all(bool((t == 0xFF).all()) for t in held)


def test_new_results_belong_to_the_stream_of_the_call():
    side = other_stream()
    ops = gated_operands(5), gated_operands(150, 1536)
    dh, gu = torch.ones(128, 128).bfloat16().cuda(), torch.ones(128, 256).bfloat16().cuda()
    g = torch.ones(40, 50).cuda()
    torch.cuda.synchronize()
    for stream in (side, None, torch.cuda.current_stream()):
        where = (stream or torch.cuda.current_stream()).cuda_stream
        made = [t for o in ops for t in fq.fp8q_gemm_swiglu(*o, with_gu=True, with_codes=True, stream=stream)]
        made += fq.fp8q_swiglu_bwd(dh, gu, with_d=True, stream=stream)
        made.append(fq.fp8q_newton_schulz(g, stream=stream))
        assert [home_of(t) for t in made] == [where] * len(made)
    with torch.cuda.stream(side):
        assert home_of(fq.fp8q_newton_schulz(g)) == side.cuda_stream
    torch.cuda.synchronize()


def test_a_result_dropped_on_the_current_stream_is_not_reused_before_it_is_read():
    # read late on the current stream, dropped at once; the call's stream then
    # takes blocks of the same size
    side = other_stream()
    ops = gated_operands(64, 512)
    want = fq.fp8q_gemm_swiglu(*ops).h.clone()

    def blocks():
        return [torch.full((64, 512), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(8)]

    with torch.cuda.stream(side):
        blocks()
    torch.cuda.synchronize()
    h = fq.fp8q_gemm_swiglu(*ops, stream=side).h
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    copy = h.clone()
    del h
    with torch.cuda.stream(side):
        held = blocks()
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and len(held) == 8


def test_another_stream_inside_a_capture():
    g = torch.randn(96, 160, generator=torch.Generator().manual_seed(2)).cuda()
    want = fq.fp8q_newton_schulz(g)
    side = other_stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = fq.fp8q_newton_schulz(g, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        got.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


# ------------------------------------------------------------------ interpreter
def test_other_threads_run_while_a_call_waits():
    # behind a kernel that sleeps, launches fill the queue until a call has to
    # wait in the driver; Python threads go on meanwhile
    dh, gu = torch.ones(128, 128).bfloat16().cuda(), torch.ones(128, 256).bfloat16().cuda()
    d = torch.empty(128, 256).bfloat16().cuda()

    def call():
        fq.fp8q_swiglu_bwd(dh, gu, with_rows=False, with_cols=False, with_h=False, d=d)

    call()
    torch.cuda.synchronize()
    stop, gaps = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(1e-3)
            now = time.perf_counter()
            gaps[0] = max(gaps[0], now - last)
            last = now

    t = threading.Thread(target=tick)
    t.start()
    torch.cuda._sleep(2_000_000_000)  # about a second
    held = 0.0
    for _ in range(6000):
        t0 = time.perf_counter()
        call()
        held = max(held, time.perf_counter() - t0)
        if held > 0.2:
            break
    stop.set()
    t.join()
    torch.cuda.synchronize()
    if held < 0.2:
        pytest.skip(f"no call had to wait ({held:.3f} s at most)")
    assert gaps[0] < held / 2, (gaps[0], held)
