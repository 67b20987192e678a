"""The smoke check's gated calls reach both kernels, in both scale modes: the few-token kernel takes up
to 64 tokens, and more while blocks of 64 columns times blocks of 64 tokens are at most 128."""
import __graft_entry__ as entry


def test_smoke_reaches_the_few_token_kernel_and_the_tiles():
    few = [M <= 64 or F // 64 * ((M + 63) // 64) <= 128 for M, F, _, _ in entry.SMOKE_GATED]
    calls = {(f, mode, call) for f, (_, _, mode, call) in zip(few, entry.SMOKE_GATED)}
    assert {(True, 0, "fp8q_gemm_swiglu"), (False, 0, "fp8q_gemm_swiglu"),
            (False, 1, "fp8q_gemm_swiglu_pow2")} <= calls
