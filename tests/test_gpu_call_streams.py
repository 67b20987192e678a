"""The memory that a call takes for itself, results and scratch, belongs to the stream that the call
is given, so that no other stream gets it while the call still works in it."""
import numpy as np
import pytest

from fp8_fine_grained_amax_gb300 import synth
from _util import bf16_to_torch, u8

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    B.load_library()
    yield
    assert B.fp8q_sync_status() == 0


def home_of(t):
    """Handle of the stream that a tensor's memory was taken on."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's memory")


class Handle:
    """Anything with a handle does for a stream."""
    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("kind", ["other", "other's handle", "none", "current"])
def test_new_results_belong_to_the_stream_of_the_call(kind):
    current, side = torch.cuda.current_stream(), torch.cuda.Stream()
    assert side.cuda_stream != current.cuda_stream
    stream = {"other": side, "other's handle": Handle(side), "none": None, "current": current}[kind]
    where = (stream or current).cuda_stream
    x = bf16_to_torch(synth.activation(256, 256, seed=91, name="home.X"))
    w = bf16_to_torch(synth.weight(256, 256, seed=92, name="home.W"))
    x32, offs = x.float(), torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    q, s = B.fp8q_quant_act(x)
    qw, sw = B.fp8q_quant_weight(w)
    qw2, sw2 = torch.stack([qw, qw]), torch.stack([sw, sw])
    torch.cuda.synchronize()
    made = [*B.fp8q_quant_act(x, stream=stream),
            *B.fp8q_quant_act_T(x, with_rows=True, stream=stream),
            *B.fp8q_requant_act_T(q, s, stream=stream),
            *B.fp8q_quant_weight(w, with_transpose=True, stream=stream),
            *B.fp8q_quant_tensor(x, stream=stream),
            B.fp8q_cast_e4m3(x32, stream=stream),
            B.fp8q_gemm(q, s, qw, sw, stream=stream),
            B.fp8q_grouped_gemm(q, s, qw2, sw2, offs, stream=stream)]
    assert [home_of(m) for m in made] == [where] * len(made)
    torch.cuda.synchronize()


def test_quant_tensor_scratch_is_not_given_away_while_the_call_runs():
    # the call waits on its stream behind a kernel that sleeps; the current stream
    # meanwhile takes and fills every block of the size that the scratch has
    x = bf16_to_torch(synth.activation(4096, 256, seed=93, name="scratch.X"))
    size = max(4, B.fp8q_quant_tensor_workspace_bytes(4096, 256))
    q0, s0 = B.fp8q_quant_tensor(x)
    side = torch.cuda.Stream()

    def blocks():
        return [torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]

    # both streams keep freed blocks of that size: no allocation below waits for the device
    with torch.cuda.stream(side):
        blocks()
        B.fp8q_quant_tensor(x)
    blocks()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # about 0.2 s
    q, s = B.fp8q_quant_tensor(x, stream=side)
    held = blocks()
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the call was over before the blocks were filled"
    torch.cuda.synchronize()
    assert np.array_equal(u8(q), u8(q0)) and torch.equal(s, s0)
    assert all(bool((t == 0x7F).all()) for t in held)
