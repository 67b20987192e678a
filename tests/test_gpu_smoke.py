"""The smoke check of the gated calls fails when a result is wrong or no number at all."""
import pytest
import torch

import __graft_entry__ as entry

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    entry.build()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


class Spoilt:
    """The binding, but one call's result has something put in the place of one value."""

    def __init__(self, call, field, value):
        self._call, self._field, self._value = call, field, value

    def __getattr__(self, name):
        f = getattr(B, name)
        if name != self._call:
            return f

        def spoil(*args, **kw):
            r = f(*args, **kw)
            t = (getattr(r, self._field) if self._field else r).clone()
            t[-1, -1] = self._value
            return r._replace(**{self._field: t}) if self._field else t
        return spoil


def test_the_calls_as_they_are_pass():
    assert 0.0 < entry._smoke_gated(B) <= 1.0


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e6])
@pytest.mark.parametrize("call,field", [("fp8q_gemm_swiglu", "h"), ("fp8q_gemm_swiglu", "gu"),
                                        ("fp8q_gemm_swiglu_pow2", "h"), ("fp8q_gemm_swiglu", "s"),
                                        ("fp8q_swiglu_bwd", "d"), ("fp8q_swiglu_bwd", "sT"),
                                        ("fp8q_newton_schulz", None)])
def test_a_wrong_value_fails(call, field, value):
    with pytest.raises(AssertionError):
        entry._smoke_gated(Spoilt(call, field, value))
