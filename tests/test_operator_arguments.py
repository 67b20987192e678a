"""Argument checks of the gated feed-forward and Newton-Schulz calls: made on
the host before any device work, so they run without a GPU."""
import pytest

P = 4096  # a non-null, 16-byte aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    from fp8_fine_grained_amax_gb300 import binding
    return binding.load_library()


@pytest.fixture(scope="module")
def B():
    from fp8_fine_grained_amax_gb300 import binding
    return binding


FWD = dict(a=P, lda=256, sa=P, ld_sa=64, b=P, ldb=256, sb=P, ld_sb=2, h=P, ldh=128, gu=P,
           ld_gu=256, q=P, ldq=128, s=P, ld_s=64, mode=0, M=64, F=128, K=256, stream=None)
BWD = dict(dh=P, ld_dh=128, gu=P, ld_gu=256, d=P, ld_d=256, q=P, ldq=256, s=P, ld_s=128, qT=P,
           ldqT=128, sT=P, ld_sT=256, hT=P, ld_hT=128, shT=P, ld_shT=128, T=128, F=128, mode=0,
           stream=None)
NS = dict(g=P, ldg=20, g_stride=200, in_dtype=1, out=P, ldo=20, o_stride=200, out_dtype=0, batch=2,
          m=10, n=20, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, ws=P, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(mode=2), "INVALID"), (dict(M=-1), "SHAPE"), (dict(F=-128), "SHAPE"), (dict(F=64), "SHAPE"),
    (dict(F=200), "SHAPE"), (dict(K=100), "SHAPE"), (dict(K=-128), "SHAPE"),
    (dict(M=1 << 31), "SHAPE"), (dict(F=1 << 30), "SHAPE"), (dict(ld_sa=63), "SHAPE"),
    (dict(lda=240), "SHAPE"), (dict(ldb=128), "SHAPE"), (dict(ld_sb=1), "SHAPE"),
    (dict(ldh=64), "SHAPE"), (dict(ld_gu=128), "SHAPE"), (dict(ldq=64), "SHAPE"),
    (dict(ld_s=63), "SHAPE"), (dict(h=None, gu=None, q=None, s=None), "INVALID"),
    (dict(s=None), "INVALID"), (dict(q=None), "INVALID"), (dict(a=None), "INVALID"),
    (dict(b=None), "INVALID"), (dict(sa=None), "INVALID"), (dict(sb=None), "INVALID"),
    (dict(a=P + 8), "ALIGN"), (dict(b=P + 1), "ALIGN"), (dict(lda=264), "ALIGN"),
    (dict(ldb=257), "ALIGN"), (dict(sa=P + 2), "ALIGN"), (dict(h=P + 2), "ALIGN"),
    (dict(ldh=130), "ALIGN"), (dict(ld_gu=260), "ALIGN"), (dict(q=P + 4), "ALIGN"),
    (dict(ldq=136), "ALIGN"), (dict(s=P + 1), "ALIGN")])
def test_forward_refusals(lib, B, change, status):
    for entry in ("fp8q_gemm_swiglu", "fp8q_gemm_swiglu_pow2"):
        assert getattr(lib, entry)(*{**FWD, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


def grouped(change):
    a = {**FWD, **change}
    a = {k: v for k, v in a.items() if k != "ld_sb"}
    out = {}
    for k, v in a.items():
        if k == "h":
            out["offs"] = change.get("offs", P)
            out["G"] = change.get("G", 4)
        if k not in ("offs", "G"):
            out[k] = v
    return out


@pytest.mark.parametrize("change,status", [
    (dict(G=0), "SHAPE"), (dict(G=1025), "SHAPE"), (dict(offs=None), "INVALID"),
    (dict(offs=P + 1), "ALIGN"), (dict(F=1 << 28, ldh=1 << 28, ld_gu=1 << 29, ldq=1 << 28, G=4), "SHAPE"),
    (dict(K=100), "SHAPE"), (dict(b=None), "INVALID"), (dict(lda=264), "ALIGN")])
def test_grouped_refusals(lib, B, change, status):
    for entry in ("fp8q_grouped_gemm_swiglu", "fp8q_grouped_gemm_swiglu_pow2"):
        assert getattr(lib, entry)(*grouped(change).values()) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(mode=-1), "INVALID"), (dict(T=-1), "SHAPE"), (dict(F=64), "SHAPE"), (dict(T=100), "SHAPE"),
    (dict(T=100, qT=None, sT=None), "SHAPE"), (dict(T=65536 * 128), "SHAPE"),
    (dict(ld_dh=64), "SHAPE"), (dict(ld_gu=128), "SHAPE"), (dict(ld_d=128), "SHAPE"),
    (dict(ldq=128), "SHAPE"), (dict(ld_s=64), "SHAPE"), (dict(ldqT=64), "SHAPE"),
    (dict(ld_sT=128), "SHAPE"), (dict(ld_hT=64), "SHAPE"), (dict(ld_shT=64), "SHAPE"),
    (dict(dh=None), "INVALID"), (dict(gu=None), "INVALID"), (dict(s=None), "INVALID"),
    (dict(sT=None), "INVALID"), (dict(hT=None), "INVALID"),
    (dict(d=None, q=None, s=None, qT=None, sT=None, hT=None, shT=None), "INVALID"),
    (dict(dh=P + 2), "ALIGN"), (dict(ld_dh=132), "ALIGN"), (dict(ld_gu=258), "ALIGN"),
    (dict(ld_d=260), "ALIGN"), (dict(ldq=264), "ALIGN"), (dict(ldqT=136), "ALIGN"),
    (dict(hT=P + 8), "ALIGN"), (dict(shT=P + 2), "ALIGN")])
def test_backward_refusals(lib, B, change, status):
    assert lib.fp8q_swiglu_bwd(*{**BWD, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(in_dtype=2), "INVALID"), (dict(out_dtype=-1), "INVALID"), (dict(steps=0), "INVALID"),
    (dict(eps=-1.0), "INVALID"), (dict(eps=float("nan")), "INVALID"), (dict(m=-1), "SHAPE"),
    (dict(n=(1 << 20) + 1), "SHAPE"), (dict(batch=-1), "SHAPE"), (dict(batch=65536), "SHAPE"),
    (dict(ldg=19), "SHAPE"), (dict(ldo=19), "SHAPE"), (dict(o_stride=199), "SHAPE"),
    (dict(g_stride=-1), "SHAPE"), (dict(g=None), "INVALID"), (dict(out=None), "INVALID"),
    (dict(ws=None), "INVALID"), (dict(ws_bytes=100), "SHAPE"), (dict(g=P + 2), "ALIGN"),
    (dict(out=P + 1), "ALIGN"), (dict(ws=P + 16), "ALIGN")])
def test_newton_schulz_refusals(lib, B, change, status):
    assert lib.fp8q_newton_schulz(*{**NS, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


def test_empty_work_succeeds(lib, B):
    none = dict(a=None, sa=None, b=None, sb=None, h=None, gu=None, q=None, s=None)
    for change in (dict(M=0), dict(F=0)):
        assert lib.fp8q_gemm_swiglu(*{**FWD, **none, **change}.values()) == B.FP8Q_OK
        assert lib.fp8q_grouped_gemm_swiglu_pow2(*grouped({**none, **change}).values()) == B.FP8Q_OK
    assert lib.fp8q_swiglu_bwd(*{**BWD, "T": 0, "dh": None, "gu": None}.values()) == B.FP8Q_OK
    for change in (dict(batch=0), dict(m=0), dict(n=0)):
        assert lib.fp8q_newton_schulz(*{**NS, **change, "g": None, "out": None,
                                        "ws": None}.values()) == B.FP8Q_OK


def test_workspace_size(lib):
    # two copies of X, A and B in FP16, their diagonals, counters and partial
    # sums; at most 76 pairs' FP32 partial tiles of 256 x 256
    f = lib.fp8q_newton_schulz_workspace_bytes
    assert f(1, 2048, 7168) == f(1, 7168, 2048)
    need = 2 * 2048 * 7168 * 2 + 2 * 2048 * 2048 * 2 + 2 * 2048 * 4
    assert need <= f(1, 2048, 7168) <= need + 76 * 256 * 256 * 4 + 32768
    assert f(1, 8, 8) <= 256 * 256 * 4 + 32768
    assert f(-1, 8, 8) == 0 and f(1, 1 << 21, 8) == 0 and f(4096, 1 << 16, 1 << 16) == 0


def test_marshalling_module_loads_and_names_its_calls(lib, B):
    m = B._calls()
    for name in ("swiglu", "swiglu_bwd", "newton_schulz"):
        with pytest.raises(TypeError):
            getattr(m, name)()


def test_binding_refuses_what_is_not_on_a_gpu(lib):
    import torch

    import fp8_fine_grained_amax_gb300 as fq
    a, sa = torch.zeros(4, 256, dtype=torch.uint8), torch.ones(2, 4)
    b, sb = torch.zeros(256, 256, dtype=torch.uint8), torch.ones(2, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_gemm_swiglu(a, sa, b, sb)
    with pytest.raises(TypeError):
        fq.fp8q_gemm_swiglu([1], sa, b, sb)
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_swiglu_bwd(torch.zeros(128, 128).bfloat16(), torch.zeros(128, 256).bfloat16())
    with pytest.raises(ValueError, match="CUDA"):
        fq.fp8q_newton_schulz(torch.zeros(8, 8))
