"""Argument checks of the norm, AdamW and router calls: made on the host before any
device work, so they run without a GPU."""
import ctypes

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


NORM = dict(x=P, ldx=256, kx=0, res=P, ld_res=256, kres=1, w=P, kw=1, eps=1e-6, r=P, ld_r=256, y=P, ldy=256, q=P,
            ldq=256, s=P, ld_s=64, rstd=P, mode=0, T=64, C=256, stream=None)
NORM_BWD = dict(dy=P, ld_dy=256, kdy=0, x=P, ldx=256, kx=0, rstd=P, w=P, kw=0, dres=P, ld_dres=256, dx=P, ld_dx=256,
                kd=0, dw=P, accumulate=0, T=64, C=256, ws=P, ws_bytes=1 << 20, stream=None)
ROUTE = dict(l=P, ld=64, kind=1, valid=P, score=0, norm=1, scale=1.0, idx=P, weight=P, counts=P, offs=P, order=P,
             slot=P, tokens=P, loss=P, T=1000, E=64, k=4, ws=P, ws_bytes=1 << 20, stream=None)
ROUTE_BWD = dict(l=P, ld=64, kind=1, valid=P, score=0, norm=1, scale=1.0, idx=P, counts=P, tokens=P, dw=P, dloss=P,
                 d=P, ld_d=64, T=100, E=64, k=4, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(kx=2), "INVALID"), (dict(kres=-1), "INVALID"), (dict(kw=2), "INVALID"), (dict(mode=2), "INVALID"),
    (dict(eps=-1.0), "INVALID"), (dict(eps=float("nan")), "INVALID"), (dict(T=-1), "SHAPE"), (dict(T=1 << 31), "SHAPE"),
    (dict(C=-8), "SHAPE"), (dict(C=12), "SHAPE"), (dict(C=200), "SHAPE"), (dict(C=32776, q=None, s=None), "SHAPE"),
    (dict(ldx=248), "SHAPE"), (dict(ld_res=248), "SHAPE"), (dict(ld_r=248), "SHAPE"), (dict(ldy=248), "SHAPE"),
    (dict(ldq=240), "SHAPE"), (dict(ld_s=63), "SHAPE"), (dict(x=None), "INVALID"), (dict(w=None), "INVALID"),
    (dict(s=None), "INVALID"), (dict(q=None), "INVALID"), (dict(res=None), "INVALID"),
    (dict(r=None, y=None, q=None, s=None, rstd=None), "INVALID"), (dict(x=P + 8), "ALIGN"), (dict(ldx=260), "ALIGN"),
    (dict(res=P + 4), "ALIGN"), (dict(ld_res=258), "ALIGN"), (dict(w=P + 8), "ALIGN"), (dict(r=P + 8), "ALIGN"),
    (dict(y=P + 2), "ALIGN"), (dict(ldy=260), "ALIGN"), (dict(q=P + 8), "ALIGN"), (dict(ldq=264), "ALIGN"),
    (dict(s=P + 2), "ALIGN"), (dict(rstd=P + 1), "ALIGN")])
def test_norm_refusals(lib, B, change, status):
    assert lib.fp8q_rmsnorm(*{**NORM, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(kdy=2), "INVALID"), (dict(kx=-1), "INVALID"), (dict(kw=3), "INVALID"), (dict(kd=2), "INVALID"),
    (dict(T=-1), "SHAPE"), (dict(C=4), "SHAPE"), (dict(C=32776), "SHAPE"), (dict(ld_dy=248), "SHAPE"),
    (dict(ldx=248), "SHAPE"), (dict(ld_dres=248), "SHAPE"), (dict(ld_dx=248), "SHAPE"), (dict(dy=None), "INVALID"),
    (dict(x=None), "INVALID"), (dict(rstd=None), "INVALID"), (dict(w=None), "INVALID"),
    (dict(dx=None), "INVALID"), (dict(dx=None, dres=None, dw=None), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(ws_bytes=100), "SHAPE"), (dict(ws=P + 8), "ALIGN"), (dict(dy=P + 2), "ALIGN"), (dict(ld_dy=260), "ALIGN"),
    (dict(x=P + 2), "ALIGN"), (dict(w=P + 4), "ALIGN"), (dict(rstd=P + 2), "ALIGN"), (dict(dres=P + 8), "ALIGN"),
    (dict(ld_dx=260), "ALIGN"), (dict(dw=P + 2), "ALIGN")])
def test_norm_backward_refusals(lib, B, change, status):
    assert lib.fp8q_rmsnorm_bwd(*{**NORM_BWD, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(kind=2), "INVALID"), (dict(score=2), "INVALID"), (dict(T=-1), "SHAPE"), (dict(T=(1 << 26) + 1), "SHAPE"),
    (dict(E=0), "SHAPE"), (dict(E=1025, ld=1025), "SHAPE"), (dict(k=0), "SHAPE"), (dict(k=65), "SHAPE"),
    (dict(k=33), "SHAPE"), (dict(T=1 << 26, k=32), "SHAPE"), (dict(ld=63), "SHAPE"), (dict(l=None), "INVALID"),
    (dict(idx=None), "INVALID"), (dict(weight=None), "INVALID"), (dict(counts=None), "INVALID"),
    (dict(offs=None), "INVALID"), (dict(order=None), "INVALID"), (dict(slot=None), "INVALID"),
    (dict(tokens=None), "INVALID"), (dict(loss=None), "INVALID"), (dict(ws=None), "INVALID"),
    (dict(ws_bytes=64), "SHAPE"), (dict(ws=P + 8), "ALIGN"), (dict(l=P + 2), "ALIGN"), (dict(idx=P + 2), "ALIGN"),
    (dict(order=P + 1), "ALIGN"), (dict(loss=P + 2), "ALIGN")])
def test_route_refusals(lib, B, change, status):
    assert lib.fp8q_route(*{**ROUTE, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(kind=-1), "INVALID"), (dict(score=-1), "INVALID"), (dict(E=0), "SHAPE"), (dict(k=65), "SHAPE"),
    (dict(ld=63), "SHAPE"), (dict(ld_d=63), "SHAPE"), (dict(l=None), "INVALID"), (dict(d=None), "INVALID"),
    (dict(idx=None), "INVALID"), (dict(counts=None), "INVALID"), (dict(tokens=None), "INVALID"),
    (dict(l=P + 1), "ALIGN"), (dict(d=P + 2), "ALIGN"), (dict(dw=P + 2), "ALIGN"), (dict(dloss=P + 2), "ALIGN")])
def test_route_backward_refusals(lib, B, change, status):
    assert lib.fp8q_route_bwd(*{**ROUTE_BWD, **change}.values()) == getattr(B, "FP8Q_ERR_" + status)


class Entry(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "ms", "vs", "copy")] + [("n", ctypes.c_int64)]


def entries(*changes):
    out = (Entry * len(changes))()
    for i, c in enumerate(changes):
        base = P + i * (1 << 20)
        for k, name in enumerate(("p", "g", "m", "v", "ms", "vs", "copy")):
            setattr(out[i], name, base + k * (1 << 16))
        out[i].n = 1000
        for name, value in c.items():
            setattr(out[i], name, value)
    return out


def adamw(lib, tensors, kp=1, kg=1, state=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, lr_dev=None,
          step_dev=None, scale=None, count=None):
    return lib.fp8q_adamw(tensors and ctypes.addressof(tensors), len(tensors or ()) if count is None else count, kp, kg,
                          state, lr, b1, b2, eps, wd, step, lr_dev, step_dev, scale, None)


@pytest.mark.parametrize("change,status", [
    (dict(kp=2), "INVALID"), (dict(kg=-1), "INVALID"), (dict(state=3), "INVALID"), (dict(state=-1), "INVALID"),
    (dict(b1=1.0), "INVALID"), (dict(b1=-0.1), "INVALID"), (dict(b2=1.0), "INVALID"), (dict(eps=-1e-8), "INVALID"),
    (dict(eps=float("nan")), "INVALID"), (dict(lr=float("inf")), "INVALID"), (dict(wd=float("nan")), "INVALID"),
    (dict(step=0), "INVALID"), (dict(count=-1), "SHAPE"), (dict(lr_dev=P + 2), "ALIGN"), (dict(step_dev=P + 4), "ALIGN"),
    (dict(scale=P + 1), "ALIGN")])
def test_adamw_refusals(lib, B, change, status):
    assert adamw(lib, entries({}, {}), **change) == getattr(B, "FP8Q_ERR_" + status)


@pytest.mark.parametrize("change,kw,status", [
    (dict(n=-1), {}, "SHAPE"), (dict(n=(1 << 42) + 1), {}, "SHAPE"), (dict(p=None), {}, "INVALID"),
    (dict(g=None), {}, "INVALID"), (dict(m=None), {}, "INVALID"), (dict(v=None), {}, "INVALID"),
    (dict(ms=None), dict(state=2), "INVALID"), (dict(vs=None), dict(state=2), "INVALID"),
    (dict(p=P + 2), {}, "ALIGN"), (dict(p=P + 1), dict(kp=0), "ALIGN"), (dict(g=P + (1 << 16) + 2), {}, "ALIGN"),
    (dict(m=P + (2 << 16) + 1), dict(state=0), "ALIGN"), (dict(copy=P + (6 << 16) + 1), {}, "ALIGN"),
    (dict(ms=P + (4 << 16) + 2), dict(state=2), "ALIGN"),
    # ranges that meet: m of one tensor inside p of it, or p of another
    (dict(m=P + 3996), {}, "INVALID"), (dict(v=P + (1 << 20)), {}, "INVALID")])
def test_adamw_tensor_refusals(lib, B, change, kw, status):
    assert adamw(lib, entries(change, {}), **kw) == getattr(B, "FP8Q_ERR_" + status)


def test_adamw_same_tensor_twice_is_refused(lib, B):
    one = entries({})
    assert adamw(lib, (Entry * 2)(one[0], one[0])) == B.FP8Q_ERR_INVALID


def test_empty_work_succeeds(lib, B):
    none = dict(x=None, res=None, w=None, r=None, y=None, q=None, s=None, rstd=None)
    for change in (dict(T=0), dict(C=0)):
        assert lib.fp8q_rmsnorm(*{**NORM, **none, **change}.values()) == B.FP8Q_OK
    assert lib.fp8q_rmsnorm(*{**NORM, "C": 0}.values()) == B.FP8Q_ERR_SHAPE  # rstd of no columns
    assert lib.fp8q_rmsnorm_bwd(*{**NORM_BWD, "C": 0, "dy": None, "x": None, "w": None, "ws": None}.values()) == B.FP8Q_OK
    assert lib.fp8q_route_bwd(*{**ROUTE_BWD, "T": 0, "l": None, "d": None}.values()) == B.FP8Q_OK
    assert adamw(lib, None) == B.FP8Q_OK
    assert adamw(lib, entries(dict(n=0, p=None, g=None, m=None, v=None))) == B.FP8Q_OK


def test_workspace_sizes(lib):
    f = lib.fp8q_rmsnorm_bwd_workspace_bytes
    assert f(1, 128) >= 512 and f(8192, 7168) >= 152 * 7168 * 4 and f(1 << 20, 7168) == f(1 << 21, 7168)
    assert f(-1, 128) == 0 and f(1, 12) == 0 and f(1, 1 << 20) == 0
    f = lib.fp8q_route_workspace_bytes
    assert f(1, 256) == f(256, 256) == 0 and f(1 << 20, 256) == f(1 << 21, 256) > 0
    assert f(-1, 8) == 0 and f(8, 0) == 0 and f(8, 1025) == 0


def test_marshalling_module_names_the_calls(lib, B):
    m = B._calls()
    for name in ("rmsnorm", "rmsnorm_bwd", "adamw", "route", "route_bwd"):
        with pytest.raises(TypeError):
            getattr(m, name)()


def test_binding_refuses_wrong_tensors(lib):
    import torch

    import fp8_fine_grained_amax_gb300 as fq
    x, w = torch.zeros(4, 256).bfloat16(), torch.ones(256)
    for call in (lambda: fq.fp8q_rmsnorm(x, w), lambda: fq.fp8q_rmsnorm_bwd(x, x, torch.ones(4), w),
                 lambda: fq.fp8q_route(torch.zeros(4, 8), 2),
                 lambda: fq.fp8q_route_bwd(torch.zeros(4, 8), torch.zeros(4, 2).int(), torch.zeros(8).int(),
                                           torch.zeros(1).int()),
                 lambda: fq.fp8q_adamw([x.float()], [x.float()], [x.float()], [x.float()], step=1, lr=1e-3)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="BFloat16 or Float"):
        fq.fp8q_rmsnorm(x.half(), w)
    with pytest.raises(ValueError, match="as long as"):
        fq.fp8q_adamw([x], [x, x], [x], [x], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="go together"):
        fq.fp8q_adamw([x], [x], [x], [x], step=1, lr=1e-3, m_scales=[x])
    with pytest.raises(TypeError):
        fq.fp8q_adamw(3, [x], [x], [x], step=1, lr=1e-3)
    with pytest.raises(TypeError):
        fq.fp8q_adamw([3], [x], [x], [x], step=1, lr=1e-3)
    assert fq.fp8q_adamw([], [], [], [], step=1, lr=1e-3) is None


@pytest.mark.parametrize("change", [dict(lr=1e39), dict(lr=-1e300), dict(wd=3.5e38), dict(eps=1e39)])
def test_adamw_numbers_past_fp32_are_refused(lib, B, change):
    # they would be infinite in the kernel
    assert adamw(lib, entries({}, {}), **change) == B.FP8Q_ERR_INVALID


def test_one_beta_alone_is_refused(lib):
    import torch

    import fp8_fine_grained_amax_gb300 as fq
    x = torch.zeros(4)
    for betas in ((None, 0.9), (0.9, None)):
        with pytest.raises(TypeError):
            fq.fp8q_adamw([x], [x], [x], [x], step=1, lr=1e-3, betas=betas)
