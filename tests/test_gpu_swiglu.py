"""The gated feed-forward calls against plain 64-bit arithmetic.

Tolerances (u = 2^-24, absdot = sum_k |a_k b_k| of the dequantised operands):
  e_sum  = (128 + K/128 + 8) * 2u * absdot: 128 products per group summed by the
           tensor cores (each step may truncate: 2u), the K/128 groups added in
           FP32, a few roundings of the scales.
  silu   : exp(-g) from exp2(-g * log2 e) in FP32, relative error below
           (4 + 2 |g|) * 2u, plus the quotient's and the product's few ulps:
           r(g) = (8 + 2 |g|) * 2u.  |silu'| <= 1.1.
  h      : |u| 1.1 e_g + (|silu(g)| + 1.1 e_g) e_u + r |h|, and 1e-35 |u| where
           exp overflows.
  BF16   : half a unit, 2^-8 relative to the value.
  E4M3   : half a code step: 2^-4 of the value, or 2^-10 of the scale below the
           smallest normal code.
"""
import numpy as np
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq
from _util import assert_within_tolerance

pytestmark = pytest.mark.gpu
U2 = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def gen(seed):
    return torch.Generator().manual_seed(seed)


def operands(M, F, K, seed, pow2=False, experts=None):
    """Random codes and scales on the CPU; g and u come out of order one."""
    g = gen(seed)
    G = experts or 1

    def scales(*shape, around):
        s = torch.exp2(torch.randn(*shape, generator=g) * 0.5) * around
        return torch.exp2(torch.round(torch.log2(s))) if pow2 else s

    a = (torch.randn(M, K, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    b = (torch.randn(G, 2 * F, K, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
    sa = scales(K // 128, M, around=1 / 60)
    sb = scales(G, 2 * F // 128, K // 128, around=1.5 / 60 / max(K, 1) ** 0.5)
    if experts is None:
        b, sb = b[0], sb[0]
    return a.view(torch.uint8), sa, b.view(torch.uint8), sb


def values(a, sa, b, sb):
    x = a.view(torch.float8_e4m3fn).double() * sa.double().t().repeat_interleave(128, 1)
    w = b.view(torch.float8_e4m3fn).double() * \
        sb.double().repeat_interleave(128, -2).repeat_interleave(128, -1)
    return x, w


def reference(x, w):
    """gu, its error bound, h, its error bound."""
    K, F = x.shape[1], w.shape[0] // 2
    gu = x @ w.t()
    e = (128 + K / 128 + 8) * U2 * (x.abs() @ w.abs().t())
    g, u, eg, eu = gu[:, :F], gu[:, F:], e[:, :F], e[:, F:]
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    eh = u.abs() * 1.1 * eg + (silu.abs() + 1.1 * eg) * eu + (8 + 2 * g.abs()) * U2 * h.abs() + \
        1e-35 * (u.abs() + eu)
    return gu, e, h, eh


def pow2_scale(amax):
    a = np.maximum(amax, 2.0 ** -116)
    e = np.floor(np.log2(a)) - 9
    while True:
        low = 448.0 * 2.0 ** e < a
        if not low.any():
            return 2.0 ** e
        e = e + low


def check_codes(q, s, v, ev, pow2, what):
    """1x128 codes q [M][C] and scales s [C/128][M] of values v within ev."""
    M, C = v.shape
    q = q.cpu().view(torch.float8_e4m3fn).double().numpy().reshape(M, C // 128, 128)
    s = s.double().cpu().numpy().T
    v, ev = v.numpy().reshape(M, C // 128, 128), ev.numpy().reshape(M, C // 128, 128)
    amax, ea = np.abs(v).max(-1), ev.max(-1)
    if pow2:
        lo, hi = pow2_scale(np.maximum(amax - ea, 0)), pow2_scale(amax + ea)
        assert np.all((s == lo) | (s == hi)), what
    else:
        want = np.maximum(amax, 2.0 ** -116) / 448
        assert_within_tolerance(s, want, ea / 448 + 4 * U2 * want, what + " scales")
    tol = np.maximum(2.0 ** -4 * (np.abs(v) + ev), 2.0 ** -10 * s[..., None]) + ev + \
        4 * U2 * np.abs(v)
    assert_within_tolerance(q * s[..., None], v, tol, what + " codes")


def check_forward(r, x, w, scale_mode, rows=slice(None)):
    gu, e, h, eh = reference(x, w)
    if r.gu is not None:
        assert_within_tolerance(r.gu[rows].double().cpu().numpy(), gu.numpy(),
                                (e + 2.0 ** -8 * (gu.abs() + e)).numpy(), "gu")
    if r.h is not None:
        assert_within_tolerance(r.h[rows].double().cpu().numpy(), h.numpy(),
                                (eh + 2.0 ** -8 * (h.abs() + eh)).numpy(), "h")
    if r.q is not None:
        check_codes(r.q[rows], r.s[:, rows], h, eh, scale_mode == fq.FP8Q_SCALE_POW2, "h")


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,F,K", [(1, 128, 128), (2, 256, 1152), (7, 128, 640), (8, 384, 256),
                                   (9, 128, 896), (17, 256, 128), (25, 128, 1024), (32, 256, 384),
                                   (33, 128, 256), (100, 256, 512), (256, 384, 128),
                                   (257, 128, 1280), (333, 640, 896), (700, 256, 640)])
def test_forward(M, F, K, pow2):
    a, sa, b, sb = operands(M, F, K, 1000 + M, pow2)
    call = fq.fp8q_gemm_swiglu_pow2 if pow2 else fq.fp8q_gemm_swiglu
    for mode in (fq.FP8Q_SCALE_FP32, fq.FP8Q_SCALE_POW2):
        r = call(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True,
                 scale_mode=mode)
        check_forward(r, *values(a, sa, b, sb), mode)


@pytest.mark.parametrize("M", [3, 70])
@pytest.mark.parametrize("want", [dict(), dict(with_gu=True), dict(with_codes=True),
                                  dict(with_h=False, with_codes=True),
                                  dict(with_h=False, with_gu=True)])
def test_forward_each_result_alone(M, want):
    a, sa, b, sb = operands(M, 256, 384, 5)
    full = fq.fp8q_gemm_swiglu(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True,
                               with_codes=True)
    r = fq.fp8q_gemm_swiglu(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), **want)
    assert (r.h is not None) == want.get("with_h", True)
    assert (r.gu is not None) == want.get("with_gu", False)
    assert (r.q is not None) == (r.s is not None) == want.get("with_codes", False)
    for got, ref in zip(r, full):
        assert got is None or torch.equal(got, ref)


@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("pow2", [False, True])
def test_forward_empty_sums_and_zero_rows(M, pow2):
    call = fq.fp8q_gemm_swiglu_pow2 if pow2 else fq.fp8q_gemm_swiglu
    floor = torch.tensor(2.0 ** -116 / 448, dtype=torch.float32)
    # K = 0
    e8 = torch.empty(M, 0, dtype=torch.uint8, device="cuda")
    r = call(e8, torch.empty(0, M, device="cuda"), e8.new_empty(256, 0),
             torch.empty(2, 0, device="cuda"), with_gu=True, with_codes=True)
    assert not r.h.any() and not r.gu.any() and not r.q.bitwise_and(0x7F).any()
    assert torch.equal(r.s.cpu(), floor.expand_as(r.s.cpu()))
    # a token of zero codes among others
    a, sa, b, sb = operands(M, 128, 256, 6, pow2)
    a[M // 2] = 0
    r = call(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True)
    check_forward(r, *values(a, sa, b, sb), fq.FP8Q_SCALE_FP32)
    assert r.s[0, M // 2].cpu() == floor
    # no tokens: nothing to do
    r = call(a[:0].cuda(), sa[:, :0].cuda(), b.cuda(), sb.cuda(), with_codes=True)
    assert r.h.shape == (0, 128) and r.q.shape == (0, 128)


@pytest.mark.parametrize("M", [4, 150])
def test_forward_large_magnitudes(M):
    # g of both signs up to thousands: exp overflows on one side, silu(g) = g on the other
    a, sa, b, sb = operands(M, 128, 256, 7)
    sa = sa * 500
    r = fq.fp8q_gemm_swiglu(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True,
                            with_codes=True)
    assert torch.isfinite(r.h.float()).all() and torch.isfinite(r.s).all()
    check_forward(r, *values(a, sa, b, sb), fq.FP8Q_SCALE_FP32)


def padded(rows, cols, pad_rows, pad_cols, dtype, fill):
    """A view of the first rows x cols of a sentinel-filled buffer, and the buffer."""
    t = torch.full((rows + pad_rows, cols + pad_cols), fill, dtype=dtype, device="cuda")
    return t[:rows, :cols], t


@pytest.mark.parametrize("M", [3, 24, 130])
@pytest.mark.parametrize("pow2", [False, True])
def test_forward_strides_and_padding(M, pow2):
    F, K = 256, 384
    a, sa, b, sb = operands(M, F, K, 8, pow2)
    av, _ = padded(M, K, 2, 48, torch.uint8, 0x7F)       # NaN codes in the padding
    bv, _ = padded(2 * F, K, 2, 16, torch.uint8, 0x7F)
    sav, _ = padded(K // 128, M, 1, 3, torch.float32, float("nan"))
    sbv, _ = padded(2 * F // 128, K // 128, 1, 2, torch.float32, float("nan"))
    for v, t in ((av, a), (bv, b), (sav, sa), (sbv, sb)):
        v.copy_(t)
    h, hb = padded(M, F, 3, 8, torch.bfloat16, 7.0)
    gu, gub = padded(M, 2 * F, 3, 24, torch.bfloat16, 7.0)
    q, qb = padded(M, F, 3, 16, torch.uint8, 0xCD)
    s, sbuf = padded(F // 128, M, 2, 5, torch.float32, -3.0)
    call = fq.fp8q_gemm_swiglu_pow2 if pow2 else fq.fp8q_gemm_swiglu
    r = call(av, sav, bv, sbv, h=h, gu=gu, q=q, s=s)
    check_forward(r, *values(a, sa, b, sb), fq.FP8Q_SCALE_FP32)
    for view, buf, fill in ((h, hb, 7.0), (gu, gub, 7.0), (q, qb, 0xCD), (s, sbuf, -3.0)):
        view.fill_(fill)
        assert bool((buf == fill).all()), "wrote outside its result"


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("offs", [[0, 0, 70, 70, 300, 333], [5, 6, 200, 201, 290, 300],
                                  [0, 333, 333, 333, 333, 333], [0, 1, 2, 3, 4, 333],
                                  [-4, 90, 40, 250, 900, 333]])
def test_experts(offs, pow2):
    M, F, K, G = 333, 256, 384, 5
    a, sa, b, sb = operands(M, F, K, 9, pow2, experts=G)
    h = torch.full((M, F), 7.0, dtype=torch.bfloat16, device="cuda")
    gu = torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((M, F), 0xCD, dtype=torch.uint8, device="cuda")
    s = torch.full((F // 128, M), -3.0, device="cuda")
    call = fq.fp8q_grouped_gemm_swiglu_pow2 if pow2 else fq.fp8q_grouped_gemm_swiglu
    r = call(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(),
             torch.tensor(offs, dtype=torch.int32, device="cuda"), h=h, gu=gu, q=q, s=s)
    # the ranges that the interface documents: clamped, never overlapping
    clamped = [min(max(o, 0), M) for o in offs]
    covered = torch.zeros(M, dtype=torch.bool)
    prev = 0
    for e in range(G):
        lo = max(clamped[e], prev)
        hi = max(lo, clamped[e + 1])
        prev = hi
        if hi > lo:
            x, w = values(a, sa, b[e], sb[e])
            check_forward(r, x[lo:hi], w, fq.FP8Q_SCALE_FP32, slice(lo, hi))
        covered[lo:hi] = True
    left = ~covered.cuda()
    assert bool((h[left] == 7.0).all() and (gu[left] == 7.0).all() and (q[left] == 0xCD).all()
                and (s[:, left] == -3.0).all())


def test_pow2_precondition_is_reported():
    for M in (4, 64):
        a, sa, b, sb = operands(M, 128, 256, 10, True)
        sa[1, 2] = 0.3
        fq.fp8q_gemm_swiglu_pow2(a.cuda(), sa.cuda(), b.cuda(), sb.cuda())
        assert B.fp8q_sync_status() == fq.binding.FP8Q_ERR_INVALID
        assert B.fp8q_sync_status() == 0


# ------------------------------------------------------------------ backward
def grads(dh, gu):
    """d = [dg | du], h and their error bounds, 64 bits."""
    F = dh.shape[1]
    y, g, u = dh.double(), gu[:, :F].double(), gu[:, F:].double()
    s = 1 / (1 + torch.exp(-g))
    silu = g * s
    r = (12 + 2 * g.abs()) * U2
    slope, slope_abs = s + silu * (1 - s), s + (silu * (1 - s)).abs()
    d = torch.cat([y * u * slope, y * silu], 1)
    # where exp overflows, s = 0 in place of a value below 1e-37
    tiny = 1e-35
    e = torch.cat([(y * u).abs() * (r * slope_abs + tiny), y.abs() * (r * silu.abs() + tiny)], 1)
    return d, e, silu * u, u.abs() * (r * silu.abs() + tiny)


def bwd_inputs(T, F, seed, spread=2.0):
    g = gen(seed)
    return (torch.randn(T, F, generator=g) * 1e-3).bfloat16(), \
        (torch.randn(T, 2 * F, generator=g) * spread).bfloat16()


def check_bwd(r, dh, gu, mode):
    d, e, h, eh = grads(dh, gu)
    pow2 = mode == fq.FP8Q_SCALE_POW2
    if r.d is not None:
        assert_within_tolerance(r.d.double().cpu().numpy(), d.numpy(),
                                (e + 2.0 ** -8 * (d.abs() + e)).numpy(), "d")
    if r.q is not None:
        check_codes(r.q, r.s, d, e, pow2, "d")
    if r.qT is not None:
        check_codes(r.qT, r.sT, d.t().contiguous(), e.t().contiguous(), pow2, "d^T")
    if r.hT is not None:
        check_codes(r.hT, r.shT, h.t().contiguous(), eh.t().contiguous(), pow2, "h^T")


@pytest.mark.parametrize("mode", [fq.FP8Q_SCALE_FP32, fq.FP8Q_SCALE_POW2])
@pytest.mark.parametrize("T,F", [(128, 128), (128, 640), (384, 256), (1024, 384)])
def test_backward(T, F, mode):
    dh, gu = bwd_inputs(T, F, 20 + T)
    r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True, scale_mode=mode)
    check_bwd(r, dh, gu, mode)


@pytest.mark.parametrize("T", [1, 3, 127, 129, 500])
@pytest.mark.parametrize("rows", [False, True])
def test_backward_any_token_count(T, rows):
    dh, gu = bwd_inputs(T, 256, 30 + T)
    r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True, with_rows=rows, with_cols=False,
                           with_h=False)
    assert r.qT is None and r.hT is None and (r.q is not None) == rows
    check_bwd(r, dh, gu, fq.FP8Q_SCALE_FP32)


def test_backward_each_result_alone():
    dh, gu = bwd_inputs(256, 256, 40)
    full = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True)
    names = ("with_d", "with_rows", "with_cols", "with_h")
    for bits in range(1, 16):
        want = {n: bool(bits >> i & 1) for i, n in enumerate(names)}
        r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), **want)
        for got, ref in zip(r, full):
            assert got is None or torch.equal(got, ref), want


def test_backward_extremes():
    # saturated and vanishing gates, zero groups, one large entry in a group
    dh, gu = bwd_inputs(128, 256, 41, spread=1.0)
    gu[:, :64] = 200.0
    gu[:, 64:128] = -200.0
    dh[:, 130] = 0
    dh[5] = 0
    gu[7, 200] = 3e4
    gu[:, 256 + 140] = 0
    r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True)
    check_bwd(r, dh, gu, fq.FP8Q_SCALE_FP32)
    floor = torch.tensor(2.0 ** -116 / 448, dtype=torch.float32)
    assert torch.equal(r.s[:, 5].cpu(), floor.expand(4)) and r.sT[0, 130].cpu() == floor
    assert r.shT[0, 140].cpu() == floor


def test_backward_matches_differences():
    # central differences of L = sum dh * silu(g) * u in 64 bits: error below
    # eps^2 |f'''| / 6 + rounding 2^-52 |f| / eps, eps = 1e-4: 1e-8 relative to
    # the terms' size, so the BF16 rounding (2^-8) and the kernel's own bound dominate
    dh, gu = bwd_inputs(64, 128, 42)
    r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True, with_rows=False, with_cols=False,
                           with_h=False)
    y, g, u = dh.double(), gu[:, :128].double(), gu[:, 128:].double()
    f = lambda g, u: y * g / (1 + torch.exp(-g)) * u  # noqa: E731
    eps = 1e-4
    diff = torch.cat([(f(g + eps, u) - f(g - eps, u)) / (2 * eps),
                      (f(g, u + eps) - f(g, u - eps)) / (2 * eps)], 1)
    d, e, _, _ = grads(dh, gu)
    size = torch.cat([(y * u).abs() * (1 + g.abs()), y.abs() * (1 + g.abs())], 1)
    assert_within_tolerance(r.d.double().cpu().numpy(), diff.numpy(),
                            (2 * e + 2.0 ** -8 * (d.abs() + e) + 1e-7 * size).numpy(), "differences")


def test_backward_strides_and_padding():
    T, F = 256, 128
    dh, gu = bwd_inputs(T, F, 43)
    dv, _ = padded(T, F, 1, 8, torch.bfloat16, float("nan"))
    gv, _ = padded(T, 2 * F, 1, 16, torch.bfloat16, float("nan"))
    dv.copy_(dh)
    gv.copy_(gu)
    outs = dict(d=(T, 2 * F, 8, torch.bfloat16, 7.0), q=(T, 2 * F, 16, torch.uint8, 0xCD),
                s=(2 * F // 128, T, 3, torch.float32, -3.0), qT=(2 * F, T, 16, torch.uint8, 0xCD),
                sT=(T // 128, 2 * F, 1, torch.float32, -3.0), hT=(F, T, 32, torch.uint8, 0xCD),
                shT=(T // 128, F, 5, torch.float32, -3.0))
    views, bufs = {}, {}
    for k, (rows, cols, pad, dt, fill) in outs.items():
        views[k], bufs[k] = padded(rows, cols, 2, pad, dt, fill)
    r = fq.fp8q_swiglu_bwd(dv, gv, **views)
    check_bwd(r, dh, gu, fq.FP8Q_SCALE_FP32)
    for k, (_, _, _, _, fill) in outs.items():
        views[k].fill_(fill)
        assert bool((bufs[k] == fill).all()), f"{k}: wrote outside its result"


def test_streams_and_graph_capture():
    a, sa, b, sb = (t.cuda() for t in operands(300, 256, 384, 50))
    dh, gu = (t.cuda() for t in bwd_inputs(256, 256, 51))
    few = (a[:6], sa[:, :6].contiguous(), b, sb)
    eager = [fq.fp8q_gemm_swiglu(a, sa, b, sb, with_gu=True, with_codes=True),
             fq.fp8q_gemm_swiglu(*few, with_gu=True, with_codes=True),
             fq.fp8q_swiglu_bwd(dh, gu, with_d=True)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [fq.fp8q_gemm_swiglu(a, sa, b, sb, with_gu=True, with_codes=True),
                 fq.fp8q_gemm_swiglu(*few, with_gu=True, with_codes=True),
                 fq.fp8q_swiglu_bwd(dh, gu, with_d=True)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [fq.fp8q_gemm_swiglu(a, sa, b, sb, with_gu=True, with_codes=True),
                    fq.fp8q_gemm_swiglu(*few, with_gu=True, with_codes=True),
                    fq.fp8q_swiglu_bwd(dh, gu, with_d=True)]
    graph.replay()
    torch.cuda.synchronize()
    for e, s, c in zip(eager, again, captured):
        for x, y, z in zip(e, s, c):
            assert torch.equal(x, y) and torch.equal(x, z)


def test_binding_refuses():
    a, sa, b, sb = (t.cuda() for t in operands(4, 128, 256, 60))
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(a, sa, b[:, :128], sb)           # another K
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(a, sa[:1], b, sb)                # scales of another K
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(a, sa, b, sb[:1])
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(a.view(torch.int8), sa, b, sb)   # codes are uint8
    with pytest.raises(ValueError):
        fq.fp8q_gemm_swiglu(a, sa, b, sb, h=torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(fq.FP8QError) as err:
        fq.fp8q_gemm_swiglu(a, sa, b, sb, with_h=False)      # nothing to compute
    assert err.value.status == B.FP8Q_ERR_INVALID
    dh, gu = (t.cuda() for t in bwd_inputs(100, 128, 61))
    with pytest.raises(fq.FP8QError) as err:
        fq.fp8q_swiglu_bwd(dh, gu)                           # 128x1 tiles of 100 tokens
    assert err.value.status == B.FP8Q_ERR_SHAPE
    with pytest.raises(ValueError):
        fq.fp8q_swiglu_bwd(dh, gu[:, :128])
    with pytest.raises(ValueError):
        fq.fp8q_swiglu_bwd(dh.float(), gu)
