"""The RMS norm and its backward pass against plain 64-bit arithmetic.

Tolerances (u = 2^-24), for C columns:
  h    : one FP32 addition, u |h|.
  rstd : the row's squares are all positive: at most 32 terms one after another in a
         thread (backward's long form: 32), 10 levels of a tree, and each square's and
         h's own rounding: (46 + 3) u relative in the sum, half of that in its root, 4 u
         for 1 / C, the root and the quotient: 32 u.
  y    : h, rstd and two products: 36 u |y|.
  BF16 : half a unit, 2^-8 of the value.
  E4M3 : half a code step: 2^-4 of the value, or 2^-10 of the scale below the smallest
         normal code.
  dx   : t = dy w and xh with a rounding each; c is a sum of C products, 42 terms deep at
         most, so off by 46 u of the sum of magnitudes / C; four more roundings of each
         term.
  dw   : at most ceil(T / 152) rows one after another in a CTA and 912 partial sums in
         32 parts and a tree, at most 40 deep: well below 160 more: as
         many u of the sum of magnitudes, and 3 for each product.
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq
from test_gpu_swiglu import check_codes, padded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def rand(seed, *shape, dtype=FP, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def near(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    ok = err <= tol
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} outside, max err/tol " \
        f"{float((err / tol.clamp_min(1e-300)).max()):.3g}"


def half(t):
    return 2.0 ** -8 if t.dtype == BF else U


def check_forward(out, x, w, res, eps, mode):
    h = x.double() + (0 if res is None else res.double())
    rstd = 1 / (h.square().mean(1, keepdim=True) + eps).sqrt()
    y = h * rstd * w.double()
    if out.r is not None:
        near(out.r, h, half(out.r) * 1.01 * h.abs() + U * h.abs() + 1e-40, "r")
    if out.rstd is not None:
        near(out.rstd, rstd[:, 0], 32 * U * rstd[:, 0], "rstd")
    ey = 36 * U * y.abs()
    if out.y is not None:
        near(out.y, y, ey + 2.0 ** -8 * (y.abs() + ey) + 1e-40, "y")
    if out.q is not None:
        check_codes(out.q, out.s, y, ey + 1e-40, mode == fq.FP8Q_SCALE_POW2, "codes")


@pytest.mark.parametrize("T,C,kx,kres", [
    (1, 128, BF, None), (1, 7168, BF, BF), (3, 256, FP, BF), (7, 384, BF, FP), (2, 1024, FP, FP), (5, 1152, FP, None),
    (33, 896, BF, FP), (130, 2048, BF, BF), (2, 32768, FP, FP), (9, 16512, BF, BF), (1000, 640, BF, BF),
    (333, 7168, FP, BF), (4, 3200, BF, None), (700, 128, FP, None)])
def test_forward(T, C, kx, kres):
    x, w = rand(T + C, T, C, dtype=kx), 1 + rand(1, C, std=0.3)
    res = None if kres is None else rand(T + C + 1, T, C, dtype=kres, std=3.0)
    for mode in (fq.FP8Q_SCALE_FP32, fq.FP8Q_SCALE_POW2):
        wk = w if mode == fq.FP8Q_SCALE_FP32 else w.to(BF)
        out = fq.fp8q_rmsnorm(x.cuda(), wk.cuda(), residual=None if res is None else res.cuda(), eps=1e-5, with_y=True,
                              with_rstd=True, scale_mode=mode)
        assert (out.r is None) == (res is None)
        check_forward(out, x, wk, res, 1e-5, mode)


@pytest.mark.parametrize("C", [8, 24, 264, 1000, 1032, 4104, 8200])
def test_forward_without_codes(C):
    x, w, res = rand(C, 37, C, dtype=BF), rand(2, C), rand(3, 37, C)
    out = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), with_y=True, with_codes=False, with_rstd=True)
    check_forward(out, x, w, res, 1e-6, 0)
    assert out.q is None and out.s is None


@pytest.mark.parametrize("C", [512, 2304])
def test_each_result_alone(C):
    x, w, res = rand(5, 11, C, dtype=BF).cuda(), rand(6, C).cuda(), rand(7, 11, C, dtype=BF).cuda()
    full = fq.fp8q_rmsnorm(x, w, residual=res, with_y=True, with_rstd=True)
    none = dict(with_r=False, with_y=False, with_codes=False, with_rstd=False)
    for name in ("r", "y", "codes", "rstd"):
        out = fq.fp8q_rmsnorm(x, w, residual=res, **{**none, f"with_{name}": True})
        for field, got in zip(out._fields, out):
            wanted = field == name or (name == "codes" and field in "qs")
            assert (got is not None) == wanted
            assert got is None or torch.equal(got, getattr(full, field))
    with pytest.raises(fq.FP8QError):
        fq.fp8q_rmsnorm(x, w, residual=res, **none)
    with pytest.raises(ValueError):
        fq.fp8q_rmsnorm(x, w, r=res)


@pytest.mark.parametrize("C", [256, 4096])
def test_zero_rows_and_large_and_small_rows(C):
    x, w = rand(8, 6, C, dtype=FP), 1 + rand(9, C, std=0.1)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-15
    x[3, 1:] = 0
    x[4] = 3e38 ** 0.5 / C ** 0.5 * 0.9
    out = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, with_y=True, with_rstd=True)
    check_forward(out, x, w, None, 1e-6, 0)
    assert not out.y[0].any() and not out.q[0].bitwise_and(0x7F).any()
    # a row that is no number leaves the others alone
    bad = x.clone()
    bad[2] = float("nan")
    bad[4, 7] = float("inf")
    got = fq.fp8q_rmsnorm(bad.cuda(), w.cuda(), eps=1e-6, with_y=True, with_rstd=True)
    keep = [0, 1, 3, 5]
    assert torch.equal(got.y[keep], out.y[keep]) and torch.equal(got.q[keep], out.q[keep])
    assert torch.isnan(got.y[2].float()).all()


@pytest.mark.parametrize("C,kres", [(256, BF), (1024, FP), (1152, FP), (7168, BF)])
def test_residual_updated_in_place_and_strides(C, kres):
    T = 21
    x, w, res = rand(10, T, C, dtype=BF), rand(11, C), rand(12, T, C, dtype=kres)
    want = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), residual=res.cuda(), with_y=True, with_rstd=True)
    nan = float("nan")
    xv, _ = padded(T, C, 2, 8, BF, nan)
    rv, rb = padded(T, C, 2, 24, kres, 7.0)
    y, yb = padded(T, C, 1, 16, BF, 7.0)
    q, qb = padded(T, C, 1, 48, torch.uint8, 0xCD)
    s, sb = padded(C // 128, T, 1, 5, FP, -3.0)
    xv.copy_(x)
    rv.copy_(res)
    out = fq.fp8q_rmsnorm(xv, w.cuda(), residual=rv, r=rv, y=y, q=q, s=s, with_rstd=True)
    assert out.r is rv and out.y is y and out.q is q and out.s is s
    for got, ref in zip(out, want):
        assert torch.equal(got, ref)
    assert (rb[:, C:] == 7).all() and (rb[T:] == 7).all() and (yb[:, C:] == 7).all() and (yb[T:] == 7).all()
    assert (qb[:, C:] == 0xCD).all() and (qb[T:] == 0xCD).all() and (sb[:, T:] == -3).all()


def test_no_rows():
    e = torch.empty(0, 256, dtype=BF, device="cuda")
    w = torch.ones(256, device="cuda")
    out = fq.fp8q_rmsnorm(e, w, residual=e, with_y=True, with_rstd=True)
    assert out.y.shape == (0, 256) and out.s.shape == (2, 0) and out.rstd.shape == (0,)
    g = fq.fp8q_rmsnorm_bwd(e, e, out.rstd, w)
    assert g.dx.shape == (0, 256) and not g.dw.any()
    dw = torch.full((256,), 3.0, device="cuda")
    fq.fp8q_rmsnorm_bwd(e, e, out.rstd, w, dw=dw, accumulate=True)
    assert (dw == 3).all()


def reference_bwd(dy, x, rstd, w, dres):
    dy, x, rs, w = dy.double(), x.double(), rstd.double()[:, None], w.double()
    C = x.shape[1]
    xh, t = x * rs, dy * w
    c, size = (t * xh).mean(1, keepdim=True), (t * xh).abs().mean(1, keepdim=True)
    dx = rs * (t - xh * c)
    tol = rs * (4 * U * (t.abs() + (xh * c).abs()) + xh.abs() * 46 * U * size)
    if dres is not None:
        dx = dx + dres.double()
        tol = tol + U * dx.abs()
    rows = -(-x.shape[0] // 152) + 160
    return dx, tol, (dy * xh).sum(0), (rows + 3) * U * (dy * xh).abs().sum(0)


SHAPES = [(1, 8, FP, FP, FP, True), (1, 128, BF, BF, BF, False), (5, 256, BF, FP, BF, True), (64, 520, FP, BF, FP, True),
          (333, 896, BF, BF, FP, False), (5000, 1024, BF, BF, BF, True), (700, 1032, BF, BF, BF, True),
          (128, 2048, BF, BF, BF, False), (77, 4104, FP, FP, FP, True), (1, 7168, BF, BF, BF, True),
          (333, 7168, BF, FP, BF, True), (310, 8192, FP, FP, FP, True), (3, 8200, BF, BF, BF, True),
          (170, 16512, FP, BF, BF, False), (2, 32768, FP, FP, FP, True)]


@pytest.mark.parametrize("T,C,kdy,kx,kd,with_dres", SHAPES)
def test_backward(T, C, kdy, kx, kd, with_dres):
    x, dy, w = rand(C, T, C, dtype=kx, std=2.0), rand(T, T, C, dtype=kdy, std=1e-3), 1 + rand(13, C, std=0.3)
    w = w.to(BF) if T % 2 else w
    rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float()
    dres = rand(14, T, C, dtype=kd, std=1e-3) if with_dres else None
    want, tol, dw, tolw = reference_bwd(dy, x, rstd, w, dres)
    kind = fq.FP8Q_OUT_BF16 if kd == BF else fq.FP8Q_OUT_FP32
    args = (dy.cuda(), x.cuda(), rstd.cuda(), w.cuda())
    g = fq.fp8q_rmsnorm_bwd(*args, dres=None if dres is None else dres.cuda(), out_dtype=kind)
    near(g.dx, want, tol + half(g.dx) * (want.abs() + tol) + 1e-40, "dx")
    near(g.dw, dw, tolw + 1e-40, "dw")
    # the same bits again, each result alone, dw added to what is there, dres as its own result
    only = fq.fp8q_rmsnorm_bwd(*args, with_dx=False)
    assert only.dx is None and torch.equal(only.dw, g.dw)
    held = torch.full_like(g.dw, 0.25)
    dx = None if dres is None else dres.cuda()
    more = fq.fp8q_rmsnorm_bwd(*args, dres=dx, dx=dx, dw=held, accumulate=True, out_dtype=kind)
    assert torch.equal(more.dw, 0.25 + g.dw) and torch.equal(more.dx, g.dx)
    only = fq.fp8q_rmsnorm_bwd(*args, dres=None if dres is None else dres.cuda(), with_dw=False, out_dtype=kind)
    assert only.dw is None and torch.equal(only.dx, g.dx)


@pytest.mark.parametrize("C", [64, 1536, 8704])
def test_backward_strides(C):
    T = 19
    x, dy, w, dres = rand(15, T, C, dtype=BF), rand(16, T, C, dtype=BF), rand(17, C), rand(18, T, C, dtype=BF)
    rstd = (x.double().square().mean(1) + 1e-6).rsqrt().float().cuda()
    want = fq.fp8q_rmsnorm_bwd(dy.cuda(), x.cuda(), rstd, w.cuda(), dres=dres.cuda())
    views = [padded(T, C, 2, p, BF, float("nan"))[0] for p in (8, 24, 40)]
    for v, t in zip(views, (dy, x, dres)):
        v.copy_(t)
    dx, buf = padded(T, C, 2, 16, BF, 7.0)
    ws = torch.full((fq.fp8q_rmsnorm_bwd_workspace_bytes(T, C) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    got = fq.fp8q_rmsnorm_bwd(views[0], views[1], rstd, w.cuda(), dres=views[2], dx=dx, workspace=ws[:-64])
    assert torch.equal(got.dx, want.dx) and torch.equal(got.dw, want.dw)
    assert (buf[:, C:] == 7).all() and (buf[T:] == 7).all() and (ws[-64:] == 0xFF).all()


def test_gradients_against_differences():
    # sum(y * dy) + sum(h * dres) of the exact forward at x +- e along random directions
    T, C, e = 4, 96, 1e-4
    x, dy, w, dres = rand(19, T, C), rand(20, T, C), 1 + rand(21, C, std=0.2), rand(22, T, C)

    def value(xx, ww):
        y = xx / (xx.square().mean(1, keepdim=True) + 1e-6).sqrt() * ww
        return float((y * dy.double()).sum() + (xx * dres.double()).sum())

    out = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), eps=1e-6, with_codes=False, with_rstd=True)
    g = fq.fp8q_rmsnorm_bwd(dy.cuda(), x.cuda(), out.rstd, w.cuda(), dres=dres.cuda(), out_dtype=fq.FP8Q_OUT_FP32)
    for seed in range(4):
        d = rand(30 + seed, T, C).double()
        slope = (value(x.double() + e * d, w.double()) - value(x.double() - e * d, w.double())) / (2 * e)
        # third differences e^2 of order one, FP32 gradients
        assert abs(slope - float((g.dx.double().cpu() * d).sum())) < 1e-5 * (1 + float(d.norm() * g.dx.double().norm().cpu()))
        d = rand(40 + seed, C).double()
        slope = (value(x.double(), w.double() + e * d) - value(x.double(), w.double() - e * d)) / (2 * e)
        assert abs(slope - float((g.dw.double().cpu() * d).sum())) < 1e-5 * (1 + float(d.norm() * g.dw.double().norm().cpu()))


def test_rows_past_32_bit_offsets():
    # 2300 rows a million elements apart: offsets of 2.3e9 elements
    T, C, ld = 2300, 256, 1_000_000
    buf = torch.empty((T - 1) * ld + C, dtype=BF, device="cuda")
    x = buf.as_strided((T, C), (ld, 1))
    data, w = rand(23, T, C, dtype=BF), rand(24, C)
    x.copy_(data)
    out = fq.fp8q_rmsnorm(x, w.cuda(), residual=x, r=x, with_y=True, with_rstd=True)
    check_forward(out, data, w, data, 1e-6, 0)
    g = fq.fp8q_rmsnorm_bwd(x, x, out.rstd, w.cuda(), dres=x, dx=x)
    h = (data.double() * 2).to(BF)
    want, tol, dw, tolw = reference_bwd(h, h, out.rstd.cpu(), w, h)
    near(g.dx, want, tol + 2.0 ** -8 * (want.abs() + tol), "dx")
    near(g.dw, dw, tolw, "dw")


# more rows than a launch has CTAs (or warps) for: each takes two to four, so the ring's places are used again
@pytest.mark.parametrize("T,C,kx,kres", [
    (6000, 520, BF, BF), (6000, 640, FP, FP), (3000, 1152, BF, BF), (3001, 1280, FP, BF), (1500, 4088, BF, FP),
    (1500, 3968, BF, None), (500, 4096, FP, FP), (400, 8320, BF, BF), (310, 16384, BF, None), (400, 16512, BF, BF),
    (310, 24576, FP, None), (200, 32768, BF, FP)])
def test_forward_of_more_rows_than_a_launch_takes(T, C, kx, kres):
    x, w = rand(T + C, T, C, dtype=kx), 1 + rand(1, C, std=0.3)
    x = (x.float() * (1 + torch.arange(T) % 7)[:, None]).to(kx)  # rows that are not mistaken for one another
    res = None if kres is None else rand(T + C + 1, T, C, dtype=kres, std=3.0)
    codes = C % 128 == 0
    out = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), with_y=True, with_rstd=True,
                          with_codes=codes)
    check_forward(out, x, w, res, 1e-6, fq.FP8Q_SCALE_FP32)
    # statistics alone: rows that end before their results
    only = fq.fp8q_rmsnorm(x.cuda(), w.cuda(), residual=None if res is None else res.cuda(), with_r=False, with_codes=False,
                           with_rstd=True)
    assert torch.equal(only.rstd, out.rstd)


@pytest.mark.parametrize("T,C,kdy,kx,kd,with_dres", [
    (9000, 256, BF, BF, BF, True), (9001, 136, FP, FP, BF, False), (8000, 8, BF, FP, FP, True), (6000, 512, BF, FP, FP, True),
    (6001, 264, FP, FP, BF, True), (3000, 1024, FP, FP, FP, True), (3000, 1152, BF, BF, BF, True), (3001, 1032, FP, FP, BF, True),
    (1500, 2048, BF, FP, FP, True), (400, 8704, BF, BF, BF, True), (400, 9216, FP, FP, BF, False), (310, 16384, BF, BF, BF, True),
    (400, 10240, FP, FP, FP, True), (310, 16512, BF, FP, FP, True), (310, 4096, FP, BF, BF, True)])
def test_backward_of_more_rows_than_a_launch_takes(T, C, kdy, kx, kd, with_dres):
    test_backward(T, C, kdy, kx, kd, with_dres)
