"""The gated feed-forward calls on every path they can take: the dense GEMM tiles, which the few-token
kernel's rule leaves only to larger calls, and the second passes of every ring, buffer and persistent
loop.  Tolerances as derived in test_gpu_swiglu.py.

Which path a call takes: the few-token kernel for up to 64 tokens, and for more while blocks of 64
columns times blocks of 64 tokens are at most 128; its K split is the largest of 4, 2 and 1 that
keeps all its CTAs resident at once, two per SM.
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq
from _util import assert_within_tolerance
from test_gpu_swiglu import bwd_inputs, check_bwd, check_codes, operands, padded, reference, values

pytestmark = pytest.mark.gpu
SMS = 152


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def blocks(M, F):
    return F // 64 * ((M + 63) // 64)


def on_tiles(M, F):
    return M > 64 and blocks(M, F) > 128


def k_split(M, F):
    return next(s for s in (4, 2, 1) if s == 1 or s * blocks(M, F) <= 2 * SMS)


def call_of(pow2):
    return fq.fp8q_gemm_swiglu_pow2 if pow2 else fq.fp8q_gemm_swiglu


def check(r, a, sa, b, sb, mode, rows=slice(None)):
    """All results against 64-bit values, whose products run on the GPU (plain torch)."""
    gu, e, h, eh = (t.cpu() for t in reference(*values(a.cuda(), sa.cuda(), b.cuda(), sb.cuda())))
    assert_within_tolerance(r.gu[rows].double().cpu().numpy(), gu.numpy(),
                            (e + 2.0 ** -8 * (gu.abs() + e)).numpy(), "gu")
    assert_within_tolerance(r.h[rows].double().cpu().numpy(), h.numpy(),
                            (eh + 2.0 ** -8 * (h.abs() + eh)).numpy(), "h")
    check_codes(r.q[rows], r.s[:, rows], h, eh, mode == fq.FP8Q_SCALE_POW2, "h")


# ------------------------------------------------------------------ dense tiles
DENSE = [(65, 8320, 128), (333, 1536, 256), (512, 1152, 640), (700, 896, 1152), (2049, 640, 384)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("mode", [fq.FP8Q_SCALE_FP32, fq.FP8Q_SCALE_POW2])
@pytest.mark.parametrize("M,F,K", DENSE)
def test_dense_tiles(M, F, K, mode, pow2):
    assert on_tiles(M, F)
    a, sa, b, sb = operands(M, F, K, 2000 + M, pow2)
    r = call_of(pow2)(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True, scale_mode=mode)
    check(r, a, sa, b, sb, mode)


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("want", [dict(), dict(with_gu=True), dict(with_codes=True),
                                  dict(with_h=False, with_codes=True),
                                  dict(with_h=False, with_gu=True),
                                  dict(with_h=False, with_gu=True, with_codes=True)])
def test_dense_tiles_each_result_alone(want, pow2):
    M, F, K = 333, 1536, 384
    assert on_tiles(M, F)
    ops = [t.cuda() for t in operands(M, F, K, 2100, pow2)]
    full = call_of(pow2)(*ops, with_gu=True, with_codes=True)
    r = call_of(pow2)(*ops, **want)
    assert (r.h is not None) == want.get("with_h", True)
    assert (r.gu is not None) == want.get("with_gu", False)
    assert (r.q is not None) == (r.s is not None) == want.get("with_codes", False)
    for got, ref in zip(r, full):
        assert got is None or torch.equal(got, ref)


@pytest.mark.parametrize("pow2", [False, True])
def test_dense_tiles_empty_sums_and_zero_rows(pow2):
    M, F = 1000, 1152
    assert on_tiles(M, F)
    floor = torch.tensor(2.0 ** -116 / 448, dtype=torch.float32)
    e8 = torch.empty(M, 0, dtype=torch.uint8, device="cuda")
    r = call_of(pow2)(e8, torch.empty(0, M, device="cuda"), e8.new_empty(2 * F, 0),
                      torch.empty(2 * F // 128, 0, device="cuda"), with_gu=True, with_codes=True)
    assert not r.h.any() and not r.gu.any() and not r.q.bitwise_and(0x7F).any()
    assert torch.equal(r.s.cpu(), floor.expand_as(r.s.cpu()))
    a, sa, b, sb = operands(M, F, 256, 2200, pow2)
    a[M // 2] = 0
    r = call_of(pow2)(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True)
    check(r, a, sa, b, sb, fq.FP8Q_SCALE_FP32)
    assert bool((r.s[:, M // 2].cpu() == floor).all())


def test_dense_tiles_large_magnitudes():
    # g of both signs up to thousands: exp overflows on one side, silu(g) = g on the other
    M, F, K = 300, 2048, 256
    assert on_tiles(M, F)
    a, sa, b, sb = operands(M, F, K, 2300)
    sa = sa * 500
    r = fq.fp8q_gemm_swiglu(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True)
    assert torch.isfinite(r.h.float()).all() and torch.isfinite(r.s).all()
    check(r, a, sa, b, sb, fq.FP8Q_SCALE_FP32)


@pytest.mark.parametrize("M", [130, 257, 383])
@pytest.mark.parametrize("pow2", [False, True])
def test_dense_tiles_strides_and_padding(M, pow2):
    F, K = 3200, 384
    assert on_tiles(M, F)
    a, sa, b, sb = operands(M, F, K, 2400, pow2)
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
    r = call_of(pow2)(av, sav, bv, sbv, h=h, gu=gu, q=q, s=s)
    check(r, a, sa, b, sb, fq.FP8Q_SCALE_FP32)
    for view, buf, fill in ((h, hb, 7.0), (gu, gub, 7.0), (q, qb, 0xCD), (s, sbuf, -3.0)):
        view.fill_(fill)
        assert bool((buf == fill).all()), "wrote outside its result"


@pytest.mark.parametrize("where", ["sa", "sb gate", "sb up"])
@pytest.mark.parametrize("grouped", [False, True])
def test_pow2_precondition_is_reported_on_tiles(grouped, where):
    M, F, K = 300, 2048, 256
    assert on_tiles(M, F)
    a, sa, b, sb = operands(M, F, K, 2500, True)
    if where == "sa":
        sa[1, 299] = 0.3
    else:
        sb[5 if where == "sb gate" else F // 128 + 5, 1] = 0.3
    ops = [t.cuda() for t in (a, sa, b, sb)]
    if grouped:
        offs = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        fq.fp8q_grouped_gemm_swiglu_pow2(ops[0], ops[1], ops[2][None], ops[3][None], offs)
    else:
        fq.fp8q_gemm_swiglu_pow2(*ops)
    assert B.fp8q_sync_status() == B.FP8Q_ERR_INVALID
    assert B.fp8q_sync_status() == 0


@pytest.mark.parametrize("pow2", [False, True])
def test_dense_tiles_several_per_pair(pow2):
    # 272 tiles on 76 pairs: the exchanges' phases, the staging behind tensor stores and both
    # accumulators are used again
    M, F, K = 4100, 2048, 256
    assert (M + 255) // 256 * (F // 128) > 3 * SMS // 2 and on_tiles(M, F)
    a, sa, b, sb = operands(M, F, K, 2600, pow2)
    r = call_of(pow2)(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True)
    check(r, a, sa, b, sb, fq.FP8Q_SCALE_FP32)


@pytest.mark.parametrize("pow2", [False, True])
def test_expert_tiles_several_per_pair(pow2):
    M, F, K, offs = 3001, 1920, 256, [0, 1, 700, 700, 2047, 3001]
    G = len(offs) - 1
    assert sum((hi - lo + 255) // 256 for lo, hi in zip(offs, offs[1:])) * (F // 128) > SMS
    a, sa, b, sb = operands(M, F, K, 2700, pow2, experts=G)
    call = fq.fp8q_grouped_gemm_swiglu_pow2 if pow2 else fq.fp8q_grouped_gemm_swiglu
    r = call(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), torch.tensor(offs, dtype=torch.int32, device="cuda"),
             with_gu=True, with_codes=True)
    for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
        if hi > lo:
            check(r, a[lo:hi], sa[:, lo:hi], b[e], sb[e], fq.FP8Q_SCALE_FP32, slice(lo, hi))


@pytest.mark.parametrize("pow2", [False, True])
def test_dense_tiles_on_streams_and_in_graphs(pow2):
    M, F, K = 700, 1152, 640
    assert on_tiles(M, F)
    ops = [[t.cuda() for t in operands(M, F, K, 2800 + i, pow2)] for i in range(2)]
    dh, gu = (t.cuda() for t in bwd_inputs(512, 512, 2810))

    def calls(o):
        # each kernel may set itself up under the end of the one before
        return [*call_of(pow2)(*o, with_gu=True, with_codes=True), *fq.fp8q_swiglu_bwd(dh, gu, with_d=True),
                *call_of(pow2)(*o, with_h=True)][:-3]

    want = [calls(o) for o in ops]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in ops], [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(calls(ops[i]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls(ops[0])
    for t in captured:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got[0].append(captured)
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(g, want[i]))


# ------------------------------------------------------------------ few tokens: every split, rings used again
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("M,F,K,split", [(9, 640, 4992, 4), (24, 640, 4992, 4), (50, 640, 4992, 4),
                                         (1, 7168, 2688, 2), (32, 7168, 2688, 2), (64, 7168, 2688, 2),
                                         (16, 10240, 1536, 1), (17, 10240, 1536, 1), (33, 10240, 1536, 1),
                                         (1000, 512, 2688, 2), (4000, 128, 1280, 2), (200, 1280, 2560, 2)])
def test_few_tokens_every_split(M, F, K, split, pow2):
    assert not on_tiles(M, F) and k_split(M, F) == split
    a, sa, b, sb = operands(M, F, K, 2900 + M, pow2)
    r = call_of(pow2)(a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), with_gu=True, with_codes=True)
    check(r, a, sa, b, sb, fq.FP8Q_SCALE_FP32)


# ------------------------------------------------------------------ backward: several rounds of tiles
def test_backward_several_tiles_per_cluster():
    T, F = 2048, 2944
    assert T // 128 * (F // 128) > 2 * SMS
    dh, gu = bwd_inputs(T, F, 3000)
    d_dh, d_gu = dh.cuda(), gu.cuda()
    full = fq.fp8q_swiglu_bwd(d_dh, d_gu, with_d=True)
    check_bwd(full, dh, gu, fq.FP8Q_SCALE_FP32)
    names = ("with_d", "with_rows", "with_cols", "with_h")
    for bits in range(1, 16):
        want = {n: bool(bits >> i & 1) for i, n in enumerate(names)}
        for _ in range(3):
            r = fq.fp8q_swiglu_bwd(d_dh, d_gu, **want)
            for got, ref in zip(r, full):
                assert got is None or torch.equal(got, ref), want


@pytest.mark.parametrize("mode", [fq.FP8Q_SCALE_FP32, fq.FP8Q_SCALE_POW2])
def test_backward_odd_tokens_several_tiles_per_cluster(mode):
    T, F = 5003, 1024
    assert (T + 127) // 128 * (F // 128) > 2 * SMS
    dh, gu = bwd_inputs(T, F, 3100)
    r = fq.fp8q_swiglu_bwd(dh.cuda(), gu.cuda(), with_d=True, with_cols=False, with_h=False, scale_mode=mode)
    check_bwd(r, dh, gu, mode)
