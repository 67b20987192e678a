"""Newton-Schulz orthogonalisation against the iteration in 64 bits.

Tolerance on |got - ref|_F / |ref|_F.  Three matrices are rounded to FP16 per
step (relative error at most 2^-11 in a unit of the last place, 2^-12 half a
unit, 2^-12 / sqrt(3) rms); an error in X, A or B enters the new X with a
weight of at most |a| + |b| + |c| = 10.3, and the roundings are independent:
  sqrt(3 * 5) * 2^-12 / sqrt(3) * 10.3 = 5.6e-3  ->  6e-3 for FP32 results,
and 2^-8 / sqrt(3) = 2.3e-3 more (in quadrature) for BF16 ones: 6.5e-3.
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu
COEFFS = (3.4445, -4.7750, 2.0315)
TOL = {torch.float32: 6e-3, torch.bfloat16: 6.5e-3}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def reference(g, steps=5, coeffs=COEFFS, eps=1e-7):
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    x = x / (torch.linalg.matrix_norm(x)[..., None, None] + eps)
    for _ in range(steps):
        A = x @ x.mT
        x = a * x + (b * A + c * A @ A) @ x
    return x.mT if tall else x


def gradient(*shape, seed=0, dtype=torch.float32, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    m, n = shape[-2:]
    r = max(1, min(m, n) // 4)
    low = torch.randn(*shape[:-2], m, r, generator=g) @ torch.randn(*shape[:-2], r, n, generator=g)
    return ((low / r ** 0.5 + 0.5 * torch.randn(*shape, generator=g)) * scale).to(dtype)


def rel(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("out", [fq.FP8Q_OUT_BF16, fq.FP8Q_OUT_FP32])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 70), (65, 1), (8, 8), (33, 64), (64, 33), (127, 129),
                                 (128, 128), (256, 256), (257, 300), (300, 257), (100, 1001),
                                 (1001, 100), (513, 640)])
def test_against_64_bits(m, n, dtype, out):
    g = gradient(m, n, seed=m * 7 + n, dtype=dtype)
    x = fq.fp8q_newton_schulz(g.cuda(), out_dtype=out)
    assert x.shape == g.shape and x.dtype == (torch.bfloat16 if out == fq.FP8Q_OUT_BF16
                                              else torch.float32)
    assert rel(x, reference(g)) <= TOL[x.dtype]


@pytest.mark.parametrize("steps", [1, 2, 3, 10])
def test_steps_and_coefficients(steps):
    g = gradient(150, 260, seed=steps)
    x = fq.fp8q_newton_schulz(g.cuda(), steps=steps, out_dtype=fq.FP8Q_OUT_FP32)
    assert rel(x, reference(g, steps)) <= TOL[torch.float32] * max(1, steps / 5) ** 0.5
    # the cubic iteration, whose fixed point is the orthogonal factor itself
    x = fq.fp8q_newton_schulz(g.cuda(), steps=steps, coeffs=(1.5, -0.5, 0.0),
                              out_dtype=fq.FP8Q_OUT_FP32)
    assert rel(x, reference(g, steps, (1.5, -0.5, 0.0))) <= TOL[torch.float32]


def test_result_is_nearly_orthogonal():
    g = gradient(200, 500, seed=3)
    s = torch.linalg.svdvals(fq.fp8q_newton_schulz(g.cuda(), out_dtype=fq.FP8Q_OUT_FP32).double())
    # five quintic steps map [0.01, 1] into [0.65, 1.25]
    assert float(s.min()) > 0.6 and float(s.max()) < 1.3


@pytest.mark.parametrize("m,n", [(96, 200), (200, 96), (300, 300)])
def test_batch_and_single_matrices(m, n):
    # how the sums along K are split follows the whole call's work, so a matrix
    # of a batch and the same matrix alone may differ by roundings: both are
    # held to the reference, and each call repeats bit by bit
    g = gradient(5, m, n, seed=4).cuda()
    g[2] = 0
    x = fq.fp8q_newton_schulz(g)
    assert torch.equal(x, fq.fp8q_newton_schulz(g))
    for i in (0, 1, 3, 4):
        ref = reference(g[i].cpu())
        assert rel(x[i], ref) <= TOL[x.dtype]
        assert rel(fq.fp8q_newton_schulz(g[i].contiguous()), ref) <= TOL[x.dtype]
    assert not x[2].any(), "a zero gradient gives a zero update"
    assert fq.fp8q_newton_schulz(g[:0]).shape == (0, m, n)


@pytest.mark.parametrize("B,m,n", [(400, 40, 50), (200, 64, 200), (90, 130, 70), (40, 300, 320),
                                   (20, 520, 300)])
def test_many_small_matrices(B, m, n):
    # several rounds of tiles per pair, one or a few K blocks each: the kernel's
    # producer, MMA, epilogue and counting warps run far apart from one another
    g = gradient(B, m, n, seed=11).cuda()
    x = fq.fp8q_newton_schulz(g)
    assert rel(x, reference(g.cpu())) <= TOL[x.dtype]
    assert torch.equal(x, fq.fp8q_newton_schulz(g))


@pytest.mark.parametrize("m,n", [(1100, 1900), (1700, 2300), (768, 9000), (9001, 260), (100, 20000),
                                 (1280, 16384)])
def test_split_and_wide_tiles(m, n):
    # long sums and more than one tile width in one call
    g = gradient(m, n, seed=12)
    x = fq.fp8q_newton_schulz(g.cuda(), out_dtype=fq.FP8Q_OUT_FP32)
    assert rel(x, reference(g)) <= TOL[torch.float32]
    assert torch.equal(x, fq.fp8q_newton_schulz(g.cuda(), out_dtype=fq.FP8Q_OUT_FP32))


def test_tall_is_the_transpose_of_wide():
    g = gradient(130, 300, seed=5).cuda()
    assert torch.equal(fq.fp8q_newton_schulz(g.t().contiguous()).t(), fq.fp8q_newton_schulz(g))


@pytest.mark.parametrize("scale", [1e-12, 1e6])
def test_scale_of_the_gradient_does_not_matter(scale):
    g = gradient(96, 160, seed=6, scale=scale)
    x = fq.fp8q_newton_schulz(g.cuda(), eps=0.0, out_dtype=fq.FP8Q_OUT_FP32)
    assert rel(x, reference(g, eps=0.0)) <= TOL[torch.float32]


def test_entries_far_below_the_largest():
    # one entry holds nearly all of the norm; the rest are 1e-4 of it, far below
    # FP16's normal range without the stored matrices' scale
    g = gradient(64, 96, seed=7, scale=1e-4)
    g[3, 5] = 1.0
    x = fq.fp8q_newton_schulz(g.cuda(), out_dtype=fq.FP8Q_OUT_FP32)
    assert rel(x, reference(g)) <= TOL[torch.float32]


@pytest.mark.parametrize("m,n", [(70, 133), (133, 70)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strides_and_padding(m, n, dtype):
    g = gradient(3, m, n, seed=8, dtype=dtype)
    gbuf = torch.full((3, m + 2, n + 5), float("nan"), dtype=dtype, device="cuda")
    obuf = torch.full((3, m + 1, n + 3), 7.0, dtype=dtype, device="cuda")
    gv, ov = gbuf[:, 1:m + 1, 3:n + 3], obuf[:, :m, 1:n + 1]
    gv.copy_(g)
    od = fq.FP8Q_OUT_FP32 if dtype == torch.float32 else fq.FP8Q_OUT_BF16
    fq.fp8q_newton_schulz(gv, out=ov, out_dtype=od)
    assert torch.equal(ov, fq.fp8q_newton_schulz(g.cuda(), out_dtype=od))
    ov.fill_(7.0)
    assert bool((obuf == 7.0).all()), "wrote outside its result"


def test_non_finite_entries_stay_in_their_matrix():
    g = gradient(3, 40, 50, seed=9).cuda()
    want = fq.fp8q_newton_schulz(g)
    g[1, 4, 5] = float("inf")
    got = fq.fp8q_newton_schulz(g)
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert not torch.isfinite(got[1].float()).all()


def test_streams_capture_and_kept_workspace():
    g = gradient(2, 160, 300, seed=10).cuda()
    ws = torch.full((fq.fp8q_newton_schulz_workspace_bytes(2, 160, 300),), 0xFF, dtype=torch.uint8,
                    device="cuda")  # NaN patterns: nothing may be read before it is written
    want = fq.fp8q_newton_schulz(g)
    assert torch.equal(fq.fp8q_newton_schulz(g, workspace=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = fq.fp8q_newton_schulz(g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fq.fp8q_newton_schulz(g, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again, want) and torch.equal(captured, want)


def test_two_streams_at_once():
    # each call fills the GPU with kernels that wait for their own CTAs
    gs = [gradient(1500, 2000, seed=20 + i).cuda() for i in range(2)]
    want = [fq.fp8q_newton_schulz(g) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fq.fp8q_newton_schulz(gs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_binding_refuses():
    g = gradient(8, 16).cuda()
    with pytest.raises(ValueError):
        fq.fp8q_newton_schulz(g.half())
    with pytest.raises(ValueError):
        fq.fp8q_newton_schulz(g.t())
    with pytest.raises(ValueError):
        fq.fp8q_newton_schulz(g[0])
    with pytest.raises(ValueError):
        fq.fp8q_newton_schulz(g, out=torch.empty(8, 16, device="cuda"))  # FP32, BF16 asked for
    for bad, status in ((dict(steps=0), B.FP8Q_ERR_INVALID), (dict(eps=-1.0), B.FP8Q_ERR_INVALID),
                        (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
                         B.FP8Q_ERR_SHAPE)):
        with pytest.raises(fq.FP8QError) as err:
            fq.fp8q_newton_schulz(g, **bad)
        assert err.value.status == status
