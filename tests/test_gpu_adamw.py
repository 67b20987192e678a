"""The AdamW step over lists of tensors against plain 64-bit arithmetic.

Tolerances (u = 2^-24):
  m : one product, one fused multiply-add, g * grad_scale and the factors' own rounding:
      6 u (|b1 m| + |(1 - b1) g|).  v the same with 8 u (all terms positive).
  p : the step's relative error: m's, half of v's, the two corrections, the root, the sum
      and the quotient: 14 u of |m-terms| / (sqrt(v) / .. + eps), lr's rounding and the
      products 4 u more; and 3 u |p|.
  BF16 half a unit, 2^-8 of the value; E4M3 half a step, 2^-4 of the value or 2^-10 of
  the scale below the smallest normal code, of a value that for sqrt(v) is first raised
  to the smallest code (up to 2^-9 of the scale away: two of those half steps).
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
KIND = {"bf16": BF, "fp32": FP}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


def near(got, want, tol, what):
    err = (got.double().cpu() - want).abs()
    ok = err <= tol
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} outside, max err/tol " \
        f"{float((err / tol.clamp_min(1e-300)).max()):.3g}"


def spread(s, n):
    return s.double().cpu().repeat_interleave(128)[:n]


class State:
    """Parameters, gradients and moments of a list of sizes on the GPU."""

    def __init__(self, sizes, p="fp32", g="fp32", state="fp32", copy=False, seed=0, offset=0):
        gen = torch.Generator().manual_seed(seed)
        self.kind, self.sizes, self.gen = state, sizes, gen

        def put(t, dtype):
            # `offset` elements behind an aligned address
            buf = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
            buf[offset:].copy_(t)
            return buf[offset:]

        self.put, self.tg = put, KIND[g]
        self.p = [put(torch.randn(n, generator=gen), KIND[p]) for n in sizes]
        self.new_gradients()
        tm = torch.uint8 if state == "e4m3" else KIND[state]
        self.m, self.v = ([put(torch.zeros(n), tm) for n in sizes] for _ in range(2))
        groups = [(n + 127) // 128 for n in sizes]
        self.ms, self.vs = ([torch.zeros(n, device="cuda") for n in groups] if state == "e4m3" else None
                            for _ in range(2))
        self.copy = [put(torch.zeros(n), BF) for n in sizes] if copy else None

    def new_gradients(self):
        r = lambda n: torch.randn(n, generator=self.gen)  # noqa: E731
        self.g = [self.put(r(n) * torch.exp(2 * r(n)) * 1e-3, self.tg) for n in self.sizes]

    def values(self, i):
        """m and v of tensor i in 64 bits."""
        m, v = self.m[i], self.v[i]
        if self.kind != "e4m3":
            return m.double().cpu(), v.double().cpu()
        n = m.numel()
        return (m.view(E4M3).double().cpu() * spread(self.ms[i], n),
                (v.view(E4M3).double().cpu() * spread(self.vs[i], n)) ** 2)

    def step(self, **kw):
        fq.fp8q_adamw(self.p, self.g, self.m, self.v, m_scales=self.ms, v_scales=self.vs, copies=self.copy, **kw)


HYPER = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def check_codes(q, s, want, tol, root, what):
    """Codes and scales of groups of 128 of values `want` known to `tol`."""
    n = want.numel()
    pad = -n % 128
    groups = torch.nn.functional.pad(want.abs(), (0, pad)).reshape(-1, 128).amax(1).clamp_min(2.0 ** -116)
    slack = torch.nn.functional.pad(tol, (0, pad)).reshape(-1, 128).amax(1)
    near(s, groups / 448, slack / 448 + 4 * U * groups / 448, what + " scales")
    sc = spread(s, n)
    if root:  # by the call's definition a positive root is at least the smallest code, 2^-9 of the scale
        want = torch.where(want > 0, torch.maximum(want, 2.0 ** -9 * sc), want)
    near(q.view(E4M3).double().cpu() * sc, want,
         torch.maximum(2.0 ** -4 * (want.abs() + tol), 2.0 ** -10 * sc) + tol + 8 * U * want.abs(), what + " codes")
    if root:
        code = q.view(E4M3).double().cpu()
        assert bool((code >= 0).all())
        assert bool((code[want > tol] >= 2.0 ** -9).all()), "a positive root became 0"


def check_step(st, step, hyper=HYPER, scale=1.0):
    """Makes one step and compares it with the same step in 64 bits."""
    before = [(p.double().cpu(), *st.values(i)) for i, p in enumerate(st.p)]
    st.step(step=step, **hyper, **({} if scale == 1.0 else dict(grad_scale=torch.tensor([scale], device="cuda"))))
    (b1, b2), lr, eps, wd = hyper["betas"], hyper["lr"], hyper["eps"], hyper["weight_decay"]
    for i, (p, m, v) in enumerate(before):
        g = st.g[i].double().cpu() * float(torch.tensor(scale, dtype=FP))
        size = (b1 * m).abs() + ((1 - b1) * g).abs()
        m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        tm, tv = 6 * U * size + 1e-44, 8 * U * v1 + 1e-44
        den = (v1 / (1 - b2 ** step)).sqrt() + eps
        move = m1 / (1 - b1 ** step) / den
        want = p - lr * (wd * p + move)
        tol = abs(lr) * 18 * U * size / (1 - b1 ** step) / den + 3 * U * (p.abs() + want.abs())
        if st.p[i].dtype == BF:
            tol = tol + 2.0 ** -8 * (want.abs() + tol)
        near(st.p[i], want, tol, f"p[{i}]")
        if st.copy is not None:
            near(st.copy[i], want, tol + 2.0 ** -8 * (want.abs() + tol), f"copy[{i}]")
        if st.kind == "e4m3":
            check_codes(st.m[i], st.ms[i], m1, tm, False, f"m[{i}]")
            check_codes(st.v[i], st.vs[i], v1.sqrt(), 8 * U * v1.sqrt() + 1e-22, True, f"v[{i}]")
        else:
            r = 2.0 ** -8 if st.kind == "bf16" else 0.0
            near(st.m[i], m1, tm + r * (m1.abs() + tm), f"m[{i}]")
            near(st.v[i], v1, tv + r * (v1 + tv), f"v[{i}]")


SIZES = [1, 7, 8, 127, 128, 129, 1000, 4095, 4096, 4097, 12345, 0, 70001]


@pytest.mark.parametrize("state", ["fp32", "bf16", "e4m3"])
@pytest.mark.parametrize("p,g,copy", [("fp32", "fp32", True), ("fp32", "bf16", False), ("bf16", "fp32", False),
                                      ("bf16", "bf16", False)])
def test_steps(p, g, copy, state):
    st = State(SIZES, p, g, state, copy)
    for step in (1, 2, 3):
        check_step(st, step, scale=1.0 if step == 1 else 0.37)
        st.new_gradients()
    check_step(st, 100000)


@pytest.mark.parametrize("state", ["fp32", "bf16", "e4m3"])
@pytest.mark.parametrize("offset", [1, 3, 4])
def test_addresses_off_16_bytes(state, offset):
    st = State([1, 130, 4099, 9000], "fp32", "bf16", state, True, seed=1, offset=offset)
    check_step(st, 1)
    check_step(st, 2)


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_many_tensors(state):
    # more than one launch takes, an empty one among them
    sizes = [(i * 37) % 301 for i in range(300)]
    check_step(State(sizes, "fp32", "fp32", state, True, seed=2), 1)


def test_moments_are_rounded_after_every_operation():
    # m and v are defined as FP32 products and sums, each rounded (in 64 bits here, then to FP32): the
    # same bits, so that 8-bit codes do not hang on how a compiler joins operations
    st = State([100001], seed=11)
    f = lambda t: t.float().double()  # noqa: E731
    b1, b2 = (float(torch.tensor(b, dtype=FP)) for b in (0.9, 0.95))
    o1, o2 = (float(torch.tensor(1 - b, dtype=FP)) for b in (0.9, 0.95))
    scale = torch.tensor([0.3], device="cuda")
    for step in (1, 2, 3):
        m, v = (t.double().cpu() for t in (st.m[0], st.v[0]))
        d = f(st.g[0].double().cpu() * float(scale))
        st.step(step=step, grad_scale=scale, **HYPER)
        m, v = f(f(b1 * m) + f(o1 * d)), f(f(b2 * v) + f(f(o2 * d) * d))
        assert torch.equal(st.m[0].double().cpu(), m) and torch.equal(st.v[0].double().cpu(), v)
        st.new_gradients()


def test_the_same_as_one_by_one():
    for state in ("fp32", "e4m3"):
        a, b = (State([5000, 333, 20000], "fp32", "fp32", state, seed=3) for _ in range(2))
        a.step(step=1, **HYPER)
        for i in range(3):
            fq.fp8q_adamw([b.p[i]], (b.g[i],), [b.m[i]], [b.v[i]], step=1, **HYPER,
                          m_scales=b.ms and [b.ms[i]], v_scales=b.vs and [b.vs[i]])
        for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v):
            assert torch.equal(x, y)


def test_zero_gradients_and_zero_moments():
    for state in ("fp32", "bf16", "e4m3"):
        st = State([300], "fp32", "fp32", state, seed=4)
        st.g[0].zero_()
        p = st.p[0].clone()
        st.step(step=1, **HYPER)
        near(st.p[0], p.double().cpu() * (1 - 1e-3), 4 * U * p.double().abs().cpu(), "decay alone")
        assert all(not (t.bitwise_and(0x7F) if t.dtype == torch.uint8 else t).any() for t in st.m + st.v)


@pytest.mark.parametrize("state", ["fp32", "bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_gradients_that_are_no_numbers(state, bad):
    # they show in their parameter and leave the others alone (8 bits: an infinite one the other groups)
    a, b = (State([300, 40], "fp32", "fp32", state, seed=6) for _ in range(2))
    a.g[0][133], b.g[0][133] = bad, 0.0
    keep = torch.ones(300, dtype=torch.bool, device="cuda")
    keep[133] = False
    for step in (1, 2):
        a.step(step=step, **HYPER)
        b.step(step=step, **HYPER)
        if state == "e4m3" and bad == float("inf"):
            keep[128:256] = False
        assert torch.isnan(a.p[0][133])
        for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v):
            kept = keep if x.numel() == 300 else slice(None)
            assert torch.equal(x[kept], y[kept])


def test_small_gradients_in_a_group_keep_their_denominator():
    # one value of a group ten million times larger than the others: their root is below half the
    # smallest code, and a step of theirs stays of the order of lr
    st = State([128], "fp32", "fp32", "e4m3", seed=5)
    hyper = dict(lr=1e-2, betas=(0.9, 0.95), eps=1e-12, weight_decay=0.0)
    for step in range(1, 30):
        st.g[0].fill_(1e-7)
        st.g[0][5] = 1.0 if step < 3 else 0.0
        before = st.p[0].clone()
        check_step(st, step, hyper)
        assert float((st.p[0] - before).abs().max()) < 10 * hyper["lr"]
        assert bool((st.v[0].view(E4M3).float() > 0).all())


@pytest.mark.parametrize("state", ["fp32", "e4m3"])
def test_zero_betas_and_odd_hyperparameters(state):
    st = State([1000], "fp32", "fp32", state, seed=6)
    check_step(st, 1, dict(lr=0.5, betas=(0.0, 0.0), eps=1e-3, weight_decay=0.0))
    check_step(st, 7, dict(lr=-0.1, betas=(0.5, 0.999), eps=1.0, weight_decay=2.0))


@pytest.mark.parametrize("beta2", [0.95, 0.999, 0.99999])
def test_step_and_rate_in_device_memory(beta2):
    hyper = dict(betas=(0.9, beta2), eps=1e-8, weight_decay=0.1)
    for step in (1, 2, 17, 5000, 10 ** 7):
        a, b = (State([3000], seed=7) for _ in range(2))
        a.step(step=step, lr=3e-3, **hyper)
        b.step(step=torch.tensor(step, device="cuda"), lr=torch.tensor([3e-3], device="cuda"), **hyper)
        # both moves are right to 18 u of their terms; FP32 corrections on the device add 8 u
        p0 = State([3000], seed=7).p[0].double().cpu()
        near(b.p[0], a.p[0].double().cpu(), 48 * U * ((a.p[0].double().cpu() - p0).abs() + 1e-2) + 2 * U * p0.abs(), "p")
        assert torch.equal(a.m[0], b.m[0]) and torch.equal(a.v[0], b.v[0])


def test_captured_call_follows_its_tensors():
    lr, step = torch.full((1,), 1e-2, device="cuda"), torch.ones(1, dtype=torch.long, device="cuda")
    hyper = dict(betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    a, b = (State([5000, 129], "fp32", "fp32", "e4m3", True, seed=8) for _ in range(2))
    a.step(step=step, lr=lr, **hyper)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        a.step(step=step, lr=lr, **hyper)
    b.step(step=torch.ones(1, dtype=torch.long, device="cuda"), lr=lr, **hyper)
    for k in (2, 3, 4):
        lr.fill_(1e-2 / k)
        graph.replay()
        b.step(step=torch.tensor([k], device="cuda"), lr=lr, **hyper)
        for x, y in zip(a.p + a.m + a.v + a.ms + a.vs + a.copy, b.p + b.m + b.v + b.ms + b.vs + b.copy):
            assert torch.equal(x, y)


def test_more_than_2_31_values():
    n = (1 << 31) + 4097 + 5
    p, g = (torch.empty(n, dtype=BF, device="cuda") for _ in range(2))
    p.fill_(1.0)
    g.fill_(0.0)
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    ms, vs = (torch.zeros((n + 127) // 128, device="cuda") for _ in range(2))
    tail = 9000
    gen = torch.Generator().manual_seed(9)
    g[-tail:].copy_(torch.randn(tail, generator=gen) * 1e-3)
    g[:tail].copy_(torch.randn(tail, generator=gen) * 1e-3)
    at = (n - tail) // 128 * 128  # a group's start

    def small(sl):
        st = State([1], "bf16", "bf16", "e4m3")
        st.p, st.g = [p[sl].clone()], [g[sl].clone()]
        k = st.p[0].numel()
        st.m, st.v = ([torch.zeros(k, dtype=torch.uint8, device="cuda")] for _ in range(2))
        st.ms, st.vs = ([torch.zeros((k + 127) // 128, device="cuda")] for _ in range(2))
        st.step(step=1, **HYPER)
        return st

    ends = [(slice(at, n), slice(at // 128, None), small(slice(at, n))),
            (slice(0, 8192), slice(0, 64), small(slice(0, 8192)))]
    fq.fp8q_adamw([p], [g], [m], [v], m_scales=[ms], v_scales=[vs], step=1, **HYPER)
    for sl, groups, st in ends:
        for got, want in ((p[sl], st.p[0]), (m[sl], st.m[0]), (v[sl], st.v[0]), (ms[groups], st.ms[0]), (vs[groups], st.vs[0])):
            assert torch.equal(got, want)


def test_refusals_on_the_device():
    st = State([100, 200], seed=10)
    with pytest.raises(fq.FP8QError):  # the same tensor twice
        fq.fp8q_adamw([st.p[0]] * 2, [st.g[0]] * 2, [st.m[0]] * 2, [st.v[0]] * 2, step=1, lr=1e-3)
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8q_adamw([st.p[1][::2]], [st.g[0]], [st.m[0]], [st.v[0]], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="elements"):
        fq.fp8q_adamw([st.p[1]], [st.g[0]], [st.m[1]], [st.v[1]], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="need m_scales"):
        fq.fp8q_adamw([st.p[0]], [st.g[0]], [st.m[0].byte()], [st.v[0].byte()], step=1, lr=1e-3)
    with pytest.raises(ValueError, match="one element"):
        st.step(step=1, lr=1e-3, grad_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="Long"):
        st.step(step=torch.ones(1, device="cuda"), lr=1e-3)
    with pytest.raises(fq.FP8QError):
        st.step(step=0, lr=1e-3)


@pytest.mark.parametrize("state", ["bf16", "e4m3"])
def test_moments_of_fewer_bits_follow_their_gradients(state):
    """600 steps of normal gradients and 600 with half of each group a hundred times smaller, with the betas that the
    call takes by itself, against moments in 64 bits.  BF16: v rests where a step moves it by less than half its last
    place, (1 - b2) |g^2 / v - 1| < 2^-8, 8 % of v and 4 % of its root.  8 bits: the root rests while (1 - b2) |g^2 /
    v - 1| / 2 < 2^-4, g^2 up to 3.5 v, a factor of 1.87.  m: errors of half a step, 2^-4 and 2^-8 at most, 1 / sqrt(3)
    of that over many, of which the last 1 / (1 - b1^2) = 5.3 remain: 0.083 and 0.0052, and half as much again."""
    n, half = 128 * 64, torch.arange(128 * 64, device="cuda") % 128 < 64
    st = State([n], "fp32", "fp32", state, seed=20)
    g = torch.Generator(device="cuda").manual_seed(21)
    m, v = (torch.zeros(n, dtype=torch.double, device="cuda") for _ in range(2))
    bound, bound_m = (1.04, 0.0078) if state == "bf16" else (1.87, 0.125)

    def check():
        got_m, got_v = (t.cuda() for t in st.values(0))
        for part in (half, ~half):
            ratio = float(got_v[part].sqrt().mean() / v[part].sqrt().mean())
            assert 1 / bound < ratio < bound, ratio
            assert float((got_m - m)[part].norm() / m[part].norm()) < bound_m

    for step in range(1, 1201):
        st.g[0].normal_(generator=g)
        if step > 600:
            st.g[0][half] *= 0.01
        st.step(step=step, lr=1e-3)
        d = st.g[0].double()
        m, v = 0.9 * m + 0.1 * d, 0.95 * v + 0.05 * d * d
        if step == 600:
            check()
    check()


def test_betas_where_none_are_given():
    for state, betas in (("fp32", (0.9, 0.999)), ("bf16", (0.9, 0.95)), ("e4m3", (0.9, 0.95))):
        a, b = (State([3000], "fp32", "fp32", state, seed=22) for _ in range(2))
        for step in (1, 2):
            a.step(step=step, lr=1e-2)
            b.step(step=step, lr=1e-2, betas=betas)
        for x, y in zip(a.p + a.m + a.v, b.p + b.m + b.v):
            assert torch.equal(x, y)


@pytest.mark.parametrize("state", ["fp32", "bf16", "e4m3"])
@pytest.mark.parametrize("eps", [1e-30, 1e-40, 1e-60])
def test_zero_gradients_with_the_smallest_eps(state, eps):
    st = State([300], "fp32", "fp32", state, seed=23)
    st.g[0].zero_()
    p = st.p[0].clone()
    st.step(step=1, **{**HYPER, "eps": eps})
    near(st.p[0], p.double().cpu() * (1 - 1e-3), 4 * U * p.double().abs().cpu(), "decay alone")
