"""The expert router and its backward pass against plain 64-bit arithmetic.

The choice, counts, offsets and order are whole numbers and have to be equal; the
reference sorts the FP32 logits, equal ones by index.

Tolerances (u = 2^-24): exp(l - m) with the difference rounded, |l - m| u, and exp's own
2 u; sums of up to E terms, 32 in a lane and 5 levels of a tree, 40 u; a reciprocal and
products: a weight is right to (60 + 2 |l - m|) u of itself (sigmoid: 2 |l| for the same
reason, and its complement likewise), with 1e-37 for what underflows.
The loss sums T such probabilities per expert, all positive: ceil(T / 152 / 16) of them
in a warp, 16 + 152 partial sums, and the experts in a tree: at most (T / 2432 + 260 +
2 * 60) u.  Gradients: the factors above on every term, 100 u more for the sums, of the
sum of magnitudes.
"""
import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq
from test_gpu_swiglu import padded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32
BIG = torch.finfo(FP).max
SOFT, SIG = 0, 1


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


def make(T, E, dtype, seed, masked):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2 + torch.randn(E, generator=g)
    valid = None
    if masked and T:
        valid = torch.rand(T, generator=g) > 0.2
        l = torch.where((torch.rand(T, 1, generator=g) < 0.3) & (torch.rand(T, E, generator=g) < 0.6), float("-inf"), l)
        l[torch.rand(T, generator=g) < 0.1] = float("-inf")
    return l.to(dtype), valid


def parts(l, valid, score):
    """Open experts, clamped logits and the logarithms of their scores in 64 bits."""
    may = l.float() > float("-inf")
    if valid is not None:
        may = may & valid[:, None]
    x = l.double().clamp_max(BIG)
    x = torch.where(may, x, float("-inf"))
    log_s = torch.nn.functional.logsigmoid(x) if score == SIG else x - torch.logsumexp(x, 1, keepdim=True)
    return may, x, torch.where(may, log_s, float("-inf"))


def reference(l, valid, k, score, normalise, scale):
    T, E = l.shape
    may, x, log_s = parts(l, valid, score)
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    has = may.gather(1, idx)
    w = torch.where(has, log_s.gather(1, idx), float("-inf"))
    w = torch.softmax(w, 1).nan_to_num(0.0) if normalise else torch.exp(w)
    idx = torch.where(has, idx, -1)
    flat = torch.where(has, idx, E).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    n = int(counts.sum())
    order[n:] = -1
    tokens = int(has[:, 0].sum()) if T else 0
    p = torch.softmax(log_s, 1).nan_to_num(0.0)
    loss = E * float((counts / max(n, 1) * p.sum(0)).sum()) / max(tokens, 1)
    return dict(idx=idx, weight=w * scale, counts=counts, offs=torch.cat([torch.zeros(1).long(), counts.cumsum(0)]),
                order=order, slot=torch.where(has, slot.reshape(T, k), -1), tokens=torch.tensor([tokens]),
                loss=torch.tensor([loss], dtype=torch.double))


def check(r, l, valid, k, score, normalise, scale):
    want = reference(l, valid, k, score, normalise, scale)
    for name in ("idx", "counts", "offs", "order", "slot", "tokens"):
        got = getattr(r, name)
        assert got.dtype == torch.int32 and torch.equal(got.cpu().long(), want[name]), name
    may, x, _ = parts(l, valid, score)
    at = want["idx"].clamp_min(0)
    val = torch.where(want["idx"] >= 0, x.gather(1, at) if l.shape[0] else x[:, :k], 0.0)
    top = x.amax(1, keepdim=True).clamp_min(-BIG) if l.shape[0] else x[:, :1]
    reach = (val.abs() if score == SIG else (top - val).abs()).clamp_max(200)
    far = reach.amax(1, keepdim=True) if normalise else reach
    near(r.weight, want["weight"], (60 + 2 * reach + 2 * far) * U * want["weight"].abs() + 1e-37 * scale, "weight")
    near(r.loss, want["loss"], (l.shape[0] / 2432 + 380 + 2 * 40) * U * want["loss"].abs() + 1e-37, "loss")


GRID = [(1, 1, 1, FP), (1, 256, 8, FP), (2, 8, 2, BF), (15, 3, 3, FP), (64, 64, 6, BF), (65, 64, 6, FP), (64, 33, 32, FP),
        (66, 128, 1, BF), (333, 64, 6, BF), (777, 160, 8, FP), (1000, 7, 2, FP), (2431, 16, 1, BF), (2433, 16, 4, FP),
        (5003, 100, 5, BF), (300, 512, 12, FP), (257, 1024, 32, FP), (70, 1000, 16, BF), (20000, 256, 8, FP),
        # one CTA, a cluster and two launches on both sides of where each ends
        (32, 256, 8, FP), (33, 200, 7, FP), (200, 256, 8, BF), (256, 256, 8, FP), (257, 256, 8, FP), (17, 600, 5, FP),
        (33, 512, 8, FP), (255, 400, 9, BF), (256, 512, 32, FP), (257, 512, 3, FP), (32, 1024, 8, FP), (33, 1000, 8, BF)]


@pytest.mark.parametrize("T,E,k,dtype", GRID)
@pytest.mark.parametrize("score,normalise,masked", [(SOFT, True, False), (SIG, True, True), (SOFT, False, True),
                                                    (SIG, False, False)])
def test_forward(T, E, k, dtype, score, normalise, masked):
    l, valid = make(T, E, dtype, T + E, masked)
    r = fq.fp8q_route(l.cuda(), k, score=score, normalise=normalise, scale=2.5, valid=None if valid is None else valid.cuda())
    check(r, l, valid, k, score, normalise, 2.5)


@pytest.mark.parametrize("T", [5, 400])
def test_ties_take_the_lowest_index(T):
    for E in (8, 40, 300):
        l = torch.zeros(T, E)
        l[1::2] = -0.0
        l[2] = torch.arange(E) % 3
        l[3] = -torch.zeros(E) * (torch.arange(E) % 2)
        check(fq.fp8q_route(l.cuda(), 5), l, None, 5, SOFT, True, 1.0)
        l = torch.randint(0, 3, (T, E), generator=torch.Generator().manual_seed(1)).to(BF)
        check(fq.fp8q_route(l.cuda(), 5, score=SIG), l, None, 5, SIG, True, 1.0)


@pytest.mark.parametrize("T", [5, 400])
@pytest.mark.parametrize("E,k", [(8, 8), (20, 3), (100, 8), (256, 1), (256, 32), (400, 16), (700, 31), (1024, 8), (1024, 32)])
@pytest.mark.parametrize("steps", [1, 4, 300])
def test_logits_that_differ_in_their_last_bits(T, E, k, steps):
    # a few values and multiples of a unit in their last place, both signs, equal ones among them:
    # groups that agree in the upper bits end inside the choice, at its end, behind more than 32
    g = torch.Generator().manual_seed(E * k + steps)
    l = torch.randint(-3, 4, (T, E), generator=g).float()
    l = l * (1 + torch.randint(0, steps, (T, E), generator=g) * 2.0 ** -23)
    l[:, E // 2] = -0.0
    l[T // 2] = 1.0
    l[T // 3, : E - 1] = float("-inf")
    out = fq.fp8q_route(l.cuda(), k)
    order = torch.sort(l.double() + 0.0, dim=1, descending=True, stable=True)
    want = torch.where(order.values > float("-inf"), order.indices, -1)[:, :k].int()
    assert torch.equal(out.idx.cpu(), want)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("E", [16, 300, 1024])
def test_infinity_counts_as_the_largest_value(E, dtype):
    # equal to it, so the lower index comes first; a weight has six roundings, 1e-6 of 0.2 at most
    l = torch.zeros(40, E, dtype=dtype)
    l[:, 3] = l[:, 7] = torch.finfo(FP).max if dtype == FP else float("inf")
    l[:, 2] = l[:, 5] = l[:, 9] = float("inf")
    out = fq.fp8q_route(l.cuda(), 6)
    assert torch.equal(out.idx.cpu(), torch.tensor([[2, 3, 5, 7, 9, 0]], dtype=torch.int32).expand(40, 6))
    near(out.weight, torch.tensor([[0.2] * 5 + [0.0]], dtype=torch.float64).expand(40, 6), torch.tensor(1e-6), "weight")


@pytest.mark.parametrize("T", [6, 300])
@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("dtype", [FP, BF])
def test_infinities_nan_and_lowest_values(T, score, dtype):
    E, k, inf = 12, 4, float("inf")
    l, _ = make(T, E, dtype, 3, False)
    low = torch.finfo(dtype).min
    l[0] = -inf                      # nothing left
    l[1] = float("nan")
    l[2, 3:] = -inf                  # fewer than k
    l[3, 5], l[3, 7] = inf, inf      # as large as can be
    l[4] = low                       # a mask of the type's lowest value everywhere
    l[5, 1:] = low
    l[5, 0] = float("nan")
    r = fq.fp8q_route(l.cuda(), k, score=score)
    for name, t in r._asdict().items():
        assert not torch.isnan(t.float()).any(), name
    want = reference(l.nan_to_num(nan=-inf, posinf=inf, neginf=-inf), None, k, score, True, 1.0)
    for name in ("idx", "counts", "offs", "order", "slot", "tokens"):
        assert torch.equal(getattr(r, name).cpu().long(), want[name]), name
    assert (r.idx[:2] == -1).all() and (r.weight[:2] == 0).all()
    assert r.idx[2].tolist()[3:] == [-1] and r.idx[3].tolist()[:2] == [5, 7] and r.idx[4].tolist() == [0, 1, 2, 3]
    if score == SOFT:
        assert (r.weight[4] == 0.25).all()
    else:  # every score underflows: no weight rather than no number
        assert (r.weight[4] == 0).all()
    ones = torch.ones(T, k, device="cuda")
    d = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=ones, dloss=torch.ones(1, device="cuda"),
                          score=score)
    assert torch.isfinite(d.float()).all() and not d[:2].any() and not d[2, 3:].any()


@pytest.mark.parametrize("T", [3, 500])
def test_no_valid_token(T):
    l, _ = make(T, 16, FP, 4, False)
    none = torch.zeros(T, dtype=torch.bool, device="cuda")
    r = fq.fp8q_route(l.cuda(), 2, valid=none)
    assert (r.idx == -1).all() and (r.order == -1).all() and (r.slot == -1).all() and not r.weight.any()
    assert not r.counts.any() and not r.offs.any() and r.loss.item() == 0 and r.tokens.item() == 0
    d = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=torch.ones(T, 2, device="cuda"),
                          dloss=torch.ones(1, device="cuda"), valid=none)
    assert not d.any()


def test_no_tokens():
    r = fq.fp8q_route(torch.empty(0, 16, device="cuda"), 2)
    assert r.idx.shape == (0, 2) and r.order.shape == (0,) and not r.counts.any() and not r.offs.any()
    assert r.loss.item() == 0 and r.tokens.item() == 0
    d = fq.fp8q_route_bwd(torch.empty(0, 16, device="cuda"), r.idx, r.counts, r.tokens, dloss=r.loss)
    assert d.shape == (0, 16)


def test_balance_loss_is_one_where_experts_are_used_alike():
    l = torch.full((64, 8), -20.0)
    l[torch.arange(64), torch.arange(64) % 8] = 20.0
    assert abs(fq.fp8q_route(l.cuda(), 1).loss.item() - 1) < 1e-6
    l[:] = -20.0
    l[:, 3] = 20.0
    assert abs(fq.fp8q_route(l.cuda(), 1).loss.item() - 8) < 1e-5


@pytest.mark.parametrize("T,E,k", [(40, 24, 3), (700, 100, 6)])
def test_strides_and_given_results(T, E, k):
    for dtype in (FP, BF):
        l, valid = make(T, E, dtype, 5, True)
        want = fq.fp8q_route(l.cuda(), k, valid=valid.cuda())
        for pad in (1, 8):
            lv, _ = padded(T, E, 2, pad, dtype, float("nan"))
            lv.copy_(l)
            i = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
            given = dict(idx=i(T, k), weight=torch.zeros(T, k, device="cuda"), counts=i(E), offs=i(E + 1), order=i(T * k),
                         slot=i(T, k), tokens=i(1), loss=torch.zeros(1, device="cuda"))
            ws = torch.full((fq.fp8q_route_workspace_bytes(T, E) + 64,), 0xFF, dtype=torch.uint8, device="cuda")
            r = fq.fp8q_route(lv, k, valid=valid.cuda().byte(), workspace=ws[:-64], **given)
            for name, t in r._asdict().items():
                assert t is given[name] and torch.equal(t, getattr(want, name)), name
            assert (ws[-64:] == 0xFF).all()
            dw, one = torch.randn(T, k, device="cuda"), torch.ones((), device="cuda")
            d0 = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dw, dloss=one, valid=valid.cuda())
            dv, buf = padded(T, E, 2, pad, dtype, 7.0)
            d1 = fq.fp8q_route_bwd(lv, r.idx, r.counts, r.tokens, dweight=dw, dloss=one, valid=valid.cuda(), dlogits=dv)
            assert d1 is dv and torch.equal(d0, d1) and (buf[:, E:] == 7).all() and (buf[T:] == 7).all()


def value(x, may, idx, counts, tokens, dw, dloss, score, normalise, scale):
    """sum(weight * dw) + dloss * loss in 64 bits, the choice and the counts held."""
    E = x.shape[1]
    log_s = torch.nn.functional.logsigmoid(x) if score == SIG else torch.log_softmax(x, 1)
    log_s = torch.where(may, log_s, float("-inf"))
    has = idx >= 0
    w = torch.where(has, log_s.gather(1, idx.clamp_min(0)), float("-inf"))
    w = torch.softmax(w, 1) if normalise else torch.exp(w)
    p = torch.softmax(log_s, 1)
    loss = E * (counts.double() / counts.sum() * p.sum(0)).sum() / tokens
    return (torch.where(has, w, 0.0) * dw).sum() * scale + dloss * loss


@pytest.mark.parametrize("T,E,k,dtype", [(1, 2, 1, FP), (3, 8, 2, FP), (50, 33, 5, BF), (333, 64, 6, BF), (600, 256, 8, FP),
                                         (100, 512, 8, FP), (64, 1000, 16, BF), (20, 128, 32, FP), (5000, 16, 4, FP)])
@pytest.mark.parametrize("score,normalise", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_backward(T, E, k, dtype, score, normalise):
    l, valid = make(T, E, dtype, T * 3 + E, T > 3)
    vc = None if valid is None else valid.cuda()
    kw = dict(score=score, normalise=normalise, scale=1.5, valid=vc)
    r = fq.fp8q_route(l.cuda(), k, **kw)
    g = torch.Generator().manual_seed(T)
    dw, dloss = torch.randn(T, k, generator=g), 0.7
    may, x, log_s = parts(l, valid, score)
    alive = may.any(1)
    idx, counts, tokens = r.idx.cpu().long(), r.counts.cpu(), int(r.tokens)
    n = T / max(tokens, 1)

    def grads(a, b):
        y = torch.where(may, x, -1e4)[alive].requires_grad_()
        v = value(y, may[alive], idx[alive], counts, tokens, a * dw[alive].double(), b * dloss, score, normalise, 1.5)
        return torch.zeros(T, E, dtype=torch.double).masked_scatter_(alive[:, None].expand(T, E),
                                                                     torch.autograd.grad(v, y)[0]) * may

    # magnitudes of the sums behind each element
    s = torch.where(may, torch.exp(log_s), 0.0)
    p = torch.where(alive[:, None], torch.softmax(log_s, 1), 0.0)
    has = idx >= 0
    u = torch.where(has, torch.exp(log_s.gather(1, idx.clamp_min(0))), 0.0)
    if normalise:
        u = u / u.sum(1, keepdim=True).clamp_min(1e-300)
    mag = torch.zeros(T, E, dtype=torch.double).scatter_add_(1, idx.clamp_min(0), u * dw.abs().double() * 1.5)
    all_u = (u * dw.abs().double() * 1.5).sum(1, keepdim=True)
    if normalise:
        mag = mag + torch.zeros(T, E, dtype=torch.double).scatter_add_(1, idx.clamp_min(0), u) * all_u
    elif score == SOFT:
        mag = mag + p * all_u
    dp = dloss * E * counts.double() / max(int(counts.sum()), 1) / max(tokens, 1)
    mag_l = p * (dp + (p * dp).sum(1, keepdim=True))
    if score == SIG:
        mag, mag_l = mag * torch.sigmoid(-x.clamp_min(-1e4)), mag_l * torch.sigmoid(-x.clamp_min(-1e4))
    reach = torch.where(may, (x.abs() if score == SIG else x.amax(1, keepdim=True) - x), 0.0).amax(1, keepdim=True)
    dwc, dlc = dw.cuda(), torch.tensor([dloss], device="cuda")
    for a, b in ((1, 1), (1, 0), (0, 1)):
        got = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dwc if a else None, dloss=dlc if b else None, **kw)
        assert got.dtype == dtype
        want = grads(a, b)
        # and the reference's own rounding, 2^-53 of its terms: where the exact sum is 0 it leaves some of that
        tol = (200 + 8 * reach) * U * (a * mag + b * mag_l) + 1e-37 + 2.0 ** -48 * (a * dw.abs().double().sum(1, keepdim=True) + b)
        near(got, want, tol + (2.0 ** -8 * (want.abs() + tol) if dtype == BF else 0), f"dlogits {a} {b}")
        again = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dwc if a else None, dloss=dlc if b else None, **kw)
        assert torch.equal(got, again)


@pytest.mark.parametrize("score,normalise", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
def test_gradients_against_differences(score, normalise):
    T, E, k, e = 6, 10, 3, 1e-4
    l, _ = make(T, E, FP, 6, False)
    r = fq.fp8q_route(l.cuda(), k, score=score, normalise=normalise)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(7))
    d = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dw.cuda(), dloss=torch.ones(1, device="cuda"),
                          score=score, normalise=normalise).double().cpu()
    may = torch.ones(T, E, dtype=torch.bool)
    f = lambda x: float(value(x, may, r.idx.cpu().long(), r.counts.cpu(), T, dw.double(), 1.0, score, normalise, 1.0))  # noqa: E731
    for seed in range(4):
        v = torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).double()
        slope = (f(l.double() + e * v) - f(l.double() - e * v)) / (2 * e)
        # third differences e^2 of order one, FP32 gradients
        assert abs(slope - float((d * v).sum())) < 1e-6 * (1 + float(d.norm() * v.norm()))


def test_choices_that_are_none_and_the_same_choice_twice():
    l, _ = make(4, 8, FP, 8, False)
    idx = torch.tensor([[1, 1], [-1, 3], [8, 2], [1 << 30, -(1 << 30)]], dtype=torch.int32, device="cuda")
    counts = torch.ones(8, dtype=torch.int32, device="cuda")
    dw = torch.ones(4, 2, device="cuda")
    d = fq.fp8q_route_bwd(l.cuda(), idx, counts, torch.tensor([4], dtype=torch.int32, device="cuda"), dweight=dw,
                          score=SIG, normalise=False).double().cpu()
    s = torch.sigmoid(l.double())
    want = torch.zeros(4, 8, dtype=torch.double)
    for t, e, n in ((0, 1, 2), (1, 3, 1), (2, 2, 1)):
        want[t, e] = n * s[t, e] * (1 - s[t, e])
    near(d, want, 100 * U * want + 1e-37, "dlogits")


def test_more_tokens_than_16_bit_counts_hold():
    # 153 CTAs of up to 65535 tokens, every token to the same expert first
    T, E, k = 10_000_001, 3, 2
    l = torch.randn(T, E, device="cuda") * 0.1
    l[:, 1] += 10
    r = fq.fp8q_route(l, k)
    second = torch.where(l[:, 2] > l[:, 0], 2, 0)
    assert (r.idx[:, 0] == 1).all() and torch.equal(r.idx[:, 1].long(), second)
    counts = torch.bincount(r.idx.reshape(-1), minlength=E)
    assert torch.equal(r.counts.long(), counts) and r.offs.tolist() == [0, *counts.cumsum(0).tolist()]
    assert torch.equal(r.order.long(), torch.sort(r.idx.reshape(-1), stable=True).indices)
    assert torch.equal(r.order[r.slot.reshape(-1).long()].long(), torch.arange(T * k, device="cuda"))
    p = torch.softmax(l.double(), 1).mean(0)
    want = E * (counts.double() / (T * k) * p).sum()
    # T / 153 / 32 probabilities one after another in a warp, 32 and 153 partial sums
    assert abs(float(r.loss) - float(want)) < (T / 153 / 32 + 500) * U * float(want)


def test_repeats_bit_by_bit():
    l, valid = make(9000, 200, FP, 9, True)
    first = fq.fp8q_route(l.cuda(), 8, valid=valid.cuda())
    for _ in range(5):
        again = fq.fp8q_route(l.cuda(), 8, valid=valid.cuda())
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def many_tokens(T, E, k, dtype, seed):
    """Logits that send most choices of neighbouring tokens to the same few experts, at other places of the choice."""
    l, valid = make(T, E, dtype, seed, True)
    l[:, : k + 2] += 6.0
    return l, valid


# more tokens than a launch has warps: each warp takes two to four, in every form
MANY = [(20000, 16, 4, FP), (20000, 30, 3, BF), (12000, 64, 6, BF), (13000, 33, 5, FP), (12000, 128, 8, FP),
        (12001, 256, 8, FP), (12000, 200, 6, BF), (11000, 512, 8, FP), (11000, 400, 8, BF), (7000, 1024, 32, FP),
        (7000, 1000, 16, BF), (6999, 1023, 8, FP)]


@pytest.mark.parametrize("T,E,k,dtype", MANY)
@pytest.mark.parametrize("score,normalise", [(SOFT, True), (SOFT, False), (SIG, True)])
def test_backward_of_more_tokens_than_warps(T, E, k, dtype, score, normalise):
    # a token's gradient is its own: the same bits as in calls of 500 tokens, which take one per warp
    l, valid = many_tokens(T, E, k, dtype, T + E)
    l, valid = l.cuda(), valid.cuda()
    kw = dict(score=score, normalise=normalise, scale=1.5)
    r = fq.fp8q_route(l, k, valid=valid, **kw)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    dloss = torch.tensor([0.7], device="cuda")
    got = fq.fp8q_route_bwd(l, r.idx, r.counts, r.tokens, dweight=dw, dloss=dloss, valid=valid, **kw)
    for lo in range(0, T, 500):
        at = slice(lo, lo + 500)
        want = fq.fp8q_route_bwd(l[at], r.idx[at], r.counts, r.tokens, dweight=dw[at], dloss=dloss, valid=valid[at], **kw)
        assert torch.equal(got[at], want), lo


@pytest.mark.parametrize("T,E,k,dtype", [c for c in MANY if c[1] > 128])
@pytest.mark.parametrize("score,normalise", [(SOFT, True), (SIG, False)])
def test_forward_of_more_tokens_than_warps(T, E, k, dtype, score, normalise):
    # several tokens per warp of many experts, and more CTAs than the second launch adds up in one go
    l, valid = many_tokens(T, E, k, dtype, T + E)
    r = fq.fp8q_route(l.cuda(), k, score=score, normalise=normalise, scale=2.5, valid=valid.cuda())
    check(r, l, valid, k, score, normalise, 2.5)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("score,normalise", [(SOFT, True), (SOFT, False), (SIG, True), (SIG, False)])
@pytest.mark.parametrize("T,E,k,dtype", [(7, 6, 5, FP), (300, 64, 6, BF), (300, 300, 8, FP), (40, 1000, 32, BF)])
def test_gradients_of_choices_that_are_none_do_not_count(T, E, k, dtype, score, normalise, bad):
    # tokens with fewer open experts than choices, with none, and padding: whatever stands in dweight there
    l, _ = make(T, E, dtype, T + E, False)
    l[::2, k - 2:] = float("-inf")
    l[1] = float("-inf")
    valid = torch.ones(T, dtype=torch.bool)
    valid[3::5] = False
    l, valid = l.cuda(), valid.cuda()
    kw = dict(score=score, normalise=normalise, scale=1.5, valid=valid)
    r = fq.fp8q_route(l, k, **kw)
    none = r.idx < 0
    assert none.any() and not none.all()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    dloss = torch.tensor([0.7], device="cuda")
    want = fq.fp8q_route_bwd(l, r.idx, r.counts, r.tokens, dweight=dw.masked_fill(none, 0.0), dloss=dloss, **kw)
    got = fq.fp8q_route_bwd(l, r.idx, r.counts, r.tokens, dweight=dw.masked_fill(none, bad), dloss=dloss, **kw)
    assert torch.isfinite(want.float()).all() and torch.equal(got, want)
    assert not got[~valid].any() and not got[1].any()
    # a choice outside the experts, of a closed one, or of a padding token is none either
    idx = torch.where(none, E + 3, r.idx)
    idx[0, k - 1] = E - 1  # closed to token 0
    idx[3] = 0             # padding
    dw = dw.masked_fill(none, bad)
    dw[3] = bad
    assert torch.equal(fq.fp8q_route_bwd(l, idx, r.counts, r.tokens, dweight=dw, dloss=dloss, **kw), want)


@pytest.mark.parametrize("score", [SOFT, SIG])
@pytest.mark.parametrize("T,E,k", [(500, 64, 1), (3000, 256, 1), (400, 600, 4), (100, 24, 1)])
def test_one_normalised_choice_is_a_constant(T, E, k, score):
    # one choice, or one open expert: its weight is the scale, and its gradient nothing
    l, _ = make(T, E, FP, 3 * T + E, False)
    if k > 1:
        l[torch.arange(E) != torch.arange(T)[:, None] % E] = float("-inf")
    r = fq.fp8q_route(l.cuda(), k, score=score, scale=2.5)
    assert (r.weight[:, 0] == 2.5).all() and not r.weight[:, 1:].any()
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T)).cuda()
    d = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dw, score=score, scale=2.5)
    assert not d.any()


@pytest.mark.parametrize("T,E", [(30, 100), (600, 300)])
@pytest.mark.parametrize("centre", [-4, -12, -40, -80])
def test_weights_of_small_sigmoids_keep_their_digits(T, E, centre):
    """exp to 1 unit in the last place (2 u), 1 + exp (u), its reciprocal to a unit (2 u): 5 u whatever the logit;
    normalised 5 u more for the sum's terms, 5 for its tree, 2 and 1 for reciprocal and product: 18 u.  The gradient
    has the factor 1 - s, 5 u of the same kind, and four products: 14 u alone; normalised the weight's 18 u, the
    mean's 18 + 6 u of its terms, a difference, two products and 1 - s: 50 u of the terms' size."""
    k = 6
    l = centre + 0.5 * torch.randn(T, E, generator=torch.Generator().manual_seed(T + centre))
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(T))
    for normalise, tol, grad_tol in ((False, 5, 14), (True, 18, 50)):
        r = fq.fp8q_route(l.cuda(), k, score=SIG, normalise=normalise)
        at = r.idx.cpu().long()
        s = torch.sigmoid(l.double().gather(1, at))
        w = s / s.sum(1, keepdim=True) if normalise else s
        near(r.weight, w, tol * U * w, "weight")
        d = fq.fp8q_route_bwd(l.cuda(), r.idx, r.counts, r.tokens, dweight=dw.cuda(), score=SIG, normalise=normalise)
        g = dw.double()
        mean = (w * g).sum(1, keepdim=True) if normalise else 0.0
        size = g.abs() + ((w * g.abs()).sum(1, keepdim=True) if normalise else 0.0)
        near(d.cpu().gather(1, at), w * (g - mean) * (1 - s), grad_tol * U * w * size, "gradient")
