"""The norm, the router and AdamW as one block's training step uses them, around the experts' products."""
import importlib.util
import os

import pytest
import torch

B = pytest.importorskip("fp8_fine_grained_amax_gb300.binding")
import fp8_fine_grained_amax_gb300 as fq

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from fp8_fine_grained_amax_gb300.build import build_library
    build_library()
    yield B.load_library()
    assert B.fp8q_sync_status() == 0


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block_step", os.path.join(ROOT, "examples", "moe_block_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inputs(T, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(T, D, generator=g, device="cuda").bfloat16() for _ in range(3)]


def plain(b, x, res, idx):
    """The block in 64 bits, the choice held: contribution, balance loss, and its leaves."""
    leaves = [t.double().requires_grad_() for t in (x.double() + res.double(), b.norm, b.router, b.w, b.wd)]
    h, norm, router, w, wd = leaves
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    p = torch.softmax(y @ router.t(), 1)
    weight = p.gather(1, idx)
    weight = weight / weight.sum(1, keepdim=True)
    out = torch.zeros_like(y)
    for e in range(b.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        gate, up = (y[t] @ w[e].t()).chunk(2, 1)
        out = out.index_add(0, t, (torch.nn.functional.silu(gate) * up) @ wd[e].t() * weight[t, j, None])
    counts = torch.bincount(idx.reshape(-1), minlength=b.E).double()
    loss = b.E * (counts / counts.sum() * p.mean(0)).sum()
    return out, loss, leaves


def test_gradients_of_the_whole_block(example):
    """Every product has two E4M3 operands, each off by at most 2^-4 and, over many values, by 0.026 of their
    norm: 0.037 per product.  The longest way to a gradient is two products forward and two backward, 0.074; half
    as much again for the gates' slopes, and the same for what the logits, BF16 y of FP32 rows, change.  The
    norm's and the router's gradients cancel partly."""
    T, D = 300, 256
    b = example.MoEBlock(D, 384, 8, 2, 5)
    b.norm.add_(torch.randn(D, generator=torch.Generator().manual_seed(6)).cuda() * 0.1)
    x, res, dout = inputs(T, D, 7)
    dout = dout.float() / T
    out, stream, loss = b.forward(x, res)
    dx = b.backward(dout)
    idx = b.r.idx.long()
    want, want_loss, leaves = plain(b, x, res, idx)
    # the choice itself: by the reference's own logits but for near ties
    far = lambda a, c: float((a.double() - c.detach()).norm() / c.detach().norm())  # noqa: E731
    assert far(out, want) < 0.08 and abs(float(loss) - float(want_loss.detach())) < 1e-2
    assert far(stream, leaves[0].detach()) < 2.0 ** -8
    grads = torch.autograd.grad((want * dout.double()).sum() + b.balance * want_loss, leaves)
    got = (dx - dout, b.dnorm, b.drouter, b.dw, b.dwd)
    for name, a, c in zip(("x", "norm", "router", "w", "wd"), got, grads):
        assert far(a, c) < 0.15, name


def test_routed_rows_are_the_tokens_rows(example):
    b = example.MoEBlock(256, 128, 5, 3, 8)
    x, res, _ = inputs(77, 256, 9)
    b.forward(x, res)
    r = b.r
    rows, slot = r.order // 3, r.slot
    assert torch.equal(rows[slot], torch.arange(77, device="cuda")[:, None].expand(77, 3).int())
    ends = r.offs.tolist()
    for e in range(5):
        assert (r.idx[rows[ends[e]:ends[e + 1]]] == e).any(1).all()
    # a token's experts one by one give the same contribution as the grouped products
    t = 13
    for j in range(3):
        e = int(r.idx[t, j])
        g = fq.fp8q_gemm_swiglu(b.n.q[t:t + 1], b.n.s[:, t:t + 1], b.qw[e], b.sw[e], with_h=False, with_codes=True)
        y = fq.fp8q_gemm(g.q, g.s, b.qwd[e], b.swd[e]).float()[0]
        assert float((y - b.y[t, j]).norm() / b.y[t, j].norm()) < 0.02  # codes of h may differ by a step


def test_training_runs_and_keeps_finite(example, capsys):
    losses = example.main(D=128, F=256, E=4, k=2, T=256, steps=3)
    assert len(losses) == 3 and all(torch.isfinite(torch.tensor(losses)))
    assert "balance" in capsys.readouterr().out


def test_captured_step_repeats_the_eager_one(example):
    """Norm, router, both backward passes and AdamW in one captured graph with its own scratch, replayed on new
    inputs beside another graph: the eager calls' bits."""
    T, D, E, k = 200, 512, 16, 4
    x, res, dy = inputs(T, D, 10)
    w = torch.ones(D, device="cuda")
    router = torch.randn(E, D, generator=torch.Generator().manual_seed(11)).cuda() / D ** 0.5
    dw0, one = torch.randn(T, k, device="cuda"), torch.ones(1, device="cuda")

    class State:
        def __init__(self):
            self.w = w.clone()
            self.m, self.v = (torch.zeros(D, dtype=torch.uint8, device="cuda") for _ in range(2))
            self.ms, self.vs = (torch.zeros(D // 128, device="cuda") for _ in range(2))
            self.step = torch.zeros(1, dtype=torch.long, device="cuda")

        def run(self, x, res, dy):
            self.step += 1
            n = fq.fp8q_rmsnorm(x, self.w, residual=res, with_y=True, with_rstd=True)
            logits = (n.y.float()[:, None] * router).sum(-1)
            r = fq.fp8q_route(logits, k)
            d = fq.fp8q_route_bwd(logits, r.idx, r.counts, r.tokens, dweight=dw0, dloss=one)
            g = fq.fp8q_rmsnorm_bwd(dy, n.r, n.rstd, self.w, dres=dy)
            fq.fp8q_adamw([self.w], [g.dw], [self.m], [self.v], m_scales=[self.ms], v_scales=[self.vs], step=self.step,
                          lr=1e-2)
            return [*n, *r, d, *g]

    a, b, c = State(), State(), State()
    bufs = [[t.clone() for t in (x, res, dy)] for _ in range(2)]
    State().run(x, res, dy)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for st, buf, graph in zip((a, b), bufs, graphs):
        with torch.cuda.graph(graph):
            outs.append(st.run(*buf))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for seed in (20, 21, 22):
        new = inputs(T, D, seed)
        for buf in bufs:
            for t, s in zip(buf, new):
                t.copy_(s)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):  # both at once
            with torch.cuda.stream(stream):
                graph.replay()
        want = c.run(*new)
        torch.cuda.synchronize()
        for out, st in zip(outs, (a, b)):
            for got, ref in zip(out + [st.w, st.m, st.v, st.ms, st.vs], want + [c.w, c.m, c.v, c.ms, c.vs]):
                assert torch.equal(got, ref)


def test_calls_run_on_the_stream_they_are_given():
    x, res, dy = inputs(400, 1536, 12)
    w = torch.ones(1536, device="cuda")
    l = torch.randn(400, 32, device="cuda")
    n = fq.fp8q_rmsnorm(x, w, residual=res, with_y=True, with_rstd=True)
    g = fq.fp8q_rmsnorm_bwd(dy, n.r, n.rstd, w, dres=dy)
    r = fq.fp8q_route(l, 4)
    d = fq.fp8q_route_bwd(l, r.idx, r.counts, r.tokens, dloss=r.loss)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 0.05 s
    n2 = fq.fp8q_rmsnorm(x, w, residual=res, with_y=True, with_rstd=True, stream=side)
    g2 = fq.fp8q_rmsnorm_bwd(dy, n2.r, n2.rstd, w, dres=dy, stream=side)
    r2 = fq.fp8q_route(l, 4, stream=side)
    d2 = fq.fp8q_route_bwd(l, r2.idx, r2.counts, r2.tokens, dloss=r2.loss, stream=side)
    p = [torch.ones(500, device="cuda") for _ in range(4)]
    fq.fp8q_adamw(p[:1], p[1:2], p[2:3], p[3:], step=1, lr=0.5, stream=side)
    # the current stream takes and fills what the allocator would hand out again
    held = [torch.full((n2.y.numel() * 2,), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.current_stream().synchronize()
    assert not side.query(), "the calls did not wait for their stream"
    torch.cuda.synchronize()
    for a, b in zip([*n, *g, *r, d], [*n2, *g2, *r2, d2]):
        assert torch.equal(a, b)
    assert (p[0] != 1).all() and all((h == 0x7F).all() for h in held)
    handles = {seg["stream"] for seg in torch.cuda.memory_snapshot() for t in (n2.y, g2.dx, r2.idx, d2)
               if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]}
    assert handles == {side.cuda_stream}


def test_two_threads_at_once():
    import threading
    l = torch.randn(3000, 64, device="cuda")
    x = torch.randn(600, 2048, device="cuda").bfloat16()
    w = torch.ones(2048, device="cuda")
    want_r, want_n = fq.fp8q_route(l, 6), fq.fp8q_rmsnorm(x, w, with_rstd=True)
    want_g = fq.fp8q_rmsnorm_bwd(x, x, want_n.rstd, w)
    torch.cuda.synchronize()
    wrong = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                r, n = fq.fp8q_route(l, 6), fq.fp8q_rmsnorm(x, w, with_rstd=True)
                g = fq.fp8q_rmsnorm_bwd(x, x, n.rstd, w)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip([*r, n.q, n.s, *g], [*want_r, want_n.q, want_n.s, *want_g])):
                    wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def plain_masked(b, x, res, idx, may):
    """`plain` for choices of -1 and experts that are closed (`may` False) to a token."""
    leaves = [t.double().requires_grad_() for t in (x.double() + res.double(), b.norm, b.router, b.w, b.wd)]
    h, norm, router, w, wd = leaves
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    alive, has = may.any(1), idx >= 0
    p = torch.softmax(torch.where(may, y @ router.t(), -1e4), 1) * alive[:, None]
    weight = torch.where(has, p.gather(1, idx.clamp_min(0)), 0.0)
    weight = weight / torch.where(alive, weight.sum(1), 1.0)[:, None]
    out = torch.zeros_like(y)
    for e in range(b.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        gate, up = (y[t] @ w[e].t()).chunk(2, 1)
        out = out.index_add(0, t, (torch.nn.functional.silu(gate) * up) @ wd[e].t() * weight[t, j, None])
    counts = torch.bincount(idx[has], minlength=b.E).double()
    loss = b.E * (counts / counts.sum() * p.sum(0)).sum() / alive.sum()
    return out, loss, leaves


def test_block_with_padding_and_closed_experts(example):
    """Tokens without a choice and with fewer than k: no rows of theirs are written, whatever is in that memory.
    Bounds as in test_gradients_of_the_whole_block."""
    T, D, E, k = 300, 256, 6, 3
    b = example.MoEBlock(D, 384, E, k, 15)
    x, res, dout = inputs(T, D, 17)
    dout = dout.float() / T
    g = torch.Generator(device="cuda").manual_seed(18)
    valid = torch.rand(T, generator=g, device="cuda") > 0.2
    closed = torch.rand(T, E, generator=g, device="cuda") < 0.6
    closed[::7] = True

    def spoil():  # free memory full of NaN: what the calls take next
        held = [torch.full((T * k * D,), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(16)]
        torch.cuda.synchronize()
        del held

    spoil()
    out, stream, loss = b.forward(x, res, valid, closed)
    spoil()
    dx = b.backward(dout)
    idx = b.r.idx.long()
    none = idx < 0
    assert none.all(1).any() and (none.any(1) & ~none.all(1)).any()
    assert not out[none.all(1)].any() and torch.equal(none, b.r.slot < 0)
    may = ~closed & valid[:, None]
    want, want_loss, leaves = plain_masked(b, x, res, idx, may)
    far = lambda a, c: float((a.double() - c.detach()).norm() / c.detach().norm())  # noqa: E731
    assert far(out, want) < 0.08 and abs(float(loss) - float(want_loss.detach())) < 1e-2
    assert far(stream, leaves[0].detach()) < 2.0 ** -8
    grads = torch.autograd.grad((want * dout.double()).sum() + b.balance * want_loss, leaves)
    got = (dx - dout, b.dnorm, b.drouter, b.dw, b.dwd)
    for name, a, c in zip(("x", "norm", "router", "w", "wd"), got, grads):
        assert far(a, c) < 0.15, name
    b.update(1e-3)
    assert all(torch.isfinite(t).all() for t in (b.norm, b.router, b.w, b.wd))


def test_block_without_any_choice(example):
    b = example.MoEBlock(256, 128, 4, 2, 16)
    x, res, dout = inputs(40, 256, 19)
    out, _, loss = b.forward(x, res, torch.zeros(40, dtype=torch.bool, device="cuda"))
    dx = b.backward(dout.float())
    assert not out.any() and loss.item() == 0 and torch.equal(dx, dout.float())
    assert not any(t.any() for t in (b.dnorm, b.drouter, b.dw, b.dwd))


def test_what_a_result_keeps_alive():
    """Results of a call share allocations; what is little, and kept, holds no more than 64 KB."""
    held = lambda t: t.untyped_storage().nbytes()  # noqa: E731
    for T, E, k in ((1, 64, 4), (2000, 64, 4), (4096, 256, 8), (40000, 256, 8)):
        r = fq.fp8q_route(torch.randn(T, E, device="cuda"), k)
        assert max(map(held, (r.loss, r.tokens, r.counts, r.offs))) <= 64 << 10
        assert all(held(t) <= max(t.nbytes, 2 << 20) for t in r)
        check = fq.fp8q_route_bwd(torch.randn(T, E, device="cuda"), r.idx, r.counts, r.tokens, dloss=r.loss)
        assert held(check) == check.nbytes
    for T, C in ((1, 7168), (40, 7168), (333, 896), (1000, 7168)):
        x = torch.randn(T, C, device="cuda").bfloat16()
        w = torch.ones(C, device="cuda")
        n = fq.fp8q_rmsnorm(x, w, residual=x, with_y=True, with_rstd=True)
        assert held(n.rstd) <= 64 << 10
        g = fq.fp8q_rmsnorm_bwd(x, n.r, n.rstd, w)
        assert all(held(t) <= max(t.nbytes, 2 << 20) for t in (*n, *g))
        # parts of one allocation do not overlap, and start where wide loads may
        parts = sorted((t.data_ptr(), t.nbytes) for t in (*n, *g))
        assert all(p + size <= q for (p, size), (q, _) in zip(parts, parts[1:])) and all(p % 256 == 0 for p, _ in parts)


def test_a_logged_loss_holds_no_more_than_itself_and_little_else():
    l = torch.randn(4000, 64, device="cuda")
    fq.fp8q_route(l, 8)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    losses = [fq.fp8q_route(l, 8).loss for _ in range(100)]
    assert torch.cuda.memory_allocated() - before <= 100 * (64 << 10)
    assert len({float(x) for x in losses}) == 1
