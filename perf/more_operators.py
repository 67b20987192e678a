"""Measured cases of the operators around the FP8 products of a training or serving step.

Operators (``op``):

- ``norm``       root-mean-square norm with the residual's addition: h = x + r, y = h / rms(h) * w, as BF16
                 and / or as the 1x128 FP8 operand of the next product.
- ``norm_bwd``   its backward pass: the gradient of h, with the residual stream's own gradient added, and of w.
- ``adamw``      one AdamW step over a list of tensors, moments in FP32, in BF16 or in 8 bits.  In 8 bits m and
                 sqrt(v) are E4M3 codes with one FP32 scale per 128 values; a positive sqrt(v) is at least the
                 smallest code, so that no denominator is rounded to zero.
- ``route``      the router of a mixture of experts: the k largest logits of each token (ties: the lowest index),
                 combine weights, counts, offsets and order of the rows sorted by expert, and the balance loss
                 E * sum_e (share of the choices that went to e) * (mean probability of e).
- ``route_bwd``  its backward pass: the gradient of the logits from those of the weights and of the loss.

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is true, with the library's
kernels.  FP8 outputs are float8_e4m3fn tensors beside their FP32 scales.
"""
import torch

own = False

E4M3 = torch.float8_e4m3fn
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
LR, BETAS, ADAM_EPS, DECAY = 3e-4, (0.9, 0.95), 1e-8, 0.1
TINY = 2.0 ** -126  # a sum of scores below it counts as this
BIG = 3.4028234663852886e38  # the largest FP32 value

# the weights of four experts: gate and up projection 4096 x 7168, down projection 7168 x 2048
EXPERTS = ",".join(["29360128,14680064"] * 4)


def listed():
    return [
        # one token in the serving loop: residual stream updated, FP8 operand of the next product
        dict(name="norm 1 token", op="norm", T=1, C=7168, x="bf16", res="bf16", y=False, codes=True, rstd=False, pow2=False),
        # an odd number of prompt tokens, FP32 residual stream, both kinds of output
        dict(name="norm 333x896", op="norm", T=333, C=896, x="bf16", res="fp32", y=True, codes=True, rstd=True, pow2=True),
        # training forward: new residual stream, FP8 operand, statistics for the backward pass
        dict(name="norm 8192x7168", op="norm", T=8192, C=7168, x="bf16", res="bf16", y=False, codes=True, rstd=True,
             pow2=False),
        # a micro-batch of a small block: launch latency counts
        dict(name="norm_bwd 128x2048", op="norm_bwd", T=128, C=2048, dy="bf16", x="bf16", dres=False, dx="bf16"),
        # training backward, the residual stream's gradient added
        dict(name="norm_bwd 8192x7168", op="norm_bwd", T=8192, C=7168, dy="bf16", x="bf16", dres=True, dx="bf16"),
        # what no weight matrix is: norms, a router, biases of odd lengths; latency counts
        dict(name="adamw 10 small", op="adamw", sizes="7168,7168,1536,512,7168,1835008,256,1,333,65537", p="fp32", g="fp32",
             state="fp32", copy=False, clip=True, step=1),
        # four experts' weights, master weights and moments in FP32, BF16 copies for the next forward pass
        dict(name="adamw experts fp32", op="adamw", sizes=EXPERTS, p="fp32", g="fp32", state="fp32", copy=True, clip=True,
             step=1000),
        # the same with moments in 8 bits
        dict(name="adamw experts 8 bits", op="adamw", sizes=EXPERTS, p="fp32", g="fp32", state="e4m3", copy=True, clip=True,
             step=1000),
        # one token in the serving loop
        dict(name="route 1 token", op="route", T=1, E=256, k=8, logits="fp32", sigmoid=False, norm=True, masked=False),
        # a training batch of 16384 tokens, some of them padding
        dict(name="route 16384x256", op="route", T=16384, E=256, k=8, logits="fp32", sigmoid=True, norm=True, masked=True),
        # a small batch, few experts, weights not normalised: latency counts
        dict(name="route_bwd 333x64", op="route_bwd", T=333, E=64, k=6, logits="bf16", sigmoid=False, norm=False,
             masked=True),
        # the training batch's gradient
        dict(name="route_bwd 16384x256", op="route_bwd", T=16384, E=256, k=8, logits="fp32", sigmoid=True, norm=True,
             masked=True),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    def flag(p=0.5):
        return rng.random() < p

    def kind():
        return rng.choice(["bf16", "fp32"])

    while True:
        op = rng.choice(["norm", "norm", "norm_bwd", "norm_bwd", "adamw", "adamw", "route", "route_bwd"])
        if op == "norm":
            codes = flag(0.7)
            C = 128 * log_int(1, 128) if codes else 8 * log_int(1, 2048)
            c = dict(op=op, T=log_int(1, 16384), C=C, x=kind(), res=rng.choice(["none", "bf16", "fp32"]),
                     y=not codes or flag(0.3), codes=codes, rstd=flag(), pow2=flag(0.3))
        elif op == "norm_bwd":
            c = dict(op=op, T=log_int(1, 16384), C=8 * log_int(1, 2048), dy=kind(), x=kind(), dres=flag(), dx=kind())
        elif op == "adamw":
            sizes = [log_int(1, 3e7) for _ in range(rng.randint(1, 10))]
            p = rng.choice(["fp32", "fp32", "bf16"])
            c = dict(op=op, sizes=",".join(map(str, sizes)), p=p, g=kind(), state=rng.choice(["fp32", "bf16", "e4m3"]),
                     copy=p == "fp32" and flag(), clip=flag(), step=log_int(1, 20000))
        else:
            E = log_int(2, 1024)
            k = rng.randint(1, min(E, 16))
            # one weight alone, normalised, is a constant
            c = dict(op=op, T=log_int(1, 32768), E=E, k=k, logits=kind(), sigmoid=flag(), norm=k > 1 and flag(),
                     masked=flag())
        if work(c)["bytes"] <= 1.2e9:
            return c


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _stream(g, T, C):
    """A residual stream: channels of different size and a few large entries."""
    x = _randn(g, T, C) * torch.exp(_randn(g, C, std=0.5))
    return torch.where(_rand(g, T, C) < 1e-3, x * 30.0, x)


def _sizes(case):
    return [int(n) for n in case["sizes"].split(",")]


def _logits(case, g):
    T, E = case["T"], case["E"]
    l = _randn(g, T, E, std=1.5) + _randn(g, E, std=0.7)
    valid = None
    if case["masked"]:
        # padding tokens, and experts that some tokens may not take
        valid = _rand(g, T) > 0.1
        l = torch.where((_rand(g, T, 1) < 0.1) & (_rand(g, T, E) < 0.5), float("-inf"), l)
    return l.to(TYPES[case["logits"]]), valid


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op == "norm":
        T, C = case["T"], case["C"]
        s["x"] = _randn(g, T, C).to(TYPES[case["x"]])
        s["res"] = None if case["res"] == "none" else _stream(g, T, C).to(TYPES[case["res"]])
        s["w"] = 1.0 + _randn(g, C, std=0.2)
    elif op == "norm_bwd":
        T, C = case["T"], case["C"]
        s["x"] = _stream(g, T, C).to(TYPES[case["x"]])
        s["rstd"] = (s["x"].double().square().mean(1) + EPS).rsqrt().float()
        s["w"] = 1.0 + _randn(g, C, std=0.2)
        s["dy"] = _randn(g, T, C, std=1e-3).to(TYPES[case["dy"]])
        s["dres"] = _randn(g, T, C, std=1e-3).to(TYPES[case["dx"]]) if case["dres"] else None
    elif op == "adamw":
        sizes, state = _sizes(case), case["state"]
        s["p"] = [_randn(g, n, std=0.02).to(TYPES[case["p"]]) for n in sizes]
        s["g"] = [(_randn(g, n) * torch.exp(_randn(g, n)) * 1e-3).to(TYPES[case["g"]]) for n in sizes]
        first = case["step"] == 1  # nothing has been averaged yet
        m = [torch.zeros(n, device="cuda") if first else _randn(g, n, std=5e-4) for n in sizes]
        r = [torch.zeros(n, device="cuda") if first else 1e-3 * torch.exp(_randn(g, n)) for n in sizes]
        if state == "e4m3":
            s["m"], s["ms"] = _pairs(_quant(t) for t in m)
            s["v"], s["vs"] = _pairs(_quant(t, True) for t in r)
            s["m"], s["v"] = [t.view(torch.uint8) for t in s["m"]], [t.view(torch.uint8) for t in s["v"]]
        else:
            s["m"], s["v"] = [t.to(TYPES[state]) for t in m], [t.square().to(TYPES[state]) for t in r]
        s["copy"] = [t.bfloat16() for t in s["p"]] if case["copy"] else None
        s["clip"] = torch.rand(1, generator=g, device="cuda") + 0.25 if case["clip"] else None
    else:
        s["l"], s["valid"] = _logits(case, g)
        s["scale"] = 2.5
        if op == "route_bwd":
            # what the forward pass left, and the gradients that reach its results
            r = _route(s)
            s["idx"], s["counts"], s["tokens"] = r["idx"], r["counts"], r["tokens"]
            s["dw"] = _randn(g, case["T"], case["k"], std=1e-2)
            s["dloss"] = torch.full((1,), 1e-3, device="cuda")
    return s


# ----------------------------------------------------------------------------- plain forms
def _pairs(it):
    a, b = zip(*it)
    return list(a), list(b)


def _scales(amax, pow2):
    """Scale of each group and the factor its values are multiplied by."""
    a = amax.clamp_min(2.0 ** -116)
    if not pow2:
        return a / 448.0, 448.0 / a
    mant, exp = torch.frexp(a / 448.0)  # a / 448 = mant * 2^exp, mant in [0.5, 1)
    e = torch.where(mant == 0.5, exp - 1, exp)
    return torch.ldexp(torch.ones_like(a), e), torch.ldexp(torch.ones_like(a), -e)


def _quant_rows(x, pow2):
    """1x128 tiles of x [T][C]: codes [T][C] and scales [C/128][T]."""
    T, C = x.shape
    t = x.reshape(T, C // 128, 128)
    s, inv = _scales(t.abs().amax(-1), pow2)
    return (t * inv[..., None]).reshape(T, C).to(E4M3), s.t().contiguous()


def _groups(x):
    """x [n] as groups of 128, the last one filled with zeros."""
    n = x.numel()
    pad = -n % 128
    return (torch.cat([x, x.new_zeros(pad)]) if pad else x).reshape(-1, 128)


def _quant(x, root=False):
    """Codes [n] and scales [n/128, rounded up] of a moment; root: of sqrt(v), positive values at least 2^-9."""
    t = _groups(x)
    s, inv = _scales(t.abs().amax(1), False)
    t = t * inv[:, None]
    if root:
        t = torch.where(t > 0, t.clamp_min(2.0 ** -9), t)
    return t.reshape(-1)[:x.numel()].to(E4M3), s


def _values(q, s):
    return (_groups(q.view(E4M3).float()) * s[:, None]).reshape(-1)[:q.numel()]


def _norm(s):
    case = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    rstd = 1.0 / (h.square().mean(1, keepdim=True) + EPS).sqrt()
    y = h * rstd * s["w"]
    out = {}
    if s["res"] is not None:
        out["r"] = h.to(s["res"].dtype)
    if case["y"]:
        out["y"] = y.bfloat16()
    if case["codes"]:
        out["q"], out["s"] = _quant_rows(y, case["pow2"])
    if case["rstd"]:
        out["rstd"] = rstd[:, 0]
    return out


def _norm_bwd(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    xh = x * rstd
    t = dy * s["w"]
    dx = rstd * (t - xh * (t * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(TYPES[s["case"]["dx"]]), "dw": (dy * xh).sum(0)}


def _adamw_one(s, i, b1, b2, c1, c2):
    """One tensor's step, in place."""
    state = s["case"]["state"]
    p, g, m, v = s["p"][i], s["g"][i].float(), s["m"][i], s["v"][i]
    if s["clip"] is not None:
        g = g * s["clip"]
    if state == "e4m3":
        m0, v0 = _values(m, s["ms"][i]), _values(v, s["vs"][i]).square()
    else:
        m0, v0 = m.float(), v.float()
    m1 = b1 * m0 + (1 - b1) * g
    v1 = b2 * v0 + (1 - b2) * g * g
    w = p.float()
    w = w - LR * (DECAY * w + m1 / c1 / ((v1 / c2).sqrt() + ADAM_EPS))
    p.copy_(w)
    if s["copy"] is not None:
        s["copy"][i].copy_(w)
    if state == "e4m3":
        q, sc = _quant(m1)
        m.copy_(q.view(torch.uint8))
        s["ms"][i].copy_(sc)
        q, sc = _quant(v1.sqrt(), True)
        v.copy_(q.view(torch.uint8))
        s["vs"][i].copy_(sc)
    else:
        m.copy_(m1)
        v.copy_(v1)


def _adamw(s):
    (b1, b2), t = BETAS, s["case"]["step"]
    [_adamw_one(s, i, b1, b2, 1 - b1 ** t, 1 - b2 ** t) for i in range(len(s["p"]))]
    return _adamw_out(s)


def _adamw_out(s):
    out = {"p": s["p"]}
    if s["case"]["state"] == "e4m3":
        out.update(m=[t.view(E4M3) for t in s["m"]], v=[t.view(E4M3) for t in s["v"]], ms=s["ms"], vs=s["vs"])
    else:
        out.update(m=s["m"], v=s["v"])
    if s["copy"] is not None:
        out["copy"] = s["copy"]
    return out


def _scores(s):
    """Logits (those that cannot be chosen at -inf), scores and probabilities, [T][E]."""
    l = s["l"].float()
    may = l > float("-inf")
    if s["valid"] is not None:
        may = may & s["valid"][:, None]
    l = torch.where(may, l.clamp_max(BIG), float("-inf"))
    if s["case"]["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-l))
        return l, may, score, score / score.sum(1, keepdim=True).clamp_min(TINY)
    top = l.amax(1, keepdim=True).clamp_min(-BIG)
    e = torch.exp(l - top)
    p = e / e.sum(1, keepdim=True).clamp_min(TINY)
    return l, may, p, p


def _route(s):
    case = s["case"]
    k, E = case["k"], case["E"]
    l, may, score, p = _scores(s)
    T = l.shape[0]
    idx = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :k]
    has = may.gather(1, idx)
    w = torch.where(has, score.gather(1, idx), 0.0)
    if case["norm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(TINY)
    idx = torch.where(has, idx, -1)
    flat = torch.where(has, idx, E).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    slot = torch.empty_like(order)
    slot[order] = torch.arange(T * k, device=l.device)
    counts = torch.zeros(E + 1, dtype=torch.long, device=l.device).scatter_add_(0, flat, torch.ones_like(flat))[:E]
    total = counts.sum()
    tokens = has[:, 0].sum()
    share = counts.float() / total.clamp_min(1).float()
    loss = E * (share * p.sum(0)).sum() / tokens.clamp_min(1).float()
    at = torch.arange(T * k, device=l.device)
    offs = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return {"idx": idx.int(), "weight": w * s["scale"], "counts": counts.int(), "offs": offs.int(),
            "order": torch.where(at < total, order, -1).int(),
            "slot": torch.where(has, slot.reshape(T, k), -1).int(),
            "tokens": tokens.int().reshape(1), "loss": loss.reshape(1)}


def _route_bwd(s):
    """Through the logarithms of the scores: d / d log s_e is u_e from the weights and v_e from the loss."""
    case = s["case"]
    E = case["E"]
    l, may, score, p = _scores(s)
    has = s["idx"] >= 0
    at = s["idx"].clamp_min(0).long()
    dw = torch.where(has, s["dw"], 0.0) * s["scale"]
    u = torch.where(has, score.gather(1, at), 0.0)
    if case["norm"]:
        u = u / u.sum(1, keepdim=True).clamp_min(TINY)
        u = u * (dw - (u * dw).sum(1, keepdim=True))
    else:
        u = u * dw
    share = s["counts"].float() / s["counts"].sum().clamp_min(1).float()
    dp = s["dloss"] * E * share / s["tokens"].clamp_min(1).float()
    d = p * (dp - (p * dp).sum(1, keepdim=True))
    if not case["sigmoid"] and not case["norm"]:
        d = d - p * u.sum(1, keepdim=True)
    d = d.scatter_add_(1, at, u)
    if case["sigmoid"]:
        d = d / (1.0 + torch.exp(l))
    return {"dlogits": torch.where(may, d, 0.0).to(TYPES[case["logits"]])}


PLAIN = {"norm": _norm, "norm_bwd": _norm_bwd, "adamw": _adamw, "route": _route, "route_bwd": _route_bwd}


# ----------------------------------------------------------------------------- the library's calls
def _own(s):
    import fp8_fine_grained_amax_gb300 as fq
    case = s["case"]
    op = case["op"]
    if op == "norm":
        r = fq.fp8q_rmsnorm(s["x"], s["w"], residual=s["res"], eps=EPS, with_y=case["y"], with_codes=case["codes"],
                            with_rstd=case["rstd"], scale_mode=fq.FP8Q_SCALE_POW2 if case["pow2"] else fq.FP8Q_SCALE_FP32)
        out = {}
        if s["res"] is not None:
            out["r"] = r.r
        if case["y"]:
            out["y"] = r.y
        if case["codes"]:
            out["q"], out["s"] = r.q.view(E4M3), r.s
        if case["rstd"]:
            out["rstd"] = r.rstd
        return out
    if op == "norm_bwd":
        r = fq.fp8q_rmsnorm_bwd(s["dy"], s["x"], s["rstd"], s["w"], dres=s["dres"],
                                out_dtype=fq.FP8Q_OUT_BF16 if case["dx"] == "bf16" else fq.FP8Q_OUT_FP32)
        return {"dx": r.dx, "dw": r.dw}
    if op == "adamw":
        fq.fp8q_adamw(s["p"], s["g"], s["m"], s["v"], m_scales=s.get("ms"), v_scales=s.get("vs"), copies=s["copy"],
                      step=case["step"], lr=LR, betas=BETAS, eps=ADAM_EPS, weight_decay=DECAY, grad_scale=s["clip"])
        return _adamw_out(s)
    kind = fq.FP8Q_SCORE_SIGMOID if case["sigmoid"] else fq.FP8Q_SCORE_SOFTMAX
    if op == "route":
        r = fq.fp8q_route(s["l"], case["k"], score=kind, normalise=case["norm"], scale=s["scale"], valid=s["valid"])
        return r._asdict()
    return {"dlogits": fq.fp8q_route_bwd(s["l"], s["idx"], s["counts"], s["tokens"], dweight=s["dw"], dloss=s["dloss"],
                                         score=kind, normalise=case["norm"], scale=s["scale"], valid=s["valid"])}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"none": 0, "bf16": 2, "fp32": 4, "e4m3": 1}
    if op == "norm":
        n = case["T"] * case["C"]
        b = n * (size[case["x"]] + 2 * size[case["res"]] + 2 * case["y"] + case["codes"]) + case["codes"] * n // 32
        return {"bytes": b + 4 * case["C"] + 4 * case["T"] * case["rstd"], "flops": 6.0 * n}
    if op == "norm_bwd":
        n = case["T"] * case["C"]
        b = n * (size[case["dy"]] + size[case["x"]] + size[case["dx"]] * (1 + case["dres"]))
        return {"bytes": b + 8 * case["C"] + 4 * case["T"], "flops": 10.0 * n}
    if op == "adamw":
        n = sum(_sizes(case))
        each = 2 * size[case["p"]] + size[case["g"]] + 4 * size[case["state"]] + 2 * case["copy"]
        return {"bytes": n * each + (n // 8 if case["state"] == "e4m3" else 0), "flops": 16.0 * n}
    T, E, k = case["T"], case["E"], case["k"]
    b = T * E * size[case["logits"]]
    if op == "route":
        return {"bytes": b + 16 * T * k + 8 * E, "flops": 6.0 * T * E}
    return {"bytes": 2 * b + 8 * T * k + 4 * E, "flops": 12.0 * T * E}


# ----------------------------------------------------------------------------- 64 bits
def _exact_codes(x, root=False):
    """Unrounded codes and scales of groups of 128 along the last axis: what E4M3 then rounds."""
    a = x.abs().unflatten(-1, (-1, 128)).max(-1).values
    a = torch.where(a < 2.0 ** -116, 2.0 ** -116, a)
    q = x / a.repeat_interleave(128, -1) * 448
    return torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q) if root else q, a / 448


def _exact_pow2(q, s):
    """The same with the scales rounded up to powers of two."""
    up = torch.exp2(torch.ceil(torch.log2(s)))
    return q * (s / up).repeat_interleave(128, -1), up


def _exact_norm(case, s):
    h = s["x"].double()
    if s["res"] is not None:
        h = torch.add(s["res"].double(), h)
    length = torch.linalg.vector_norm(h, dim=1)
    rstd = torch.rsqrt(length * length / case["C"] + EPS)
    y = torch.einsum("tc,t,c->tc", h, rstd, s["w"].double())
    out = {}
    if s["res"] is not None:
        out["r"] = h
    if case["y"]:
        out["y"] = y
    if case["codes"]:
        q, sc = _exact_codes(y)
        if case["pow2"]:
            q, sc = _exact_pow2(q, sc)
        out["q"], out["s"] = q, sc.t().contiguous()
    if case["rstd"]:
        out["rstd"] = rstd
    return out


def _exact_norm_bwd(s):
    """By differentiating y with rstd's own dependence on x, row by row: a projection off x's direction."""
    x, dy, rstd, w = (s[n].double() for n in ("x", "dy", "rstd", "w"))
    t = torch.einsum("tc,c->tc", dy, w)
    along = torch.einsum("tc,tc->t", t, x) * rstd.pow(3) / x.shape[1]
    dx = torch.einsum("tc,t->tc", t, rstd) - torch.einsum("tc,t->tc", x, along)
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return {"dx": dx, "dw": torch.einsum("tc,tc,t->c", dy, x, rstd)}


def _exact_fill(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 128))


def _exact_adamw(case, s):
    (b1, b2), t = BETAS, case["step"]
    out = {}

    def put(**kw):
        [out.setdefault(k, []).append(v) for k, v in kw.items()]

    def one(i):
        g, p = s["g"][i].double(), s["p"][i].double()
        n = p.numel()
        if s["clip"] is not None:
            g = g * s["clip"].double()
        m, v = s["m"][i], s["v"][i]
        if case["state"] == "e4m3":
            m = m.view(E4M3).double() * s["ms"][i].double().repeat_interleave(128)[:n]
            v = (v.view(E4M3).double() * s["vs"][i].double().repeat_interleave(128)[:n]) ** 2
        m = torch.lerp(m.double(), g, 1 - b1)
        v = torch.lerp(v.double(), g * g, 1 - b2)
        step = (m / (1 - b1 ** t)) / (torch.sqrt(v) / (1 - b2 ** t) ** 0.5 + ADAM_EPS)
        p = p * (1 - LR * DECAY) - LR * step
        put(p=p)
        if case["state"] == "e4m3":
            q, sc = _exact_codes(_exact_fill(m))
            put(m=q[:n], ms=sc)
            q, sc = _exact_codes(_exact_fill(torch.sqrt(v)), True)
            put(v=q[:n], vs=sc)
        else:
            put(m=m, v=v)
        if case["copy"]:
            put(copy=p)

    [one(i) for i in range(len(s["p"]))]
    return out


def _exact_open(case, s, l):
    may = ~(torch.isneginf(l) | torch.isnan(l))
    return may if s["valid"] is None else may & s["valid"].reshape(-1, 1)


def _exact_weights(case, l, may, chosen):
    """Scores of the chosen experts (a mask) and probabilities, through logarithms."""
    gone = float("-inf")
    log_score = torch.nn.functional.logsigmoid(l) if case["sigmoid"] else torch.log_softmax(l, 1)
    log_score = torch.where(may, log_score, gone)
    p = torch.where(may, torch.exp(log_score - torch.logsumexp(log_score, 1, keepdim=True)), 0.0)
    if case["norm"]:
        kept = torch.where(chosen, log_score, gone)
        log_score = kept - torch.logsumexp(kept, 1, keepdim=True)
    return torch.where(chosen, torch.exp(torch.where(chosen, log_score, 0.0)), 0.0), p


def _exact_route(case, s):
    l = s["l"].double()
    T, E = l.shape
    may = _exact_open(case, s, l)
    l = torch.where(may, l, -1e4)  # far below every logit that is open
    # ties go to the lowest index: a rank of each value among its row's, as whole numbers
    rank = torch.argsort(torch.argsort(torch.where(may, -l, float("inf")), dim=1, stable=True), dim=1)
    chosen = (rank < case["k"]) & may
    w, p = _exact_weights(case, l, may, chosen)
    place = torch.where(chosen, rank, case["k"])
    weight = torch.zeros(T, case["k"] + 1, dtype=torch.float64, device=l.device).scatter_(1, place, w)[:, :case["k"]]
    n, total = int(may.any(1).sum()), int(chosen.sum())
    loss = E * torch.dot(chosen.double().sum(0) / max(total, 1), p.sum(0) / max(n, 1))
    none = dict.fromkeys(("idx", "counts", "offs", "order", "slot", "tokens"))
    return {**none, "weight": weight * s["scale"], "loss": loss.reshape(1)}


def _exact_route_bwd(case, s):
    """Automatic differentiation of the weights and the loss, with the choice and the counts held."""
    l = s["l"].double()
    T, E = l.shape
    may = _exact_open(case, s, l)
    l = torch.where(may, l, -1e4).requires_grad_()
    has = s["idx"] >= 0
    column = torch.where(has, s["idx"].long(), E)
    spread = torch.zeros(T, E + 1, dtype=torch.float64, device=l.device)
    chosen = spread.scatter(1, column, 1.0)[:, :E] > 0
    dw = spread.scatter(1, column, s["dw"].double())[:, :E]
    alive = may.any(1)
    if not bool(alive.any()):
        return {"dlogits": torch.zeros(T, E, dtype=torch.float64, device=l.device)}
    w, p = _exact_weights(case, l[alive], may[alive], chosen[alive])
    f = s["counts"].double() / int(s["counts"].sum())
    loss = E * (f * p.sum(0)).sum() / int(alive.sum())
    value = (dw[alive] * w).sum() * s["scale"] + s["dloss"].double().sum() * loss
    return {"dlogits": torch.autograd.grad(value, l)[0] * may}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        return _exact_norm(case, s)
    if op == "norm_bwd":
        return _exact_norm_bwd(s)
    if op == "adamw":
        return _exact_adamw(case, s)
    return _exact_route(case, s) if op == "route" else _exact_route_bwd(case, s)
