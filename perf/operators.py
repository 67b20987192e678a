"""Measured cases of the gated feed-forward operators and of the Newton-Schulz orthogonalisation.

Operators (``op``):

- ``ffn``      both projections of a gated feed-forward block, the activation and the product,
               from FP8 codes: h = silu(X Wg^T) * (X Wu^T).  X is E4M3 with one scale per 1x128
               tile, [Wg; Wu] is E4M3 with one scale per 128x128 block.
- ``experts``  the same for tokens sorted by expert, each segment with its expert's weights.
- ``ffn_bwd``  its backward pass down to the gradients of the two projections' outputs, as BF16
               and / or as the FP8 operands of the following Dgrad and Wgrad products.
- ``ortho``    the orthogonalised update of a weight gradient: a fixed number of Newton-Schulz
               steps X <- a X + (b A + c A^2) X, A = X X^T, from X = G / (|G| + eps).

``run`` computes them from elementary torch operations in 32 bits, or, where ``own`` is true, with
the library's kernels.  FP8 outputs are float8_e4m3fn tensors beside their FP32 scales.
"""
import torch

own = False

E4M3 = torch.float8_e4m3fn
COEFFS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # one token in the serving loop: two 2048 x 7168 projections, FP8 result for the down projection
        dict(name="ffn 1 token", op="ffn", M=1, F=2048, K=7168, pow2=False, h=False, gu=False, codes=True),
        # a batch of decoding requests through a wide block
        dict(name="ffn 24 tokens", op="ffn", M=24, F=7168, K=7168, pow2=False, h=False, gu=False, codes=True),
        # an odd number of prompt tokens through a small block, every output asked for
        dict(name="ffn 333 tokens", op="ffn", M=333, F=640, K=896, pow2=False, h=True, gu=True, codes=True),
        # training forward: the projections are kept for the backward pass, FP8 result for the down projection
        dict(name="ffn 8192 tokens", op="ffn", M=8192, F=2048, K=7168, pow2=False, h=False, gu=True, codes=True),
        # training forward with power-of-two scales, wide block, BF16 result
        dict(name="ffn 4096 pow2", op="ffn", M=4096, F=7168, K=7168, pow2=True, h=True, gu=True, codes=False),
        # mixture of experts: 16 experts with uneven shares of 16384 tokens, one of them empty
        dict(name="experts 16x16384", op="experts", M=16384, G=16, F=2048, K=7168, pow2=False, h=True, gu=False,
             codes=True),
        # a micro-batch of 128 tokens of a small block, all gradients: launch latency counts
        dict(name="ffn_bwd 128x640", op="ffn_bwd", T=128, F=640, d=True, rows=True, cols=True, h=True),
        # training backward: FP8 operands of Dgrad and of both Wgrads
        dict(name="ffn_bwd 8192x2048", op="ffn_bwd", T=8192, F=2048, d=False, rows=True, cols=True, h=True),
        # an odd number of tokens, wide block: BF16 gradient and the FP8 operand of Dgrad
        dict(name="ffn_bwd 5003x7168", op="ffn_bwd", T=5003, F=7168, d=True, rows=True, cols=False, h=False),
        # the weight gradient of a 2048 x 7168 projection, accumulated in FP32
        dict(name="ortho 2048x7168", op="ortho", B=1, m=2048, n=7168, bf16=False, steps=5),
        # sixteen experts' tall BF16 gradients in one call
        dict(name="ortho 16x896x640", op="ortho", B=16, m=896, n=640, bf16=True, steps=5),
        # one small matrix of odd sizes: latency counts
        dict(name="ortho 301x999", op="ortho", B=1, m=301, n=999, bf16=False, steps=5),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    while True:
        op = rng.choice(["ffn", "ffn", "ffn", "experts", "ffn_bwd", "ffn_bwd", "ortho", "ortho"])
        F, K = 128 * log_int(1, 56), 128 * log_int(1, 56)
        outs = rng.choice([(True, False, False), (False, False, True), (True, True, False), (False, True, True)])
        if op == "ffn":
            pow2 = rng.random() < 0.4
            c = dict(op=op, M=log_int(1, 16384), F=F, K=K, pow2=pow2, h=outs[0] or pow2, gu=outs[1],
                     codes=outs[2] and not pow2)
        elif op == "experts":
            G = log_int(2, 32)
            pow2 = rng.random() < 0.4
            c = dict(op=op, M=log_int(16, 16384), G=G, F=F, K=K, pow2=pow2, h=outs[0] or pow2, gu=outs[1],
                     codes=outs[2] and not pow2)
        elif op == "ffn_bwd":
            T = log_int(1, 16384)
            if rng.random() < 0.7:
                T = 128 * (T // 128 + 1)
            cols = T % 128 == 0
            c = dict(op=op, T=T, F=F, d=rng.random() < 0.5 or not cols, rows=rng.random() < 0.7, cols=cols,
                     h=cols and rng.random() < 0.7)
        else:
            c = dict(op=op, B=log_int(1, 16), m=log_int(64, 4096), n=log_int(64, 7168), bf16=rng.random() < 0.5,
                     steps=5)
        w = work(c)
        # no dearer than the largest listed case, and with inputs that are quickly made; 3072 is no size
        # of this repository's workloads
        if w["flops"] <= 6.5e11 and w["bytes"] <= 6.5e8 and 3072 not in c.values():
            return c


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))


def _randn(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std)


def _scales(amax, pow2):
    """Scale of each group and the factor its values are multiplied by."""
    a = amax.clamp_min(2.0 ** -116)
    if not pow2:
        return a / 448.0, 448.0 / a
    mant, exp = torch.frexp(a / 448.0)  # a / 448 = mant * 2^exp, mant in [0.5, 1)
    e = torch.where(mant == 0.5, exp - 1, exp)
    return torch.ldexp(torch.ones_like(a), e), torch.ldexp(torch.ones_like(a), -e)


def _quant_rows(x, pow2):
    """1x128 tiles of x [M][K]: codes [M][K] and scales [K/128][M]."""
    M, K = x.shape
    t = x.reshape(M, K // 128, 128)
    s, inv = _scales(t.abs().amax(-1), pow2)
    return (t * inv[..., None]).reshape(M, K).to(E4M3), s.t().contiguous()


def _quant_cols(x, pow2):
    """128x1 tiles of x [T][C]: transposed codes [C][T] and scales [T/128][C]."""
    T, C = x.shape
    t = x.reshape(T // 128, 128, C)
    s, inv = _scales(t.abs().amax(1), pow2)
    return (t * inv[:, None, :]).reshape(T, C).t().contiguous().to(E4M3), s.contiguous()


def _quant_blocks(w, pow2):
    """128x128 blocks of w [N][K]: codes [N][K] and scales [N/128][K/128]."""
    N, K = w.shape
    t = w.reshape(N // 128, 128, K // 128, 128)
    s, inv = _scales(t.abs().amax((1, 3)), pow2)
    return (t * inv[:, None, :, None]).reshape(N, K).to(E4M3), s.contiguous()


def _tokens(g, M, K, pow2):
    """Activations with a few outlier entries, rounded to BF16, then quantised."""
    x = _randn(g, M, K)
    x = torch.where(torch.rand(M, K, generator=g, device="cuda") < 1e-3, x * 100.0, x)
    q, s = _quant_rows(x.bfloat16().float(), pow2)
    return q.view(torch.uint8), s


def _weights(g, N, K, pow2):
    q, s = _quant_blocks(_randn(g, N, K, std=0.02).bfloat16().float(), pow2)
    return q.view(torch.uint8), s


def _offsets(M, G, seed):
    """Row offsets of G experts over M tokens: uneven shares, the second expert empty."""
    r = torch.Generator().manual_seed(int(seed) + 77)
    share = torch.rand(G, generator=r) + 0.05
    share[1] = 0.0
    edges = torch.cat([torch.zeros(1), torch.cumsum(share / share.sum(), 0)])
    offs = (edges * M).round().long().clamp_(0, M)
    offs[-1] = M
    return offs.tolist()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=dict(case))
    if op in ("ffn", "experts"):
        F, K, pow2 = case["F"], case["K"], case["pow2"]
        s["a"], s["sa"] = _tokens(g, case["M"], K, pow2)
        if op == "ffn":
            s["b"], s["sb"] = _weights(g, 2 * F, K, pow2)
        else:
            G = case["G"]
            s["b"] = torch.empty(G, 2 * F, K, dtype=torch.uint8, device="cuda")
            s["sb"] = torch.empty(G, 2 * F // 128, K // 128, device="cuda")
            for e in range(G):
                s["b"][e], s["sb"][e] = _weights(g, 2 * F, K, pow2)
            s["rows"] = _offsets(case["M"], G, seed)
            s["offs"] = torch.tensor(s["rows"], dtype=torch.int32, device="cuda")
    elif op == "ffn_bwd":
        T, F = case["T"], case["F"]
        s["dh"] = _randn(g, T, F, std=1e-3).bfloat16()
        s["gu"] = _randn(g, T, 2 * F, std=1.7).bfloat16()
    else:
        # a gradient: a decaying spectrum of directions over a floor of noise
        B, m, n = case["B"], case["m"], case["n"]
        r = max(1, min(m, n) // 8)
        decay = torch.arange(1, r + 1, device="cuda", dtype=torch.float32).rsqrt()
        G = (_randn(g, B, m, r) * decay) @ _randn(g, B, r, n)
        G = G / G.square().mean().sqrt() + _randn(g, B, m, n)
        s["g"] = (G * 1e-4).to(torch.bfloat16 if case["bf16"] else torch.float32)
    return s


# ----------------------------------------------------------------------------- plain forms
def _values_rows(q, s):
    M, K = q.shape
    return (q.view(E4M3).float().reshape(M, K // 128, 128) * s.t()[..., None]).reshape(M, K)


def _values_blocks(q, s):
    N, K = q.shape
    return (q.view(E4M3).float().reshape(N // 128, 128, K // 128, 128) * s[:, None, :, None]).reshape(N, K)


def _ffn_outputs(case, gu):
    F = case["F"]
    g, u = gu[:, :F], gu[:, F:]
    h = g / (1.0 + torch.exp(-g)) * u
    out = {}
    if case["h"]:
        out["h"] = h.bfloat16()
    if case["gu"]:
        out["gu"] = gu.bfloat16()
    if case["codes"]:
        out["q"], out["s"] = _quant_rows(h, False)
    return out


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ffn":
        return _ffn_outputs(case, _values_rows(s["a"], s["sa"]) @ _values_blocks(s["b"], s["sb"]).t())
    if op == "experts":
        x = _values_rows(s["a"], s["sa"])
        parts = [x[lo:hi] @ _values_blocks(s["b"][e], s["sb"][e]).t()
                 for e, (lo, hi) in enumerate(zip(s["rows"], s["rows"][1:])) if hi > lo]
        return _ffn_outputs(case, torch.cat(parts))
    if op == "ffn_bwd":
        F = case["F"]
        dh, gu = s["dh"].float(), s["gu"].float()
        g, u = gu[:, :F], gu[:, F:]
        sig = 1.0 / (1.0 + torch.exp(-g))
        d = torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1)
        out = {}
        if case["d"]:
            out["d"] = d.bfloat16()
        if case["rows"]:
            out["q"], out["s"] = _quant_rows(d, False)
        if case["cols"]:
            out["qT"], out["sT"] = _quant_cols(d, False)
        if case["h"]:
            out["hT"], out["shT"] = _quant_cols(g * sig * u, False)
        return out
    a, b, c = COEFFS
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(case["steps"]):
        A = x @ x.transpose(1, 2)
        x = a * x + (b * A + c * (A @ A)) @ x
    return (x.transpose(1, 2) if tall else x).contiguous().bfloat16()


def _own(s):
    import fp8_fine_grained_amax_gb300 as fq
    case = s["case"]
    op = case["op"]
    if op in ("ffn", "experts"):
        want = dict(with_h=case["h"], with_gu=case["gu"], with_codes=case["codes"])
        if op == "ffn":
            call = fq.fp8q_gemm_swiglu_pow2 if case["pow2"] else fq.fp8q_gemm_swiglu
            r = call(s["a"], s["sa"], s["b"], s["sb"], **want)
        else:
            call = fq.fp8q_grouped_gemm_swiglu_pow2 if case["pow2"] else fq.fp8q_grouped_gemm_swiglu
            r = call(s["a"], s["sa"], s["b"], s["sb"], s["offs"], **want)
        out = {}
        if case["h"]:
            out["h"] = r.h
        if case["gu"]:
            out["gu"] = r.gu
        if case["codes"]:
            out["q"], out["s"] = r.q.view(E4M3), r.s
        return out
    if op == "ffn_bwd":
        r = fq.fp8q_swiglu_bwd(s["dh"], s["gu"], with_d=case["d"], with_rows=case["rows"], with_cols=case["cols"],
                               with_h=case["h"])
        out = {}
        if case["d"]:
            out["d"] = r.d
        if case["rows"]:
            out["q"], out["s"] = r.q.view(E4M3), r.s
        if case["cols"]:
            out["qT"], out["sT"] = r.qT.view(E4M3), r.sT
        if case["h"]:
            out["hT"], out["shT"] = r.hT.view(E4M3), r.shT
        return out
    return fq.fp8q_newton_schulz(s["g"], steps=case["steps"], coeffs=COEFFS, eps=EPS)


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op in ("ffn", "experts"):
        M, F, K = case["M"], case["F"], case["K"]
        G = case.get("G", 1)
        # an expert without tokens reads no weights
        G = max(1, min(G - 1, M)) if op == "experts" else 1
        b = M * K + M * K // 32 + G * (2 * F * K + 2 * F * K // 4096)
        b += M * F * (2 * case["h"] + 4 * case["gu"]) + case["codes"] * (M * F + M * F // 32)
        return {"bytes": b, "flops": 4.0 * M * F * K}
    if op == "ffn_bwd":
        n = case["T"] * case["F"]
        b = 6 * n + 4 * n * case["d"] + 2 * n * case["rows"] + 2 * n * case["cols"] + n * case["h"]
        b += n // 32 * (2 * case["rows"] + 2 * case["cols"] + case["h"])
        return {"bytes": b, "flops": 20.0 * n}
    B, m, n = case["B"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # X X^T and A A are symmetric: half of each is enough
    return {"bytes": B * m * n * (2 if case["bf16"] else 4) + 2 * B * m * n,
            "flops": 1.0 * B * case["steps"] * (3.0 * m * m * n + m * m * m)}


# ----------------------------------------------------------------------------- 64 bits
def _exact_rows(x):
    """Unrounded 1x128 codes and scales: what E4M3 then rounds."""
    M, K = x.shape
    a = x.abs().reshape(M, K // 128, 128).max(-1).values
    return (x.reshape(M, K // 128, 128) / a[..., None] * 448).reshape(M, K), a.t() / 448


def _exact_cols(x):
    q, s = _exact_rows(x.t().contiguous())
    return q, s


def _exact_ffn(case, gu):
    g, u = gu.split(case["F"], 1)
    h = 0.5 * g * (1 + torch.tanh(0.5 * g)) * u
    out = {}
    if case["h"]:
        out["h"] = h
    if case["gu"]:
        out["gu"] = gu
    if case["codes"]:
        out["q"], out["s"] = _exact_rows(h)
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("ffn", "experts"):
        x = s["a"].view(E4M3).double() * s["sa"].double().t().repeat_interleave(128, 1)
        rows = s.get("rows", [0, case["M"]])
        b = s["b"].reshape(-1, 2 * case["F"], case["K"])
        sb = s["sb"].reshape(b.shape[0], 2 * case["F"] // 128, case["K"] // 128)
        gu = torch.empty(case["M"], 2 * case["F"], dtype=torch.float64, device="cuda")
        for e in range(b.shape[0]):
            w = sb[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1) * b[e].view(E4M3).double()
            gu[rows[e]:rows[e + 1]] = torch.mm(x[rows[e]:rows[e + 1]], w.t())
        return _exact_ffn(case, gu)
    if op == "ffn_bwd":
        dh = s["dh"].double()
        g, u = s["gu"].double().split(case["F"], 1)
        t = torch.tanh(0.5 * g)
        silu = 0.5 * g * (1 + t)
        slope = 0.5 * (1 + t) + 0.25 * g * (1 - t * t)
        d = torch.cat([dh * u * slope, dh * silu], 1)
        out = {}
        if case["d"]:
            out["d"] = d
        if case["rows"]:
            out["q"], out["s"] = _exact_rows(d)
        if case["cols"]:
            out["qT"], out["sT"] = _exact_cols(d)
        if case["h"]:
            out["hT"], out["shT"] = _exact_cols(silu * u)
        return out
    # the iteration acts on the singular values alone: an odd polynomial of each, applied through the
    # eigenvectors of the Gram matrix of the shorter side
    a, b, c = COEFFS
    x = s["g"].double()
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + EPS)
    lam, V = torch.linalg.eigh(x @ x.mT)
    gain = torch.ones_like(lam)
    for _ in range(case["steps"]):
        p = a + b * lam + c * lam * lam
        gain, lam = gain * p, lam * p * p
    x = (V * gain[:, None, :]) @ (V.mT @ x)
    return (x.mT if tall else x).contiguous()
