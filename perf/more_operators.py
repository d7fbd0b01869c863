"""What the operators around the FP8 products of a transformer layer are measured
on: the root-mean-square norm with the residual's addition and quantised
outputs (with its gradient), a whole gated mixture-of-experts layer for a few
tokens, and the norm and clipping of a model's gradients.

Each case runs in a plain form (``own`` false: elementary torch operations in
32 bits, long sums in 64) or through the library's entry points (``own`` true).
Codes are e4m3 in 1x128 groups along the features (row codes), 128x1 groups
along the tokens (column codes, written transposed) and 128x128 weight tiles,
with s = max(amax, 1e-12) / 448 and q = RNE(x / s).
"""
import math

import torch

own = False

LIB = "blockwise_scaled_fp8_gb300"
BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-12
SUM_FLOOR = 1e-20   # of the chosen scores' sum, where weights are renormalised
NORM_FLOOR = 1e-6   # added to the gradients' norm before the division
F8 = torch.float8_e4m3fn
DTYPES = dict(bf16=torch.bfloat16, fp16=torch.float16, fp32=torch.float32)


def _lib():
    import importlib
    return importlib.import_module(LIB)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of a served model enters a layer: residual added, codes for the next product and the bf16 row
        # that a router reads; pure latency
        dict(name="norm one token", op="norm", T=1, K=4096, residual=True, cols=False, out=True, weight="bf16", grad=False,
             dh=False),
        # a prompt's tokens, the first norm of a model (no residual yet), a ragged count
        dict(name="norm prompt", op="norm", T=2047, K=5120, residual=False, cols=False, out=False, weight="bf16",
             grad=False, dh=False),
        # a training step: codes for the forward and the weight gradient, backward with the residual stream's gradient
        dict(name="norm step", op="norm", T=16384, K=4096, residual=True, cols=True, out=False, weight="fp32", grad=True,
             dh=True),
        # a smaller model's step with sizes that are multiples of nothing, no gradient from the stream
        dict(name="norm step odd", op="norm", T=5003, K=2001, residual=True, cols=True, out=True, weight="fp32", grad=True,
             dh=False),
        # one new token through the eight gated experts that its router picks: latency and one read of their weights
        dict(name="layer one token", op="layer", T=1, E=64, k=8, K=4096, I=2048, N=4096, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0, dtype="bf16"),
        # a small batch that reaches most experts; sigmoid scores in groups, a bias for balance
        dict(name="layer batch", op="layer", T=16, E=64, k=8, K=4096, I=2048, N=4096, score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renorm=True, scale=2.5, dtype="fp32"),
        # a few tokens of a model with many narrow experts
        dict(name="layer narrow", op="layer", T=5, E=128, k=6, K=1920, I=704, N=1920, score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renorm=False, scale=16.0, dtype="bf16"),
        # gradients of a small model, clipped into the optimizer's fp32 buffers: latency
        dict(name="clip small", op="clip", tensors=40, numel=2_000_000, dtype="bf16", out="fp32", ragged=True, clip=True),
        # gradients of some layers of a large model, clipped
        dict(name="clip layers", op="clip", tensors=48, numel=1_200_000_000, dtype="bf16", out="bf16", ragged=False,
             clip=True),
        # the norm alone, of tensors of several types, for a log
        dict(name="norm of mixed", op="clip", tensors=61, numel=150_000_000, dtype="mixed", out="none", ragged=True,
             clip=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "layer", "clip"])
    if op == "norm":
        K = rng.choice([_log(rng, 64, 8192) // 8 * 8, _log(rng, 128, 8192) // 128 * 128, _log(rng, 33, 8192)])
        grad = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, min(20000, 64_000_000 // K)), K=K, residual=rng.random() < 0.6,
                    cols=rng.random() < 0.5, out=rng.random() < 0.5, weight=rng.choice(["bf16", "fp32"]), grad=grad,
                    dh=grad and rng.random() < 0.5)
    if op == "layer":
        score = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4])
        E = groups * _log(rng, 8, 96 // groups)
        K = rng.choice([_log(rng, 256, 4096) // 128 * 128, _log(rng, 200, 4096)])
        return dict(op=op, T=rng.randint(1, 16), E=E, k=rng.randint(1, min(8, E // groups)), K=K,
                    I=_log(rng, 128, 1536) // 64 * 64, N=_log(rng, 256, 4096) // 128 * 128, score=score,
                    bias=score == "sigmoid" and rng.random() < 0.5, groups=groups,
                    top_groups=groups if groups == 1 else rng.randint(2, groups), group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["bf16", "fp32"]))
    clip = rng.random() < 0.7
    return dict(op=op, tensors=rng.randint(1, 60), numel=_log(rng, 1000, 300_000_000),
                dtype=rng.choice(["bf16", "fp16", "fp32", "mixed"]), out=rng.choice(["bf16", "fp32"]) if clip else "none",
                ragged=rng.random() < 0.6, clip=clip)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _codes_of(w):
    """128x128 tiles of w [E, N, K]: the library's code buffer [E*N, K up to a multiple of 16] and scales [E*Nb, Kb]."""
    E, N, K = w.shape
    Nb, Kb = -(-N // BLOCK), -(-K // BLOCK)
    q = torch.zeros(E, N, -(-K // 16) * 16, dtype=torch.uint8, device=w.device)
    s = torch.empty(E, Nb, Kb, device=w.device)
    for e in range(0, E, 8):  # (eight experts at a time, for the room that the 32-bit forms take)
        v = w[e:e + 8]
        p = torch.zeros(v.shape[0], Nb * BLOCK, Kb * BLOCK, device=w.device)
        p[:, :N, :K] = v
        p = p.view(-1, Nb, BLOCK, Kb, BLOCK)
        s[e:e + 8] = p.abs().amax((2, 4)).clamp_min(AMAX_FLOOR) / E4M3_MAX
        p = (p / s[e:e + 8, :, None, :, None]).view(-1, Nb * BLOCK, Kb * BLOCK)
        q[e:e + 8, :, :K] = p[:, :N, :K].to(F8).view(torch.uint8)
    return q.view(E * N, -1), s.view(E * Nb, Kb)


def _sizes(case):
    """Elements of each tensor of a model: most of them in a few matrices, the rest small."""
    n, total = case["tensors"], case["numel"]
    big = max(1, n // 2)
    sizes = [max(1, total // big - (i * 37 if case["ragged"] else 0)) for i in range(big)]
    return (sizes + [max(1, min(4096, total // n) - (i if case["ragged"] else 0)) for i in range(n - big)])[:n]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    bf = torch.bfloat16
    s = dict(case=case, eps=1e-6)
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        # a residual stream: tokens of different sizes, a few features much larger than the rest
        wide = 1 + 8 * (torch.rand(K, generator=g, device="cuda") < 0.01)
        s["x"] = (n(T, K) * (0.2 + 2 * torch.rand(T, 1, generator=g, device="cuda")) * wide).to(bf)
        s["residual"] = (n(T, K) * wide).to(bf) if case["residual"] else None
        s["weight"] = (1 + 0.2 * n(K)).to(DTYPES[case["weight"]])
        s["dy"] = n(T, K).mul_(1e-3).to(bf) if case["grad"] else None
        s["dh"] = n(T, K).mul_(1e-3).to(bf) if case["dh"] else None
        return s
    if case["op"] == "layer":
        T, E, K, I, N = (case[i] for i in ("T", "E", "K", "I", "N"))
        s["x"] = n(T, K).to(bf)
        s["logits"] = (1.5 * n(T, E) + 0.7 * n(E)).to(DTYPES[case["dtype"]])
        s["bias"] = 0.05 * n(E) if case["bias"] else None
        # the experts' weights, quantised once: gate rows, then up rows, of each expert; then the way down
        s["qgu"], s["sgu"] = _codes_of(n(E, 2 * I, K).mul_(1.3 / K ** 0.5).to(bf))
        s["qd"], s["sd"] = _codes_of(n(E, N, I).mul_(1.3 / I ** 0.5).to(bf))
        return s
    kinds = ["bf16", "fp32", "fp16"]
    s["grads"], s["out"] = [], [] if case["clip"] else None
    for i, size in enumerate(_sizes(case)):
        kind = DTYPES[kinds[i % 3] if case["dtype"] == "mixed" else case["dtype"]]
        off = i % 3 if case["ragged"] else 0  # views of a larger buffer that start anywhere in it
        buf = torch.empty(size + off, dtype=kind, device="cuda")
        buf[off:] = n(size).mul_(1e-2 / (1 + i % 5))
        s["grads"].append(buf[off:].view(-1, 4096) if size % 4096 == 0 else buf[off:])
        if case["clip"]:
            s["out"].append(torch.empty_like(s["grads"][-1], dtype=DTYPES[case["out"]]))
    s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _group_quant(x):
    """1x128 groups of x [T, K] fp32: codes [T, K] and scales [Kb, T]."""
    T, K = x.shape
    p = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(T, -1, BLOCK)
    s = p.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (p / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(F8)
    return q.view(T, -1)[:, :K], s.t()


def _norm(st):
    case, bf = st["case"], torch.bfloat16
    h = st["x"]
    out = {}
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(bf)
        out["h"] = h
    hf, w = h.float(), st["weight"].float()
    rstd = 1 / torch.sqrt((hf * hf).sum(1) / case["K"] + st["eps"])
    y = hf * rstd[:, None] * w
    out["rstd"] = rstd
    out["q_row"], out["s_row"] = _group_quant(y)
    if case["cols"]:
        out["q_col"], out["s_col"] = _group_quant(y.t())
    if case["out"]:
        out["y"] = y.to(bf)
    if case["grad"]:
        dy = st["dy"].float()
        n, g = hf * rstd[:, None], dy * w
        dx = rstd[:, None] * (g - n * ((g * n).sum(1) / case["K"])[:, None])
        out["dx"] = (dx if st["dh"] is None else dx + st["dh"].float()).to(bf)
        out["dweight"] = (dy * n).sum(0, dtype=torch.float64).float()
    return out


def _route(st):
    """The experts of each token [T, k] and their weights."""
    case, logits = st["case"], st["logits"].float()
    T, E = logits.shape
    G = case["groups"]
    if case["score"] == "sigmoid":
        p = 1 / (1 + torch.exp(-logits))
        c = p if st["bias"] is None else p + st["bias"]
        g = c
    else:
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        p, c, g = e / e.sum(1, keepdim=True), logits, e
    if G > 1:
        best = torch.sort(g.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    idx = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :case["k"]]
    w = p.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(SUM_FLOOR)
    return idx, case["scale"] * w


def _weight_of(q, s, e, N, K, real):
    """Expert e's weight [N, K] from its codes and scales."""
    Nb = -(-N // BLOCK)
    s = s[e * Nb:(e + 1) * Nb].to(real).repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]
    return q[e * N:(e + 1) * N].view(F8)[:, :K].to(real) * s


def _group_values(x):
    """x [T, K] fp32 after its quantisation in 1x128 groups."""
    q, s = _group_quant(x)
    return q.float() * s.t().repeat_interleave(BLOCK, 1)[:, :x.shape[1]]


def _layer(st):
    case = st["case"]
    T, E, K, I, N = (case[i] for i in ("T", "E", "K", "I", "N"))
    idx, w = _route(st)
    dense = torch.zeros(T, E, device=w.device).scatter_(1, idx, w)
    x = _group_values(st["x"].float())
    y = torch.zeros(T, N, device=w.device)
    for e in range(E):  # every token through every expert, most of them with weight 0
        gu = torch.matmul(x, _weight_of(st["qgu"], st["sgu"], e, 2 * I, K, torch.float32).t())
        gate, up = gu[:, :I], gu[:, I:]
        a = _group_values(gate / (1 + torch.exp(-gate)) * up)
        y += dense[:, e:e + 1] * torch.matmul(a, _weight_of(st["qd"], st["sd"], e, N, I, torch.float32).t())
    return dict(y=y.to(torch.bfloat16))


def _clip(st):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in st["grads"]:
        f = t.float()
        total += (f * f).sum(dtype=torch.float64)
    norm = torch.sqrt(total).float()
    out = dict(norm=norm)
    if st["out"] is not None:
        coef = (st["max_norm"] / (norm + NORM_FLOOR)).clamp_max(1.0)
        for t, o in zip(st["grads"], st["out"]):
            o.copy_(t.float() * coef)
        out["grads"] = st["out"]
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    B = _lib()
    case = st["case"]
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        r = B.rms_norm_quant(st["x"], st["weight"], residual=st["residual"], eps=st["eps"], cols=case["cols"],
                             out=case["out"])
        out = dict(rstd=r.rstd, q_row=r.q_row.view(F8)[:, :K], s_row=r.s_row[:, :T])
        if case["residual"]:
            out["h"] = r.h
        if case["cols"]:
            out |= dict(q_col=r.q_col.view(F8)[:, :T], s_col=r.s_col[:, :K])
        if case["out"]:
            out["y"] = r.y
        if case["grad"]:
            out["dx"], out["dweight"] = B.rms_norm_bwd(st["dy"], r.h, st["weight"], r.rstd, dh=st["dh"])
        return out
    if case["op"] == "layer":
        return dict(y=B.moe_mlp_decode(st["x"], st["logits"], case["k"], st["qgu"], st["sgu"], st["qd"], st["sd"],
                                       I=case["I"], N=case["N"], bias=st["bias"], score=case["score"],
                                       groups=case["groups"], top_groups=case["top_groups"],
                                       group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"]))
    if st["out"] is None:
        return dict(norm=B.grad_norm(st["grads"]))
    return dict(norm=B.clip_grads(st["grads"], st["max_norm"], out=st["out"]), grads=st["out"])


def run(st):
    if own:
        return _run_own(st)
    return dict(norm=_norm, layer=_layer, clip=_clip)[st["case"]["op"]](st)


def work(case):
    if case["op"] == "norm":
        T, K = case["T"], case["K"]
        Kb, Tb = -(-K // BLOCK), -(-T // BLOCK)
        w = 2 if case["weight"] == "bf16" else 4
        n, b, f = T * K, 2 * T * K + w * K + 4 * T, 6 * T * K
        b += n + 4 * Kb * T + (4 * n if case["residual"] else 0) + (2 * n if case["out"] else 0)
        if case["cols"]:
            b, f = b + n + 4 * Tb * K, f + 3 * n
        if case["grad"]:  # dy, the stream and its gradient in; dx and the weight's gradient out
            b, f = b + 6 * n + (2 * n if case["dh"] else 0) + (w + 4) * K + 4 * T, f + 10 * n
        return dict(bytes=b, flops=f)
    if case["op"] == "layer":
        T, E, k, K, I, N = (case[i] for i in ("T", "E", "k", "K", "I", "N"))
        # the experts that T tokens with k distinct choices each reach, were all liked alike
        reached = E * (1 - (1 - k / E) ** T)
        tiles = -(-2 * I // BLOCK) * -(-K // BLOCK) + -(-N // BLOCK) * -(-I // BLOCK)
        el = 2 if case["dtype"] == "bf16" else 4
        return dict(bytes=reached * (2 * I * K + N * I + 4 * tiles) + 2 * T * K + el * T * E + 2 * T * N,
                    flops=2 * T * k * (2 * I * K + N * I))
    size = dict(bf16=2, fp16=2, fp32=4, mixed=8 / 3, none=0)
    n = sum(_sizes(case))
    return dict(bytes=n * (size[case["dtype"]] + size[case["out"]]), flops=(3 if case["clip"] else 2) * n)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_quant(x):
    """x [A, C] in 64 bits: x / s before rounding, and s, of groups of 128 along C."""
    A, C = x.shape
    full = torch.nn.functional.pad(x, (0, -C % BLOCK)).view(A, -1, BLOCK)
    s = full.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (full / s[:, :, None]).reshape(A, -1)[:, :C], s.t()


def _exact_norm(st):
    case, d = st["case"], torch.float64
    x = st["x"].to(d)
    out = {}
    if st["residual"] is not None:
        out["h"] = x + st["residual"].to(d)
        x = (st["x"].float() + st["residual"].float()).to(torch.bfloat16).to(d)  # the stream that is kept is bf16
    w = st["weight"].to(d)
    rstd = (x.square().mean(1) + st["eps"]).rsqrt()
    n = x * rstd[:, None]
    y = n * w
    out["rstd"] = rstd
    out["q_row"], out["s_row"] = _exact_quant(y)
    if case["cols"]:
        out["q_col"], out["s_col"] = _exact_quant(y.t().contiguous())
    if case["out"]:
        out["y"] = y
    if case["grad"]:
        dy = st["dy"].to(d)
        out["dweight"] = (dy * n).sum(0)
        dn = dy * w
        # the derivative of n = x (mean(x^2) + eps)^-1/2
        dx = dn * rstd[:, None] - x * (rstd ** 3 * (dn * x).mean(1))[:, None]
        out["dx"] = dx if st["dh"] is None else dx + st["dh"].to(d)
    return out


def _exact_layer(st):
    case, d = st["case"], torch.float64
    T, E, k, G, I, N, K = (case[i] for i in ("T", "E", "k", "groups", "I", "N", "K"))
    l = st["logits"].to(d)
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    c = p if st["bias"] is None else p + st["bias"].to(d)
    if G > 1:
        score = c.view(T, G, -1).topk(min(case["group_top"], E // G), 2).values.sum(2)
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, score.topk(case["top_groups"], 1).indices, True)
        c = c.view(T, G, -1).masked_fill(~keep[:, :, None], -math.inf).reshape(T, E)
    idx = c.topk(k, 1).indices
    w = p.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(SUM_FLOOR)
    w = w * case["scale"]

    def held(v):  # the values that the e4m3 codes of 1x128 groups stand for
        q, s = _exact_quant(v)
        q = q.float().to(F8).to(d)
        return q * s.t().repeat_interleave(BLOCK, 1)[:, :v.shape[1]]

    # the input's scales and quotients are fp32 ones, one division each
    full = torch.nn.functional.pad(st["x"].float(), (0, -K % BLOCK)).view(T, -1, BLOCK)
    s = full.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR) / E4M3_MAX
    x = ((full / s).to(F8).to(d) * s.to(d)).view(T, -1)[:, :K]
    y = torch.zeros(T, N, dtype=d, device="cuda")
    for e in idx.unique().tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        gu = x[t] @ _weight_of(st["qgu"], st["sgu"], e, 2 * I, K, d).t()
        a = held(torch.nn.functional.silu(gu[:, :I]) * gu[:, I:])
        y[t] += w[t, j][:, None] * (a @ _weight_of(st["qd"], st["sd"], e, N, I, d).t())
    return dict(y=y)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(st)
    if case["op"] == "layer":
        return _exact_layer(st)
    norm = torch.stack([torch.linalg.vector_norm(t.reshape(-1), dtype=torch.float64) for t in st["grads"]]).norm()
    out = dict(norm=norm)
    if st["out"] is not None:
        coef = min(1.0, st["max_norm"] / (float(norm) + NORM_FLOOR))
        out["grads"] = [t.double() * coef for t in st["grads"]]
    return out
