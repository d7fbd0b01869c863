"""What the mixture-of-experts operators are measured on: the router (scores,
choice and weights of the experts, with its gradient), the plan that sorts the
routed slots by expert, the dispatch that gathers tokens into quantised
operands, the combine of the experts' outputs (with its gradient), and the
routed FP8 product of decode-sized batches.

Each case runs in a plain form (``own`` false: elementary torch operations in
32 bits) or through the library's entry points (``own`` true).  A slot is a
(token t, choice j) pair, flat index t * k + j; a row is a place of the
sorted buffers; row[t, j] is a slot's row (-1: the slot goes nowhere) and
src[r] a row's slot (-1: padding).
"""
import math

import torch

own = False

LIB = "blockwise_scaled_fp8_gb300"
BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 1e-12
SUM_FLOOR = 1e-20  # of the chosen scores' sum, where weights are renormalised


def _lib():
    import importlib
    return importlib.import_module(LIB)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one new token of a served model picks its experts: pure latency
        dict(name="route one token", op="route", T=1, E=64, k=6, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=True, scale=1.0, dtype="bf16", grad=False, empty=0.0),
        # a training batch over many experts in groups, sigmoid scores, a bias for balance, padding tokens masked
        dict(name="route groups", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, renorm=True, scale=2.5, dtype="fp32", grad=False, empty=0.01),
        # a training step's router, forward and backward; a ragged token count, an odd expert count
        dict(name="route step", op="route", T=50021, E=160, k=6, score="softmax", bias=False, groups=1, top_groups=1,
             group_top=1, renorm=False, scale=16.0, dtype="bf16", grad=True, empty=0.0),
        # slots of a decode batch, packed without padding
        dict(name="plan decode", op="plan", T=48, E=256, k=8, align=1, empty=0.0),
        # slots of a training batch, every expert on a 128-row boundary, padding tokens routed nowhere
        dict(name="plan train", op="plan", T=16384, E=256, k=8, align=128, empty=0.01),
        # forward dispatch of the MoE-mid token count, two experts a token
        dict(name="dispatch mid", op="dispatch", T=4096, E=8, k=2, K=4096, weighted=False, cols=True, empty=0.0),
        # backward dispatch of a training batch, eight experts a token, rows scaled by the routing weights
        dict(name="dispatch train", op="dispatch", T=16384, E=64, k=8, K=4096, weighted=True, cols=True, empty=0.01),
        # a decode batch's experts joined
        dict(name="combine decode", op="combine", T=48, E=256, k=8, N=4096, align=1, grad=False, dye=False, empty=0.0),
        # a training step's combine: outputs, the gradient of the experts' outputs and of the weights
        dict(name="combine step", op="combine", T=16384, E=64, k=8, N=4096, align=128, grad=True, dye=True, empty=0.01),
        # one new token through its eight experts: eight weights read once
        dict(name="product one token", op="product", T=1, E=64, k=8, N=2048, K=4096),
        # a decode batch that reaches nearly every expert
        dict(name="product batch", op="product", T=32, E=64, k=8, N=2048, K=4096),
        # few experts with dozens of rows each, ragged sizes, a last K-block of 80
        dict(name="product ragged", op="product", T=150, E=8, k=2, N=1000, K=2000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "plan", "dispatch", "combine", "product"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 8, 256 // groups if groups > 1 else 384)
        score = rng.choice(["softmax", "sigmoid"])
        top = groups if groups == 1 else rng.randint(groups // 2, groups)
        k = rng.randint(1, min(8, E // groups))
        grad = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 32768 if grad else 65536), E=E, k=k, score=score,
                    bias=score == "sigmoid" and rng.random() < 0.5, groups=groups, top_groups=top,
                    group_top=rng.choice([1, 2]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["bf16", "fp32"]), grad=grad, empty=rng.choice([0.0, 0.02]))
    if op == "plan":
        return dict(op=op, T=_log(rng, 1, 20000), E=_log(rng, 4, 512), k=rng.randint(1, 8), align=rng.choice([1, 128]),
                    empty=rng.choice([0.0, 0.02]))
    if op == "dispatch":
        return dict(op=op, T=_log(rng, 16, 8192), E=_log(rng, 4, 128), k=rng.randint(1, 8),
                    K=rng.choice([_log(rng, 128, 4096) // 8 * 8, _log(rng, 128, 4096) // 128 * 128, _log(rng, 100, 2000)]),
                    weighted=rng.random() < 0.5, cols=rng.random() < 0.7, empty=rng.choice([0.0, 0.02]))
    if op == "combine":
        grad = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 12000), E=_log(rng, 8, 256), k=rng.randint(1, 8), N=_log(rng, 128, 4096),
                    align=rng.choice([1, 128]), grad=grad, dye=grad and rng.random() < 0.5, empty=rng.choice([0.0, 0.02]))
    E = _log(rng, 4, 64)
    return dict(op=op, T=_log(rng, 1, 128), E=E, k=rng.randint(1, min(8, E)), N=_log(rng, 128, 2048),
                K=rng.choice([_log(rng, 128, 4096), _log(rng, 128, 4096) // 128 * 128]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(T, k, E, align):
    n = T * k
    return (n + min(E, n) * (align - 1)) // align * align


def _choices(g, T, E, k, empty):
    """Distinct experts a token, unevenly liked, some tokens routed nowhere."""
    like = torch.randn(E, generator=g, device="cuda") * 0.5
    idx = torch.topk(torch.randn(T, E, generator=g, device="cuda") + like, min(k, E), dim=1).indices.to(torch.int32)
    if k > E:
        idx = torch.cat([idx, torch.full((T, k - E), -1, dtype=torch.int32, device="cuda")], 1)
    if empty:
        idx = torch.where(torch.rand(T, 1, generator=g, device="cuda") < empty, -1, idx)
    return idx.contiguous()


def _plan_plain(idx, E, align):
    """Slots sorted by expert, in slot order within one; each expert's first row a multiple of align."""
    T, k = idx.shape
    R = _rows(T, k, E, align)
    flat = idx.reshape(-1).to(torch.int64)
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    counts = torch.bincount(key, minlength=E + 1)
    offs = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    offs[1:] = torch.cumsum((counts[:E] + align - 1) // align * align, 0)
    order = torch.sort(key, stable=True).indices
    first = torch.cumsum(counts, 0) - counts
    k_sorted = key[order]
    place = torch.arange(T * k, device=idx.device) - first[k_sorted] + offs[k_sorted]
    place = torch.where(k_sorted < E, place, -1)
    row = torch.empty(T * k, dtype=torch.int64, device=idx.device)
    row[order] = place
    src = torch.full((R + 1,), -1, dtype=torch.int64, device=idx.device)
    src[torch.where(place >= 0, place, R)] = order
    return dict(offs=offs.to(torch.int32), row=row.reshape(T, k).to(torch.int32), src=src[:R].to(torch.int32),
                counts=counts[:E].to(torch.int32))


def _tile_quant(w):
    """128x128 tiles of w [E, N, K] bf16: codes [E, N, K] and scales [E, Nb, Kb]."""
    E, N, K = w.shape
    Nb, Kb = -(-N // BLOCK), -(-K // BLOCK)
    p = torch.zeros(E, Nb * BLOCK, Kb * BLOCK, device=w.device)
    p[:, :N, :K] = w.float()
    p = p.view(E, Nb, BLOCK, Kb, BLOCK)
    s = p.abs().amax((2, 4)).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (p / s[:, :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(E, Nb * BLOCK, Kb * BLOCK)[:, :N, :K].contiguous(), s


def _group_quant(x):
    """1x128 groups of x [T, K]: codes [T, K] float8, scales [Kb, T]."""
    T, K = x.shape
    Kb = -(-K // BLOCK)
    p = torch.zeros(T, Kb * BLOCK, device=x.device)
    p[:, :K] = x
    p = p.view(T, Kb, BLOCK)
    s = p.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    q = (p / s[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(T, Kb * BLOCK)[:, :K], s.t().contiguous()


def _pad16(codes):
    """The library's code buffers: bytes, rows of a multiple of 16."""
    n = codes.shape[1]
    buf = torch.zeros(codes.shape[0], -(-n // 16) * 16, dtype=torch.uint8, device=codes.device)
    buf[:, :n] = codes.view(torch.uint8)
    return buf


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    s = dict(case=case)
    if op == "route":
        # logits of a trained router: a spread of a few units, experts unevenly liked
        s["logits"] = (1.5 * n(T, E) + 0.7 * n(E)).to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        if case["empty"]:  # padding tokens: every expert masked
            s["logits"][torch.rand(T, generator=g, device="cuda") < case["empty"]] = -math.inf
        s["bias"] = 0.05 * n(E) if case["bias"] else None
        s["dw"] = 1e-3 * n(T, k) if case["grad"] else None
        return s
    idx = _choices(g, T, E, k, case.get("empty", 0.0))
    if op == "plan":
        s["idx"] = idx
        return s
    s["plan"] = _plan_plain(idx, E, case.get("align", 1 if op == "product" else BLOCK))
    R = s["plan"]["src"].numel()
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    w = w / w.sum(1, keepdim=True)
    if op == "dispatch":
        s["x"] = n(T, case["K"]).mul_(1e-3 if case["weighted"] else 1.0).to(torch.bfloat16)
        s["w"] = w if case["weighted"] else None
    elif op == "combine":
        s["ye"] = n(R, case["N"]).to(torch.bfloat16)
        s["dy"] = n(T, case["N"]).mul_(1e-3).to(torch.bfloat16) if case["grad"] else None
        s["w"] = w
    else:
        N, K = case["N"], case["K"]
        q, s["sb"] = _tile_quant((0.02 * n(E, N, K)).to(torch.bfloat16))
        s["qb"] = _pad16(q.reshape(E * N, K))
        s["sb"] = s["sb"].reshape(-1, s["sb"].shape[2]).contiguous()
        del q
        qa, s["sa"] = _group_quant(n(T, K).to(torch.bfloat16).float())
        s["qa"] = _pad16(qa)
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _chosen(c, g, case):
    """The experts of each token: idx [T, k] int64, -1 where none is left.  c
    [T, E]: what is compared (-inf: not eligible), g: what a group's score sums
    the largest of."""
    T, E = c.shape
    k, G = case["k"], case["groups"]
    none = torch.full_like(c, -math.inf)
    c = torch.where(torch.isneginf(g), none, c)
    if G > 1:
        best = torch.sort(g.view(T, G, E // G), dim=2, descending=True).values[:, :, :case["group_top"]]
        score = torch.where(torch.isneginf(best), torch.zeros_like(best), best).sum(2)
        score = torch.where(torch.isneginf(best[:, :, 0]), none[:, :G], score)
        kept = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        mask = torch.zeros(T, G, dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = torch.where(mask.repeat_interleave(E // G, 1), c, none)
    top = torch.sort(c, dim=1, descending=True, stable=True)
    return torch.where(torch.isneginf(top.values[:, :k]), -1, top.indices[:, :k])


def _scores(logits, case, real):
    """Scores [T, E] and the eligible experts, in the type `real`."""
    l = logits.to(real)
    ok = l > torch.finfo(logits.dtype).min
    l = torch.where(ok, l, torch.full_like(l, -math.inf))
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
        e = s
    else:
        top = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(torch.isneginf(top), torch.zeros_like(top), top))
        s = e / e.sum(1, keepdim=True).clamp_min(torch.finfo(real).tiny)
    return l, e, s, ok


def _route(st, real):
    case, logits, bias = st["case"], st["logits"], st["bias"]
    l, e, s, ok = _scores(logits, case, real)
    none = torch.full_like(s, -math.inf)
    if case["score"] == "sigmoid":
        c = s if bias is None else s + bias.to(real)
        g = c
    else:
        c, g = l, e  # the softmax keeps the logits' order; a group's sum needs no common denominator
    idx = _chosen(torch.where(ok, c, none), torch.where(ok, g, none), case)
    live = idx >= 0
    zero = torch.zeros((), dtype=real, device=s.device)
    sel = torch.where(live, s.gather(1, idx.clamp_min(0)), zero)
    total = sel.sum(1, keepdim=True).clamp_min(SUM_FLOOR)
    w = case["scale"] * (sel / total if case["renorm"] else sel)
    out = dict(idx=idx.to(torch.int32), w=w.to(real))
    if case["grad"]:
        dw = torch.where(live, st["dw"].to(real), zero)
        if case["renorm"]:
            ds = (case["scale"] * dw - (dw * w).sum(1, keepdim=True)) / total
            ds = torch.where(live, ds, zero)
        else:
            ds = case["scale"] * dw
        dense = torch.zeros_like(s).scatter_add_(1, idx.clamp_min(0), ds)
        if case["score"] == "sigmoid":
            dl = dense * s * (1 - s)
        else:
            dl = s * (dense - (ds * sel).sum(1, keepdim=True))
        out["dlogits"] = torch.where(ok, dl, zero)
    return out


def _gathered(st):
    """The dispatched rows [R, K]: the token of each row, scaled by its weight; zeros on padding."""
    src, k = st["plan"]["src"].long(), st["case"]["k"]
    at = src.clamp_min(0)
    x = st["x"][at // k].float()
    if st["w"] is not None:
        x = x * st["w"].reshape(-1)[at][:, None]
    return torch.where((src >= 0)[:, None], x, torch.zeros((), device=x.device))


def _dispatch(st):
    x = _gathered(st)
    q, s = _group_quant(x)
    out = dict(q_row=q, s_row=s)
    if st["case"]["cols"]:
        q, s = _group_quant(x.t())
        out |= dict(q_col=q, s_col=s)
    return out


def _combine(st, real):
    case, row = st["case"], st["plan"]["row"].long()
    live = row >= 0
    ye = torch.where(live[:, :, None], st["ye"][row.clamp_min(0)].to(real), torch.zeros((), dtype=real, device=row.device))
    w = torch.where(live, st["w"].to(real), torch.zeros((), dtype=real, device=row.device))
    out = dict(y=(ye * w[:, :, None]).sum(1))
    if case["grad"]:
        dy = st["dy"].to(real)
        out["dw"] = (ye * dy[:, None, :]).sum(2)
        if case["dye"]:
            src, k = st["plan"]["src"].long(), case["k"]
            at = src.clamp_min(0)
            d = dy[at // k] * w.reshape(-1)[at][:, None]
            out["dye"] = torch.where((src >= 0)[:, None], d, torch.zeros((), dtype=real, device=row.device))
    return out


def _product(st, real):
    """Row r of the routed product: the codes of its slot's token against its expert's weight."""
    case, plan = st["case"], st["plan"]
    T, E, k, N, K = (case[i] for i in ("T", "E", "k", "N", "K"))
    Kb, Nb = -(-K // BLOCK), -(-N // BLOCK)
    b = st["qb"].view(torch.float8_e4m3fn)[:, :K].to(real).view(E, N, K)
    b = b * st["sb"].to(real).view(E, Nb, Kb).repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    a = st["qa"].view(torch.float8_e4m3fn)[:, :K].to(real)
    a = a * st["sa"].to(real).t().repeat_interleave(BLOCK, 1)[:, :K]
    every = torch.matmul(a, b.view(E * N, K).t()).view(T, E, N)  # every token against every expert
    src = plan["src"].long()
    r = torch.arange(src.numel(), device=src.device)
    e = torch.searchsorted(plan["offs"].long(), r, right=True) - 1
    return every[src // k, e]


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def _run_own(st):
    B = _lib()
    case, op = st["case"], st["case"]["op"]
    if op == "route":
        how = dict(score=case["score"], groups=case["groups"], top_groups=case["top_groups"], group_top=case["group_top"],
                   renormalize=case["renorm"], scale=case["scale"])
        idx, w = B.moe_route(st["logits"], case["k"], bias=st["bias"], **how)
        out = dict(idx=idx, w=w)
        if case["grad"]:
            out["dlogits"] = B.moe_route_bwd(st["logits"], idx, w, st["dw"], score=case["score"],
                                             renormalize=case["renorm"], scale=case["scale"])
        return out
    if op == "plan":
        p = B.moe_plan(st["idx"], case["E"], align=case["align"])
        return dict(offs=p.offs, row=p.row, src=p.src, counts=p.counts)
    plan = B.MoePlan(**st["plan"])
    if op == "dispatch":
        q, s, qt, stt = B.moe_dispatch(st["x"], plan, weight=st["w"], cols=case["cols"])
        f8 = torch.float8_e4m3fn
        out = dict(q_row=q.view(f8)[:, :case["K"]], s_row=s)
        if case["cols"]:
            out |= dict(q_col=qt.view(f8)[:, :plan.src.numel()], s_col=stt[:, :case["K"]])
        return out
    if op == "combine":
        out = dict(y=B.moe_combine(st["ye"], plan, st["w"]))
        if case["grad"]:
            dye, out["dw"] = B.moe_combine_bwd(st["dy"], st["ye"], plan, st["w"], with_dye=case["dye"])
            if case["dye"]:
                out["dye"] = dye
        return out
    return dict(c=B.gemm_routed_1x128_128x128(st["qa"], st["sa"], st["qb"], st["sb"], plan, case["N"], case["K"]))


def run(st):
    if own:
        return _run_own(st)
    case, op, real = st["case"], st["case"]["op"], torch.float32
    bf = torch.bfloat16
    if op == "route":
        out = _route(st, real)
        if case["grad"]:
            out["dlogits"] = out["dlogits"].to(st["logits"].dtype)
        return out
    if op == "plan":
        return _plan_plain(st["idx"], case["E"], case["align"])
    if op == "dispatch":
        return _dispatch(st)
    if op == "combine":
        out = _combine(st, real)
        return {name: v if name == "dw" else v.to(bf) for name, v in out.items()}
    return dict(c=_product(st, real).to(bf))


def work(case):
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    if op == "route":
        el = 2 if case["dtype"] == "bf16" else 4
        b = T * E * el + T * k * 8
        f = T * E * 8
        if case["grad"]:  # logits again, the choice and its gradient in, the logits' gradient out
            b, f = b + 2 * T * E * el + T * k * 12, 2 * f
        return dict(bytes=b, flops=f)
    R = _rows(T, k, E, case.get("align", 1 if op == "product" else BLOCK))
    if op == "plan":
        return dict(bytes=4 * (2 * T * k + R + 2 * E + 1), flops=4 * T * k)
    if op == "dispatch":
        K = case["K"]
        Kb, Rb = -(-K // BLOCK), -(-R // BLOCK)
        b = 2 * T * K + 4 * R + R * K + 4 * Kb * R + (4 * T * k if case["weighted"] else 0)
        if case["cols"]:
            b += R * K + 4 * Rb * K
        return dict(bytes=b, flops=(6 if case["cols"] else 3) * R * K)
    if op == "combine":
        N = case["N"]
        b, f = 2 * T * k * N + 2 * T * N + 8 * T * k, 2 * T * k * N
        if case["grad"]:
            b, f = b + 2 * T * k * N + 2 * T * N + 12 * T * k, f + 2 * T * k * N
            if case["dye"]:
                b, f = b + 2 * R * N, f + T * k * N
        return dict(bytes=b, flops=f)
    N, K = case["N"], case["K"]
    # the experts that T tokens with k distinct choices each reach, were all liked alike
    reached = E * (1 - (1 - min(k, E) / E) ** T)
    return dict(bytes=reached * (N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK)) + T * K + 2 * R * N, flops=2 * R * N * K)


# ---------------------------------------------------------------------------
# The definitions in 64 bits, one token, group or row at a time in form
# ---------------------------------------------------------------------------

def _exact_route(st):
    case = st["case"]
    T, E, k, G = (case[i] for i in ("T", "E", "k", "groups"))
    raw = st["logits"]
    ok = raw > torch.finfo(raw.dtype).min
    l = raw.double().masked_fill(~ok, -math.inf)
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1).nan_to_num(0.0)
    c = p.clone() if st["bias"] is None else p + st["bias"].double()
    c[~ok] = -math.inf
    if G > 1:
        best = c.view(T, G, -1).topk(min(case["group_top"], E // G), 2).values
        score = best.masked_fill(best == -math.inf, 0.0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        order = torch.argsort(score, dim=1, descending=True, stable=True)
        rank = torch.empty_like(order).scatter_(1, order, torch.arange(G, device=order.device).expand(T, G).contiguous())
        c = c.view(T, G, -1).masked_fill((rank >= case["top_groups"])[:, :, None], -math.inf).reshape(T, E)
    idx = torch.empty(T, k, dtype=torch.long, device=c.device)
    for j in range(k):  # one choice after another, the lowest index of equal ones
        best = c.amax(1, keepdim=True)
        first = (c == best).to(torch.uint8).argmax(1)
        idx[:, j] = torch.where(best[:, 0] == -math.inf, -1, first)
        c.scatter_(1, first[:, None], -math.inf)
    on = idx >= 0
    at = idx.clamp_min(0)
    w = p.gather(1, at) * on
    total = w.sum(1, keepdim=True).clamp_min(SUM_FLOOR)
    if case["renorm"]:
        w = w / total
    out = dict(idx=None, w=case["scale"] * w)
    if case["grad"]:
        dw = st["dw"].double() * on * case["scale"]
        if case["renorm"]:  # the derivative of s_j / sum(s)
            dw = (dw - (dw * w).sum(1, keepdim=True)) / total * on
        dp = torch.zeros_like(p).scatter_add_(1, at, dw)
        if case["score"] == "sigmoid":
            out["dlogits"] = dp * p * (1 - p)
        else:
            out["dlogits"] = p * dp - p * (p * dp).sum(1, keepdim=True)
    return out


def _exact_quant(x, block):
    """x [A, C] in 64 bits: x / s before rounding, and s, of blocks along C."""
    A, C = x.shape
    full = torch.nn.functional.pad(x, (0, -C % block)).view(A, -1, block)
    s = full.abs().amax(2).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (full / s[:, :, None]).reshape(A, -1)[:, :C], s.t()


def exact(case, seed):
    st = prepare(case, seed)
    op, k = case["op"], case["k"]
    if op == "route":
        return _exact_route(st)
    if op == "plan":
        return None
    if op == "dispatch":
        src = st["plan"]["src"].long()
        x = torch.zeros(src.numel(), case["K"], dtype=torch.float64, device="cuda")
        on = torch.nonzero(src >= 0)[:, 0]
        x[on] = st["x"][src[on] // k].double()
        if st["w"] is not None:
            x[on] *= st["w"].flatten()[src[on]].double()[:, None]
        q, s = _exact_quant(x, BLOCK)
        out = dict(q_row=q, s_row=s)
        if case["cols"]:
            q, s = _exact_quant(x.t().contiguous(), BLOCK)
            out |= dict(q_col=q, s_col=s)
        return out
    if op == "combine":
        T, N, row = case["T"], case["N"], st["plan"]["row"].long()
        y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        dye = torch.zeros(st["ye"].shape, dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(row[:, j] >= 0)[:, 0]
            e = st["ye"][row[t, j]].double()
            y[t] += e * st["w"][t, j].double()[:, None]
            if case["grad"]:
                dw[t, j] = (e * st["dy"][t].double()).sum(1)
                dye[row[t, j]] = st["dy"][t].double() * st["w"][t, j].double()[:, None]
        out = dict(y=y)
        if case["grad"]:
            out["dw"] = dw
            if case["dye"]:
                out["dye"] = dye
        return out
    N, K = case["N"], case["K"]
    Nb = -(-N // BLOCK)
    offs, src = st["plan"]["offs"].tolist(), st["plan"]["src"].long()
    c = torch.zeros(src.numel(), N, dtype=torch.float64, device="cuda")
    wide = lambda s, n: s.double().repeat_interleave(BLOCK, 0)[:n]  # noqa: E731
    for e in range(case["E"]):
        if offs[e + 1] > offs[e]:
            rows = src[offs[e]:offs[e + 1]] // k
            a = st["qa"].view(torch.float8_e4m3fn)[rows, :K].double() * wide(st["sa"][:, rows], K).t()
            sb = wide(wide(st["sb"][e * Nb:(e + 1) * Nb], N).t(), K).t()
            c[offs[e]:offs[e + 1]] = a @ (st["qb"].view(torch.float8_e4m3fn)[e * N:(e + 1) * N, :K].double() * sb).t()
    return dict(c=c)
