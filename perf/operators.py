"""Mixture-of-experts operators on quantized weights: the cases they are timed
and checked on, with each operator in plain torch operations.

    moe_route             expert choice: softmax or sigmoid scores, a balancing
                          bias, groups of experts, top-k, renormalised weights
    moe_sort              (token, expert) pairs in expert order, with offsets
    qlinear_experts_bf16  the experts' quantized products (FP8_Dynamic,
                          W8A8_INT8), gate / up with the gated activation or
                          a plain projection
    moe_combine           weighted sum of each token's expert outputs

`own` selects what run() does: False, the plain forms below; True, the calls a
user makes of the library.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
INT8_MAX = 127.0
FLOAT_MAX = 3.4028234663852886e38


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _route(name, T, E, k, score, bias, groups, keep, top, renorm, dtype, masked=0.0, scale=1.0):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias, "groups": groups,
            "keep": keep, "top": top, "renorm": renorm, "dtype": dtype, "masked": masked, "scale": scale}


def _sort(name, T, k, E, dropped=0.0):
    return {"name": name, "op": "sort", "T": T, "k": k, "E": E, "dropped": dropped}


def _experts(name, fmt, T, k, E, K, N, act, skew=0.0):
    """N: output columns (the width after the activation when act is set)."""
    return {"name": name, "op": "experts", "fmt": fmt, "T": T, "k": k, "E": E, "K": K, "N": N, "act": act,
            "skew": skew}


def _combine(name, T, k, H, add, dropped=0.0):
    return {"name": name, "op": "combine", "T": T, "k": k, "H": H, "add": add, "dropped": dropped}


def listed():
    return [
        # one decoded token, choice by biased sigmoid scores inside the best half of 8 groups: all latency
        _route("route_one_token", 1, 256, 8, "sigmoid", True, 8, 4, 2, True, "float32", scale=2.5),
        # a ragged batch over an odd expert count, plain softmax choice, a few experts masked out for some tokens
        _route("route_ragged_batch", 257, 60, 5, "softmax", False, 1, 1, 1, False, "bfloat16", masked=0.3),
        # a prefill batch: biased sigmoid scores, groups
        _route("route_prefill", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, "float32", scale=2.5),
        # one decode step of 32 sequences
        _sort("sort_decode", 32, 8, 128),
        # a padded prefill batch: the pairs of padding tokens (expert -1) are dropped
        _sort("sort_prefill_padded", 32768, 8, 256, dropped=0.125),
        # gate and up projections of one decoded token, int8: eight experts' weights stream once
        _experts("int8_gate_up_one_token", "w8a8_int8", 1, 8, 64, 4096, 1024, True),
        # down projection of a 32-sequence decode step, fp8: every expert, a few rows each
        _experts("fp8_down_decode", "fp8_dynamic", 32, 8, 64, 1024, 4096, False),
        # down projection of an odd batch, int8, odd widths
        _experts("int8_down_odd", "w8a8_int8", 75, 6, 60, 1408, 2048, False),
        # gate and up projections of a short prefill, fp8, uneven expert loads
        _experts("fp8_gate_up_short_prefill", "fp8_dynamic", 517, 4, 32, 2048, 1792, True, skew=0.5),
        # gate and up projections of a long prefill, int8: bound by the tensor cores
        _experts("int8_gate_up_prefill", "w8a8_int8", 8192, 8, 64, 4096, 1024, True, skew=0.5),
        # outputs of one decoded token gathered and weighted
        _combine("combine_one_token", 1, 8, 4096, True),
        # the same for a prefill batch with padding
        _combine("combine_prefill", 8192, 8, 4096, True, dropped=0.05),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "sort", "experts", "experts", "experts", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = _log_int(rng, 4, 64 if groups > 1 else 512)
        E = groups * per
        keep = rng.randint(1, groups)
        return dict(_route("", _log_int(rng, 1, 16384), E, min(rng.randint(1, 10), keep * per),
                           rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, keep, rng.choice([1, 2]),
                           rng.random() < 0.7, rng.choice(["float32", "bfloat16"]),
                           masked=rng.choice([0.0, 0.0, 0.2]), scale=rng.choice([1.0, 2.5])))
    if op == "sort":
        E = _log_int(rng, 4, 512)
        return dict(_sort("", _log_int(rng, 1, 32768), rng.randint(1, min(8, E)), E,
                          dropped=rng.choice([0.0, 0.0, 0.1])))
    if op == "combine":
        return dict(_combine("", _log_int(rng, 1, 8192), rng.randint(1, 8), 8 * _log_int(rng, 16, 512),
                             rng.random() < 0.5, dropped=rng.choice([0.0, 0.05])))
    while True:
        E = _log_int(rng, 4, 128)
        act = rng.random() < 0.5
        c = _experts("", rng.choice(["w8a8_int8", "fp8_dynamic"]), _log_int(rng, 1, 8192), rng.randint(1, min(8, E)), E,
                     16 * _log_int(rng, 16, 256), 16 * _log_int(rng, 8, 128 if act else 256), act,
                     skew=rng.choice([0.0, 0.5]))
        rows = c["N"] * (2 if act else 1)
        if E * rows * c["K"] <= 1 << 30 and c["T"] * c["k"] * rows * c["K"] <= 8192 * 8 * 2048 * 4096:
            return dict(c)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _choose(T, E, k, skew, g):
    """k different experts a token, int32 [T, k]; skew: spread of the experts' popularity."""
    z = torch.rand(T, E, device="cuda", generator=g).clamp_min(1e-30)
    pop = skew * torch.randn(E, device="cuda", generator=g)
    gumbel = -torch.log((-torch.log(z)).clamp_min(1e-30))
    return torch.topk(gumbel + pop, k, dim=1).indices.to(torch.int32)


def _plan(ids, E):
    """offsets, order and positions of the pairs in expert order (-1: dropped)."""
    flat = ids.reshape(-1).long()
    P = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = counts[:E].cumsum(0)
    n = int(offsets[-1])
    pos = torch.full((P,), -1, dtype=torch.int64, device=ids.device)
    pos[order[:n]] = torch.arange(n, device=ids.device)
    order[n:] = -1
    return offsets.int(), order.int(), pos.int().view(ids.shape), counts[:E].tolist()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * torch.randn(T, E, device="cuda", generator=g)
        logits += 0.5 * torch.randn(E, device="cuda", generator=g)
        if case["masked"]:
            # some tokens may not take some experts; a few tokens (padding) may take none
            hide = torch.rand(T, E, device="cuda", generator=g) < case["masked"]
            hide |= torch.rand(T, 1, device="cuda", generator=g) < 0.02
            logits.masked_fill_(hide, float("-inf"))
        s["logits"] = logits.to(getattr(torch, case["dtype"])).contiguous()
        s["bias"] = 0.1 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None
    elif op == "sort":
        ids = _choose(case["T"], case["E"], case["k"], 0.5, g)
        if case["dropped"]:
            ids[torch.rand(case["T"], device="cuda", generator=g) < case["dropped"]] = -1
        s["ids"] = ids
    elif op == "experts":
        T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
        rows = N * (2 if case["act"] else 1)
        s["offsets"], order, _, s["counts"] = _plan(_choose(T, E, k, case["skew"], g), E)
        # the gate and up projections gather each pair's token; the down projection's rows are in expert order
        s["order"] = order if case["act"] else None
        x = torch.randn(T if case["act"] else T * k, K, device="cuda", generator=g)
        x[:, torch.randint(0, K, (max(1, K // 100),), device="cuda", generator=g)] *= 20.0  # outlier channels
        s["x"] = x.bfloat16()
        if case["fmt"] == "w8a8_int8":
            s["wq"] = torch.randint(-127, 128, (E, rows, K), device="cuda", generator=g, dtype=torch.int8)
            step = 0.04 / INT8_MAX
        else:
            wq = torch.empty(E, rows, K, device="cuda", dtype=torch.float8_e4m3fn)
            for e in range(E):
                w = 112.0 * torch.randn(rows, K, device="cuda", generator=g)
                wq[e] = w.clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s["wq"] = wq
            step = 0.02 / 112.0
        s["sw"] = step * (0.5 + torch.rand(E, rows, device="cuda", generator=g))
        s["y"] = torch.zeros(T * k, N, device="cuda", dtype=torch.bfloat16)
    else:
        T, k, H = case["T"], case["k"], case["H"]
        P = T * k
        s["h"] = torch.randn(P, H, device="cuda", generator=g).bfloat16()
        pos = torch.randperm(P, device="cuda", generator=g).to(torch.int32).view(T, k)
        if case["dropped"]:
            pos[torch.rand(T, k, device="cuda", generator=g) < case["dropped"]] = -1
        s["pos"] = pos.contiguous()
        w = torch.rand(T, k, device="cuda", generator=g) + 0.05
        s["weights"] = w / w.sum(1, keepdim=True)
        s["add"] = torch.randn(T, H, device="cuda", generator=g).bfloat16() if case["add"] else None
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _pick(value, count, limit):
    """Indices of the `count` largest of each row, largest first, ties to the
    lowest index; -1 where only -inf is left."""
    value = value.clone()
    cols = torch.arange(value.shape[1], device=value.device)
    out = []
    for _ in range(count):
        best = value.amax(1, keepdim=True)
        i = torch.where(value == best, cols, limit).amin(1, keepdim=True)
        value = torch.where(cols == i, float("-inf"), value)
        out.append(torch.where(best == float("-inf"), -1, i))
    return torch.cat(out, 1)


def _plain_route(logits, bias, k, score, groups, keep, top, renorm, scale):
    x = logits.double()
    x = torch.where(torch.isnan(x), float("-inf"), x).clamp_max(FLOAT_MAX)
    able = x > float("-inf")
    if score == "softmax":
        m = x.amax(1, keepdim=True)
        e = torch.where(able, torch.exp(x - torch.where(m > float("-inf"), m, 0.0)), 0.0)
        total = e.sum(1, keepdim=True)
        s = e / torch.where(total > 0, total, 1.0)
    else:
        s = torch.where(able, 1.0 / (1.0 + torch.exp(-x)), 0.0)
    choice = s if bias is None else s + bias.double()
    choice = torch.where(able, choice, float("-inf"))
    value = x if bias is None else choice  # without a bias the scores' order is the logits'
    T, E = x.shape
    if keep < groups:
        c = (value if top == 1 else choice).view(T, groups, E // groups)
        first = c.amax(2)
        if top == 2:
            cols = torch.arange(E // groups, device=x.device)
            i = torch.where(c == first[..., None], cols, E).amin(2, keepdim=True)
            second = torch.where(cols == i, float("-inf"), c).amax(2)
            first = torch.where(second > float("-inf"), first + second, first)
        best = _pick(first, keep, groups)
        kept = (best[:, :, None] == torch.arange(groups, device=x.device)).any(1)
        value = torch.where(kept.repeat_interleave(E // groups, 1), value, float("-inf"))
    ids = _pick(value, k, E)
    w = torch.where(ids >= 0, s.gather(1, ids.clamp_min(0)), 0.0)
    if renorm:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return (w * scale).float(), ids.int()


def _plain_sort(ids, E):
    flat = ids.reshape(-1).long()
    P = flat.numel()
    hot = torch.arange(E, device=ids.device)[:, None] == flat
    rank = torch.cumsum(hot, 1, dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = rank[:, -1].cumsum(0)
    ok = (flat >= 0) & (flat < E)
    at = flat.clamp(0, E - 1)
    pos = torch.where(ok, offsets[at] + rank.gather(0, at[None])[0] - 1, -1)
    order = torch.full((P + 1,), -1, dtype=torch.int32, device=ids.device)
    order[torch.where(ok, pos, P).long()] = torch.arange(P, dtype=torch.int32, device=ids.device)
    return offsets, order[:P], pos.int().view(ids.shape)


def _plain_quantize(x, fmt):
    x = x.float()
    top = torch.full((1,), E4M3_MAX if fmt == "fp8_dynamic" else INT8_MAX, device=x.device)
    scale = x.abs().amax(1).clamp_min(1e-12) / top
    q = x / scale[:, None]
    if fmt == "fp8_dynamic":
        return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float(), scale
    return q.round().clamp(-INT8_MAX, INT8_MAX), scale


def _plain_experts(s):
    case = s["case"]
    q, scale = _plain_quantize(s["x"], case["fmt"])
    y, begin, N = s["y"], 0, case["N"]
    for e, n in enumerate(s["counts"]):
        if n:
            rows = slice(begin, begin + n)
            at = rows if s["order"] is None else torch.div(s["order"][rows], case["k"], rounding_mode="floor").long()
            v = (q[at] @ s["wq"][e].float().t()) * scale[at][:, None] * s["sw"][e]
            if case["act"]:
                gate, up = v[:, :N], v[:, N:]
                v = gate / (1.0 + torch.exp(-gate)) * up
            y[rows] = v.bfloat16()
            begin += n
    return y


def _plain_combine(h, pos, weights, add):
    y = torch.zeros(pos.shape[0], h.shape[1], device=h.device) if add is None else add.float()
    for j in range(pos.shape[1]):
        p = pos[:, j].long()
        y = y + torch.where(p >= 0, weights[:, j], 0.0)[:, None] * h[p.clamp_min(0)].float()
    return y.bfloat16()


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import quantized_gemm_decode_b200 as qgd
    if op == "route":
        if own:
            return qgd.moe_route(state["logits"], case["k"], score=case["score"], bias=state["bias"],
                                 groups=case["groups"], topk_groups=case["keep"], group_top=case["top"],
                                 renormalize=case["renorm"], scale=case["scale"])
        return _plain_route(state["logits"], state["bias"], case["k"], case["score"], case["groups"], case["keep"],
                            case["top"], case["renorm"], case["scale"])
    if op == "sort":
        if own:
            return qgd.moe_sort(state["ids"], case["E"])
        return _plain_sort(state["ids"], case["E"])
    if op == "experts":
        if own:
            fmt = qgd.FMT_W8A8_INT8 if case["fmt"] == "w8a8_int8" else qgd.FMT_FP8_DYNAMIC
            return qgd.qlinear_experts_bf16(fmt, state["x"], state["wq"], state["sw"], state["offsets"],
                                            order=state["order"], top_k=case["k"] if case["act"] else 1,
                                            act=qgd.ACT_SILU_MUL if case["act"] else qgd.ACT_NONE, y=state["y"])
        return _plain_experts(state)
    if own:
        return qgd.moe_combine(state["h"], state["pos"], state["weights"], add=state["add"])
    return _plain_combine(state["h"], state["pos"], state["weights"], state["add"])


# ---------------------------------------------------------------------------
# Bytes and operations
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": 5 * T * E}
    if op == "sort":
        P = case["T"] * case["k"]
        return {"bytes": 12 * P + 4 * (case["E"] + 1), "flops": P}
    if op == "combine":
        T, k, H = case["T"], case["k"], case["H"]
        live = T * k * (1.0 - case["dropped"])
        return {"bytes": int(2 * live * H + 2 * T * H * (2 if case["add"] else 1) + 8 * T * k),
                "flops": int(2 * live * H)}
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    rows = N * (2 if case["act"] else 1)
    live = E * (1.0 - (1.0 - k / E) ** T)  # experts that at least one token takes, on average
    x = 2 * (T if case["act"] else T * k) * K
    return {"bytes": int(x + live * rows * (K + 4) + 2 * T * k * N + 4 * (E + 1) + (4 * T * k if case["act"] else 0)),
            "flops": 2 * T * k * rows * K}


# ---------------------------------------------------------------------------
# The operators' definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(logits, bias, c):
    z = logits.double()
    z[torch.isnan(z)] = -math.inf
    z[z == math.inf] = FLOAT_MAX
    live = z != -math.inf
    if c["score"] == "softmax":
        p = torch.softmax(torch.where(live, z, -1e300), 1) * live
    else:
        p = torch.sigmoid(z) * live
    key = z.clone() if bias is None else (p + bias.double()).masked_fill(~live, -math.inf)
    T, E = z.shape
    if c["keep"] < c["groups"]:
        per = E // c["groups"]
        src = key if c["top"] == 1 else (p if bias is None else key).masked_fill(~live, -math.inf)
        ranked = src.view(T, c["groups"], per).sort(dim=2, descending=True).values
        value = ranked[..., 0].clone()
        if c["top"] == 2 and per > 1:
            value += ranked[..., 1].masked_fill(ranked[..., 1] == -math.inf, 0.0)
        winners = value.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        open_ = torch.zeros(T, c["groups"], dtype=torch.bool, device=z.device).scatter_(1, winners, True)
        key = key.view(T, c["groups"], per).masked_fill(~open_[..., None], -math.inf).view(T, E)
    top = key.sort(dim=1, descending=True, stable=True)
    ids = top.indices[:, :c["k"]].clone()
    none = top.values[:, :c["k"]] == -math.inf
    w = p.gather(1, ids).masked_fill(none, 0.0)
    ids[none] = -1
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(5e-324)
    return w * c["scale"], ids.int()


def _exact_codes(x, fmt):
    """Codes and scales of the dynamic quantizer: scale and quotient are each
    one division rounded to 32 bits, the code the nearest one, ties to even."""
    v = x.double()
    top = E4M3_MAX if fmt == "fp8_dynamic" else INT8_MAX
    scale = (v.abs().amax(1).clamp_min(float(torch.tensor(1e-12, dtype=torch.float32))) / top).float().double()
    q = (v / scale[:, None]).float().double()
    if fmt != "fp8_dynamic":
        return q.round().clamp(-INT8_MAX, INT8_MAX), scale
    size = q.abs().clamp_max(E4M3_MAX)
    step = torch.exp2(torch.floor(torch.log2(size.clamp_min(2.0 ** -6))) - 3.0)
    return torch.sign(q) * ((size / step).round() * step).clamp_max(E4M3_MAX), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(s["logits"], s["bias"], case)
    if op == "sort":
        offsets, order, pos, _ = _plan(s["ids"], case["E"])
        return offsets, order, pos
    if op == "combine":
        keep = s["pos"] >= 0
        w = torch.where(keep, s["weights"], torch.zeros_like(s["weights"])).double()
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for t in range(0, case["T"], 512):
            rows = s["h"][s["pos"][t:t + 512].clamp_min(0).long()].double()
            out[t:t + 512] = torch.einsum("tk,tkh->th", w[t:t + 512], rows)
        return out if s["add"] is None else out + s["add"].double()
    codes, scale = _exact_codes(s["x"], case["fmt"])
    N, k = case["N"], case["k"]
    out = torch.zeros(case["T"] * k, N, dtype=torch.float64, device="cuda")
    bounds = s["offsets"].tolist()
    for e in range(case["E"]):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        src = torch.arange(a, b, device="cuda") if s["order"] is None else s["order"][a:b].long() // k
        full = (codes[src] @ s["wq"][e].double().T) * scale[src][:, None] * s["sw"][e].double()
        out[a:b] = full[:, :N] * torch.sigmoid(full[:, :N]) * full[:, N:] if case["act"] else full
    return out
