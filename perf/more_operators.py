"""Measured cases of the gated router and the int8 products.

Two operators, each with its plain form (elementary torch operations) and the
call of this package that does the same:

  route    a router's logits, their scores (softmax over the experts, or a
           sigmoid each), a bias that counts for the choice only, the choice of
           groups of experts and of the K experts in them, and the weights of
           the chosen (renormalised or not, scaled);
  product  products grouped by expert of int8 rows with a scale each (tokens)
           and int8 matrices with a scale for each output channel, plain or with
           the SwiGLU of two matrices.

route, for a token x with logits l_e = x . router_w[e] (+ router_bias[e]) and
scores s_e: the choice values are c_e = s_e + select_bias[e]. With G groups of
E/G consecutive experts, a group's value is its largest c or the sum of its two
largest; the group_topk groups of the largest values stay. Of their experts, the
K with the largest c are taken, in descending order. Ties go to the lower index
throughout; a value of -inf is never taken (id -1, weight 0). The weights are
the scores of the chosen, divided by their sum if renorm, times scale.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a small decode: two of 16 experts, balanced by a bias
        {"name": "route-1-token", "op": "route", "T": 1, "d": 4096, "E": 16, "K": 2, "act": "bf16",
         "score": "softmax", "select": True, "disabled": 0, "groups": 1, "group_topk": 1, "group_by": "max",
         "renorm": True, "scale": 1.0},
        # a decode batch, grouped experts, sigmoid scores
        {"name": "route-decode-63", "op": "route", "T": 63, "d": 8192, "E": 64, "K": 6, "act": "bf16",
         "score": "sigmoid", "select": True, "disabled": 0, "groups": 8, "group_topk": 3, "group_by": "top2",
         "renorm": True, "scale": 2.5},
        # prompt processing of the large layer's shape
        {"name": "route-prefill-16", "op": "route", "T": 16384, "d": 8192, "E": 16, "K": 2, "act": "bf16",
         "score": "sigmoid", "select": True, "disabled": 0, "groups": 1, "group_topk": 1, "group_by": "max",
         "renorm": True, "scale": 1.0},
        # prompt processing with many experts that several GPUs share
        {"name": "route-prefill-256", "op": "route", "T": 8192, "d": 4096, "E": 256, "K": 8, "act": "bf16",
         "score": "sigmoid", "select": True, "disabled": 0, "groups": 8, "group_topk": 4, "group_by": "top2",
         "renorm": True, "scale": 2.5},
        # an odd number of fp32 tokens, three experts taken out of service, weights as they are
        {"name": "route-ragged-f32", "op": "route", "T": 2999, "d": 4096, "E": 60, "K": 4, "act": "f32",
         "score": "softmax", "select": True, "disabled": 3, "groups": 4, "group_topk": 2, "group_by": "max",
         "renorm": False, "scale": 1.0},
        # one token through the layer's gate/up: two experts' weights are read
        {"name": "swiglu-1-token", "op": "product", "T": 1, "d": 4096, "f": 14336, "E": 16, "K": 2, "skew": 0.0,
         "gather": True, "swiglu": True, "out": "bf16", "scale": "bf16"},
        # a decode batch of the large layer: every expert's down weights are read
        {"name": "down-decode-64", "op": "product", "T": 64, "d": 24576, "f": 8192, "E": 16, "K": 2, "skew": 0.0,
         "gather": False, "swiglu": False, "out": "f32", "scale": "bf16"},
        # a dense MLP's gate/up at decode: one expert takes every token
        {"name": "dense-64", "op": "product", "T": 64, "d": 8192, "f": 24576, "E": 1, "K": 1, "skew": 0.0,
         "gather": False, "swiglu": True, "out": "bf16", "scale": "bf16"},
        # a short prompt, unevenly spread, sizes that fill no tile
        {"name": "swiglu-ragged-333", "op": "product", "T": 333, "d": 4160, "f": 1472, "E": 40, "K": 3, "skew": 0.5,
         "gather": True, "swiglu": True, "out": "bf16", "scale": "f32"},
        # prompt processing
        {"name": "swiglu-prefill", "op": "product", "T": 8192, "d": 4096, "f": 14336, "E": 16, "K": 2, "skew": 0.0,
         "gather": True, "swiglu": True, "out": "bf16", "scale": "bf16"},
        # the largest: the down product of a long prompt chunk, two experts crowded
        {"name": "down-skewed", "op": "product", "T": 16384, "d": 24576, "f": 8192, "E": 16, "K": 2, "skew": 1.0,
         "gather": False, "swiglu": False, "out": "f32", "scale": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["route", "product"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        size = _log_int(rng, 2 if groups > 1 else 4, 256 // groups)
        E = groups * size
        group_topk = rng.randint(1, groups)
        case = {"op": op, "T": _log_int(rng, 1, 16384), "d": _log_int(rng, 256, 8192, 64), "E": E,
                "K": rng.randint(1, min(8, group_topk * size)), "act": rng.choice(["bf16", "bf16", "f32"]),
                "score": rng.choice(["softmax", "sigmoid"]), "select": rng.random() < 0.75, "disabled": 0,
                "groups": groups, "group_topk": group_topk, "group_by": rng.choice(["max", "top2"]),
                "renorm": rng.random() < 0.75, "scale": rng.choice([1.0, 2.5])}
        if case["select"] and rng.random() < 0.25:
            case["disabled"] = rng.randint(1, max(1, E // 8))
        while work(case)["flops"] > 2 * 8192 * 4096 * 256:
            case["T"] = max(1, case["T"] // 2)
        return case
    E = _log_int(rng, 1, 64)
    case = {"op": op, "T": _log_int(rng, 1, 16384), "d": _log_int(rng, 256, 24576, 64),
            "f": _log_int(rng, 256, 24576, 64), "E": E, "K": min(E, rng.choice([1, 2, 2, 4, 8])),
            "skew": rng.choice([0.0, 0.5, 1.0]), "gather": rng.random() < 0.5, "swiglu": rng.random() < 0.5,
            "out": rng.choice(["bf16", "f32"]), "scale": rng.choice(["bf16", "f32"])}
    while E * 2 * case["d"] * case["f"] > 16 * 8192 * 24576:
        case["f"] = max(256, case["f"] // 2 // 64 * 64)
    while work(case)["flops"] > 1.3e13:
        case["T"] = max(1, case["T"] // 2)
    return case


# ------------------------------------------------------------------ inputs

def _draw_int8(gen, rows, cols, sigma):
    """Normal numbers as int8 with a scale a row: codes [rows, cols], scales [rows], drawn in slabs of rows."""
    q = torch.empty(rows, cols, dtype=torch.int8, device=DEV)
    s = torch.empty(rows, device=DEV)
    slab = max(1, (1 << 27) // cols)
    for r in range(0, rows, slab):
        n = min(slab, rows - r)
        v = torch.randn(n, cols, generator=gen, device=DEV) * sigma
        top = v.abs().amax(1) / 127
        q[r:r + n] = torch.round(v / top.unsqueeze(1)).clamp(-127, 127).to(torch.int8)
        s[r:r + n] = top
    return q, s


def _draw_routing(gen, T, E, K, skew):
    """Slots grouped by expert; skew crowds the first experts and leaves late ones empty."""
    logits = torch.randn(T, E, generator=gen, device=DEV)
    logits -= skew * 0.5 * torch.arange(E, device=DEV)
    ids = logits.topk(K, dim=1).indices.reshape(-1)
    slots = torch.argsort(ids, stable=True).to(torch.int32)
    counts = torch.bincount(ids, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return slots, offsets, counts.tolist()


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": dict(case)}
    T, d, E, K = case["T"], case["d"], case["E"], case["K"]

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=gen, device=DEV) * scale).to(dtype)

    if case["op"] == "route":
        dt = DTYPES[case["act"]]
        st["x"] = randn(T, d, dtype=dt)
        st["router_w"] = randn(E, d, dtype=dt, scale=0.02)
        st["router_bias"] = randn(E, scale=0.1) if case["score"] == "softmax" else None
        st["select_bias"] = None
        if case["select"]:
            # a balancing bias is of the size of the differences between scores
            b = randn(E, scale=0.05 if case["score"] == "sigmoid" else 0.2 / E)
            off = torch.randperm(E, generator=gen, device=DEV)[:case["disabled"]]
            b[off] = -math.inf
            st["select_bias"] = b
        if own:
            import int8_weight_moe_amd as m
            st["gate"] = m.Gate(
                score=m.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else m.MOE_SCORE_SOFTMAX,
                select_bias=st["select_bias"], groups=case["groups"], group_topk=case["group_topk"],
                group_by=m.MOE_GROUP_TOP2 if case["group_by"] == "top2" else m.MOE_GROUP_MAX,
                renorm=case["renorm"], scale=case["scale"])
        return st

    f = case["f"]
    st["slots"], st["offsets"], st["counts"] = _draw_routing(gen, T, E, K, case["skew"])
    st["a_q"], st["a_s"] = _draw_int8(gen, T if case["gather"] else T * K, d, 1.0)
    for name in ("w0", "w1") if case["swiglu"] else ("w0",):
        q, s = _draw_int8(gen, E * f, d, 0.02)
        q, s = q.view(E, f, d), s.view(E, f).to(DTYPES[case["scale"]])
        if own:
            import int8_weight_moe_amd as m
            q = m.moe_pack_rows(q)
        st[name + "_q"], st[name + "_s"] = q, s
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import int8_weight_moe_amd as m
    c = st["case"]
    if c["op"] == "route":
        return m.moe_route_gated(st["x"], st["router_w"], st["router_bias"], c["K"], st["gate"])
    return m.moe_grouped_mm_int8(st["a_q"], st["a_s"], st["offsets"], st["w0_q"], st["w0_s"], DTYPES[c["out"]],
                                 sorted_slots=st["slots"] if c["gather"] else None, K=c["K"] if c["gather"] else 1,
                                 w2_q=st.get("w1_q"), w2_s=st.get("w1_s"))


def _run_plain(st):
    c = st["case"]
    E, K = c["E"], c["K"]
    if c["op"] == "route":
        # in 64 bits: which of two values that differ by their rounding is larger decides the ids
        l = st["x"].double() @ st["router_w"].double().t()
        if st["router_bias"] is not None:
            l = l + st["router_bias"].double()
        if c["score"] == "softmax":
            z = torch.exp(l - l.amax(1, keepdim=True))
            score = z / z.sum(1, keepdim=True)
        else:
            score = 1 / (1 + torch.exp(-l))
        choice = score if st["select_bias"] is None else score + st["select_bias"].double()
        G = c["groups"]
        if G > 1:
            by_group = choice.view(-1, G, E // G)
            if c["group_by"] == "top2":
                value = by_group.sort(2, descending=True).values[:, :, :2].sum(2)
            else:
                value = by_group.amax(2)
            dropped = value.sort(dim=1, descending=True, stable=True).indices[:, c["group_topk"]:]
            mask = torch.zeros_like(value, dtype=torch.bool).scatter_(1, dropped, True)
            choice = torch.where(mask.unsqueeze(2), -math.inf, by_group).view(-1, E)
        top = choice.sort(dim=1, descending=True, stable=True)
        taken = top.values[:, :K] > -math.inf
        w = torch.where(taken, score.gather(1, top.indices[:, :K]), 0.0)
        if c["renorm"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, 0.0)
        return torch.where(taken, top.indices[:, :K], -1).to(torch.int32), (w * c["scale"]).float()

    out = torch.empty(c["T"] * K, c["f"], dtype=DTYPES[c["out"]], device=DEV)
    r0 = 0
    for e in range(E):
        r1 = r0 + st["counts"][e]
        if r1 == r0:
            continue
        rows = st["slots"][r0:r1] // K if c["gather"] else slice(r0, r1)
        a, a_s = st["a_q"][rows].float(), st["a_s"][rows].unsqueeze(1)
        p = [(a @ st[n + "_q"][e].float().t()) * st[n + "_s"][e].float() * a_s
             for n in (("w0", "w1") if c["swiglu"] else ("w0",))]
        out[r0:r1] = (p[0] / (1 + torch.exp(-p[0])) * p[1] if len(p) == 2 else p[0]).to(out.dtype)
        r0 = r1
    return out


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    T, d, E, K = case["T"], case["d"], case["E"], case["K"]
    if case["op"] == "route":
        b = 2 if case["act"] == "bf16" else 4
        biases = E * 4 * ((case["score"] == "softmax") + case["select"])
        return {"bytes": (T + E) * d * b + biases + T * K * 8, "flops": 2 * T * d * E}
    f, S = case["f"], T * K
    hit = min(E, S)   # experts with rows, at most
    mats = 2 if case["swiglu"] else 1
    weights = hit * mats * f * (d + (2 if case["scale"] == "bf16" else 4))
    rows = T if case["gather"] else S
    return {"bytes": weights + rows * (d + 4) + S * f * (2 if case["out"] == "bf16" else 4),
            "flops": 2 * mats * S * d * f}


# ------------------------------------------------------------------ the definition in 64 bits

def _first_max(v):
    """Index of the largest value of each row, the lowest of equal ones."""
    n = v.shape[1]
    i = torch.arange(n, device=v.device).expand_as(v)
    return torch.where(v == v.amax(1, keepdim=True), i, n).amin(1)


def _exact_route(case, st):
    E, K, G = case["E"], case["K"], case["groups"]
    logits = torch.empty(case["T"], E, dtype=torch.float64, device=DEV)
    w = st["router_w"].double()
    for t in range(0, case["T"], 2048):
        logits[t:t + 2048] = torch.mm(st["x"][t:t + 2048].double(), w.t())
    if st["router_bias"] is not None:
        logits += st["router_bias"].double()
    if case["score"] == "softmax":
        s = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    else:
        s = torch.where(logits > 0, 1 / (1 + torch.exp(-logits.abs())),
                        torch.exp(-logits.abs()) / (1 + torch.exp(-logits.abs())))
    c = s.clone()
    if st["select_bias"] is not None:
        c += st["select_bias"].double()
    rows = torch.arange(case["T"], device=DEV)
    if G > 1:
        size = E // G
        value = torch.empty(case["T"], G, dtype=torch.float64, device=DEV)
        for g in range(G):
            part = c[:, g * size:(g + 1) * size].clone()
            first = _first_max(part)
            value[:, g] = part[rows, first]
            if case["group_by"] == "top2":
                part[rows, first] = -math.inf
                value[:, g] += part.amax(1)
        keep = torch.zeros(case["T"], G, dtype=torch.bool, device=DEV)
        for _ in range(case["group_topk"]):
            # a group of value -inf may stay too: below it are only those already kept
            g = _first_max(torch.where(keep, -math.inf, value.clamp(min=-1e300)))
            keep[rows, g] = True
        c = torch.where(keep.repeat_interleave(size, dim=1), c, -math.inf)
    ids = torch.full((case["T"], K), -1, dtype=torch.int32, device=DEV)
    wt = torch.zeros(case["T"], K, dtype=torch.float64, device=DEV)
    for k in range(K):
        e = _first_max(c)
        ok = c[rows, e] > -math.inf
        ids[:, k] = torch.where(ok, e, -1).to(torch.int32)
        wt[:, k] = torch.where(ok, s[rows, e], 0.0)
        c[rows, e] = -math.inf
    if case["renorm"]:
        total = wt.sum(1, keepdim=True)
        wt = wt / torch.where(total > 0, total, 1.0)
    return ids, wt * case["scale"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "route":
        return _exact_route(case, st)
    names = ("w0", "w1") if case["swiglu"] else ("w0",)
    N, d = case["f"], case["d"]
    out = torch.empty(case["T"] * case["K"], N, dtype=torch.float64, device=DEV)
    slab = max(16, (1 << 26) // d)
    ends = torch.tensor(st["counts"]).cumsum(0).tolist()
    for e, r1 in enumerate(ends):
        r0 = r1 - st["counts"][e]
        if r0 == r1:
            continue
        src = torch.arange(r0, r1, device=DEV)
        if case["gather"]:
            src = torch.div(st["slots"][r0:r1].long(), case["K"], rounding_mode="floor")
        a = st["a_q"][src].double() * st["a_s"][src].double().unsqueeze(1)
        for c0 in range(0, N, slab):
            p = [torch.mm(a, (st[n + "_q"][e, c0:c0 + slab].double() * st[n + "_s"][e, c0:c0 + slab].double()[:, None]).t())
                 for n in names]
            out[r0:r1, c0:c0 + slab] = p[0] * torch.sigmoid(p[0]) * p[1] if len(p) == 2 else p[0]
    return out
