"""What stands between the products of an FP8 mixture-of-experts block, as cases to be timed and compared.

Four operators, those that are trained through with their gradients:

* ``norm``      root-mean-square norm of x plus the residual, written as the E4M3 operand of the next product (1x128 scales)
* ``route``     a router's logits to experts and weights: softmax or sigmoid scores, a bias, groups, top-k, renormalised
* ``gate``      silu(gate) * up between an expert's two products, as the second one's E4M3 operand (1x128, or 128x1 for its
  weight's gradient)
* ``dispatch``  quantized token rows, with their scales, in the experts' order

``run`` computes them in plain torch operations in 32 bits, choices of experts in 64 (``own`` false), or by the library's entry
points (``own`` true).  ``exact`` computes them in 64 bits from their definitions.
"""

import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of a single sequence: the norm in front of a projection of the headline weight, latency
        {"name": "norm one token", "op": "norm", "part": "fwd", "rows": 1, "K": 8192, "dtype": "bf16", "residual": True, "y": False, "stats": False},
        # a prompt in front of an expert layer: the FP8 operand, and the row itself for the router
        {"name": "norm prompt", "op": "norm", "part": "fwd", "rows": 8192, "K": 7184, "dtype": "bf16", "residual": True, "y": True, "stats": False},
        # training in fp32 at a width that no vector load divides, an odd number of tokens
        {"name": "norm odd", "op": "norm", "part": "fwd", "rows": 4095, "K": 7183, "dtype": "fp32", "residual": False, "y": False, "stats": True},
        # training: gradients of the norm's input and weight, the residual's own gradient added
        {"name": "norm gradient", "op": "norm", "part": "grad", "rows": 8191, "K": 7184, "dtype": "bf16", "residual": True},
        # the router of one decoding batch: latency
        {"name": "route batch", "op": "route", "part": "fwd", "T": 48, "E": 32, "topk": 2, "dtype": "fp32", "score": "softmax", "bias": False, "groups": 1,
         "topk_groups": 1, "group_top": 1, "renormalize": True, "scale": 1.0, "masked": 0},
        # a training batch over many experts: sigmoid scores, a balancing bias, the best half of eight groups
        {"name": "route training", "op": "route", "part": "fwd", "T": 65536, "E": 256, "topk": 8, "dtype": "fp32", "score": "sigmoid", "bias": True, "groups": 8,
         "topk_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5, "masked": 0},
        # training: the gradient of softmax weights that are not renormalised reaches every logit
        {"name": "route gradient", "op": "route", "part": "grad", "T": 65536, "E": 256, "topk": 8, "dtype": "fp32", "score": "softmax", "renormalize": False, "scale": 1.0},
        # a decoding batch between the two products of its experts: 48 tokens, two experts each
        {"name": "gate batch", "op": "gate", "part": "rows", "rows": 96, "H": 4096, "dtype": "bf16"},
        # training: the operand of the second weight's gradient, an odd number of rows
        {"name": "gate columns", "op": "gate", "part": "columns", "rows": 16379, "H": 4096, "dtype": "bf16"},
        # training: the gradient of both halves
        {"name": "gate gradient", "op": "gate", "part": "grad", "rows": 8191, "H": 7184, "dtype": "bf16"},
        # a decoding batch over the expert stack
        {"name": "dispatch batch", "op": "dispatch", "T": 48, "topk": 2, "E": 32, "K": 7184, "align": 1},
        # a prompt over the expert stack, parts of 128 rows
        {"name": "dispatch prompt", "op": "dispatch", "T": 8191, "topk": 4, "E": 32, "K": 7184, "align": 128},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """A size in lo..hi: any number one time in four, else a multiple of 16."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["norm", "norm", "route", "route", "gate", "gate", "dispatch"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "norm":
        K = _odd(rng, 96, 8192)
        rows = min(_log(rng, 1, 16384), (1 << 25) // K)
        case = {"op": op, "part": rng.choice(["fwd", "fwd", "grad"]), "rows": rows, "K": K, "dtype": dtype, "residual": rng.random() < 0.7}
        return case if case["part"] == "grad" else case | {"y": rng.random() < 0.5, "stats": rng.random() < 0.5}
    if op == "route":
        E = rng.choice([8, 16, 32, 60, 64, 72, 128, 160, 256, 384, 512])
        case = {"op": op, "part": rng.choice(["fwd", "fwd", "grad"]), "T": min(_log(rng, 1, 65536), (1 << 24) // E), "E": E, "topk": rng.choice([1, 2, 4, 6, 8]),
                "dtype": dtype, "score": rng.choice(["softmax", "sigmoid"]), "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5])}
        if case["part"] == "grad":
            return case
        groups = rng.choice([1, 1, 4, 8]) if E % 8 == 0 and E >= 32 else 1
        return case | {"bias": rng.random() < 0.5, "groups": groups, "topk_groups": max(1, groups // 2), "group_top": rng.choice([1, 2]),
                       "masked": rng.choice([0, 0, 2])}
    if op == "gate":
        H = _odd(rng, 96, 8192)
        return {"op": op, "part": rng.choice(["plain", "rows", "rows", "columns", "grad"]), "rows": min(_log(rng, 1, 16384), (1 << 24) // H), "H": H, "dtype": dtype}
    return {"op": op, "T": _log(rng, 1, 8192), "topk": rng.choice([1, 2, 4]), "E": rng.choice([8, 32, 64]), "K": _odd(rng, 128, 7184), "align": rng.choice([1, 128])}


def _cdiv(a, b):
    return -(-a // b)


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def _capacity(case):
    """Rows that the experts' order has room for: each expert's part is rounded up to `align` rows."""
    n = case["T"] * case["topk"]
    return n + min(case["E"], n) * (case["align"] - 1)


def work(case):
    op = case["op"]
    if op == "norm":
        n, es, K, rows = case["rows"] * case["K"], _size(case), case["K"], case["rows"]
        if case["part"] == "grad":
            return {"bytes": n * es * (3 + case["residual"]) + K * (es + 4) + 4 * rows, "flops": 10 * n}
        return {"bytes": n * es * (1 + 2 * case["residual"] + case["y"]) + n + rows * _cdiv(K, 128) + K * es + 4 * rows * case["stats"], "flops": 6 * n}
    if op == "route":
        T, E, a = case["T"], case["E"], case["T"] * case["topk"]
        if case["part"] == "fwd":
            return {"bytes": T * E * _size(case) + 8 * a + 4 * E * case["bias"], "flops": 8 * T * E}
        # the other forms need the chosen experts' logits alone
        read = T * E if case["score"] == "softmax" and not case["renormalize"] else a
        return {"bytes": (read + T * E) * _size(case) + 8 * a, "flops": 6 * read + 6 * a}
    if op == "gate":
        n, es = case["rows"] * case["H"], _size(case)
        if case["part"] == "grad":
            return {"bytes": 5 * n * es, "flops": 16 * n}
        out = {"plain": n * es, "rows": n + case["rows"] * _cdiv(case["H"], 128), "columns": n + _cdiv(case["rows"], 128) * case["H"]}[case["part"]]
        return {"bytes": 2 * n * es + out, "flops": 8 * n}
    row = case["K"] + _cdiv(case["K"], 128)
    # the rows of no choice are written too: they come out as zero
    return {"bytes": (case["T"] + _capacity(case)) * row + 4 * _capacity(case), "flops": 0}


# ------------------------------------------------------------------ inputs


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(g, rows, K, dtype):
    """Rows of N(0, 1) at scales of their own, a few columns much larger, as hidden states have them."""
    x = torch.randn(rows, K, device="cuda", generator=g)
    x *= torch.exp2(torch.randn(rows, 1, device="cuda", generator=g))
    x[:, torch.randint(0, K, (max(1, K // 512),), device="cuda", generator=g)] *= 30.0
    return x.to(dtype)


def _logits(g, T, E, dtype):
    """Some experts are liked by most tokens, and tokens differ in how sure they are."""
    liking = 0.5 * torch.randn(E, device="cuda", generator=g)
    sure = torch.exp2(0.5 * torch.randn(T, 1, device="cuda", generator=g))
    return (torch.randn(T, E, device="cuda", generator=g) * sure + liking).to(dtype)


def _distinct(g, T, topk, E):
    """Experts [T, topk], distinct within a token, some far more popular than others."""
    liking = 1.5 * torch.randn(E, device="cuda", generator=g)
    noise = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)
    return (liking - torch.log(-torch.log(noise))).topk(topk, dim=1).indices


def _source(ids, E, align):
    """The choice (token * topk + place) at each row of the experts' order, -1 where there is none; each expert's part is rounded up
    to `align` rows."""
    flat = ids.reshape(-1)
    n = flat.numel()
    count = torch.bincount(flat, minlength=E)
    room = (count + align - 1) // align * align
    begin, first = room.cumsum(0) - room, count.cumsum(0) - count
    by = torch.sort(flat, stable=True).indices
    source = torch.full((n + min(E, n) * (align - 1),), -1, dtype=torch.int32, device=ids.device)
    source[begin[flat[by]] + torch.arange(n, device=ids.device) - first[flat[by]]] = by.int()
    return source


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "norm":
        rows, K, dt = case["rows"], case["K"], _dtype(case["dtype"])
        s["weight"] = (1 + 0.2 * torch.randn(K, device="cuda", generator=g)).to(dt)
        if case["part"] == "fwd":
            s["x"] = _activations(g, rows, K, dt)
            s["residual"] = _activations(g, rows, K, dt) if case["residual"] else None
            return s
        s["h"] = _activations(g, rows, K, dt)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["g"] = (1e-3 * torch.randn(rows, K, device="cuda", generator=g)).to(dt)
        s["g_h"] = (1e-3 * torch.randn(rows, K, device="cuda", generator=g)).to(dt) if case["residual"] else None
        return s
    if op == "route":
        s["logits"] = _logits(g, case["T"], case["E"], _dtype(case["dtype"]))
        if case["part"] == "fwd":
            s["bias"] = 0.05 * torch.randn(case["E"], device="cuda", generator=g) if case["bias"] else None
            if case["masked"]:  # experts that are out of service
                s["logits"][:, torch.randperm(case["E"], device="cuda", generator=g)[: case["masked"]]] = -math.inf
            return s
        s["ids"] = (s["logits"].float() + 0.1 * torch.randn(case["T"], case["E"], device="cuda", generator=g)).topk(case["topk"], dim=1).indices.int()
        s["g"] = torch.randn(case["T"], case["topk"], device="cuda", generator=g)
        return s
    if op == "gate":
        s["x"] = _activations(g, case["rows"], 2 * case["H"], _dtype(case["dtype"]))
        if case["part"] == "grad":
            s["g"] = (1e-3 * torch.randn(case["rows"], case["H"], device="cuda", generator=g)).to(s["x"].dtype)
        return s
    s["source"] = _source(_distinct(g, case["T"], case["topk"], case["E"]), case["E"], case["align"])
    s["data"], s["scales"] = _quant_rows(_activations(g, case["T"], case["K"], torch.float32))
    return s


# ------------------------------------------------------------- plain forms


def _power(e):
    """2^e in fp32 for whole numbers e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _quant_rows(x):
    """fp32 [n, K] -> (E4M3 bytes, UE8M0 codes [n, ceil(K/128)]): per 128 elements of a row the least power of two 2^s with amax <=
    448 * 2^s, s in [-127, 127]; a block that holds a NaN or an infinity has code 255 and NaN payloads."""
    n, K = x.shape
    nb = _cdiv(K, 128)
    v = torch.nn.functional.pad(x, (0, nb * 128 - K)).reshape(n, nb, 128)
    amax = v.abs().amax(2)
    bad = ~(amax < math.inf)
    m, e = torch.frexp(torch.where(bad, torch.ones_like(amax), amax))  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    s = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-127, 127)
    s = torch.where(amax > 0, s, torch.full_like(s, -127))
    data = (v * _power(-s)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    data = torch.where(bad[..., None], torch.full_like(data, 0x7F), data)
    return data.reshape(n, nb * 128)[:, :K].contiguous(), torch.where(bad, torch.full_like(s, 255), s + 127).to(torch.uint8)


def _norm(s):
    case, w = s["case"], s["weight"].float()
    if case["part"] == "grad":
        n = s["h"].float() * s["rstd"][:, None]
        g = s["g"].float()
        d = g * w
        d_h = (d - n * (d * n).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["g_h"] is not None:
            d_h = d_h + s["g_h"].float()
        return {"h": d_h.to(s["h"].dtype), "weight": (g * n).sum(0)}
    h = s["x"] if s["residual"] is None else (s["x"].float() + s["residual"].float()).to(s["x"].dtype)
    hf = h.float()
    rstd = torch.rsqrt(hf.square().mean(1) + EPS)
    y = hf * rstd[:, None] * w
    data, scales = _quant_rows(y)
    out = {"data": data, "scales": scales}
    if s["residual"] is not None:
        out["h"] = h
    if case["y"]:
        out["y"] = y.to(h.dtype)
    if case["stats"]:
        out["rstd"] = rstd
    return out


def _descending(v):
    """The places of v's values along the last axis, largest first, equal ones by their place."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices


def _route(s):
    case, topk = s["case"], s["case"]["topk"]
    if case["part"] == "grad":
        x, ids, g = s["logits"].float(), s["ids"].long(), s["g"]
        if case["score"] == "softmax":
            e = torch.exp(x - x.amax(1, keepdim=True))
            p = e / e.sum(1, keepdim=True)
        else:
            p = 1 / (1 + torch.exp(-x))
        chosen = p.gather(1, ids)
        d = g * case["scale"]
        if case["renormalize"]:
            total = chosen.sum(1, keepdim=True)
            d = (d - (d * chosen).sum(1, keepdim=True) / total) / total
        d = torch.zeros_like(p).scatter_add_(1, ids, d)
        d = p * (d - (p * d).sum(1, keepdim=True)) if case["score"] == "softmax" else d * p * (1 - p)
        return d.to(s["logits"].dtype)
    # which expert is ahead is decided in 64 bits
    x = s["logits"].double()
    T, E = x.shape
    if case["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    c = p if s["bias"] is None else p + s["bias"].double()
    c = torch.where(x > -math.inf, c, torch.full_like(c, -math.inf))
    if case["groups"] > 1:
        by_group = c.view(T, case["groups"], -1)
        top = by_group.sort(dim=2, descending=True).values[..., : case["group_top"]]
        total = torch.where((top > -math.inf).any(2), torch.where(top > -math.inf, top, torch.zeros_like(top)).sum(2), torch.full_like(top[..., 0], -math.inf))
        kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, _descending(total)[:, : case["topk_groups"]], True)
        c = torch.where(kept[..., None], by_group, torch.full_like(by_group, -math.inf)).view(T, E)
    ids = _descending(c)[:, :topk]
    there = c.gather(1, ids) > -math.inf
    w = torch.where(there, p.gather(1, ids), torch.zeros_like(p[:, :1])).float()
    if case["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(there, w / total, torch.zeros_like(w))
    return {"ids": torch.where(there, ids, torch.full_like(ids, -1)).int(), "weights": w * case["scale"]}


def _gate(s):
    case, x = s["case"], s["x"].float()
    gate, up = x[:, : case["H"]], x[:, case["H"] :]
    sig = 1 / (1 + torch.exp(-gate))
    if case["part"] == "grad":
        g = s["g"].float()
        return torch.cat([g * up * sig * (1 + gate * (1 - sig)), g * gate * sig], 1).to(s["x"].dtype)
    a = gate * sig * up
    if case["part"] == "plain":
        return a.to(s["x"].dtype)
    if case["part"] == "rows":
        data, scales = _quant_rows(a)
        return {"data": data, "scales": scales}
    data, scales = _quant_rows(a.t())
    return {"data": data.t().contiguous(), "scales": scales.t().contiguous()}


def _dispatch(s):
    there = (s["source"] >= 0)[:, None]
    token = torch.div(s["source"].clamp(min=0), s["case"]["topk"], rounding_mode="floor").long()
    return {"data": torch.where(there, s["data"][token], torch.zeros_like(s["data"][:1])), "scales": torch.where(there, s["scales"][token], torch.zeros_like(s["scales"][:1]))}


# --------------------------------------------------------- the library's


def _norm_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    case = s["case"]
    if case["part"] == "grad":
        d_h, d_weight = mxq.mxq_rmsnorm_grad(s["g"], s["h"], s["weight"], s["rstd"], g_h=s["g_h"])
        return {"h": d_h, "weight": d_weight}
    r = mxq.mxq_rmsnorm(s["x"], s["weight"], residual=s["residual"], eps=EPS, normed=case["y"], stats=case["stats"])
    out = {"data": r.data, "scales": r.scales}
    if s["residual"] is not None:
        out["h"] = r.h
    if case["y"]:
        out["y"] = r.y
    if case["stats"]:
        out["rstd"] = r.rstd
    return out


def _route_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    case = s["case"]
    if case["part"] == "grad":
        return mxq.mxq_moe_route_grad(s["g"], s["logits"], s["ids"], score=case["score"], renormalize=case["renormalize"], scale=case["scale"])
    ids, weights = mxq.mxq_moe_route(s["logits"], case["topk"], bias=s["bias"], score=case["score"], groups=case["groups"], topk_groups=case["topk_groups"],
                                     group_top=case["group_top"], renormalize=case["renormalize"], scale=case["scale"])
    return {"ids": ids, "weights": weights}


def _gate_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    part = s["case"]["part"]
    if part == "grad":
        return mxq.mxq_silu_mul_grad(s["g"], s["x"])
    if part == "plain":
        return mxq.mxq_silu_mul(s["x"])
    data, scales = (mxq.mxq_fp8_silu_mul_1x128 if part == "rows" else mxq.mxq_fp8_silu_mul_128x1)(s["x"])
    return {"data": data, "scales": scales}


def _dispatch_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    data, scales = mxq.mxq_fp8_dispatch(s["data"], s["scales"], s["source"], s["case"]["topk"])
    return {"data": data, "scales": scales}


def run(state):
    op = state["case"]["op"]
    if own:
        out = {"norm": _norm_own, "route": _route_own, "gate": _gate_own, "dispatch": _dispatch_own}[op](state)
    else:
        out = {"norm": _norm, "route": _route, "gate": _gate, "dispatch": _dispatch}[op](state)
    if isinstance(out, dict) and "data" in out:  # bytes as the values that they stand for
        out["data"], out["scales"] = out["data"].view(torch.float8_e4m3fn), out["scales"].view(torch.float8_e8m0fnu)
    return out


# ------------------------------------------------------------ in 64 bits


def _two_to(e):
    """2^e in 64 bits for whole numbers e in [-400, 400]."""
    return torch.tensor([math.ldexp(1.0, k) for k in range(-400, 401)], dtype=torch.float64, device="cuda")[e.long() + 400]


def _quant64(x):
    """The payloads, before they are rounded to E4M3, and the scales of each 128 elements of a row, in 64 bits."""
    n, K = x.shape
    nb = _cdiv(K, 128)
    b = torch.nn.functional.pad(x, (0, nb * 128 - K)).reshape(n, nb, 128)
    amax = b.abs().amax(2, keepdim=True)
    s = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127)
    s = torch.where(amax <= 448 * _two_to(s - 1), s - 1, s)  # a logarithm that was rounded across a whole number
    s = torch.where(amax > 448 * _two_to(s), s + 1, s).clamp(-127, 127)
    return (b / _two_to(s)).reshape(n, -1)[:, :K], _two_to(s)[..., 0]


def _sigmoid64(x):
    return torch.where(x >= 0, 1 / (1 + torch.exp(-x.abs())), torch.exp(-x.abs()) / (1 + torch.exp(-x.abs())))


def _places(c):
    """The place of each value of a row in descending order, equal ones by their index: how many are ahead of it."""
    earlier = torch.ones(c.shape[1], c.shape[1], dtype=torch.bool, device=c.device).tril(-1)  # [value, other]: other comes first
    return torch.cat([((p[:, None] > p[..., None]) | (p[:, None] == p[..., None]) & earlier).sum(2) for p in c.split(512)])


def exact(case, seed):
    op = case["op"]
    if op == "dispatch":
        return None
    s = prepare(case, seed)
    if op == "norm":
        w, K = s["weight"].double(), case["K"]
        if case["part"] == "grad":
            # the derivative of sum(g y) at h, with the row's statistic as the call is given it
            h, r, v = s["h"].double(), s["rstd"].double()[:, None], s["g"].double() * w
            d = r * v - h * r**3 * ((v * h).sum(1, keepdim=True) / K)
            return {"h": d if s["g_h"] is None else d + s["g_h"].double(), "weight": (s["g"].double() * h * r).sum(0)}
        h = s["x"].double()
        out = {}
        if s["residual"] is not None:
            h = (h + s["residual"].double()).to(s["x"].dtype).double()  # the sum that the model carries on is rounded to its type
            out["h"] = h
        ms = (h * h).sum(1, keepdim=True) / K + EPS
        y = h / torch.sqrt(ms) * w
        out["data"], out["scales"] = _quant64(y)
        if case["y"]:
            out["y"] = y
        if case["stats"]:
            out["rstd"] = 1 / torch.sqrt(ms[:, 0])
        return out
    if op == "route":
        x = s["logits"].double()
        if case["part"] == "grad":
            ids, g = s["ids"].long(), s["g"].double() * case["scale"]
            p = torch.softmax(x, 1) if case["score"] == "softmax" else _sigmoid64(x)
            chosen = p.gather(1, ids)
            # d w_j / d x_e by the quotient's rule on logarithms: d log s_j / d x_e is [j = e] - s_e (softmax) or [j = e](1 - s_e)
            w = chosen / chosen.sum(1, keepdim=True) if case["renormalize"] else chosen
            t = g * w
            if case["renormalize"]:
                t = t - w * t.sum(1, keepdim=True)
            if case["score"] == "sigmoid":
                return torch.zeros_like(x).scatter_(1, ids, t * _sigmoid64(-x).gather(1, ids))
            d = torch.zeros_like(x).scatter_(1, ids, t)
            return d if case["renormalize"] else d - p * t.sum(1, keepdim=True)
        p = torch.softmax(x, 1) if case["score"] == "softmax" else _sigmoid64(x)
        c = p if s["bias"] is None else p + s["bias"].double()
        c = c.masked_fill(x == -math.inf, -math.inf)
        if case["groups"] > 1:
            best = c.view(case["T"], case["groups"], -1).topk(case["group_top"], dim=2).values
            total = best.clamp(min=0).sum(2) if s["bias"] is None else torch.nan_to_num(best, neginf=0.0).sum(2)
            kept = _places(total.masked_fill((best == -math.inf).all(2), -math.inf)) < case["topk_groups"]
            c = c.masked_fill(~kept.repeat_interleave(case["E"] // case["groups"], 1), -math.inf)
        place = _places(c)
        chosen = (place < case["topk"]) & (c > -math.inf)
        w = p * chosen
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        # each expert's weight to its place; the others go to one place more, which is cut off
        out = torch.zeros(case["T"], case["topk"] + 1, dtype=torch.float64, device="cuda")
        out.scatter_(1, place.clamp(max=case["topk"]), w * case["scale"])
        return {"ids": None, "weights": out[:, :-1]}
    gate, up = s["x"][:, : case["H"]].double(), s["x"][:, case["H"] :].double()
    sig = _sigmoid64(gate)
    if case["part"] == "grad":
        g = s["g"].double()
        return torch.cat([g * up * (sig + gate * sig * _sigmoid64(-gate)), g * gate * sig], 1)
    a = gate * sig * up
    if case["part"] == "plain":
        return a
    if case["part"] == "rows":
        data, scales = _quant64(a)
        return {"data": data, "scales": scales}
    data, scales = _quant64(a.t())
    return {"data": data.t(), "scales": scales.t()}
