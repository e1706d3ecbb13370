"""The FP8 linear layer and the mixture-of-experts operators, as cases to be timed and compared.

Five operators stand on the 128x128 blockwise weights that this library converts:

* ``quant``    activations to E4M3 with one power-of-two scale per 128 elements, along rows (1x128) or columns (128x1)
* ``matmul``   the matrix product of such operands, forward and for both gradients
* ``grouped``  the same product for rows sorted by expert, each expert with its own weight
* ``sort``     tokens' choices of experts, brought into the experts' order
* ``moe``      rows taken to the experts' order and back with the router's weights, and the gradients of both

``run`` computes them in plain torch operations in 32 bits (``own`` false) or by the library's entry points (``own``
true).  ``exact`` computes them in 64 bits from their definitions.
"""

import math

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases


def listed():
    return [
        # activations of a prompt on their way into a projection of the expert stack's width (7184 = 56 blocks and 16)
        {"name": "quant rows prompt", "op": "quant", "axis": "rows", "rows": 8192, "K": 7184, "dtype": "bf16"},
        # fp32 gradients of an odd number of tokens, quantised along the tokens for the weight gradient
        {"name": "quant columns odd", "op": "quant", "axis": "columns", "rows": 4099, "K": 4096, "dtype": "fp32"},
        # one decoding step of a single sequence: latency and the weight's bytes
        {"name": "matmul one token", "op": "matmul", "dir": "fwd", "M": 1, "N": 8192, "K": 8192, "out": "bf16"},
        # a decoding batch through a wide projection
        {"name": "matmul batch", "op": "matmul", "dir": "fwd", "M": 96, "N": 7184, "K": 4096, "out": "bf16"},
        # a prompt through the headline weight
        {"name": "matmul prompt", "op": "matmul", "dir": "fwd", "M": 8192, "N": 8192, "K": 8192, "out": "bf16"},
        # training: the gradient of the input, an odd number of tokens
        {"name": "matmul input gradient", "op": "matmul", "dir": "dgrad", "M": 4099, "N": 4096, "K": 7184, "out": "bf16"},
        # training: the gradient of the weight, kept in fp32
        {"name": "matmul weight gradient", "op": "matmul", "dir": "wgrad", "M": 4099, "N": 4096, "K": 4096, "out": "fp32"},
        # a decoding batch over the expert stack: most experts see a few tokens, some none
        {"name": "grouped batch", "op": "grouped", "dir": "fwd", "T": 48, "topk": 2, "E": 32, "N": 4096, "K": 7184, "out": "bf16"},
        # a prompt over the expert stack, the loads of the experts uneven
        {"name": "grouped prompt", "op": "grouped", "dir": "fwd", "T": 4096, "topk": 4, "E": 32, "N": 4096, "K": 7184, "out": "bf16"},
        # the router's choices of one decoding batch: latency
        {"name": "sort batch", "op": "sort", "T": 48, "topk": 2, "E": 32, "align": 1},
        # the router's choices of a training batch, over many experts, in blocks of 128 rows
        {"name": "sort training", "op": "sort", "T": 65536, "topk": 8, "E": 256, "align": 128},
        # the gradient of the way back: the experts' rows and the router's weights
        {"name": "moe combine gradient", "op": "moe", "part": "combine_grad", "T": 8191, "topk": 4, "E": 32, "H": 7184, "align": 1, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _odd(rng, lo, hi):
    """A size in lo..hi: any number one time in four, else a multiple of 16."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(16, n // 16 * 16)


def draw(rng):
    op = rng.choice(["quant", "matmul", "matmul", "grouped", "sort", "moe"])
    if op == "quant":
        rows = _log(rng, 1, 16384)
        K = min(_odd(rng, 96, 8192), (1 << 26) // rows)
        return {"op": op, "axis": rng.choice(["rows", "columns"]), "rows": rows, "K": max(K, 16), "dtype": rng.choice(["bf16", "fp32"])}
    if op == "matmul":
        return {"op": op, "dir": rng.choice(["fwd", "dgrad", "wgrad"]), "M": _log(rng, 1, 8192), "N": _odd(rng, 128, 8192), "K": _odd(rng, 128, 8192),
                "out": rng.choice(["bf16", "fp32"])}
    E, topk = rng.choice([8, 16, 32, 64, 128, 256]), rng.choice([1, 2, 4, 6, 8])
    align = rng.choice([1, 128])
    if op == "sort":
        return {"op": op, "T": _log(rng, 1, 65536), "topk": topk, "E": E, "align": align}
    if op == "moe":
        return {"op": op, "part": rng.choice(["dispatch", "dispatch_grad", "combine", "combine_grad"]), "T": _log(rng, 1, 8192), "topk": min(topk, 4), "E": min(E, 64),
                "H": _odd(rng, 256, 7184), "align": align, "dtype": rng.choice(["bf16", "fp32"])}
    E, topk = min(E, 64), min(topk, 4)
    N = _odd(rng, 128, 4096)
    K = min(_odd(rng, 128, 7184), (1 << 30) // (E * N) // 16 * 16)
    return {"op": op, "dir": rng.choice(["fwd", "dgrad", "wgrad"]), "T": _log(rng, 1, 4096), "topk": topk, "E": E, "N": N, "K": K, "out": rng.choice(["bf16", "fp32"])}


def _cdiv(a, b):
    return -(-a // b)


def _capacity(case, align):
    """Rows that the experts' order has room for: each expert's part is rounded up to `align` rows."""
    return case["T"] * case["topk"] + (min(case["E"], case["T"] * case["topk"]) * (align - 1))


def _group_align(case):
    return 128 if case["dir"] == "wgrad" else 1


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["K"]
        blocks = case["rows"] * _cdiv(case["K"], 128) if case["axis"] == "rows" else _cdiv(case["rows"], 128) * case["K"]
        return {"bytes": n * (3 if case["dtype"] == "bf16" else 5) + blocks, "flops": 2 * n}
    if op == "sort":
        a = case["T"] * case["topk"]
        return {"bytes": 4 * (2 * a + _capacity(case, case["align"]) + case["E"] + 1), "flops": a}
    if op == "moe":
        a, es = case["T"] * case["topk"], 2 if case["dtype"] == "bf16" else 4
        token, rows, cap = case["T"] * case["H"] * es, a * case["H"] * es, _capacity(case, case["align"]) * case["H"] * es
        bytes_ = {"dispatch": token + cap, "dispatch_grad": rows + token, "combine": rows + token + 4 * a, "combine_grad": token + rows + cap + 8 * a}[case["part"]]
        return {"bytes": bytes_ + 4 * a, "flops": 2 * a * case["H"]}
    es = 2 if case["out"] == "bf16" else 4
    N, K = case["N"], case["K"]
    M = case["M"] if op == "matmul" else case["T"] * case["topk"]
    # of the stacked weights only those that tokens choose have to be read, or their gradients computed: the choices are skewed, so
    # this counts the experts that a uniform choice would touch on average
    E = 1 if op == "matmul" else case["E"]
    touched = 1 if op == "matmul" else E * (1 - (1 - 1 / E) ** M)
    w = N * K * touched
    if case["dir"] == "fwd":
        b = M * K + w + M * N * es
    elif case["dir"] == "dgrad":
        b = M * N + w + M * K * es
    else:
        b = M * N + M * K + N * K * E * es
    return {"bytes": b, "flops": 2 * M * N * K}


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


def _weight(g, E, N, K):
    """(E4M3 payload bytes [E, N, K], fp32 tile scales [E, N/128, K/128]) of N(0, 1) weights on the E2M1 grid: 1x32 blocks a few
    binary orders apart below their 128x128 tile's largest, as the blockwise conversion leaves them."""
    grid = torch.tensor(_E2M1, device="cuda")
    mid = (grid[1:] + grid[:-1]) / 2
    table = torch.stack([grid * 2.0 ** (6 - s) for s in range(4)])
    table = torch.cat([table, -table], 1).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)  # [4 spreads x 16 signed codes]
    nb = _cdiv(K, 32)
    data = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, device="cuda", generator=g)
        code = torch.bucketize((w * 2.5).abs_(), mid, out_int32=True) + 8 * (w < 0)
        spread = torch.randint(0, 4, (N, nb), device="cuda", generator=g, dtype=torch.int32).repeat_interleave(32, 1)[:, :K]
        data[e] = table[(code + 16 * spread).reshape(-1)].view(N, K)
    tile = torch.exp2(torch.randint(-14, -10, (E, _cdiv(N, 128), _cdiv(K, 128)), device="cuda", generator=g).float())
    return data, tile


def _choices(g, T, topk, E):
    """Experts [T, topk] of each token, distinct within a token, some experts far more popular than others and some tokens
    dropped by a full expert (-1)."""
    liking = 1.5 * torch.randn(E, device="cuda", generator=g)
    noise = torch.rand(T, E, device="cuda", generator=g).clamp_(1e-9, 1 - 1e-7)
    ids = (liking - torch.log(-torch.log(noise))).topk(min(topk, E), dim=1).indices.to(torch.int32)
    if topk > E:
        ids = torch.cat([ids, ids[:, : topk - E]], 1)
    ids[torch.rand(T, topk, device="cuda", generator=g) < 0.01] = -1
    return ids


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op == "quant":
        return {"case": case, "x": _activations(g, case["rows"], case["K"], _dtype(case["dtype"]))}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        s = {"case": case}
        if case["dir"] == "wgrad":
            s["g"], s["g_scales"] = _quant_columns(_activations(g, M, N, torch.float32))
            s["x"], s["x_scales"] = _quant_columns(_activations(g, M, K, torch.float32))
            return s
        s["x"], s["x_scales"] = _quant_rows(_activations(g, M, K if case["dir"] == "fwd" else N, torch.float32))
        w, tile = _weight(g, 1, N, K)
        return s | {"w": w[0], "tile": tile[0]}
    ids = _choices(g, case["T"], case["topk"], case["E"])
    if op == "sort":
        return {"case": case, "ids": ids}
    align = case["align"] if op == "moe" else _group_align(case)
    order = _sort(ids, case["E"], align)
    s = {"case": case, "order": order}
    cap = order["source"].numel()
    if op == "moe":
        dt, H, part = _dtype(case["dtype"]), case["H"], case["part"]
        if part in ("dispatch", "combine_grad"):
            s["tokens"] = _activations(g, case["T"], H, dt)
        if part != "dispatch":
            s["rows"] = _activations(g, cap, H, dt)
        if part.startswith("combine"):
            s["weights"] = torch.softmax(torch.randn(case["T"], case["topk"], device="cuda", generator=g), 1)
        return s
    N, K = case["N"], case["K"]
    s["most"] = max(1, int(order["offsets"].diff().max()))  # the longest part, which the plain form pads the others to
    fill = (order["source"] >= 0)[:, None]
    if case["dir"] == "wgrad":
        s["g"], s["g_scales"] = _quant_columns(_activations(g, cap, N, torch.float32) * fill)
        s["x"], s["x_scales"] = _quant_columns(_activations(g, cap, K, torch.float32) * fill)
        return s
    s["x"], s["x_scales"] = _quant_rows(_activations(g, cap, K if case["dir"] == "fwd" else N, torch.float32) * fill)
    s["w"], s["tile"] = _weight(g, case["E"], N, K)
    return s


# ------------------------------------------------------------- plain forms


def _power(e):
    """2^e in fp32 for whole numbers e in [-127, 127], from its bits."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _blocks_to_fp8(v):
    """[n, b] fp32 blocks -> (E4M3 bytes, UE8M0 codes): the scale is the least power of two 2^s with amax <= 448 * 2^s, s in
    [-127, 127]; a block that holds a NaN or an infinity has code 255 and NaN payloads."""
    amax = v.abs().amax(1)
    bad = ~(amax < math.inf)
    m, e = torch.frexp(torch.where(bad, torch.ones_like(amax), amax))  # amax = m 2^e, m in [1/2, 1); 448 = 0.875 * 2^9
    s = (e - 9 + (m > 0.875).to(e.dtype)).clamp(-127, 127)
    s = torch.where(amax > 0, s, torch.full_like(s, -127))
    scaled = v * _power(-s)[:, None]
    data = torch.where(bad[:, None], torch.full_like(v, math.nan), scaled).to(torch.float8_e4m3fn).view(torch.uint8)
    data = torch.where(bad[:, None], torch.full_like(data, 0x7F), data)
    return data, torch.where(bad, torch.full_like(s, 255), s + 127).to(torch.uint8)


def _quant_rows(x):
    rows, K = x.shape
    nb = _cdiv(K, 128)
    v = torch.nn.functional.pad(x.float(), (0, nb * 128 - K)).view(rows * nb, 128)
    data, codes = _blocks_to_fp8(v)
    return data.view(rows, nb * 128)[:, :K].contiguous(), codes.view(rows, nb)


def _quant_columns(x):
    data, codes = _quant_rows(x.t())
    return data.t().contiguous(), codes.t().contiguous()


def _decode_rows(data, scales):
    """fp32 [rows, K] of E4M3 bytes with scales [rows, ceil(K/128)]."""
    s = _power(scales.to(torch.int32).clamp(max=254) - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return data.view(torch.float8_e4m3fn).float() * s.repeat_interleave(128, -1)[..., : data.shape[-1]]


def _decode_columns(data, scales):
    return _decode_rows(data.t().contiguous(), scales.t()).t()


def _decode_weight(w, tile):
    s = tile.repeat_interleave(128, -2)[..., : w.shape[-2], :].repeat_interleave(128, -1)[..., : w.shape[-1]]
    return w.view(torch.float8_e4m3fn).float() * s


def _matmul(s):
    case = s["case"]
    if case["dir"] == "wgrad":
        y = _decode_columns(s["g"], s["g_scales"]).t() @ _decode_columns(s["x"], s["x_scales"])
    else:
        w = _decode_weight(s["w"], s["tile"])
        y = _decode_rows(s["x"], s["x_scales"]) @ (w.t() if case["dir"] == "fwd" else w)
    return y.to(_dtype(case["out"]))


def _parts(s, rows):
    """rows [cap, n] as [E, most, n], each expert's part padded with zero rows; and the place of each row in it."""
    off = s["order"]["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=rows.device)
    inside = at < off[1:, None]
    return rows[at.clamp(max=rows.shape[0] - 1)] * inside[..., None], at, inside


def _grouped(s):
    case, order = s["case"], s["order"]
    if case["dir"] == "wgrad":
        gp = _parts(s, _decode_columns(s["g"], s["g_scales"]))[0]
        xp = _parts(s, _decode_columns(s["x"], s["x_scales"]))[0]
        return torch.bmm(gp.transpose(1, 2), xp).to(_dtype(case["out"]))
    xp, at, inside = _parts(s, _decode_rows(s["x"], s["x_scales"]))
    w = _decode_weight(s["w"], s["tile"])
    y = torch.bmm(xp, w.transpose(1, 2) if case["dir"] == "fwd" else w).to(_dtype(case["out"]))
    cap = order["source"].numel()
    out = torch.zeros(cap + 1, y.shape[-1], dtype=y.dtype, device=y.device)  # rows behind the last part are zero
    out[torch.where(inside, at, cap)] = y
    return out[:cap]


def _sort(ids, E, align):
    """offsets [E+1]: where each expert's part begins, rounded up to `align` rows; source [capacity]: the choice (token * topk +
    place) at each row, -1 where there is none; slots [T, topk]: the row of each choice, -1 for a dropped one."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, torch.full_like(flat, E))
    by = torch.sort(key, stable=True).indices
    count = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(count, 0) - count
    room = torch.div(count[:E] + align - 1, align, rounding_mode="floor") * align
    offsets = torch.cat([torch.zeros(1, dtype=torch.long, device=ids.device), torch.cumsum(room, 0)])
    rank = torch.empty_like(by)
    rank[by] = torch.arange(n, device=ids.device)
    slots = torch.where(valid, torch.cat([offsets[:E], offsets[:1]])[key] + rank - first[key], torch.full_like(key, -1))
    cap = n + min(E, n) * (align - 1)
    source = torch.full((cap + 1,), -1, dtype=torch.long, device=ids.device)
    source[torch.where(valid, slots, torch.full_like(slots, cap))] = torch.arange(n, device=ids.device)
    source[cap] = -1
    return {"offsets": offsets.int(), "source": source[:cap].int(), "slots": slots.view(ids.shape).int()}


def _moe(s):
    case, order = s["case"], s["order"]
    topk, T, H, dt = case["topk"], case["T"], case["H"], _dtype(case["dtype"])
    source, slots = order["source"].long(), order["slots"].long()
    if case["part"] == "dispatch":
        taken = s["tokens"][torch.div(source.clamp(min=0), topk, rounding_mode="floor")]
        return torch.where((source >= 0)[:, None], taken, torch.zeros_like(taken))
    there = (slots >= 0)[..., None]
    rows = torch.where(there, s["rows"][slots.clamp(min=0)].float(), torch.zeros((), device=slots.device))  # [T, topk, H]
    if case["part"] == "dispatch_grad":
        return rows.sum(1).to(dt)
    w = s["weights"]
    if case["part"] == "combine":
        return (rows * w[..., None]).sum(1).to(dt)
    grad = s["tokens"].float()
    d_rows = torch.zeros(source.numel() + 1, H, dtype=dt, device=slots.device)
    d_rows[torch.where(slots >= 0, slots, source.numel()).view(-1)] = (grad[:, None] * w[..., None]).to(dt).view(-1, H)
    return {"rows": d_rows[: source.numel()], "weights": (rows * grad[:, None]).sum(-1)}


# --------------------------------------------------------- the library's


def _quant_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    return (mxq.mxq_fp8_quant_1x128 if s["case"]["axis"] == "rows" else mxq.mxq_fp8_quant_128x1)(s["x"])


def _product_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    case, dt = s["case"], _dtype(s["case"]["out"])
    if case["op"] == "grouped":
        off = s["order"]["offsets"]
        if case["dir"] == "wgrad":
            return mxq.mxq_fp8_grouped_matmul_wgrad(s["g"], s["g_scales"], s["x"], s["x_scales"], off, out_dtype=dt)
        f = mxq.mxq_fp8_grouped_matmul if case["dir"] == "fwd" else mxq.mxq_fp8_grouped_matmul_dgrad
        return f(s["x"], s["x_scales"], s["w"], s["tile"], off, out_dtype=dt)
    if case["dir"] == "wgrad":
        return mxq.mxq_fp8_matmul_wgrad(s["g"], s["g_scales"], s["x"], s["x_scales"], out_dtype=dt)
    f = mxq.mxq_fp8_matmul if case["dir"] == "fwd" else mxq.mxq_fp8_matmul_dgrad
    return f(s["x"], s["x_scales"], s["w"], s["tile"], out_dtype=dt)


def _sort_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    order = mxq.mxq_moe_sort(s["ids"], s["case"]["E"], align=s["case"]["align"])
    return {"offsets": order.offsets, "source": order.source, "slots": order.slots}


def _moe_own(s):
    import block_scaled_precision_x32_gb300 as mxq

    part, order, topk = s["case"]["part"], s["order"], s["case"]["topk"]
    if part == "dispatch":
        return mxq.mxq_moe_dispatch(s["tokens"], order["source"], topk)
    if part == "dispatch_grad":
        return mxq.mxq_moe_dispatch_grad(s["rows"], order["slots"])
    if part == "combine":
        return mxq.mxq_moe_combine(s["rows"], order["slots"], s["weights"])
    d_rows, d_weights = mxq.mxq_moe_combine_grad(s["tokens"], s["rows"], order["source"], order["slots"], s["weights"])
    return {"rows": d_rows, "weights": d_weights}


def run(state):
    op = state["case"]["op"]
    if op == "quant":
        plain = _quant_rows if state["case"]["axis"] == "rows" else _quant_columns
        data, scales = _quant_own(state) if own else plain(state["x"])
        return {"data": data.view(torch.float8_e4m3fn), "scales": scales.view(torch.float8_e8m0fnu)}
    if op == "matmul":
        return _product_own(state) if own else _matmul(state)
    if op == "grouped":
        return _product_own(state) if own else _grouped(state)
    if op == "sort":
        return _sort_own(state) if own else _sort(state["ids"], state["case"]["E"], state["case"]["align"])
    return _moe_own(state) if own else _moe(state)


# ------------------------------------------------------------ in 64 bits


def _fp8_values():
    """The 256 values of E4M3 bytes: sign, four exponent bits of bias 7, three of fraction; the last of each sign is NaN."""
    v = []
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        m = math.nan if c & 127 == 127 else f * 2.0**-9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        v.append(-m if c & 128 else m)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _values64(data, scale_of):
    """E4M3 bytes [..., r, c] in 64 bits, times the scale of their place."""
    return _fp8_values()[data.int()] * scale_of


def _two_to(e):
    """2^e in 64 bits for whole numbers e in [-400, 400]."""
    return torch.tensor([math.ldexp(1.0, k) for k in range(-400, 401)], dtype=torch.float64, device="cuda")[e.long() + 400]


def _power64(codes):
    return _two_to(codes.long() - 127)


def _along(s, n, axis):
    """Block scales spread over the n elements of an axis, 128 each."""
    return s.index_select(axis, torch.arange(n, device="cuda") // 128)


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    s = prepare(case, seed)
    if op == "quant":
        # the nearest value of the grid that the block's scale leaves, found from the number's own binary exponent
        x = s["x"].double() if case["axis"] == "rows" else s["x"].double().t()
        nb = _cdiv(x.shape[1], 128)
        b = torch.nn.functional.pad(x, (0, nb * 128 - x.shape[1])).reshape(x.shape[0], nb, 128)
        amax = b.abs().amax(2, keepdim=True)
        s = torch.ceil(torch.log2(amax / 448)).clamp(-127, 127)
        s = torch.where(amax <= 448 * _two_to(s - 1), s - 1, s)  # a logarithm that was rounded across a whole number
        s = torch.where(amax > 448 * _two_to(s), s + 1, s).clamp(-127, 127)
        v = b / _two_to(s)
        top = torch.floor(torch.log2(v.abs().clamp(min=2.0**-6)))
        top = torch.where(v.abs() >= 2 * _two_to(top), top + 1, torch.where((v.abs() < _two_to(top)) & (top > -6), top - 1, top))
        step = _two_to(top - 3)
        q = (torch.round(v / step) * step).reshape(x.shape[0], -1)[:, : x.shape[1]]
        scale = _two_to(s)[..., 0]
        return {"data": q, "scales": scale} if case["axis"] == "rows" else {"data": q.t(), "scales": scale.t()}
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        if case["dir"] == "wgrad":
            return _values64(s["g"], _along(_power64(s["g_scales"]), M, 0)).t() @ _values64(s["x"], _along(_power64(s["x_scales"]), M, 0))
        x = _values64(s["x"], _along(_power64(s["x_scales"]), s["x"].shape[1], 1))
        w = _values64(s["w"], _along(_along(s["tile"].double(), N, 0), K, 1))
        return x @ (w.t() if case["dir"] == "fwd" else w)
    off, source = s["order"]["offsets"].tolist(), s["order"]["source"]
    if op == "grouped":
        N, K, cap = case["N"], case["K"], source.numel()
        if case["dir"] == "wgrad":
            gd = _values64(s["g"], _along(_power64(s["g_scales"]), cap, 0))
            xd = _values64(s["x"], _along(_power64(s["x_scales"]), cap, 0))
            return torch.stack([gd[off[e] : off[e + 1]].t() @ xd[off[e] : off[e + 1]] for e in range(case["E"])])
        xd = _values64(s["x"], _along(_power64(s["x_scales"]), s["x"].shape[1], 1))
        y = torch.zeros(cap, N if case["dir"] == "fwd" else K, dtype=torch.float64, device="cuda")
        for e in range(case["E"]):
            if off[e] < off[e + 1]:
                w = _values64(s["w"][e], _along(_along(s["tile"][e].double(), N, 0), K, 1))
                y[off[e] : off[e + 1]] = xd[off[e] : off[e + 1]] @ (w.t() if case["dir"] == "fwd" else w)
        return y
    topk, H, part, slots = case["topk"], case["H"], case["part"], s["order"]["slots"].long()
    cap = source.numel()
    if part == "dispatch":
        y = torch.zeros(cap, H, dtype=torch.float64, device="cuda")
        at = torch.nonzero(source >= 0)[:, 0]
        y[at] = s["tokens"].double()[source[at].long() // topk]
        return y
    if part != "combine_grad":
        y = torch.zeros(case["T"], H, dtype=torch.float64, device="cuda")
        for k in range(topk):
            at = torch.nonzero(slots[:, k] >= 0)[:, 0]
            r = s["rows"][slots[at, k]].double()
            y[at] += r if part == "dispatch_grad" else r * s["weights"][at, k, None].double()
        return y
    d_rows, d_w = torch.zeros(cap, H, dtype=torch.float64, device="cuda"), torch.zeros(case["T"], topk, dtype=torch.float64, device="cuda")
    for k in range(topk):
        at = torch.nonzero(slots[:, k] >= 0)[:, 0]
        g = s["tokens"][at].double()
        d_rows[slots[at, k]] = g * s["weights"][at, k, None].double()
        d_w[at, k] = (g * s["rows"][slots[at, k]].double()).sum(1)
    return {"rows": d_rows, "weights": d_w}
