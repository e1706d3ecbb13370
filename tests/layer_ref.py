"""64-bit references of the FP8 linear layer and the mixture-of-experts
operators, in numpy and from their definitions alone."""

import numpy as np


def _e4m3_table():
    """Values of the codes 0..126: four exponent bits of bias 7, three of fraction."""
    v = []
    for c in range(127):
        e, f = c >> 3, c & 7
        v.append(f * 2.0**-9 if e == 0 else (8 + f) * 2.0 ** (e - 10))
    return np.array(v)


E4M3 = _e4m3_table()
_MID = (E4M3[1:] + E4M3[:-1]) / 2


def e4m3_decode(b):
    b = np.asarray(b, dtype=np.uint8)
    v = np.append(E4M3, np.nan)[b & 0x7F]
    return np.where(b & 0x80, -v, v)


def e4m3_encode(v):
    """Nearest code of finite |v| <= 448, ties to the even code, the sign kept."""
    a = np.abs(v)
    code = np.searchsorted(_MID, a, side="left")  # a midpoint belongs to the code below it ...
    tie = (code < len(_MID)) & (a == _MID[np.minimum(code, len(_MID) - 1)])
    code = np.where(tie & (code % 2 == 1), code + 1, code)  # ... unless that one is odd
    return (code | (np.signbit(v) << 7)).astype(np.uint8)


def ue8m0(c):
    c = np.asarray(c).astype(np.int64)
    return np.where(c == 255, np.nan, np.ldexp(1.0, np.minimum(c, 254) - 127))


def quant_rows(x):
    """x float64 [rows, K] -> (E4M3 bytes, UE8M0 codes [rows, ceil(K/128)])."""
    rows, K = x.shape
    nb = -(-K // 128)
    data = np.zeros((rows, K), np.uint8)
    codes = np.zeros((rows, nb), np.uint8)
    for j in range(nb):
        b = x[:, 128 * j:128 * j + 128]
        bad = ~np.isfinite(b).all(1)
        amax = np.where(bad, 0.0, np.abs(np.where(bad[:, None], 0.0, b)).max(1))
        m, e = np.frexp(amax)  # 448 = 0.875 * 2^9
        s = np.where(amax > 0, np.clip(e - 9 + (m > 0.875), -127, 127), -127)
        enc = e4m3_encode(np.where(bad[:, None], 0.0, b) * np.ldexp(1.0, -s)[:, None])
        data[:, 128 * j:128 * j + 128] = np.where(bad[:, None], 0x7F, enc)
        codes[:, j] = np.where(bad, 255, s + 127)
    return data, codes


def quant_columns(x):
    d, c = quant_rows(np.ascontiguousarray(x.T))
    return np.ascontiguousarray(d.T), np.ascontiguousarray(c.T)


def gather(x, index, div):
    """Row index[i] // div of x, zeros for a negative index or one that leaves x."""
    t = np.where(index < 0, -1, index // div)
    ok = (t >= 0) & (t < x.shape[0])
    out = np.zeros((len(index),) + x.shape[1:], x.dtype)
    out[ok] = x[t[ok]]
    return out


def decode_rows(data, codes):
    return e4m3_decode(data) * np.repeat(ue8m0(codes), 128, 1)[:, : data.shape[1]]


def decode_columns(data, codes):
    return e4m3_decode(data) * np.repeat(ue8m0(codes), 128, 0)[: data.shape[0]]


def decode_weight(w, tile):
    """[..., N, K] bytes and [..., N/128, K/128] tile scales."""
    s = np.repeat(np.repeat(tile.astype(np.float64), 128, -2), 128, -1)
    return e4m3_decode(w) * s[..., : w.shape[-2], : w.shape[-1]]


def product(a, b):
    """(a b^T, |a| |b|^T) in 64 bits for a [m, d], b [n, d]."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def clamp_offsets(offsets, rows):
    return np.maximum.accumulate(np.clip(offsets.astype(np.int64), 0, rows))


def moe_sort(ids, E, align):
    T, topk = ids.shape
    n = T * topk
    flat = ids.reshape(-1)
    cap = n + min(E, n) * (align - 1)
    offsets = np.zeros(E + 1, np.int64)
    source = np.full(cap, -1, np.int64)
    slots = np.full(n, -1, np.int64)
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        at = offsets[e] + np.arange(len(mine))
        source[at] = mine
        slots[mine] = at
        offsets[e + 1] = offsets[e] + -(-len(mine) // align) * align
    return offsets, source, slots.reshape(T, topk)
