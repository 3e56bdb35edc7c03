"""The attention side of a serving step in FP64: block tables, norms with rotation, the 4-bit
key/value cache and attention over it.

TEST INFRASTRUCTURE (oracle): see the header of ``oracle/formats.py`` for who may
import it.  Shares no code with the CUDA library.

``attention`` and ``norm_rope`` also return a bound on what an FP32-accumulating implementation
may differ by, element by element (``oracle.decode.within`` compares with it)."""
from __future__ import annotations

import numpy as np

from . import fp4 as FP4
from .formats import bf16_to_f64, f64_to_bf16

U = 2.0 ** -24                 # half a step of FP32, relative
MIN_BYTE, MAX_BYTE = 63, 190   # scales of the cache: 2^-64 .. 2^63


# ---------------------------------------------------------------------- block tables
def block_tables(context, new, free, count, table, t, page, num_pages):
    """The step's arrays, request by request and page by page; None if the step has to be refused."""
    context, new, free, table = (np.array(x, np.int64) for x in (context, new, free, table))
    s, width = table.shape
    if (context < 0).any() or (new < -1).any() or not 0 <= count <= len(free):
        return None
    stack = list(free[:count])
    for r in range(s):
        if -(-(context[r] + max(new[r], 0)) // page) > width:
            return None
        if new[r] < 0:
            stack += [int(x) for x in table[r, :-(-context[r] // page)]]
    if len(stack) > len(free) or sum(max(int(x), 0) for x in new) > t:
        return None
    free[:len(stack)] = stack
    slots, positions = np.full(t, -1, np.int64), np.full(t, -1, np.int64)
    start, lens = np.zeros(s + 1, np.int64), np.zeros(s, np.int64)
    at, bad_page = 0, False
    for r in range(s):
        start[r] = at
        if new[r] < 0:
            continue
        lens[r] = context[r] + new[r]
        for j in range(-(-context[r] // page), -(-lens[r] // page)):
            if not stack:
                return None
            table[r, j] = stack.pop()
        for pos in range(context[r], lens[r]):
            p = table[r, pos // page]
            ok = 0 <= p < num_pages
            bad_page |= not ok
            slots[at], positions[at] = (p * page + pos % page if ok else -1), pos
            at += 1
    start[s] = at
    return {"table": table, "free": free, "count": len(stack), "start": start, "lens": lens, "slots": slots,
            "positions": positions, "bad_page": bad_page}


# -------------------------------------------------------------------- norms, rotation
def norm_rope(x, w, eps, positions, cos_sin, interleaved):
    """x [T, H, D]; w [D] or None; cos_sin [max_pos, rot].  (values, bound)."""
    x = np.asarray(x, np.float64)
    d, rot = x.shape[-1], cos_sin.shape[1]
    y = x
    if w is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    cs = np.asarray(cos_sin, np.float64)[positions][:, None]
    cos, sin = cs[..., :rot // 2], cs[..., rot // 2:]
    i = np.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    out, size = y.copy(), np.abs(y)
    out[..., a], out[..., b] = y[..., a] * cos - y[..., b] * sin, y[..., b] * cos + y[..., a] * sin
    size[..., a] = np.abs(y[..., a] * cos) + np.abs(y[..., b] * sin)
    size[..., b] = np.abs(y[..., b] * cos) + np.abs(y[..., a] * sin)
    # x^2 summed over D elements, the mean, rsqrt (2 units), two products, the rotation's product and sum:
    # half the sum's relative error goes through the root
    return out, size * (d / 2 + 8) * 2 * U


# ------------------------------------------------------------------------------ cache
def encode(x):
    """x [.., D] -> (E2M1 codes [.., D], scale bytes [.., D / 32]) of finite values."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    u = np.clip(FP4.ue8m0_for_amax_fp4(np.abs(g).max(-1)).astype(np.int64), MIN_BYTE, MAX_BYTE)
    return FP4.f64_to_e2m1(g * 2.0 ** (127.0 - u)[..., None]).reshape(x.shape), u.astype(np.uint8)


def nibbles(d, kind):
    """Nibble of its row that each element of a key ("k") or value ("v") row stands in."""
    b, e = d // 32, np.arange(d)
    block, i = e // 32, e % 32
    per = 8 if kind == "k" else 4
    return (i // per * b + block) * per + i % per


def rows(codes, kind):
    """Codes [.., D] in elements' order -> bytes [.., D / 2] as the cache holds them."""
    out = np.zeros_like(codes)
    out[..., nibbles(codes.shape[-1], kind)] = codes
    return FP4.pack_fp4(out)


def decode(row, sf, kind):
    """Cache bytes [.., D / 2] and scales [.., D / 32] -> FP64 values [.., D]."""
    codes = FP4.unpack_fp4(row)
    codes = codes[..., nibbles(codes.shape[-1], kind)]
    v = FP4.e2m1_to_f64(codes).reshape(*codes.shape[:-1], codes.shape[-1] // 32, 32)
    return (v * 2.0 ** (sf.astype(np.float64) - 127.0)[..., None]).reshape(codes.shape)


def cached(table_row, n, codes, sf, kind, head):
    """FP64 [n, D]: the first n cached tokens of one head of one request."""
    page = codes.shape[2]
    j = np.arange(n)
    p = np.asarray(table_row, np.int64)[j // page]
    return decode(codes[p, head, j % page], sf[p, head, j % page], kind)


# -------------------------------------------------------------------------- attention
def attention(q, kc, ks, vc, vs, table, start, lens, scale, window=0, weight=2.0 ** -11, floor=2.0 ** -33):
    """q [T, Hq, D] FP64 values.  (out, bound, used): rows of requests are True in `used`.

    Bound, row by row: a score of D products, whose absolute values add up to S, is off by D + 8 units of S in
    FP32 (products and partial sums; q's conversion to FP16 after a power-of-two scaling is exact down to 2^-22 of
    the row's largest, 2^-33 of it absolute); the exponential adds 8 units; a weight times its value's scale is
    rounded to FP16, 2^-11 of itself (``weight``) or 2^-33 (``floor``) of the row's largest; sums over n keys are off by n + 16 units (n / 16
    accumulations and the joins).  Numerator and denominator errors add up."""
    t, hq, d = q.shape
    hkv = kc.shape[1]
    group = hq // hkv
    out, bound, used = np.zeros(q.shape), np.zeros(q.shape), np.zeros(t, bool)
    for r in range(len(lens)):
        t0, n, length = int(start[r]), int(start[r + 1] - start[r]), int(lens[r])
        used[t0:t0 + n] = True
        if n == 0 or length == 0:
            continue
        pos = np.arange(length - n, length)[:, None]
        j = np.arange(length)[None]
        seen = (j <= pos) & ((j > pos - window) if window else True)
        for h in range(hkv):
            k, v = cached(table[r], length, kc, ks, "k", h), cached(table[r], length, vc, vs, "v", h)
            vscale = np.repeat(2.0 ** (np.stack([vs[int(table[r][i // kc.shape[2]]), h, i % kc.shape[2]] for i in range(length)])
                                       .astype(np.float64) - 127.0), 32, axis=1)
            for hh in range(h * group, (h + 1) * group):
                x = q[t0:t0 + n, hh]
                s = x @ k.T * scale
                size = np.abs(x) @ np.abs(k).T * scale
                low = np.abs(x).max(1, keepdims=True) * 2.0 ** -33 * np.abs(k).sum(1)[None] * scale
                s = np.where(seen, s, -np.inf)
                top = s.max(1, keepdims=True)
                any_key = np.isfinite(top)
                p = np.where(seen, np.exp(s - np.where(any_key, top, 0.0)), 0.0)
                total = np.where(any_key, p.sum(1, keepdims=True), 1.0)
                p /= total
                ds = np.where(seen, (size * (d + 8) + np.abs(np.where(seen, s, 0.0)) * 4) * 2 * U + low, 0.0) + 8 * 2 * U
                ds = np.expm1(np.minimum(ds, 1.0))
                o = p @ v
                largest = np.max(p[:, :, None] * vscale[None], axis=(1, 2))[:, None]
                num = (p * (ds + weight)) @ np.abs(v) + (p @ np.abs(v)) * (length + 16) * 2 * U
                num += floor * largest * 6 * seen.sum(1, keepdims=True)
                den = (p * ds).sum(1, keepdims=True) + (length + 16) * 2 * U
                out[t0:t0 + n, hh] = o
                bound[t0:t0 + n, hh] = num + np.abs(o) * den
    return out, bound, used


def bf16(x):
    """FP64 values rounded to BF16: (bit patterns, their values)."""
    bits = f64_to_bf16(np.asarray(x, np.float64))
    return bits, bf16_to_f64(bits)
