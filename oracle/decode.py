"""The operators of an MoE decode step in FP64: router, whole MoE MLP, projection with
per-token adapters.

TEST INFRASTRUCTURE (oracle): see the header of ``oracle/formats.py`` for who may
import it.  Shares no code with the CUDA library.

``moe_mlp`` and ``lora`` also return a bound on what an FP32-accumulating implementation may
differ by, element by element, worked out from the operands:

* a sum of n products whose absolute values add up to S, accumulated step by step in FP32 by
  truncating adders, is off by at most n * 2^-23 * S, n counting the accumulation steps (the
  tensor core adds 32 FP8 or 16 BF16 products at a time; each partial sum joined later is one
  more step);
* E4M3 rounding of an FP32 value y known to within dy: whatever lies between the codes of
  y - dy and y + dy, under either scale if the group's maximum is that close to the next power;
* the result itself is rounded once, so it lies between the roundings of the two ends
  (``within``)."""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import fp4 as FP4
from .gemm import block_scales, dequant_k_major, row_scales

U = 2.0 ** -23


def within(got, ref, out) -> np.ndarray:
    """Whether each value lies between the roundings of d - bound and d + bound to the output type."""
    d, bound = ref
    r = (lambda x: F.bf16_to_f64(F.f64_to_bf16(x))) if out == "bf16" else (lambda x: x.astype(np.float32).astype(np.float64))
    return (got >= r(d - bound)) & (got <= r(d + bound))


# ------------------------------------------------------------------------ router
def route_keys(logits, bias, score, n_group, topk_group):
    """(scores, keys): keys of experts outside the chosen groups and of -inf/NaN logits are -inf."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    dead = np.isnan(x) | np.isneginf(x)
    x = np.where(dead, -np.inf, x)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-x))
        else:
            top = x.max(axis=1, keepdims=True)
            ex = np.where(dead, 0.0, np.exp(x - np.where(np.isfinite(top), top, 0.0)))
            s = ex / np.maximum(ex.sum(axis=1, keepdims=True), 1e-300)
    key = x.copy() if bias is None else np.where(dead, -np.inf, s + np.asarray(bias, np.float64))
    key = np.where(np.isnan(key), -np.inf, key)
    if n_group > 1:
        per = e // n_group
        for i in range(t):
            by = -np.sort(-key[i].reshape(n_group, per), axis=1)
            top = by[:, 0] if bias is None or per == 1 else by[:, 0] + by[:, 1]
            out = np.argsort(-top, kind="stable")[topk_group:]
            for g in out:
                key[i, g * per:(g + 1) * per] = -np.inf
    return s, key


def route(logits, topk, bias=None, score="softmax", n_group=1, topk_group=1, renormalize=True, scale=1.0):
    """(ids int32 [T, topk], weights float64 [T, topk]); ties to the lowest index, empty slots -1 and 0."""
    s, key = route_keys(logits, bias, score, n_group, topk_group)
    order = np.argsort(-key, axis=1, kind="stable")[:, :topk]
    live = np.take_along_axis(key, order, 1) > -np.inf
    w = np.where(live, np.take_along_axis(s, order, 1), 0.0)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return np.where(live, order, -1).astype(np.int32), w * scale


# ---------------------------------------------------------------------- MoE MLP
def _weights(q, sf, fp4):
    n = q.shape[0]
    if fp4:
        k = q.shape[1] * 2
        return FP4.dequant_mxfp4(q, FP4.mx_scales(sf, n, k))
    return dequant_k_major(q, block_scales(sf, n, q.shape[1]))


def _requantised(y, dy):
    """E4M3 1x128 requantisation of y (its FP32 rounding decides) and the interval it may fall in."""
    q, sf = F.quantize_rows(y.astype(np.float32).astype(np.float64))
    scale = lambda b: np.repeat(F.ue8m0_to_f64(b), 128, axis=1)  # noqa: E731
    value = F.e4m3_to_f64(q) * scale(sf)
    lo, hi = value.copy(), value.copy()
    g = np.abs(y).reshape(y.shape[0], -1, 128)
    d = dy.reshape(g.shape)
    for amax in ((g - d).max(axis=2), (g + d).max(axis=2)):
        sc = scale(F.ue8m0_for_amax(np.maximum(amax, 0.0)))
        for v in (y - dy, y + dy):
            r = F.e4m3_to_f64(F.f64_to_e4m3(np.clip(v / sc, -448, 448))) * sc
            lo, hi = np.minimum(lo, r), np.maximum(hi, r)
    return value, np.maximum(value - lo, hi - value)


def moe_mlp(a, sfa, w13, sf13, w2, sf2, ids, weights, expert_base=0, fp4=False):
    """(D float64 [T, H], bound float64 [T, H] before D's rounding): see ``fg_fp8_moe_mlp``."""
    t, h = a.shape
    e, i = w13.shape[0], w13.shape[1] // 2
    x = dequant_k_major(a, row_scales(sfa, t, h))
    d, err, mag = np.zeros((t, h)), np.zeros((t, h)), np.zeros((t, h))
    steps1, used = h // 32 + 8, 0
    for j in range(e):
        hit = np.asarray(ids) == expert_base + j
        rows = np.nonzero(hit.any(axis=1))[0]
        if not len(rows):
            continue
        used += 1
        w = np.where(hit, np.asarray(weights, np.float64), 0.0).sum(axis=1)[rows, None]
        m13, m2 = _weights(w13[j], sf13[j], fp4), _weights(w2[j], sf2[j], fp4)
        hid = x[rows] @ m13.T
        dh = steps1 * U * (np.abs(x[rows]) @ np.abs(m13).T)
        gate, up, dg, du = hid[:, :i], hid[:, i:], dh[:, :i], dh[:, i:]
        with np.errstate(over="ignore"):
            act = gate / (1.0 + np.exp(-gate))
        y = w * act * up
        # |SiLU'| <= 1.1; the FP32 exponential, quotient and products: 64 units together
        dy = np.abs(w) * (1.1 * dg * np.abs(up) + np.abs(act) * du + 1.1 * dg * du) + 64 * U * np.abs(y)
        q, dq = _requantised(y, dy)
        d[rows] += q @ m2.T
        err[rows] += dq @ np.abs(m2).T
        mag[rows] += np.abs(q) @ np.abs(m2).T
    return d, err + (used * (i // 32) + 8) * U * mag


# ------------------------------------------------------------------------- LoRA
def lora(a, sfa, b, sfb, x, lora_a, lora_b, scaling, ids, out="bf16"):
    """(D float64 [M, N], bound float64 [M, N] before D's rounding): see ``fg_fp8_gemm_nt_lora``; x, lora_a, lora_b
    hold BF16 values.

    Steps that add exact zeros (another token's adapter, padded ranks) leave an accumulator as it is, so
    a row counts its own only: K / 32 of FP8 products, whose partial sums stay below ``mag``, then
    one for each BF16 part and 16 ranks of its own adapter, and a join for every K-group and every
    adapter step that a cut may separate."""
    m, k = a.shape
    n = b.shape[0]
    wa, wb = dequant_k_major(a, row_scales(sfa, m, k)), dequant_k_major(b, block_scales(sfb, n, k))
    d = wa @ wb.T
    mag = np.abs(wa) @ np.abs(wb).T
    err = (k // 32) * U * mag
    r = lora_a.shape[1]
    for i in range(m):
        j = int(ids[i])
        steps = 0
        if 0 <= j < lora_a.shape[0]:
            s = float(scaling[j])
            v = s * (lora_a[j] @ x[i])
            dv = (k // 16 + 8) * U * abs(s) * (np.abs(lora_a[j]) @ np.abs(x[i]))
            dv += (2.0 ** -16 if out == "bf16" else 2.0 ** -23) * (np.abs(v) + dv)       # the BF16 parts
            d[i] += lora_b[j] @ v
            err[i] += np.abs(lora_b[j]) @ dv
            mag[i] += np.abs(lora_b[j]) @ np.abs(v)
            steps = (2 if out == "bf16" else 3) * ((r + 15) // 16)
        err[i] += (k // 128 + 2 * steps) * U * mag[i]
    return d, err
