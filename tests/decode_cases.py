"""Seeded cases of the MoE decode operators (router, MoE MLP, projection with adapters),
encoded by the oracle's quantisers."""
from __future__ import annotations

import numpy as np

from oracle import formats as F
from oracle import fp4 as FP4


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def bf16(x):
    """FP64 values rounded to BF16: (bit patterns, their values)."""
    bits = F.f64_to_bf16(x)
    return bits, F.bf16_to_f64(bits)


def moe_case(seed, t, h, i, e, topk, routed=None, fp4=False, base=0):
    g = rng(seed)
    routed = routed or e
    qa, sa = F.quantize_rows(g.standard_normal((t, h)))

    def weights(n, k):
        w = g.standard_normal((n, k)) * 0.05
        if fp4:
            q, s = FP4.quantize_mxfp4(w)
            return q, FP4.pack_mx_scales(s)
        q, s = F.quantize_blocks(w)
        return q, F.pack_ue8m0(s)

    w13, w2 = [weights(2 * i, h) for _ in range(e)], [weights(h, i) for _ in range(e)]
    ids = np.argsort(g.random((t, routed)), axis=1)[:, :topk].astype(np.int32)
    w = g.random((t, topk)).astype(np.float32) + np.float32(0.1)
    return {"a": qa, "sfa": F.pack_ue8m0(sa), "w13": np.stack([x[0] for x in w13]), "sf13": np.stack([x[1] for x in w13]),
            "w2": np.stack([x[0] for x in w2]), "sf2": np.stack([x[1] for x in w2]), "ids": ids, "weights": w,
            "base": base, "fp4": fp4}


def lora_case(seed, m, n, k, l, r, none=0.2):
    g = rng(seed)
    xb, x = bf16(g.standard_normal((m, k)))
    a, sa = F.quantize_rows(x)
    b, sb = F.quantize_blocks(g.standard_normal((n, k)) * 0.05)
    la_bits, la = bf16(g.standard_normal((l, r, k)) * k ** -0.5)
    lb_bits, lb = bf16(g.standard_normal((l, n, r)) * r ** -0.5)
    ids = np.where(g.random(m) < none, -1, g.integers(0, l, m)).astype(np.int32)
    return {"a": a, "sfa": F.pack_ue8m0(sa), "b": b, "sfb": F.pack_ue8m0(sb), "x_bits": xb, "x": x, "la_bits": la_bits,
            "la": la, "lb_bits": lb_bits, "lb": lb, "scaling": (g.random(l) * 2 - 0.5).astype(np.float32), "ids": ids}


def lora_args(c):
    return [c[k] for k in ("a", "sfa", "b", "sfb", "x", "la", "lb", "scaling", "ids")]


def parts_case(seed, m, n, k, l, r):
    """A case whose result is x @ lora_a^T alone, value by value: FP8 rows of zeros, one element in each
    row of x, and rows of lora_b that pick one rank (even rows) or the difference of two ranks whose
    values are neighbours in BF16 (odd rows).  Every token has an adapter."""
    c = lora_case(seed, m, n, k, l, r, none=0.0)
    g = rng(seed + 1)
    c["a"] = np.zeros_like(c["a"])
    x = np.zeros((m, k))
    x[np.arange(m), g.integers(0, k, m)] = g.standard_normal(m)
    lb = np.zeros((l, n, r))
    for j in range(l):
        lb[j, np.arange(n), g.integers(0, r, n)] = g.choice([-1.0, 0.5, 1.0], n)
        lb[j, 1::2] = 0.0
        pair = 2 * g.integers(0, r // 2, n // 2)
        lb[j, np.arange(1, n, 2), pair] = 1.0
        lb[j, np.arange(1, n, 2), pair + 1] = -1.0
    c["la_bits"][:, 1::2] = c["la_bits"][:, 0::2] + 1
    c["la"] = F.bf16_to_f64(c["la_bits"])
    c["x_bits"], c["x"] = bf16(x)
    c["lb_bits"], c["lb"] = bf16(lb)
    return c
