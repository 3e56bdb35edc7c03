"""Seeded cases of the attention side of a serving step, encoded by the oracle."""
from __future__ import annotations

import numpy as np

from oracle import serving as O


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def cache_case(seed, lens, new, hq, hkv, d, page, spread=2, extra_rows=2, q_scale=1.5):
    """Requests of `lens` cached tokens of which the last `new` bring queries, in shuffled pages.  What no
    request holds is garbage: pages, rows behind a request's length (scale bytes that are infinite or
    huge), block-table entries behind its pages, rows of q behind the last request's."""
    g = rng(seed)
    lens, new = np.array(lens, np.int64), np.array(new, np.int64)
    need = -(-lens // page)
    width = int(max(1, need.max(initial=1))) + 1
    pages = int(need.sum()) + 3
    perm = g.permutation(pages)
    table = g.choice(np.array([-1, 2 ** 31 - 1, pages]), (len(lens), width))
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = perm[at:at + n]
        at += n
    kc, vc = (g.integers(0, 256, (pages, hkv, page, d // 2), dtype=np.uint8) for _ in range(2))
    ks, vs = (g.choice(np.array([255, 254, 0], np.uint8), (pages, hkv, page, d // 32)) for _ in range(2))
    for r, n in enumerate(lens):
        p, o = table[r, np.arange(n) // page], np.arange(n) % page
        for codes, sf, kind in ((kc, ks, "k"), (vc, vs, "v")):
            x = g.standard_normal((n, hkv, d)) * 2.0 ** g.integers(-spread, spread + 1, (n, hkv, 1))
            c, s = O.encode(x)
            codes[p, :, o], sf[p, :, o] = O.rows(c, kind), s
    start = np.concatenate([[0], np.cumsum(new)])
    t = int(start[-1]) + extra_rows
    q_bits, q = O.bf16(g.standard_normal((t, hq, d)) * q_scale)
    return {"q_bits": q_bits, "q": q, "kc": kc, "ks": ks, "vc": vc, "vs": vs, "table": table.astype(np.int32),
            "start": start.astype(np.int32), "lens": lens.astype(np.int32), "page": page, "d": d, "hq": hq, "hkv": hkv,
            "pages": pages}


def wide(c, tokens=1 << 18):
    """The same case with room for longer contexts in its block table (what is faster is chosen by that)."""
    more = max(0, tokens // c["page"] - c["table"].shape[1])
    return dict(c, table=np.pad(c["table"], ((0, 0), (0, more)), constant_values=-1))


def many_rows(c, window=0):
    """Whether the tensor cores take 128 rows or more at a time."""
    group, s, d = c["hq"] // c["hkv"], len(c["lens"]), c["d"]
    new = -(-len(c["q"]) // s)
    rows, keys = new * group, c["table"].shape[1] * c["page"]
    if window:
        keys = min(keys, window + new)
    blocks, few = keys // 128 + 1, min({64: 32, 128: 16, 256: 8}[d], 8 if rows <= 8 else 16 if rows <= 16 else 32)
    here, there = s * c["hkv"] * -(-rows // few) * (5 + blocks), s * c["hkv"] * -(-rows // 128) * (3 + blocks)
    return s <= 1024 and rows > 32 and here > {64: 2.1, 128: 3.2, 256: 9.0}[d] * there + 2300


def reference(c, scale=None, window=0):
    return O.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["table"], c["start"], c["lens"],
                       c["d"] ** -0.5 if scale is None else scale, window, 2.0 ** (-8 if many_rows(c, window) else -11))


def tables_case(seed, s, page, longest, width, mode):
    g = rng(seed)
    context = g.integers(0, longest + 1, s)
    new = {"decode": lambda: g.choice([1, 1, 1, 0, -1], s), "prompts": lambda: g.integers(-1, 60, s)}[mode]()
    total = int((-(-context // page)).sum() + (-(-np.maximum(new, 0) // page) + 1).sum()) + 2
    perm = g.permutation(total)
    table = np.full((s, width), -5)
    at = 0
    for r in range(s):
        n = -(-context[r] // page)
        table[r, :n] = perm[at:at + n]
        at += n
    free = np.concatenate([perm[at:], np.full(at, -9)])
    return {"context": context, "new": new, "table": table, "free": free, "count": total - at, "pages": total,
            "t": int(np.maximum(new, 0).sum())}
