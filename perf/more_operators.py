"""The attention side of a serving step over a key/value cache held in 4 bits, as cases that can
be timed and compared.

Four operators, each in a plain form (elementary torch operations, rounded once) and as calls of
the library (``own``):

* pages: block tables, slots and positions of a step's tokens from the requests' lengths
         (``build_block_tables``);
* rope:  norms of queries and keys for each head with the position rotation (``qk_norm_rope``);
* kv:    keys and values into the 4-bit cache, and back out of it (``kv_append_mxfp4``,
         ``kv_gather_mxfp4``);
* attn:  attention of each request's new tokens over its cached ones (``paged_attention_mxfp4``).

A cache row of one head and token holds D E2M1 codes and one UE8M0 scale per 32 of them.  Codes
stand in the order the attention reads them in (B = D / 32): element 32 b + 8 c + j of a key is
nibble (c B + b) 8 + j, element 32 b + 4 g + j of a value is nibble (g B + b) 4 + j.

``exact`` states each operator that computes numbers again in FP64."""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step of 256 requests, one token each, a few of them finished: latency
        {"name": "pages_256_decode", "op": "pages", "S": 256, "T": 256, "page": 64, "context": 4096, "mode": "decode"},
        # a step that admits prompts: up to 8192 tokens over 48 requests, small pages
        {"name": "pages_48_prompts", "op": "pages", "S": 48, "T": 8192, "page": 16, "context": 2048, "mode": "prompts"},
        # one new token: latency
        {"name": "rope_1", "op": "rope", "T": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "norm": True, "pairs": False},
        # a prompt of 8192 tokens, queries and keys side by side in the projection's output
        {"name": "rope_8192", "op": "rope", "T": 8192, "Hq": 64, "Hkv": 8, "D": 128, "rot": 128, "norm": True, "pairs": False},
        # an odd batch of small heads, half of each rotated, neighbours as pairs, no norm
        {"name": "rope_333_half", "op": "rope", "T": 333, "Hq": 12, "Hkv": 4, "D": 64, "rot": 32, "norm": False, "pairs": True},
        # an odd decode batch into the cache
        {"name": "kv_37", "op": "kv", "T": 37, "Hkv": 8, "D": 128, "page": 64},
        # a prompt of 8192 tokens into the cache
        {"name": "kv_8192", "op": "kv", "T": 8192, "Hkv": 8, "D": 128, "page": 64},
        # one request with a short context: launches and latency
        {"name": "attn_1x129", "op": "attn", "S": 1, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "context": 129, "new": 1,
         "ragged": False, "window": 0},
        # a decode batch of 64 requests of uneven lengths up to 8192
        {"name": "attn_64x8192_ragged", "op": "attn", "S": 64, "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "context": 8192,
         "new": 1, "ragged": True, "window": 0},
        # one request with a very long context
        {"name": "attn_1x131072", "op": "attn", "S": 1, "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "context": 131072, "new": 1,
         "ragged": False, "window": 0},
        # drafts of 4 tokens being verified, small heads, a sliding window, pages of 16
        {"name": "attn_24x4_window", "op": "attn", "S": 24, "Hq": 24, "Hkv": 8, "D": 64, "page": 16, "context": 3000, "new": 4,
         "ragged": True, "window": 1024},
        # prompts being read in pieces of up to 512 tokens over what is cached of them
        {"name": "attn_4x512_prompts", "op": "attn", "S": 4, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "context": 6000,
         "new": 512, "ragged": True, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "kv", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "pages":
        mode = rng.choice(["decode", "prompts"])
        s = _log_int(rng, 1, 512 if mode == "decode" else 64)
        return {"op": op, "S": s, "T": s + rng.randint(0, 32) if mode == "decode" else _log_int(rng, 64, 8192), "page": page,
                "context": _log_int(rng, 1, 4096), "mode": mode}
    heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 8, 12, 16])
    dim = rng.choice([64, 128, 128, 256])
    if op == "rope":
        t = _log_int(rng, 1, 8192)
        while t * heads * (group + 1) * dim > 8192 * 72 * 128:
            t //= 2
        return {"op": op, "T": t, "Hq": heads * group, "Hkv": heads, "D": dim, "rot": rng.choice([32, 64, dim]),
                "norm": rng.random() < 0.6, "pairs": rng.random() < 0.4}
    if op == "kv":
        t = _log_int(rng, 1, 8192)
        while t * heads * dim > 8192 * 8 * 128:
            t //= 2
        return {"op": op, "T": t, "Hkv": heads, "D": dim, "page": page}
    new = rng.choice([1, 1, 1, 1, rng.randint(2, 8), _log_int(rng, 16, 512)])
    context = _log_int(rng, 1, 32768 if new <= 8 else 6000)
    s = _log_int(rng, 1, 64 if new <= 8 else 4)
    while s > 1 and s * heads * dim * (context + new) > 64 * 8 * 128 * 8192:
        s //= 2
    while new > 8 and s * new * heads * group * dim * (context + new) > 4 * 512 * 32 * 128 * 6000:
        new //= 2
    return {"op": op, "S": s, "Hq": heads * group, "Hkv": heads, "D": dim, "page": page, "context": context, "new": new,
            "ragged": rng.random() < 0.7, "window": rng.choice([0, 0, _log_int(rng, 16, 4096)])}


def _row_bytes(d):
    return d // 2 + d // 32


def work(case):
    op = case["op"]
    if op == "pages":
        s, t = case["S"], case["T"]
        return {"bytes": 4 * (2 * s + 2 * s + 1 + 2 * t + t // case["page"] + s), "flops": 4 * (s + t)}
    if op == "rope":
        t, rot = case["T"], case["rot"]
        n = t * (case["Hq"] + case["Hkv"]) * case["D"]
        return {"bytes": 4 * n + t * 4 + t * rot * 4, "flops": 8 * n}
    if op == "kv":
        n = case["T"] * case["Hkv"]
        return {"bytes": 2 * n * (4 * case["D"] + 2 * _row_bytes(case["D"])) + 8 * case["T"], "flops": 8 * n * case["D"]}
    s, new, group = case["S"], case["new"], case["Hq"] // case["Hkv"]
    c = case["context"] * (0.5 if case["ragged"] else 1.0)
    n = (new + 1) // 2 if case["ragged"] and new > 8 else new
    keys = c + n / 2                                      # keys that a new token looks at
    seen = c + n                                          # keys that a request reads
    if case["window"]:
        keys, seen = min(keys, case["window"]), min(seen, case["window"] + n)
    d = case["D"]
    return {"bytes": s * seen * case["Hkv"] * 2 * _row_bytes(d) + 4 * s * n * case["Hq"] * d,
            "flops": 4 * s * n * case["Hkv"] * group * d * keys}


# ------------------------------------------------------------------------- prepare
def _codes(x):
    """Values [.., D] -> E2M1 codes [.., D] and scale bytes [.., D / 32]: the smallest power of two (kept within 2^-64
    and 2^63) that brings a block's largest magnitude within 6, codes to the nearest, ties to the even one."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = g.abs().amax(-1)
    fr, ex = torch.frexp(amax)
    e = torch.where(amax > 0, torch.where(fr <= 0.75, ex - 3, ex - 2), torch.zeros_like(ex)).clamp(-64, 63)
    v = (g * ((127 - e).to(torch.int32) << 23).view(torch.float32)[..., None]).reshape(x.shape)
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for mid, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= mid if up else a > mid).to(torch.uint8)
    return code | torch.signbit(v).to(torch.uint8) << 3, (e + 127).to(torch.uint8)


def _pack(code, per):
    """Codes [.., D] in elements' order -> row bytes [.., D / 2]; per = 8 for keys, 4 for values."""
    d = code.shape[-1]
    c = code.reshape(*code.shape[:-1], d // 32, 32 // per, per).transpose(-2, -3).reshape(*code.shape[:-1], d // 2, 2)
    return c[..., 0] | c[..., 1] << 4


def _values(row, sf, per):
    """Row bytes [.., D / 2] and scale bytes [.., D / 32] -> FP32 values [.., D]."""
    d = row.shape[-1] * 2
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=row.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(row & 15).int()], table[(row >> 4).int()]], -1)
    v = v.reshape(*row.shape[:-1], 32 // per, d // 32, per).transpose(-2, -3).reshape(*row.shape[:-1], d // 32, 32)
    return (v * (sf.to(torch.int32) << 23).view(torch.float32)[..., None]).reshape(*row.shape[:-1], d)


def _lengths(n, hi, gen, ragged):
    if not ragged:
        return torch.full((n,), hi, device=DEV)
    return (1 + (hi - 1) * torch.rand(n, generator=gen, device=DEV)).round().long()


def _tables(lens, longest, extra, page, gen):
    """Shuffled pages: a block table that holds `lens` tokens a row, rows of up to `longest` tokens and `extra` more pages
    in all, the pages left over and the number of all."""
    need = (lens + page - 1) // page
    width = (longest + page - 1) // page + 1
    total = len(lens) * (width - 1) + extra
    perm = torch.randperm(total, generator=gen, device=DEV)
    start = need.cumsum(0) - need
    col = torch.arange(width, device=DEV)[None]
    table = torch.where(col < need[:, None], perm[(start[:, None] + col).clamp(max=total - 1)], torch.zeros_like(col))
    return table.to(torch.int32).contiguous(), perm[int(need.sum()):].to(torch.int32).contiguous(), total


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 29)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEV) * std

    s = dict(case)
    op = case["op"]
    if op == "pages":
        n, t, page = case["S"], case["T"], case["page"]
        context = _lengths(n, case["context"], gen, True)
        if case["mode"] == "decode":
            new = torch.ones(n, dtype=torch.long, device=DEV)
            new[torch.rand(n, generator=gen, device=DEV) < 0.05] = -1            # finished: gives its pages back
        else:                                             # prompts share the step's tokens; some requests wait
            share = torch.rand(n, generator=gen, device=DEV)
            new = (share / share.sum() * t).floor().long()
            context[torch.rand(n, generator=gen, device=DEV) < 0.5] = 0          # admitted in this step
        longest = case["context"] + (1 if case["mode"] == "decode" else t)
        s["table"], free, s["pages"] = _tables(context, longest, 3, page, gen)
        s["context_lens"], s["new_lens"] = context.to(torch.int32), new.to(torch.int32)
        s["free"] = torch.cat([free, torch.zeros(s["pages"] - len(free), dtype=torch.int32, device=DEV)])
        s["count"] = torch.tensor([len(free)], dtype=torch.int32, device=DEV)
        s["count_out"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["start"] = torch.empty(n + 1, dtype=torch.int32, device=DEV)
        s["lens"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["slots"], s["positions"] = (torch.empty(t, dtype=torch.int32, device=DEV) for _ in range(2))
        return s
    d, hkv = case["D"], case["Hkv"]
    if op == "rope":
        t, hq, rot = case["T"], case["Hq"], case["rot"]
        qkv = normal(t, (hq + 2 * hkv) * d, std=2.0).to(torch.bfloat16)          # the projection's output
        s["q"] = qkv[:, :hq * d].view(t, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        far = 16384
        inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
        angle = torch.arange(far, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()
        first = int(torch.randint(0, far - t, (1,), generator=gen, device=DEV))
        s["positions"] = torch.arange(first, first + t, dtype=torch.int32, device=DEV)
        s["qw"], s["kw"] = ((1.0 + normal(d, std=0.1)).to(torch.bfloat16) if case["norm"] else None for _ in range(2))
        s["qo"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["ko"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        return s
    page = case["page"]
    if op == "kv":
        t = case["T"]
        pages = (t + page - 1) // page + 5
        qkv = normal(t, 2 * hkv * d).to(torch.bfloat16)
        s["k"], s["v"] = qkv[:, :hkv * d].view(t, hkv, d), qkv[:, hkv * d:].view(t, hkv, d)
        perm = torch.randperm(pages, generator=gen, device=DEV)
        at = torch.arange(t, device=DEV) + page // 2
        s["slots"] = (perm[at // page] * page + at % page).to(torch.int32)
        for name in ("k", "v"):
            s[name + "c"] = torch.zeros(pages, hkv, page, d // 2, dtype=torch.uint8, device=DEV)
            s[name + "s"] = torch.zeros(pages, hkv, page, d // 32, dtype=torch.uint8, device=DEV)
            s[name + "o"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        return s
    n, hq = case["S"], case["Hq"]
    context = _lengths(n, case["context"], gen, case["ragged"])
    if case["ragged"] and case["new"] > 8:                # prompts share the step's tokens
        t = n * (case["new"] + 1) // 2
        share = 0.2 + torch.rand(n, generator=gen, device=DEV)
        new = (share / share.sum() * t).floor().long().clamp(1, case["new"])
    else:
        t = n * case["new"]
        new = torch.full((n,), case["new"], device=DEV)
    lens = context + new
    s["table"], _, pages = _tables(lens, case["context"] + case["new"], 3, page, gen)
    start = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), new.cumsum(0)])
    s["start"], s["lens"] = start.to(torch.int32), lens.to(torch.int32)
    s["widest"] = case["new"]
    s["q"] = normal(t, hq, d, std=1.5).to(torch.bfloat16)
    s["out"] = torch.zeros(t, hq, d, dtype=torch.bfloat16, device=DEV)           # rows behind the last request's stay
    for name, per in (("k", 8), ("v", 4)):
        s[name + "c"] = torch.empty(pages, hkv, page, d // 2, dtype=torch.uint8, device=DEV)
        s[name + "s"] = torch.empty(pages, hkv, page, d // 32, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (hkv * page * d))
        for i in range(0, pages, step):
            code, sf = _codes(normal(min(step, pages - i), hkv, page, d))
            s[name + "c"][i:i + step], s[name + "s"][i:i + step] = _pack(code, per), sf
    if own:                                              # the workspace that a program keeps beside its cache
        import moe_fp8_e4m3_gb300 as fg
        s["workspace"] = fg.paged_attention_workspace(t, n, hq, hkv, d)
    return s


# ----------------------------------------------------------------------------- run
def run(s):
    if own:
        import moe_fp8_e4m3_gb300 as fg
        if s["op"] == "pages":
            fg.build_block_tables(s["context_lens"], s["new_lens"], s["free"], s["count"], s["table"], s["start"], s["lens"],
                                  s["slots"], s["positions"], s["count_out"], page_size=s["page"], num_pages=s["pages"])
            return s["table"], s["start"], s["lens"], s["slots"], s["positions"], s["free"], s["count_out"]
        if s["op"] == "rope":
            fg.qk_norm_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["qo"], s["ko"], q_weight=s["qw"], k_weight=s["kw"],
                            eps=1e-6, interleaved=s["pairs"])
            return s["qo"], s["ko"]
        if s["op"] == "kv":
            fg.kv_append_mxfp4(s["k"], s["v"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"])
            fg.kv_gather_mxfp4(s["slots"], s["kc"], s["ks"], s["vc"], s["vs"], s["ko"], s["vo"])
            return s["ko"], s["vo"]
        fg.paged_attention_mxfp4(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["start"], s["lens"], s["out"],
                                 s["workspace"], window=s["window"])
        return s["out"]
    return {"pages": _pages_plain, "rope": _rope_plain, "kv": _kv_plain, "attn": _attn_plain}[s["op"]](s)


def _pages_plain(s):
    page, t, n = s["page"], s["T"], s["S"]
    context, new = s["context_lens"].long(), s["new_lens"].long()
    done = new < 0
    new = new.clamp(min=0)
    held = (context + page - 1) // page
    col = torch.arange(s["table"].shape[1], device=DEV)[None]
    # finished requests' pages on top of the free ones, in the requests' order
    back = torch.where(done, held, torch.zeros_like(held))
    at = s["count"].long() + back.cumsum(0) - back
    free = torch.cat([s["free"], s["free"][:1]])                     # one more place for what is not given back
    where = torch.where((col < back[:, None]), at[:, None] + col, torch.full_like(col, len(s["free"])))
    free = free.scatter(0, where.reshape(-1), s["table"].reshape(-1))[:-1]
    count = s["count"].long() + back.sum()
    # new pages from the top, in the requests' order
    lens = torch.where(done, torch.zeros_like(context), context + new)
    more = torch.where(done, torch.zeros_like(held), (lens + page - 1) // page - held)
    first = more.cumsum(0) - more
    fresh = (col >= held[:, None]) & (col < (held + more)[:, None])
    top = (count - 1 - first[:, None] - (col - held[:, None])).clamp(0, len(s["free"]) - 1)
    table = torch.where(fresh, free[top], s["table"])
    start = torch.cat([torch.zeros_like(count), new.cumsum(0)])
    i = torch.arange(t, device=DEV)
    r = torch.searchsorted(start[1:].contiguous(), i, right=True).clamp(max=n - 1)
    used = i < start[-1]
    pos = context[r] + i - start[r]
    slots = table[r, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    minus = torch.full_like(i, -1)
    i32 = torch.int32
    return (table, start.to(i32), lens.to(i32), torch.where(used, slots, minus).to(i32), torch.where(used, pos, minus).to(i32),
            free, (count - more.sum()).to(i32))


def _rope_plain(s):
    rot, half = s["rot"], s["rot"] // 2
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., :half], cs[..., half:]
    out = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        turn = x[..., :rot]
        if s["pairs"]:
            a, b = turn[..., 0::2], turn[..., 1::2]
            turn = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = turn[..., :half], turn[..., half:]
            turn = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out.append(torch.cat([turn, x[..., rot:]], -1).to(torch.bfloat16))
    return tuple(out)


def _kv_plain(s):
    page = s["page"]
    slot = s["slots"].long()
    p, o = slot // page, slot % page
    out = []
    for name, per in (("k", 8), ("v", 4)):
        code, sf = _codes(s[name].float())
        cache, scales = s[name + "c"], s[name + "s"]
        cache[p, :, o], scales[p, :, o] = _pack(code, per), sf
        out.append(_values(cache[p, :, o], scales[p, :, o], per).to(torch.bfloat16))
    return tuple(out)


def _attn_plain(s):
    n, hkv, d, page = s["S"], s["Hkv"], s["D"], s["page"]
    group = s["Hq"] // hkv
    start, lens, widest = s["start"].long(), s["lens"].long(), s["widest"]
    table = s["table"][:, :-1].long()

    def rows(name, per):                                  # [S, Hkv, keys, D]
        c, f = s[name + "c"][table], s[name + "s"][table]
        c = c.transpose(1, 2).reshape(n, hkv, -1, d // 2)
        return _values(c, f.transpose(1, 2).reshape(n, hkv, -1, d // 32), per)

    k = rows("k", 8)
    i = torch.arange(widest, device=DEV)
    new = start[1:] - start[:-1]
    token = (start[:-1, None] + i).clamp(max=len(s["q"]) - 1)                     # [S, widest]
    q = s["q"][token].float().reshape(n, widest, hkv, group, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, widest * group, d)
    x = (q @ k.transpose(2, 3)) * d ** -0.5
    del k
    pos = (lens - new)[:, None] + i                       # [S, widest]
    j = torch.arange(x.shape[3], device=DEV)
    seen = j[None, None] <= pos[..., None]
    if s["window"]:
        seen &= j[None, None] > pos[..., None] - s["window"]
    seen = seen.repeat_interleave(group, 1)[:, None]
    x = torch.where(seen, x, torch.full((), -math.inf, device=DEV))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x = x / x.sum(-1, keepdim=True)
    o = (x @ rows("v", 4)).reshape(n, hkv, widest, group, d).permute(0, 2, 1, 3, 4).reshape(n * widest, hkv * group, d)
    t = torch.arange(len(s["q"]), device=DEV)
    r = torch.searchsorted(start[1:].contiguous(), t, right=True)
    used = r < n
    r = r.clamp(max=n - 1)
    o = o[(r * widest + t - start[r]).clamp(max=len(o) - 1)].to(torch.bfloat16)
    return torch.where(used[:, None, None], o, s["out"])


# --------------------------------------------------------------------------- exact
def exact(case, seed):
    """The same outputs from the operators' definitions in FP64, request by request."""
    if case["op"] == "pages":
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        rot = case["rot"]
        pos = s["positions"].long()
        c, z = s["cos_sin"][pos].double()[:, None].chunk(2, -1)
        outs = []
        for x, w in ((s["q"].double(), s["qw"]), (s["k"].double(), s["kw"])):
            if w is not None:
                x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            at = torch.arange(rot, device=DEV)
            first, second = (at[0::2], at[1::2]) if case["pairs"] else (at[:rot // 2], at[rot // 2:])
            y = x.clone()
            turned = torch.complex(x[..., first], x[..., second]) * torch.complex(c, z)
            y[..., first], y[..., second] = turned.real, turned.imag
            outs.append(y)
        return tuple(outs)
    if case["op"] == "kv":
        return tuple(_exact_mx(s[name].double()) for name in ("k", "v"))
    d, group = case["D"], case["Hq"] // case["Hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    start, lens = s["start"].tolist(), s["lens"].tolist()
    for r in range(case["S"]):
        n, t0 = lens[r], start[r]
        new = start[r + 1] - t0
        pages = s["table"][r, :(n + case["page"] - 1) // case["page"]].long()
        first = max(0, n - new + 1 - case["window"]) if case["window"] else 0
        for h in range(case["Hkv"]):
            k = _exact_row(s["kc"][pages, h].reshape(-1, d // 2)[first:n], s["ks"][pages, h].reshape(-1, d // 32)[first:n], 8)
            v = _exact_row(s["vc"][pages, h].reshape(-1, d // 2)[first:n], s["vs"][pages, h].reshape(-1, d // 32)[first:n], 4)
            q = s["q"][t0:t0 + new, h * group:(h + 1) * group].double()
            x = torch.einsum("igd,jd->igj", q, k) / math.sqrt(d)
            i, j = torch.arange(n - new, n, device=DEV)[:, None], torch.arange(first, n, device=DEV)[None]
            hide = j > i
            if case["window"]:
                hide |= j <= i - case["window"]
            x.masked_fill_(hide[:, None], -math.inf)
            out[t0:t0 + new, h * group:(h + 1) * group] = torch.einsum("igj,jd->igd", torch.softmax(x, -1), v)
    return out


def _exact_row(row, sf, per):
    """FP64 values of cache rows, element by element from where each one stands."""
    d = row.shape[1] * 2
    b = d // 32
    e = torch.arange(d, device=DEV)
    block, part, j = e // 32, e % 32 // per, e % per
    nibble = (part * b + block) * per + j
    code = row.long()[:, nibble // 2] >> (nibble % 2 * 4) & 15
    ex, man = code >> 1 & 3, code & 1
    v = torch.where(ex == 0, man.double() / 2, (1 + man.double() / 2) * torch.pow(2.0, ex.double() - 1))
    return torch.where(code >= 8, -v, v) * torch.pow(2.0, sf.double()[:, block] - 127)


def _exact_mx(x):
    """Values that the 4-bit cache holds for x, in FP64: the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times the block's scale."""
    g = x.reshape(*x.shape[:-1], -1, 32)
    amax = g.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(amax / 6).nan_to_num(neginf=0.0))
    e = torch.where(amax > 6 * torch.pow(2.0, e), e + 1, e)
    e = torch.where(amax <= 6 * torch.pow(2.0, e - 1), e - 1, e)
    scale = torch.where(amax > 0, torch.pow(2.0, e.clamp(-64, 63)), torch.ones_like(amax))
    v = (g / scale).clamp(-6, 6)
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1)
    return (torch.round(v / step) * step * scale).reshape(x.shape)
