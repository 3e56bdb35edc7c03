"""The operators of an MoE decode step, as cases that can be timed and compared.

Three operators, each in a plain form (elementary torch operations in FP32, rounded once) and
as a call of the library (``own``):

* route: router logits -> top-k expert ids and routing weights (``moe_route``);
* moe:   a whole MoE MLP for at most 128 tokens: gate-up, SwiGLU, E4M3 requantisation, down
         projection and weighted sum, with E4M3 or MXFP4 weights (``fp8_moe_mlp``,
         ``fp8_fp4_moe_mlp``);
* lora:  an FP8 projection shared by all requests plus each token's own low-rank adapter
         (``fp8_gemm_nt_lora``).

``exact`` states each of them again in FP64."""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # the router of one new token over 256 experts in 8 groups, with a balancing bias: latency
        {"name": "route_1_256_grouped", "op": "route", "T": 1, "E": 256, "topk": 8, "groups": 8, "keep": 4,
         "score": "sigmoid", "bias": True},
        # the router of a prompt of 8192 tokens, top-6 of 256 (the contiguous benchmark's routing)
        {"name": "route_8192_256", "op": "route", "T": 8192, "E": 256, "topk": 6, "groups": 1, "keep": 1,
         "score": "softmax", "bias": False},
        # one token of a small model: launches and latency
        {"name": "moe_1_small", "op": "moe", "T": 1, "H": 1024, "I": 512, "E": 8, "routed": 8, "topk": 2, "fp4": False},
        # one token, the benchmark's expert size (gate-up N = K = 4096): pure weight streaming
        {"name": "moe_1_4096", "op": "moe", "T": 1, "H": 4096, "I": 2048, "E": 32, "routed": 32, "topk": 6, "fp4": False},
        # a shard of 32 of 256 experts, 16 tokens in flight: most of a token's experts live elsewhere
        {"name": "moe_16_shard_4096", "op": "moe", "T": 16, "H": 4096, "I": 2048, "E": 32, "routed": 256, "topk": 6,
         "fp4": False},
        # the widest layer and the fullest batch: every expert is read once
        {"name": "moe_128_7168", "op": "moe", "T": 128, "H": 7168, "I": 2048, "E": 32, "routed": 32, "topk": 6,
         "fp4": False},
        # an odd batch on MXFP4 weights
        {"name": "moe_37_4096_fp4", "op": "moe", "T": 37, "H": 4096, "I": 2048, "E": 32, "routed": 32, "topk": 6,
         "fp4": True},
        # few tokens on odd sizes (11 and 5 K-groups), MXFP4 weights
        {"name": "moe_3_1408_fp4", "op": "moe", "T": 3, "H": 1408, "I": 640, "E": 60, "routed": 60, "topk": 4, "fp4": True},
        # one request with an adapter
        {"name": "lora_1_4096", "op": "lora", "M": 1, "N": 4096, "K": 4096, "L": 8, "R": 16, "ids": "mixed", "f32": False},
        # a decode batch of 64 requests (the benchmark's decode GEMM), nearly every one with an adapter of its own
        {"name": "lora_64_7168", "op": "lora", "M": 64, "N": 7168, "K": 4096, "L": 128, "R": 16, "ids": "mixed",
         "f32": False},
        # a ragged batch, a last row block of 112 rows, a rank below the tensor cores' step, FP32 out
        {"name": "lora_33_1008_f32", "op": "lora", "M": 33, "N": 1008, "K": 2048, "L": 12, "R": 8, "ids": "mixed",
         "f32": True},
        # a prefill step: prompts of a few requests one after another, high-rank adapters
        {"name": "lora_2048_segments", "op": "lora", "M": 2048, "N": 4096, "K": 4096, "L": 16, "R": 64, "ids": "segments",
         "f32": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "lora", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        per = _log_int(rng, 4, 512 // groups)
        e = groups * per
        keep = rng.randint(1, groups)
        topk = rng.randint(1, min(16, keep * per))
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": _log_int(rng, 1, 8192), "E": e, "topk": topk, "groups": groups, "keep": keep,
                "score": score, "bias": score == "sigmoid" and rng.random() < 0.6}
    if op == "moe":
        h, i = 128 * _log_int(rng, 4, 56), 128 * _log_int(rng, 2, 16)
        e = _log_int(rng, 4, 64)
        while e * h * i > 32 * 7168 * 2048:
            e -= 1
        routed = e * rng.choice([1, 1, 1, 2, 8])
        return {"op": op, "T": _log_int(rng, 1, 128), "H": h, "I": i, "E": e, "routed": routed,
                "topk": rng.randint(1, min(8, routed)), "fp4": rng.random() < 0.5}
    m = _log_int(rng, 1, 2048)
    return {"op": op, "M": m, "N": 16 * _log_int(rng, 16, 448), "K": 128 * _log_int(rng, 4, 32),
            "L": _log_int(rng, 1, 128), "R": rng.choice([8, 16, 24, 32, 64, 128]) if m <= 256 else rng.choice([8, 16, 32, 64]),
            "ids": "segments" if m > 256 else "mixed", "f32": rng.random() < 0.3}


def _distinct(n, p, tries):
    """Expected number of n items that are named when each of `tries` draws names each with probability p."""
    return n * (1.0 - (1.0 - p) ** tries)


def work(case):
    if case["op"] == "route":
        t, e, k = case["T"], case["E"], case["topk"]
        return {"bytes": t * e * 4 + (e * 4 if case["bias"] else 0) + t * k * 8, "flops": 8 * t * e}
    if case["op"] == "moe":
        t, h, i, e, k = (case[n] for n in ("T", "H", "I", "E", "topk"))
        p = min(1.0, k / case["routed"])
        per = 3 * h * i * (0.5 + 1 / 32 if case["fp4"] else 1.0 + 1 / 16384)
        return {"bytes": _distinct(e, p, t) * per + t * (h * (1 + 1 / 128) + k * 8 + h * 2), "flops": 6 * t * p * e * h * i}
    m, n, k, l, r = (case[x] for x in ("M", "N", "K", "L", "R"))
    with_adapter = 0.9 * m
    used = _distinct(l, 0.9 / l, m) if case["ids"] == "mixed" else min(l, _segments(m))
    return {"bytes": n * k * (1 + 1 / 16384) + m * k * (1 + 1 / 128 + 2) + used * r * (k + n) * 2 + m * n * (4 if case["f32"] else 2) + m * 4,
            "flops": 2 * m * n * k + 2 * with_adapter * r * (k + n)}


def _segments(m):
    return max(1, round(m / 384))


# ------------------------------------------------------------------------- prepare
def _groups_exponent(amax):
    """Smallest e with amax <= 448 * 2^e (0 for an empty group)."""
    fr, ex = torch.frexp(amax)
    e = torch.where(fr <= 0.875, ex - 9, ex - 8)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _pack(byte, ld):
    """Scale bytes [.., K-group, MN] -> packed words [.., ceil(K-groups / 4), ld]."""
    kg, mn = byte.shape[-2:]
    full = torch.zeros(*byte.shape[:-2], (kg + 3) // 4 * 4, ld, dtype=torch.uint8, device=byte.device)
    full[..., :kg, :mn] = byte
    full = full.reshape(*byte.shape[:-2], (kg + 3) // 4, 4, ld).transpose(-1, -2).contiguous()
    return full.view(torch.int32).squeeze(-1)


def _pow2(e):
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _align4(x):
    return (x + 3) // 4 * 4


def _e4m3_rows(x):
    """Rows [M, K] -> E4M3 codes and packed scales of their 1x128 groups."""
    m, k = x.shape
    g = x.reshape(m, k // 128, 128)
    e = _groups_exponent(g.abs().amax(-1))
    q = (g * _pow2(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(m, k)
    return q, _pack((e + 127).to(torch.uint8).T.contiguous(), _align4(m))


def _e4m3_blocks(w):
    """Weights [N, K] -> E4M3 codes and packed scales of their 128x128 blocks."""
    n, k = w.shape
    nb = (n + 127) // 128
    pad = torch.zeros(nb * 128, k, device=w.device)
    pad[:n] = w
    g = pad.reshape(nb, 128, k // 128, 128)
    e = _groups_exponent(g.abs().amax((1, 3)))
    q = (g * _pow2(-e)[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(nb * 128, k)[:n]
    return q.contiguous(), _pack((e + 127).to(torch.uint8).T.contiguous(), _align4(nb))


def _mxfp4(w):
    """Weights [N, K] -> packed E2M1 codes and the scale words of their 1x32 blocks."""
    n, k = w.shape
    g = w.reshape(n, k // 32, 32)
    amax = g.abs().amax(-1)
    fr, ex = torch.frexp(amax)
    e = torch.where(amax > 0, torch.where(fr <= 0.75, ex - 3, ex - 2), torch.zeros_like(ex))
    v = (g * _pow2(-e)[..., None]).reshape(n, k)
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for mid, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= mid if up else a > mid).to(torch.uint8)          # ties to the even code
    code |= (v < 0).to(torch.uint8) << 3
    sf = torch.zeros(k // 128, _align4(n), 4, dtype=torch.uint8, device=w.device)
    sf[:, :n] = (e + 127).to(torch.uint8).reshape(n, k // 128, 4).transpose(0, 1)
    return (code[:, 0::2] | code[:, 1::2] << 4).contiguous(), sf.view(torch.int32).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 7919 + 13)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=DEV) * std

    s = dict(case)
    if case["op"] == "route":
        t, e, k = case["T"], case["E"], case["topk"]
        s["logits"] = normal(t, e, std=2.0)
        s["b"] = normal(e, std=0.1) if case["bias"] else None
        s["ids"] = torch.empty(t, k, dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(t, k, device=DEV)
    elif case["op"] == "moe":
        t, h, i, e, k, routed = (case[n] for n in ("T", "H", "I", "E", "topk", "routed"))
        s["a"], s["sfa"] = _e4m3_rows(normal(t, h))
        quant = _mxfp4 if case["fp4"] else _e4m3_blocks
        s["w13"], s["sf13"], s["w2"], s["sf2"] = (
            torch.stack(x) for x in zip(*(quant(normal(2 * i, h, std=0.02)) + quant(normal(h, i, std=0.02)) for _ in range(e))))
        logits = normal(t, routed)
        top, ids = logits.topk(k, dim=1)
        s["ids"] = ids.to(torch.int32)
        s["weights"] = torch.softmax(top, 1)
        s["base"] = (routed - e) // 2                     # this shard holds experts base .. base + E - 1
        s["out"] = torch.empty(t, h, dtype=torch.bfloat16, device=DEV)
    else:
        m, n, k, l, r = (case[x] for x in ("M", "N", "K", "L", "R"))
        x = normal(m, k)
        s["x"] = x.to(torch.bfloat16)
        s["a"], s["sfa"] = _e4m3_rows(s["x"].float())
        s["w"], s["sfw"] = _e4m3_blocks(normal(n, k, std=0.02))
        s["lora_a"] = normal(l, r, k, std=k ** -0.5).to(torch.bfloat16)
        s["lora_b"] = normal(l, n, r, std=0.3 * r ** -0.5).to(torch.bfloat16)
        s["scaling"] = 0.5 + 1.5 * torch.rand(l, generator=gen, device=DEV)
        if case["ids"] == "mixed":
            ids = torch.randint(0, l, (m,), generator=gen, device=DEV)
            none = torch.rand(m, generator=gen, device=DEV) < 0.1
        else:                                            # prompts one after another, each with one adapter or none
            cuts = torch.randint(0, m, (_segments(m) - 1,), generator=gen, device=DEV).sort().values
            seg = torch.searchsorted(cuts, torch.arange(m, device=DEV), right=True)
            ids = torch.randint(0, l, (_segments(m),), generator=gen, device=DEV)[seg]
            none = (torch.rand(_segments(m), generator=gen, device=DEV) < 0.1)[seg]
        s["ids"] = torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32)
        s["out"] = torch.empty(m, n, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
    if own and case["op"] != "route":                    # the workspace that a program keeps beside its weights
        import moe_fp8_e4m3_gb300 as fg
        s["workspace"] = (fg.moe_mlp_workspace(case["T"], case["H"], case["I"], case["E"]) if case["op"] == "moe" else
                          fg.lora_workspace(case["M"], case["N"], case["K"], case["R"]))
    return s


# ----------------------------------------------------------------------------- run
def run(s):
    if own:
        import moe_fp8_e4m3_gb300 as fg
        if s["op"] == "route":
            fg.moe_route(s["logits"], s["ids"], s["weights"], bias=s["b"], score=s["score"], n_group=s["groups"],
                         topk_group=s["keep"])
            return s["ids"], s["weights"]
        if s["op"] == "moe":
            call = fg.fp8_fp4_moe_mlp if s["fp4"] else fg.fp8_moe_mlp
            call(s["a"], s["sfa"], s["w13"], s["sf13"], s["w2"], s["sf2"], s["ids"], s["weights"], s["out"], s["workspace"],
                 expert_base=s["base"])
            return s["out"]
        fg.fp8_gemm_nt_lora(s["a"], s["sfa"], s["w"], s["sfw"], s["x"], s["lora_a"], s["lora_b"], s["scaling"], s["ids"],
                            s["out"], s["workspace"])
        return s["out"]
    return {"route": _route_plain, "moe": _moe_plain, "lora": _lora_plain}[s["op"]](s)


def _route_plain(s):
    x = s["logits"]
    t, e = x.shape
    if s["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-x))
    key = x if s["b"] is None else p + s["b"]
    if s["groups"] > 1:
        by = key.reshape(t, s["groups"], -1).sort(dim=2, descending=True).values
        top = by[..., 0] if s["b"] is None or by.shape[2] == 1 else by[..., 0] + by[..., 1]
        best = top.sort(dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        keep = torch.zeros(t, s["groups"], dtype=torch.bool, device=x.device).scatter_(1, best, True)
        key = torch.where(keep.repeat_interleave(e // s["groups"], 1), key, torch.full_like(key, -math.inf))
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    w = p.gather(1, ids)
    return ids.to(torch.int32), w / w.sum(1, keepdim=True)


def _scales(sf, mn, kg):
    """Packed words [.., words, ld] -> FP32 scales [.., MN, K-group]."""
    b = sf.unsqueeze(-1).view(torch.uint8)[..., :mn, :]                     # [.., words, MN, 4]
    b = b.transpose(-2, -3).reshape(*sf.shape[:-2], mn, -1)[..., :kg]
    return (b.to(torch.int32) << 23).view(torch.float32)


def _rows_f32(q, sf):
    m, k = q.shape
    v = q.view(torch.float8_e4m3fn).float().reshape(m, k // 128, 128)
    return (v * _scales(sf, m, k // 128)[..., None]).reshape(m, k)


def _blocks_f32(q, sf):
    *g, n, k = q.shape
    sc = _scales(sf, (n + 127) // 128, k // 128).repeat_interleave(128, -2)[..., :n, :]
    return (q.view(torch.float8_e4m3fn).float().reshape(*g, n, k // 128, 128) * sc[..., None]).reshape(*g, n, k)


def _fp4_f32(q, sf):
    *g, n, half = q.shape
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=q.device)
    table = torch.cat([table, -table])
    v = torch.stack([table[(q & 15).int()], table[(q >> 4).int()]], -1).reshape(*g, n, half // 16, 32)
    return (v * _scales(sf, n, half // 16)[..., None]).reshape(*g, n, 2 * half)


def _requantised(y):
    """E4M3 values (times their scales) of y's 1x128 groups along its last axis."""
    g = y.reshape(*y.shape[:-1], -1, 128)
    e = _groups_exponent(g.abs().amax(-1))[..., None]
    return ((g * _pow2(-e)).to(torch.float8_e4m3fn).float() * _pow2(e)).reshape(y.shape)


def _moe_plain(s):
    t, h, i, e, k = (s[n] for n in ("T", "H", "I", "E", "topk"))
    decode = _fp4_f32 if s["fp4"] else _blocks_f32
    x = _rows_f32(s["a"], s["sfa"])
    ids = s["ids"].long() - s["base"]
    here = (ids >= 0) & (ids < e)
    w = torch.where(here, s["weights"], torch.zeros_like(s["weights"]))
    ids = torch.where(here, ids, torch.zeros_like(ids))
    if t * k < e:                                        # few pairs: each reads its own expert
        sel = ids.reshape(-1)
        w13, w2 = decode(s["w13"][sel], s["sf13"][sel]), decode(s["w2"][sel], s["sf2"][sel])
        xs, wy = x.repeat_interleave(k, 0)[:, None, :], w.reshape(-1, 1, 1)
    else:                                                # many: every expert once, on every token
        w13, w2 = decode(s["w13"], s["sf13"]), decode(s["w2"], s["sf2"])
        xs, wy = x[None], torch.zeros(t, e, device=x.device).scatter_add_(1, ids, w).T[..., None]
    hid = xs @ w13.transpose(1, 2)
    gate, up = hid[..., :i], hid[..., i:]
    y = _requantised(wy * (gate / (1.0 + torch.exp(-gate))) * up)
    o = y @ w2.transpose(1, 2)
    o = o.reshape(t, k, h).sum(1) if t * k < e else o.sum(0)
    return o.to(torch.bfloat16)


def _lora_plain(s):
    m, n, l, r = (s[x] for x in ("M", "N", "L", "R"))
    base = _rows_f32(s["a"], s["sfa"]) @ _blocks_f32(s["w"], s["sfw"]).T
    ids = s["ids"].long().clamp(min=0)
    scale = torch.where(s["ids"] >= 0, s["scaling"][ids], torch.zeros(m, device=base.device))
    x = s["x"].float()
    if m < l:                                            # each token reads its own adapter
        v = (s["lora_a"][ids].float() @ x[:, :, None]) * scale[:, None, None]
        delta = (s["lora_b"][ids].float() @ v)[..., 0]
    else:                                                # all adapters at once, the others' parts masked
        v = (x @ s["lora_a"].float().reshape(l * r, -1).T).reshape(m, l, r)
        mine = (torch.arange(l, device=ids.device)[None] == ids[:, None]).float() * scale[:, None]
        delta = (v * mine[..., None]).reshape(m, l * r) @ s["lora_b"].float().transpose(1, 2).reshape(l * r, n)
    return (base + delta).to(s["out"].dtype)


# --------------------------------------------------------------------------- exact
def exact(case, seed):
    """The same outputs from the operators' definitions in FP64, expert by expert and adapter by adapter."""
    s = prepare(case, seed)
    if case["op"] == "route":
        x = s["logits"].double()
        p = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        key = x.clone() if s["b"] is None else p + s["b"].double()
        per = case["E"] // case["groups"]
        if case["groups"] > 1:
            two = 1 if s["b"] is None or per == 1 else 2
            score = key.reshape(-1, case["groups"], per).topk(two, 2).values.sum(2)
            out = score.topk(case["groups"] - case["keep"], 1, largest=False).indices
            for j in range(out.shape[1]):
                group = torch.arange(case["E"], device=DEV)[None] // per
                key[group == out[:, j:j + 1]] = -math.inf
        ids = key.topk(case["topk"], 1).indices
        w = p.gather(1, ids)
        return ids.to(torch.int32), w / w.sum(1, keepdim=True)
    if case["op"] == "moe":
        t, h, i, e = (case[n] for n in ("T", "H", "I", "E"))
        x = _exact_decode(s["a"], s["sfa"], 1, 128)
        out = torch.zeros(t, h, dtype=torch.float64, device=DEV)
        for j in range(e):
            hit = s["ids"] == s["base"] + j
            rows = hit.any(1).nonzero()[:, 0]
            if not len(rows):
                continue
            w = (s["weights"].double() * hit).sum(1)[rows]
            how = (1, 32) if case["fp4"] else (128, 128)
            gate_up = x[rows] @ _exact_decode(s["w13"][j], s["sf13"][j], *how).T
            y = torch.sigmoid(gate_up[:, :i]) * gate_up[:, :i] * gate_up[:, i:] * w[:, None]
            out.index_add_(0, rows, _exact_e4m3(y) @ _exact_decode(s["w2"][j], s["sf2"][j], *how).T)
        return out
    x = s["x"].double()
    out = _exact_decode(s["a"], s["sfa"], 1, 128) @ _exact_decode(s["w"], s["sfw"], 128, 128).T
    for j in range(case["L"]):
        rows = (s["ids"] == j).nonzero()[:, 0]
        if len(rows):
            v = x[rows] @ s["lora_a"][j].double().T
            out.index_add_(0, rows, s["scaling"][j].double() * (v @ s["lora_b"][j].double().T))
    return out


def _exact_decode(q, sf, rows, cols):
    """FP64 values of codes with one scale per rows x cols block (cols == 32: packed E2M1)."""
    def value(code, exp_bits, man_bits, bias):
        man, ex = code & ((1 << man_bits) - 1), code >> man_bits & ((1 << exp_bits) - 1)
        v = man * 2.0 ** (1 - bias - man_bits) if ex == 0 else (1 + man / (1 << man_bits)) * 2.0 ** (ex - bias)
        return -v if code >> (man_bits + exp_bits) & 1 else v
    if cols == 32:
        lut = torch.tensor([value(c, 2, 1, 1) for c in range(16)], dtype=torch.float64, device=q.device)
        n, half = q.shape
        v = torch.empty(n, 2 * half, dtype=torch.float64, device=q.device)
        v[:, 0::2], v[:, 1::2] = lut[q.long() % 16], lut[q.long() // 16]
    else:
        lut = torch.tensor([value(c, 4, 3, 7) for c in range(256)], dtype=torch.float64, device=q.device)
        v = lut[q.long()]
    n, k = v.shape
    block, group = torch.arange(n, device=q.device) // rows, torch.arange(k // cols, device=q.device)
    byte = sf.long()[group // 4][:, block] >> (8 * (group % 4))[:, None] & 255
    return (v.reshape(n, k // cols, cols) * torch.pow(2.0, byte.T.double() - 127)[..., None]).reshape(n, k)


def _exact_e4m3(y):
    """y rounded to E4M3 times the power of two of each 1x128 group, in FP64."""
    g = y.reshape(y.shape[0], -1, 128)
    amax = g.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(amax / 448).nan_to_num(neginf=0.0))
    e = torch.where(amax > 448 * torch.pow(2.0, e), e + 1, e)
    e = torch.where(amax <= 448 * torch.pow(2.0, e - 1), e - 1, e)
    scale = torch.where(amax > 0, torch.pow(2.0, e), torch.ones_like(e))
    v = g / scale
    step = torch.pow(2.0, torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step * scale).reshape(y.shape)
