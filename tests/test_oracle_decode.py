"""Pins of ``oracle/decode.py`` (CPU): the router, the MoE MLP and the adapters against loops
over single elements, closed forms, and the stated rules for ties, groups and empty slots."""
import math

import numpy as np
import pytest

import decode_cases as D
from oracle import decode as O
from oracle import formats as F
from oracle import fp4 as FP4


def brute_route(row, topk, bias, score, n_group, topk_group, renormalize, scale):
    e = len(row)
    live = [j for j in range(e) if row[j] > -math.inf]
    total = sum(math.exp(row[j]) for j in live)
    s = [0.0] * e
    for j in live:
        s[j] = 1 / (1 + math.exp(-row[j])) if score == "sigmoid" else math.exp(row[j]) / total
    key = {j: (row[j] if bias is None else s[j] + bias[j]) for j in live}
    per = e // n_group
    if n_group > 1:
        gs = []
        for g in range(n_group):
            ks = sorted((key.get(j, -math.inf) for j in range(g * per, (g + 1) * per)), reverse=True)
            gs.append((-(ks[0] + ks[1] if bias is not None and per > 1 else ks[0]), g))
        keep = {g for _, g in sorted(gs)[:topk_group]}
        key = {j: v for j, v in key.items() if j // per in keep}
    chosen = sorted(key, key=lambda j: (-key[j], j))[:topk]
    w = [s[j] for j in chosen]
    if renormalize and sum(w) > 0:
        w = [v / sum(w) for v in w]
    pad = topk - len(chosen)
    return chosen + [-1] * pad, [v * scale for v in w] + [0.0] * pad


@pytest.mark.parametrize("score,bias,n_group,topk_group", [("softmax", False, 1, 1), ("sigmoid", False, 1, 1),
                                                           ("sigmoid", True, 4, 2), ("softmax", False, 4, 3),
                                                           ("softmax", True, 2, 1)])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_against_loops(score, bias, n_group, topk_group, renormalize):
    g = D.rng(5)
    x = np.round(g.standard_normal((40, 12)) * 4) / 4          # many ties
    x[3, 2], x[4, :], x[5, 1:] = -math.inf, -math.inf, -math.inf
    b = np.round(g.standard_normal(12) * 8) / 64 if bias else None
    ids, w = O.route(x, 3, b, score, n_group, topk_group, renormalize, 2.5)
    for i in range(40):
        bi, bw = brute_route(list(x[i]), 3, b, score, n_group, topk_group, renormalize, 2.5)
        assert list(ids[i]) == bi, i
        np.testing.assert_allclose(w[i], bw, rtol=1e-12, atol=1e-15)


def scalar_e4m3(v):
    return float(F.e4m3_to_f64(F.f64_to_e4m3(np.array([v])))[0])


@pytest.mark.parametrize("fp4", [False, True])
def test_moe_mlp_against_loops(fp4):
    c = D.moe_case(7, t=3, h=128, i=128, e=3, topk=2, routed=5, fp4=fp4, base=1)
    c["ids"][0] = [2, 2]                                        # one expert twice: its weights add up
    c["ids"][1] = [-1, 7]                                       # nothing here
    got, bound = O.moe_mlp(c["a"], c["sfa"], c["w13"], c["sf13"], c["w2"], c["sf2"], c["ids"], c["weights"], c["base"], fp4)
    assert np.all(got[1] == 0) and np.all(bound[1] == 0)

    def element(q, sf, n, k):
        if fp4:
            byte = int(q[n, k // 2])
            code = byte >> 4 if k % 2 else byte & 15
            u = int(sf[k // 128, n]) >> (8 * (k % 128 // 32)) & 255
            return FP4.e2m1_value(code) * 2.0 ** (u - 127)
        u = int(sf[k // 512, n // 128]) >> (8 * (k // 128 % 4)) & 255
        return F.e4m3_value(int(q[n, k])) * 2.0 ** (u - 127)

    for t in (0, 2):
        want = np.zeros(128)
        for e in range(3):
            w = sum(float(c["weights"][t, j]) for j in range(2) if c["ids"][t, j] == 1 + e)
            if not any(c["ids"][t, j] == 1 + e for j in range(2)):
                continue
            x = [F.e4m3_value(int(c["a"][t, k])) * 2.0 ** ((int(c["sfa"][0, t]) & 255) - 127) for k in range(128)]
            hid = [sum(x[k] * element(c["w13"][e], c["sf13"][e], n, k) for k in range(128)) for n in range(256)]
            y = [float(np.float32(w * hid[n] / (1 + math.exp(-hid[n])) * hid[128 + n])) for n in range(128)]
            sc = 1.0
            amax = max(abs(v) for v in y)
            sc = 2.0 ** math.ceil(math.log2(amax / 448))
            q = [scalar_e4m3(v / sc) * sc for v in y]
            want += [sum(q[k] * element(c["w2"][e], c["sf2"][e], n, k) for k in range(128)) for n in range(128)]
        np.testing.assert_allclose(got[t], want, rtol=1e-10, atol=1e-12)


def test_moe_bound_is_small_and_holds_for_fp32():
    """The bound is a few times BF16's rounding, and an FP32 evaluation of the definition keeps it."""
    c = D.moe_case(9, t=4, h=256, i=256, e=4, topk=2)
    got, bound = O.moe_mlp(c["a"], c["sfa"], c["w13"], c["sf13"], c["w2"], c["sf2"], c["ids"], c["weights"])
    rms = np.sqrt(np.mean(got ** 2))
    assert np.max(bound) < 0.05 * rms and np.median(bound) < 2e-3 * rms
    x = O.dequant_k_major(c["a"], O.row_scales(c["sfa"], 4, 256)).astype(np.float32)
    out = np.zeros((4, 256), np.float32)
    for e in range(4):
        m13 = O._weights(c["w13"][e], c["sf13"][e], False).astype(np.float32)
        m2 = O._weights(c["w2"][e], c["sf2"][e], False).astype(np.float32)
        for t in range(4):
            for j in range(2):
                if c["ids"][t, j] == e:
                    hid = m13 @ x[t]
                    y = c["weights"][t, j] * (hid[:256] / (1 + np.exp(-hid[:256]))) * hid[256:]
                    q, s = F.quantize_rows(y[None].astype(np.float64))
                    out[t] += m2 @ (F.e4m3_to_f64(q[0]) * np.repeat(F.ue8m0_to_f64(s[0]), 128)).astype(np.float32)
    assert np.all(O.within(out.astype(np.float64), (got, bound), "f32"))


def test_lora_against_loops():
    c = D.lora_case(11, m=3, n=16, k=128, l=2, r=8, none=0.0)
    c["ids"][:] = [1, -1, 0]
    got, _ = O.lora(c["a"], c["sfa"], c["b"], c["sfb"], c["x"], c["la"], c["lb"], c["scaling"], c["ids"])
    for i in range(3):
        sa = 2.0 ** ((int(c["sfa"][0, i]) & 255) - 127)
        sb = 2.0 ** ((int(c["sfb"][0, 0]) & 255) - 127)
        for n in range(16):
            want = sum(F.e4m3_value(int(c["a"][i, k])) * sa * F.e4m3_value(int(c["b"][n, k])) * sb for k in range(128))
            if c["ids"][i] >= 0:
                l = c["ids"][i]
                for r in range(8):
                    v = sum(c["x"][i, k] * c["la"][l, r, k] for k in range(128))
                    want += float(c["scaling"][l]) * v * c["lb"][l, n, r]
            assert abs(got[i, n] - want) < 1e-10


def test_planted_mistakes_are_seen():
    """The checks tell these apart from the definition: gate and up swapped, the routing weight
    dropped, the bias used as a weight, the adapter of another token."""
    c = D.moe_case(13, t=2, h=128, i=128, e=2, topk=1)
    args = [c[k] for k in ("a", "sfa", "w13", "sf13", "w2", "sf2", "ids", "weights")]
    d, bound = O.moe_mlp(*args)
    swapped = [x for x in args]
    swapped[2] = np.concatenate([c["w13"][:, 128:], c["w13"][:, :128]], axis=1)
    swapped[3] = c["sf13"][:, :, [1, 0, 2, 3]]
    assert np.any(np.abs(O.moe_mlp(*swapped)[0] - d) > bound)
    flat = [x for x in args]
    flat[7] = np.ones_like(c["weights"])
    assert np.any(np.abs(O.moe_mlp(*flat)[0] - d) > bound)
    x = D.rng(1).standard_normal((4, 8))
    b = np.linspace(-1, 1, 8)
    assert not np.allclose(O.route(x, 2, b, "sigmoid")[1], O.route(x, 2, None, "sigmoid")[1])
    lc = D.lora_case(17, m=4, n=16, k=128, l=3, r=8, none=0.0)
    largs = [lc[k] for k in ("a", "sfa", "b", "sfb", "x", "la", "lb", "scaling", "ids")]
    d, bound = O.lora(*largs)
    largs[8] = np.roll(lc["ids"] + 1, 1) % 3
    assert np.any(np.abs(O.lora(*largs)[0] - d) > bound)
