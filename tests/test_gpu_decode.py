"""GPU parity of the MoE decode operators (router, whole MoE MLP, projection with per-token
adapters) against the FP64 oracle, whose bounds are derived from the operands
(``oracle/decode.py``); ids, untouched memory and zero rows are compared exactly."""
import numpy as np
import pytest

import decode_cases as D
from oracle import decode as O

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_fp8_e4m3_gb300 as lib
    return lib


def _ok(fg):
    st, detail = fg.get_device_error()
    assert st == 0, (st, hex(detail))


# ------------------------------------------------------------------------ router
def run_route(fg, x, topk, bias=None, **kw):
    from gpu_util import dev
    t = x.shape[0]
    ids = torch.full((t + 2, topk), -77, dtype=torch.int32, device="cuda")
    w = torch.full((t + 2, topk), -77.0, device="cuda")
    fg.moe_route(dev(x.astype(np.float32)), ids[1:t + 1], w[1:t + 1], bias=None if bias is None else dev(bias.astype(np.float32)),
                 **kw)
    _ok(fg)
    assert torch.all(ids[0] == -77) and torch.all(ids[-1] == -77) and torch.all(w[0] == -77) and torch.all(w[-1] == -77)
    return ids[1:t + 1].cpu().numpy(), w[1:t + 1].cpu().numpy()


# FP32 scores: exp and the quotients are within a few units (2^-24) of the exact value, the sums
# of E <= 1024 terms by shuffles within 15 more; weights agree to 64 * 2^-24 of themselves
ROUTE_RTOL = 64 * 2.0 ** -24


@pytest.mark.parametrize("t,e,topk", [(1, 1, 1), (1, 8, 8), (5, 33, 3), (130, 60, 4), (7, 256, 8), (4, 512, 16),
                                      (3, 1024, 32)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_choice_and_weights(fg, t, e, topk, score):
    g = D.rng(100 + e + t)
    # distinct multiples of 1/64 per row: no two keys are near each other
    x = np.stack([g.permutation(e) for _ in range(t)]) / 64.0 - e / 128.0
    for kw in (dict(), dict(renormalize=False, scale=2.5)):
        ids, w = run_route(fg, x, topk, score=score, **kw)
        rid, rw = O.route(x, topk, score=score, **kw)
        assert np.array_equal(ids, rid)
        np.testing.assert_allclose(w, rw, rtol=ROUTE_RTOL)


@pytest.mark.parametrize("t,e,topk,groups,keep", [(9, 64, 6, 8, 3), (1, 256, 8, 8, 4), (33, 60, 4, 4, 1), (5, 8, 2, 8, 2),
                                                  (3, 1024, 16, 32, 5)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_groups_and_bias(fg, t, e, topk, groups, keep, biased):
    g = D.rng(e + groups)
    x = g.standard_normal((t, e)).astype(np.float32).astype(np.float64)
    bias = (g.integers(-64, 65, e) / 256.0) if biased else None
    ids, w = run_route(fg, x, topk, bias, score="sigmoid", n_group=groups, topk_group=keep)
    s, key = O.route_keys(x, bias, "sigmoid", groups, keep)
    rid, rw = O.route(x, topk, bias, "sigmoid", groups, keep)
    # FP32 keys (|key| < 2) are within 8 units of 2^-23: where the oracle's own order is clearer
    # than that, the ids are the oracle's
    srt = -np.sort(-key, axis=1)[:, :topk + 1]
    with np.errstate(invalid="ignore"):
        clear = np.all(-np.diff(srt, axis=1) > 2.0 ** -19, axis=1)
    assert clear.mean() > 0.5
    assert np.array_equal(ids[clear], rid[clear])
    np.testing.assert_allclose(w[clear], rw[clear], rtol=ROUTE_RTOL)


def test_route_ties_and_masked_experts(fg):
    x = np.zeros((6, 40))
    x[1, 7] = x[1, 33] = 1.0
    x[2, :] = -np.inf
    x[3, :] = -np.inf
    x[3, [39, 4]] = 2.0, 2.0
    x[4, :] = np.nan
    x[4, 12] = -3.0
    x[5, ::2] = np.nan
    x[5, 1::4] = -np.inf
    for score in ("softmax", "sigmoid"):
        ids, w = run_route(fg, x, 3, score=score)
        rid, rw = O.route(x, 3, score=score)
        assert np.array_equal(ids, rid)
        np.testing.assert_allclose(w, rw, rtol=ROUTE_RTOL, atol=0)
    assert list(ids[0]) == [0, 1, 2] and list(ids[2]) == [-1, -1, -1] and list(ids[3]) == [4, 39, -1]
    ids, w = run_route(fg, np.array([[-0.0, 0.0, -0.0, 0.0]]), 4)     # -0 and 0 tie
    assert list(ids[0]) == [0, 1, 2, 3]


# ----------------------------------------------------------------------- MoE MLP
def moe_inputs(c):
    from gpu_util import dev
    return [dev(c[k]) for k in ("a", "sfa", "w13", "sf13", "w2", "sf2", "ids", "weights")]


def run_moe(fg, c, out="bf16", ws=None, args=None, stream=None):
    from gpu_util import GuardedOut
    t, h = c["a"].shape
    e, i = c["w13"].shape[0], c["w13"].shape[1] // 2
    args = args or moe_inputs(c)
    ws = fg.moe_mlp_workspace(t, h, i, e) if ws is None else ws
    o = GuardedOut(t, h, out)
    (fg.fp8_fp4_moe_mlp if c["fp4"] else fg.fp8_moe_mlp)(*args, o.tensor, ws, expert_base=c["base"], stream=stream)
    _ok(fg)
    o.check_guards()
    return o.values()


def moe_ref(c):
    return O.moe_mlp(*[c[k] for k in ("a", "sfa", "w13", "sf13", "w2", "sf2", "ids", "weights")], expert_base=c["base"],
                     fp4=c["fp4"])


def check(got, ref, out="bf16"):
    ok = O.within(got, ref, out)
    at = np.unravel_index(int(np.argmin(ok)), ok.shape)
    assert ok.all(), f"{(~ok).sum()} of {ok.size} outside; {at}: got {got[at]}, {ref[0][at]} within {ref[1][at]}"


MOE = [  # T, H, I, E, topk, routed, base
    (1, 128, 128, 1, 1, 1, 0), (1, 384, 256, 8, 2, 8, 0), (2, 640, 128, 5, 3, 5, 0), (7, 1152, 640, 12, 4, 48, 12),
    (16, 256, 384, 8, 8, 8, 0), (17, 256, 256, 8, 2, 16, 4), (33, 512, 128, 40, 5, 40, 0), (64, 128, 512, 3, 1, 3, 0),
    (65, 384, 128, 8, 2, 8, 0), (128, 256, 256, 6, 2, 6, 0),
]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,h,i,e,topk,routed,base", MOE)
def test_moe_mlp(fg, fp4, t, h, i, e, topk, routed, base):
    c = D.moe_case(t + h + i, t, h, i, e, topk, routed, fp4, base)
    for out in ("bf16", "f32"):
        check(run_moe(fg, c, out), moe_ref(c), out)


def test_moe_ids_masks_and_duplicates(fg):
    """Ids of other shards, -1, an expert named twice, a zero and a negative routing weight, tokens
    without any expert (their rows hold NaN codes and are exact zeros in D)."""
    c = D.moe_case(3, t=20, h=256, i=256, e=6, topk=3, routed=6, base=10)
    g = D.rng(4)
    c["ids"] += 10
    c["ids"][0] = [10, 10, 11]
    c["ids"][1] = [-1, -1, -1]
    c["ids"][2] = [9, 16, 2 ** 31 - 1]
    c["ids"][3] = [-2 ** 31, -5, 12]
    c["weights"][4] = 0.0
    c["weights"][5, 0] = -0.7
    c["a"][1] = 0x7F
    c["a"][2] = g.integers(0, 256, 256)
    got = run_moe(fg, c)
    clean = dict(c, a=c["a"].copy())
    clean["a"][1:3] = 0
    check(got, moe_ref(clean))
    assert np.all(got[1] == 0) and np.all(got[2] == 0) and np.all(got[4] == 0)


@pytest.mark.parametrize("t", [1, 40])
def test_moe_no_expert_here(fg, t):
    c = D.moe_case(5, t, 256, 128, 4, 2, base=100)
    for out in ("bf16", "f32"):
        assert np.all(run_moe(fg, c, out) == 0)


def test_moe_non_finite_rows_stay_apart(fg):
    c = D.moe_case(6, t=9, h=256, i=128, e=4, topk=2)
    c["a"][3, 17] = 0x7F                    # NaN code in token 3
    c["weights"][5, 1] = np.nan
    c["weights"][6, 0] = np.inf
    got = run_moe(fg, c)
    assert np.all(np.isnan(got[3])) and np.all(np.isnan(got[5])) and np.all(np.isnan(got[6]))
    rest = [0, 1, 2, 4, 7, 8]
    ok = dict(c, a=c["a"].copy(), weights=np.nan_to_num(c["weights"], nan=0.0, posinf=0.0))
    ok["a"][3] = 0
    d, bound = moe_ref(ok)
    check(got[rest], (d[rest], bound[rest]))


@pytest.mark.parametrize("sms", [1, 3, 37])
@pytest.mark.parametrize("fp4", [False, True])
def test_moe_any_number_of_shares(fg, sms, fp4):
    """The work is cut into as many shares as there are SMs: cuts inside tiles, between experts,
    several tiles in a share, one share in all."""
    c = D.moe_case(8, t=19, h=640, i=384, e=5, topk=2, fp4=fp4)
    ref = moe_ref(c)
    try:
        fg.set_num_sms(sms)
        check(run_moe(fg, c), ref)
    finally:
        fg.set_num_sms(0)


def test_moe_same_bits_again_and_workspace_reuse(fg):
    """Results do not depend on which share arrives last, on what an earlier call (with another
    batch) left in the workspace, on the stream, or on programmatic launches."""
    big, small = D.moe_case(1, 16, 1024, 512, 8, 4), D.moe_case(2, 3, 1024, 512, 8, 2)
    ws = fg.moe_mlp_workspace(16, 1024, 512, 8)
    args = moe_inputs(big)
    first = run_moe(fg, big, ws=ws, args=args)
    check(first, moe_ref(big))
    for _ in range(20):
        assert np.array_equal(run_moe(fg, big, ws=ws, args=args), first)
    check(run_moe(fg, small, ws=ws), moe_ref(small))
    ws.view(torch.uint8)[fg.lib.fg_moe_mlp_workspace(1, 1024, 512, 8) // 2:].fill_(0xFF)     # past the counters
    assert np.array_equal(run_moe(fg, big, ws=ws, args=args), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    from gpu_util import GuardedOut
    o = GuardedOut(16, 1024, "bf16")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fg.fp8_moe_mlp(*args, o.tensor, ws)
    torch.cuda.synchronize()
    assert np.array_equal(o.values(), first)
    fg.set_pdl(False)
    try:
        assert np.array_equal(run_moe(fg, big, ws=ws, args=args), first)
    finally:
        fg.set_pdl(True)


def test_one_workspace_for_many_sizes(fg):
    """A workspace that served one size (or operator) serves any other that fits."""
    cases = [D.moe_case(51, 1, 256, 384, 60, 4), D.moe_case(52, 70, 256, 384, 60, 2), D.moe_case(53, 16, 512, 128, 3, 2),
             D.lora_case(54, 70, 272, 256, 12, 24), D.moe_case(55, 2, 512, 256, 9, 3, fp4=True), D.lora_case(56, 5, 1008, 512, 3, 64)]
    ws = torch.zeros(128 << 20, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for c in cases:
            if "w13" in c:
                check(run_moe(fg, c, ws=ws), moe_ref(c))
            else:
                check(run_lora(fg, c, ws=ws), lora_ref(c))


def test_moe_refusals(fg):
    c = D.moe_case(1, 4, 256, 128, 2, 1)
    args = moe_inputs(c)
    ws = fg.moe_mlp_workspace(4, 256, 128, 2)
    d = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        fg.fp8_moe_mlp(*args, d[:3], ws)
    with pytest.raises(ValueError):
        fg.fp8_moe_mlp(*args, d, ws[:1000])
    with pytest.raises(TypeError):
        fg.fp8_moe_mlp(*args, d.half(), ws)
    with pytest.raises(TypeError):
        fg.fp8_moe_mlp(*args[:6], args[6].long(), args[7], d, ws)
    with pytest.raises(fg.FgError):
        fg.moe_mlp_workspace(200, 256, 128, 2)


# -------------------------------------------------------------------------- LoRA
def lora_inputs(c):
    from gpu_util import dev
    bf = lambda bits: dev(bits.view(np.int16)).view(torch.bfloat16)  # noqa: E731
    return [dev(c["a"]), dev(c["sfa"]), dev(c["b"]), dev(c["sfb"]), bf(c["x_bits"]), bf(c["la_bits"]), bf(c["lb_bits"]),
            dev(c["scaling"]), dev(c["ids"])]


def run_lora(fg, c, out="bf16", ws=None, args=None, status=0):
    from gpu_util import GuardedOut
    m, k = c["a"].shape
    n, r = c["b"].shape[0], c["la"].shape[1]
    ws = fg.lora_workspace(m, n, k, r) if ws is None else ws
    o = GuardedOut(m, n, out)
    fg.fp8_gemm_nt_lora(*(args or lora_inputs(c)), o.tensor, ws)
    assert fg.get_device_error()[0] == status
    o.check_guards()
    return o.values()


def lora_ref(c, out="bf16"):
    return O.lora(*[c[k] for k in ("a", "sfa", "b", "sfb", "x", "la", "lb", "scaling", "ids")], out=out)


LORA = [  # M, N, K, L, R
    (1, 16, 128, 1, 8), (1, 272, 512, 5, 16), (3, 48, 128, 3, 24), (16, 1008, 256, 20, 16), (17, 256, 384, 2, 64),
    (33, 528, 256, 40, 32), (64, 256, 512, 130, 16), (65, 144, 128, 9, 72), (128, 512, 256, 128, 8), (100, 256, 128, 7, 128),
    (129, 272, 256, 4, 40), (300, 512, 128, 33, 16),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,l,r", LORA)
def test_lora(fg, m, n, k, l, r, out):
    c = D.lora_case(m + n + r, m, n, k, l, r)
    check(run_lora(fg, c, out), lora_ref(c, out), out)


@pytest.mark.parametrize("kind", ["none", "one", "last"])
@pytest.mark.parametrize("m", [5, 150])
def test_lora_adapter_patterns(fg, kind, m):
    """No adapter in the whole call, one adapter for all, adapters in the last token tile only."""
    c = D.lora_case(21, m, 272, 256, 4, 16)
    c["ids"][:] = 3 if kind == "one" else -1
    if kind == "last":
        c["ids"][-1] = 2
    check(run_lora(fg, c), lora_ref(c))


def test_lora_without_adapters_is_the_projection(fg):
    from gpu_util import GuardedOut
    c = D.lora_case(22, 40, 272, 512, 4, 16)
    c["ids"][:] = -1
    got = run_lora(fg, c, "f32")
    o = GuardedOut(40, 272, "f32")
    fg.fp8_gemm_nt(*lora_inputs(c)[:4], o.tensor)
    _ok(fg)
    check(o.values(), lora_ref(c, "f32"), "f32")
    check(got, lora_ref(c, "f32"), "f32")


def test_lora_bad_ids_and_non_finite_tokens(fg):
    """An id >= L is reported and treated as no adapter; ids below 0 are no adapter; a NaN in x
    reaches its own token only, and only through an adapter."""
    c = D.lora_case(23, 20, 272, 256, 4, 16, none=0.0)
    c["ids"][4] = 4
    c["ids"][5] = -2 ** 31
    got = run_lora(fg, c, status=fg.FG_ERR_DEVICE_CONTRACT)
    check(got, lora_ref(c))
    c["ids"][4] = -1
    c["x_bits"][[4, 7], 3] = 0x7FC0
    got = run_lora(fg, c)
    ref = lora_ref(c)
    assert np.all(np.isnan(got[7]))
    rest = [i for i in range(20) if i != 7]
    check(got[rest], (ref[0][rest], ref[1][rest]))


@pytest.mark.parametrize("sms", [1, 5, 64])
def test_lora_any_number_of_shares(fg, sms):
    c = D.lora_case(24, 140, 528, 512, 30, 32)
    ref = lora_ref(c)
    try:
        fg.set_num_sms(sms)
        check(run_lora(fg, c), ref)
    finally:
        fg.set_num_sms(0)


def test_lora_same_bits_again_and_workspace_reuse(fg):
    c, d = D.lora_case(25, 48, 784, 1024, 30, 16), D.lora_case(26, 40, 784, 1024, 9, 16)
    ws = fg.lora_workspace(48, 784, 1024, 16)
    args = lora_inputs(c)
    first = run_lora(fg, c, ws=ws, args=args)
    for _ in range(20):
        assert np.array_equal(run_lora(fg, c, ws=ws, args=args), first)
    check(run_lora(fg, d, ws=ws), lora_ref(d))
    check(run_lora(fg, d, "f32", ws=ws), lora_ref(d, "f32"), "f32")
    assert np.array_equal(run_lora(fg, c, ws=ws, args=args), first)


def test_lora_refusals(fg):
    c = D.lora_case(27, 4, 256, 128, 2, 8)
    args = lora_inputs(c)
    ws = fg.lora_workspace(4, 256, 128, 8)
    d = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        fg.fp8_gemm_nt_lora(*args, d[:3], ws)
    with pytest.raises(TypeError):
        fg.fp8_gemm_nt_lora(*args[:4], args[4].float(), *args[5:], d, ws)
    with pytest.raises(ValueError):
        fg.fp8_gemm_nt_lora(*args, d, ws[:256])


# ------------------------------------------------------------------- as a step
def test_decode_step_in_a_graph(fg):
    """Projection with adapters -> quantise -> router -> MoE MLP, captured once in a CUDA graph and
    replayed on new logits, ids and activations: bit for bit what the calls give one by one."""
    from gpu_util import dev
    lc, mc = D.lora_case(31, 12, 256, 256, 6, 16), D.moe_case(32, 12, 256, 256, 8, 3)
    largs, margs = lora_inputs(lc), moe_inputs(mc)
    lws, mws = fg.lora_workspace(12, 256, 256, 16), fg.moe_mlp_workspace(12, 256, 256, 8)
    y = torch.empty(12, 256, device="cuda")
    out = torch.empty(12, 256, dtype=torch.bfloat16, device="cuda")
    logits = torch.randn(12, 8, device="cuda", generator=torch.Generator("cuda").manual_seed(1))

    def step():
        fg.fp8_gemm_nt_lora(*largs, y, lws)
        fg.quantize_1x128_rows(y, margs[0], margs[1])
        fg.moe_route(logits, margs[6], margs[7])
        fg.fp8_moe_mlp(*margs, out, mws)

    step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for seed in range(3):
        g = torch.Generator("cuda").manual_seed(10 + seed)
        logits.copy_(torch.randn(12, 8, device="cuda", generator=g))
        largs[8].copy_(torch.randint(-1, 6, (12,), device="cuda", generator=g, dtype=torch.int32))
        largs[4].copy_(torch.randn(12, 256, device="cuda", generator=g))
        step()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    _ok(fg)


@pytest.mark.parametrize("which", ["moe", "lora"])
def test_stalled_pipeline_times_out_and_context_survives(fg, which):
    """The bounded waits: with the weight producer holding back its first stage (host-side stall
    hook) the call records a time-out and returns; with a zeroed workspace the next one is right."""
    c = D.moe_case(41, 8, 512, 256, 4, 2) if which == "moe" else D.lora_case(42, 8, 512, 512, 3, 16)
    args = moe_inputs(c) if which == "moe" else lora_inputs(c)
    ws = fg.moe_mlp_workspace(8, 512, 256, 4) if which == "moe" else fg.lora_workspace(8, 512, 512, 16)
    d = torch.empty(8, 512, dtype=torch.bfloat16, device="cuda")
    call = fg.fp8_moe_mlp if which == "moe" else fg.fp8_gemm_nt_lora
    assert fg.get_device_error()[0] == 0
    fg.debug_inject_stall(True, 200_000)
    try:
        call(*args, d, ws)
        st, detail = fg.get_device_error()
    finally:
        fg.debug_inject_stall(False)
    assert st == fg.FG_ERR_DEVICE_TIMEOUT and detail & 0x200, (st, hex(detail))
    ws.zero_()
    if which == "moe":
        check(run_moe(fg, c, ws=ws, args=args), moe_ref(c))
    else:
        check(run_lora(fg, c, ws=ws, args=args), lora_ref(c))


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,l,r,sms", [
    # several token tiles in clusters: many adapters, a last tile of 44 tokens, a last block of 16 rows, more
    # pieces than FP8 units
    (200, 272, 640, 60, 128, 0), (300, 528, 2304, 3, 16, 0), (129, 144, 128, 40, 64, 0),
    # whole tiles, one round and several; equal shares
    (400, 272, 128, 2, 8, 0), (400, 528, 256, 2, 16, 5), (200, 528, 384, 60, 128, 20)])
def test_lora_prompt_shares(fg, m, n, k, l, r, sms, out):
    c = D.lora_case(m + n + l, m, n, k, l, r)
    try:
        fg.set_num_sms(sms)
        check(run_lora(fg, c, out), lora_ref(c, out), out)
    finally:
        fg.set_num_sms(0)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,sms", [(9, 0), (40, 0), (70, 0), (20, 37)])
def test_moe_more_tiles_than_sms(fg, t, sms, fp4):
    """Whole tiles in several rounds."""
    c = D.moe_case(31 + t, t, 256, 128, 170, 16, 170, fp4)
    try:
        fg.set_num_sms(sms)
        check(run_moe(fg, c), moe_ref(c))
    finally:
        fg.set_num_sms(0)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,h,i,e,topk", [(6, 512, 256, 5, 2), (20, 384, 128, 6, 1), (40, 512, 256, 5, 2), (100, 640, 128, 6, 1),
                                          (3, 1024, 128, 2, 1)])
def test_moe_non_finite_weights_stay_with_their_tokens(fg, fp4, t, h, i, e, topk):
    """A NaN code and NaN scales in one expert's weights reach the tokens that use it, and no others."""
    c = D.moe_case(41 + t, t, h, i, e, topk, fp4=fp4)
    ref = moe_ref(c)
    bad = 1
    if fp4:
        c["sf13"][bad, 0, 3] |= 0xFF                          # K-block 0 of a gate row
        c["sf2"][bad, 0, h - 1] |= 0xFF
    else:
        c["w2"][bad, h - 1, 5] = 0x7F
        c["w2"][bad, 17, i - 1] = 0xFF
        c["w13"][bad, 2 * i - 1, 0] = 0x7F
    uses = (c["ids"] == bad).any(axis=1)
    assert uses.any() and not uses.all()
    for out in ("bf16", "f32"):
        got = run_moe(fg, c, out)
        assert np.isnan(got[uses]).any()
        check(got[~uses], (ref[0][~uses], ref[1][~uses]), out)


@pytest.mark.parametrize("m,n,k,l,r,sms", [(20, 272, 256, 4, 16, 0), (64, 528, 384, 12, 64, 0), (300, 272, 256, 4, 16, 0),
                                           (400, 528, 256, 3, 16, 5), (200, 528, 384, 60, 128, 20)])
def test_lora_non_finite_adapters_stay_with_their_tokens(fg, m, n, k, l, r, sms):
    """Infinities and NaN in one adapter's A and B reach the tokens that use it, and no others."""
    c = D.lora_case(51 + m, m, n, k, l, r)
    refs = {out: lora_ref(c, out) for out in ("bf16", "f32")}
    bad = 2
    c["lb_bits"][bad, n - 1, 0] = 0x7F80
    c["lb_bits"][bad, 3, r - 1] = 0x7FC0
    c["la_bits"][bad, 1, k - 1] = 0xFF80
    uses = c["ids"] == bad
    assert uses.any() and not uses.all()
    try:
        fg.set_num_sms(sms)
        for out, ref in refs.items():
            got = run_lora(fg, c, out)
            assert not np.isfinite(got[uses]).all()
            check(got[~uses], (ref[0][~uses], ref[1][~uses]), out)
    finally:
        fg.set_num_sms(0)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,sms", [(5, 3), (40, 3), (100, 4), (40, 2)])
def test_moe_more_down_tiles_than_sms(fg, t, sms, fp4):
    """The down projection's tiles do not fit the SMs: no clusters, no third launch."""
    c = D.moe_case(61 + t, t, 1152, 128, 3, 2, fp4=fp4)
    ref = moe_ref(c)
    try:
        fg.set_num_sms(sms)
        for out in ("bf16", "f32"):
            check(run_moe(fg, c, out), ref, out)
    finally:
        fg.set_num_sms(0)


@pytest.mark.parametrize("m,sms", [(1, 3), (8, 5), (40, 3), (100, 2)])
def test_lora_more_tiles_than_sms(fg, m, sms):
    c = D.lora_case(71 + m, m, 1600, 256, 5, 16)
    try:
        fg.set_num_sms(sms)
        check(run_lora(fg, c), lora_ref(c))
    finally:
        fg.set_num_sms(0)
