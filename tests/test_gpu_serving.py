"""GPU parity of the attention side of a serving step (block tables, norms with rotation, the 4-bit cache,
attention over it) against the FP64 oracle, whose bounds are derived from the operands; codes, tables and
untouched memory are compared exactly."""
import numpy as np
import pytest

import serving_cases as C
from gpu_util import dev
from oracle import serving as O
from oracle.decode import within

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


@pytest.fixture(scope="module")
def fg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_fp8_e4m3_gb300 as lib
    lib.get_device_error()
    return lib


def expect(fg, status=0, detail=0):
    assert fg.get_device_error() == (status, detail)


def bf(bits):
    return dev(np.asarray(bits).view(np.int16)).view(BF)


def f64(t):
    return t.double().cpu().numpy()


# -------------------------------------------------------------------------- attention
def attend(fg, c, window=0, scale=None, out=None, ws=None, stream=None):
    q = bf(c["q_bits"])
    out = torch.full_like(q, -77.0) if out is None else out
    ws = fg.paged_attention_workspace(q.shape[0], len(c["lens"]), c["hq"], c["hkv"], c["d"]) if ws is None else ws
    fg.paged_attention_mxfp4(q, dev(c["kc"]), dev(c["ks"]), dev(c["vc"]), dev(c["vs"]), dev(c["table"]), dev(c["start"]),
                             dev(c["lens"]), out, ws, scale=scale, window=window, stream=stream)
    return out, ws


def check(c, out, window=0, scale=None):
    ref, bound, used = C.reference(c, scale, window)
    got = f64(out)
    assert (got[~used] == -77.0).all(), "rows behind the last request were written"
    bad = ~within(got[used], (ref[used], bound[used]), "bf16")
    assert not bad.any(), (bad.sum(), np.abs(got[used] - ref[used])[bad].max(), np.argwhere(bad)[:4])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 1), (6, 2), (12, 3), (32, 2)])
@pytest.mark.parametrize("page", [16, 48, 128])
def test_decode_over_ragged_lengths(fg, d, hq, hkv, page):
    lens = [1, 15, 16, 17, 0, 127, 128, 129, 300]
    c = C.cache_case(hq + d + page, lens, [min(n, 1) for n in lens], hq, hkv, d, page)
    out, ws = attend(fg, c)
    expect(fg)
    check(c, out)
    assert not ws[:7680].any(), "counters are left as they were"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(2, 2), (8, 2), (5, 1), (16, 1)])
@pytest.mark.parametrize("window", [0, 1, 7, 100])
def test_several_new_tokens(fg, d, hq, hkv, window):
    """Rows of one request at different positions: causal masks, chunks that end inside a token's heads, windows."""
    c = C.cache_case(hq + d + window, [40, 5, 333, 130, 70], [3, 5, 1, 0, 37], hq, hkv, d, 32)
    out, _ = attend(fg, c, window)
    expect(fg)
    check(c, out, window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,new", [(2, 2, [70, 64, 65]), (8, 1, [30, 0, 17]), (6, 2, [1, 100, 9]), (16, 1, [8, 8, 3]),
                                        (16, 1, [40, 5, 61]), (4, 2, [300, 1, 150])])
@pytest.mark.parametrize("window", [0, 33])
@pytest.mark.parametrize("page", [16, 80])
def test_many_rows_a_request(fg, d, hq, hkv, new, window, page):
    """Chunks of 128 rows on the tensor cores: ends inside a token's heads, requests of few rows among them, tiles that
    end behind the keys, windows that begin inside a tile."""
    lens = [n + extra for n, extra in zip(new, (0, 200, 131))]
    extra_rows = 3 * 2048 if window else 3 * -(-256 * hkv // hq)
    c = C.wide(C.cache_case(d + hq + sum(new) + window + page, lens, new, hq, hkv, d, page, extra_rows=extra_rows))
    assert C.many_rows(c, window)
    out, ws = attend(fg, c, window)
    expect(fg)
    check(c, out, window)
    assert not ws[:7680].any(), "counters are left as they were"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 50, 400])
def test_many_requests_of_many_rows(fg, d, window):
    """More items than CTAs, windows that begin inside a tile, requests without rows among them."""
    g = C.rng(d + window)
    new = g.integers(0, 40, 60)
    c = C.cache_case(d + window, new + g.integers(0, 200, 60), new, 8, 2, d, 16, extra_rows=2000)
    assert C.many_rows(c, window)
    out, ws = attend(fg, c, window)
    expect(fg)
    check(c, out, window)
    assert not ws[:7680].any(), "counters are left as they were"


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [512, 1 << 18])
@pytest.mark.parametrize("rows", [24, 32, 33, 48, 64, 65, 80, 128, 136])
def test_row_counts_around_the_choice_of_kernel(fg, d, tokens, rows):
    c = C.wide(C.cache_case(rows, [rows + 40, 400], [rows, rows], 1, 1, d, 16, extra_rows=0), tokens)
    out, _ = attend(fg, c)
    expect(fg)
    check(c, out)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[40, 1], [70, 60]])
def test_many_rows_over_long_contexts_are_split_and_joined(fg, d, new):
    c = C.wide(C.cache_case(d, [2500, 1800], new, 8, 1, d, 32))
    assert C.many_rows(c)
    out, ws = attend(fg, c)
    expect(fg)
    check(c, out)
    for _ in range(3):
        again, _ = attend(fg, c, ws=ws)
        assert torch.equal(again, out)


@pytest.mark.parametrize("new", [20, 50, 70])
def test_many_rows_scores_that_keep_rising(fg, new):
    """Keys whose scores rise by far more than a step of the running maximum, tile by tile, and fall again."""
    c = C.wide(C.cache_case(12, [1000], [new], 8, 1, 64, 16))
    assert C.many_rows(c)
    c["q"][:] = np.abs(c["q"])
    c["q_bits"], c["q"] = O.bf16(c["q"])
    n = np.arange(1000)
    x = np.zeros((1000, 1, 64))
    x[:] = (np.where(n < 700, n, 1400 - n) / 50.0)[:, None, None]
    codes, sf = O.encode(x)
    p, o = c["table"][0, n // 16], n % 16
    c["kc"][p, :, o], c["ks"][p, :, o] = O.rows(codes, "k"), sf
    out, _ = attend(fg, c)
    expect(fg)
    check(c, out)


@pytest.mark.parametrize("hq", [4, 16, 32])
def test_many_rows_contract_violations_and_non_finite_queries(fg, hq):
    c = C.wide(C.cache_case(13, [300, 90], [40, 30], hq, 2, 128, 16))
    assert C.many_rows(c)
    c = dict(c, q_bits=np.concatenate([c["q_bits"]] * 1), table=c["table"].copy())
    ref = O.attention(c["q"], c["kc"], c["ks"], c["vc"], c["vs"], c["table"], c["start"], c["lens"], 128 ** -0.5, 0, 2.0 ** -8)
    c["q_bits"][5, 1, 7] = 0x7FC0
    c["q_bits"][6, 3, 0] = 0x7F80
    c["table"][1, 2] = -1
    out, _ = attend(fg, c)
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x10A)
    got = f64(out)
    assert np.isnan(got[5, 1]).all() and np.isnan(got[6, 3]).any()
    ok = np.ones((40, hq), bool)
    ok[5, 1] = ok[6, 3] = False
    assert within(got[:40][ok], (ref[0][:40][ok], ref[1][:40][ok]), "bf16").all()
    # request 1 without the tokens of its third page: the others move up, positions and all
    keep = np.r_[0:32, 48:90]
    small = {k: c[k].copy() for k in ("kc", "ks", "vc", "vs")}
    page, off = c["table"][1, keep // 16], keep % 16
    at = np.arange(len(keep))
    for k in small:
        small[k][c["table"][0, at // 16], :, at % 16] = c[k][page, :, off]
    one = O.attention(c["q"][40:70], *[small[k] for k in ("kc", "ks", "vc", "vs")], c["table"][:1], [0, 30], [74], 128 ** -0.5, 0, 2.0 ** -8)
    assert within(got[40:70], one[:2], "bf16").all()
    assert (got[70:] == -77).all()


@pytest.mark.parametrize("hq", [4, 32])
def test_a_stalled_wait_times_out_and_the_context_survives(fg, hq):
    """The bounded waits of the tensor-core kernel, of one row tile and two: with its first key tile held back (host-side
    hook) the call records a time-out and returns, and the same call is right afterwards, on a workspace zeroed anew."""
    c = C.wide(C.cache_case(21, [300, 190], [70, 80], hq, 1 if hq == 32 else 2, 128, 16))
    assert C.many_rows(c)
    fg.debug_inject_stall(True, 200_000)
    try:
        out, ws = attend(fg, c)
        status, detail = fg.get_device_error()
    finally:
        fg.debug_inject_stall(False)
    assert status == fg.FG_ERR_DEVICE_TIMEOUT and detail & 0xF00 == 0x200
    ws.zero_()
    out, _ = attend(fg, c, ws=ws)
    expect(fg)
    check(c, out)


def test_rows_before_the_first_key(fg):
    """More rows than cached tokens: the rows before position 0 look at nothing and become zero."""
    c = C.cache_case(3, [3, 0, 20], [3, 0, 2], 4, 2, 128, 16, extra_rows=9)
    c["start"] = np.array([0, 5, 9, 11], np.int32)
    out, _ = attend(fg, c)
    expect(fg)
    check(c, out)
    got = f64(out)
    assert not got[:2].any() and not got[5:9].any()


@pytest.mark.parametrize("hkv,length", [(1, 20000), (2, 9000)])
def test_one_long_request_is_split_and_joined(fg, hkv, length):
    c = C.cache_case(length, [length], [1], 8 * hkv, hkv, 128, 64)
    out, ws = attend(fg, c)
    expect(fg)
    check(c, out)
    for _ in range(3):                                       # the order of arrival does not matter
        again, _ = attend(fg, c, ws=ws)
        assert torch.equal(again, out)


@pytest.mark.parametrize("d,hq,new", [(64, 8, 1), (64, 16, 1), (64, 8, 3), (128, 16, 1), (128, 8, 1), (256, 8, 1), (256, 16, 1)])
def test_long_requests_beside_short_ones(fg, d, hq, new):
    """Many pieces an item, joined eight at a time, of one and more row tiles; items that end inside a group of eight."""
    c = C.cache_case(d + hq, [9000, 3, 17, 6500], [new, 1, 0, new], hq, 1, d, 32)
    out, ws = attend(fg, c)
    expect(fg)
    check(c, out)
    assert not ws[:7680].any(), "counters are left as they were"
    again, _ = attend(fg, c, ws=ws)
    assert torch.equal(again, out)


def test_a_workspace_serves_calls_of_other_sizes(fg):
    ws = fg.paged_attention_workspace(64, 1, 32, 1, 256)
    for seed, (lens, new, hq, hkv, d) in enumerate([([700, 3], [2, 1], 8, 2, 128), ([5000], [1], 4, 1, 256),
                                                    ([90] * 5, [4] * 5, 16, 4, 64), ([700], [40], 8, 2, 256),
                                                    ([5000, 17], [1, 1], 3, 3, 128), ([60, 300], [60, 9], 4, 1, 64)]):
        c = C.wide(C.cache_case(seed, lens, new, hq, hkv, d, 32))
        out, _ = attend(fg, c, ws=ws)
        expect(fg)
        check(c, out)


@pytest.mark.parametrize("spread", [0, 12, 28])
def test_scales_far_apart(fg, spread):
    """Block scales of different tokens 2^-spread to 2^spread apart, of keys (a few dominate) and values."""
    c = C.cache_case(spread, [260, 33, 7], [2, 1, 4], 4, 2, 128, 16, spread=spread, q_scale=2.0 ** -spread)
    out, _ = attend(fg, c)
    expect(fg)
    check(c, out)


@pytest.mark.parametrize("power", [-100, -20, 20, 60])
def test_queries_of_any_size(fg, power):
    c = C.cache_case(power + 200, [77, 150], [1, 3], 8, 2, 128, 16)
    c["q_bits"], c["q"] = O.bf16(c["q"] * 2.0 ** power)
    scale = 128 ** -0.5 * 2.0 ** -power
    out, _ = attend(fg, c, scale=scale)
    expect(fg)
    check(c, out, scale=float(np.float32(scale)))


def test_non_finite_queries_stay_in_their_rows(fg):
    c = C.cache_case(9, [60, 300], [2, 1], 8, 2, 128, 16)
    ref, bound, used = C.reference(c)
    bits = c["q_bits"].copy()
    bits[0, 1, 5] = 0x7FC0
    bits[1, 6, 0] = 0x7F80
    out, _ = attend(fg, dict(c, q_bits=bits))
    expect(fg)
    got = f64(out)
    assert np.isnan(got[0, 1]).all() and np.isnan(got[1, 6]).any()
    used = np.repeat(used[:, None], 8, 1)
    used[0, 1] = used[1, 6] = False
    assert within(got[used], (ref[used], bound[used]), "bf16").all()


def test_contract_violations_leave_the_others_right(fg):
    lens, new = [50, 20, 64, 33], [1, 1, 2, 1]
    c = C.cache_case(4, lens, new, 4, 2, 64, 16)
    ref, bound, _ = C.reference(c)

    def run(**kw):
        out, _ = attend(fg, dict(c, **{k: np.array(v, np.int32) for k, v in kw.items()}))
        expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x10A)
        return f64(out)

    def right(got, rows):
        assert within(got[rows], (ref[rows], bound[rows]), "bf16").all()

    got = run(lens=[50, -1, 64, 33])
    right(got, [0, 2, 3, 4])
    assert (got[1] == -77).all()
    got = run(lens=[50, 20, 64, 10 ** 6])
    right(got, [0, 1, 2, 3])
    assert (got[4] == -77).all()
    got = run(start=[0, 1, 2, 4, 99])
    right(got, [0, 1, 2, 3])
    assert (got[4:] == -77).all()
    got = run(start=[0, 1, -3, 4, 5])
    right(got, [0, 4])
    assert (got[1:4] == -77).all()
    table = c["table"].copy()
    table[1, 1] = c["pages"]
    table[2, 0] = -4
    got = run(table=table)
    right(got, [0, 4])
    # request 1 without its second page, request 2 without its first: the other tokens alone
    one = O.attention(c["q"][1:2], c["kc"], c["ks"], c["vc"], c["vs"], c["table"][1:2], [0, 1], [16], 64 ** -0.5)
    assert within(got[1:2], one[:2], "bf16").all()
    two = O.attention(c["q"][2:4], c["kc"], c["ks"], c["vc"], c["vs"], c["table"][2:3, 1:], [0, 2], [48], 64 ** -0.5)
    assert within(got[2:4], two[:2], "bf16").all()


@pytest.mark.parametrize("s,new", [(8, 4), (300, 1), (6, 100), (700, 3)])
@pytest.mark.parametrize("tokens", [16, 1 << 18])
def test_requests_that_claim_the_same_rows(fg, s, new, tokens):
    """query_start goes up and down over all rows again and again: nothing is written, and the next call is right."""
    c = C.wide(C.cache_case(s, [new + 3] * s, [new] * s, 4, 2, 64, 16), tokens)
    out, ws = attend(fg, dict(c, start=np.resize(np.array([0, s * new], np.int32), s + 1)))
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x10A)
    assert (f64(out) == -77).all()
    out, _ = attend(fg, c, ws=ws)
    expect(fg)
    check(c, out)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_prompt_among_many_decodes(fg, d):
    new = [1] * 40
    new[17] = 260
    lens = [30 + 7 * i for i in range(40)]
    lens[17] = 400
    c = C.cache_case(d, lens, new, 8, 2, d, 16, extra_rows=0)
    out, _ = attend(fg, c)
    expect(fg)
    check(c, out)


def test_streams_and_graph_replays_with_new_lengths(fg):
    """Lengths are read on the device: a captured call serves whatever they are when it is replayed."""
    c = C.cache_case(6, [200, 90, 31], [1, 1, 1], 8, 2, 128, 32)
    q, cache = bf(c["q_bits"]), [dev(c[k]) for k in ("kc", "ks", "vc", "vs")]
    table, start, lens = dev(c["table"]), dev(c["start"]), dev(c["lens"])
    out = torch.full_like(q, -77.0)
    ws = fg.paged_attention_workspace(q.shape[0], 3, 8, 2, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fg.paged_attention_mxfp4(q, *cache, table, start, lens, out, ws)
    side.synchronize()
    check(c, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fg.paged_attention_mxfp4(q, *cache, table, start, lens, out, ws)
        fg.paged_attention_mxfp4(q, *cache, table, start, lens, out, ws, window=64)
    for now in ([200, 90, 31], [130, 1, 0], [1, 89, 16]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(dict(c, lens=np.array(now, np.int32)), out, window=64)
    expect(fg)


def test_rows_past_32_bits_of_offset(fg):
    """A cache of 4.4 GB a kind: its last pages lie past 2^32 bytes."""
    hkv, d, page, pages = 8, 128, 64, 140000
    if torch.cuda.get_device_properties(0).total_memory < 40 << 30:
        pytest.skip("needs 10 GB")
    cache = [torch.empty(pages, hkv, page, n, dtype=torch.uint8, device="cuda") for n in (64, 4, 64, 4)]
    g = C.rng(8)
    n = 100
    bits, x = O.bf16(g.standard_normal((2, n, hkv, d)))
    order = np.array([pages - 1, pages - 2])
    slots = order[np.arange(n) // page] * page + np.arange(n) % page
    fg.kv_append_mxfp4(bf(bits[0]), bf(bits[1]), dev(slots.astype(np.int32)), *cache)
    k, v = (torch.empty(n, hkv, d, dtype=BF, device="cuda") for _ in range(2))
    fg.kv_gather_mxfp4(dev(slots.astype(np.int32)), *cache, k, v)
    small = [np.zeros((2, hkv, page, m), np.uint8) for m in (64, 4, 64, 4)]
    for i, kind in enumerate("kv"):
        codes, sf = O.encode(x[i])
        small[2 * i][np.arange(n) // page, :, np.arange(n) % page] = O.rows(codes, kind)
        small[2 * i + 1][np.arange(n) // page, :, np.arange(n) % page] = sf
        assert np.array_equal(f64(k if kind == "k" else v), O.decode(O.rows(codes, kind), sf, kind))
    q_bits, q = O.bf16(g.standard_normal((1, 16, d)))
    out = torch.empty(1, 16, d, dtype=BF, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fg.paged_attention_mxfp4(bf(q_bits), *cache, i32(*order)[None], i32(0, 1), i32(n), out, fg.paged_attention_workspace(1, 1, 16, hkv, d))
    ref = O.attention(q, *small, np.array([[0, 1]]), [0, 1], [n], d ** -0.5)
    assert within(f64(out), ref[:2], "bf16").all()
    expect(fg)


# ------------------------------------------------------------------------------ cache
def empty_cache(pages, heads, page, d):
    return [torch.full((pages, heads, page, n), 0xA5, dtype=torch.uint8, device="cuda") for n in (d // 2, d // 32) * 2]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("t,heads,page", [(1, 1, 16), (37, 3, 48), (301, 8, 64)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_and_gather(fg, d, t, heads, page, strided):
    g = C.rng(d + t)
    pages = t // page + 4
    slots = g.permutation(pages * page)[:t]
    slots[::5] = -1 - np.arange(len(slots[::5]))            # skipped
    x = g.standard_normal((2, t, heads, d)) * 2.0 ** g.integers(-12, 13, (2, t, heads, 1))
    x[0, t // 2, 0, :32] = 0.0
    bits, x = O.bf16(x)
    kv = torch.zeros(t, 2 * heads * d + (24 if strided else 0), dtype=BF, device="cuda")
    k, v = kv[:, :heads * d].view(t, heads, d), kv[:, heads * d:2 * heads * d].view(t, heads, d)
    k.copy_(bf(bits[0])), v.copy_(bf(bits[1]))
    cache = empty_cache(pages, heads, page, d)
    want = [c.cpu().numpy() for c in cache]
    fg.kv_append_mxfp4(k, v, dev(slots.astype(np.int32)), *cache)
    expect(fg)
    live = slots >= 0
    p, o = slots[live] // page, slots[live] % page
    back = []
    for i, kind in enumerate("kv"):
        codes, sf = O.encode(x[i])
        want[2 * i][p, :, o], want[2 * i + 1][p, :, o] = O.rows(codes, kind)[live], sf[live]
        back.append(O.decode(O.rows(codes, kind), sf, kind))
    for got, w in zip(cache, want):
        assert np.array_equal(got.cpu().numpy(), w)
    out = torch.full((t, 2 * heads * d + (24 if strided else 0)), 5.0, dtype=BF, device="cuda")
    ko, vo = out[:, :heads * d].view(t, heads, d), out[:, heads * d:2 * heads * d].view(t, heads, d)
    fg.kv_gather_mxfp4(dev(slots.astype(np.int32)), *cache, ko, vo)
    expect(fg)
    for got, w in zip((ko, vo), back):
        got = f64(got)
        assert np.array_equal(got[live], w[live]) and (got[~live] == 5.0).all()
    assert (out[:, 2 * heads * d:] == 5.0).all()


def test_append_of_non_finite_and_extreme_values(fg):
    x = np.zeros((3, 1, 64))
    x[0, 0, :4] = [2.0 ** 100, -2.0 ** 64, 2.0 ** 62, 1.0]
    x[1, 0, 0], x[1, 0, 33] = 2.0 ** -63, 2.0 ** -100
    bits, x = O.bf16(x)
    bits[2, 0, :4] = [0x7F80, 0xFF80, 0x7FC0, 0x3F80]       # inf, -inf, NaN, 1
    bits[2, 0, 32:35] = [0x7FC0, 0x4000, 0xC040]            # NaN, 2, -3
    cache = empty_cache(1, 1, 16, 64)
    slots = dev(np.arange(3, dtype=np.int32))
    fg.kv_append_mxfp4(bf(bits), bf(bits), slots, *cache)
    k, v = (torch.empty(3, 1, 64, dtype=BF, device="cuda") for _ in range(2))
    fg.kv_gather_mxfp4(slots, *cache, k, v)
    expect(fg)
    codes, sf = O.encode(x[:2])
    want = np.zeros((3, 1, 64))
    want[:2] = O.decode(O.rows(codes, "k"), sf, "k")
    top = 6 * 2.0 ** 63
    want[2, 0, :3] = [top, -top, top]
    want[2, 0, 32:35] = [6 * 0.5, 2.0, -3.0]                # the block's largest number is 3: scale 2^-1
    assert np.array_equal(f64(k), want) and np.array_equal(f64(v), want)


def test_slots_past_the_cache(fg):
    bits, _ = O.bf16(C.rng(1).standard_normal((4, 2, 128)))
    cache = empty_cache(2, 2, 16, 128)
    for slot in (32, 2 ** 31 - 1):
        slots = dev(np.array([0, slot, 31, -1], np.int32))
        fg.kv_append_mxfp4(bf(bits), bf(bits), slots, *cache)
        expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x108)
        k, v = (torch.full((4, 2, 128), 5.0, dtype=BF, device="cuda") for _ in range(2))
        fg.kv_gather_mxfp4(slots, *cache, k, v)
        expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x108)
        assert (k[[1, 3]] == 5.0).all() and not (k[[0, 2]] == 5.0).all()
    touched = cache[0][:, 0].reshape(32, 64)[[0, 31]]
    assert not (touched == 0xA5).all() and (cache[0][:, 0].reshape(32, 64)[1:31] == 0xA5).all()


# ------------------------------------------------------------------- norms, rotation
@pytest.mark.parametrize("d,rot", [(8, 0), (64, 64), (64, 32), (96, 96), (128, 128), (128, 16), (192, 64), (256, 256), (40, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["both", "q", "none"])
def test_norm_and_rotation(fg, d, rot, interleaved, norm):
    t, hq, hkv = 11, 5, 2
    g = C.rng(d + rot)
    qb, q = O.bf16(g.standard_normal((t, hq, d)) * 3)
    kb, k = O.bf16(g.standard_normal((t, hkv, d)) * 3)
    wb, w = O.bf16(1 + 0.3 * g.standard_normal((2, d)))
    angle = g.random((50, rot // 2)) * 6.28
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = g.integers(0, 50, t).astype(np.int32)
    pos[4] = -1
    qo = torch.full((t, hq, d), 5.0, dtype=BF, device="cuda")
    ko = torch.full((t, hkv, d), 5.0, dtype=BF, device="cuda")
    wq, wk = norm != "none", norm == "both"
    fg.qk_norm_rope(bf(qb), bf(kb), dev(pos), dev(cs), qo, ko, q_weight=bf(wb[0]) if wq else None,
                    k_weight=bf(wb[1]) if wk else None, eps=1e-5, interleaved=interleaved)
    expect(fg)
    for got, x, weight in ((qo, q, w[0] if wq else None), (ko, k, w[1] if wk else None)):
        got = f64(got)
        ref = O.norm_rope(x, weight, float(np.float32(1e-5)), np.maximum(pos, 0), cs, interleaved)
        live = pos >= 0
        assert within(got[live], (ref[0][live], ref[1][live]), "bf16").all()
        assert (got[~live] == 5.0).all()


@pytest.mark.parametrize("t,hq,hkv", [(1, 1, 1), (3, 7, 0), (700, 33, 5), (2048, 16, 6)])
def test_norm_and_rotation_in_place_of_a_projections_rows(fg, t, hq, hkv):
    """Queries and keys side by side in rows that hold more; outputs over the inputs; sizes on both sides of the one
    from which a lane keeps four heads."""
    d = 128
    g = C.rng(t)
    width = (hq + hkv) * d + 40
    xb, x = O.bf16(g.standard_normal((t, width)))
    angle = g.random((t + 3, 64)) * 6.28
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    pos = (np.arange(t) + 3).astype(np.int32)
    wb, w = O.bf16(1 + 0.3 * g.standard_normal((2, d)))
    buf = bf(xb)
    q, k = buf[:, :hq * d].view(t, hq, d), buf[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    fg.qk_norm_rope(q, k, dev(pos), dev(cs), q, k, q_weight=bf(wb[0]), k_weight=bf(wb[1]))
    expect(fg)
    got = f64(buf)
    for lo, n, weight in ((0, hq, w[0]), (hq * d, hkv, w[1])):
        ref = O.norm_rope(x[:, lo:lo + n * d].reshape(t, n, d), weight, float(np.float32(1e-6)), pos, cs, False)
        assert within(got[:, lo:lo + n * d].reshape(t, n, d), ref, "bf16").all()
    assert np.array_equal(got[:, (hq + hkv) * d:], x[:, (hq + hkv) * d:])


def test_positions_past_the_table(fg):
    x = torch.ones(3, 2, 64, dtype=BF, device="cuda")
    cs = torch.zeros(10, 64, device="cuda")
    qo, ko = torch.full_like(x, 5.0), torch.full_like(x, 5.0)
    fg.qk_norm_rope(x, x, dev(np.array([9, 10, 2 ** 31 - 1], np.int32)), cs, qo, ko)
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x109)
    assert not qo[0].any() and not ko[0].any() and (qo[1:] == 5.0).all() and (ko[1:] == 5.0).all()


def test_norm_of_zeros_and_large_values(fg):
    x = torch.zeros(2, 1, 128, dtype=BF, device="cuda")
    x[1, 0, 3] = 2.0 ** 60
    cs = torch.cat([torch.ones(4, 64), torch.zeros(4, 64)], 1).cuda()
    w = torch.ones(128, dtype=BF, device="cuda")
    qo, ko = torch.empty_like(x), torch.empty_like(x)
    fg.qk_norm_rope(x, x, dev(np.array([0, 1], np.int32)), cs, qo, ko, q_weight=w, k_weight=w)
    expect(fg)
    assert not qo[0].any()
    assert float(qo[1, 0, 3]) == float(torch.tensor(128 ** 0.5).to(BF)) and not qo[1, 0, 4:].any()


# ---------------------------------------------------------------------- block tables
def tables(fg, c, t, page, alias=False):
    i32 = lambda x: dev(np.asarray(x).astype(np.int32))  # noqa: E731
    a = {"context": i32(c["context"]), "new": i32(c["new"]), "free": i32(c["free"]), "count": i32([c["count"]]),
         "table": i32(c["table"])}
    s = len(c["context"])
    a["start"] = torch.full((s + 1,), -77, dtype=torch.int32, device="cuda")
    a["lens"] = a["context"] if alias else torch.full((s,), -77, dtype=torch.int32, device="cuda")
    a["count_out"] = a["count"] if alias else torch.full((1,), -77, dtype=torch.int32, device="cuda")
    a["slots"], a["positions"] = (torch.full((t,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    fg.build_block_tables(a["context"], a["new"], a["free"], a["count"], a["table"], a["start"], a["lens"], a["slots"],
                          a["positions"], a["count_out"], page_size=page, num_pages=c["pages"])
    return a


def check_tables(a, c, t, page):
    ref = O.block_tables(c["context"], c["new"], c["free"], c["count"], c["table"], t, page, c["pages"])
    for k in ("table", "free", "start", "lens", "slots", "positions"):
        assert np.array_equal(a[k].cpu().numpy(), ref[k]), k
    assert int(a["count_out"]) == ref["count"]


@pytest.mark.parametrize("s,page,longest,mode", [(1, 1, 3, "decode"), (5, 16, 40, "prompts"), (33, 7, 100, "decode"),
                                                 (1030, 16, 50, "decode"), (90, 16, 33, "prompts"), (4000, 64, 200, "decode")])
@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("spare", [0, 5, 2000])
def test_block_tables(fg, s, page, longest, mode, alias, spare):
    c = C.tables_case(s + page, s, page, longest, (longest + 60) // page + 2, mode)
    a = tables(fg, c, c["t"] + spare, page, alias)
    expect(fg)
    check_tables(a, c, c["t"] + spare, page)


def test_block_tables_again_on_the_same_inputs(fg):
    c = C.tables_case(1, 20, 16, 60, 9, "prompts")
    a = tables(fg, c, c["t"], 16)
    first = {k: v.clone() for k, v in a.items()}
    fg.build_block_tables(a["context"], a["new"], a["free"], a["count"], a["table"], a["start"], a["lens"], a["slots"],
                          a["positions"], a["count_out"], page_size=16, num_pages=c["pages"])
    expect(fg)
    assert all(torch.equal(first[k], a[k]) for k in a)


def test_block_tables_of_no_request(fg):
    c = {"context": [], "new": [], "free": [4], "count": 1, "table": np.zeros((0, 2)), "pages": 9}
    a = tables(fg, c, 3, 16)
    expect(fg)
    assert int(a["start"][0]) == 0 and (a["slots"] == -1).all() and int(a["count_out"]) == 1


@pytest.mark.parametrize("change", [
    dict(context=[20, -1, 5]), dict(new=[1, -2, 1]), dict(context=[20, 81, 5]), dict(new=[61, 0, 0]), dict(count=0),
    dict(count=-1), dict(count=13), dict(t=2), dict(new=[1, 2 ** 31 - 1, 1]), dict(context=[20, 2 ** 31 - 1, 5]),
    dict(new=[-1, 1, 1], count=11)])
def test_steps_that_are_refused_are_empty(fg, change):
    """Three requests, pages of 16, rows of 5 pages, 12 places in the free list, 4 tokens at most."""
    c = {"context": [20, 16, 5], "new": [1, 1, 1], "free": list(range(10, 22)), "count": 4,
         "table": np.arange(15).reshape(3, 5), "pages": 30}
    c.update(change)
    a = tables(fg, c, c.pop("t", 4), 16)
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x107)
    assert not a["start"].any() and (a["slots"] == -1).all() and (a["positions"] == -1).all()
    assert a["lens"].tolist() == [max(x, 0) for x in c["context"]] and int(a["count_out"]) == c["count"]
    assert np.array_equal(a["table"].cpu().numpy(), c["table"]) and a["free"].tolist() == c["free"]


def test_page_ids_outside_the_cache_get_no_slot(fg):
    c = {"context": [20, 16, 5], "new": [2, 1, 1], "free": [77, 1, 2], "count": 1, "table": np.array([[3, 30], [4, 0], [-2, 0]]),
         "pages": 30}
    a = tables(fg, c, 5, 16)
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x107)
    assert a["slots"].tolist() == [-1] * 5 and a["positions"].tolist() == [20, 21, 16, 5, -1]


# ------------------------------------------------------------------- steps of a model
def test_steps_of_a_layer(fg):
    """What a serving loop does with one layer: requests come, go on and finish; tables, rotation, append and attention
    run one after another on the same stream without the host reading anything in between."""
    hq, hkv, d, page, pages, width, s, t = 8, 2, 128, 16, 40, 8, 4, 48
    g = C.rng(11)
    cache = empty_cache(pages, hkv, page, d)
    host = [c.cpu().numpy() for c in cache]
    i32 = lambda x: dev(np.asarray(x).astype(np.int32))  # noqa: E731
    lens, count, table = i32([0] * s), i32([pages]), i32(np.full((s, width), -1))
    free = i32(g.permutation(pages))
    start, slots, positions = i32([0] * (s + 1)), i32([0] * t), i32([0] * t)
    angle = np.arange(width * page)[:, None] * 0.1 ** np.arange(64)[None]
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    wb, w = O.bf16(1 + 0.1 * g.standard_normal((2, d)))
    ws = fg.paged_attention_workspace(t, s, hq, hkv, d)
    for new in ([20, 5, 0, 17], [1, 1, 30, 1], [1, -1, 1, 1], [1, 16, -1, 4], [-1, 1, 2, 1], [15, 1, 1, 0]):
        bits, _ = O.bf16(g.standard_normal((t, (hq + 2 * hkv) * d)))
        qkv = bf(bits)
        q, k, v = (x.view(t, -1, d) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
        fg.build_block_tables(lens, i32(new), free, count, table, start, lens, slots, positions, count, page_size=page, num_pages=pages)
        fg.qk_norm_rope(q, k, positions, dev(cs), q, k, q_weight=bf(wb[0]), k_weight=bf(wb[1]))
        fg.kv_append_mxfp4(k, v, slots, *cache)
        qc = q.contiguous()
        out = torch.full_like(qc, -77.0)
        fg.paged_attention_mxfp4(qc, *cache, table, start, lens, out, ws)
        expect(fg)
        sl = slots.cpu().numpy()
        for i, (kind, x) in enumerate((("k", k), ("v", v))):
            codes, sf = O.encode(f64(x)[sl >= 0])
            p, o = sl[sl >= 0] // page, sl[sl >= 0] % page
            host[2 * i][p, :, o], host[2 * i + 1][p, :, o] = O.rows(codes, kind), sf
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(cache, host))
        ref, bound, used = O.attention(f64(qc), *host, table.cpu().numpy(), start.cpu().numpy(), lens.cpu().numpy(), d ** -0.5)
        got = f64(out)
        assert within(got[used], (ref[used], bound[used]), "bf16").all() and (got[~used] == -77.0).all()
        held = sum(-(-int(x) // page) for x in lens.cpu().numpy())
        assert int(count) + held == pages


# ------------------------------------------------------------------- the module in C++
def native_calls(fg):
    bind = fg._native()
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    bf16 = lambda *n: torch.zeros(n, dtype=BF, device="cuda")  # noqa: E731
    caches = list(fg.kv_cache_mxfp4(4, 2, 16, 128))
    free = torch.arange(9, dtype=torch.int32, device="cuda")
    ws = fg.paged_attention_workspace(5, 2, 8, 2, 128)
    q, k = bf16(5, 8, 128), bf16(5, 2, 128)
    w = bf16(128)
    return {
        "tables": (bind.tables, [i32(2), i32(2), free, i32(1), i32(2, 4), i32(3), i32(2), i32(5), i32(5), i32(1), 16, 9]),
        "rope": (bind.rope, [q, k, i32(5), torch.ones(9, 128, device="cuda"), q.clone(), k.clone(), w, w, 1e-6, True]),
        "append": (bind.append, [k, k, i32(5) - 1] + caches),
        "gather": (bind.gather, [k.clone(), k.clone(), i32(5)] + caches),
        "attention": (bind.attention, [q] + caches + [i32(2, 4), i32(3), i32(2), q.clone(), ws, 0.1, 7]),
    }


@pytest.mark.parametrize("name", ["tables", "rope", "append", "gather", "attention"])
def test_native_calls_take_good_arguments_only(fg, name):
    call, args = native_calls(fg)[name]
    assert call(*args) == fg.FG_OK
    expect(fg)
    for i, x in enumerate(args):
        wrong = [object(), "x", 2 ** 40] + ([] if isinstance(x, float) else [0.5])
        if torch.is_tensor(x):
            wrong.append(x.cpu())
            if not (name == "attention" and i == 9):        # a workspace is of any type
                wrong.append(x.double())
            if x.numel() > 1:
                wrong.append(torch.stack([x, x], -1)[..., 0])                  # elements apart
        for y in wrong:
            assert call(*args[:i], y, *args[i + 1:]) is None, (i, y)
    expect(fg)


def test_native_calls_refuse_shapes_that_do_not_belong_together(fg):
    calls = native_calls(fg)
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    bf16 = lambda *n: torch.zeros(n, dtype=BF, device="cuda")  # noqa: E731
    u8 = lambda *n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
    for name, i, y in [("tables", 0, i32(3)), ("tables", 1, i32(1)), ("tables", 3, i32(2)), ("tables", 4, i32(8)), ("tables", 4, i32(3, 4)),
                       ("tables", 5, i32(2)), ("tables", 6, i32(1)), ("tables", 8, i32(4)), ("tables", 9, i32(2)),
                       ("rope", 0, bf16(4, 8, 128)), ("rope", 0, bf16(5, 8, 64)), ("rope", 1, bf16(5, 3, 128)), ("rope", 2, i32(4)),
                       ("rope", 3, torch.ones(128, device="cuda")), ("rope", 4, bf16(5, 4, 128)), ("rope", 5, bf16(5, 8, 128)),
                       ("rope", 6, bf16(64)), ("rope", 0, bf16(5, 8, 256)[:, :, ::2]), ("rope", 0, bf16(5, 9, 128)[:, ::2]),
                       ("append", 0, bf16(5, 3, 128)), ("append", 1, bf16(4, 2, 128)), ("append", 2, i32(4)), ("append", 3, u8(4, 2, 16, 32)),
                       ("append", 4, u8(4, 2, 16, 3)), ("gather", 0, bf16(5, 2, 64)), ("gather", 5, u8(3, 2, 16, 64)),
                       ("gather", 6, u8(4, 2, 16, 8)), ("gather", 3, u8(4 * 2 * 16, 64)),
                       ("attention", 0, bf16(5, 8, 64)), ("attention", 0, bf16(4, 8, 128)), ("attention", 0, bf16(40, 128)),
                       ("attention", 5, i32(3, 4)), ("attention", 5, i32(8)), ("attention", 6, i32(2)), ("attention", 7, i32(3)),
                       ("attention", 8, bf16(5, 4, 128)), ("attention", 9, u8(1000))]:
        call, args = calls[name]
        assert call(*args[:i], y, *args[i + 1:]) is None, (name, i)
    expect(fg)


def test_native_calls_and_the_binding_agree(fg):
    """A call without a stream goes through the module, one with the current stream through the binding."""
    c = C.cache_case(77, [50, 300, 0], [3, 1, 0], 8, 2, 128, 16)
    out, ws = attend(fg, c)
    other, _ = attend(fg, c, ws=ws, stream=torch.cuda.current_stream())
    assert torch.equal(out, other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other, _ = attend(fg, c)
    side.synchronize()
    assert torch.equal(out, other)
    check(c, out)
    with pytest.raises(fg.FgError):
        attend(fg, c, scale=-1.0)
    with pytest.raises(ValueError):
        attend(fg, c, ws=ws[:1000])
    expect(fg)
