"""The serving step's operators at the limits of their arguments: windows as large as their type, requests that claim
the same rows, pages of more than 2^30 tokens, value scales far apart within a token, scales that
leave no score, scores of any size."""
import numpy as np
import pytest

import serving_cases as C
from oracle import serving as O
from oracle.decode import within
from test_gpu_serving import attend, check, expect, f64, fg, tables  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# ---------------------------------------------------------------------------- windows
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 3, 40, 2 ** 30, 2 ** 31 - 4, 2 ** 31 - 1])
def test_windows_over_rows_before_the_first_key(fg, d, window):
    """Requests of more rows than cached tokens: rows before position 0 look at nothing, the others at what the window
    holds, however large it is."""
    c = C.cache_case(d + window % 97, [3, 0, 20, 9], [3, 0, 2, 9], 4, 2, d, 16, extra_rows=9)
    c["start"] = np.array([0, 9, 12, 14, 23], np.int32)
    out, _ = attend(fg, c, window)
    expect(fg)
    check(c, out, window)
    got = f64(out)
    assert not got[:6].any() and not got[9:12].any() and got[6:9].any(axis=(1, 2)).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq", [8, 32])
@pytest.mark.parametrize("window", [20, 2 ** 31 - 4, 2 ** 31 - 1])
def test_windows_over_many_rows_before_the_first_key(fg, d, hq, window):
    c = C.wide(C.cache_case(d + hq, [30, 90], [30, 40], hq, 1, d, 16, extra_rows=3 * 2048))
    c["start"] = np.array([0, 70, 110], np.int32)
    assert C.many_rows(c, window)
    out, _ = attend(fg, c, window)
    expect(fg)
    check(c, out, window)
    got = f64(out)
    assert not got[:40].any() and got[40:70].any(axis=(1, 2)).all()


# ------------------------------------------------------------- rows claimed more than once
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("s", [3, 300, 1000])
@pytest.mark.parametrize("tokens", [16, 1 << 18])
def test_a_few_rows_claimed_twice(fg, d, s, tokens):
    """query_start falls once and by little: requests 0 and 2 both claim rows 3 and 4, all requests together fewer rows
    than the call has.  Nothing is written, whatever the order of the two, and the next call is right."""
    new = [5, 0, 5] + [1] * (s - 3)
    c = C.wide(C.cache_case(s + d, [n + 3 for n in new], new, 4, 2, d, 16, extra_rows=40 * s if tokens > 16 else 8), tokens)
    assert C.many_rows(c) == (tokens > 16)
    start = c["start"].copy()
    start[2:] -= 2
    out, ws = attend(fg, dict(c, start=start))
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x10A)
    assert (f64(out) == -77).all()
    out, _ = attend(fg, c, ws=ws)
    expect(fg)
    check(c, out)


def test_many_chunks_a_request_and_rows_claimed_twice(fg):
    """Requests of more chunks than one thread walks take another way through the plan."""
    c = C.cache_case(31, [600, 20, 600], [600, 0, 600], 4, 1, 64, 16, extra_rows=8)
    c["start"] = np.array([0, 600, 598, 1198], np.int32)
    assert not C.many_rows(c)
    out, _ = attend(fg, c)
    expect(fg, fg.FG_ERR_DEVICE_CONTRACT, 0x10A)
    assert (f64(out) == -77).all()


# ------------------------------------------------------------------------- block tables
@pytest.mark.parametrize("page,width,context,new", [
    (2 ** 31 - 1, 1, [5, 0, 2 ** 31 - 4], [3, 0, 2]), (2 ** 30 + 16, 1, [2 ** 30, 7, 0], [9, -1, 1]),
    (2 ** 30 - 8, 2, [2 ** 30 - 9, 2 ** 30, 2 ** 31 - 20], [2, 1, -1]), (2 ** 29 + 1, 3, [2 ** 30, 2 ** 29 + 1, 2], [4, 1, 1])])
def test_block_tables_of_pages_past_2_30_tokens(fg, page, width, context, new):
    """Rounding up to pages passes 2^31 on the way: the tables are the oracle's all the same."""
    held = [-(-n // page) for n in context]
    table, at = np.full((3, width), -5), 0
    for r, n in enumerate(held):
        table[r, :n] = np.arange(at, at + n) % ((2 ** 31 - 1) // page)
        at += n
    c = {"context": context, "new": new, "free": [0] * 8, "count": 4, "table": table, "pages": (2 ** 31 - 1) // page}
    a = tables(fg, c, sum(max(n, 0) for n in new) + 2, page)
    expect(fg)
    check_block_tables(a, c, page)


def check_block_tables(a, c, page):
    """O.block_tables walks every position; here only the new ones are walked."""
    stack, table = list(c["free"][:c["count"]]), c["table"].copy()
    for r, n in enumerate(c["new"]):
        if n < 0:
            stack += [int(x) for x in table[r, :-(-c["context"][r] // page)]]
    free = np.array(stack + list(c["free"][len(stack):]))
    slots, positions, lens, start = [], [], [], [0]
    for r, n in enumerate(c["new"]):
        lens.append(c["context"][r] + n if n >= 0 else 0)
        for j in range(-(-c["context"][r] // page), -(-lens[r] // page)):
            table[r, j] = stack.pop()
        for pos in range(c["context"][r], lens[r]):
            slots.append(int(table[r, pos // page]) * page + pos % page)
            positions.append(pos)
        start.append(len(slots))
    spare = [-1] * (a["slots"].numel() - len(slots))
    assert a["slots"].tolist() == slots + spare and a["positions"].tolist() == positions + spare
    assert a["lens"].tolist() == lens and a["start"].tolist() == start and int(a["count_out"]) == len(stack)
    assert np.array_equal(a["table"].cpu().numpy(), table) and np.array_equal(a["free"].cpu().numpy(), free)


# ------------------------------------------------------ value scales far apart in a token
def values_apart(c, seed, spread, fall, tokens=None):
    """The case with values whose 32-element blocks differ by up to 2^(2 spread) within a token: anyhow, or (fall) from
    the first block down to the last one in every token; tokens: only these of every request."""
    g = C.rng(seed)
    d, hkv, page = c["d"], c["hkv"], c["page"]
    for r, n in enumerate(c["lens"]):
        t = np.arange(n) if tokens is None else np.array([i for i in tokens if i < n], np.int64)
        e = g.integers(-spread, spread + 1, (len(t), hkv, d // 32, 1))
        if fall:
            e[:] = np.linspace(spread, -spread, d // 32).round().astype(np.int64)[:, None]
        x = g.standard_normal((len(t), hkv, d // 32, 32)) * 2.0 ** e
        codes, sf = O.encode(x.reshape(len(t), hkv, d))
        p, o = c["table"][r, t // page], t % page
        c["vc"][p, :, o], c["vs"][p, :, o] = O.rows(codes, "v"), sf
    return c


def check_by_block(c, out, window=0):
    """A weight times a block's scale is off by 2^-11 of itself (2^-8 where the tensor cores take many rows) or by 2^-25
    of the largest such product of the same row and block; the exponent that both are taken of, up to 2^8, is off by 2^-17."""
    got = f64(out)
    weight = 2.0 ** (-8 if C.many_rows(c, window) else -11) + 2.0 ** -16
    for b in range(c["d"] // 32):
        # with block b's scales in the place of all, the oracle's largest product is block b's
        vs = np.repeat(c["vs"][..., b:b + 1], c["d"] // 32, -1)
        ref, bound, used = O.attention(c["q"], c["kc"], c["ks"], c["vc"], vs, c["table"], c["start"], c["lens"], c["d"] ** -0.5,
                                       window, weight, floor=2.0 ** -25)
        e = slice(32 * b, 32 * b + 32)
        bad = ~within(got[used][..., e], (ref[used][..., e], bound[used][..., e]), "bf16")
        assert not bad.any(), (b, bad.sum(), np.argwhere(bad)[:4], got[used][..., e][bad][:4], ref[used][..., e][bad][:4])


@pytest.mark.parametrize("d,hq", [(64, 1), (64, 16), (64, 32), (128, 8), (128, 16), (256, 5)])
@pytest.mark.parametrize("spread", [3, 12, 31])
@pytest.mark.parametrize("fall", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_value_scales_far_apart_within_a_token(fg, d, hq, spread, fall, window):
    c = values_apart(C.cache_case(d + hq + spread, [150, 17, 1, 0, 64], [2, 1, 1, 0, 3], hq, 1, d, 16), 5, spread, fall)
    out, _ = attend(fg, c, window)
    expect(fg)
    check_by_block(c, out, window)


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 16), (256, 8)])
@pytest.mark.parametrize("tokens", [[3], [130, 131], [299]])
def test_a_token_with_scales_far_apart_among_others(fg, d, hq, tokens):
    """One block of one token far above everything else: the other blocks keep the other tokens' digits."""
    c = values_apart(C.cache_case(d + tokens[0], [300, 300], [1, 1], hq, 1, d, 32), 7, 25, True, tokens)
    out, _ = attend(fg, c)
    expect(fg)
    check_by_block(c, out)


def test_value_blocks_of_zeros_beside_small_ones(fg):
    """A block of zeros has scale 1, however small its neighbours are."""
    c = C.cache_case(41, [200, 90], [1, 2], 8, 2, 128, 16)
    g = C.rng(41)
    for r, n in enumerate(c["lens"]):
        x = g.standard_normal((n, 2, 128)) * 2.0 ** -45
        x[:, :, 32:64] = 0.0
        codes, sf = O.encode(x)
        p, o = c["table"][r, np.arange(n) // 16], np.arange(n) % 16
        c["vc"][p, :, o], c["vs"][p, :, o] = O.rows(codes, "v"), sf
    out, _ = attend(fg, c)
    expect(fg)
    check_by_block(c, out)
    assert not out[:3, :, 32:64].any()


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 8), (128, 16), (256, 8)])
@pytest.mark.parametrize("fall", [False, True])
def test_value_scales_far_apart_over_a_long_context(fg, d, hq, fall):
    """Pieces of one item in several CTAs, their maxima far apart."""
    c = values_apart(C.cache_case(d + hq + 1, [5000], [1], hq, 1, d, 64), 9, 25, fall)
    out, ws = attend(fg, c)
    expect(fg)
    check_by_block(c, out)
    again, _ = attend(fg, c, ws=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("hq", [8, 32])
def test_many_rows_and_value_scales_far_apart(fg, hq):
    c = values_apart(C.wide(C.cache_case(hq, [150, 60], [70, 50], hq, 1, 128, 16)), 11, 31, True)
    assert C.many_rows(c)
    out, _ = attend(fg, c)
    expect(fg)
    check_by_block(c, out)


# -------------------------------------------------------------------- scores of any size
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [2.0 ** -23, 2.0 ** -40, 2.0 ** -126, 2.0 ** -149])
def test_scales_that_leave_no_score(fg, d, scale):
    """Queries of zeros and small ones, the smallest scales: every key that a row looks at counts the same, and no other."""
    c = C.cache_case(d, [37, 300, 5], [3, 1, 5], 4, 2, d, 16)
    c["q"][0] = 0.0
    c["q"][1] *= 2.0 ** -120
    c["q_bits"], c["q"] = O.bf16(c["q"])
    for many in (False, True):
        if many:
            c = C.wide(dict(c, q=np.concatenate([c["q"]] + [c["q"][:1]] * 300), q_bits=np.concatenate([c["q_bits"]] + [c["q_bits"][:1]] * 300)))
            assert C.many_rows(c)
        out, _ = attend(fg, c, scale=scale)
        expect(fg)
        check(c, out, scale=scale)


def peaked(c, sign, power, tie):
    """Keys 2^-min(|j - middle|, tie) in every element, queries of one value, `sign` times 2^power to 2^(power + 1), in every
    element of a row: scores differ by at least a factor of two, so that a row's output is the mean of the values whose
    score is the largest, the middle key's or (sign -1) the farthest ones'.  Returns the outputs' exact values."""
    d, page = c["d"], c["page"]
    c["q"][:] = sign * 2.0 ** power * (1 + C.rng(power).integers(0, 128, c["q"].shape[:2] + (1,)) / 128)
    c["q_bits"], c["q"] = O.bf16(c["q"])
    out = np.zeros(c["q"].shape)
    for r, n in enumerate(c["lens"]):
        j = np.arange(n)
        level = -np.minimum(np.abs(j - n // 2), tie)
        codes, sf = O.encode(np.broadcast_to((2.0 ** level)[:, None, None], (n, c["hkv"], d)))
        p, o = c["table"][r, j // page], j % page
        c["kc"][p, :, o], c["ks"][p, :, o] = O.rows(codes, "k"), sf
        t0, new = c["start"][r], c["start"][r + 1] - c["start"][r]
        for h in range(c["hkv"]):
            v = O.cached(c["table"][r], n, c["vc"], c["vs"], "v", h)
            for i in range(new):
                s = sign * level[:n - new + i + 1]
                top = np.flatnonzero(s == s.max(initial=-99))
                group = c["hq"] // c["hkv"]
                out[t0 + i, h * group:(h + 1) * group] = v[top].mean(0) if len(top) else 0.0
    return out


def check_peaked(c, out, want):
    """The other weights are 2^-(2^18) of the largest and less.  Each of up to n equal weights and their sum is rounded
    to FP32, a weight (times a scale) to FP16 or BF16: a term of up to n is off by at most 2^-8 of |v| together."""
    got, n = f64(out), int(c["start"][-1])
    size = max(np.abs(want[:n]).max(), 2.0 ** -8)
    assert np.isfinite(got[:n]).all()
    assert (np.abs(got[:n] - want[:n]) <= 2.0 ** -8 * np.abs(want[:n]) + 2.0 ** -8 * 24.0 * size).all(), np.abs(got[:n] - want[:n]).max()


@pytest.mark.parametrize("d,hq", [(64, 8), (64, 32), (128, 8), (128, 16), (256, 8)])
@pytest.mark.parametrize("power", [18, 24, 27, 30, 50, 100, 110])
@pytest.mark.parametrize("sign,tie", [(1, 8), (-1, 8), (1, 0)])
def test_scores_of_any_size(fg, d, hq, power, sign, tie):
    c = C.cache_case(d + hq, [1, 37, 300], [1, 2, 1], hq, 1, d, 16, spread=0)
    want = peaked(c, sign, power, tie)
    out, _ = attend(fg, c)
    expect(fg)
    check_peaked(c, out, want)


@pytest.mark.parametrize("d,hq", [(64, 8), (128, 8), (128, 32), (256, 8)])
@pytest.mark.parametrize("power", [18, 24, 30, 50, 100, 110])
@pytest.mark.parametrize("sign,tie", [(1, 8), (-1, 8), (1, 0)])
def test_many_rows_and_scores_of_any_size(fg, d, hq, power, sign, tie):
    c = C.wide(C.cache_case(d + hq, [70, 300], [70, 60], hq, 1, d, 16, spread=0))
    assert C.many_rows(c)
    want = peaked(c, sign, power, tie)
    out, _ = attend(fg, c)
    expect(fg)
    check_peaked(c, out, want)
