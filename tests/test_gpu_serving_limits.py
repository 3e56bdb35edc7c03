"""The serving step's operators at the limits of their arguments: windows as large as their type, requests that claim
the same rows, pages of more than 2^30 tokens."""
import numpy as np
import pytest

import serving_cases as C
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
