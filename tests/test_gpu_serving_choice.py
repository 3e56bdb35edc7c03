"""Which kernel an attention call over the 4-bit cache takes, as the library prints it: ``serving_cases.many_rows`` states
the rule a second time and sets the other tests' tolerances, so both sides of every border are launched once (lengths of
zero: only the printed choice is looked at here)."""
import re

import numpy as np
import pytest

import serving_cases as C

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def fg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_fp8_e4m3_gb300 as lib
    return lib


def sizes(d, s, hq, hkv, tokens, new):
    return {"d": d, "hq": hq, "hkv": hkv, "page": 16, "lens": [0] * s, "q": range(s * new), "table": np.zeros((s, tokens // 16))}


def launched(fg, capfd, c, window):
    """(rows of an item, whether the tensor-core kernel runs)"""
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    t, s = len(c["q"]), len(c["lens"])
    q = torch.zeros(t, c["hq"], c["d"], dtype=torch.bfloat16, device="cuda")
    ws = fg.paged_attention_workspace(t, s, c["hq"], c["hkv"], c["d"])
    capfd.readouterr()
    fg.paged_attention_mxfp4(q, *fg.kv_cache_mxfp4(2, c["hkv"], 16, c["d"]), i32(*c["table"].shape), i32(s + 1), i32(s), q.clone(), ws,
                             window=window)
    torch.cuda.synchronize()
    line = [x for x in capfd.readouterr().err.splitlines() if x.startswith("[fg] paged_attention_mxfp4")][-1]
    return int(re.search(r"rows=(\d+)", line).group(1)), line.endswith("(tcgen05)")


def few_rows(d, rows):
    return min(8 if rows <= 8 else 16 if rows <= 16 else 32, {64: 32, 128: 16, 256: 8}[d])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("s,hq,hkv,tokens,window", [(1, 8, 1, 8192, 0), (16, 32, 4, 8192, 0), (4, 64, 8, 131072, 0), (64, 6, 2, 512, 0),
                                                    (16, 16, 8, 131072, 1024), (1024, 4, 4, 1024, 0)])
def test_both_sides_of_the_choice(fg, capfd, monkeypatch, d, s, hq, hkv, tokens, window):
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    group = hq // hkv
    new = next(n for n in range(1, 5000) if C.many_rows(sizes(d, s, hq, hkv, tokens, n), window))
    assert new > 1
    rows, tensor_cores = launched(fg, capfd, sizes(d, s, hq, hkv, tokens, new - 1), window)
    assert not tensor_cores and rows == few_rows(d, (new - 1) * group)
    rows, tensor_cores = launched(fg, capfd, sizes(d, s, hq, hkv, tokens, new), window)
    assert tensor_cores and rows == (256 if d <= 128 and new * group >= 512 else 128)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_both_sides_of_256_rows(fg, capfd, monkeypatch, d):
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    for new, rows in ((511, 128), (512, 256 if d <= 128 else 128)):
        assert launched(fg, capfd, sizes(d, 2, 4, 4, 8192, new), 0) == (rows, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32])
def test_row_tiles_of_few_rows(fg, capfd, monkeypatch, d, rows):
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    assert launched(fg, capfd, sizes(d, 3, rows, 1, 8192, 1), 0) == (few_rows(d, rows), False)


def test_many_requests_take_the_kernel_of_few_rows(fg, capfd, monkeypatch):
    monkeypatch.setenv("FG_PRINT_CONFIGS", "1")
    c = sizes(128, 1025, 8, 1, 8192, 16)
    assert not C.many_rows(c) and launched(fg, capfd, c, 0) == (16, False)
