"""Pins of the serving oracle: closed forms and definitions written out by hand."""
import numpy as np
import pytest

import serving_cases as C
from oracle import fp4 as FP4
from oracle import serving as O


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["k", "v"])
def test_rows_hold_every_element_once(d, kind):
    n = O.nibbles(d, kind)
    assert sorted(n) == list(range(d))
    b = d // 32
    for e in (0, 7, 33, d - 1):
        if kind == "k":
            assert n[e] == (e % 32 // 8 * b + e // 32) * 8 + e % 8
        else:
            assert n[e] == (e % 32 // 4 * b + e // 32) * 4 + e % 4


def test_codes_are_the_weight_quantisers_within_its_range():
    x = C.rng(3).standard_normal((40, 128)) * 2.0 ** C.rng(4).integers(-20, 20, (40, 1))
    x[7, 32:64] = 0.0
    codes, sf = O.encode(x)
    packed, s = FP4.quantize_mxfp4(x)
    assert np.array_equal(FP4.pack_fp4(codes), packed) and np.array_equal(sf, s)
    for kind in "kv":
        assert np.array_equal(O.decode(O.rows(codes, kind), sf, kind), FP4.dequant_mxfp4(packed, s))


def test_scales_are_clamped():
    x = np.zeros((3, 64))
    x[0, 0], x[0, 1] = 2.0 ** 100, -1.0
    x[1, 0] = 2.0 ** -63
    x[2, 40] = 2.0 ** -80
    codes, sf = O.encode(x)
    v = O.decode(O.rows(codes, "k"), sf, "k")
    assert v[0, 0] == 6 * 2.0 ** 63 and v[0, 1] == 0.0 and v[1, 0] == 2.0 ** -63 and not v[2].any()


def test_attention_of_equal_keys_is_the_mean():
    c = C.cache_case(1, [5, 1, 0], [2, 1, 0], 2, 1, 64, 16)
    c["q"][:] = 0.0
    out, bound, used = C.reference(c)
    v = O.cached(c["table"][0], 5, c["vc"], c["vs"], "v", 0)
    # five terms of |v| <= 32, each off by 2^-53 of itself twice (the weight, the sum): 5 * 32 * 2^-52
    np.testing.assert_allclose(out[0], np.broadcast_to(v[:4].mean(0), (2, 64)), rtol=0, atol=160 * 2.0 ** -52)
    np.testing.assert_allclose(out[1], np.broadcast_to(v.mean(0), (2, 64)), rtol=0, atol=160 * 2.0 ** -52)
    assert used.tolist() == [True] * 3 + [False] * 2 and (bound[:3] >= 0).all()
    out, _, _ = C.reference(c, window=1)
    np.testing.assert_allclose(out[1, 0], v[4], rtol=1e-12)


def test_attention_rows_before_the_first_key_are_zero():
    c = C.cache_case(2, [3], [3], 1, 1, 64, 16)
    c["start"] = np.array([0, 5], np.int32)                 # five rows, three keys: rows 0 and 1 stand before key 0
    out, _, _ = C.reference(c)
    assert not out[:2].any() and out[2:5].any(axis=(1, 2)).all()


def test_rotation_keeps_lengths_and_turns_by_the_angle():
    g = C.rng(5)
    x = g.standard_normal((4, 2, 64))
    angle = g.random((9, 16)) * 6
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    pos = np.array([0, 3, 8, 2])
    for inter in (False, True):
        y, bound = O.norm_rope(x, None, 0.0, pos, cs, inter)
        i = np.arange(16)
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + 16)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * angle[pos])[:, None]
        np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, rtol=1e-12)
        assert np.array_equal(y[..., 32:], x[..., 32:]) and (bound > 0).any()
    y, _ = O.norm_rope(x, np.full(64, 2.0), 0.0, pos, cs[:, :0], False)
    np.testing.assert_allclose((y * y).mean(-1), 4.0, rtol=1e-12)


def test_block_tables_by_hand():
    # pages of 4: request 0 goes on within its page and into a new one, 1 is finished, 2 waits, 3 begins
    out = O.block_tables([3, 5, 4, 0], [3, -1, 0, 5], [10, 11, -1, -1, -1], 2,
                         [[7, -1, -1], [8, 9, -1], [6, -1, -1], [-1, -1, -1]], 9, 4, 20)
    assert out["free"][:4].tolist() == [10, 11, 8, 9] and out["count"] == 1
    assert out["table"].tolist() == [[7, 9, -1], [8, 9, -1], [6, -1, -1], [8, 11, -1]]
    assert out["start"].tolist() == [0, 3, 3, 3, 8] and out["lens"].tolist() == [6, 0, 4, 5]
    assert out["slots"].tolist() == [31, 36, 37, 32, 33, 34, 35, 44, -1]
    assert out["positions"].tolist() == [3, 4, 5, 0, 1, 2, 3, 4, -1]
    assert O.block_tables([3], [6], [1], 1, [[0, 0, 0]], 9, 4, 20) is None       # two pages wanted, one free
    assert O.block_tables([3], [6], [1, 2], 2, [[0, 0]], 9, 4, 20) is None       # a row of two pages
    assert O.block_tables([3], [6], [1, 2], 2, [[0, 0, 0]], 5, 4, 20) is None    # five tokens at most
