"""How closely the bound of ``oracle.decode.lora`` (CPU) looks: x @ lora_a^T enters the second product as
BF16 parts, two for a BF16 result and three for an FP32 one, and a part that is left out is seen."""
import numpy as np
import pytest

import decode_cases as D
from oracle import decode as O
from oracle import formats as F


def with_parts(c, parts):
    """D in FP64 with x @ lora_a^T as a sum of that many BF16 parts, and nothing else rounded."""
    zero = dict(c, ids=np.full_like(c["ids"], -1))
    d = O.lora(*D.lora_args(zero))[0]
    for i, j in enumerate(c["ids"]):
        if 0 <= j < c["la"].shape[0]:
            rest = float(c["scaling"][j]) * (c["la"][j] @ c["x"][i])
            v = np.zeros_like(rest)
            for _ in range(parts):
                h = F.bf16_to_f64(F.f64_to_bf16(rest))
                v, rest = v + h, rest - h
            d[i] += c["lb"][j] @ v
    return d


def rounded(d, out):
    return F.bf16_to_f64(F.f64_to_bf16(d)) if out == "bf16" else d.astype(np.float32).astype(np.float64)


@pytest.mark.parametrize("out,needed", [("bf16", 2), ("f32", 3)])
@pytest.mark.parametrize("m,k,l,r", [(16, 128, 5, 8), (33, 256, 12, 16), (150, 128, 4, 64), (1, 128, 1, 8)])
def test_a_missing_part_is_seen(m, k, l, r, out, needed):
    c = D.parts_case(m + r, m, 64, k, l, r)
    ref = O.lora(*D.lora_args(c), out=out)
    assert O.within(rounded(with_parts(c, needed), out), ref, out).all()
    for parts in range(1, needed):
        assert not O.within(rounded(with_parts(c, parts), out), ref, out).all(), parts


@pytest.mark.parametrize("m,n,k,l,r", [(16, 1008, 256, 20, 16), (100, 256, 128, 7, 128), (200, 272, 640, 60, 128)])
def test_one_part_is_seen_among_ordinary_values(m, n, k, l, r):
    c = D.lora_case(m + n + l, m, n, k, l, r)
    assert not O.within(rounded(with_parts(c, 1), "f32"), O.lora(*D.lora_args(c), out="f32"), "f32").all()


def test_bound_of_a_row_does_not_grow_with_the_other_rows():
    c = D.lora_case(5, 40, 32, 256, 9, 16, none=0.0)
    alone = {k: (v[:1] if k in ("a", "x", "ids") else v) for k, v in c.items()}
    alone["sfa"] = c["sfa"][:, :4]
    many, one = O.lora(*D.lora_args(c))[1][0], O.lora(*D.lora_args(alone))[1][0]
    np.testing.assert_allclose(many, one, rtol=1e-12)
