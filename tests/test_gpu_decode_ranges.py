"""The MoE decode operators at the ends of their number ranges."""
import numpy as np
import pytest

import decode_cases as D
from oracle import decode as O
from test_gpu_decode import ROUTE_RTOL, check, fg, lora_ref, run_lora, run_route  # noqa: F401  (fg: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


# exp of a difference of logits: FP32 rounds the difference (below 128) to 2^-18 at worst, which the
# exponential passes on to the weight
FAR_RTOL = ROUTE_RTOL + 2.0 ** -18


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
@pytest.mark.parametrize("level", [-87.5, -88.5, -100.0, -300.0])
def test_route_weights_of_scores_below_fp32(fg, score, biased, groups, keep, level):  # noqa: F811
    """Renormalised weights are ratios of the chosen scores, whatever the scores' size: all logits far
    below zero, and (with a bias that chooses them) far below the row's largest."""
    g = D.rng(int(-level) + groups)
    e, t, topk = 40, 6, 4
    x = np.stack([level + g.permutation(e) / 8.0 - 2.5 for _ in range(t)])
    x[1] = level                                            # all equal
    x[2, :20] -= 60.0
    x[3, 7] = -20.0
    bias = g.permutation(e) * 4.0 if biased else None
    if biased:
        x[4, int(np.argmin(bias))] = 3.0                    # the row's largest, not chosen
    ids, w = run_route(fg, x, topk, bias, score=score, n_group=groups, topk_group=keep)
    x32 = x.astype(np.float32).astype(np.float64)
    rid, rw = O.route(x32, topk, bias, score, groups, keep)
    assert np.array_equal(ids, rid)
    np.testing.assert_allclose(w, rw, rtol=FAR_RTOL, atol=2.0 ** -149)
    np.testing.assert_allclose(w.sum(axis=1), 1.0, rtol=1e-5)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m", [3, 20, 200])
def test_adapter_products_between_bf16_and_fp32_range(fg, m, out):  # noqa: F811
    """scaling * x @ lora_a^T above the largest BF16 value: its parts are finite, and so is the result."""
    c = D.lora_case(81 + m, m, 32, 128, 2, 8, none=0.0)
    x = np.zeros((m, 128))
    x[:, 0] = 1.0
    x[1::2, 0] = -1.0
    c["x_bits"], c["x"] = D.bf16(x)
    c["la_bits"], c["la"] = D.bf16(np.ones_like(c["la"]))
    lb = np.zeros_like(c["lb"])
    lb[:, :, 3] = 2.0 ** -20
    c["lb_bits"], c["lb"] = D.bf16(lb)
    c["scaling"][:] = [3.4e38, 3.397e38]
    got = run_lora(fg, c, out)
    assert np.isfinite(got).all()
    check(got, lora_ref(c, out), out)
