"""The MoE MLP on a shard of the experts, call after call on one workspace: steps in which no
token uses an expert of the shard, at sizes whose tiles are cut (H of 2048 and more)."""
import numpy as np
import pytest

import decode_cases as D
from test_gpu_decode import check, fg, moe_inputs, moe_ref, run_moe  # noqa: F401  (fg: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

COUNTER_BYTES = 2 * 512 * 4          # the head of a workspace: both launches' arrival counters


def counters_are_zero(ws):
    return int(torch.count_nonzero(ws[:COUNTER_BYTES])) == 0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t", [1, 12, 40])
@pytest.mark.parametrize("h,i,e", [(2048, 256, 3), (4096, 128, 4), (7168, 128, 2), (1408, 256, 3)])
def test_calls_without_a_local_expert_leave_no_trace(fg, h, i, e, t, fp4):  # noqa: F811
    """Ordinary, empty, empty, one expert, ordinary: zeros from the empty calls, the counters back at
    zero behind every call, and the first call's bits again from the last."""
    c = D.moe_case(h + t, t, h, i, e, min(2, e), fp4=fp4, base=5)
    c["ids"] += 5
    args = moe_inputs(c)
    ws = fg.moe_mlp_workspace(t, h, i, e)
    first = run_moe(fg, c, ws=ws, args=args)
    check(first, moe_ref(c))
    assert counters_are_zero(ws)
    none = list(args)
    for away in (-1, 4, 5 + e):
        none[6] = torch.full_like(args[6], away)
        for out in ("bf16", "f32"):
            got = run_moe(fg, c, out, ws=ws, args=none)
            assert np.array_equal(got, np.zeros_like(got))
            assert counters_are_zero(ws)
    one = dict(c, ids=np.full_like(c["ids"], -1))
    one["ids"][:, 0] = 5 + e - 1
    check(run_moe(fg, one, ws=ws), moe_ref(one))
    assert counters_are_zero(ws)
    assert np.array_equal(run_moe(fg, c, ws=ws, args=args), first)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("t,sms", [(3, 3), (40, 4)])
def test_empty_calls_on_few_sms(fg, t, sms, fp4):  # noqa: F811
    """The same with more output tiles than SMs: neither clusters nor the third launch."""
    c = D.moe_case(t, t, 2048, 128, 2, 1, fp4=fp4)
    args = moe_inputs(c)
    ws = fg.moe_mlp_workspace(t, 2048, 128, 2)
    none = list(args)
    none[6] = torch.full_like(args[6], -1)
    try:
        fg.set_num_sms(sms)
        first = run_moe(fg, c, ws=ws, args=args)
        check(first, moe_ref(c))
        for _ in range(2):
            got = run_moe(fg, c, ws=ws, args=none)
            assert np.array_equal(got, np.zeros_like(got))
            assert counters_are_zero(ws)
        assert np.array_equal(run_moe(fg, c, ws=ws, args=args), first)
    finally:
        fg.set_num_sms(0)
