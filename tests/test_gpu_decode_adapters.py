"""The projection with per-token adapters where its adapters decide: results that are one value of
x @ lora_a^T (so that the low BF16 parts show), and single tokens that do have an adapter."""
import numpy as np
import pytest

import decode_cases as D
from test_gpu_decode import check, fg, lora_ref, run_lora  # noqa: F401  (fg: the fixture)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,l,r", [(1, 64, 128, 1, 8), (16, 64, 128, 5, 8), (33, 272, 256, 12, 16), (64, 256, 512, 60, 32),
                                       (150, 64, 128, 4, 64), (300, 272, 256, 3, 128)])
def test_every_part_of_the_adapters_products_counts(fg, m, n, k, l, r, out):  # noqa: F811
    c = D.parts_case(m + r, m, n, k, l, r)
    check(run_lora(fg, c, out), lora_ref(c, out), out)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,l,r", [(16, 128, 1, 8), (272, 512, 5, 16), (1008, 384, 3, 72), (48, 2048, 2, 128)])
def test_one_token_with_an_adapter(fg, n, k, l, r, out):  # noqa: F811
    c = D.lora_case(n + r, 1, n, k, l, r, none=0.0)
    assert c["ids"][0] >= 0
    check(run_lora(fg, c, out), lora_ref(c, out), out)


@pytest.mark.parametrize("sms", [1, 3])
def test_one_token_with_an_adapter_and_more_tiles_than_sms(fg, sms):  # noqa: F811
    c = D.lora_case(72, 1, 1600, 256, 5, 16, none=0.0)
    assert c["ids"][0] >= 0
    try:
        fg.set_num_sms(sms)
        check(run_lora(fg, c), lora_ref(c))
    finally:
        fg.set_num_sms(0)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,l,r", [(1, 272, 256, 1, 16), (20, 272, 256, 3, 8), (70, 144, 128, 5, 72), (150, 272, 256, 5, 16),
                                       (300, 528, 384, 3, 8), (300, 272, 128, 200, 16), (200, 528, 384, 60, 128)])
def test_workspace_for_the_adapters_there_are(fg, m, n, k, l, r, out):  # noqa: F811
    """A workspace of exactly the bytes that the call needs, between guards, with one byte less refused."""
    c = D.lora_case(m + l + r, m, n, k, l, r)
    dtype = torch.bfloat16 if out == "bf16" else torch.float32
    size = fg.lora_workspace(m, n, k, r, adapters=l, dtype=dtype).nbytes
    assert size <= fg.lora_workspace(m, n, k, r).nbytes
    buf = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[4096:4096 + size]
    ws.zero_()
    for _ in range(2):
        check(run_lora(fg, c, out, ws=ws), lora_ref(c, out), out)
    assert torch.all(buf[:4096] == 0xA5) and torch.all(buf[4096 + size:] == 0xA5)
    with pytest.raises(ValueError):
        run_lora(fg, c, out, ws=ws[:-1])
