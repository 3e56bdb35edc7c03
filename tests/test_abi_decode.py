"""Refusals of the MoE decode operators on a host without a GPU: every bad argument is an
error code before anything is launched, and workspace sizes are plain host arithmetic."""
import pytest

FAKE = 1 << 20          # an aligned non-null "device" address; never dereferenced


@pytest.fixture(scope="module")
def fg():
    import moe_fp8_e4m3_gb300 as lib
    return lib


def route(fg, t=4, e=64, topk=4, groups=1, keep=1, score=0, logits=FAKE, bias=None, ids=FAKE, w=FAKE):
    return fg.lib.fg_moe_route(t, e, topk, groups, keep, score, 1, 1.0, logits, bias, ids, w, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), -1), (dict(e=0), -1), (dict(topk=0), -1), (dict(topk=65), -1), (dict(groups=0), -1),
    (dict(groups=5), -1), (dict(groups=4, keep=5), -1), (dict(groups=4, keep=0), -1),
    (dict(groups=8, keep=1, topk=9), -1), (dict(score=2), -1), (dict(logits=None), -1), (dict(ids=None), -1),
    (dict(w=FAKE + 2), -1), (dict(bias=FAKE + 1), -1), (dict(e=1025), -2), (dict(e=128, topk=33), -2),
    (dict(groups=64, keep=64), -2), (dict(t=0), 0),
])
def test_route_argument_errors(fg, kw, want):
    assert route(fg, **kw) == want


def moe(fg, fp4, t=4, h=256, i=128, e=8, topk=2, base=0, a=FAKE, sfa=FAKE, w13=FAKE, sf13=FAKE, w2=FAKE, sf2=FAKE,
        ids=FAKE, w=FAKE, d=FAKE, dtype=0, ws=FAKE):
    fn = fg.lib.fg_fp8_fp4_moe_mlp if fp4 else fg.lib.fg_fp8_moe_mlp
    return fn(t, h, i, e, topk, base, a, sfa, w13, sf13, w2, sf2, ids, w, d, dtype, ws, None)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), -1), (dict(h=200), -1), (dict(h=0), -1), (dict(i=64), -1), (dict(e=0), -1), (dict(topk=0), -1),
    (dict(base=-1), -1), (dict(dtype=3), -1), (dict(t=129), -2), (dict(e=1025), -2), (dict(topk=33), -2),
    (dict(a=None), -1), (dict(ws=None), -1), (dict(ws=FAKE + 128), -1), (dict(w2=FAKE + 8), -1), (dict(ids=FAKE + 2), -1),
    (dict(d=FAKE + 8), -1), (dict(sf2=FAKE + 4), -1), (dict(t=0), 0),
])
def test_moe_argument_errors(fg, fp4, kw, want):
    assert moe(fg, fp4, **kw) == want


def test_moe_fp4_weights_need_32_byte_alignment(fg):
    assert moe(fg, True, w13=FAKE + 16) == -1


def lora(fg, m=4, n=256, k=256, l=3, r=16, a=FAKE, sfa=FAKE, b=FAKE, sfb=FAKE, x=FAKE, la=FAKE, lb=FAKE, sc=FAKE, ids=FAKE,
         d=FAKE, dtype=0, ws=FAKE):
    return fg.lib.fg_fp8_gemm_nt_lora(m, n, k, l, r, a, sfa, b, sfb, x, la, lb, sc, ids, d, dtype, ws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(m=-1), -1), (dict(n=24), -1), (dict(n=0), -1), (dict(k=192), -1), (dict(l=0), -1), (dict(r=0), -1),
    (dict(r=12), -1), (dict(r=136), -1), (dict(m=65537), -1), (dict(dtype=2), -1), (dict(l=1025), -2),
    (dict(x=None), -1), (dict(la=FAKE + 8), -1), (dict(lb=FAKE + 2), -1), (dict(ids=None), -1), (dict(ws=FAKE + 16), -1),
    (dict(m=0), 0),
])
def test_lora_argument_errors(fg, kw, want):
    assert lora(fg, **kw) == want


def test_workspace_sizes(fg):
    L = fg.lib
    assert L.fg_moe_mlp_workspace(129, 256, 128, 8) == -1 and L.fg_moe_mlp_workspace(4, 100, 128, 8) == -1
    assert L.fg_lora_workspace(4, 250, 256, 16) == -1 and L.fg_lora_workspace(4, 256, 256, 7) == -1
    sizes = [L.fg_moe_mlp_workspace(t, 4096, 2048, 32) for t in (1, 16, 17, 64, 128)]
    assert sizes[0] <= sizes[1] < sizes[2] < sizes[3] < sizes[4]
    assert L.fg_lora_workspace(1, 4096, 4096, 16) < L.fg_lora_workspace(128, 4096, 4096, 16)


def test_no_device_fails_loudly(fg):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert route(fg) == fg.FG_ERR_CUDA
    assert moe(fg, False) == fg.FG_ERR_CUDA and moe(fg, True) == fg.FG_ERR_CUDA
    assert lora(fg) == fg.FG_ERR_CUDA


@pytest.mark.parametrize("fp4", [False, True])
def test_moe_experts_end_within_the_ids_type(fg, fp4):
    """Past it, ids from -2^31 on would count as experts of the shard."""
    for base in (2 ** 31 - 1, 2 ** 31 - 8):
        assert moe(fg, fp4, e=8, base=base) == fg.FG_ERR_INVALID_ARG
    assert moe(fg, fp4, t=0, e=8, base=2 ** 31 - 9) == fg.FG_OK
