"""Refusals of the attention side of a serving step on a host without a GPU: every bad argument is an error
code before anything is launched, and the Python binding names tensors that do not fit."""
import pytest

from test_binding_decode import Fake

torch = pytest.importorskip("torch")
FAKE = 1 << 20          # an aligned non-null "device" address; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def fg():
    import moe_fp8_e4m3_gb300 as lib
    return lib


def tables(fg, s=4, t=8, page=16, pages=10, width=5, free=10, **kw):
    names = ["context", "new", "free_pages", "count", "table", "start", "lens", "slots", "positions", "count_out"]
    return fg.lib.fg_build_block_tables(s, t, page, pages, width, free, *[kw.get(n, FAKE) for n in names], None)


@pytest.mark.parametrize("kw,want", [
    (dict(s=-1), -1), (dict(t=-1), -1), (dict(page=0), -1), (dict(pages=0), -1), (dict(width=0), -1), (dict(free=-1), -1),
    (dict(page=2 ** 20, pages=2 ** 12), -1), (dict(page=2 ** 20, width=2 ** 12), -1), (dict(s=4001), -2), (dict(t=2 ** 18 + 1), -2),
    (dict(width=2 ** 18 + 1), -2), (dict(free=2 ** 30 + 1), -2), (dict(context=None), -1), (dict(new=None), -1), (dict(free_pages=None), -1),
    (dict(count=None), -1), (dict(table=None), -1), (dict(start=None), -1), (dict(lens=None), -1), (dict(slots=None), -1),
    (dict(positions=None), -1), (dict(count_out=None), -1), (dict(table=FAKE + 2), -1), (dict(slots=FAKE + 1), -1)])
def test_block_tables_argument_errors(fg, kw, want):
    assert tables(fg, **kw) == want


def rope(fg, t=4, hq=4, hkv=2, d=128, rot=64, far=100, q=FAKE, qs=512, k=FAKE, ks=256, qw=FAKE, kw=FAKE, eps=1e-6, pos=FAKE,
         cs=FAKE, qo=FAKE, qos=512, ko=FAKE, kos=256):
    return fg.lib.fg_qk_norm_rope(t, hq, hkv, d, rot, far, q, qs, k, ks, qw, kw, eps, pos, cs, 0, qo, qos, ko, kos, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), -1), (dict(hq=0), -1), (dict(hkv=-1), -1), (dict(d=0), -1), (dict(d=100), -1), (dict(rot=-16), -1),
    (dict(rot=144), -1), (dict(rot=24), -1), (dict(far=0), -1), (dict(eps=-1.0), -1), (dict(eps=NAN), -1), (dict(qs=504), -1),
    (dict(qs=516), -1), (dict(ks=255), -1), (dict(qos=500), -1), (dict(kos=260), -1), (dict(d=264, qs=1056, ks=528, qos=1056, kos=528), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(pos=None), -1), (dict(cs=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(q=FAKE + 8), -1), (dict(kw=FAKE + 2), -1), (dict(cs=FAKE + 4), -1), (dict(pos=FAKE + 1), -1), (dict(t=0), 0)])
def test_norm_rope_argument_errors(fg, kw, want):
    assert rope(fg, **kw) == want


def kv(fg, gather, t=4, heads=2, d=128, page=16, pages=10, k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE, kc=FAKE, ksf=FAKE,
       vc=FAKE, vsf=FAKE):
    if gather:
        return fg.lib.fg_kv_gather_mxfp4(t, heads, d, page, pages, slots, kc, ksf, vc, vsf, k, ks, v, vs, None)
    return fg.lib.fg_kv_append_mxfp4(t, heads, d, page, pages, k, ks, v, vs, slots, kc, ksf, vc, vsf, None)


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), -1), (dict(heads=0), -1), (dict(d=0), -1), (dict(page=0), -1), (dict(pages=0), -1), (dict(page=2 ** 20, pages=2 ** 12), -1),
    (dict(ks=248), -1), (dict(vs=257), -1), (dict(d=96), -2), (dict(d=512, ks=1024, vs=1024), -2), (dict(page=24), -2),
    (dict(k=None), -1), (dict(v=FAKE + 8), -1), (dict(slots=None), -1), (dict(kc=None), -1), (dict(ksf=FAKE + 4), -1),
    (dict(vc=FAKE + 8), -1), (dict(vsf=None), -1), (dict(t=0), 0)])
def test_cache_argument_errors(fg, gather, kw, want):
    assert kv(fg, gather, **kw) == want


def attention(fg, t=4, s=2, hq=8, hkv=2, d=128, page=16, pages=10, width=5, scale=0.1, window=0, **kw):
    names = ["q", "kc", "ks", "vc", "vs", "table", "start", "lens"]
    return fg.lib.fg_paged_attention_mxfp4(t, s, hq, hkv, d, page, pages, width, *[kw.get(n, FAKE) for n in names], scale, window,
                                           kw.get("out", FAKE), kw.get("ws", FAKE), None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), -1), (dict(s=-1), -1), (dict(hq=0), -1), (dict(hkv=0), -1), (dict(hq=7), -1), (dict(d=0), -1), (dict(page=0), -1),
    (dict(pages=0), -1), (dict(width=0), -1), (dict(window=-1), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=NAN), -1),
    (dict(scale=INF), -1), (dict(page=2 ** 20, pages=2 ** 12), -1), (dict(page=2 ** 20, width=2 ** 12), -1), (dict(d=96), -2),
    (dict(page=24), -2), (dict(s=4097), -2), (dict(t=2 ** 18 + 1), -2), (dict(hq=514), -2), (dict(q=None), -1), (dict(kc=None), -1),
    (dict(ks=FAKE + 8), -1), (dict(vc=FAKE + 8), -1), (dict(vs=None), -1), (dict(table=None), -1), (dict(start=FAKE + 2), -1),
    (dict(lens=None), -1), (dict(out=None), -1), (dict(ws=None), -1), (dict(ws=FAKE + 128), -1), (dict(t=0), 0), (dict(s=0), 0)])
def test_attention_argument_errors(fg, kw, want):
    assert attention(fg, **kw) == want


def test_calls_with_their_arguments_in_one_record(fg):
    """A record reaches the entry point that it names, word by word: each bad argument is the one that is found."""
    call, n = fg.lib.fg_call, FAKE
    assert call(-1, b"") == -1 and call(5, bytes(200)) == -1 and call(0, None) == -1
    tables_ok = [4, 8, 16, 10, 5, 10] + [n] * 10 + [0]
    rope_ok = [4, 4, 2, 128, 64, 100, n, 512, n, 256, n, n, 1e-6, n, n, 0, n, 512, n, 256, 0]
    append_ok = [4, 2, 128, 16, 10, n, 256, n, 256] + [n] * 5 + [0]
    gather_ok = [4, 2, 128, 16, 10] + [n] * 6 + [256, n, 256, 0]
    attention_ok = [4, 2, 8, 2, 128, 16, 10, 5] + [n] * 8 + [0.1, 0, n, n, 0]
    bad = {"int": -1, "ptr": n + 2, "stride": 17, "float": NAN}
    for i, (args, form, kinds) in enumerate([
            (tables_ok, fg._TABLES_ARGS, "iiiiii" + "p" * 10), (rope_ok, fg._ROPE_ARGS, "iiiiiipspsppfpp.psps"),
            (append_ok, fg._APPEND_ARGS, "iiiiipspsppppp"), (gather_ok, fg._APPEND_ARGS, "iiiiippppppsps"),
            (attention_ok, fg._ATTENTION_ARGS, "iiiiiiii" + "p" * 8 + "fipp")]):
        assert call(i, form.pack(*args)) in (fg.FG_OK, fg.FG_ERR_CUDA) if not torch.cuda.is_available() else True
        for j, kind in enumerate(kinds):
            if kind == ".":
                continue
            wrong = bad[{"i": "int", "p": "ptr", "s": "stride", "f": "float"}[kind]]
            assert call(i, form.pack(*args[:j], wrong, *args[j + 1:])) == -1, (i, j)
    # sizes past 32 bits are refused, not cut
    assert call(4, fg._ATTENTION_ARGS.pack(*([2 ** 32 + 4] + attention_ok[1:]))) == -1


def test_workspace_sizes(fg):
    size = fg.lib.fg_paged_attention_workspace
    assert size(4, 2, 7, 2, 128) == -1 and size(-1, 2, 8, 2, 128) == -1 and size(4, 2, 8, 2, 96) == -1
    assert 0 < size(1, 1, 8, 1, 128) == size(63, 7, 1, 1, 64) == size(1, 0, 1, 1, 256) < size(64, 1, 1, 1, 128) < size(64, 1, 1, 1, 256)
    for hq in (1, 8, 64):                   # what serves many rows serves fewer, of any number of requests
        for d in (64, 128, 256):
            sizes = [size(t, s, hq, 1, d) for t in (1, 4, 7, 8, 31, 32, 63, 64, 255, 256, 8192) for s in (1, 4096)]
            assert sizes == sorted(sizes)


def test_no_device_fails_loudly(fg):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert {tables(fg), rope(fg), kv(fg, False), kv(fg, True), attention(fg)} == {fg.FG_ERR_CUDA}


# ---------------------------------------------------------------------------- binding
BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


class Strided(Fake):
    """A stand-in with strides; contiguous in its last two dimensions unless told otherwise."""

    def __init__(self, *shape, dtype=BF, first=None, inner=1):
        super().__init__(*shape, dtype=dtype, contiguous=first is None and inner == 1)
        self.first, self.inner = first, inner

    def stride(self):
        t, h, d = self.shape
        return (h * d if self.first is None else self.first), d * self.inner, self.inner


def i32(*shape):
    return Fake(*shape, dtype=I32)


@pytest.fixture
def stub(fg, monkeypatch):
    fg.calls = 0

    def call(*args):
        fg.calls += 1
        return fg.FG_OK

    monkeypatch.setattr(fg, "_call", call)
    return fg


def cache(pages=10, heads=2, page=16, d=128):
    return {"k_cache": Fake(pages, heads, page, d // 2), "k_sf": Fake(pages, heads, page, d // 32),
            "v_cache": Fake(pages, heads, page, d // 2), "v_sf": Fake(pages, heads, page, d // 32)}


ARGS = {
    "build_block_tables": lambda fg: dict(
        context_lens=i32(4), new_lens=i32(4), free_pages=i32(9), free_count=i32(1), block_table=i32(4, 6), query_start=i32(5),
        seq_lens=i32(4), slots=i32(7), positions=i32(7), free_count_out=i32(1), page_size=16, num_pages=9),
    "qk_norm_rope": lambda fg: dict(
        q=Strided(5, 4, 128, first=1024), k=Strided(5, 2, 128, first=1024), positions=i32(5), cos_sin=Fake(50, 64, dtype=F32),
        q_out=Strided(5, 4, 128), k_out=Strided(5, 2, 128), q_weight=Fake(128, dtype=BF), k_weight=Fake(128, dtype=BF)),
    "kv_append_mxfp4": lambda fg: dict(k=Strided(5, 2, 128, first=512), v=Strided(5, 2, 128), slots=i32(5), **cache()),
    "kv_gather_mxfp4": lambda fg: dict(k=Strided(5, 2, 128, first=512), v=Strided(5, 2, 128), slots=i32(5), **cache()),
    "paged_attention_mxfp4": lambda fg: dict(
        q=Fake(5, 8, 128, dtype=BF), block_table=i32(3, 6), query_start=i32(4), seq_lens=i32(3), out=Fake(5, 8, 128, dtype=BF),
        workspace=Fake(fg.lib.fg_paged_attention_workspace(5, 3, 8, 2, 128)), **cache()),
}

WRONG = [
    ("build_block_tables", dict(new_lens=i32(3))), ("build_block_tables", dict(query_start=i32(4))), ("build_block_tables", dict(positions=i32(6))),
    ("build_block_tables", dict(free_count=i32(2))), ("build_block_tables", dict(seq_lens=i32(5))),
    ("build_block_tables", dict(slots=Fake(7, dtype=torch.int64))), ("build_block_tables", dict(block_table=Fake(4, 6, dtype=I32, contiguous=False))),
    ("qk_norm_rope", dict(k=Strided(4, 2, 128))), ("qk_norm_rope", dict(q_out=Strided(5, 4, 64))), ("qk_norm_rope", dict(q=Strided(5, 4, 128, inner=2))),
    ("qk_norm_rope", dict(q=Strided(5, 4, 128, dtype=F32))), ("qk_norm_rope", dict(q_weight=Fake(64, dtype=BF))),
    ("qk_norm_rope", dict(k_weight=Fake(128, dtype=F32))), ("qk_norm_rope", dict(positions=i32(4))), ("qk_norm_rope", dict(cos_sin=Fake(50, 64, dtype=BF))),
    ("kv_append_mxfp4", dict(k=Strided(5, 3, 128))), ("kv_append_mxfp4", dict(v=Strided(5, 2, 64))), ("kv_append_mxfp4", dict(slots=i32(4))),
    ("kv_append_mxfp4", dict(k_sf=Fake(10, 2, 16, 2))), ("kv_append_mxfp4", dict(v_cache=Fake(9, 2, 16, 64))),
    ("kv_append_mxfp4", dict(v_sf=Fake(10, 2, 16, 4, dtype=I32))), ("kv_gather_mxfp4", dict(v=Strided(4, 2, 128))),
    ("kv_gather_mxfp4", dict(k_cache=Fake(10, 2, 16, 64, contiguous=False))), ("kv_gather_mxfp4", dict(k_sf=Fake(10, 2, 8, 4))),
    ("paged_attention_mxfp4", dict(q=Fake(5, 8, 64, dtype=BF))), ("paged_attention_mxfp4", dict(out=Fake(4, 8, 128, dtype=BF))),
    ("paged_attention_mxfp4", dict(query_start=i32(3))), ("paged_attention_mxfp4", dict(seq_lens=i32(4))),
    ("paged_attention_mxfp4", dict(workspace=Fake(4096))), ("paged_attention_mxfp4", dict(out=Fake(5, 8, 128, dtype=F32))),
    ("paged_attention_mxfp4", dict(block_table=Fake(3, 6, dtype=I32, contiguous=False))), ("paged_attention_mxfp4", dict(v_sf=Fake(10, 2, 16, 2))),
]


@pytest.mark.parametrize("name", list(ARGS))
def test_binding_takes_the_documented_shapes(stub, name):
    getattr(stub, name)(**ARGS[name](stub), stream=0)
    assert stub.calls == 1


@pytest.mark.parametrize("name,wrong", WRONG)
def test_binding_refuses_other_shapes_and_types(stub, name, wrong):
    with pytest.raises((ValueError, TypeError)):
        getattr(stub, name)(**dict(ARGS[name](stub), **wrong), stream=0)
    assert stub.calls == 0


# ------------------------------------------------------------------- the module in C++
def test_native_calls_leave_what_they_do_not_take_to_the_binding(fg):
    bind = fg._native()
    i32, b16, u8, f32 = (lambda *n, t=t: torch.zeros(n, dtype=t) for t in (I32, BF, torch.uint8, F32))
    tensors = [i32(2), i32(2), i32(9), i32(1), i32(2, 4), i32(3), i32(2), i32(5), i32(5), i32(1)]
    caches = [u8(4, 2, 16, 64), u8(4, 2, 16, 4)] * 2
    k = b16(5, 2, 128)
    calls = [(bind.tables, tensors + [16, 9]), (bind.rope, [k, k, i32(5), f32(9, 128), k, k, None, None, 1e-6, False]),
             (bind.append, [k, k, i32(5)] + caches), (bind.gather, [k, k, i32(5)] + caches),
             (bind.attention, [k] + caches + [i32(2, 4), i32(3), i32(2), k, u8(1 << 24), None, 0])]
    for call, args in calls:
        assert call(*args) is None                          # tensors of the CPU
        assert call(*args[:-1]) is None and call(*args, None) is None and call() is None
        assert call(*([None] * len(args))) is None and call(*([2 ** 70] * len(args))) is None
