"""Shapes that the Python binding of the MoE decode operators refuses, on a host without a GPU: the
tensors are stand-ins with a shape and a dtype, and the library call behind the binding is a stub
that must not be reached with arrays that are smaller than what a kernel reads."""
import pytest

torch = pytest.importorskip("torch")


class Fake:
    """What the binding asks of a CUDA tensor."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.uint8, contiguous=True):
        self.shape, self.dtype, self.contiguous = torch.Size(shape), dtype, contiguous

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.shape.numel()

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20


def align4(x):
    return (x + 3) // 4 * 4


def i32(*shape):
    return Fake(*shape, dtype=torch.int32)


@pytest.fixture
def fg(monkeypatch):
    import moe_fp8_e4m3_gb300 as lib
    lib.calls = 0

    def stub(*args):
        lib.calls += 1
        return lib.FG_OK

    for name in ("fg_fp8_moe_mlp", "fg_fp8_fp4_moe_mlp", "fg_fp8_gemm_nt_lora"):
        monkeypatch.setattr(lib.lib, name, stub)
    return lib


def moe_args(fg, fp4, t=5, h=640, i=384, e=3, topk=2):
    kw, k2 = (h // 2, i // 2) if fp4 else (h, i)
    sf13, sf2 = ((e, h // 128, align4(2 * i)), (e, i // 128, align4(h))) if fp4 else \
        ((e, (h + 511) // 512, align4(2 * i // 128)), (e, (i + 511) // 512, align4(h // 128)))
    return {"a": Fake(t, h), "sfa": i32((h + 511) // 512, align4(t)), "w13": Fake(e, 2 * i, kw), "sf13": i32(*sf13),
            "w2": Fake(e, h, k2), "sf2": i32(*sf2), "topk_ids": i32(t, topk), "topk_weights": Fake(t, topk, dtype=torch.float32),
            "d": Fake(t, h, dtype=torch.bfloat16), "workspace": Fake(fg.lib.fg_moe_mlp_workspace(t, h, i, e))}


def call_moe(fg, fp4, args):
    (fg.fp8_fp4_moe_mlp if fp4 else fg.fp8_moe_mlp)(**args, stream=0)


@pytest.mark.parametrize("fp4", [False, True])
def test_moe_takes_the_documented_shapes(fg, fp4):
    call_moe(fg, fp4, moe_args(fg, fp4))
    for t, h, i, e, topk in ((1, 128, 128, 1, 1), (128, 1408, 640, 60, 4), (4, 512, 512, 2, 2)):
        call_moe(fg, fp4, moe_args(fg, fp4, t, h, i, e, topk))
    assert fg.calls == 4


@pytest.mark.parametrize("fp4", [False, True])
def test_moe_refuses_weights_of_the_other_kind(fg, fp4):
    args = moe_args(fg, fp4)
    other = moe_args(fg, not fp4)
    for names in (("w13",), ("w2",), ("w13", "w2"), ("w13", "sf13", "w2", "sf2")):
        with pytest.raises(ValueError):
            call_moe(fg, fp4, dict(args, **{n: other[n] for n in names}))
    assert fg.calls == 0


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("name", ["w13 K", "w2 K", "w13 rows", "sfa", "sf13", "sf2", "workspace bytes", "workspace strided"])
def test_moe_refuses_arrays_that_are_too_small(fg, fp4, name):
    args = moe_args(fg, fp4)
    half = 2 if fp4 else 1
    args.update({
        "w13 K": lambda: {"w13": Fake(3, 768, 512 // half)},
        "w2 K": lambda: {"w2": Fake(3, 640, 256 // half)},
        "w13 rows": lambda: {"w13": Fake(3, 769, 640 // half)},
        "sfa": lambda: {"sfa": i32(1, 8)},
        "sf13": lambda: {"sf13": i32(2, *args["sf13"].shape[1:])},
        "sf2": lambda: {"sf2": i32(3, 1, 4)},
        "workspace bytes": lambda: {"workspace": Fake(args["workspace"].nbytes - 1)},
        "workspace strided": lambda: {"workspace": Fake(args["workspace"].nbytes, contiguous=False)},
    }[name]())
    if name == "sf2" and not fp4:
        args["sf2"] = i32(3, 1, 7)
    with pytest.raises(ValueError):
        call_moe(fg, fp4, args)
    assert fg.calls == 0


def lora_args(fg, m=5, n=272, k=640, l=3, r=16):
    bf = torch.bfloat16
    return {"a": Fake(m, k), "sfa": i32((k + 511) // 512, align4(m)), "b": Fake(n, k),
            "sfb": i32((k + 511) // 512, align4((n + 127) // 128)), "x": Fake(m, k, dtype=bf), "lora_a": Fake(l, r, k, dtype=bf),
            "lora_b": Fake(l, n, r, dtype=bf), "scaling": Fake(l, dtype=torch.float32), "ids": i32(m), "d": Fake(m, n, dtype=bf),
            "workspace": Fake(fg.lib.fg_lora_workspace(m, n, k, r))}


def test_lora_takes_the_documented_shapes(fg):
    fg.fp8_gemm_nt_lora(**lora_args(fg), stream=0)
    fg.fp8_gemm_nt_lora(**lora_args(fg, 1, 16, 128, 1, 8), stream=0)
    fg.fp8_gemm_nt_lora(**lora_args(fg, 300, 1600, 1024, 9, 128), stream=0)
    assert fg.calls == 3


@pytest.mark.parametrize("name,small", [
    ("sfa", (1, 8)), ("sfb", (2, 3)), ("workspace", None), ("lora_b", (3, 272, 8)), ("lora_a", (3, 16, 512)), ("b", (272, 512))])
def test_lora_refuses_arrays_that_are_too_small(fg, name, small):
    args = lora_args(fg)
    args[name] = (Fake(args[name].nbytes, contiguous=False) if small is None else Fake(*small, dtype=args[name].dtype))
    with pytest.raises(ValueError):
        fg.fp8_gemm_nt_lora(**args, stream=0)
    assert fg.calls == 0
