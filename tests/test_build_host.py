"""The build script on a host without a GPU: what it builds where torch or Python's headers are missing.  The compilers are
stood in for by a function that writes the files they are asked for."""
import importlib.util
import os
import subprocess
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build script with its outputs in tmp_path; .commands: what it ran."""
    spec = importlib.util.spec_from_file_location("fg_build_under_test", os.path.join(ROOT, "moe_fp8_e4m3_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    for name, file in (("BUILD", "_build"), ("LIB", "libfg.so"), ("BIND", "fg_bind.so")):
        monkeypatch.setattr(mod, name, str(tmp_path / file))
    mod.commands, mod.fails = [], lambda cmd: False

    def run(cmd, **kw):
        mod.commands.append(cmd)
        if mod.fails(cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="fatal error: Python.h: No such file or directory")
        out = cmd[cmd.index("-o") + 1]
        text = " ".join(cmd)
        for x in cmd:                                       # objects go into what is linked from them
            if x.endswith(".o") and x != out and os.path.exists(x):
                with open(x) as f:
                    text += f.read()
        with open(out, "w") as f:
            f.write(text)
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(mod, "subprocess", types.SimpleNamespace(run=run, PIPE=subprocess.PIPE))
    return mod


def without_torch(monkeypatch, mod):
    real = importlib.util.find_spec
    fake = types.SimpleNamespace(util=types.SimpleNamespace(find_spec=lambda n, *a: None if n == "torch" else real(n, *a)))
    monkeypatch.setattr(mod, "importlib", fake)


def test_the_library_is_built_without_torch(build, monkeypatch):
    without_torch(monkeypatch, build)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BIND) and not any("fg_bind.cpp" in " ".join(c) for c in build.commands)
    n = len(build.commands)
    build.build()
    assert len(build.commands) == n, "nothing is out of date"


def test_the_library_is_built_where_the_module_does_not_compile(build):
    pytest.importorskip("torch")
    build.fails = lambda cmd: any("fg_bind" in x for x in cmd)
    with pytest.warns(RuntimeWarning, match="Python.h"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)
    with open(build.BIND, "w") as f:                         # one of older sources is not left to be loaded
        f.write("old")
    os.utime(build.BIND, (0, 0))
    with pytest.warns(RuntimeWarning):
        build.build()
    assert not os.path.exists(build.BIND)
    n = len(build.commands)
    build.fails = lambda cmd: False
    build.build()
    assert os.path.exists(build.BIND)
    assert all("fg_bind" in " ".join(c) for c in build.commands[n:]), "the library was up to date"


def test_both_are_built_once(build):
    pytest.importorskip("torch")
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.BIND)
    n = len(build.commands)
    build.build()
    assert len(build.commands) == n
    build.build(force=True)
    assert len(build.commands) == 2 * n


def test_a_library_that_does_not_link_is_an_error(build):
    build.fails = lambda cmd: "-shared" in cmd
    with pytest.raises(RuntimeError):
        build.build()


@pytest.mark.parametrize("what", ["torch", "python"])
def test_the_module_is_built_anew_for_another_torch_or_python(build, tmp_path, monkeypatch, what):
    """File times say nothing about it: the packages may be older than the module."""
    pytest.importorskip("torch")
    build.build()
    assert build.bind_fits()
    n = len(build.commands)
    if what == "torch":
        other = tmp_path / "torch"
        other.mkdir()
        (other / "version.py").write_text("__version__ = '0.0'")
        monkeypatch.setattr(build, "_torch", lambda: str(other))
    else:
        monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-300")
    assert not build.bind_fits()
    build.build()
    assert build.bind_fits() and len(build.commands) > n
    assert all("fg_bind" in " ".join(c) for c in build.commands[n:])


@pytest.mark.parametrize("why", ["missing", "other"])
def test_calls_go_through_the_binding_where_the_module_does_not_fit(why, tmp_path, monkeypatch):
    torch = pytest.importorskip("torch")
    import moe_fp8_e4m3_gb300 as fg
    from moe_fp8_e4m3_gb300 import build as mod

    from test_abi_serving import ARGS
    if why == "other":
        (tmp_path / "fg_bind.so").write_text("of another torch")
    monkeypatch.setattr(mod, "BIND", str(tmp_path / "fg_bind.so"))
    monkeypatch.setattr(fg, "_bind", None)
    monkeypatch.setattr(fg, "_stream", lambda stream: 0)
    calls = []
    monkeypatch.setattr(fg, "_call", lambda *a: calls.append(a[0]) or fg.FG_OK)
    with pytest.warns(RuntimeWarning, match="fg_bind.so"):
        fg.build_block_tables(**ARGS["build_block_tables"](fg))
    for name in ("qk_norm_rope", "kv_append_mxfp4", "kv_gather_mxfp4", "paged_attention_mxfp4"):
        getattr(fg, name)(**ARGS[name](fg))
    assert calls == [0, 1, 2, 3, 4]
    with pytest.raises(TypeError):
        fg.build_block_tables(**dict(ARGS["build_block_tables"](fg), slots=torch.zeros(7, dtype=torch.int32)))
