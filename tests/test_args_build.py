"""The library's build does not depend on the module that packs tensor views: without torch or a working g++ the
binding packs them itself."""
import os
import subprocess
import sys
import sysconfig

import pytest

from fp8_attention_forward_gb300 import build


def test_the_module_is_named_by_interpreter_and_torch():
    a, b = build.args_path("2.9.1"), build.args_path("2.11.0")
    assert a != b and a.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and os.path.dirname(a) == build.BUILD
    torch = pytest.importorskip("torch")
    from fp8_attention_forward_gb300 import fa8

    out = build.build_args()
    assert out in (None, build.args_path(torch.__version__))
    assert (fa8._args_module() is not None) == (out is not None)


def test_no_torch_no_module(monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert build.build_args() is None


@pytest.mark.parametrize("how", ["fails", "fails silently", "is missing"])
def test_a_compiler_that_does_not_work_leaves_the_library(how, monkeypatch, tmp_path):
    """build() goes on to link the library; an older module does not stay."""
    pytest.importorskip("torch")
    import torch

    if build.build_args() is None:
        pytest.skip("no headers here")
    run, built = subprocess.run, []

    def fake(cmd, **kw):
        if cmd[0] == "g++":
            if how == "is missing":
                raise FileNotFoundError("g++")
            return subprocess.CompletedProcess(cmd, 1, "", "no such header" if how == "fails" else "")
        built.append(cmd)
        return run(["touch", cmd[cmd.index("-o") + 1]], **kw)

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfa8.so"))
    stale = build.args_path(torch.__version__)
    open(stale, "w").close()
    os.utime(stale, (0, 0))
    monkeypatch.setattr(build.subprocess, "run", fake)
    with pytest.warns(UserWarning, match="fa8_args"):
        lib = build.build()
    assert os.path.exists(lib) and any("-shared" in c for c in built) and not os.path.exists(stale)


def test_another_folder_gets_the_library_alone(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "build_args", lambda: pytest.fail("not for this folder"))
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **kw: (
        open(cmd[cmd.index("-o") + 1], "w").close(), subprocess.CompletedProcess(cmd, 0, "", ""))[1])
    assert os.path.exists(build.build(out_dir=str(tmp_path)))
