"""Building the extension that checks tensor arguments: for one interpreter and one torch, and not without
notice where it could be built."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

from moe_decode_layer_mxfp8_gb300 import build as mb


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Builds into a folder of the test's, by a compiler that writes its name: the commands that it got."""
    seen = []

    def run(cmd, **kw):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(mb, "ARGS_LIB", str(tmp_path / os.path.basename(mb.ARGS_LIB)))
    monkeypatch.setattr(mb, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(mb.subprocess, "run", run)
    return seen


def test_its_name_is_that_of_one_interpreter():
    assert os.path.basename(mb.ARGS_LIB) == "_args" + sysconfig.get_config_var("EXT_SUFFIX")
    assert f"{sys.version_info[0]}{sys.version_info[1]}" in os.path.basename(mb.ARGS_LIB)


def test_it_is_built_once_for_an_interpreter_and_a_torch(fake, tmp_path, monkeypatch):
    old = tmp_path / "_args.so"  # without a tag, another interpreter would load it
    old.write_text("for some interpreter")
    assert mb.build_args() == mb.ARGS_LIB and len(fake) == 1 and not old.exists()
    assert mb.build_args() == mb.ARGS_LIB and len(fake) == 1
    mine = mb.ARGS_LIB
    monkeypatch.setattr(mb, "ARGS_LIB", str(tmp_path / "_args.cpython-399-other.so"))
    assert mb.build_args() == mb.ARGS_LIB and len(fake) == 2
    # the other interpreter's torch says nothing of this one's file
    with monkeypatch.context() as c:
        c.setattr(torch, "__version__", "99.0")
        assert mb.build_args() and len(fake) == 3
        c.setattr(mb, "ARGS_LIB", mine)
        assert mb.build_args() and len(fake) == 4
    assert mb.build_args(force=True) and len(fake) == 5


def test_it_is_there_where_it_can_be_built():
    """The operators work without it; a source that does not compile is not to pass for missing headers."""
    torch_h = os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "Dtype.h")
    if not (os.path.exists(torch_h) and os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))):
        pytest.skip("no headers of torch or Python")
    assert mb.build_args() == mb.ARGS_LIB
    code = "from moe_decode_layer_mxfp8_gb300 import cache as c; assert c._args and c._vec is c._args.vec"
    subprocess.run([sys.executable, "-c", code], cwd=mb.ROOT, check=True)
