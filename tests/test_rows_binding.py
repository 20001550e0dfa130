"""The row operators' binding, host only: streams and the argument checks' library."""
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

import token_choice_routing_amd as tcr
from token_choice_routing_amd import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_stream_of_another_device_is_refused():
    """The call's tensors are on the current device, so its stream has to be as well."""
    assert tcr._row_stream(SimpleNamespace(cuda_stream=16, device_index=0), 0) == 16
    assert tcr._row_stream(SimpleNamespace(cuda_stream=16), 0) == 16  # a handle of another library
    assert tcr._row_stream(32, 1) == 32
    with pytest.raises(ValueError, match="stream: expected one of the current device"):
        tcr._row_stream(SimpleNamespace(cuda_stream=16, device_index=1), 0)


def _without_checks(path):
    """A fresh process whose binding looks for its checks at path (a file or none)."""
    code = f"""
import torch, token_choice_routing_amd as tcr
tcr.MARSHAL_PATH = {path!r}
lib = tcr.load_library()
dims = tcr.make_dims(64, 64, 8, 8, 2, 64, 0, tcr.MOE_BF16)
assert tcr.workspace_bytes(dims, tcr.MOE_WS_LAYER) > 0
try:
    tcr.moe_act8_pack(torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
except ImportError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout


def test_layer_calls_do_not_need_the_argument_checks(tmp_path):
    """Without the native checks the library still loads; the row operators name what is
    missing."""
    missing = str(tmp_path / "_marshal.so")
    assert f"{missing} (argument checks of the row operators) is not built" in _without_checks(missing)


def test_argument_checks_that_do_not_load(monkeypatch):
    monkeypatch.setattr(tcr, "_marshal", None)

    def fail(*a):
        raise ImportError("undefined symbol")

    monkeypatch.setattr(tcr.importlib, "import_module", fail)
    with pytest.raises(ImportError, match="_marshal.so does not load with this torch.*undefined symbol"):
        tcr.moe_act8_pack(torch.zeros(4, 64), None, None)


def test_build_without_a_host_compiler(tmp_path, monkeypatch, capsys):
    """The checks' compiler is missing or fails: a warning, and no checks of an earlier build."""
    old = tmp_path / "_marshal.so"
    monkeypatch.setattr(B, "MARSHAL", str(old))
    for cmd, word in (([str(tmp_path / "no-such-compiler")], "no-such-compiler"),
                      ([sys.executable, "-c", "print('no headers'); raise SystemExit(3)"], "no headers")):
        old.write_text("old")
        monkeypatch.setattr(B, "_marshal_cmd", lambda out, cmd=cmd: cmd)
        problem = B._compile_marshal(str(old) + ".tmp")
        assert word in problem
        B._install_marshal(str(old) + ".tmp", problem)
        assert not old.exists() and "row operators will refuse" in capsys.readouterr().err
    new = tmp_path / "new"
    new.write_text("new")
    B._install_marshal(str(new), "")
    assert old.read_text() == "new" and capsys.readouterr().err == ""
