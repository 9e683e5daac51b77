"""The binding of the request calls: its absence, a failed build or one for another torch take away those calls and no
others.  CPU only."""
import os
import subprocess
import sys

import pytest
import torch

import block_sparse_attention_pbsa_b200 as P
from block_sparse_attention_pbsa_b200 import _lib, build

WITHOUT = """
import sys
sys.path.insert(0, sys.argv[1])
import block_sparse_attention_pbsa_b200 as P
assert P.__file__.startswith(sys.argv[1])
assert P.pbsa_workspace_bytes(P.make_geom(2, 128, 8, 8, 8, 8, 0.1, "bf16"), 4, 4) >= 256
assert P.pbsa_q4_block_bytes(P.make_req_geom(2, 2, 64, 0.1, "bf16")) == 4608
assert "unsupported" in P.pbsa_status_string(2)
for call in (lambda: P.pbsa_append_q4(None, None, None, None, None, 1), lambda: P.pbsa_request_tables(*[None] * 10)):
    try:
        call()
    except RuntimeError as e:
        assert "python -m block_sparse_attention_pbsa_b200.build" in str(e), e
    else:
        raise SystemExit("the call went through")
"""


def test_the_library_loads_without_the_binding(tmp_path):
    build.build()
    pkg = tmp_path / "block_sparse_attention_pbsa_b200"
    pkg.mkdir()
    for n in os.listdir(build.PKG):
        if n.endswith(".py") or n == "libpbsa.so":
            os.symlink(os.path.join(build.PKG, n), pkg / n)
    # (a module of the untagged name, as older builds left, is not taken for it)
    (pkg / "_requests.so").write_bytes(b"not a library")
    code = tmp_path / "without.py"
    code.write_text(WITHOUT)
    r = subprocess.run([sys.executable, str(code), str(tmp_path)], capture_output=True, text=True, cwd=tmp_path, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_a_binding_that_cannot_be_built_leaves_the_library(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "binding_path", lambda: str(tmp_path / "_requests.so"))
    monkeypatch.setenv("CXX", "false")
    with pytest.warns(UserWarning, match="binding"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(tmp_path / "_requests.so")


def test_the_binding_is_for_one_torch_and_one_interpreter(monkeypatch):
    build.build()
    monkeypatch.setattr(build.subprocess, "run", lambda *a, **k: pytest.fail("rebuilt"))
    build._binding()                                   # as it was built: nothing to do
    monkeypatch.setattr(torch, "__version__", "1.2.3")
    with pytest.raises(pytest.fail.Exception, match="rebuilt"):
        build._binding()
    monkeypatch.setattr(_lib, "_binding", None)
    with pytest.raises(RuntimeError, match="1.2.3"):   # there is none for that one
        P.pbsa_append_q4(P.make_req_geom(2, 2, 64, 0.1, "bf16"), None, None, None, None, 1)
    monkeypatch.undo()
    before = _lib.binding_path()
    monkeypatch.setattr(_lib.sysconfig, "get_config_var", lambda name: ".cpython-399-x86_64-linux-gnu.so")
    assert _lib.binding_path() != before
