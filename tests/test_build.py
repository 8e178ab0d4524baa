"""The extension module: rebuilt when what it was built against changes, and
needed by its own calls only (CPU)."""
import os
import subprocess
import sys

import pytest
import torch

from long_context_causal_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def built(tmp_path, monkeypatch):
    """A module newer than its sources, with the record of what it was built against."""
    monkeypatch.setattr(build, "BINDING_LIB", str(tmp_path / "module.so"))
    monkeypatch.setattr(build, "BINDING_KEY", str(tmp_path / "module.key"))
    (tmp_path / "module.so").write_bytes(b"")
    (tmp_path / "module.key").write_text(build._binding_key())
    return tmp_path


def test_the_module_that_was_built_is_up_to_date(built, monkeypatch):
    assert build.binding_up_to_date()
    monkeypatch.setattr(build, "_nvcc", lambda: pytest.fail("a built tree needs no compiler"))
    assert build.binding_up_to_date()


@pytest.mark.parametrize("what", ["torch", "abi", "python", "no key", "no module", "older"])
def test_the_module_is_rebuilt_for_another_torch(built, monkeypatch, what):
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "1.2.3")
    elif what == "abi":
        monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    elif what == "python":
        monkeypatch.setattr(sys, "version", "2.7")
    elif what == "no key":
        os.remove(built / "module.key")
    elif what == "no module":
        os.remove(built / "module.so")
    else:
        os.utime(built / "module.so", (0, 0))
    assert not build.binding_up_to_date()


WITHOUT = """
import sys
sys.modules["long_context_causal_gb300._dfa_torch"] = None      # as where it does not load
import torch
from long_context_causal_gb300 import dfa
assert dfa.dfa_build_worklist(4, 4, 2)[2] > 0 and dfa.dfa_ckpt8_size(1, 4, 2, 300, 128) > 0
q = torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16)
for call in (lambda: dfa.dfa_attn_fwd_sink(q, q, q, 4), lambda: dfa.dfa_ckpt8_save(q, q, q, q)):
    try:
        call()
    except ImportError as e:
        assert "build()" in str(e)
    else:
        raise AssertionError("no error")
"""


def test_the_other_entry_points_do_not_need_the_module():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
