"""The binding of the operators around the mixer is bound to one PyTorch; the
package and the mixer are not."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import importlib.abc, sys
import torch

class Refused(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._efla_block"):
            raise ImportError("undefined symbol: _ZN2at6Tensor")

if sys.argv[1] == "unloadable":
    sys.meta_path.insert(0, Refused())
elif sys.argv[1] == "other version":
    torch.__version__ = "9.9.9"
import delta_rule_linear_03_b200 as efla
assert efla.version() >= 100 and efla.prefill_bwd_workspace_size(1, 2, 8, 64) > 0
for call in (lambda: efla.norm_fwd(None, None), lambda: efla.conv_step(None, None, None), lambda: efla.scan_step(*[None] * 6)):
    try:
        call()
    except ImportError as e:
        assert "build.py" in str(e) and sys.argv[2] in str(e), e
    else:
        raise SystemExit("no error")
assert efla.scan_fwd_workspace_size(8, 2048, 1024, 1, 16) == 0
"""


@pytest.mark.parametrize("how,said", [("unloadable", "undefined symbol"), ("other version", "9.9.9")])
def test_the_mixer_needs_no_binding(how, said):
    r = subprocess.run([sys.executable, "-c", PROGRAM, how, said], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_another_version_makes_the_binding_stale(monkeypatch):
    spec = importlib.util.spec_from_file_location("efla_builder", os.path.join(ROOT, "delta_rule_linear_03_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    assert "torch " in b.binding_for()
    with open(b.BUILT_FOR) as f:
        assert f.read() == b.binding_for()
    library = b.stale_library()
    monkeypatch.setattr(b, "binding_for", lambda: "torch 9.9.9 cpython-999")
    assert b.stale_binding() and b.stale() and b.stale_library() == library
