"""What the package needs of torch: nothing until an operator on tensors (or a Decoder) is used."""

import os
import subprocess
import sys

from persistent_monokernel_sm_b200 import build

build.build()
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STAR = """
import sys
from persistent_monokernel_sm_b200 import *
assert "torch" not in sys.modules
import persistent_monokernel_sm_b200 as kd
assert load_library() and kd_strerror(0) == "ok" and {"linear", "prompt_attention", "kd_linear"} <= set(dir(kd))
assert "torch" not in sys.modules
assert callable(kd.linear) and "torch" in sys.modules
"""


def test_a_star_import_leaves_torch_alone():
    r = subprocess.run([sys.executable, "-c", STAR], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_the_library_builds_without_torch(monkeypatch):
    """_kd_torch.so is left out where torch is not installed, and built again for another torch."""
    def run(*a, **k):
        raise AssertionError("a compiler was started")

    real = build._torch_version()
    monkeypatch.setattr(build.subprocess, "check_call", run)
    monkeypatch.setattr(build, "_torch_version", lambda: None)
    assert build.build() == build.OUT
    monkeypatch.setattr(build, "_torch_version", lambda: "0.0")
    assert build._torch_stale("0.0")
    try:
        build.build()
    except AssertionError as e:
        assert "compiler" in str(e)
    else:
        raise AssertionError("not built for another torch")
    monkeypatch.setattr(build, "_torch_version", lambda: real)
    build.build()
