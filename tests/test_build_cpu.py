"""The build: the C library needs nvcc and no torch; the marshalling module is compiled again for another torch or Python, and
refuses to work with one that it was not compiled against."""
import os
import subprocess
import sys

import pytest

from diffusion_transformer_w4a4_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

NO_TORCH = r'''
import sys
class Hidden:
    def find_spec(self, name, path=None, target=None):
        if name.split(".")[0] == "torch":
            raise ModuleNotFoundError("No module named 'torch'", name="torch")
sys.path.insert(0, ROOT)
import importlib.util
find = importlib.util.find_spec
importlib.util.find_spec = lambda name, *a: None if name.split(".")[0] == "torch" else find(name, *a)
sys.meta_path.insert(0, Hidden())
from diffusion_transformer_w4a4_b200 import build
build.MARSHAL = OUT
print(build.build())
import diffusion_transformer_w4a4_b200 as svdq
print(svdq.svdq_status_string(0))
assert "torch" not in sys.modules
'''


def test_library_builds_and_loads_without_torch(tmp_path):
    build.build()  # (the library itself is up to date below)
    out = str(tmp_path / "marshal.so")
    code = NO_TORCH.replace("ROOT", repr(ROOT)).replace("OUT", repr(out))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    assert build.LIB in r.stdout and not os.path.exists(out)


def test_module_of_other_versions_is_stale(tmp_path, monkeypatch):
    build.build()
    assert not build._marshal_stale()
    stamp = tmp_path / "stamp"
    monkeypatch.setattr(build, "MARSHAL_STAMP", str(stamp))
    assert build._marshal_stale()  # built before versions were noted
    for text in ("python 3.1 torch 2.11.0", build._marshal_versions() + "x"):
        stamp.write_text(text)
        assert build._marshal_stale()
    stamp.write_text(build._marshal_versions())
    assert not build._marshal_stale()


def test_module_refuses_another_torch():
    import torch

    build.build()
    import diffusion_transformer_w4a4_b200 as svdq

    m = svdq._calls()
    with pytest.raises(RuntimeError, match="built for torch"):
        m.bind(0, 0, 0, 0, None, None, None, "1.0.0")
    with pytest.raises(ValueError, match="CUDA tensor"):  # and goes on as it was bound
        svdq.svdq_qk_norm_rope(torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16))
