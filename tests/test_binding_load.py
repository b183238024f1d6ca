"""The package without its C++ binding, or with one built against another torch: everything but the bounded-memory
operators works, and those say what is wrong.  The build notices another torch."""
import os
import subprocess
import sys

import pytest

from test_abi import ROOT, load_build_module

PKG = os.path.join(ROOT, "route_kv_memory_b200")

PROGRAM = """
import route_kv_memory_b200 as mka
from fastmka_inputs import CONFIGS
assert "sm_100a" in mka.mka_version()
assert mka.mka_state_size(mka.make_config(CONFIGS["qwen7b_4k"]), 100) > 0
assert mka.mka_kv8_attention_workspace_size(mka.make_kv8_config(1, 10, 1, 1, 64)) > 0
for _ in range(2):
    try:
        mka.mka_kv8_append(None, None, None, None, None)
    except ImportError as e:
        assert "_build.py" in str(e), e
        print("refused:", e)
"""


@pytest.fixture()
def copy(tmp_path):
    """A package that shares the library but has no binding."""
    load_build_module().build_library()
    p = tmp_path / "route_kv_memory_b200"
    p.mkdir()
    for name in ("__init__.py", "libmka.so"):
        os.symlink(os.path.join(PKG, name), p / name)
    return p


def run(copy):
    env = dict(os.environ, PYTHONPATH=f"{copy.parent}{os.pathsep}{ROOT}")
    # (the package finds its files beside its own, copied, name)
    src = (copy / "__init__.py")
    if src.is_symlink():
        text = src.read_text()
        src.unlink()
        src.write_text(text)
    return subprocess.run([sys.executable, "-c", PROGRAM], env=env, cwd=copy.parent, capture_output=True, text=True)


def test_without_the_binding(copy):
    r = run(copy)
    assert r.returncode == 0 and r.stdout.count("refused:") == 2, r.stderr[-2000:]


def test_binding_of_another_torch(copy):
    (copy / "_binding.py").write_text("torch_version = '0.0.1'\n")
    r = run(copy)
    assert r.returncode == 0 and r.stdout.count("0.0.1") == 2, r.stdout + r.stderr[-2000:]


def test_build_notices_another_torch(tmp_path):
    m = load_build_module()
    m.BINDING, m.BINDING_TORCH = str(tmp_path / "_binding.so"), str(tmp_path / "torch.txt")
    assert not m.binding_is_current("2.0")  # neither file
    open(m.BINDING, "w").close()
    assert not m.binding_is_current("2.0")  # unknown torch
    with open(m.BINDING_TORCH, "w") as f:
        f.write("2.0")
    assert m.binding_is_current("2.0") and not m.binding_is_current("2.1")
    os.utime(m.BINDING, (0, 0))
    assert not m.binding_is_current("2.0")  # older than its source


def test_the_built_binding_is_this_torch_s():
    import torch
    load_build_module().build_library()
    from route_kv_memory_b200 import _binding
    assert _binding.torch_version == torch.__version__
