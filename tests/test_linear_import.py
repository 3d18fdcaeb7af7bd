"""The package without the torch side of its linear operators: everything that
does not need it goes on, and what needs it says what is missing."""
import importlib.machinery
import importlib.util
import os
import subprocess
import sys

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "lds_tiled_matrix_amd")

USE = """
import lds_tiled_matrix_amd as X
assert X.__file__.startswith(%r), X.__file__
assert X.xpose_sgemm_plan(64, 64, 64, 256, 64, 65536, 64, 131072, 64)[0] == X.XPOSE_OK
assert X.fp8_gemm_plan(1, 4096, 4096)["tile_n"] == 16
import torch
assert X.plan_for(torch.zeros(300, 200))
for call in (lambda: X.fp8_quantize(torch.zeros(4, 4)), lambda: X.layer_norm(torch.zeros(4, 4)),
             lambda: X.clip_grad_norm([torch.zeros(4)], 1.0)):
    try:
        call()
    except ImportError as e:
        assert "_linear.so" in str(e) and "build.py" in str(e), e
    else:
        raise AssertionError("no error")
print("fine")
"""


@pytest.mark.parametrize("other", ["missing", "broken"])
def test_package_without_the_torch_side(tmp_path, other):
    """As a checkout whose _linear.so is not built, or was built for another
    torch or Python."""
    package = tmp_path / "lds_tiled_matrix_amd"
    package.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py") or name == "libxpose.so":
            os.symlink(os.path.join(PACKAGE, name), package / name)
    if other == "broken":
        (package / "_linear.so").write_bytes(b"no library")
    env = dict(os.environ, PYTHONPATH=str(tmp_path), PYTHONDONTWRITEBYTECODE="1")
    got = subprocess.run([sys.executable, "-c", USE % str(tmp_path)], env=env, cwd=tmp_path, capture_output=True,
                         text=True, timeout=300)
    assert got.returncode == 0 and got.stdout.strip() == "fine", got.stderr


def test_build_without_hip_in_torch(tmp_path, monkeypatch):
    """A torch for the CPU alone has no libraries to link with: the library
    itself is built all the same."""
    spec = importlib.util.spec_from_file_location("xpose_build", os.path.join(PACKAGE, "build.py"))
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    origin = str(tmp_path / "torch" / "__init__.py")
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: importlib.machinery.ModuleSpec(name, None, origin=origin))

    def run(*a, **k):
        raise AssertionError(a)
    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build_torch() is None
