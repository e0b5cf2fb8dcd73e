"""The library builds, and the binding loads, without the CPython extension of the paged calls: it depends on the installed torch, the
library on nvcc alone (no GPU is used)."""
import os
import shutil
import subprocess
import sys

import pytest

from long_context_fm_gb300 import build as fmbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def apart(tmp_path, monkeypatch):
    """The build of one small source, in a folder of its own."""
    monkeypatch.setattr(fmbuild, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(fmbuild, "LIB", str(tmp_path / "libfm.so"))
    monkeypatch.setattr(fmbuild, "CALL", str(tmp_path / "_fm_call.so"))
    monkeypatch.setattr(fmbuild, "SOURCES", ["fm_mask.cpp"])
    return tmp_path


def test_the_library_builds_where_the_extension_does_not(apart, monkeypatch):
    monkeypatch.setattr(fmbuild, "_call_command", lambda nvcc, out: [sys.executable, "-c", "import sys; sys.exit('no torch headers')"])
    with pytest.warns(RuntimeWarning, match="no torch headers"):
        lib = fmbuild.build()
    assert os.path.exists(lib) and not os.path.exists(fmbuild.CALL)


def test_the_library_builds_without_torch(apart, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch raises ImportError
    with pytest.warns(RuntimeWarning):
        lib = fmbuild.build()
    assert os.path.exists(lib) and not os.path.exists(fmbuild.CALL)


def test_another_torch_gets_an_extension_of_its_own(apart, monkeypatch):
    import torch

    made = []

    def command(nvcc, out):
        made.append(torch.__version__)
        return [sys.executable, "-c", f"open({out!r}, 'w').write('x')"]

    monkeypatch.setattr(fmbuild, "_call_command", command)
    lib = fmbuild.build()
    when = os.path.getmtime(lib)
    fmbuild.build()
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    fmbuild.build()
    assert made[1:] == ["9.9.9"] and os.path.getmtime(lib) == when      # and the library as it was
    fmbuild.build()
    assert len(made) == 2


LOADED = """
import torch
{before}
from long_context_fm_gb300 import fm
assert fm.fm_plan_bytes(1, 1, 256) > 0 and fm.fm_paged_plan_bytes(fm.PagedStep(4, 64, 8, 10, 40, 32, 8, 4, 128, 0, 0)) > 0
x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
cache = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
for call in (lambda: fm.fm_paged_append(x, x, torch.zeros(4, dtype=torch.int64), cache, cache, torch.zeros(1, dtype=torch.int32)),):
    try:
        call()
    except TypeError:
        print("refused")
"""


@pytest.mark.parametrize("extension", ["missing", "of another torch", "broken", "as built"])
@pytest.mark.parametrize("before", ["", "del torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice   # a torch without CUDA"])
def test_the_binding_loads(tmp_path, extension, before):
    fmbuild.build()
    package = tmp_path / "long_context_fm_gb300"
    (package / "_lib").mkdir(parents=True)
    for name in ("__init__.py", "fm.py", "build.py"):
        shutil.copy(os.path.join(fmbuild.HERE, name), package / name)
    os.symlink(fmbuild.LIB, package / "_lib" / "libfm.so")
    if extension != "missing":
        for name in os.listdir(fmbuild.OUT_DIR):
            if name.startswith("_fm_call"):
                shutil.copy(os.path.join(fmbuild.OUT_DIR, name), package / "_lib" / name)
    if extension == "broken":
        (package / "_lib" / "_fm_call.so").write_text("not a library")
    elif extension == "of another torch":
        # (its functions would be called all the same: what is loaded has to be known to fit)
        (package / "_lib" / "_fm_call.so").write_text("not a library")
        (package / "_lib" / "_fm_call.tag").write_text("torch 1.0")
    r = subprocess.run([sys.executable, "-c", LOADED.format(before=before)], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.split() == ["refused"], r.stderr
