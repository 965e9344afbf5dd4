"""The token-by-token calls' CPython extension is optional for everything else:
the package imports and serves its other calls without it, its build follows
the Python and torch that it was made for (CPU)."""
import importlib.util
import os
import subprocess
import sys

import pytest

import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import _abi

PKG = os.path.dirname(os.path.abspath(dl.__file__))

USE = """
import torch
import long_context_diffusion_b200 as dl
from long_context_diffusion_b200 import pipeline
assert dl.__file__.startswith({tmp!r}), dl.__file__
desc = dl.make_desc(1, 4, 4, 64, 128, 8, 64, 2, 2, torch.float32)
assert dl.dl_workspace_size(desc) > 0
try:
    dl.dl_decode_attn(desc, None, None, None, None, None, None, None, None)
except ImportError as e:
    assert "decode_attn" in str(e) and "build" in str(e), e
else:
    raise SystemExit("no ImportError")
"""


@pytest.mark.parametrize("calls", ["missing", "not a library"])
def test_the_package_serves_its_other_calls_without_the_extension(calls, tmp_path):
    pkg = tmp_path / "long_context_diffusion_b200"
    (pkg / "lib").mkdir(parents=True)
    for f in os.listdir(PKG):
        if f.endswith(".py"):
            os.symlink(os.path.join(PKG, f), pkg / f)
    os.symlink(_abi.LIB_PATH, pkg / "lib" / os.path.basename(_abi.LIB_PATH))
    if calls != "missing":
        (pkg / "lib" / "_calls.so").write_bytes(b"no library")
    r = subprocess.run([sys.executable, "-c", USE.format(tmp=str(tmp_path))], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def build(tmp_path):
    """The build module with its outputs under tmp_path."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(PKG, "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.BUILD, mod.CALLS = str(tmp_path), str(tmp_path / "_calls.so")
    return mod


def test_the_extension_is_built_again_for_another_python_or_torch(build, monkeypatch):
    assert build.build_calls() == build.CALLS
    first = os.stat(build.CALLS)
    build.build_calls()
    assert os.stat(build.CALLS).st_ino == first.st_ino  # nothing changed
    was = build._calls_stamp
    monkeypatch.setattr(build, "_calls_stamp", lambda: was() + " another torch")
    build.build_calls()
    assert os.stat(build.CALLS).st_ino != first.st_ino
    mod = _abi._load_calls(build.CALLS)
    with pytest.raises(RuntimeError, match="not bound"):
        mod.decode_attn()


def test_without_the_exchange_table_in_the_headers_the_library_still_builds(build, monkeypatch, tmp_path, capsys):
    inc = tmp_path / "include"
    (inc / "ATen").mkdir(parents=True)
    (inc / "ATen" / "dlpack.h").write_text("// an older DLPack\n")
    (tmp_path / "_calls.so").write_bytes(b"of another torch")
    monkeypatch.setattr(build, "_torch_include", lambda: str(inc))
    assert build.build_calls() is None
    assert not os.path.exists(build.CALLS) and "DLPackExchangeAPI" in capsys.readouterr().err


def test_an_extension_for_another_python_says_so(tmp_path):
    """bind_calls.cpp built with the version macros of another Python."""
    spec = importlib.util.spec_from_file_location("_b", os.path.join(PKG, "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    src = tmp_path / "other.cpp"
    src.write_text('#include <Python.h>\n#undef PY_MINOR_VERSION\n#define PY_MINOR_VERSION 1\n'
                   f'#include "{os.path.join(b.CSRC, "bind_calls.cpp")}"\n')
    out = str(tmp_path / "_calls.so")
    import sysconfig
    subprocess.run(["g++", "-O0", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(b.ROOT, "include"), "-I",
                    sysconfig.get_paths()["include"], "-I", b._torch_include(), str(src), "-o", out], check=True,
                   capture_output=True)
    mod = _abi._load_calls(out)
    with pytest.raises(ImportError, match="built for Python 3.1,"):
        mod.decode_attn
