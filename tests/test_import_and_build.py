"""The package's import and build where a part of the machine is missing."""
import ctypes
import os
import subprocess
import sys

import pytest

from exact_attention_58_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)


def test_import_with_a_pytorch_without_cuda():
    """A CPU-only PyTorch lacks the private functions that name the current
    stream and device; the package imports all the same."""
    res = python("import torch\n"
                 "for name in [n for n in dir(torch._C) if n.startswith('_cuda_')]:\n"
                 "    delattr(torch._C, name)\n"
                 "import exact_attention_58_gb300 as ea\n"
                 "assert ea.attn_fwd_paged\n")
    assert res.returncode == 0, res.stderr


def test_library_stands_where_the_extension_does_not_compile(monkeypatch, tmp_path):
    """build() reports the extension's error, after linking the library, and
    leaves no extension of an older build beside it."""
    if not os.path.exists(_build.LIB_PATH):
        _build.build()
    for name in ("LIB_PATH", "STAMP", "BINDING_PATH", "BINDING_STAMP"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    broken = tmp_path / "binding.cpp"
    broken.write_text("#error no headers\n")
    monkeypatch.setattr(_build, "BINDING_SRC", str(broken))
    (tmp_path / "_binding.so").write_text("old")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        _build.build()
    lib = ctypes.CDLL(str(tmp_path / "libgbattn.so"))
    assert lib.attn_version() > 0
    assert not os.path.exists(tmp_path / "_binding.so")
