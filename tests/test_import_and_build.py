"""The package's import and build where a part of the machine is missing."""
import os
import subprocess
import sys

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
