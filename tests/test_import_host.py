"""Importing the package needs no CUDA build of PyTorch: what only such a build has is
asked for at the first call that needs it."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_a_cuda_build_of_torch():
    code = ("import torch\n"
            "for n in [n for n in dir(torch._C) if n.startswith('_cuda')]:\n"
            "    delattr(torch._C, n)\n"
            "import moe_decode_expert_gb300 as m, moe_decode_expert_gb300.decode_layer\n"
            "x = torch.zeros(2, 64, dtype=torch.bfloat16)\n"
            "try:\n"
            "    m._launch_stream(-1, None)\n"
            "except ValueError as e:\n"
            "    print(e)\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "CUDA" in r.stdout, r.stderr
