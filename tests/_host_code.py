"""The kernels' arithmetic (csrc/moe_exact.h) in a host library, with a test's own
loops over it."""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_decode_expert_gb300", "csrc")


def host_library(tmp_path, code):
    """``code`` (extern "C" functions) compiled behind moe_exact.h, loaded."""
    src, lib = tmp_path / "host.cpp", tmp_path / "host.so"
    src.write_text('#include <cstring>\n#include "moe_exact.h"\nusing namespace moe;\n' + code)
    subprocess.run(["g++", "-O2", "-std=c++17", "-ffp-contract=off", "-Wno-unknown-pragmas", "-shared", "-fPIC", "-I", CSRC,
                    str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))
