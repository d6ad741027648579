"""C++ of the kernels' index arithmetic compiled for the host, for tests that go to its edges."""
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_layer_sigmoid_gb300", "csrc")


def library(folder, source):
    """The C functions of `source` as a ctypes library; arithmetic that overflows ends the process."""
    src, lib = os.path.join(folder, "host.cpp"), os.path.join(folder, "host.so")
    with open(src, "w") as f:
        f.write(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, src, "-o", lib], check=True)
    return ctypes.CDLL(lib)
