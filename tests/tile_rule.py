"""The library's rule for which kernel an int8 product takes, compiled for the
host from its own header."""
import collections
import ctypes
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_expert_load_ue_amd", "csrc")
SHIM = """
#include "ue_tiles.h"
extern "C" const char *choose(int M, long long N, int K, int G, int gated, int grouped,
                              int wide, int num_cu, long long *out) {
    const ue::I8Size z{M, N, K, G, gated != 0, grouped != 0, wide != 0, num_cu};
    const ue::I8Kernel k = ue::i8_kernel(z);
    out[0] = ue::i8_workgroups(k, z);
    out[1] = out[0] * ue::i8_tile(k).threads <= ue::kLaunchThreads;
    return ue::i8_tile(k).name;
}
"""
Choice = collections.namedtuple("Choice", "name workgroups fits")


def compile_rule(folder):
    src, lib = os.path.join(folder, "rule.cpp"), os.path.join(folder, "rule.so")
    with open(src, "w") as f:
        f.write(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC,
                    "-o", lib, src], check=True)
    f = ctypes.CDLL(lib).choose
    f.restype = ctypes.c_char_p
    f.argtypes = ([ctypes.c_int, ctypes.c_longlong] + [ctypes.c_int] * 6 +
                  [ctypes.POINTER(ctypes.c_longlong * 2)])

    def rule(M, N, K, G=1, gated=False, grouped=False, wide=False, num_cu=256):
        out = (ctypes.c_longlong * 2)()
        name = f(M, N, K, G, gated, grouped, wide, num_cu, ctypes.byref(out))
        return Choice(name.decode(), out[0], bool(out[1]))
    return rule
