"""csrc/mx_rules.h (which kernel and tile a product's sizes choose) compiled
for the host: the rules that the library itself is built from."""
import ctypes
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "lossless_bf16_tensor_exp_amd", "csrc")
SHIM = """
#include "mx_rules.h"
extern "C" {
int matmul_kernel(uint64_t t, uint64_t n, uint64_t k, uint32_t g, int o, int mx8) { return mx_matmul_kernel({t, n, k, g, o != 0}, mx8 != 0); }
int scaled_kernel(uint64_t t, uint64_t n, uint64_t k, uint32_t g, int o) { return mx_scaled_kernel({t, n, k, g, o != 0}); }
int dx_kernel(uint64_t t, uint64_t n, uint64_t k, uint32_t g, int o) { return mx_dx_kernel({t, n, k, g, o != 0}); }
uint32_t dx_parts(uint64_t t, uint64_t n, uint64_t k, uint32_t g) { return mx_dx_parts(t, n, k, g); }
uint64_t unit_groups(uint64_t rows, uint64_t cols) { return mx_unit_groups(rows, cols); }
uint64_t tile_groups(int op, uint32_t bm, uint32_t bn, uint64_t t, uint64_t n, uint64_t k, uint32_t g, int o, uint32_t parts) {
  return mx_tile_groups(op, bm, bn, {t, n, k, g, o != 0}, parts);
}
uint32_t wgrad_parts(uint64_t t, uint64_t n, uint64_t k, uint32_t g) { return mx_wgrad_parts(t, n, k, g); }
}
"""
KERNELS = ("few128", "few16", "32x128", "64x128", "128x128", "128x256", "32x256", "64x256", "256x128")
_rules = None


def rules():
    global _rules
    if _rules is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "shim.cpp"), os.path.join(d, "shim.so")
            with open(src, "w") as f:
                f.write(SHIM)
            subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-Wno-unused-function", "-shared", "-fPIC",
                            "-I", CSRC, "-o", so, src], check=True)
            _rules = ctypes.CDLL(so)
        u64, u32, i32 = ctypes.c_uint64, ctypes.c_uint32, ctypes.c_int
        for name, tail, res in (("matmul_kernel", [i32, i32], i32), ("scaled_kernel", [i32], i32), ("dx_kernel", [i32], i32),
                                ("dx_parts", [], u32), ("wgrad_parts", [], u32)):
            f = getattr(_rules, name)
            f.argtypes, f.restype = [u64, u64, u64, u32] + tail, res
        _rules.unit_groups.argtypes, _rules.unit_groups.restype = [u64, u64], u64
        _rules.tile_groups.argtypes, _rules.tile_groups.restype = [i32, u32, u32, u64, u64, u64, u32, i32, u32], u64
    return _rules


def kernel(op, tokens, n, k, groups=1, offsets=None):
    """Name of the kernel of a product: op "bf16" or "mx8" (matmul by x's form), "scaled" or "dx"."""
    o = int(groups > 1 if offsets is None else offsets)
    r = rules()
    if op in ("bf16", "mx8"):
        return KERNELS[r.matmul_kernel(tokens, n, k, groups, o, int(op == "mx8"))]
    return KERNELS[(r.scaled_kernel if op == "scaled" else r.dx_kernel)(tokens, n, k, groups, o)]
