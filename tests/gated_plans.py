"""The kernels that the rules of the gated products choose, asked on the CPU as tests/ops_plans.py does."""
import ctypes
import os
import subprocess
import tempfile

from tests.ops_plans import ACTS, ROOT, available  # noqa: F401

SHIM = r"""
#include "mpgemm_ops_host.hpp"
using namespace mpg_host;
static void put(const OpPlan &p, int64_t *o) {
    o[0] = p.skinny; o[1] = p.fm; o[2] = p.w; o[3] = p.waves; o[4] = p.rows; o[5] = p.tiles_m; o[6] = p.tiles_n;
}
extern "C" {
void plan_gated(int64_t groups, int64_t rows, int64_t n, int64_t k, int tb, int act, int kept, int64_t *o) {
    put(gated_plan(groups, rows, n, k, tb, gated_weight(act, kept)), o);
}
void plan_gated_grad(int64_t groups, int64_t rows, int64_t n, int64_t k, int act, int h, int64_t *o) {
    put(gated_grad_plan(groups, rows, n, k, gated_grad_weight(act, h)), o);
}
}
"""
_i64 = ctypes.c_int64
_lib = None


def _load():
    global _lib
    if _lib is None:
        csrc = os.path.join(ROOT, "mixed_precision_dense_amd", "csrc")
        with tempfile.TemporaryDirectory() as d:
            src, lib = os.path.join(d, "plans.cpp"), os.path.join(d, "plans.so")
            with open(src, "w") as f:
                f.write(SHIM)
            subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o",
                            lib, src, os.path.join(csrc, "mpgemm_host.cpp"), os.path.join(csrc, "mpgemm_ops_host.cpp")],
                           check=True)
            _lib = ctypes.CDLL(lib)
    return _lib


def _kernel(o):
    """("few", block rows, blocks of columns, waves) or ("tile", edge)."""
    return ("few", o[1], o[2], o[3]) if o[0] else ("tile", o[4])


def gated(groups, rows, n, k, tb, act="silu", kept=False):
    o = (_i64 * 7)()
    _load().plan_gated(_i64(groups), _i64(rows), _i64(n), _i64(k), int(tb), ACTS[act], int(kept), o)
    return _kernel(o)


def gated_grad(groups, rows, n, k, act="silu", h=False):
    o = (_i64 * 7)()
    _load().plan_gated_grad(_i64(groups), _i64(rows), _i64(n), _i64(k), ACTS[act], int(h), o)
    return _kernel(o)
