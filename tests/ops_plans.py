"""The kernels that the library's rules choose, asked on the CPU: the host-only sources built beside a
few lines that hand their plans out."""
import ctypes
import os
import shutil
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = r"""
#include "mpgemm_ops_host.hpp"
using namespace mpg_host;
static void put(const OpPlan &p, int64_t *o) {
    o[0] = p.skinny; o[1] = p.fm; o[2] = p.w; o[3] = p.waves; o[4] = p.rows; o[5] = p.tiles_m; o[6] = p.tiles_n;
}
extern "C" {
void plan_forward(int64_t m, int64_t n, int64_t k, int tb, int act, int aux, int c, int64_t *o) {
    put(op_plan(m, n, k, tb, forward_weight(act, aux, c)), o);
}
void plan_slope(int64_t m, int64_t n, int64_t k, int tb, int act, int64_t *o) { put(op_plan(m, n, k, tb, slope_weight(act)), o); }
void plan_grouped(int64_t rows, int64_t groups, int64_t n, int64_t k, int tb, int act, int aux, int64_t *o) {
    put(grouped_plan(rows, groups, n, k, tb, forward_weight(act, aux, false)), o);
}
void plan_grouped_grad(int64_t rows, int64_t groups, int64_t n, int64_t k, int tb, int act, int64_t *o) {
    put(grouped_plan(rows, groups, n, k, tb, slope_weight(act)), o);
}
void plan_wgrad(int64_t groups, int64_t rows, int64_t m, int64_t n, int64_t *o) { put(wgrad_plan(groups, rows, m, n), o); }
int plan_ce(int64_t m, int64_t n, int64_t k, int train, int64_t *logits, int64_t *dw, int64_t *dx, int64_t *other) {
    CeLayout L;
    if (!ce_layout(m, n, k, train != 0, L)) return 0;
    put(L.logits, logits);
    if (train && m > 0) {
        put(L.dw, dw);
        put(L.dx, dx);
    }
    other[0] = L.outer; other[1] = L.splits; other[2] = L.listed; other[3] = L.piece; other[4] = L.pieces;
    return 1;
}
}
"""
_i64, _int = ctypes.c_int64, ctypes.c_int
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_lib = None


def available():
    return shutil.which("g++") is not None


def _load():
    global _lib
    if _lib is None:
        csrc = os.path.join(ROOT, "mixed_precision_dense_amd", "csrc")
        with tempfile.TemporaryDirectory() as d:
            src, lib = os.path.join(d, "plans.cpp"), os.path.join(d, "plans.so")
            with open(src, "w") as f:
                f.write(SHIM)
            subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-o", lib,
                            src, os.path.join(csrc, "mpgemm_host.cpp"), os.path.join(csrc, "mpgemm_ops_host.cpp")], check=True)
            _lib = ctypes.CDLL(lib)
    return _lib


def _kernel(o):
    """("few", block rows, blocks of columns, waves) or ("tile", edge)."""
    return ("few", o[1], o[2], o[3]) if o[0] else ("tile", o[4])


def _ask(name, *args):
    o = (_i64 * 7)()
    getattr(_load(), name)(*args, o)
    return _kernel(o)


def forward(m, n, k, tb, act="none", aux=False, c=False):
    return _ask("plan_forward", _i64(m), _i64(n), _i64(k), int(tb), ACTS[act], int(aux), int(c))


def slope(m, n, k, tb, act):
    return _ask("plan_slope", _i64(m), _i64(n), _i64(k), int(tb), ACTS[act])


def grouped(rows, groups, n, k, tb, act="none", aux=False):
    return _ask("plan_grouped", _i64(rows), _i64(groups), _i64(n), _i64(k), int(tb), ACTS[act], int(aux))


def grouped_grad(rows, groups, n, k, tb, act):
    return _ask("plan_grouped_grad", _i64(rows), _i64(groups), _i64(n), _i64(k), int(tb), ACTS[act])


def wgrad(groups, rows, m, n):
    return _ask("plan_wgrad", _i64(groups), _i64(rows), _i64(m), _i64(n))


def cross_entropy(m, n, k, train):
    """{"logits", "dw", "dx": kernels, "outer", "splits", "listed", "piece", "pieces"}; the middle ones with train."""
    a, b, c, d = ((_i64 * 7)() for _ in range(4))
    assert _load().plan_ce(_i64(m), _i64(n), _i64(k), int(train), a, b, c, d)
    got = {"logits": _kernel(a)}
    if train:
        got.update(dw="outer" if d[0] else _kernel(b), dx=_kernel(c))
    got.update(splits=d[1], listed=bool(d[2]), piece=d[3], pieces=d[4])
    return got
