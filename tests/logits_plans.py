"""The kernels that the rules of the losses and log probabilities choose, asked on the CPU as tests/ops_plans.py does."""
import ctypes
import os
import subprocess
import tempfile

from tests.ops_plans import ROOT, available  # noqa: F401

SHIM = r"""
#include "mpgemm_ops_host.hpp"
using namespace mpg_host;
extern "C" {
int plan_merge_picks(int64_t m, int64_t top, int64_t k) { return merge_picks(m, top, k); }
void plan_logprobs(int64_t m, int64_t n, int bytes, int64_t top, int64_t *o) {
    const LogprobLayout L = logprob_layout(m, n, bytes, top);
    o[0] = L.waves; o[1] = L.parts; o[2] = L.part_vectors;
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


def merge_picks(m, top, k):
    """Whether the kernel that joins a loss's statistics forms the logits at the teacher's columns itself."""
    return bool(_load().plan_merge_picks(_i64(m), _i64(top), _i64(k)))


def logprobs(m, n, t, top):
    """(waves of a workgroup, parts of a row, 16-byte vectors of a part)."""
    o = (_i64 * 3)()
    _load().plan_logprobs(_i64(m), _i64(n), 4 if t == "f32" else 2, _i64(top), o)
    return tuple(o)
