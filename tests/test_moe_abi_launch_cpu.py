"""What the entry points of include/awq_moe.h hand to the launches, without a GPU: moe_abi.hip's host code built by the
host compiler beside launches that only record their arguments. Pointers are fake and never dereferenced."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
moe = pytest.importorskip("post_quantization_mean_amd.moe")

FAKE, OK = 0x10000, 0
F32, BF16 = 0, 1

RECORDER = r"""
#include <stdarg.h>
#include <stdio.h>
#include "abi_status.h"
#include "moe.h"
static char text[512];
static int calls;
namespace awq {
int fail(int status, const char* fmt, ...) { va_list a; va_start(a, fmt); vsnprintf(text, sizeof text, fmt, a); va_end(a); return status; }
int ok() { return 0; }
int hip_fail(hipError_t, const char*) { return 7; }
BlockNormArgs norm;
GroupedArgs grouped;
hipError_t launch_block_norm(const BlockNormArgs& a, int, Mat, Mat, hipStream_t) { norm = a; ++calls; return hipSuccess; }
size_t block_norm_backward_stats_bytes(int64_t, int64_t) { return 0; }
size_t block_norm_backward_partial_floats(int64_t, int64_t) { return 0; }
hipError_t launch_block_norm_backward(const BlockNormArgs& a, int, CMat, CMat, Mat, Mat, float*, float*, void*, int64_t, void*,
                                      float*, hipStream_t) { norm = a; ++calls; return hipSuccess; }
int moe_sort_blocks(int64_t) { return 1; }
hipError_t launch_moe_sort(const void*, bool, int, int, int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_moe_gather(const RouteArgs&, int, CMat, Mat, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_moe_combine(const RouteArgs&, int, CMat, const float*, Mat, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_moe_combine_backward(const RouteArgs&, int, CMat, CMat, const float*, Mat, float*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_w4a16_grouped(const GroupedArgs& a, int, bool, hipStream_t) { grouped = a; ++calls; return hipSuccess; }
hipError_t launch_w4a16_grouped_backward(const GroupedArgs& a, int, bool, hipStream_t) { grouped = a; ++calls; return hipSuccess; }
}  // namespace awq
#define SEEN extern "C" __attribute__((visibility("default")))
SEEN const char* awq_last_error() { return text; }
SEEN int seen_calls() { return calls; }
SEEN int64_t seen_ld_gate() { return awq::norm.ld_gate; }
SEEN float seen_res_scale() { return awq::norm.res_scale; }
SEEN int64_t seen_ld_x() { return awq::grouped.x.ld; }
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("no host compiler or HIP headers")
    at = tmp_path_factory.mktemp("moe_abi")
    (at / "recorder.cpp").write_text(RECORDER)
    csrc = os.path.join(ROOT, "post_quantization_mean_amd", "csrc")
    so = str(at / "recorder.so")
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + csrc, "-x", "c++", os.path.join(csrc, "moe_abi.hip"),
                    str(at / "recorder.cpp"), "-o", so], check=True, capture_output=True, timeout=100)
    lib = ctypes.CDLL(so)
    for name, (res, args) in moe._SIGNATURES.items():
        getattr(lib, name).restype, getattr(lib, name).argtypes = res, args
    lib.awq_last_error.restype = ctypes.c_char_p
    lib.seen_ld_gate.restype = lib.seen_ld_x.restype = ctypes.c_int64
    lib.seen_res_scale.restype = ctypes.c_float
    return lib


def _launched(lib, call):
    """Does `call` reach a launch? Its status otherwise has to be an error."""
    before = lib.seen_calls()
    status = call()
    assert (status == OK) == (lib.seen_calls() == before + 1), lib.awq_last_error().decode()
    return status == OK


def _norm(lib, **kw):
    v = dict(y=FAKE, ld_y=64, residual=FAKE, ld_r=64, dtype=BF16, n=4, d=64, w_post=FAKE, gate=None, ld_gate=0, scale=0.5,
             w_pre=FAKE, eps=1e-6, res_out=FAKE, ld_ro=64, h=FAKE + 64, ld_h=64)
    assert not set(kw) - set(v)
    v.update(kw)
    return lib.awq_block_norm(*v.values(), None)


def _norm_backward(lib, **kw):
    v = dict(y=FAKE, ld_y=64, residual=FAKE, ld_r=64, dtype=BF16, n=4, d=64, w_post=FAKE, gate=None, ld_gate=0, scale=0.5,
             w_pre=FAKE, eps=1e-6, d_res=FAKE, ld_dr=64, d_h=FAKE, ld_dh=64, d_y=FAKE, ld_dy=64, d_residual=FAKE, ld_do=64,
             d_w_post=FAKE, d_w_pre=FAKE, d_gate=None, ld_dg=0, ws=FAKE, nb=0)
    assert not set(kw) - set(v)
    v.update(kw)
    return lib.awq_block_norm_backward(*v.values(), None)


@pytest.mark.parametrize("f", [_norm, _norm_backward])
def test_a_pitch_without_a_gate_is_no_gate_per_token(lib, f):
    """The kernels read a gate of each token's own wherever the pitch is not zero."""
    assert _launched(lib, lambda: f(lib, gate=None, ld_gate=64)) and lib.seen_ld_gate() == 0
    assert _launched(lib, lambda: f(lib, gate=None, ld_gate=-5)) and lib.seen_ld_gate() == 0
    assert _launched(lib, lambda: f(lib, gate=FAKE, ld_gate=72)) and lib.seen_ld_gate() == 72
    assert _launched(lib, lambda: f(lib, gate=FAKE)) and lib.seen_ld_gate() == 0


@pytest.mark.parametrize("f,parts", [(_norm, dict(res_out=None)), (_norm_backward, dict(d_y=None, d_w_post=None))])
def test_without_y_there_is_no_residual_scale(lib, f, parts):
    """r' is the residual then; an infinite scale times the zeros that stand for y would be NaN."""
    for scale in (0.5, float("inf"), float("nan")):
        assert _launched(lib, lambda: f(lib, y=None, w_post=None, scale=scale, **parts)) and lib.seen_res_scale() == 1.0
    assert _launched(lib, lambda: f(lib, scale=0.25)) and lib.seen_res_scale() == 0.25
