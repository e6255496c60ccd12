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


ELSE = FAKE + 0x1000000


@pytest.mark.parametrize("f,there", [
    (_norm, dict(y=ELSE, ld_y=72, res_out=ELSE, ld_ro=64)), (_norm, dict(residual=ELSE, ld_r=72, res_out=ELSE, ld_ro=64)),
    (_norm, dict(y=ELSE, ld_y=64, h=ELSE, ld_h=72)), (_norm, dict(residual=ELSE, ld_r=64, h=ELSE, ld_h=65)),
    (_norm_backward, dict(d_res=ELSE, ld_dr=64, d_residual=ELSE, ld_do=80)),
    (_norm_backward, dict(d_h=ELSE, ld_dh=80, d_y=ELSE, ld_dy=64))])
def test_in_place_with_another_pitch_is_refused(lib, f, there):
    """A row's output would lie over rows that other blocks still read. One row has no other, and equal pitches none over it."""
    apart = dict(y=FAKE, residual=FAKE + 0x10000, res_out=FAKE + 0x20000, h=FAKE + 0x30000) if f is _norm else \
        dict(d_res=FAKE, d_h=FAKE + 0x10000, d_y=FAKE + 0x20000, d_residual=FAKE + 0x30000)
    assert _launched(lib, lambda: f(lib, **apart))
    assert not _launched(lib, lambda: f(lib, **{**apart, **there})) and b"pitch" in lib.awq_last_error()
    assert _launched(lib, lambda: f(lib, **{**apart, **there}, n=1))
    same = {k: 72 if k.startswith("ld") else v for k, v in there.items()}
    assert _launched(lib, lambda: f(lib, **{**apart, **same}))


def test_combining_gradients_in_place_with_another_pitch_is_refused(lib):
    def call(rows, ld_rows, d_rows, ld_d_rows, n_rows=8):
        return lib.awq_moe_combine_backward(ELSE, 64, rows, ld_rows, BF16, n_rows, 64, FAKE, FAKE, 4, 2, d_rows, ld_d_rows, FAKE,
                                            None)
    assert _launched(lib, lambda: call(FAKE, 72, FAKE, 72)) and _launched(lib, lambda: call(FAKE, 72, ELSE, 64))
    assert not _launched(lib, lambda: call(FAKE, 72, FAKE, 64)) and b"pitch" in lib.awq_last_error()
    assert _launched(lib, lambda: call(FAKE, 72, FAKE, 64, n_rows=1))


def _grouped(lib, backward, n, ld_x, x=FAKE):
    """128 inputs and 300 outputs."""
    mode = () if backward else (0,)
    f = lib.awq_w4a16_grouped_gemm_backward if backward else lib.awq_w4a16_grouped_gemm
    return f(x, ld_x, BF16, FAKE, FAKE, FAKE, FAKE, 4, n, 128, 300, *mode, FAKE, 304, F32, None)


@pytest.mark.parametrize("backward,width", [(False, 128), (True, 300)])
def test_the_pitch_of_a_single_row_means_nothing(lib, backward, width):
    for ld in (width, width + 3, width + 4, 1 << 23):
        assert _launched(lib, lambda: _grouped(lib, backward, 1, ld)), ld
        assert lib.seen_ld_x() == (width + 7) // 8 * 8  # rows past the last one lie past the row's end for the kernels
        assert _launched(lib, lambda: _grouped(lib, backward, 2, ld)) == (ld % 8 == 0 and ld < 1 << 22)
    assert not _launched(lib, lambda: _grouped(lib, backward, 1, width - 1))
    assert not _launched(lib, lambda: _grouped(lib, backward, 1, width, FAKE + 8))
    assert _launched(lib, lambda: _grouped(lib, backward, 2, 304)) and lib.seen_ld_x() == 304
