"""The C ABI of the mixture-of-experts block without a GPU: every symbol include/awq_moe.h declares is
exported and bound, and bad arguments are refused on the host before anything reaches the device. Fake
non-NULL pointers are used only in calls that must fail validation."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
b = pytest.importorskip("post_quantization_mean_amd.binding")
moe = pytest.importorskip("post_quantization_mean_amd.moe")
torch = pytest.importorskip("torch")

FAKE = 0x10000  # never dereferenced: every call below fails validation first
OK, NULL, SHAPE, NO_TOKENS, ARG, UNSUPPORTED, WORKSPACE = range(7)
F32, BF16, F16 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(b.LIB_PATH):
        pytest.skip("library not built")
    return moe._load()


def _err(lib):
    return lib.awq_last_error().decode()


def test_every_declared_symbol_is_exported_and_bound(lib):
    src = open(os.path.join(ROOT, "include", "awq_moe.h"), encoding="utf-8").read()
    names = sorted(set(re.findall(r"AWQ_API[^;(]*?\b(awq_\w+)\s*\(", src)))
    assert sorted(moe.exported_symbols()) == names
    for n in names:
        assert hasattr(lib, n), n


def _norm(lib, **kw):
    v = dict(y=FAKE, ld_y=64, residual=FAKE, ld_r=64, dtype=BF16, n=4, d=64, w_post=FAKE, gate=None, ld_gate=0, scale=1.0,
             w_pre=FAKE, eps=1e-6, res_out=FAKE, ld_ro=64, h=FAKE + 64, ld_h=64)
    assert not set(kw) - set(v)
    v.update(kw)
    return lib.awq_block_norm(*v.values(), None)


@pytest.mark.parametrize("want,kw", [
    (UNSUPPORTED, dict(dtype=3)), (UNSUPPORTED, dict(dtype=-1)),
    (SHAPE, dict(n=-1)), (NO_TOKENS, dict(n=0)), (SHAPE, dict(d=0)), (UNSUPPORTED, dict(n=1 << 31)),
    (UNSUPPORTED, dict(d=32769, ld_y=40000, ld_r=40000)),
    (NULL, dict(residual=None)), (NULL, dict(y=None)), (NULL, dict(y=None, w_post=None, gate=FAKE)),
    (NULL, dict(y=None, w_post=None)),  # res_out without y
    (NULL, dict(w_pre=None)), (NULL, dict(h=None)), (NULL, dict(w_pre=None, h=None, res_out=None)),
    (ARG, dict(ld_y=63)), (ARG, dict(ld_r=0)), (ARG, dict(ld_ro=63)), (ARG, dict(ld_h=-64)),
    (ARG, dict(gate=FAKE, ld_gate=63)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=float("nan"))), (ARG, dict(eps=float("inf"))),
    (ARG, dict(h=FAKE)),  # h in res_out
    (UNSUPPORTED, dict(y=FAKE + 1)), (UNSUPPORTED, dict(w_pre=FAKE + 1)), (UNSUPPORTED, dict(dtype=F32, h=FAKE + 2)),
])
def test_block_norm_refusals(lib, want, kw):
    assert _norm(lib, **kw) == want, _err(lib)
    assert _err(lib)


def _norm_backward(lib, **kw):
    ws = lib.awq_block_norm_backward_workspace_bytes(4, 64)
    v = dict(y=FAKE, ld_y=64, residual=FAKE, ld_r=64, dtype=F16, n=4, d=64, w_post=FAKE, gate=FAKE, ld_gate=0, scale=1.0,
             w_pre=FAKE, eps=1e-6, d_res=FAKE, ld_dr=64, d_h=FAKE, ld_dh=64, d_y=FAKE, ld_dy=64, d_residual=FAKE, ld_do=64,
             d_w_post=FAKE, d_w_pre=FAKE, d_gate=FAKE, ld_dg=0, ws=FAKE, nb=ws)
    assert not set(kw) - set(v)
    v.update(kw)
    return lib.awq_block_norm_backward(*v.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NO_TOKENS, dict(n=0)), (UNSUPPORTED, dict(dtype=9)), (NULL, dict(d_h=None)), (NULL, dict(w_pre=None)),
    (NULL, dict(w_pre=None, d_h=None, d_res=None)), (NULL, dict(w_post=None)), (NULL, dict(gate=None)),
    (NULL, dict(d_y=None, d_residual=None, d_w_post=None, d_w_pre=None, d_gate=None)),
    (NULL, dict(y=None, w_post=None, gate=None, d_w_post=None, d_gate=None)),  # d_y without y
    (ARG, dict(ld_dr=63)), (ARG, dict(ld_dh=1)), (ARG, dict(ld_dy=63)), (ARG, dict(ld_do=63)),
    (ARG, dict(ld_gate=64, ld_dg=63)), (UNSUPPORTED, dict(d_w_post=FAKE + 2)), (UNSUPPORTED, dict(d_gate=FAKE + 2)),
    (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(nb=16)), (UNSUPPORTED, dict(ws=FAKE + 64)),
])
def test_block_norm_backward_refusals(lib, want, kw):
    assert _norm_backward(lib, **kw) == want, _err(lib)


def test_workspace_queries(lib):
    assert lib.awq_block_norm_backward_workspace_bytes(0, 64) == 0
    assert lib.awq_block_norm_backward_workspace_bytes(4, 32769) == 0
    nb = lib.awq_block_norm_backward_workspace_bytes(1, 65)
    assert nb >= 3 * 65 * 4 and nb % 256 == 0
    assert lib.awq_moe_sort_workspace_bytes(1, 8, 64) == 0  # one launch, nothing kept
    assert lib.awq_moe_sort_workspace_bytes(1 << 20, 8, 64) > 0
    for bad in ((0, 8, 64), (4, 0, 64), (4, 65, 64), (4, 8, 0), (4, 8, 1025), (1 << 40, 8, 64)):
        assert lib.awq_moe_sort_workspace_bytes(*bad) == 0


def _sort(lib, **kw):
    v = dict(ids=FAKE, id_bytes=8, n=4, k=2, e=8, offsets=FAKE, order=FAKE, position=FAKE, ws=None, nb=0)
    v.update(kw)
    return lib.awq_moe_sort(*v.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NO_TOKENS, dict(n=0)), (SHAPE, dict(n=-4)), (ARG, dict(k=0)), (ARG, dict(k=65)), (ARG, dict(e=0)), (ARG, dict(e=1025)),
    (UNSUPPORTED, dict(n=(1 << 22) + 1)), (UNSUPPORTED, dict(n=1 << 62, k=64)), (UNSUPPORTED, dict(id_bytes=2)),
    (NULL, dict(ids=None)), (UNSUPPORTED, dict(ids=FAKE + 4)), (NULL, dict(offsets=None)), (NULL, dict(order=None)),
    (NULL, dict(position=None)), (WORKSPACE, dict(n=1 << 20)), (WORKSPACE, dict(n=1 << 20, ws=FAKE, nb=64)),
    (UNSUPPORTED, dict(n=1 << 20, ws=FAKE + 8, nb=1 << 30)),
])
def test_sort_refusals(lib, want, kw):
    assert _sort(lib, **kw) == want, _err(lib)


def _gather(lib, **kw):
    v = dict(x=FAKE, ld_x=64, dtype=F32, n=4, d=64, position=FAKE, k=2, ids=FAKE, id_bytes=4, scales=FAKE, e=8, rows=FAKE,
             ld_rows=64, n_rows=8)
    v.update(kw)
    return lib.awq_moe_gather(*v.values(), None)


@pytest.mark.parametrize("want,kw", [
    (NO_TOKENS, dict(n=0)), (SHAPE, dict(d=0)), (UNSUPPORTED, dict(d=1 << 25, ld_x=1 << 25, ld_rows=1 << 25)),
    (UNSUPPORTED, dict(dtype=5)), (NULL, dict(x=None)), (NULL, dict(rows=None)), (NULL, dict(position=None)),
    (NULL, dict(ids=None)), (UNSUPPORTED, dict(id_bytes=1)), (ARG, dict(e=0)), (ARG, dict(ld_x=63)), (ARG, dict(ld_rows=8)),
    (SHAPE, dict(n_rows=-1)), (UNSUPPORTED, dict(n_rows=(1 << 23) + 1)), (UNSUPPORTED, dict(x=FAKE + 2)),
    (UNSUPPORTED, dict(scales=FAKE + 2)), (ARG, dict(k=0)),
])
def test_gather_refusals(lib, want, kw):
    assert _gather(lib, **kw) == want, _err(lib)


def test_combine_refusals(lib):
    f, g = lib.awq_moe_combine, lib.awq_moe_combine_backward
    assert f(FAKE, 64, BF16, 8, 64, FAKE, None, 4, 2, FAKE, 64, None) == NULL and "weights" in _err(lib)
    assert f(FAKE, 64, BF16, 8, 64, FAKE, FAKE, 0, 2, FAKE, 64, None) == NO_TOKENS
    assert f(FAKE, 64, BF16, 8, 64, FAKE, FAKE, 4, 2, FAKE, 63, None) == ARG
    assert f(None, 64, BF16, 8, 64, FAKE, FAKE, 4, 2, FAKE, 64, None) == NULL
    assert g(FAKE, 64, FAKE, 64, BF16, 8, 64, FAKE, FAKE, 4, 2, None, 64, None, None) == NULL
    assert g(FAKE, 63, FAKE, 64, BF16, 8, 64, FAKE, FAKE, 4, 2, FAKE, 64, FAKE, None) == ARG
    assert g(FAKE, 64, FAKE, 64, BF16, 8, 64, FAKE, FAKE, 4, 2, FAKE, 64, FAKE + 2, None) == UNSUPPORTED
    assert lib.awq_moe_gather_backward(FAKE, 64, BF16, 8, 64, None, 4, 2, None, 4, None, 0, FAKE, 64, None) == NULL


def _grouped(lib, backward=False, **kw):
    v = dict(x=FAKE, ld_x=128, dtype=BF16, codes=FAKE, steps=FAKE, zeros=FAKE, offsets=FAKE, e=4, n=8, d_in=128, d_out=32)
    if not backward:
        v["mode"] = 0
    v |= dict(y=FAKE, ld_y=128, y_dtype=F32)
    v.update(kw)
    return (lib.awq_w4a16_grouped_gemm_backward if backward else lib.awq_w4a16_grouped_gemm)(*v.values(), None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("want,kw", [
    (NO_TOKENS, dict(n=0)), (SHAPE, dict(n=-1)), (UNSUPPORTED, dict(n=(1 << 23) + 1)), (ARG, dict(e=0)), (ARG, dict(e=1025)),
    (SHAPE, dict(d_in=192)), (SHAPE, dict(d_in=0)), (SHAPE, dict(d_out=0)), (UNSUPPORTED, dict(dtype=F32)),
    (UNSUPPORTED, dict(y_dtype=F16)), (NULL, dict(x=None)), (NULL, dict(codes=None)), (NULL, dict(steps=None)),
    (NULL, dict(zeros=None)), (NULL, dict(offsets=None)), (NULL, dict(y=None)), (UNSUPPORTED, dict(x=FAKE + 8)),
    (UNSUPPORTED, dict(ld_x=132)), (UNSUPPORTED, dict(codes=FAKE + 8)), (UNSUPPORTED, dict(ld_x=1 << 22)),
    (ARG, dict(ld_y=16)), (ARG, dict(ld_x=24)), (UNSUPPORTED, dict(d_in=1 << 22, ld_x=1 << 23, ld_y=1 << 23)),
])
def test_grouped_refusals(lib, backward, want, kw):
    assert _grouped(lib, backward, **kw) == want, _err(lib)


def test_grouped_modes(lib):
    assert _grouped(lib, mode=3) == ARG and _grouped(lib, mode=-1) == ARG
    assert _grouped(lib, mode=1, d_out=33) == SHAPE
    assert _grouped(lib, mode=2, ld_y=15) == ARG  # 16 outputs


def test_binding_refuses_what_the_library_cannot_see():
    x = torch.zeros((4, 128), dtype=torch.bfloat16)
    pos = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        moe.awq_block_norm(x, x)
    with pytest.raises(TypeError, match="residual"):
        moe.awq_block_norm(x, x.double())
    with pytest.raises(ValueError, match="device"):
        moe.awq_moe_sort(torch.zeros((4, 2), dtype=torch.int64), 8)
    with pytest.raises(ValueError, match="top_k"):
        moe._slots(pos.reshape(-1), "position", torch.int32)
    with pytest.raises(TypeError, match="rows must be"):
        moe._export_args(x.float(), None, None, None, None)
    with pytest.raises(ValueError, match="codes"):
        moe._export_args(x, torch.zeros((2, 64), dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError, match="steps_f16"):
        moe._export_args(x, torch.zeros((2, 8, 64), dtype=torch.uint8), torch.zeros((2, 8, 2), dtype=torch.int16), None, None)
    with pytest.raises(ValueError, match="needs expert_ids"):
        moe._scale_args(torch.ones((2, 128)), None, 4, 2, 128, x.device)
    with pytest.raises(ValueError, match="act"):
        moe.awq_w4a16_grouped_gemm(x, None, None, None, None, act="gelu")
