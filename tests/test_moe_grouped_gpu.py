"""The experts' 4-bit products on the GPU against oracle/awq_moe.py.

* Exact-arithmetic inputs (activations in [-8, 8], power-of-two steps): every product and partial sum is exact in
  float32, so plain products and their gradients equal the oracle bit for bit whatever the order.
* Others: an output is a chain of at most K = d_in (d_out for the gradient) float32 additions of exact products:
  |y - y*| <= K U sum |x| |w|, U = 2^-24, and half a step of a 16-bit result. For the gated product with g and u off
  by dg and du: silu' and relu' are at most 1.1, silu(g) is at most |g|, and e^-g adds (|g| + 8) 2 U relative, so
  |h - h*| <= 1.1 dg (|u| + du) + (|g| + dg) du + (|g| + 8) 2 U |h|, and its rounding. U absolute covers float16's
  subnormal step."""
import numpy as np
import pytest

from oracle import awq_moe as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import DTYPES, U, dev, export, export_dev, half_step, host, within  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _offsets(rng, n_rows, e, kept):
    """A random split of `kept` of n_rows rows over e experts, some of them without any."""
    cuts = np.sort(rng.integers(0, kept + 1, e - 1)) if e > 1 else np.zeros(0, int)
    if e > 3:
        cuts[1] = cuts[0]  # an empty expert
    return np.concatenate([[0], np.sort(cuts), [kept]]).astype(np.int32)


def _case(rng, n_rows, e, d_in, d_out, dtype, exact, kept=None, backward=False):
    ex = export(rng, e, d_out, d_in, exact)
    off = _offsets(rng, n_rows, e, n_rows if kept is None else kept)
    width = d_out if backward else d_in
    x = rng.integers(-8, 9, (n_rows, width)).astype(np.float64) if exact else rng.normal(size=(n_rows, width))
    x[off[-1]:] = np.nan  # rows past the last expert's are not read
    pitch = (width + 7) // 8 * 8
    xt = torch.full((n_rows, pitch), 3.0, dtype=DTYPES[dtype], device="cuda")[:, :width]
    xt.copy_(dev(x, dtype))
    return xt, ex, torch.from_numpy(off).cuda(), off


def _plain_bound(x, W, off, K, backward, want, hs):
    mag = M.grouped(np.abs(x), [np.abs(w) for w in W], off, np.zeros(want.shape), backward=backward)
    return K * U * mag * (1 + hs) + hs * np.abs(want) + (U if hs else 0)


# rows that are few for an expert, some tens, hundreds and thousands; ragged outputs, groups and rows
SHAPES = [(1, 1, 128, 1), (1, 8, 256, 40), (2, 8, 4096, 64), (7, 3, 384, 300), (16, 1, 640, 33), (40, 60, 128, 272),
          (64, 4, 1152, 48), (100, 5, 256, 520), (300, 2, 384, 260), (513, 7, 128, 130), (1030, 3, 256, 264),
          (2100, 2, 640, 520), (4200, 12, 128, 96), (700, 2, 256, 64), (650, 2, 256, 40), (700, 1, 384, 192), (2100, 3, 128, 128)]
# outputs of enough 256 x 256 tiles for these; odd and even steps of the contraction, tails below and above 128 rows
SHAPES += [(16400, 3, 256, 520), (9000, 5, 640, 1100), (33000, 12, 128, 100), (11000, 3, 640, 520), (25700, 40, 128, 300)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("out", ["f32", "same"])
@pytest.mark.parametrize("n_rows,e,d_in,d_out", SHAPES)
@pytest.mark.parametrize("backward", [False, True])
def test_exact_arithmetic_bit_exact(moe, dtype, out, n_rows, e, d_in, d_out, backward):
    rng = np.random.default_rng(n_rows * 31 + d_in + d_out)
    print(f"[gpu grouped] exact rows={n_rows} e={e} d_in={d_in} d_out={d_out} {dtype} out={out} backward={backward}", flush=True)
    kept = n_rows - n_rows // 10
    x, ex, off_t, off = _case(rng, n_rows, e, d_in, d_out, dtype, True, kept, backward)
    ot = torch.float32 if out == "f32" else DTYPES[dtype]
    y = torch.full((n_rows, d_in if backward else d_out), 7.0, dtype=ot, device="cuda")
    f = moe.awq_w4a16_grouped_gemm_backward if backward else moe.awq_w4a16_grouped_gemm
    got = f(x, *export_dev(*ex), off_t, **{"dx" if backward else "y": y})
    assert got is y
    want = M.grouped(host(x), M.expert_weights(*ex, dtype), off, np.full(y.shape, 7.0), backward=backward)
    assert np.array_equal(want.astype(np.float32).astype(np.float64), want)  # exact indeed
    want_t = torch.from_numpy(want).to(ot)
    bad = (got.cpu() != want_t).numpy()
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} differ, first at {np.argwhere(bad)[0]}"


# many experts with few, some and tens of rows and outputs for thousands of waves; rows too long for shared memory;
# experts' tiles that fill the compute units
@pytest.mark.parametrize("n_rows,e,d_in,d_out", [(130, 40, 128, 3300), (300, 40, 128, 3300), (700, 40, 128, 3300),
                                                 (1200, 40, 128, 3300), (3, 2, 34816, 20), (60, 4, 34816, 18), (450, 9, 256, 2200),
                                                 (3200, 64, 1024, 40), (3200, 64, 1024, 90)])
@pytest.mark.parametrize("backward", [False, True])
def test_exact_arithmetic_of_many_experts_and_long_rows(moe, n_rows, e, d_in, d_out, backward):
    test_exact_arithmetic_bit_exact(moe, "bf16", "same", n_rows, e, d_in, d_out, backward)
    test_exact_arithmetic_bit_exact(moe, "f16", "f32", n_rows, e, d_in, d_out, backward)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n_rows,e,d_in,d_out", [(3, 8, 4096, 66), (50, 4, 512, 130), (700, 3, 1280, 200), (2500, 2, 384, 300),
                                                 (17000, 2, 384, 300)])
def test_real_values(moe, dtype, n_rows, e, d_in, d_out):
    rng = np.random.default_rng(n_rows + d_out)
    for backward in (False, True):
        x, ex, off_t, off = _case(rng, n_rows, e, d_in, d_out, dtype, False, backward=backward)
        W = M.expert_weights(*ex, dtype)
        f = moe.awq_w4a16_grouped_gemm_backward if backward else moe.awq_w4a16_grouped_gemm
        for ot, hs in ((torch.float32, 0.0), (DTYPES[dtype], half_step(dtype))):
            got = f(x, *export_dev(*ex), off_t, out_dtype=ot)
            want = M.grouped(host(x), W, off, np.zeros(got.shape), backward=backward)
            within(host(got), want, _plain_bound(host(x), W, off, d_out if backward else d_in, backward, want, hs), "y")


@pytest.mark.parametrize("act", ["silu", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n_rows,e,d_in,d_out", [(1, 2, 128, 2), (2, 8, 4096, 96), (30, 3, 640, 130), (90, 4, 256, 258),
                                                 (300, 3, 384, 520), (1300, 4, 256, 258), (2600, 1, 128, 1030), (17000, 4, 256, 258), (34000, 1, 128, 130)])
def test_gated(moe, act, dtype, n_rows, e, d_in, d_out):
    rng = np.random.default_rng(n_rows + d_in)
    kept = n_rows - n_rows // 20
    x, ex, off_t, off = _case(rng, n_rows, e, d_in, d_out, dtype, False, kept)
    W, half = M.expert_weights(*ex, dtype), d_out // 2
    gu = M.grouped(host(x), W, off, np.zeros((n_rows, d_out)))
    mag = M.grouped(np.abs(host(x)), [np.abs(w) for w in W], off, np.zeros((n_rows, d_out)))
    g, u = gu[:, :half], gu[:, half:]
    dg, du = d_in * U * mag[:, :half], d_in * U * mag[:, half:]
    for ot, hs in ((torch.float32, 0.0), (DTYPES[dtype], half_step(dtype))):
        y = torch.full((n_rows, half), 7.0, dtype=ot, device="cuda")
        got = moe.awq_w4a16_grouped_gemm(x, *export_dev(*ex), off_t, act=act, y=y)
        want = M.grouped(host(x), W, off, np.full((n_rows, half), 7.0), act=act)
        tol = 1.1 * dg * (np.abs(u) + du) + (np.abs(g) + dg) * du + (np.abs(g) + 8) * 2 * U * np.abs(want)
        within(host(got), want, tol * (1 + hs) + hs * np.abs(want) + U, act)


def test_strided_rows_and_outputs(moe):
    rng = np.random.default_rng(43)
    for n_rows in (9, 400, 2100, 33000):
        x, ex, off_t, off = _case(rng, n_rows, 3, 256, 72, "bf16", True)
        wide = torch.full((n_rows, 264), 3.0, dtype=torch.bfloat16, device="cuda")
        wide[:, :256] = x
        buf = torch.full((n_rows, 77), 5.0, device="cuda")
        got = moe.awq_w4a16_grouped_gemm(wide[:, :256], *export_dev(*ex), off_t, y=buf[:, 1:73])
        ref = moe.awq_w4a16_grouped_gemm(x, *export_dev(*ex), off_t, out_dtype=torch.float32)
        assert torch.equal(got, ref) and torch.all(buf[:, 0] == 5) and torch.all(buf[:, 73:] == 5)
        dy = torch.full((n_rows, 80), 3.0, dtype=torch.bfloat16, device="cuda")
        dy[:, :72] = torch.from_numpy(rng.integers(-4, 5, (n_rows, 72))).to(torch.bfloat16)
        buf = torch.full((n_rows, 261), 5.0, dtype=torch.bfloat16, device="cuda")
        got = moe.awq_w4a16_grouped_gemm_backward(dy[:, :72], *export_dev(*ex), off_t, dx=buf[:, 3:259])
        ref = moe.awq_w4a16_grouped_gemm_backward(dy[:, :72].contiguous(), *export_dev(*ex), off_t)
        assert torch.equal(got, ref) and torch.all(buf[:, :3] == 5) and torch.all(buf[:, 259:] == 5)


@pytest.mark.parametrize("n_rows", [5, 200, 2100, 33000])
def test_non_finite_rows_stay_their_own(moe, n_rows):
    rng = np.random.default_rng(47)
    x, ex, off_t, off = _case(rng, n_rows, 2, 256, 64, "bf16", True)
    ref = moe.awq_w4a16_grouped_gemm(x, *export_dev(*ex), off_t)
    x2 = x.clone()
    x2[n_rows // 2, 5], x2[0, 7] = float("nan"), float("inf")
    got = moe.awq_w4a16_grouped_gemm(x2, *export_dev(*ex), off_t)
    fine = torch.ones(n_rows, dtype=torch.bool)
    fine[[0, n_rows // 2]] = False
    assert torch.equal(got.cpu()[fine], ref.cpu()[fine])
    assert torch.isnan(got[n_rows // 2]).all() and not torch.isfinite(got[0]).all()


@pytest.mark.parametrize("n_rows", [5, 40, 60, 200, 33000])
def test_non_finite_gradients_stay_their_own(moe, n_rows):
    rng = np.random.default_rng(59)
    dy, ex, off_t, off = _case(rng, n_rows, 2, 256, 70, "bf16", True, backward=True)
    assert dy.stride(0) == 72  # what fills the pitch, and the next row, is not multiplied
    ref = moe.awq_w4a16_grouped_gemm_backward(dy, *export_dev(*ex), off_t)
    wide = torch.as_strided(dy, (n_rows, 72), (72, 1))
    wide[:, 70:] = float("nan")
    assert torch.equal(moe.awq_w4a16_grouped_gemm_backward(dy, *export_dev(*ex), off_t), ref)
    dy[n_rows // 2, 69], dy[0, 7] = float("nan"), float("inf")
    got = moe.awq_w4a16_grouped_gemm_backward(dy, *export_dev(*ex), off_t)
    fine = torch.ones(n_rows, dtype=torch.bool)
    fine[[0, n_rows // 2]] = False
    assert torch.equal(got.cpu()[fine], ref.cpu()[fine])
    assert torch.isnan(got[n_rows // 2]).all() and not torch.isfinite(got[0]).all()


def test_no_rows_at_all_and_offsets_outside_the_rows(moe):
    """Offsets are the caller's to change: they are clamped to the rows and to ascend."""
    rng = np.random.default_rng(53)
    for n_rows in (6, 300, 2100, 33000):
        x, ex, off_t, off = _case(rng, n_rows, 4, 128, 32, "bf16", True)
        y = torch.full((n_rows, 32), 7.0, device="cuda")
        moe.awq_w4a16_grouped_gemm(x, *export_dev(*ex), torch.zeros_like(off_t), y=y)
        assert torch.all(y == 7)
        wild = torch.tensor([-5, n_rows // 2, n_rows // 2, n_rows // 2, 1 << 30], dtype=torch.int32, device="cuda")
        tame = torch.tensor([0, n_rows // 2, n_rows // 2, n_rows // 2, n_rows], dtype=torch.int32, device="cuda")
        for f in (moe.awq_w4a16_grouped_gemm,):
            assert torch.equal(f(x, *export_dev(*ex), wild), f(x, *export_dev(*ex), tame))
        dy = x[:, :32].contiguous()
        f = moe.awq_w4a16_grouped_gemm_backward
        assert torch.equal(f(dy, *export_dev(*ex), wild), f(dy, *export_dev(*ex), tame))


def test_one_expert_is_the_plain_product(moe):
    """With one expert the call computes what awq_w4a16_gemm does (exact inputs: bit for bit)."""
    from post_quantization_mean_amd import binding as B
    rng = np.random.default_rng(59)
    for n_rows in (1, 24, 1200):
        x, ex, off_t, off = _case(rng, n_rows, 1, 384, 80, "f16", True)
        codes, steps, zeros = export_dev(*ex)
        assert torch.equal(moe.awq_w4a16_grouped_gemm(x, codes, steps, zeros, off_t),
                           B.awq_w4a16_gemm(x, codes[0], steps[0], zeros[0], out_dtype=torch.float16))


def test_refusals(moe):
    rng = np.random.default_rng(61)
    x, ex, off, _ = _case(rng, 6, 4, 128, 32, "bf16", True)
    ex = export_dev(*ex)
    f = moe.awq_w4a16_grouped_gemm
    for bad in (lambda: f(x, ex[0][:, :, :32], *ex[1:], off), lambda: f(x, *ex, off[:-1]), lambda: f(x, *ex, off, act="tanh"),
                lambda: f(x, ex[0], ex[1][:3], ex[2], off), lambda: f(x[:, :64], *ex, off), lambda: f(x, ex[0][0], *ex[1:], off),
                lambda: f(x, *ex, off, y=torch.empty((6, 33), device="cuda")), lambda: f(x.t(), *ex, off),
                lambda: f(x, ex[0].transpose(0, 1).contiguous().transpose(0, 1), *ex[1:], off)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(x.float(), *ex, off), lambda: f(x, *ex, off.long()), lambda: f(x, *ex, off, out_dtype=torch.float16),
                lambda: f(x, ex[0].int(), *ex[1:], off)):
        with pytest.raises(TypeError):
            bad()
    wide = torch.zeros((6, 132), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.AwqError) as e:  # rows that are not 16-byte aligned
        f(wide[:, :128], *ex, off)
    assert e.value.status == 5
