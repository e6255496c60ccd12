"""awq_rope and awq_rope_backward on the GPU against oracle/awq_attn.py.

Bounds, U = 2^-24: the cosine and sine are within 2 U (the reduced angle's rounding, the series' roundings, its end), their
product with the scale adds U, the two products and their sum 2 U: 5 U (|x_a| + |x_b|) |scale|, and one rounding of the
result. U absolute covers float16's subnormal step. Copied channels are equal."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import DTYPES, U, dev, half_step, host, within  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _case(rng, n, heads, d, rot, axes, dtype, far=100000):
    x = host(dev(rng.standard_normal((n, heads, d)), dtype))
    positions = rng.integers(-far, far, (axes, n))
    inv_freq = (10000.0 ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)
    axis = rng.integers(0, axes, rot // 2).astype(np.int32)
    return x, positions, inv_freq, axis


def _bound(x, y, rot, pairs, scale, dtype):
    half = rot // 2
    mag = np.abs(x[..., :rot])
    if pairs:
        s = np.repeat(mag[..., 0::2] + mag[..., 1::2], 2, -1)
    else:
        s = np.tile(mag[..., :half] + mag[..., half:], 2)
    b = np.zeros(x.shape)
    b[..., :rot] = 5 * U * s * abs(scale) + half_step(dtype) * np.abs(y[..., :rot]) * (1 + 5 * U) + U
    return b


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("style", ["half", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,heads,d,rot,axes", [(1, 1, 2, 2, 1), (1, 40, 128, 128, 1), (7, 3, 80, 80, 2), (65, 5, 128, 64, 3),
                                                (33, 72, 128, 128, 3), (9, 2, 30, 18, 2), (5, 9, 512, 512, 8), (4, 300, 34, 2, 1),
                                                (3, 1, 511, 6, 3), (2, 1024, 16, 16, 1)])
def test_rope(attn, n, heads, d, rot, axes, dtype, style, backward):
    rng = np.random.default_rng(n + heads + d + rot)
    print(f"[gpu rope] n={n} heads={heads} d={d} rot={rot} axes={axes} {dtype} {style} backward={backward}", flush=True)
    x, positions, inv_freq, axis = _case(rng, n, heads, d, rot, axes, dtype)
    scale = 1.25 if rot == 64 else 1.0
    f = attn.awq_rope_backward if backward else attn.awq_rope
    p = torch.from_numpy(positions).to(torch.int64 if n % 2 else torch.int32).cuda()
    got = f(dev(x, dtype), p, torch.from_numpy(inv_freq).cuda(), axis=None if axes == 1 else torch.from_numpy(axis).cuda(), style=style,
            scale=scale)
    want = A.rope(x, positions, inv_freq, None if axes == 1 else axis, style == "pairs", scale, backward)
    within(host(got), want, _bound(x, want, rot, style == "pairs", scale, dtype), "rope")


@pytest.mark.parametrize("layout", ["fused", "odd", "heads first"])
@pytest.mark.parametrize("style", ["half", "pairs"])
def test_rope_of_views_and_in_place(attn, style, layout):
    rng = np.random.default_rng(5)
    n, heads, d, rot = 37, 6, 96, 64
    x, positions, inv_freq, axis = _case(rng, n, heads, d, rot, 3, "bf16")
    p, f, a = (torch.from_numpy(t).cuda() for t in (positions, inv_freq, axis))
    want = attn.awq_rope(dev(x, "bf16"), p, f, a, style)
    if layout == "fused":  # the first heads of a wider row
        buf = torch.full((n, heads + 5, d), 7.0, dtype=torch.bfloat16, device="cuda")
        view = buf[:, :heads]
    elif layout == "odd":  # rows that start anywhere
        buf = torch.full((n * heads * 101 + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
        view = buf[1:].view(n, heads, 101)[..., :d]
    else:
        buf = torch.full((heads, n, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
        view = buf.transpose(0, 1)[..., :d]
    view.copy_(dev(x, "bf16"))
    assert torch.equal(attn.awq_rope(view, p, f, a, style), want)
    rest = int((buf == 7).sum())
    assert attn.awq_rope(view, p, f, a, style, out=view) is view
    assert torch.equal(view, want) and int((buf == 7).sum()) == rest
    # positions that are a part of a wider matrix
    wide = torch.zeros((3, n + 11), dtype=torch.int32, device="cuda")
    wide[:, 4:n + 4] = p
    assert torch.equal(attn.awq_rope(dev(x, "bf16"), wide[:, 4:n + 4], f, a, style), want)


def test_rope_far_positions_and_bad_axes(attn):
    rng = np.random.default_rng(6)
    x, _, inv_freq, _ = _case(rng, 64, 2, 64, 64, 1, "f32")
    inv_freq[:4] = [1.0, 0.75, 3.0, 1e-30]
    positions = rng.integers(-(1 << 31) + 1, 1 << 31, (1, 64))
    positions[0, :4] = [0, 1, (1 << 31) - 1, -(1 << 31) + 1]
    got = attn.awq_rope(dev(x, "f32"), torch.from_numpy(positions).cuda(), torch.from_numpy(inv_freq).cuda())
    want = A.rope(x, positions, inv_freq, None, False, 1.0)
    within(host(got), want, _bound(x, want, 64, False, 1.0, "f32"), "far")
    axis = np.array([0, 1, -1, 5, 2, 1 << 30, -(1 << 31), 0] * 4, np.int32)
    positions = rng.integers(0, 5000, (3, 64))
    got = attn.awq_rope(dev(x, "f32"), torch.from_numpy(positions).cuda(), torch.from_numpy(inv_freq).cuda(), torch.from_numpy(axis).cuda())
    want = A.rope(x, positions, inv_freq, axis, False, 1.0)
    within(host(got), want, _bound(x, want, 64, False, 1.0, "f32"), "axes")


@pytest.mark.parametrize("style", ["half", "pairs"])
def test_rope_gradient_is_the_transpose(attn, style):
    """The rotation is linear: column i of its matrix is the difference that one in channel i makes, to float32's rounding."""
    d, rot = 12, 10
    positions = torch.tensor([[3], [17]], dtype=torch.int32, device="cuda")
    f = torch.tensor([1.0, 0.5, 0.25, 0.03, 0.001], device="cuda")
    axis = torch.tensor([0, 1, 0, 1, 1], dtype=torch.int32, device="cuda")
    base = torch.randn((1, 1, d), device="cuda")
    at = attn.awq_rope(base, positions, f, axis, style, 0.5)
    jac = torch.stack([attn.awq_rope(base + torch.eye(d, device="cuda")[i], positions, f, axis, style, 0.5) - at for i in range(d)])[:, 0, 0]
    back = torch.stack([attn.awq_rope_backward(torch.eye(d, device="cuda")[i][None, None], positions, f, axis, style, 0.5) for i in range(d)])[:, 0, 0]
    # jac[i, j] = d out_j / d x_i; back[j, i] the same; values below 8 leave differences 2^-20 off
    assert float((jac - back.t()).abs().max()) < 2.0 ** -19
    x, g = torch.randn((50, 3, d), device="cuda"), torch.randn((50, 3, d), device="cuda")
    p = torch.randint(0, 9999, (2, 50), device="cuda")
    a = (attn.awq_rope(x, p, f, axis, style).double() * g).sum()
    b = (attn.awq_rope_backward(g, p, f, axis, style).double() * x).sum()
    assert abs(float(a - b)) < 50 * 3 * d * 2.0 ** -19


def test_rope_passes_nan_and_infinity(attn):
    x = torch.ones((2, 1, 8), device="cuda")
    x[0, 0, 1], x[1, 0, 7] = float("nan"), float("inf")
    y = attn.awq_rope(x, torch.zeros(2, dtype=torch.int32, device="cuda"), torch.ones(3, device="cuda"))
    assert host(torch.isnan(y[0, 0])).tolist() == [0, 1, 0, 0, 1, 0, 0, 0] and float(y[1, 0, 7]) == float("inf")
