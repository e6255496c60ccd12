"""Infinities and NaN in the inputs of awq_block_norm and its gradient: NaN, infinities and finite values lie where the
formulas put them in float64. The finite values that are left beside them are products of zero, copies, or one product of
three factors (3 U and a rounding), U = 2^-24."""
import numpy as np
import pytest

from oracle import awq_moe as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import U, dev, half_step, host, within  # noqa: E402

EPS = 2.0 ** -20
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _make(seed, n, d, dtype, **parts):
    """Values away from zero (0 * inf would be another pattern); parts: names with the changes {element: value}."""
    rng = np.random.default_rng(seed)
    mk = lambda *s: rng.choice([-1.0, 1.0], s) * rng.uniform(0.25, 2.0, s)  # noqa: E731
    v = {"y": mk(n, d), "residual": mk(n, d), "w_pre": mk(d), "w_post": mk(d), "gate": mk(d), "d_res": mk(n, d), "d_h": mk(n, d)}
    for name, change in parts.items():
        if change is None:
            v[name] = None
            continue
        if name == "gate" and change.get("token"):
            v[name] = mk(n, d)
        for at, value in change.items():
            if at != "token":
                v[name][..., at] = value
    t = {k: None if a is None else dev(a, dtype) for k, a in v.items()}
    return t, {k: None if a is None else host(a) for k, a in t.items()}


def _forward(moe, t, v, a, dtype):
    got = moe.awq_block_norm(t["y"], t["residual"], t["w_pre"], t["w_post"], t["gate"], a, EPS)
    with np.errstate(invalid="ignore"):
        want = dict(zip(("residual", "h"), M.block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], a, EPS)))
    return got, want


def _backward(moe, t, v, a, wanted):
    got = moe.awq_block_norm_backward(t["y"], t["residual"], t["d_res"], t["d_h"], t["w_pre"], t["w_post"], t["gate"], a, EPS,
                                      wanted=wanted)
    with np.errstate(invalid="ignore"):
        want = M.block_norm_backward(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], a, EPS, v["d_res"], v["d_h"])
    return got, want


# widths that leave lanes of a block without whole chunks, registers and wide rows; an element of the row's end, and one of
# the chunk before it that the moved-back last chunk covers too
RAGGED = [(3, 257, "bf16", 256), (2, 520, "bf16", 519), (3, 1037, "bf16", 1030), (3, 1037, "bf16", 1036), (2, 4100, "f32", 4099),
          (2, 4099, "f16", 4093), (2, 20000, "bf16", 19999), (1, 28670, "f32", 28666)]


@pytest.mark.parametrize("name,token", [("gate", False), ("gate", True), ("w_post", False)])
@pytest.mark.parametrize("n,d,dtype,at", RAGGED)
def test_infinite_weights_at_the_end_of_ragged_rows(moe, n, d, dtype, at, name, token):
    """One infinity in r' makes its norm infinite: h is 0 wherever r' is finite, and NaN where it is not."""
    t, v = _make(d, n, d, dtype, **{name: {at: INF, "token": token} if token else {at: INF}})
    got, want = _forward(moe, t, v, 0.5, dtype)
    assert np.isnan(want["h"]).sum() == n and np.all(np.delete(want["h"], at, 1) == 0)
    within(host(got["h"]), want["h"], 0.0, "h")


@pytest.mark.parametrize("name", ["gate", "w_post"])
@pytest.mark.parametrize("n,d,dtype,at", [c for c in RAGGED if c[1] <= 8192])
def test_gradients_of_infinite_weights_at_the_end_of_ragged_rows(moe, n, d, dtype, at, name):
    """Without a norm behind the residual: t is infinite in one element, and d_y = (t - u mean(t u)) / n1 in all."""
    t, v = _make(d, n, d, dtype, w_pre=None, d_h=None, **{name: {at: INF}})
    got, want = _backward(moe, t, v, 0.5, ["d_y"])
    assert np.isinf(want["d_y"]).sum() == n * (d - 1)
    within(host(got["d_y"]), want["d_y"], 0.0, "d_y")


@pytest.mark.parametrize("n,d,dtype,at", [c for c in RAGGED if c[1] <= 8192])
def test_gradients_of_an_infinite_norm_weight_at_the_end_of_ragged_rows(moe, n, d, dtype, at):
    t, v = _make(d, n, d, dtype, w_pre={at: INF})
    got, want = _backward(moe, t, v, 0.5, ["d_residual"])
    assert np.isinf(want["d_residual"]).sum() == n * (d - 1)
    within(host(got["d_residual"]), want["d_residual"], 0.0, "d_residual")


# registers, strips of columns, rows narrower than a chunk
@pytest.mark.parametrize("bad", [INF, float("nan")])
@pytest.mark.parametrize("name", ["residual", "y", "w_post", "gate"])
@pytest.mark.parametrize("d", [5, 520, 4096, 9003])
def test_a_gradient_that_does_not_pass_the_norm_does_not_see_its_input(moe, d, name, bad):
    """Without a norm behind it, d_residual is d_res_out whatever r' holds."""
    t, v = _make(d, 3, d, "bf16", w_pre=None, d_h=None, **{name: {d // 2: bad}})
    got, want = _backward(moe, t, v, 0.5, ["d_residual"])
    assert np.array_equal(host(got["d_residual"]), v["d_res"]) and np.array_equal(want["d_residual"], v["d_res"])


@pytest.mark.parametrize("bad", [INF, float("nan")])
@pytest.mark.parametrize("d", [5, 520, 4096, 9003])
def test_the_gradient_of_a_block_without_a_norm_does_not_see_its_output(moe, d, bad):
    """r' = residual + a gate y, without norms: d_y = a gate d_res_out, whatever y holds; d_gate has y in it."""
    t, v = _make(d, 3, d, "bf16", w_pre=None, w_post=None, d_h=None, y={d // 2: bad})
    got, want = _backward(moe, t, v, 0.5, ["d_y", "d_residual", "d_gate"])
    assert np.isfinite(want["d_y"]).all()
    hs = half_step("bf16")
    for k in ("d_y", "d_residual"):
        within(host(got[k]), want[k], (3 * U * (1 + hs) + hs) * np.abs(want[k]), k)
    within(host(got["d_gate"]), want["d_gate"], 6 * U * 3 * 4, "d_gate")  # three terms of at most a d_res y = 2


@pytest.mark.parametrize("scale", [INF, float("nan")])
@pytest.mark.parametrize("d", [5, 520, 28672])
def test_without_y_the_residual_scale_is_not_used(moe, d, scale):
    t, v = _make(d, 3, d, "bf16", y=None, w_post=None, gate=None)
    ref = moe.awq_block_norm(None, t["residual"], t["w_pre"], eps=EPS)["h"]
    assert torch.isfinite(ref).all()
    assert torch.equal(moe.awq_block_norm(None, t["residual"], t["w_pre"], res_scale=scale, eps=EPS)["h"], ref)
    args = (None, t["residual"], t["d_res"], t["d_h"], t["w_pre"], None, None)
    ref = moe.awq_block_norm_backward(*args, 1.0, EPS)
    got = moe.awq_block_norm_backward(*args, scale, EPS)
    assert all(torch.equal(got[k], ref[k]) for k in ref)
