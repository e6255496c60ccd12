"""awq_block_norm and its gradient on the GPU against oracle/awq_moe.py in float64.

Bounds. Every float32 operation is off by at most U = 2^-24 of its result. A sum of squares over a row is a
chain of at most 32 additions in a thread, 6 across a wave and 16 across waves, so it is within 56 U, its
square root's reciprocal within 28 U plus the division, root, addition and product (4 U): 32 U. A value of
a stage is a sum of at most three products with such factors: within C1 = 64 of U times the sum of the
magnitudes that form it. r' takes one stage; h two (its norm sees r' off by a stage: where r' is smaller than the
sum of its terms' magnitudes, k = |terms| / |r'| in the 2-norm, the norm's relative error grows by k). The
gradients take at most four stages, each with the magnitudes of the one before: C4 = 256. The sums over
tokens add a chain of (rows per block) + (blocks / 16) + 16 additions. A 16-bit result is rounded once: half
a step of its value. U times 1e-3 absolute covers results below float16's normal range (2^-24 is half of its
step there, so the bound adds U)."""
import numpy as np
import pytest

from oracle import awq_moe as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import DTYPES, U, dev, half_step, host, pitched, within  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _inputs(rng, n, d, gate):
    mk = lambda *s: rng.normal(size=s)  # noqa: E731
    return {"y": mk(n, d) * 3, "residual": mk(n, d), "w_pre": 1 + 0.3 * mk(d), "w_post": 1 + 0.3 * mk(d),
            "gate": {"channel": lambda: mk(d), "token": lambda: mk(n, d), None: lambda: None}[gate]()}


def _dev_inputs(v, dtype):
    t = {k: None if a is None else dev(a, dtype) for k, a in v.items()}
    return t, {k: None if a is None else host(a) for k, a in t.items()}


def _norm(x, eps):
    return np.sqrt(np.mean(x * x, 1, keepdims=True) + eps)


def _terms(v, a, eps):
    """Magnitudes that form r', and the factor k of the docstring."""
    r = np.abs(v["residual"])
    if v["y"] is not None:
        z = np.abs(v["y"])
        if v["w_post"] is not None:
            z = z / _norm(v["y"], eps) * np.abs(v["w_post"])
        r = r + abs(a) * (z if v["gate"] is None else np.abs(v["gate"]) * z)
    real, _ = M.block_norm(v["y"], v["residual"], None, v["w_post"], v["gate"], a, eps)
    k = 1 + np.sqrt(np.sum(r * r, 1, keepdims=True) / np.maximum(np.sum(real * real, 1, keepdims=True), 1e-30))
    return r, real, k


def _check_forward(got, v, a, eps, dtype):
    want, h = M.block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], a, eps)
    hs, (mag, _, k) = half_step(dtype), _terms(v, a, eps)
    if "residual" in got:
        within(host(got["residual"]), want, 64 * U * mag + hs * np.abs(want) + U, "residual")
    if "h" in got:
        tol = 128 * U * k * mag / _norm(want, eps) * np.abs(v["w_pre"]) + hs * np.abs(h) * (1 + 256 * U * k) + U
        within(host(got["h"]), h, tol, "h")


def _check_backward(got, v, g, a, eps, dtype):
    want = M.block_norm_backward(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], a, eps, g["d_res"], g["d_h"])
    hs, (mag, real, k) = half_step(dtype), _terms(v, a, eps)
    n = real.shape[0]
    c = 256 * U * k
    D = np.zeros_like(real) if g["d_res"] is None else np.abs(g["d_res"])
    tols = {}
    rows = (n + 255) // 256 + 64  # the chain over tokens, for any number of blocks of at least 256
    if v["w_pre"] is not None:
        n2 = _norm(real, eps)
        u2, gh = mag / n2, np.abs(g["d_h"] * v["w_pre"])
        D = D + (gh + u2 * np.mean(gh * u2, 1, keepdims=True)) / n2
        tols["d_w_pre"] = np.sum((c + rows * U) * np.abs(g["d_h"]) * u2, 0)
    tols["d_residual"] = c * D
    if v["y"] is not None:
        n1 = _norm(v["y"], eps) if v["w_post"] is not None else 1.0
        u1 = np.abs(v["y"]) / n1
        z = u1 if v["w_post"] is None else u1 * np.abs(v["w_post"])
        gt = 1.0 if v["gate"] is None else np.abs(v["gate"])
        dz = abs(a) * D * gt
        t = dz if v["w_post"] is None else dz * np.abs(v["w_post"])
        tols["d_y"] = c * t if v["w_post"] is None else c * (t + u1 * np.mean(t * u1, 1, keepdims=True)) / n1
        tols["d_w_post"] = np.sum((c + rows * U) * dz * u1, 0)
        dg = abs(a) * D * z
        tols["d_gate"] = c * dg if np.ndim(v["gate"]) == 2 else np.sum((c + rows * U) * dg, 0)
    for name, t in got.items():
        rounded = 0.0 if t.dtype == torch.float32 else hs * np.abs(want[name]) * (1 + 256 * U) + U
        within(host(t), want[name], tols[name] * (1 + hs) + rounded + 1e-30, name)
    return want


SHAPES = [(1, 1), (3, 5), (2, 64), (1, 4096), (5, 511), (4, 520), (3, 1032), (7, 2047), (2, 4100), (3, 8192), (2, 11008),
          (1, 16392), (2, 28672), (1, 32768), (300, 128), (1030, 257)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,d", SHAPES)
def test_forward_and_backward(moe, dtype, n, d):
    rng = np.random.default_rng(n * 100003 + d)
    gate = ["channel", "token", None][(n + d) % 3]
    print(f"[gpu norm] n={n} d={d} {dtype} gate={gate}", flush=True)
    t, v = _dev_inputs(_inputs(rng, n, d, gate), dtype)
    eps = float(np.float32(1e-6))
    got = moe.awq_block_norm(t["y"], t["residual"], t["w_pre"], t["w_post"], t["gate"], 0.5, eps)
    assert sorted(got) == ["h", "residual"]
    _check_forward(got, v, 0.5, eps, dtype)
    g = {"d_res": dev(rng.normal(size=(n, d)), dtype), "d_h": dev(rng.normal(size=(n, d)), dtype)}
    got = moe.awq_block_norm_backward(t["y"], t["residual"], g["d_res"], g["d_h"], t["w_pre"], t["w_post"], t["gate"], 0.5,
                                      eps)
    assert sorted(got) == sorted(["d_residual", "d_y", "d_w_pre", "d_w_post"] + (["d_gate"] if gate else []))
    _check_backward(got, v, {k: host(x) for k, x in g.items()}, 0.5, eps, dtype)


# with the norm before the next block, the norm after the block, a block's output, its gate, a gradient of r'
PARTS = [(pre, post, block, gate, d_res) for pre, post, block in ((True, False, True), (False, True, True), (False, False, True),
                                                                  (True, False, False))
         for gate in (None, "channel", "token") for d_res in (True, False) if (block or not gate) and (pre or d_res)]


@pytest.mark.parametrize("n,d", [(5, 300), (3, 9003), (700, 7)])
@pytest.mark.parametrize("pre,post,block,gate,with_d_res", PARTS)
def test_parts_left_out(moe, pre, post, block, gate, with_d_res, n, d):
    rng = np.random.default_rng(17)
    v = _inputs(rng, n, d, gate)
    for name, there in (("w_pre", pre), ("w_post", post), ("y", block)):
        v[name] = v[name] if there else None
    t, v = _dev_inputs(v, "bf16")
    eps = float(np.float32(1e-5))
    got = moe.awq_block_norm(t["y"], t["residual"], t["w_pre"], t["w_post"], t["gate"], -1.25, eps)
    assert sorted(got) == (["h"] if pre else []) + (["residual"] if block else [])
    _check_forward(got, v, -1.25, eps, "bf16")
    d_res = dev(rng.normal(size=(n, d)), "bf16") if with_d_res else None
    d_h = dev(rng.normal(size=(n, d)), "bf16") if pre else None
    got = moe.awq_block_norm_backward(t["y"], t["residual"], d_res, d_h, t["w_pre"], t["w_post"], t["gate"], -1.25, eps)
    _check_backward(got, v, {"d_res": None if d_res is None else host(d_res), "d_h": None if d_h is None else host(d_h)},
                    -1.25, eps, "bf16")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [1037, 8221])
def test_pitched_unaligned_rows_and_in_place(moe, dtype, d):
    rng = np.random.default_rng(23)
    n, ld, eps = 6, d + 6, float(np.float32(1e-6))
    t, v = _dev_inputs(_inputs(rng, n, d, "token"), dtype)
    y, _ = pitched(v["y"], dtype, ld)
    r, rbuf = pitched(v["residual"], dtype, ld + 2)
    gate, _ = pitched(v["gate"], dtype, ld + 5)
    h, hbuf = pitched(np.zeros((n, d)), dtype, ld + 1)
    ref = moe.awq_block_norm(t["y"], t["residual"], t["w_pre"], t["w_post"], t["gate"], 0.5, eps)
    got = moe.awq_block_norm(y, r, t["w_pre"], t["w_post"], gate, 0.5, eps, out={"residual": r, "h": h})  # r in place
    assert got["residual"].data_ptr() == r.data_ptr() and got["h"].data_ptr() == h.data_ptr()
    assert torch.equal(r, ref["residual"]) and torch.equal(h, ref["h"])
    for buf, step in ((rbuf, ld + 2), (hbuf, ld + 1)):  # what lies between the rows is untouched
        assert buf[0] == 7 and torch.all(buf[1:].view(n, step)[:, d:] == 7)
    d_res, d_h = dev(rng.normal(size=(n, d)), dtype), dev(rng.normal(size=(n, d)), dtype)
    args = dict(w_pre=t["w_pre"], w_post=t["w_post"], res_scale=0.5, eps=eps)
    ref = moe.awq_block_norm_backward(t["y"], t["residual"], d_res, d_h, gate=t["gate"], **args)
    dr, dbuf = pitched(host(d_res), dtype, ld)
    dh, _ = pitched(host(d_h), dtype, ld)
    got = moe.awq_block_norm_backward(y, t["residual"], dr, dh, gate=gate, out={"d_residual": dr, "d_y": dh}, **args)
    assert got["d_residual"] is dr and got["d_y"] is dh
    for name in ref:
        assert torch.equal(got[name], ref[name]), name
    assert torch.all(dbuf[1:].view(n, ld)[:, d:] == 7)


def test_rows_of_zeros_infinities_and_nan_stay_their_own(moe):
    rng = np.random.default_rng(29)
    v = _inputs(rng, 6, 520, "channel")
    v["y"][0], v["residual"][1] = 0.0, 0.0
    v["y"][2, 3], v["residual"][3, 7], v["y"][4, 5] = np.nan, np.nan, np.inf
    t, v = _dev_inputs(v, "f32")
    eps = float(np.float32(1e-6))
    got = moe.awq_block_norm(t["y"], t["residual"], t["w_pre"], t["w_post"], t["gate"], 0.5, eps)
    fine = {k: None if a is None else (a[[0, 1, 5]] if a.ndim == 2 else a) for k, a in v.items()}
    _check_forward({k: x[[0, 1, 5]] for k, x in got.items()}, fine, 0.5, eps, "f32")
    assert torch.isnan(got["h"][2:4]).all() and torch.isnan(got["h"][4]).any()


def test_the_gradients_of_one_row_and_of_many_agree_with_differences(moe):
    """The kernel's gradients against central differences of the oracle in float64 along random directions:
    sum(grad * delta) is off by at most the summed bounds of _check_backward, and the difference by h^2."""
    rng = np.random.default_rng(31)
    eps, a = float(np.float32(1e-3)), 0.75
    for n, d in ((1, 40), (600, 24)):
        t, v = _dev_inputs(_inputs(rng, n, d, "channel"), "f32")
        d_res, d_h = dev(rng.normal(size=(n, d)), "f32"), dev(rng.normal(size=(n, d)), "f32")
        got = moe.awq_block_norm_backward(t["y"], t["residual"], d_res, d_h, t["w_pre"], t["w_post"], t["gate"], a, eps)
        for name, key in (("d_y", "y"), ("d_residual", "residual"), ("d_w_pre", "w_pre"), ("d_w_post", "w_post"),
                          ("d_gate", "gate")):
            delta = rng.normal(size=v[key].shape)

            def loss(s):
                w = {**v, key: v[key] + s * delta}
                r, h = M.block_norm(w["y"], w["residual"], w["w_pre"], w["w_post"], w["gate"], a, eps)
                return np.sum(r * host(d_res)) + np.sum(h * host(d_h))

            step = 1e-4
            want = (loss(step) - loss(-step)) / (2 * step)
            parts = host(got[name]) * delta
            # the third derivative along delta is of the loss's own size times (|delta| / |x|)^3: 1e-8 * 1e2
            assert abs(parts.sum() - want) < 1e-5 * np.abs(parts).sum() + 1e-6 * abs(want), name


def test_wanted_limits_what_is_computed(moe):
    rng = np.random.default_rng(37)
    t, _ = _dev_inputs(_inputs(rng, 9, 260, "channel"), "f16")
    d_res, d_h = dev(rng.normal(size=(9, 260)), "f16"), dev(rng.normal(size=(9, 260)), "f16")
    args = (t["y"], t["residual"], d_res, d_h, t["w_pre"], t["w_post"], t["gate"])
    full = moe.awq_block_norm_backward(*args)
    for wanted in (["d_y"], ["d_residual"], ["d_w_pre"], ["d_w_post", "d_y"], ["d_gate"]):
        got = moe.awq_block_norm_backward(*args, wanted=wanted)
        assert sorted(got) == sorted(wanted)
        for name in wanted:
            assert torch.equal(got[name], full[name]), name
    with pytest.raises(ValueError, match="d_gate"):
        moe.awq_block_norm_backward(*args[:6], wanted=["d_gate"])
    ws = torch.empty(moe.awq_block_norm_backward_workspace_bytes(9, 260), dtype=torch.uint8, device="cuda")
    got = moe.awq_block_norm_backward(*args, workspace=ws)
    assert all(torch.equal(got[k], full[k]) for k in full)
    with pytest.raises(ValueError, match="workspace"):
        moe.awq_block_norm_backward(*args, workspace=ws[:-1])


def test_refusals(moe):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.awq_block_norm(x, x[:3], w)
    with pytest.raises(TypeError):
        moe.awq_block_norm(x, x, w.float())
    with pytest.raises(ValueError):
        moe.awq_block_norm(x, x, w[:63])
    with pytest.raises(ValueError):
        moe.awq_block_norm(x.t(), x.t(), torch.ones(4, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        moe.awq_block_norm(x, x, w, gate=w[None].expand(4, 64))
    with pytest.raises(ValueError):
        moe.awq_block_norm(x, x, w, out={"h": torch.empty((4, 65), dtype=torch.bfloat16, device="cuda")})
    with pytest.raises(moe.AwqError) as e:
        moe.awq_block_norm(x[:0], x[:0], w)
    assert e.value.status in (1, 3)  # an empty tensor has no pointer either
    with pytest.raises(moe.AwqError):
        moe.awq_block_norm(x, x, w, eps=-1.0)
    big = torch.zeros((1, 32776), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(moe.AwqError) as e:
        moe.awq_block_norm(big, big, big[0])
    assert e.value.status == 5
