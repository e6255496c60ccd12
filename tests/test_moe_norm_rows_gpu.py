"""awq_block_norm and its gradient with more rows than a launch has blocks, so that a block takes several rows in turn,
against the formulas in float64 on the device.

Bounds as in test_moe_norm_gpu.py: r' within 64 U of the magnitudes that form it (U = 2^-24), h within 128 U k, gradients
within 256 U k, where k = 1 + |terms| / |r'| carries what r' is off through its norm. A sum over tokens adds its chain of
additions: the rows of one block (at least 32 blocks share them, or there is one row each), the blocks of one of 16 runs (at
most 4096 / 16) and the runs. A 16-bit result is off by half a step more, and U covers float16 below its normal range."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import DTYPES, U, half_step  # noqa: E402

EPS = 2.0 ** -20


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def inputs(seed, n, d, dtype, gate="channel", pre=True, post=True, block=True):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    v = {"residual": rnd(n, d), "y": 3 * rnd(n, d) if block else None, "w_pre": 1 + 0.3 * rnd(d) if pre else None,
         "w_post": 1 + 0.3 * rnd(d) if post else None,
         "gate": {"channel": lambda: rnd(d), "token": lambda: rnd(n, d), None: lambda: None}[gate]()}
    grads = {"d_res": rnd(n, d), "d_h": rnd(n, d) if pre else None}
    to = lambda m: {k: None if t is None else t.to(DTYPES[dtype]) for k, t in m.items()}  # noqa: E731
    return to(v), to(grads)


def near(got, want, tol, name):
    """|got - want| <= tol, with NaN and infinities in the same places."""
    got, tol = got.double(), torch.as_tensor(tol, device=got.device).expand(want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{name}: infinities"
    off = (got - want).abs()[fine] - tol[fine]
    assert not off.numel() or off.max() <= 0, f"{name}: {float(off.max()):.3g} past the bound in {int((off > 0).sum())}"


def reference(v, g, a):
    """(outputs, bounds in units of the magnitudes) in float64."""
    f = {k: None if t is None else t.double() for k, t in {**v, **(g or {})}.items()}
    rms = lambda t: torch.sqrt(t.square().mean(1, keepdim=True) + EPS)  # noqa: E731
    r, block = f["residual"], f["y"] is not None
    n, one = r.shape[0], torch.ones((), dtype=torch.float64, device=r.device)
    n1 = rms(f["y"]) if f["w_post"] is not None else one
    w1, gt = (one if f[k] is None else f[k] for k in ("w_post", "gate"))
    u1 = f["y"] / n1 if block else None
    real, mag = (r + a * gt * u1 * w1, r.abs() + abs(a) * (gt * u1 * w1).abs()) if block else (r, r.abs())
    k = 1 + torch.sqrt(mag.square().sum(1, keepdim=True) / real.square().sum(1, keepdim=True).clamp(min=1e-30))
    want, tol = {}, {}
    if block:
        want["residual"], tol["residual"] = real, 64 * U * mag
    n2 = rms(real)
    if f["w_pre"] is not None:
        want["h"], tol["h"] = real / n2 * f["w_pre"], 128 * U * k * mag / n2 * f["w_pre"].abs()
    if g is None:
        return want, tol
    want, tol, c = {}, {}, 256 * U * k
    chain = (n + 31) // 32 + 4096 // 16 + 16
    D, M = (torch.zeros_like(r), torch.zeros_like(r)) if f["d_res"] is None else (f["d_res"], f["d_res"].abs())
    if f["w_pre"] is not None:
        u2, m2, gh = real / n2, mag / n2, f["d_h"] * f["w_pre"]
        D = D + (gh - u2 * (gh * u2).mean(1, keepdim=True)) / n2
        M = M + (gh.abs() + m2 * (gh.abs() * m2).mean(1, keepdim=True)) / n2
        want["d_w_pre"], tol["d_w_pre"] = (f["d_h"] * u2).sum(0), ((c + chain * U) * f["d_h"].abs() * m2).sum(0)
    want["d_residual"], tol["d_residual"] = D, c * M
    if block:
        dz, mz = a * D * gt, abs(a) * M * gt.abs()
        t, mt = dz * w1, mz * w1.abs()
        if f["w_post"] is None:
            want["d_y"], tol["d_y"] = t, c * mt
        else:
            want["d_y"] = (t - u1 * (t * u1).mean(1, keepdim=True)) / n1
            tol["d_y"] = c * (mt + u1.abs() * (mt * u1.abs()).mean(1, keepdim=True)) / n1
            want["d_w_post"], tol["d_w_post"] = (dz * u1).sum(0), ((c + chain * U) * mz * u1.abs()).sum(0)
        if f["gate"] is not None:
            dg, mg = a * D * u1 * w1, abs(a) * M * (u1 * w1).abs()
            token = f["gate"].dim() == 2
            want["d_gate"] = dg if token else dg.sum(0)
            tol["d_gate"] = c * mg if token else ((c + chain * U) * mg).sum(0)
    return want, tol


def check(got, want, tol, dtype):
    hs = half_step(dtype)
    assert sorted(got) == sorted(want)
    for name, t in got.items():
        rounded = 0.0 if t.dtype == torch.float32 else hs * want[name].abs() * (1 + 256 * U) + U
        near(t, want[name], tol[name] * (1 + hs) + rounded + 1e-30, name)


# rows past the blocks of every variant: one chunk a thread (ragged), two, weights kept and the next row loaded ahead;
# gradients of one, two, three chunks (ahead) and four (float32, not ahead); rows past 8192 in strips of columns; forward
# rows past 16384 without the kept weights (four chunks; float32 eight); rows narrower than a chunk
ROWS = [(4500, 257, ("bf16", "f32")), (2100, 520, ("bf16", "f16")), (1200, 4096, ("bf16", "f16", "f32")),
        (700, 6000, ("f32",)), (700, 8192, ("f32", "bf16")), (600, 11008, ("bf16", "f32")), (600, 20000, ("f16",)),
        (300, 28672, ("bf16", "f32")), (9000, 7, ("bf16",)), (530000, 3, ("f32", "f16"))]
CASES = [(n, d, t) for n, d, types in ROWS for t in types]


@pytest.mark.parametrize("gate", ["channel", "token", None])
@pytest.mark.parametrize("n,d,dtype", CASES)
def test_blocks_that_take_several_rows(moe, n, d, dtype, gate):
    print(f"[gpu norm rows] n={n} d={d} {dtype} gate={gate}", flush=True)
    v, g = inputs(n + d, n, d, dtype, gate)
    got = moe.awq_block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], 0.5, EPS)
    check(got, *reference(v, None, 0.5), dtype)
    got = moe.awq_block_norm_backward(v["y"], v["residual"], g["d_res"], g["d_h"], v["w_pre"], v["w_post"], v["gate"], 0.5, EPS)
    check(got, *reference(v, g, 0.5), dtype)


@pytest.mark.parametrize("pre,post", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("n,d,dtype", [(4500, 257, "bf16"), (1200, 4096, "bf16"), (700, 8192, "f32"), (300, 28672, "bf16")])
def test_several_rows_with_one_norm_or_none(moe, n, d, dtype, pre, post):
    """One sum over a row, or none, between a row and the next one."""
    print(f"[gpu norm rows] n={n} d={d} {dtype} pre={pre} post={post}", flush=True)
    v, g = inputs(n, n, d, dtype, "token", pre, post)
    got = moe.awq_block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], -1.25, EPS)
    check(got, *reference(v, None, -1.25), dtype)
    got = moe.awq_block_norm_backward(v["y"], v["residual"], g["d_res"], g["d_h"], v["w_pre"], v["w_post"], v["gate"], -1.25, EPS)
    check(got, *reference(v, g, -1.25), dtype)


@pytest.mark.parametrize("n,d,dtype", [(4500, 257, "bf16"), (2100, 520, "f16"), (1200, 4096, "bf16"), (700, 8192, "f32")])
def test_several_rows_in_place(moe, n, d, dtype):
    """r' over the residual, h over y; d_residual over d_res_out, d_y over d_h: the bits of separate outputs."""
    v, g = inputs(n, n, d, dtype, "token")
    args = dict(w_pre=v["w_pre"], w_post=v["w_post"], gate=v["gate"], res_scale=0.5, eps=EPS)
    ref = moe.awq_block_norm(v["y"], v["residual"], **args)
    back = moe.awq_block_norm_backward(v["y"], v["residual"], g["d_res"], g["d_h"], **args)
    y, r = v["y"].clone(), v["residual"].clone()
    moe.awq_block_norm(y, r, out={"residual": r, "h": y}, **args)
    assert torch.equal(r, ref["residual"]) and torch.equal(y, ref["h"])
    got = moe.awq_block_norm_backward(v["y"], v["residual"], g["d_res"], g["d_h"], out={"d_residual": g["d_res"], "d_y": g["d_h"]},
                                      **args)
    for name in back:
        assert torch.equal(got[name], back[name]), name


@pytest.mark.parametrize("n,d,dtype", [(4500, 257, "bf16"), (2100, 520, "bf16"), (1200, 4096, "bf16"), (1200, 4096, "f32"),
                                       (600, 11008, "f16"), (300, 28672, "bf16")])
def test_the_first_norm_of_a_model_takes_several_rows(moe, n, d, dtype):
    """Without y every row's r' is its residual, the rows behind a block's first one too."""
    print(f"[gpu norm rows] first norm n={n} d={d} {dtype}", flush=True)
    v, g = inputs(n, n, d, dtype, None, post=False, block=False)
    got = moe.awq_block_norm(None, v["residual"], v["w_pre"], eps=EPS)
    check(got, *reference(v, None, 1.0), dtype)
    got = moe.awq_block_norm_backward(None, v["residual"], g["d_res"], g["d_h"], v["w_pre"], eps=EPS)
    check(got, *reference(v, g, 1.0), dtype)
