"""awq_moe_sort, awq_moe_gather, awq_moe_combine and the gradients on the GPU against oracle/awq_moe.py.

Integer outputs are equal. Bounds of the others, U = 2^-24: a gathered value is one float32 product (U) and one
rounding; a combined one a chain of top_k fused additions, each off by at most U times the sum of the
magnitudes, and one rounding; d_weights a chain of at most d / 64 + 6 additions. U absolute covers
float16's subnormal step."""
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


def _ids(rng, n, k, e, dropped=0.1):
    ids = np.stack([rng.permutation(max(e, k))[:k] for _ in range(n)]).astype(np.int64)
    ids[rng.random((n, k)) < dropped] = -1
    return ids


@pytest.mark.parametrize("id_type", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,k,e", [(1, 1, 1), (1, 8, 64), (3, 2, 8), (64, 1, 1), (65, 1, 2), (257, 4, 60), (1024, 2, 8),
                                   (1025, 2, 1024), (4099, 3, 37), (20000, 8, 128), (1 << 18, 4, 300)])
def test_sort(moe, id_type, n, k, e):
    rng = np.random.default_rng(n + k + e)
    ids = rng.integers(-2, e + 2, (n, k))  # out of range on both sides; the same expert twice in a token too
    print(f"[gpu sort] n={n} k={k} e={e} {id_type}", flush=True)
    got = moe.awq_moe_sort(torch.from_numpy(ids).to(id_type).cuda(), e)
    for g, w, name in zip((got["offsets"], got["order"], got["position"]), M.sort_slots(ids, e), ("offsets", "order", "position")):
        assert np.array_equal(host(g), w), name


def test_sort_of_extremes(moe):
    for ids in (np.full((500, 8), -1), np.full((500, 8), 7), np.full((3000, 2), 1 << 40), np.arange(4096)[:, None] % 64,
                np.full((1, 1), -(1 << 62))):
        got = moe.awq_moe_sort(torch.from_numpy(ids).cuda(), 64)
        for g, w in zip((got["offsets"], got["order"], got["position"]), M.sort_slots(ids, 64)):
            assert np.array_equal(host(g), w)


def test_sort_into_given_buffers(moe):
    ids = torch.from_numpy(np.random.default_rng(3).integers(0, 8, (4000, 2))).cuda()
    ref = moe.awq_moe_sort(ids, 8)
    nb = moe.awq_moe_sort_workspace_bytes(4000, 2, 8)
    assert nb > 0
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    out = {"offsets": torch.empty(9, dtype=torch.int32, device="cuda"), "order": torch.empty(8000, dtype=torch.int32, device="cuda"),
           "position": torch.empty((4000, 2), dtype=torch.int32, device="cuda")}
    got = moe.awq_moe_sort(ids, 8, workspace=ws, out=out)
    for name in out:
        assert got[name] is out[name] and torch.equal(got[name], ref[name])
    with pytest.raises(ValueError):
        moe.awq_moe_sort(ids, 8, workspace=ws[:-1])
    with pytest.raises(ValueError):
        moe.awq_moe_sort(ids, 9, out=out)
    with pytest.raises(TypeError):
        moe.awq_moe_sort(ids.to(torch.int16), 8)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,e,d,scaled", [(1, 1, 1, 1, True), (1, 8, 64, 2048, True), (5, 2, 8, 130, False), (33, 3, 5, 515, True),
                                            (40, 8, 16, 2051, True), (17, 6, 60, 4096, False), (7, 2, 4, 11011, True)])
@pytest.mark.parametrize("strided", [False, True])
def test_gather_and_combine(moe, dtype, n, k, e, d, scaled, strided):
    rng = np.random.default_rng(n * 7 + d)
    print(f"[gpu route] n={n} k={k} e={e} d={d} {dtype} scaled={scaled} strided={strided}", flush=True)
    ids = _ids(rng, n, k, e)
    ids_t = torch.from_numpy(ids).cuda()
    pos_t = moe.awq_moe_sort(ids_t, e)["position"]
    pos, R = host(pos_t), n * k
    make = (lambda a: pitched(a, dtype, d + 3)[0]) if strided else (lambda a: dev(a, dtype))  # noqa: E731
    scales = torch.from_numpy(np.exp(0.5 * rng.normal(size=(e, d))).astype(np.float32)).cuda() if scaled else None
    sc = host(scales) if scaled else None
    kw = dict(expert_ids=ids_t, in_scales=scales) if scaled else {}
    x, rows, w = make(rng.normal(size=(n, d))), make(rng.normal(size=(R, d)) * 2), rng.normal(size=(n, k)).astype(np.float32)
    w[pos < 0] = np.nan  # the weights of dropped slots are not read
    wt, hs = torch.from_numpy(w).cuda(), half_step(dtype)

    buf = make(np.full((R, d), 5.0))
    got = moe.awq_moe_gather(x, pos_t, out=buf, **kw)
    want = M.gather(host(x), pos, ids, sc, np.full((R, d), 5.0))
    within(host(got), want, (U + hs) * np.abs(want) * (1 + U) + U, "rows")

    got = moe.awq_moe_combine(rows, pos_t, wt, out=make(np.zeros((n, d))))
    want, mag = M.combine(host(rows), pos, w.astype(np.float64)), M.combine(np.abs(host(rows)), pos, np.abs(w.astype(np.float64)))
    within(host(got), want, k * U * mag + hs * np.abs(want) * (1 + k * U) + hs * k * U * mag + U, "out")

    g = make(rng.normal(size=(n, d)))
    got = moe.awq_moe_combine_backward(g, rows, pos_t, wt, out={"d_rows": make(np.full((R, d), 5.0))})
    want, dw = M.combine_backward(host(g), host(rows), pos, w.astype(np.float64), np.full((R, d), 5.0))
    within(host(got["d_rows"]), want, (U + hs) * np.abs(want) * (1 + U) + U, "d_rows")
    _, mag = M.combine_backward(np.abs(host(g)), np.abs(host(rows)), pos, np.abs(w.astype(np.float64)), np.zeros((R, d)))
    within(host(got["d_weights"]), dw, (d / 64 + 7) * U * mag, "d_weights")

    got = moe.awq_moe_gather_backward(rows, pos_t, out=make(np.zeros((n, d))), **kw)
    want, mag = M.gather_backward(host(rows), pos, ids, sc), M.gather_backward(np.abs(host(rows)), pos, ids, sc)
    within(host(got), want, k * U * mag * (1 + hs) + hs * np.abs(want) * (1 + k * U) + U, "d_x")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,k,d", [(4099, 4, 2051), (9001, 2, 1000), (16811, 1, 1024), (1100003, 1, 17), (300007, 2, 9),
                                   (270011, 3, 3)])
def test_many_rows(moe, dtype, n, k, d):
    """Rows of more than 32 MiB, and tokens past one dimension of a grid, against torch in float64 on the device
    (one factor or k terms each: the bounds of the test above)."""
    print(f"[gpu route] many rows n={n} k={k} d={d} {dtype}", flush=True)
    g = torch.Generator("cuda").manual_seed(n)
    e, t, hs = 7, DTYPES[dtype], half_step(dtype)
    ids = torch.randint(-1, e, (n, k), generator=g, device="cuda")
    pos = moe.awq_moe_sort(ids, e)["position"]
    scales = torch.rand((e, d), generator=g, device="cuda") + 0.5
    x = torch.randn((n, d), generator=g, device="cuda").to(t)
    w = torch.randn((n, k), generator=g, device="cuda")
    at, kept = pos.clamp(min=0).long(), pos >= 0

    def near(got, want, tol):
        for a in range(0, len(want), 8192):
            assert bool((torch.abs(got[a:a + 8192].double() - want[a:a + 8192]) <= tol[a:a + 8192]).all())

    def rows_of(factor):  # the kept slots' rows from x and factors [n, d] per choice, fives elsewhere
        want = torch.full((n * k, d), 5.0, dtype=torch.float64, device="cuda")
        for j in range(k):
            want[at[kept[:, j], j]] = (x.double() * factor(j))[kept[:, j]]
        return want

    for kw, factor in (({}, lambda j: 1.0), (dict(expert_ids=ids, in_scales=scales), lambda j: scales[ids[:, j].clamp(min=0)].double())):
        want = rows_of(factor)
        got = moe.awq_moe_gather(x, pos, out=torch.full((n * k, d), 5.0, dtype=t, device="cuda"), **kw)
        near(got, want, (U + hs) * want.abs() * (1 + U) + U)
        back = moe.awq_moe_gather_backward(got, pos, **kw)
        terms = [torch.where(kept[:, j, None], got[at[:, j]].double() * factor(j), 0.0) for j in range(k)]
        want, mag = sum(terms), sum(v.abs() for v in terms)
        near(back, want, k * U * mag * (1 + hs) + hs * want.abs() * (1 + k * U) + U)
    rows = got
    out = moe.awq_moe_combine(rows, pos, w)
    terms = [torch.where(kept[:, j, None], rows[at[:, j]].double() * w[:, j, None].double(), 0.0) for j in range(k)]
    want, mag = sum(terms), sum(v.abs() for v in terms)
    near(out, want, k * U * mag * (1 + hs) + hs * want.abs() * (1 + k * U) + U)
    b = moe.awq_moe_combine_backward(x, rows, pos, w, out={"d_rows": torch.full((n * k, d), 5.0, dtype=t, device="cuda")})
    want = rows_of(lambda j: w[:, j, None].double())
    near(b["d_rows"], want, (U + hs) * want.abs() * (1 + U) + U)
    for j in range(k):
        terms = torch.where(kept[:, j, None], rows[at[:, j]].double() * x.double(), 0.0)
        near(b["d_weights"][:, j:j + 1], terms.sum(1, keepdim=True), (d / 64 + 7) * U * terms.abs().sum(1, keepdim=True))


def test_rows_past_the_buffer_and_bad_entries_are_skipped(moe):
    """position is the caller's to change: entries outside [0, n_rows), and ids outside the experts, are skipped."""
    x = torch.ones((3, 64), dtype=torch.float32, device="cuda")
    pos = torch.tensor([[0, 9], [-7, 2], [1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    rows = moe.awq_moe_gather(x, pos, out=torch.full((4, 64), 5.0, device="cuda"))
    assert rows[:, 0].tolist() == [1.0, 5.0, 1.0, 5.0]
    w = torch.ones((3, 2), device="cuda")
    assert moe.awq_moe_combine(rows, pos, w)[:, 0].tolist() == [1.0, 1.0, 0.0]
    b = moe.awq_moe_combine_backward(x, rows, pos, w, out={"d_rows": torch.full((4, 64), 3.0, device="cuda")})
    assert b["d_weights"].tolist() == [[64.0, 0.0], [0.0, 64.0], [0.0, 0.0]] and b["d_rows"][:, 5].tolist() == [1.0, 3.0, 1.0, 3.0]
    ids = torch.tensor([[0, 1], [0, 5], [0, -1]], dtype=torch.int32, device="cuda")
    rows = moe.awq_moe_gather(x, pos, expert_ids=ids, in_scales=torch.full((2, 64), 2.0, device="cuda"),
                              out=torch.full((4, 64), 5.0, device="cuda"))
    assert rows[:, 0].tolist() == [2.0, 5.0, 5.0, 5.0]


def test_a_token_without_experts_and_masked_infinities(moe):
    ids = torch.tensor([[-1, -1], [1, 0], [-1, 1]], device="cuda")
    plan = moe.awq_moe_sort(ids, 2)
    rows = torch.full((6, 128), float("inf"), dtype=torch.bfloat16, device="cuda")
    rows[:3] = torch.tensor([[2.0], [3.0], [4.0]], dtype=torch.bfloat16, device="cuda")  # rows from 3 on belong to nobody
    w = torch.tensor([[float("nan"), float("inf")], [1.0, 10.0], [float("nan"), 0.5]], device="cuda")
    out = moe.awq_moe_combine(rows, plan["position"], w)
    assert host(plan["offsets"]).tolist() == [0, 1, 3]
    assert torch.all(out[0] == 0) and torch.all(out[1] == 23) and torch.all(out[2] == 2)
    assert torch.all(moe.awq_moe_gather_backward(rows, plan["position"])[0] == 0)


def test_backward_in_place_and_single_outputs(moe):
    rng = np.random.default_rng(41)
    ids = torch.from_numpy(_ids(rng, 20, 3, 6)).cuda()
    pos = moe.awq_moe_sort(ids, 6)["position"]
    rows, g = dev(rng.normal(size=(60, 520)), "bf16"), dev(rng.normal(size=(20, 520)), "bf16")
    w = torch.rand((20, 3), device="cuda")
    ref = moe.awq_moe_combine_backward(g, rows, pos, w, out={"d_rows": rows.clone()})
    buf = rows.clone()
    got = moe.awq_moe_combine_backward(g, buf, pos, w, out={"d_rows": buf})
    assert torch.equal(got["d_rows"], ref["d_rows"]) and torch.equal(got["d_weights"], ref["d_weights"])


def test_refusals(moe):
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    for bad in (lambda: moe.awq_moe_gather(x, pos.long()), lambda: moe.awq_moe_combine(x, pos, w.double()),
                lambda: moe.awq_moe_gather(x.double(), pos)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: moe.awq_moe_gather(x, pos[:3]), lambda: moe.awq_moe_combine(x, pos, w[:, :1]),
                lambda: moe.awq_moe_gather(x, pos, in_scales=torch.ones((2, 64), device="cuda")),
                lambda: moe.awq_moe_gather(x, pos, expert_ids=pos, in_scales=torch.ones((2, 63), device="cuda")),
                lambda: moe.awq_moe_combine_backward(x[:3], x, pos, w),
                lambda: moe.awq_moe_gather(x, pos, out=torch.empty((8, 65), dtype=torch.bfloat16, device="cuda")),
                lambda: moe.awq_moe_combine(x, pos.t(), w)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.AwqError) as e:
        moe.awq_moe_sort(torch.zeros((4, 65), dtype=torch.int32, device="cuda"), 8)
    assert e.value.status == 4
