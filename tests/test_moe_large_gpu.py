"""The mixture-of-experts block on buffers whose offsets pass 32 bits, and with slots that name the same row.

Rows far apart give the bits of the same rows side by side: the arithmetic does not depend on pitches."""
import numpy as np
import pytest

from oracle import awq_moe as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import U, dev, export, export_dev, half_step, host, within  # noqa: E402

FAR = (1 << 28) + 8  # elements from row to row: nine rows and more pass 2^31 elements


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _far(t, buf):
    """The rows of t, FAR elements apart in buf."""
    n, d = t.shape
    m = buf.view(-1)[:(n - 1) * FAR + d].as_strided((n, d), (FAR, 1))
    m.copy_(t)
    return m


@pytest.fixture(scope="module")
def bufs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return [torch.empty(13 * FAR, dtype=torch.bfloat16, device="cuda") for _ in range(3)]


def test_norms_of_rows_far_apart(moe, bufs):
    rng = np.random.default_rng(5)
    for d in (5, 333, 8200):
        y, r, dr, dh = (dev(rng.normal(size=(12, d)), "bf16") for _ in range(4))
        w1, w2, gate = (dev(1 + 0.3 * rng.normal(size=d), "bf16") for _ in range(3))
        print(f"[gpu large] norms d={d}", flush=True)
        ref = moe.awq_block_norm(y, r, w1, w2, gate, 0.5)
        fy, fr = _far(y, bufs[0]), _far(r, bufs[1])
        got = moe.awq_block_norm(fy, fr, w1, w2, gate, 0.5, out={"residual": fr, "h": fy})
        assert torch.equal(got["residual"], ref["residual"]) and torch.equal(got["h"], ref["h"])
        ref = moe.awq_block_norm_backward(y, r, dr, dh, w1, w2, gate, 0.5)
        fy, fr, fh = _far(y, bufs[0]), _far(r, bufs[1]), _far(dh, bufs[2])
        got = moe.awq_block_norm_backward(fy, fr, dr, fh, w1, w2, gate, 0.5, out={"d_y": fh})
        for name in ref:
            assert torch.equal(got[name], ref[name]), name


def test_routes_of_rows_far_apart(moe, bufs):
    rng = np.random.default_rng(7)
    ids = torch.from_numpy(rng.integers(0, 3, (6, 2))).cuda()
    pos = moe.awq_moe_sort(ids, 3)["position"]
    w = torch.rand((6, 2), device="cuda")
    for d in (3, 523):
        scales = torch.rand((3, d), device="cuda") + 0.5
        x, g = dev(rng.normal(size=(6, d)), "bf16"), dev(rng.normal(size=(6, d)), "bf16")
        print(f"[gpu large] routes d={d}", flush=True)
        ref = moe.awq_moe_gather(x, pos, ids, scales)
        rows = _far(torch.zeros_like(ref), bufs[0])
        assert torch.equal(moe.awq_moe_gather(_far(x, bufs[1]), pos, ids, scales, out=rows), ref)
        out = moe.awq_moe_combine(rows, pos, w, out=_far(x, bufs[1]))
        assert torch.equal(out, moe.awq_moe_combine(ref, pos, w))
        assert torch.equal(moe.awq_moe_gather_backward(rows, pos, ids, scales), moe.awq_moe_gather_backward(ref, pos, ids, scales))
        a = moe.awq_moe_combine_backward(g, ref, pos, w)
        b = moe.awq_moe_combine_backward(_far(g, bufs[1]), rows, pos, w, out={"d_rows": rows})
        assert torch.equal(a["d_rows"], b["d_rows"]) and torch.equal(a["d_weights"], b["d_weights"])


@pytest.mark.parametrize("n_rows,far", [(12, FAR), (600, (1 << 22) - 8)])
def test_products_of_rows_far_apart(moe, bufs, n_rows, far):
    rng = np.random.default_rng(11)
    ex = export_dev(*export(rng, 2, 264, 256, True))
    off = torch.tensor([0, n_rows // 2, n_rows], dtype=torch.int32, device="cuda")
    x, dy = dev(rng.integers(-8, 9, (n_rows, 256)), "bf16"), dev(rng.integers(-8, 9, (n_rows, 264)), "bf16")
    print(f"[gpu large] products n_rows={n_rows} pitch={far}", flush=True)

    def spread(t, buf):  # the products take inputs of pitches below 2^22
        m = buf.as_strided(t.shape, (min(far, (1 << 22) - 8), 1))
        m.copy_(t)
        return m

    for f, t, width in ((moe.awq_w4a16_grouped_gemm, x, 256 + 8), (moe.awq_w4a16_grouped_gemm_backward, dy, 256)):
        out = bufs[1].as_strided((n_rows, width), (far, 1))
        got = f(spread(t, bufs[0]), *ex, off, **{"y" if f is moe.awq_w4a16_grouped_gemm else "dx": out})
        assert torch.equal(got, f(t, *ex, off))


def test_slots_that_name_the_same_row(moe):
    rng = np.random.default_rng(13)
    pos = np.array([[0, 0, 1], [2, 1, 1], [2, 2, 2]], np.int32)
    ids = rng.integers(0, 4, (3, 3))
    rows, scales, w = dev(rng.normal(size=(4, 75)), "bf16"), np.exp(rng.normal(size=(4, 75))).astype(np.float32), rng.normal(size=(3, 3)).astype(np.float32)
    pt, it, hs, r = torch.from_numpy(pos).cuda(), torch.from_numpy(ids).cuda(), half_step("bf16"), host(rows)
    # three fused additions in float32 and one rounding
    got = moe.awq_moe_combine(rows, pt, torch.from_numpy(w).cuda())
    want, mag = M.combine(r, pos, w.astype(np.float64)), M.combine(np.abs(r), pos, np.abs(w.astype(np.float64)))
    within(host(got), want, 3 * U * mag * (1 + hs) + hs * np.abs(want), "out")
    got = moe.awq_moe_gather_backward(rows, pt, it, torch.from_numpy(scales).cuda())
    s = scales.astype(np.float64)
    want, mag = M.gather_backward(r, pos, ids, s), M.gather_backward(np.abs(r), pos, ids, s)
    within(host(got), want, 3 * U * mag * (1 + hs) + hs * np.abs(want), "d_x")
    x = dev(rng.normal(size=(3, 75)), "bf16")
    got, xs = moe.awq_moe_gather(x, pt, out=torch.zeros((4, 75), dtype=torch.bfloat16, device="cuda")), host(x)
    for row, from_ in ((0, [0]), (1, [0, 1]), (2, [1, 2])):
        assert np.all(np.any([host(got)[row] == xs[t] for t in from_], axis=0))
    assert torch.all(got[3] == 0)
