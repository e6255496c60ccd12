"""awq_kv4_attention on the GPU against oracle/awq_attn.py; the bounds are attn_cases.attention_bound's, and one rounding of the
output. The logarithm of a row's sum: off by the scores' error and the numerators' 2^-10, and float32's rounding."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import attention_bound, cache_dev, paged, random_cache  # noqa: E402
from moe_cases import DTYPES, U, dev, half_step, host, within  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _run(attn, rng, q_len, kv_len, heads, kv, d, page, dtype="bf16", causal=True, window=0, max_kv=None, exact=False, out="same",
         apart=0, uniform=None, table_edit=None, cache=None, q_scale=1.5, check_lse=True):
    table, pages = paged(rng, kv_len, page, wide=rng.integers(0, 2))
    if table_edit:
        table_edit(table)
    codes, params = random_cache(rng, pages, kv, d, page, exact) if cache is None else cache(pages)
    offsets = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    n = int(offsets[-1])
    q = rng.integers(-4, 5, (n, heads, d)) / 4.0 if exact else q_scale * rng.standard_normal((n, heads, d))
    q = host(dev(q, dtype))
    c, p = cache_dev(codes, params, apart)
    kw = {}
    if uniform is None:
        uniform = len(set(q_len)) == 1
    if not uniform:
        kw["q_offsets"] = torch.from_numpy(offsets).cuda()
    out_t = DTYPES[dtype] if out == "same" else torch.float32
    got, lse = attn.awq_kv4_attention(dev(q, dtype), c, p, torch.from_numpy(table).cuda(), torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
                                      causal=causal, window=window, max_kv=max(kv_len) if max_kv is None else max_kv, out_dtype=out_t,
                                      lse=True, **kw)
    scale = d ** -0.5
    want, want_lse = A.attention(q, codes, params, table, kv_len, offsets, scale, causal, window)
    bound = attention_bound(q, codes, params, table, kv_len, offsets, scale, causal, window, want, exact)
    half = U if out == "f32" else half_step(dtype)
    fine = np.isfinite(want)
    within(host(got), want, np.where(fine, bound, 0) + half * np.abs(np.where(fine, want, 0)) + U, "out")
    if check_lse:
        e = 2.0 ** -10 + 2.0 ** -20 * (np.abs(np.where(np.isfinite(want_lse), want_lse, 0)) + 4)
        if not exact:
            e = e + np.max(np.abs(q), -1) * d * scale * 8 * (2.0 ** -11 + d * 2.0 ** -24)  # cached numbers are below 8
        within(host(lse), want_lse, e, "lse")
    return got, lse


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,kv_len,heads,kv,d,page", [
    ([1], [1], 1, 1, 32, 16), ([1], [31], 4, 2, 64, 16), ([1], [2047], 8, 8, 128, 64), ([1], [5000], 16, 2, 128, 32),
    ([1], [777], 3, 1, 96, 16), ([1, 1, 1], [33, 0, 1000], 8, 1, 128, 64), ([1] * 5, [16, 17, 300, 1, 64], 20, 4, 256, 16),
    ([1] * 2, [900, 40], 5, 1, 160, 128), ([1], [1500], 64, 2, 192, 64), ([1, 1], [129, 4100], 16, 1, 224, 1024)])
def test_single_tokens(attn, q_len, kv_len, heads, kv, d, page, dtype):
    rng = np.random.default_rng(sum(kv_len) + heads + d)
    print(f"[gpu attend] q={q_len} kv={kv_len} heads={heads}/{kv} d={d} page={page} {dtype}", flush=True)
    _run(attn, rng, q_len, kv_len, heads, kv, d, page, dtype)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,kv_len,heads,kv,d,page", [
    ([5, 5], [300, 77], 8, 2, 128, 16), ([3, 0, 9, 1], [40, 100, 9, 513], 4, 4, 64, 32), ([17], [17], 2, 1, 32, 16), ([40], [129], 6, 2, 96, 64),
    ([7, 30, 64], [7, 200, 64], 5, 1, 128, 64), ([33, 2], [1000, 65], 2, 2, 256, 16), ([130], [400], 1, 1, 192, 32), ([1, 200], [3, 210], 4, 1, 64, 16)])
def test_several_tokens(attn, q_len, kv_len, heads, kv, d, page, causal):
    rng = np.random.default_rng(sum(kv_len) + heads + d)
    print(f"[gpu attend] q={q_len} kv={kv_len} heads={heads}/{kv} d={d} page={page} causal={causal}", flush=True)
    _run(attn, rng, q_len, kv_len, heads, kv, d, page, "bf16" if d % 64 else "f16", causal, out="f32" if sum(q_len) % 2 else "same", apart=1)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 100, 5000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(attn, window, causal):
    rng = np.random.default_rng(window)
    print(f"[gpu attend] window={window} causal={causal}", flush=True)
    _run(attn, rng, [1, 1], [700, 64], 8, 2, 128, 16, causal=causal, window=window)
    _run(attn, rng, [1, 40, 6], [300, 200, 6], 4, 2, 64, 32, "f16", causal=causal, window=window)


@pytest.mark.parametrize("q_len,kv_len,d", [([1], [3000], 128), ([4, 4], [513, 100], 64), ([50], [200], 256)])
def test_exact_scores(attn, q_len, kv_len, d):
    """Keys, values and scores without rounding: only the softmax's own errors are left."""
    rng = np.random.default_rng(d)
    _run(attn, rng, q_len, kv_len, 8, 2, d, 32, "f16", exact=True, out="f32")
    _run(attn, rng, q_len, kv_len, 8, 2, d, 32, "bf16", exact=True, out="f32")


@pytest.mark.parametrize("max_kv", [1, 64, 4000, 100000])
def test_the_longest_length_changes_no_result(attn, max_kv):
    rng = np.random.default_rng(3)
    _run(attn, rng, [1, 1], [4000, 257], 8, 2, 128, 64, max_kv=max_kv)
    _run(attn, rng, [20, 3], [4000, 257], 2, 1, 64, 64, max_kv=max_kv)


def test_rows_that_see_nothing(attn):
    """Fewer cached tokens than new ones: the first new tokens stand before the cache's beginning."""
    rng = np.random.default_rng(4)
    got, lse = _run(attn, rng, [9, 4, 20], [4, 0, 1], 4, 2, 64, 16)
    assert not bool(got[:5].any()) and bool((lse[:5] == -float("inf")).all()) and bool(got[5:9].any(-1).all())
    got, _ = _run(attn, rng, [1, 1], [0, 0], 4, 2, 128, 16)
    assert not bool(got.any())


@pytest.mark.parametrize("q_len", [4, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_what_a_padding_query_holds_does_not_matter(attn, q_len, dtype):
    """Queries of NaN and infinities: zeros where the row sees nothing (before the cache's beginning, or on pages outside it),
    NaN where it sees a token, and no other row is touched."""
    rng = np.random.default_rng(17)
    codes, params = random_cache(rng, 40, 2, 64, 16)
    c, p = cache_dev(codes, params)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(2, 20)
    table[1] = -1
    kv_len = torch.tensor([q_len - 2, 60], dtype=torch.int32, device="cuda")  # the first sequence's rows 0, 1 see nothing
    q = dev(rng.standard_normal((2 * q_len, 4, 64)), dtype)
    clean, clean_lse = attn.awq_kv4_attention(q, c, p, table, kv_len, lse=True)
    bad = q.clone()
    bad[0, 0, 3], bad[1, 1, 5], bad[1, 2, :] = float("nan"), float("inf"), -float("inf")
    bad[q_len:, :, 7] = float("nan")
    bad[3, 1, 9], bad[3, 2, 8] = float("nan"), float("inf")
    got, lse = attn.awq_kv4_attention(bad, c, p, table, kv_len, lse=True)
    for x, y in ((got, clean), (lse, clean_lse)):
        assert bool(x[3, 1:3].isnan().all())
        x[3, 1:3] = y[3, 1:3]
        assert torch.equal(x, y)
    assert not bool(got[:2].any()) and not bool(got[q_len:].any())
    assert bool((lse[:2] == -float("inf")).all()) and bool((lse[q_len:] == -float("inf")).all())


def test_pages_outside_the_cache_are_not_seen(attn):
    rng = np.random.default_rng(5)

    def edit(table):
        table[0, 1], table[0, 3], table[1, 0], table[2, :] = -1, 1 << 30, -(1 << 31), -7

    _run(attn, rng, [1, 1, 1], [300, 40, 100], 8, 2, 128, 32, table_edit=edit)
    _run(attn, rng, [40, 5, 3], [300, 40, 100], 2, 2, 64, 32, table_edit=edit)


def test_lengths_past_the_table_are_clamped(attn):
    rng = np.random.default_rng(6)
    codes, params = random_cache(rng, 4, 1, 64, 16)
    c, p = cache_dev(codes, params)
    q = dev(rng.standard_normal((3, 2, 64)), "bf16")
    table = torch.tensor([[0, 1], [2, 3], [1, 0]], dtype=torch.int32, device="cuda")
    a = attn.awq_kv4_attention(q, c, p, table, torch.tensor([1 << 30, -5, 32], dtype=torch.int32, device="cuda"))
    b = attn.awq_kv4_attention(q, c, p, table, torch.tensor([32, 0, 32], dtype=torch.int32, device="cuda"))
    assert torch.equal(a, b)


def test_offsets_that_leave_rows_out(attn):
    rng = np.random.default_rng(7)
    codes, params = random_cache(rng, 8, 2, 64, 16)
    c, p = cache_dev(codes, params)
    q = dev(rng.standard_normal((60, 4, 64)), "bf16")
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    kv = torch.tensor([50, 64], dtype=torch.int32, device="cuda")
    out = torch.full((60, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((60, 4), 3.0, device="cuda")
    attn.awq_kv4_attention(q, c, p, table, kv, q_offsets=torch.tensor([20, 21, 47], dtype=torch.int32, device="cuda"), out=out, lse=lse)
    assert bool((out[:20] == 3).all()) and bool((out[47:] == 3).all()) and bool((lse[:20] == 3).all()) and bool((lse[47:] == 3).all())
    alone = attn.awq_kv4_attention(q[20:47].contiguous(), c, p, table, kv, q_offsets=torch.tensor([0, 1, 27], dtype=torch.int32, device="cuda"))
    assert torch.equal(out[20:47], alone)
    # offsets outside the rows, and ones that do not ascend, are clamped
    for bad in ([-5, 200, 300], [50, 10, 20], [1 << 30, -(1 << 30), 1 << 30]):
        got = attn.awq_kv4_attention(q, c, p, table, kv, q_offsets=torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert got.shape == q.shape and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("d", [64, 256])
def test_nan_only_where_it_is_seen(attn, d):
    """Keys or values of NaN, or of infinite parameters, behind a row's place, in the pages' unwritten rest and on pages that
    nobody names leave the row alone; seen values of NaN reach the channels of their group."""
    rng = np.random.default_rng(8)
    for at, which, group in ((150, 0, 0), (150, 1, 0), (20, 1, (d - 1) // 128), (0, 1, 0), (199, 0, 0), (198, 1, 0)):
        tables = []

        def cache(pages):
            codes, params = random_cache(rng, pages, 2, d, 16)
            table = tables[0]
            used = set(table[0].tolist()) - {-1}
            for i in range(pages):
                if i not in used:
                    params[i] = np.nan
            params[table[0, 12], :, :, :, 8:] = np.inf  # 200 of 208 tokens are cached
            params[table[0, at // 16], which, 1, group, at % 16, at % 2] = np.nan if at % 3 else -np.inf
            return codes, params

        print(f"[gpu attend] nan at {at} of {'kv'[which]} d={d}", flush=True)
        _run(attn, rng, [60], [200], 4, 2, d, 16, cache=cache, table_edit=tables.append)
        _run(attn, rng, [3], [200], 4, 2, d, 16, cache=cache, table_edit=lambda t: tables.__setitem__(0, t))


def test_queries_of_every_size(attn):
    """bfloat16 queries past float16's range and below it, NaN and infinity in single rows."""
    rng = np.random.default_rng(9)
    codes, params = random_cache(rng, 4, 2, 64, 16)
    params[:, 0] *= np.float16(2.0 ** -10)
    c, p = cache_dev(codes, params)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    kv = torch.tensor([64], dtype=torch.int32, device="cuda")
    base = dev(rng.standard_normal((8, 4, 64)), "bf16")
    want = attn.awq_kv4_attention(base, c, p, table, kv, scale=2.0 ** 7, lse=True)
    for e in (100, 20, -20, -100):  # the same scores by way of the scale
        got = attn.awq_kv4_attention(base * 2.0 ** e, c, p, table, kv, scale=2.0 ** (7 - e), lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), e
    odd = base.clone()
    odd[2, 1, 5], odd[4, 3, 0] = float("nan"), float("inf")
    got = attn.awq_kv4_attention(odd, c, p, table, kv, scale=2.0 ** 7)
    bad = torch.zeros((8, 4), dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[4, 3] = True
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[0][~bad])


def test_a_long_tail_of_small_weights_counts(attn):
    """One token 17 powers of two above 8000 others that together weigh as much as a sixteenth of it: weights below float16's
    normal numbers relative to the largest."""
    d, n = 64, 8192
    codes, params = np.zeros((n // 64, 2, 1, 64, d // 2), np.uint8), np.zeros((n // 64, 2, 1, 1, 64, 2), np.float16)
    params[:, 1, 0, 0, :, 1] = 1.0  # every value is one ...
    params[0, 1, 0, 0, 0, 1] = 0.0  # ... but the first token's
    params[0, 0, 0, 0, 0, 1] = 17.0 / d * np.log(2.0)  # its score: 17 log 2
    c, p = cache_dev(codes, params)
    table = torch.arange(n // 64, dtype=torch.int32, device="cuda").view(1, -1)
    for m in (n, 3000, 40):
        q = torch.ones((1, 1, d), dtype=torch.float16, device="cuda")
        got = attn.awq_kv4_attention(q, c, p, table, torch.tensor([m], dtype=torch.int32, device="cuda"), scale=1.0, out_dtype=torch.float32)
        top = float(np.float16(17.0 / d * np.log(2.0))) * d
        want = (m - 1) / (m - 1 + np.exp(top))
        assert abs(float(got[0, 0, 0]) / want - 1) < 2.0 ** -9 + m * 2.0 ** -24, m


def test_layouts_and_in_place(attn):
    rng = np.random.default_rng(10)
    codes, params = random_cache(rng, 20, 2, 96, 16)
    c, p = cache_dev(codes, params, 3)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    kv = torch.tensor([150, 77], dtype=torch.int32, device="cuda")
    for n in (2, 60):
        q = dev(rng.standard_normal((n, 6, 96)), "bf16")
        want, want_lse = attn.awq_kv4_attention(q, c, p, table, kv, lse=True)
        wide = torch.zeros((n, 10, 96), dtype=torch.bfloat16, device="cuda")
        wide[:, 2:8] = q
        odd = torch.zeros((n * 6 * 101 + 1,), dtype=torch.bfloat16, device="cuda")[1:].view(n, 6, 101)[..., :96]
        odd.copy_(q)
        for view in (wide[:, 2:8], odd, q.transpose(0, 1).contiguous().transpose(0, 1)):
            lse = torch.empty((n, 6), device="cuda")
            table_wide = torch.full((2, 13), -1, dtype=torch.int32, device="cuda")
            table_wide[:, :10] = table
            assert torch.equal(attn.awq_kv4_attention(view, c, p, table_wide[:, :10], kv, lse=lse, out=torch.zeros_like(odd))[0], want)
            assert torch.equal(lse, want_lse)
            assert attn.awq_kv4_attention(view, c, p, table, kv, out=view) is view and torch.equal(view, want)


def test_given_workspace_and_repeated_calls(attn):
    rng = np.random.default_rng(11)
    codes, params = random_cache(rng, 260, 2, 128, 64)
    c, p = cache_dev(codes, params)
    table = torch.from_numpy(rng.permutation(260).astype(np.int32)).cuda().view(2, 130)
    kv = torch.tensor([8300, 5000], dtype=torch.int32, device="cuda")
    q = dev(rng.standard_normal((2, 16, 128)), "bf16")
    nb = attn.awq_kv4_attention_workspace_bytes(2, 2, False, 16, 2, 128, True, 0, 8300)
    assert nb > 0
    ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")
    want = attn.awq_kv4_attention(q, c, p, table, kv, max_kv=8300)
    for _ in range(3):
        assert torch.equal(attn.awq_kv4_attention(q, c, p, table, kv, max_kv=8300, workspace=ws), want)
    with pytest.raises(ValueError):
        attn.awq_kv4_attention(q, c, p, table, kv, max_kv=8300, workspace=ws[:-1])
