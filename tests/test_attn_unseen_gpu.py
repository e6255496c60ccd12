"""awq_kv4_attention beside memory that was never written: finite steps and offsets whose numbers pass float16's largest, in places
that a row does not see, leave it alone; where they are seen they count as +-65504 (include/awq_attn.h)."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import attention_bound, cache_dev, random_cache  # noqa: E402
from moe_cases import dev, half_step, host, within  # noqa: E402

F16_MAX = 65504.0


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _cache(rng, kv_len, n_kv, d, page):
    """Sequences in pages 2 .., the first of them behind a page that no table names; page 0, page 1 and what lies behind a sequence's
    last token hold zeros. Returns (codes, params, table, mask of unwritten places [pages, page])."""
    used = [(m + page - 1) // page for m in kv_len]
    codes, params = random_cache(rng, 2 + sum(used), n_kv, d, page)
    table = np.full((len(kv_len), max(used)), -1, np.int32)
    unwritten = np.ones((2 + sum(used), page), bool)
    at = 2
    for s, m in enumerate(kv_len):
        table[s, :used[s]] = np.arange(at, at + used[s])
        unwritten[at:at + used[s]] = (np.arange(used[s] * page) >= m).reshape(-1, page)
        at += used[s]
    params.transpose(0, 4, 1, 2, 3, 5)[unwritten] = 0
    return codes, params, table, unwritten


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [32, 96, 128, 256])
@pytest.mark.parametrize("q_len,kv_len,heads,kv", [([1, 1, 1], [77, 1, 300], 8, 2), ([1], [4001], 16, 2), ([4, 4], [513, 100], 8, 2), ([200], [211], 2, 1),
                                                   ([90, 90], [90, 1001], 4, 2)])
def test_unwritten_places_do_not_matter(attn, q_len, kv_len, heads, kv, d, dtype):
    rng = np.random.default_rng(sum(kv_len) + d)
    page = 64
    print(f"[gpu unseen] q={q_len} kv={kv_len} d={d} {dtype}", flush=True)
    codes, params, table, unwritten = _cache(rng, kv_len, kv, d, page)
    codes.transpose(0, 3, 1, 2, 4)[unwritten] = 0xF2  # codes 2 and 15
    q = dev(rng.standard_normal((sum(q_len), heads, d)), dtype)
    tables = torch.from_numpy(table).cuda()
    # a hole: the second page of the first sequence is on no page where it is long enough
    if kv_len[0] > 2 * page:
        tables[0, 1] = -1
    lens = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    want = attn.awq_kv4_attention(q, *cache_dev(codes, params), tables, lens, lse=True)
    assert bool(torch.isfinite(want[0]).all())
    for step, offset in ((40000.0, 0.0), (40000.0, 60000.0), (-40000.0, -60000.0), (5000.0, 65504.0)):
        params.transpose(0, 4, 1, 2, 3, 5)[unwritten] = step, offset
        got = attn.awq_kv4_attention(q, *cache_dev(codes, params), tables, lens, lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (step, offset)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,heads,d", [(5, 4, 64), (5, 4, 256), (20, 2, 128), (70, 4, 64), (70, 4, 128), (70, 4, 256)])
def test_rows_before_a_large_value_do_not_see_it(attn, q_len, heads, d, dtype):
    """A value past float16's largest in the middle of the new tokens: rows before it as if it were not there, rows from it on have
    65504 in its place."""
    rng = np.random.default_rng(q_len + d)
    page, m = 16, 300
    print(f"[gpu unseen] q={q_len} d={d} {dtype}", flush=True)
    codes, params, table, _ = _cache(rng, [m], 1, d, page)
    place = m - q_len // 2 - 1  # the token of new token q_len - q_len // 2 - 1
    at = table[0, place // page], place % page
    codes[at[0], 1, :, at[1]] = rng.integers(0, 3, codes.shape[4]) * 16 + rng.integers(0, 3, codes.shape[4])
    q = host(dev(rng.standard_normal((q_len, heads, d)) / 2, dtype))
    lens, tables = torch.tensor([m], dtype=torch.int32, device="cuda"), torch.from_numpy(table).cuda()
    out = {}
    for sign in (1, -1):
        params[at[0], 1, :, :, at[1]] = 0.0
        clean = attn.awq_kv4_attention(dev(q, dtype), *cache_dev(codes, params), tables, lens, lse=True)
        params[at[0], 1, :, :, at[1], 0] = sign * 40000.0
        got = attn.awq_kv4_attention(dev(q, dtype), *cache_dev(codes, params), tables, lens, lse=True)
        first = q_len - q_len // 2 - 1
        assert torch.equal(got[0][:first], clean[0][:first]) and torch.equal(got[1], clean[1])
        # from there on: the definition with numbers of 80000 as 65504
        page_of, in_page = table[0][np.arange(m) // page], np.arange(m) % page
        k, v = (x[:, 0] for x in A.cached(codes, params, page_of, in_page))
        v = v.clip(-F16_MAX, F16_MAX)
        want = np.zeros((q_len, heads, d))
        for i in range(q_len):
            for h in range(heads):
                x = k[:m - q_len + i + 1] @ q[i, h] * d ** -0.5
                w = np.exp(x - x.max())
                want[i, h] = w @ v[:len(x)] / w.sum()
        offsets = np.array([0, q_len], np.int32)
        bound = attention_bound(q, codes, params, table, [m], offsets, d ** -0.5, True, 0, want)
        within(host(got[0]), want, bound + half_step(dtype) * np.abs(want), f"sign {sign}")
        out[sign] = got[0]
    assert not torch.equal(out[1], out[-1])
