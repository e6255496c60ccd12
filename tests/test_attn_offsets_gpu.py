"""awq_kv4_attention with offsets outside the rows: they are taken as the nearest row, and every row that belongs to a sequence then is
written."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import attention_bound, cache_dev, random_cache  # noqa: E402
from moe_cases import dev, half_step, host, within  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


@pytest.mark.parametrize("n,heads,page", [(6, 4, 16), (60, 4, 16), (60, 64, 16), (600, 4, 256)])
@pytest.mark.parametrize("offsets", [(-5, 0.3, 2.0), (0.5, 0.6, 1e9), (-(2.0 ** 31), 0.9, 1.0), (-40, -3, 0.4), (1.5, 2.0, 3.0), (0.2, 1.1, 1e8)])
def test_offsets_outside_the_rows(attn, n, heads, page, offsets):
    rng = np.random.default_rng(n + heads)
    d, kv, kv_len = 64, 2, [4 * page - 3, 3 * page]
    # fractions are of n, whole negative numbers as they are
    offsets = np.array([int(x) if x < 0 else min(int(x * n), 2 ** 31 - 1) for x in offsets], np.int64).astype(np.int32)
    print(f"[gpu attend] n={n} heads={heads} offsets={offsets.tolist()}", flush=True)
    codes, params = random_cache(rng, 8, kv, d, page)
    table = rng.permutation(8).astype(np.int32).reshape(2, 4)
    q = host(dev(rng.standard_normal((n, heads, d)), "bf16"))
    out, lse = torch.full((n, heads, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((n, heads), 3.0, device="cuda")
    attn.awq_kv4_attention(dev(q, "bf16"), *cache_dev(codes, params), torch.from_numpy(table).cuda(), torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
                           q_offsets=torch.from_numpy(offsets).cuda(), out=out, lse=lse)
    inside = offsets.clip(0, n)
    start, start_lse = np.full((n, heads, d), 3.0), np.full((n, heads), 3.0)
    want, want_lse = A.attention(q, codes, params, table, kv_len, inside, d ** -0.5, True, 0, start, start_lse)
    mine = np.zeros(n, bool)
    mine[inside[0]:inside[-1]] = True
    bound = attention_bound(q, codes, params, table, kv_len, inside, d ** -0.5, True, 0, want)
    within(host(out), want, bound + half_step("bf16") * np.abs(want) * mine[:, None, None], "out")
    got = host(lse)
    assert np.array_equal(got[~mine], want_lse[~mine]) and np.array_equal(np.isfinite(got), np.isfinite(want_lse))
    assert np.abs(got - want_lse)[np.isfinite(want_lse)].max(initial=0) < 0.25  # (a row that is not written has 3)
