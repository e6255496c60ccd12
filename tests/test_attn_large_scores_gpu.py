"""awq_kv4_attention where scores are far larger than their differences. Queries and keys are chosen so that every score, and every
partial sum of one, is a float32 without rounding; values are small whole numbers. What is left of the errors:

* weights: a score's distance to the largest times scale * log2(e), rounded three times (2^-22 of the exponent, which matters up to 40);
* numerators, rounded to float16 by half a step of 2^-11, in the sum as well: 2^-10;
* numerators below 2^-31 of the largest are lost; float32 sums of n of them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import dev, host, within  # noqa: E402

PAGE = 64


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _cache(rng, kv_len, d, k_codes, step, offset):
    """One sequence, one key head: keys of k_codes [kv_len, d] with one step and offset, values of -8 .. 7. (cache on the device, table, v)."""
    groups, pages = (d + 127) // 128, (kv_len + PAGE - 1) // PAGE
    full = np.zeros((2, pages * PAGE, d), np.uint8)
    full[0, :kv_len] = k_codes
    full[1] = rng.integers(0, 16, full[1].shape)
    packed = (full[..., 0::2] | full[..., 1::2] << 4).reshape(2, pages, 1, PAGE, d // 2).transpose(1, 0, 2, 3, 4)
    params = np.zeros((pages, 2, 1, groups, PAGE, 2), np.float16)
    params[:, 0] = step, offset
    params[:, 1] = 1.0, -8.0
    order = rng.permutation(pages)
    codes, placed = np.empty(packed.shape, np.uint8), np.empty(params.shape, np.float16)
    codes[order], placed[order] = packed, params
    table = torch.from_numpy(order.astype(np.int32)).cuda().view(1, pages)
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(placed).cuda()), table, full[1, :kv_len] - 8.0


def _check(attn, q, k, v, cache, table, scale, dtype):
    """q [q_len, heads, d], k [kv_len, d] and v as float64; causal."""
    q_len, heads, _ = q.shape
    kv_len = len(k)
    scale = float(np.float32(scale))
    lens = torch.tensor([kv_len], dtype=torch.int32, device="cuda")
    qt = dev(q, dtype)
    assert np.array_equal(host(qt), q)
    got, lse = attn.awq_kv4_attention(qt, *cache, table, lens, scale=scale, max_kv=kv_len, out_dtype=torch.float32, lse=True)
    want, tol, want_lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for i in range(q_len):
        n = kv_len - q_len + i + 1
        x = k[:n] @ q[i].T  # exact: [n, heads]
        w = np.exp((x - x.max(0)) * scale)
        want_lse[i] = x.max(0) * scale + np.log(w.sum(0))
        w /= w.sum(0)
        want[i] = w.T @ v[:n]
        tol[i] = (w.T @ np.abs(v[:n])) * (2.0 ** -10 + 2.0 ** -16 + n * 2.0 ** -24) + n * 2.0 ** -31 * 8
    within(host(got), want, tol, "out")
    within(host(lse), want_lse, np.abs(want_lse) * 2.0 ** -21 + 2.0 ** -9, "lse")


SHAPES = [(1, 200), (1, 3000), (5, 700), (30, 1500), (100, 100), (100, 1100)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv_len", SHAPES)
def test_scores_far_larger_than_their_differences(attn, q_len, kv_len, d, dtype):
    """Scores d 2^15 +- a few, times a power of two: base-2 exponents of +-2^20 to +-2^43 whose differences are from 1/8 up, with many
    ties."""
    rng = np.random.default_rng(q_len + kv_len + d)
    heads = 2
    codes = np.zeros((kv_len, d), np.uint8)
    codes[:, 5] = rng.integers(0, 16, kv_len)
    cache, table, v = _cache(rng, kv_len, d, codes, 32.0, 32768.0)
    k = 32768.0 + 32.0 * codes
    print(f"[gpu large scores] q={q_len} kv={kv_len} d={d} {dtype}", flush=True)
    for sign in (1.0, -1.0):
        q = np.full((q_len, heads, d), sign)
        q[..., 5] *= d * 2.0 ** -13  # the differences: code * d / 256
        q[:, 1] /= 2.0
        for e in (-1, 0, 3, 7, 9, 13, 20):
            _check(attn, q, k, v, cache, table, np.log(2.0) * 2.0 ** e * 64 / d, dtype)
        _check(attn, -q, k, v, cache, table, -np.log(2.0) * 2.0 ** 5, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,kv_len", SHAPES)
def test_scores_of_every_size_in_one_row(attn, q_len, kv_len, dtype):
    """The largest score so far grows from far below to far above, or falls, or neither; a few of 40 queries have all of them small."""
    rng = np.random.default_rng(q_len + kv_len)
    d, heads = 64, 4
    q = rng.choice([-1.0, 1.0], (q_len, heads, d)) * 2.0 ** -rng.integers(0, 9, (q_len, heads, d))
    q[:, 1] *= 2.0 ** -rng.integers(0, 7, (q_len, 1))
    codes = rng.integers(0, 16, (kv_len, d)).astype(np.uint8)
    order = np.argsort(codes @ q[0, 0])
    print(f"[gpu large scores] mixed q={q_len} kv={kv_len} {dtype}", flush=True)
    for turn in (order, order[::-1], np.arange(kv_len)):
        cache, table, v = _cache(rng, kv_len, d, codes[turn], 1.0, 0.0)
        for e in (4, 10, 13, 14, 20, 40):
            _check(attn, q, codes[turn].astype(np.float64), v, cache, table, np.log(2.0) * 2.0 ** e, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,kv_len", SHAPES)
def test_scores_far_below_zero_are_seen(attn, q_len, kv_len, dtype):
    """Scores from -2^30 down to below float32's range, by the queries' size and by the scale's: the largest of them has the weight. A
    logarithm past float32 is -infinity, and the row has its weights all the same."""
    rng = np.random.default_rng(q_len * kv_len)
    d, heads = 64, 2
    codes = np.zeros((kv_len, d), np.uint8)
    codes[:, 5] = rng.integers(0, 16, kv_len)
    cache, table, v = _cache(rng, kv_len, d, codes, 32.0, 32768.0)
    k = 32768.0 + 32.0 * codes
    lens = torch.tensor([kv_len], dtype=torch.int32, device="cuda")
    print(f"[gpu large scores] below q={q_len} kv={kv_len} {dtype}", flush=True)
    sizes = [(0, e) for e in (10, 70, 90, 100, 105, 120, 127)]
    if dtype == "bf16":
        sizes += [(e, 0) for e in (70, 90, 105, 120)] + [(100, 40), (126, 127), (-120, 127)]
    for of_query, of_scale in sizes:
        for sign in (-1.0, 1.0):
            q = np.full((q_len, heads, d), sign * 2.0 ** of_query)
            q[..., 5] *= 2.0 ** -7
            got, lse = attn.awq_kv4_attention(dev(q, dtype), *cache, table, lens, scale=2.0 ** of_scale, max_kv=kv_len,
                                              out_dtype=torch.float32, lse=True)
            x = k @ (q[0, 0] / 2.0 ** of_query)  # exact, the same for every row
            for i in range(q_len):
                n = kv_len - q_len + i + 1
                e = np.longdouble(2.0) ** (of_query + of_scale)
                w = np.exp(np.maximum((x[:n] - x[:n].max()) * e, -11000)).astype(np.float64)
                want = w @ v[:n] / w.sum()
                # longdouble holds what float64 does not; float32's range ends at 2^128
                log = float(x[:n].max() * e + np.log(np.longdouble(w.sum())))
                tol = (w @ np.abs(v[:n]) / w.sum()) * (2.0 ** -10 + 2.0 ** -16 + n * 2.0 ** -24) + n * 2.0 ** -31 * 8
                within(host(got[i]), np.broadcast_to(want, (heads, d)), np.broadcast_to(tol, (heads, d)), f"out {of_query} {of_scale} {sign}")
                if abs(log) < 2.0 ** 127 * 1.99:
                    within(host(lse[i]), np.full(heads, log), np.full(heads, abs(log) * 2.0 ** -21 + 2.0 ** -9), "lse")
                elif abs(log) > 2.0 ** 128:
                    assert bool((lse[i] == (float("inf") if log > 0 else -float("inf"))).all()), (of_query, of_scale, sign)
