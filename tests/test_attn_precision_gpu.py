"""awq_kv4_attention's precision, as tight as its roundings are, so that a token left out or counted twice, or a rounding more, shows.

Three kinds of tests. Outputs are float32, without a rounding that matters.
* Queries of zero: every weight is the same power of two, values are small whole numbers, every sum is exact. Left: one division, 2^-21.
* A few tokens, exact scores: float16 rows of few carry their numerators as two float16 numbers (2^-22 and less), the others as one.
* Any caches, at the sizes of real use: roundings are independent, so the error's variance is the sum of theirs. A float16 number of
  step u is off by u / sqrt(12) (root mean square); a numerator's step is 2^-10 of the power of two below it, over all places
  between two powers 0.2123 2^-10 of it. A weight's error e moves an output by w e (v - out). The squares' mean over the outputs
  has to be within 1.5 of the one expected, and no output further off than 8 of its own.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import cache_dev, paged, random_cache  # noqa: E402
from moe_cases import DTYPES, dev, host, within  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,kv_len,heads,kv,d,page", [
    ([1], [1], 1, 1, 32, 16), ([1], [2047], 32, 32, 128, 64), ([1] * 7, [300, 8191, 0, 31, 33, 5000, 129], 64, 8, 128, 64), ([1], [131071], 64, 8, 128, 64),
    ([1, 1], [4097, 6000], 16, 8, 256, 64), ([1] * 3, [8000, 77, 4001], 32, 8, 64, 16), ([5] * 4, [2001, 5, 700, 3333], 16, 8, 256, 32),
    ([4] * 3, [6000, 200, 33], 64, 8, 128, 64), ([7, 1, 0, 8], [4000, 1, 9, 500], 4, 1, 96, 16), ([100], [100], 4, 4, 128, 64),
    ([500, 31, 260], [500, 1000, 777], 8, 2, 64, 64), ([300], [1300], 4, 1, 128, 128), ([150], [801], 2, 1, 256, 16)])
def test_equal_weights(attn, q_len, kv_len, heads, kv, d, page, dtype):
    """Every seen token counts once: the mean of the values, and log n."""
    rng = np.random.default_rng(sum(kv_len) + d)
    table, pages = paged(rng, kv_len, page)
    codes, params = random_cache(rng, pages, kv, d, page)
    params[:, 1] = 1.0, -8.0  # values -8 .. 7; sums below 2^24 / 2^7
    if max(kv_len) > 16000:
        codes[:, 1] &= 0x11
        params[:, 1] = 1.0, 0.0
    offsets = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    n = int(offsets[-1])
    for causal, window in ((True, 0), (False, 0), (True, 129)):
        print(f"[gpu precision] equal q={q_len} kv={kv_len} d={d} {dtype} causal={causal} window={window}", flush=True)
        got, lse = attn.awq_kv4_attention(torch.zeros((n, heads, d), dtype=DTYPES[dtype], device="cuda"), *cache_dev(codes, params),
                                          torch.from_numpy(table).cuda(), torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
                                          q_offsets=torch.from_numpy(offsets).cuda(), causal=causal, window=window, max_kv=max(kv_len),
                                          out_dtype=torch.float32, lse=True)
        want, want_lse = np.zeros((n, heads, d)), np.full((n, heads), -np.inf)
        for s, m in enumerate(kv_len):
            place = np.arange(m)
            v = codes[table[s][place // page], 1, :, place % page]
            v = np.stack([v & 15, v >> 4], -1).reshape(m, kv, d) * 1.0 + float(params[0, 1, 0, 0, 0, 1])
            total = np.concatenate([np.zeros((1, kv, d)), np.cumsum(v, 0)])
            for i in range(q_len[s]):
                p = m - q_len[s] + i
                hi, lo = (min(m, p + 1) if causal else m), (max(0, p - window + 1) if window else 0)
                if hi > lo:
                    want[offsets[s] + i] = np.repeat((total[hi] - total[lo]) / (hi - lo), heads // kv, 0)
                    want_lse[offsets[s] + i] = np.log(hi - lo)
        within(host(got), want, np.abs(want) * 2.0 ** -21, "out")
        within(host(lse), want_lse, 2.0 ** -20 * (1 + np.abs(np.where(np.isfinite(want_lse), want_lse, 0))), "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len,kv_len,heads", [(1, 3, 4), (1, 12, 8), (2, 40, 8), (8, 30, 4), (40, 47, 4)])
def test_numerators(attn, q_len, kv_len, heads, d, dtype):
    """Exact scores that lie within 12 powers of two, of a few tokens. Exponents: three roundings of numbers below 2^4, 2^-19 of a weight.
    Numerators: 2^-21 as two float16 numbers, 2^-11 and as much in the sum as one."""
    rng = np.random.default_rng(q_len + kv_len + d)
    codes, params = random_cache(rng, 4, 1, d, 16, exact=True)
    q = rng.integers(-4, 5, (q_len, heads, d)) / 4.0
    k, v = _numbers(torch.from_numpy(codes), torch.from_numpy(params), torch.arange(4), kv_len, 16)
    x = k[:, 0].numpy() @ q.reshape(-1, d).T
    scale = float(np.float32(12 / (x.max(0) - x.min(0)).max() * np.log(2)))
    got, lse = attn.awq_kv4_attention(dev(q, dtype), *cache_dev(codes, params), torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4),
                                      torch.tensor([kv_len], dtype=torch.int32, device="cuda"), scale=scale, out_dtype=torch.float32, lse=True)
    few = q_len * heads <= 64
    numerator = 2.0 ** -21 if few and dtype == "f16" else 2.0 ** -10
    x, v = x.reshape(kv_len, q_len, heads) * scale, v[:, 0].numpy()
    want, tol, want_lse = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:2])
    for i in range(q_len):
        n = kv_len - q_len + i + 1
        w = np.exp(x[:n, i] - x[:n, i].max(0))
        want_lse[i] = x[:n, i].max(0) + np.log(w.sum(0))
        w /= w.sum(0)
        want[i] = w.T @ v[:n]
        tol[i] = (w.T @ np.abs(v[:n])) * (numerator + 2.0 ** -18 + n * 2.0 ** -23)
    within(host(got), want, tol, "out")
    within(host(lse), want_lse, numerator + 2.0 ** -18 + np.abs(want_lse) * 2.0 ** -21, "lse")


def _numbers(codes, params, pages, n, page):
    """Keys and values [n, kv, d] in float64 of the first n tokens in `pages`."""
    out = []
    for which in (0, 1):
        c = codes[pages, which].transpose(1, 2).flatten(0, 1)[:n]
        p = params[pages, which].permute(0, 3, 1, 2, 4).flatten(0, 1)[:n].double()
        c = torch.stack([c & 15, c >> 4], -1).flatten(-2)
        d = c.shape[-1]
        step, offset = (p[..., i].repeat_interleave(128, -1)[..., :d] for i in (0, 1))
        out.append(c * step + offset)
    return out


def _step_of(x):
    """float16's step at x (normal numbers)."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -14))) - 10)


def _expected(q, k, v, scale, few, pair):
    """(out, variance of its error) of rows q [rows, d] over tokens k, v [n, d], all float64."""
    x = (q @ k.T) * scale
    w = torch.softmax(x, -1)
    out = w @ v
    # scores: keys as float16 numbers (prompts), or sums of d products with codes + 1024, whose sums over queries of either sign
    # stay within 2 * 1264 times the queries' norm, in units of the keys' steps (0.45 at most)
    if few:
        e = (2.0 ** -24 * 0.29 * k.shape[1] ** 0.5 * 2 * 1264 * q.norm(dim=-1, keepdim=True) * 0.45 * scale) ** 2
    else:
        e = (q ** 2) @ (_step_of(k) ** 2 / 12).T * scale ** 2
    e = e + (2.0 ** -23 * (x.abs() + x.abs().max(-1, keepdim=True).values)) ** 2  # exponents
    if not pair:
        e = e + (0.2123 * 2.0 ** -10) ** 2
    w2 = w ** 2
    # sum of w^2 e (v - out)^2, and the values' own rounding
    a, b, c = (w2 * e) @ (v ** 2), (w2 * e) @ v, (w2 * e).sum(-1, keepdim=True)
    var = (a - 2 * out * b + out ** 2 * c).clamp_min(0) + w2 @ (_step_of(v) ** 2 / 12)
    return out, var + (2.0 ** -22 * (w @ v.abs())) ** 2


SIZES = [([1] * 12, [8192, 5000, 31, 777, 8000, 64, 4096, 1, 2500, 6001, 129, 3333], 64, 8, 128, 64), ([1], [131071], 64, 8, 128, 64),
         ([1] * 6, [8000, 7777, 100, 4096, 2049, 6000], 32, 8, 64, 64), ([1] * 4, [3000, 6000, 517, 99], 16, 8, 256, 64),
         ([4] * 5, [6000, 5000, 300, 4097, 128], 64, 8, 128, 64), ([5] * 6, [2001] * 6, 16, 8, 256, 64), ([1] * 8, [1024] * 8, 32, 32, 96, 16),
         ([300, 200], [1300, 200], 8, 2, 64, 64), ([512], [2560], 16, 2, 128, 64), ([140, 260], [700, 1025], 4, 2, 256, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("q_len,kv_len,heads,kv,d,page", SIZES)
def test_errors_are_those_of_the_roundings(attn, q_len, kv_len, heads, kv, d, page, dtype):
    rng = np.random.default_rng(sum(kv_len) + d)
    print(f"[gpu precision] q={q_len} kv={kv_len} heads={heads}/{kv} d={d} {dtype}", flush=True)
    table, pages = paged(rng, kv_len, page)
    codes, params = (t.cuda() for t in map(torch.from_numpy, random_cache(rng, pages, kv, d, page)))
    n, scale, group = sum(q_len), d ** -0.5, heads // kv
    q = torch.from_numpy(1.5 * rng.standard_normal((n, heads, d))).cuda().to(DTYPES[dtype])
    offsets = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
    got = attn.awq_kv4_attention(q, codes, params, torch.from_numpy(table).cuda(), torch.tensor(kv_len, dtype=torch.int32, device="cuda"),
                                 q_offsets=torch.from_numpy(offsets).cuda(), max_kv=max(kv_len), out_dtype=torch.float32).double()
    few = -(-n // len(q_len)) * group <= 64
    square, expected = 0.0, 0.0
    for s, m in enumerate(kv_len):
        k, v = _numbers(codes, params, torch.from_numpy(table[s][:-(-m // page)].astype(np.int64)).cuda(), m, page)
        for i in range(q_len[s]):
            seen = m - q_len[s] + i + 1
            row = offsets[s] + i
            for h in range(kv):
                mine = slice(h * group, (h + 1) * group)
                want, var = _expected(q[row, mine].double(), k[:seen, h], v[:seen, h], scale, few, few and dtype == "f16")
                off = (got[row, mine] - want) ** 2
                assert bool((off <= 64 * var).all()), f"row {row}, head {h}: {(off / var).max().item() ** 0.5:.1f} of its own"
                square += off.sum().item()
                expected += var.sum().item()
    print(f"[gpu precision] {(square / expected) ** 0.5:.3f} of the error expected", flush=True)
    assert square <= 1.5 ** 2 * expected
