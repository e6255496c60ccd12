"""awq_kv4_write and awq_kv4_read on the GPU against oracle/awq_attn.py. Codes, steps and offsets are equal. A number read back
is one fused float32 operation (U = 2^-24 of it) and one rounding; U absolute covers float16's subnormal step."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import cache_dev, random_cache  # noqa: E402
from moe_cases import DTYPES, U, dev, half_step, host, within  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _written(codes, params, slots, k, v):
    """What the cache holds after the tokens are written."""
    codes, params = codes.copy(), params.copy()
    size = codes.shape[3]
    for which, x in ((0, k), (1, v)):
        q, step, offset = A.quantize(x)
        packed = A.pack(q)
        for i, s in enumerate(slots):
            if 0 <= s < codes.shape[0] * size:
                codes[s // size, which, :, s % size] = packed[i]
                params[s // size, which, :, :, s % size] = np.stack([step[i], offset[i]], -1)
    return codes, params


def _check(attn, codes, params, slots, k, v, dtype, apart=0, kt=None, vt=None, slot_type=torch.int64):
    c, p = cache_dev(codes, params, apart)
    st = torch.from_numpy(np.asarray(slots)).to(slot_type).cuda()
    kt, vt = dev(k, dtype) if kt is None else kt, dev(v, dtype) if vt is None else vt
    attn.awq_kv4_write(kt, vt, c, p, st)
    want_c, want_p = _written(codes, params, slots, host(kt), host(vt))
    assert np.array_equal(c.cpu().numpy(), want_c), "codes"
    assert np.array_equal(p.cpu().numpy().view(np.uint16) & 0x7FFF, want_p.view(np.uint16) & 0x7FFF), "params"
    assert np.array_equal(p.cpu().numpy(), want_p, equal_nan=True), "signs of params"
    return c, p, want_c, want_p, st


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,kv,d,page", [(1, 1, 32, 16), (1, 8, 128, 64), (3, 2, 64, 16), (17, 1, 96, 32), (100, 3, 256, 64), (65, 2, 160, 16),
                                         (33, 5, 224, 128), (300, 8, 128, 1024), (2100, 2, 128, 64), (70000, 1, 64, 64)])
def test_write_and_read(attn, n, kv, d, page, dtype):
    rng = np.random.default_rng(n + kv + d)
    print(f"[gpu kv4] n={n} kv={kv} d={d} page={page} {dtype}", flush=True)
    pages = (n + page - 1) // page + 2
    codes, params = random_cache(rng, pages, kv, d, page)
    slots = rng.permutation(pages * page)[:n] if n < 2000 else np.arange(n) + 5
    slots = np.where(rng.random(n) < 0.1, rng.choice([-1, pages * page, 1 << 40, -(1 << 40)]) if n > 1 else slots, slots)
    k = rng.standard_normal((n, kv, d)) * np.exp(rng.standard_normal((n, kv, 1)))
    v = rng.standard_normal((n, kv, d)) + 3 * rng.standard_normal((n, kv, 1))
    c, p, wc, wp, st = _check(attn, codes, params, slots, k, v, dtype, apart=n % 3)
    for out_t in ("bf16", "f16", "f32"):
        out = tuple(torch.full((n, kv, d), 5.0, dtype=DTYPES[out_t], device="cuda") for _ in range(2))
        assert attn.awq_kv4_read(c, p, st, out=out) is not None
        there = (slots >= 0) & (slots < pages * page)
        s = np.where(there, slots, 0)
        for got, want in zip(out, A.cached(wc, wp, s // page, s % page)):
            want = np.where(there[:, None, None], want, 5.0)
            within(host(got), want, np.abs(want) * (half_step(out_t) + U) + U, f"read {out_t}")


def test_write_takes_any_layout_and_reads_one_side(attn):
    rng = np.random.default_rng(4)
    n, kv, d, page = 50, 4, 96, 16
    codes, params = random_cache(rng, 6, kv, d, page)
    slots = rng.permutation(96)[:n]
    rows = torch.full((n, 3 * kv, d), 7.0, dtype=torch.bfloat16, device="cuda")  # a fused row: query, key and value heads
    rows.copy_(torch.randn(rows.shape, device="cuda"))
    _check(attn, codes, params, slots, None, None, "bf16", kt=rows[:, kv:2 * kv], vt=rows[:, 2 * kv:], slot_type=torch.int32)
    odd = torch.randn((n * kv * 101 + 1,), device="cuda").bfloat16()[1:].view(n, kv, 101)[..., :d]
    heads_first = torch.randn((kv, n, d), device="cuda").bfloat16().transpose(0, 1)
    c, p, wc, wp, st = _check(attn, codes, params, slots, None, None, "bf16", kt=odd, vt=heads_first)
    k, v = attn.awq_kv4_read(c, p, st)
    for which, want in ((0, k), (1, v)):
        out = torch.zeros((kv, n, d + 8), dtype=torch.bfloat16, device="cuda").transpose(0, 1)[..., :d]
        pair = (out, None) if which == 0 else (None, out)
        assert attn.awq_kv4_read(c, p, st, out=pair)[which] is out
        assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_write_of_borders_and_extremes(attn, dtype):
    """Numbers on and beside the borders of two codes, constant groups, zeros, subnormal steps, the largest numbers."""
    rng = np.random.default_rng(8)
    d, n = 128, 400
    x = np.empty((n, 1, d))
    for i in range(n):
        step, offset = np.float16(2.0 ** rng.integers(-6, 3) * rng.integers(1, 9)), np.float16(rng.integers(-40, 5))
        q = rng.integers(0, 31, d) / 2.0  # half of them on a border
        q[:2] = 0, 15
        x[i, 0] = float(offset) + q * float(step)
        if i % 4 == 1:
            x[i, 0, 2:] *= 1 + rng.choice([-1, 0, 1], d - 2) * 2.0 ** -23
        if i % 4 == 2:
            x[i, 0, 2:] *= 1 + rng.choice([-1, 0, 1], d - 2) * 2.0 ** -8
    x[0], x[1], x[2], x[3] = 0.0, 1.7, -3e-9, 1e30 if dtype != "f16" else 6e4
    x[4] = np.linspace(-65504, 65504, d) if dtype == "f16" else np.linspace(-1e6, 1e6, d)
    x[5] = rng.standard_normal(d) * 1e-6
    x[6] = 1000 + rng.standard_normal(d) * 0.01
    x[7] = -65504
    x[8, 0, :64], x[8, 0, 64:] = 65504, -65504
    k = np.broadcast_to(x, (n, 1, d)).copy()
    codes, params = random_cache(rng, n // 16, 1, d, 16)
    _check(attn, codes, params, np.arange(n), k, -k, dtype)


def test_steps_are_rounded_once(attn):
    """(max - min) / 15 next to the middle of two float16 numbers: by way of float32 it would be rounded twice."""
    rng = np.random.default_rng(9)
    x = np.zeros((512, 1, 32))
    for i in range(512):
        mid = float(np.float16(rng.uniform(0.1, 1))) * (1 + 2.0 ** -11)
        x[i, 0, 5] = np.float32(15 * mid)
        x[i, 0, 6] = -np.float32(rng.choice([0, 2.0 ** -40, 2.0 ** -30]))
    codes, params = random_cache(rng, 32, 1, 32, 16)
    _check(attn, codes, params, np.arange(512), x, x, "f32")


@pytest.mark.parametrize("d", [64, 192])
def test_groups_with_nan_and_infinity(attn, d):
    rng = np.random.default_rng(10)
    x = rng.standard_normal((20, 2, d))
    x[3, 0, 7], x[4, 1, d - 1], x[5, 0, 0], x[6, 1, 63] = np.nan, np.inf, -np.inf, np.nan
    x[7] = np.nan
    codes, params = random_cache(rng, 2, 2, d, 16)
    c, p, wc, wp, st = _check(attn, codes, params, np.arange(20), x, x[::-1].copy(), "bf16")
    k, v = attn.awq_kv4_read(c, p, st)
    for got, want in zip((k, v), A.cached(wc, wp, np.arange(20) // 16, np.arange(20) % 16)):
        within(host(got), want, np.abs(want) * (half_step("bf16") + U) + U, "nan")
    assert bool(torch.isnan(k[3, 0, :64]).all()) and not bool(torch.isnan(k[3, 1]).any())
    # a foreign cache's infinite step or offset stands for NaNs too
    p[0, 0, 0, 0, 2, 0], p[0, 0, 1, 0, 8, 1] = float("inf"), float("-inf")
    k, _ = attn.awq_kv4_read(c, p, st)
    assert bool(torch.isnan(k[2, 0, :64]).all()) and bool(torch.isnan(k[8, 1, :64]).all())


def test_the_last_of_two_writes_stays(attn):
    rng = np.random.default_rng(11)
    codes, params = random_cache(rng, 4, 2, 64, 16)
    a, b = rng.standard_normal((30, 2, 64)), rng.standard_normal((30, 2, 64))
    c, p = cache_dev(codes, params)
    st = torch.from_numpy(rng.permutation(64)[:30]).cuda()
    attn.awq_kv4_write(dev(a, "bf16"), dev(a, "bf16"), c, p, st)
    attn.awq_kv4_write(dev(b, "bf16"), dev(a, "bf16"), c, p, st)
    wc, wp = _written(codes, params, st.cpu().numpy(), host(dev(b, "bf16")), host(dev(a, "bf16")))
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(p.cpu().numpy(), wp)
