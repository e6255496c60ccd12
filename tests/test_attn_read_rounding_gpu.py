"""awq_kv4_read rounds offset + code * step once to its type, also where the sum is no float32: the results are equal to the sum in
float64, where it is exact, rounded to the nearest (ties to even)."""
import numpy as np
import pytest

from oracle import awq_attn as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import DTYPES, host  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


def _rounded(x, dtype):
    if dtype != "bf16":
        with np.errstate(over="ignore"):
            return x.astype({"f16": np.float16, "f32": np.float32}[dtype]).astype(np.float64)
    m, e = np.frexp(x)
    return np.ldexp(np.rint(m * 256) / 256, e)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [32, 128, 160])
def test_sums_that_float32_does_not_hold(attn, d, dtype):
    rng = np.random.default_rng(d)
    pages, page, kv, g = 40, 64, 2, (d + 127) // 128
    codes = rng.integers(0, 256, (pages, 2, kv, page, d // 2)).astype(np.uint8)
    shape = (pages, 2, kv, g, page)
    # offsets on the middle of two bfloat16 numbers, and small steps of both signs; any finite pairs; subnormal ones; zeros
    mid = (rng.integers(128, 256, shape) + 0.5) * 2.0 ** rng.integers(-8, 4, shape) * rng.choice([-1, 1], shape)
    small = rng.integers(1024, 2048, shape) * 2.0 ** -24 * rng.choice([-1, 1], shape) * 2.0 ** rng.integers(0, 6, shape)
    params = np.stack([small, mid], -1).astype(np.float16)
    any_bits = rng.integers(0, 0x7C00, (*shape, 2)).astype(np.uint16) | rng.integers(0, 2, (*shape, 2)).astype(np.uint16) << 15
    params[10:20] = any_bits.view(np.float16)[10:20]
    params[20:25, ..., 0] = rng.integers(0, 40, shape)[20:25] * 2.0 ** -24
    params[25:30, ..., 1] = 0.0
    params[30:35] = params[30:35, ..., ::-1]  # large steps, small offsets
    slots = rng.permutation(pages * page)
    out = tuple(torch.zeros((pages * page, kv, d), dtype=DTYPES[dtype], device="cuda") for _ in range(2))
    print(f"[gpu kv4] read d={d} {dtype}", flush=True)
    attn.awq_kv4_read(torch.from_numpy(codes).cuda(), torch.from_numpy(params).cuda(), torch.from_numpy(slots).cuda(), out=out)
    twice = 0
    for got, exact in zip(out, A.cached(codes, params, slots // page, slots % page)):
        want = _rounded(exact, dtype)
        assert np.array_equal(host(got), want), f"{(host(got) != want).sum()} of {want.size}"
        twice += int((_rounded(exact.astype(np.float32).astype(np.float64), dtype) != want).sum())
    assert dtype != "bf16" or twice > 0  # the inputs hold sums that two roundings get wrong
