"""Inputs and exact conversions shared by the GPU tests of the mixture-of-experts block."""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = 2.0 ** -24  # half a step of float32


def half_step(dtype) -> float:
    return torch.finfo(DTYPES[dtype]).eps / 2


def host(t):
    """A device tensor's values, exactly, in float64 (integers stay integers)."""
    t = t.detach().cpu()
    return t.double().numpy() if t.is_floating_point() else t.numpy()


def dev(a, dtype):
    return torch.from_numpy(np.asarray(a, np.float64)).to(DTYPES[dtype]).cuda()


def pitched(a, dtype, ld):
    """A [n, d] device matrix inside a buffer of pitch ld that starts one element late, so that no row is
    aligned; the rest of the buffer holds 7."""
    n, d = np.shape(a)
    buf = torch.full((n * ld + 1,), 7.0, dtype=DTYPES[dtype], device="cuda")
    m = buf[1:].view(n, ld)[:, :d]
    m.copy_(dev(a, dtype))
    return m, buf


def export(rng, n_experts, d_out, d_in, exact=False):
    """(codes, step bits, packed zero points) of stacked experts: any nibbles; steps powers of two from 2^-8 to
    2^-4 (`exact`) or uniform."""
    g = d_in // 128
    q = rng.integers(0, 16, (n_experts, d_out, d_in)).astype(np.uint8)
    z = rng.integers(0, 16, (n_experts, d_out, 2 * ((g + 1) // 2))).astype(np.uint8)
    s = 2.0 ** rng.integers(-8, -3, (n_experts, d_out, g)) if exact else rng.uniform(0.002, 0.02, (n_experts, d_out, g))
    return q[..., 0::2] | (q[..., 1::2] << 4), s.astype(np.float16).view(np.uint16), z[..., 0::2] | (z[..., 1::2] << 4)


def export_dev(codes, steps, zeros):
    return (torch.from_numpy(codes).cuda(), torch.from_numpy(steps.view(np.int16)).cuda(), torch.from_numpy(zeros).cuda())


def within(got, want, tol, what):
    """|got - want| <= tol, with NaN and infinities in the same places."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), f"{what}: infinities"
    off = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert not off.size or off.max() <= 0, f"{what}: {off.max():.3g} past the bound, at most {np.abs(got - want)[fine].max():.3g} off"
