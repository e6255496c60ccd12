"""Rows of the experts' products that start anywhere: single rows of any pitch, and contiguous gradients of any width. Exact
inputs: the bits of padded rows."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import export, export_dev  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _offsets(n):
    return torch.tensor([0, n // 3, n // 3, n], dtype=torch.int32, device="cuda")


def _padded(x):
    """The same rows with a pitch of a multiple of 8, at the start of a buffer."""
    n, d = x.shape
    p = torch.zeros((n, (d + 7) // 8 * 8), dtype=x.dtype, device="cuda")[:, :d]
    p.copy_(x)
    return p


@pytest.mark.parametrize("d_out", [300, 33])
def test_a_single_row_of_any_pitch(moe, d_out):
    rng = np.random.default_rng(d_out)
    ex, off = export_dev(*export(rng, 3, d_out, 256, True)), _offsets(1)
    wide = torch.from_numpy(rng.integers(-8, 9, (3, 263))).to(torch.bfloat16).cuda()
    got = moe.awq_w4a16_grouped_gemm(wide[:1, :256], *ex, off)
    assert torch.equal(got, moe.awq_w4a16_grouped_gemm(wide[:1, :256].clone(memory_format=torch.contiguous_format), *ex, off))
    dy = torch.from_numpy(rng.integers(-8, 9, (1, d_out))).to(torch.bfloat16).cuda()
    assert torch.equal(moe.awq_w4a16_grouped_gemm_backward(dy, *ex, off), moe.awq_w4a16_grouped_gemm_backward(_padded(dy), *ex, off))


# few rows (several kernels), tiles with whole and cut contractions
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d_out", [(2, 1), (9, 300), (40, 33), (100, 70), (700, 130), (33000, 100)])
def test_a_contiguous_gradient_of_any_width(moe, dtype, n, d_out):
    """What a contiguous product of the same layout gives back; one that starts between 16-byte boundaries too."""
    rng = np.random.default_rng(n + d_out)
    print(f"[gpu grouped rows] n={n} d_out={d_out} {dtype}", flush=True)
    ex, off = export_dev(*export(rng, 3, d_out, 256, True)), _offsets(n)
    buf = torch.from_numpy(rng.integers(-8, 9, n * d_out + 1)).to(dtype).cuda()
    for dy in (buf[:-1].view(n, d_out), buf[1:].view(n, d_out)):
        kept = dy.clone()
        want = moe.awq_w4a16_grouped_gemm_backward(_padded(dy), *ex, off)
        assert torch.equal(moe.awq_w4a16_grouped_gemm_backward(dy, *ex, off), want) and torch.equal(dy, kept)
