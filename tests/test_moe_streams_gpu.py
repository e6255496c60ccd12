"""Calls of the mixture-of-experts block with `stream=`, beside work on the current stream that allocates memory of the same
sizes and overwrites it: the results of calls without."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import moe
    moe._load()
    return moe


def _beside(call, workspace_bytes):
    """call(stream) on a side stream that has some milliseconds of other work first, while the current stream overwrites
    all the new memory it can get of the workspace's and outputs' sizes."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        a = torch.ones((2048, 2048), device="cuda")
        for _ in range(40):
            a = a @ a * 2.0 ** -11
    got = call(side)
    took = [torch.full((max(nb, 1),), 0x7B, dtype=torch.uint8, device="cuda") for nb in workspace_bytes for _ in range(8)]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(bool((t == 0x7B).all()) for t in took) and bool((a == 1).all())
    return got


def test_sort_on_a_side_stream(moe):
    ids = torch.randint(-1, 64, (4000, 8), device="cuda")
    ref = moe.awq_moe_sort(ids, 64)
    nb = moe.awq_moe_sort_workspace_bytes(4000, 8, 64)
    assert nb > 0
    got = _beside(lambda s: moe.awq_moe_sort(ids, 64, stream=s), [nb, 4 * 32000, 4 * 65])
    assert all(torch.equal(got[k], ref[k]) for k in ref)


@pytest.mark.parametrize("n,d", [(700, 1040), (300, 9000)])
def test_norms_on_a_side_stream(moe, n, d):
    y, r, dr, dh = (torch.randn((n, d), device="cuda").bfloat16() for _ in range(4))
    w1, w2, gate = (torch.randn(d, device="cuda").bfloat16() for _ in range(3))
    ref, back = moe.awq_block_norm(y, r, w2, w1, gate), moe.awq_block_norm_backward(y, r, dr, dh, w2, w1, gate)
    got = _beside(lambda s: moe.awq_block_norm(y, r, w2, w1, gate, stream=s), [2 * n * d])
    assert all(torch.equal(got[k], ref[k]) for k in ref)
    nb = moe.awq_block_norm_backward_workspace_bytes(n, d)
    got = _beside(lambda s: moe.awq_block_norm_backward(y, r, dr, dh, w2, w1, gate, stream=s), [nb, 2 * n * d, 4 * d])
    assert all(torch.equal(got[k], back[k]) for k in back)


def test_rows_on_a_side_stream(moe):
    ids = torch.randint(0, 8, (900, 2), device="cuda")
    x, w = torch.randn((900, 512), device="cuda").bfloat16(), torch.rand((900, 2), device="cuda")
    pos = moe.awq_moe_sort(ids, 8)["position"]
    rows = moe.awq_moe_gather(x, pos)
    nb = [rows.numel() * 2, x.numel() * 2]
    for f, args in ((moe.awq_moe_gather, (x, pos)), (moe.awq_moe_combine, (rows, pos, w)), (moe.awq_moe_gather_backward, (rows, pos)),
                    (lambda *a, **k: moe.awq_moe_combine_backward(*a, **k)["d_weights"], (x, rows, pos, w))):
        assert torch.equal(_beside(lambda s: f(*args, stream=s), nb), f(*args))
