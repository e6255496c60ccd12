"""Attention over the 4-bit cache as a model runs it, on the GPU: the exported QKV product, rotary positions, the cache's write,
attention, the exported output product, for prompts and then for single tokens; calls captured in graphs, on side streams and two at
a time; sizes at which every kernel, the split and the joining of parts are at work."""
import math

import numpy as np
import pytest

from oracle import awq_attn as A
from oracle import awq_w4a16 as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from attn_cases import attention_bound, paged  # noqa: E402
from moe_cases import dev, export, export_dev, half_step, host  # noqa: E402


@pytest.fixture(scope="module")
def attn():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import attn
    attn._load()
    return attn


# ---------------------------------------------------------------- a reference for large sizes


def _numbers(codes, params):
    """float64 numbers of codes [..., m, d / 2] with params [..., groups, m, 2]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    s, o = params.double().transpose(-3, -2).repeat_interleave(128, -2)[..., :q.shape[-1], :].unbind(-1)
    return q * s + o


def _check_rows(got, lse, q, codes, params, table, kv_len, offsets, s, h, causal, window, what):
    """The rows of sequence s and key head h against float64 on the device, by the bounds of attn_cases.attention_bound."""
    n, heads, d = q.shape
    group, page = heads // codes.shape[2], codes.shape[3]
    first, last, m = int(offsets[s]), int(offsets[s + 1]), int(kv_len[s])
    at = slice(h * group, (h + 1) * group)
    if not m or first == last:
        assert not bool(got[first:last, at].any()), what
        return
    pages = table[s, :(m + page - 1) // page].long()
    k, v = (_numbers(codes[pages, w, h], params[pages, w, h]).flatten(0, 1)[:m] for w in (0, 1))
    x = (q[first:last, at].double() @ k.t()) * d ** -0.5
    p = torch.arange(first, last, device=q.device)[:, None, None] - last + m
    j = torch.arange(m, device=q.device)
    seen = (j <= p) if causal else torch.ones_like(j <= p)
    if window:
        seen = seen & (j > p - window)
    x = x.masked_fill(~seen, -math.inf)
    any_seen = seen.any(-1, keepdim=True)
    w = torch.softmax(x, -1).masked_fill(~any_seen, 0.0)
    want = w @ v
    e = ((q[first:last, at].double().abs() @ k.abs().t()).masked_fill(~seen, 0).amax(-1, keepdim=True) * d ** -0.5 * (2.0 ** -11 + d * 2.0 ** -24)
         + (x.masked_fill(~seen, 0).abs().amax(-1, keepdim=True) + 1) * 2.0 ** -22)
    bound = (w @ v.abs()) * (2 * e + 2.0 ** -9 + 2.0 ** -11 + m * 2.0 ** -24) + m * 2.0 ** -31 * v.abs().amax(0)
    bound = bound + want.abs() * torch.finfo(got.dtype).eps / 2 + 2.0 ** -24
    off = (got[first:last, at].double() - want).abs() - bound
    assert float(off.max()) <= 0, f"{what}: {float(off.max()):.3g} past the bound"
    if lse is not None:
        want = torch.logsumexp(x, -1)
        off = (lse[first:last, at].double() - want).abs() - (e[..., 0] + 2.0 ** -10 + 2.0 ** -20 * (want.abs() + 4))
        assert float(off[any_seen.expand(-1, group, -1)[..., 0]].max()) <= 0, f"{what}: lse"


def _device_cache(rng, n_pages, kv, d, page):
    g = (d + 127) // 128
    gen = torch.Generator(device="cuda").manual_seed(int(rng.integers(1 << 30)))
    codes = torch.randint(0, 256, (n_pages, 2, kv, page, d // 2), generator=gen, device="cuda", dtype=torch.uint8)
    step = 0.15 + 0.3 * torch.rand((n_pages, 2, kv, g, page), generator=gen, device="cuda")
    offset = -3.5 + 2 * torch.rand((n_pages, 2, kv, g, page), generator=gen, device="cuda")
    return codes, torch.stack([step, offset], -1).half()


@pytest.mark.parametrize("q_len,kv_len,heads,kv,d,page,causal,window", [
    # single tokens: a split over all compute units, with whole sequences, ends and beginnings in a block
    ([1], [131071], 64, 8, 128, 128, True, 0), ([1] * 37, None, 64, 8, 128, 64, True, 0), ([1] * 700, None, 8, 2, 64, 16, True, 0),
    ([1] * 1100, None, 4, 1, 128, 32, True, 0), ([1] * 3000, None, 2, 2, 128, 16, True, 0), ([1] * 5, None, 128, 1, 64, 64, True, 0),
    ([1] * 20, None, 16, 8, 256, 16, True, 900), ([1], [40000], 32, 32, 96, 64, True, 0),
    # drafts
    ([5] * 24, None, 16, 8, 256, 16, True, 2048), ([4] * 9, None, 64, 8, 128, 64, True, 0), ([7] * 3, None, 20, 5, 64, 32, False, 0),
    # prompts: split and not, tiles of several sequences, group sizes that do not divide a tile
    ([700], [700], 8, 8, 128, 64, True, 0), ([2100], [6000], 16, 2, 128, 64, True, 0), ([300] * 4, None, 40, 8, 64, 32, True, 0),
    ([513, 0, 90, 1, 1200], None, 12, 4, 128, 16, True, 0), ([1000], [1500], 6, 2, 256, 64, True, 0), ([257, 300], None, 10, 2, 160, 128, False, 0),
    ([1500], [1500], 14, 2, 64, 64, True, 300), ([64] * 20, None, 64, 8, 128, 64, True, 0), ([400] * 30, None, 32, 4, 96, 64, True, 0)])
def test_large(attn, q_len, kv_len, heads, kv, d, page, causal, window):
    rng = np.random.default_rng(len(q_len) + heads + d)
    if kv_len is None:
        kv_len = [max(n, int(v)) for n, v in zip(q_len, rng.integers(1, 6000 if len(q_len) < 100 else 900, len(q_len)))]
        if len(kv_len) > 2 and q_len[2] == 1:
            kv_len[2] = 0
    print(f"[gpu attend] {len(q_len)} sequences, {sum(q_len)} tokens, kv {min(kv_len)}..{max(kv_len)}, heads={heads}/{kv} d={d} page={page} "
          f"causal={causal} window={window}", flush=True)
    table, pages = paged(rng, kv_len, page)
    codes, params = _device_cache(rng, pages, kv, d, page)
    offsets = np.concatenate([[0], np.cumsum(q_len)])
    table = torch.from_numpy(table).cuda()
    lens = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    dtype = "f16" if heads % 3 else "bf16"
    q = dev(1.5 * rng.standard_normal((sum(q_len), heads, d)), dtype)
    kw = {} if len(set(q_len)) == 1 else {"q_offsets": torch.from_numpy(offsets.astype(np.int32)).cuda()}
    got, lse = attn.awq_kv4_attention(q, codes, params, table, lens, causal=causal, window=window, max_kv=max(kv_len), lse=True, **kw)
    again = attn.awq_kv4_attention(q, codes, params, table, lens, causal=causal, window=window, max_kv=max(kv_len), **kw)
    assert torch.equal(got, again)  # the order of sums is fixed
    for s in set(rng.integers(0, len(q_len), 6).tolist()) | {0, len(q_len) - 1, min(2, len(q_len) - 1)}:
        for h in {0, kv - 1, int(rng.integers(kv))}:
            _check_rows(got, lse, q, codes, params, table, kv_len, offsets, s, h, causal, window, f"sequence {s}, head {h}")


def test_offsets_past_32_bits(attn):
    """A cache of more than 4 GiB of codes, and one whose pages are that far apart."""
    rng = np.random.default_rng(1)
    kv, d, page = 8, 128, 64
    pages = (1 << 32) // (2 * kv * page * d // 2) + 40
    codes = torch.zeros((pages, 2, kv, page, d // 2), dtype=torch.uint8, device="cuda")
    params = torch.zeros((pages, 2, kv, 1, page, 2), dtype=torch.float16, device="cuda")
    n = 300
    slots = torch.arange(n, device="cuda") + (pages - 20) * page + 5
    k, v = (torch.randn((n, kv, d), device="cuda").bfloat16() for _ in range(2))
    attn.awq_kv4_write(k, v, codes, params, slots)
    ck, cv = attn.awq_kv4_read(codes, params, slots, dtype=torch.float32)
    assert float((ck - k.float()).abs().max()) < 0.4 and float((cv - v.float()).abs().max()) < 0.4 and bool(ck.any(-1).all())
    table = torch.arange(pages - 20, pages, dtype=torch.int32, device="cuda")[None]
    assert int(codes[:pages - 20].max()) == 0
    for n_q, group in ((1, 8), (40, 4)):
        q = dev(rng.standard_normal((n_q, kv * group, d)), "bf16")
        got, lse = attn.awq_kv4_attention(q, codes, params, table, torch.tensor([n + 5], dtype=torch.int32, device="cuda"), lse=True)
        _check_rows(got, lse, q, codes, params, table, [n + 5], [0, n_q], 0, kv - 1, True, 0, "far pages")
    # one layer of pages of many: two pages more than 2 GiB apart
    wide = torch.zeros((2, (1 << 31) // (2 * 16 * 16) + 8, 2, 1, 16, 16), dtype=torch.uint8, device="cuda")[:, 7]
    part = torch.zeros((2, 2, 1, 1, 16, 2), dtype=torch.float16, device="cuda")
    k = torch.randn((32, 1, 32), device="cuda").bfloat16()
    attn.awq_kv4_write(k, k, wide, part, torch.arange(32, device="cuda"))
    near = attn.kv4_cache(2, 1, 32, 16)
    attn.awq_kv4_write(k, k, *near, torch.arange(32, device="cuda"))
    assert torch.equal(wide, near[0]) and torch.equal(part, near[1]) and bool(wide.any())
    q = torch.randn((1, 4, 32), device="cuda").bfloat16()
    args = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), torch.tensor([32], dtype=torch.int32, device="cuda")
    assert torch.equal(attn.awq_kv4_attention(q, wide, part, *args), attn.awq_kv4_attention(q, *near, *args))


def test_pitches_past_32_bits(attn):
    """Rotary positions, a write and attention of rows that lie more than 2^31 elements apart."""
    big = torch.zeros((2, (1 << 31) + 4096), dtype=torch.bfloat16, device="cuda")
    x = big[:, 16:16 + 4 * 64].unflatten(1, (4, 64))
    x.copy_(torch.randn((2, 4, 64), device="cuda"))
    small = x.clone()
    pos, f = torch.tensor([3, 9], dtype=torch.int32, device="cuda"), torch.rand(32, device="cuda")
    want = attn.awq_rope(small, pos, f)
    assert torch.equal(attn.awq_rope(x, pos, f, out=x), want) and torch.equal(x, want)
    a, b = attn.kv4_cache(1, 4, 64, 16), attn.kv4_cache(1, 4, 64, 16)
    slots = torch.tensor([2, 7], device="cuda")
    attn.awq_kv4_write(x, x, *a, slots)
    attn.awq_kv4_write(want, want, *b, slots)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    args = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.tensor([9], dtype=torch.int32, device="cuda")
    assert torch.equal(attn.awq_kv4_attention(x, *a, *args), attn.awq_kv4_attention(want, *a, *args))


# ---------------------------------------------------------------- together


class _Layer:
    """One attention layer with exported 4-bit QKV and output products."""

    def __init__(self, rng, d_model, heads, kv, d, page):
        self.heads, self.kv, self.d, self.page = heads, kv, d, page
        self.qkv, self.out = ([t[0] for t in export(rng, 1, r, c)] for r, c in (((heads + 2 * kv) * d, d_model), (d_model, heads * d)))
        self.dev = [export_dev(*w) for w in (self.qkv, self.out)]
        self.inv_freq = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
        self.axis = (np.arange(d // 2) % 3).astype(np.int32)
        self.f, self.a = torch.from_numpy(self.inv_freq).cuda(), torch.from_numpy(self.axis).cuda()

    def run(self, attn, B, x, positions, cache, slots, table, kv_len, offsets, max_kv):
        """The layer's output and what it gives on the way."""
        n = x.shape[0]
        row = B.awq_w4a16_gemm(x, *self.dev[0])
        if row.dtype != x.dtype:
            row = row.to(x.dtype)
        row = row.view(n, self.heads + 2 * self.kv, self.d)
        qk = row[:, :self.heads + self.kv]
        attn.awq_rope(qk, positions, self.f, axis=self.a, out=qk)
        attn.awq_kv4_write(qk[:, self.heads:], row[:, self.heads + self.kv:], *cache, slots)
        y = attn.awq_kv4_attention(qk[:, :self.heads], *cache, table, kv_len, q_offsets=offsets, max_kv=max_kv)
        return B.awq_w4a16_gemm(y.view(n, -1), *self.dev[1]), row, y


def test_a_layer_over_prompts_and_then_single_tokens(attn):
    from post_quantization_mean_amd import binding as B
    rng = np.random.default_rng(2)
    heads, kv, d, page, d_model = 8, 2, 64, 16, 256
    layer = _Layer(rng, d_model, heads, kv, d, page)
    prompts = [70, 9, 0, 33]
    total = [n + 3 for n in prompts]
    table, pages = paged(rng, total, page)
    cache = attn.kv4_cache(pages, kv, d, page)
    tt = torch.from_numpy(table).cuda()
    lens = np.zeros(4, np.int64)
    for step in range(4):
        q_len = prompts if step == 0 else [1] * 4
        n = sum(q_len)
        x = host(dev(rng.standard_normal((n, d_model)), "bf16"))
        places = np.concatenate([lens[s] + np.arange(q) for s, q in enumerate(q_len)]).astype(np.int64)
        seqs = np.repeat(np.arange(4), q_len)
        positions = np.stack([places, places // 2, places % 7])
        slots = table[seqs, places // page].astype(np.int64) * page + places % page
        lens += q_len
        offsets = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        got, row, y = layer.run(attn, B, dev(x, "bf16"), torch.from_numpy(positions).cuda(), cache, torch.from_numpy(slots).cuda(), tt,
                                torch.from_numpy(lens.astype(np.int32)).cuda(), torch.from_numpy(offsets).cuda() if step == 0 else None, int(lens.max()))
        # each link of the chain from what the link before it gave: the product, the rotation, the cache, attention, the product.
        # A product is a float32 chain (each addition off by at most 2^-24 of the magnitudes' sum) and one rounding.
        rows = host(row)
        w, size = W.w4a16_matmul(x, *layer.qkv), W.abs_product_sums(x, *layer.qkv)
        bound = np.abs(w) * half_step("bf16") + size * (d_model + 8) * 2.0 ** -24
        qkv = w.reshape(n, heads + 2 * kv, d)
        assert (np.abs(rows[:, heads + kv:] - qkv[:, heads + kv:]) <= bound.reshape(qkv.shape)[:, heads + kv:]).all()
        turned = A.rope(qkv[:, :heads + kv], positions, layer.inv_freq, layer.axis, False, 1.0)
        pair = np.tile((np.abs(qkv) * 2.0 ** -8 + bound.reshape(qkv.shape))[..., :d // 2] + (np.abs(qkv) * 2.0 ** -8 + bound.reshape(qkv.shape))[..., d // 2:], 2)
        assert (np.abs(rows[:, :heads + kv] - turned) <= pair[:, :heads + kv] * (1 + 2.0 ** -8) + np.abs(turned) * 2.0 ** -8).all()
        q, k, v = rows[:, :heads], rows[:, heads:heads + kv], rows[:, heads + kv:]
        if w is not None:
            assert np.abs(v.reshape(n, -1) - w[:, (heads + kv) * d:]).max() <= 0.02 * np.abs(w).max()
        codes, params = cache[0].cpu().numpy(), cache[1].cpu().numpy()
        for which, t in ((0, k), (1, v)):
            c, s, o = A.quantize(t)
            assert np.array_equal(codes[slots // page, which, :, slots % page], A.pack(c)), (step, which)
            assert np.array_equal(params[slots // page, which, :, :, slots % page], np.stack([s, o], -1))
        want, _ = A.attention(q, codes, params, table, lens, offsets, d ** -0.5, True, 0)
        bound = attention_bound(q, codes, params, table, lens, offsets, d ** -0.5, True, 0, want)
        assert (np.abs(host(y) - want) <= bound + np.abs(want) * half_step("bf16") + 2.0 ** -24).all()
        flat = host(y).reshape(n, -1)
        want, size = W.w4a16_matmul(flat, *layer.out), W.abs_product_sums(flat, *layer.out)
        assert (np.abs(host(got) - want) <= np.abs(want) * half_step("bf16") + size * (heads * d + 8) * 2.0 ** -24).all()
    # the same tokens in one go: queries of the last step see the same cache
    got2, _ = attn.awq_kv4_attention(dev(q, "bf16"), *cache, tt, torch.from_numpy(lens.astype(np.int32)).cuda(), lse=True)
    assert torch.equal(got2, y)


def _decode_state(attn, rng, seqs, heads, kv, d, page, longest):
    cap = (longest + page - 1) // page
    table = torch.from_numpy(rng.permutation(seqs * cap).astype(np.int32).reshape(seqs, cap)).cuda()
    codes, params = _device_cache(rng, seqs * cap, kv, d, page)
    row = torch.randn((seqs, heads + 2 * kv, d), device="cuda").bfloat16()
    return table, codes, params, row


@pytest.mark.parametrize("heads,kv,d", [(32, 8, 128), (16, 16, 64)])
def test_captured_steps(attn, heads, kv, d):
    """Rotation, write and attention of a decoded batch in a graph, replayed with other rows and lengths."""
    rng = np.random.default_rng(3)
    seqs, page, longest = 6, 16, 3000
    table, codes, params, row = _decode_state(attn, rng, seqs, heads, kv, d, page, longest)
    lens = torch.ones(seqs, dtype=torch.int32, device="cuda")
    f = torch.rand(d // 2, device="cuda")
    qk = torch.empty((seqs, heads + kv, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.empty((seqs, heads, d), dtype=torch.bfloat16, device="cuda"), torch.empty((seqs, heads), device="cuda")
    nb = attn.awq_kv4_attention_workspace_bytes(seqs, seqs, False, heads, kv, d, True, 0, longest)
    ws = torch.empty(max(nb, 1), dtype=torch.uint8, device="cuda")

    def step(codes, params, out, lse, ws):
        at = lens - 1
        attn.awq_rope(row[:, :heads + kv], at, f, out=qk)
        slots = table[torch.arange(seqs, device="cuda"), (at // page).long()].long() * page + at % page
        attn.awq_kv4_write(qk[:, heads:], row[:, heads + kv:], codes, params, slots)
        attn.awq_kv4_attention(qk[:, :heads], codes, params, table, lens, max_kv=longest, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(codes, params, out, lse, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(codes, params, out, lse, ws)
    for replay in range(5):
        lens.copy_(torch.from_numpy(rng.integers(1, longest, seqs).astype(np.int32)))
        row.copy_(torch.randn(row.shape, device="cuda"))
        want = [codes.clone(), params.clone(), torch.empty_like(out), torch.empty_like(lse)]
        step(*want, torch.empty_like(ws))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[2]) and torch.equal(lse, want[3]) and torch.equal(codes, want[0]) and torch.equal(params, want[1]), replay


def test_a_gradient_in_a_graph_beside_an_eager_graph_of_the_same_leaf(attn):
    x = torch.randn((50, 4, 64), device="cuda", requires_grad=True)
    eager = (x * 2).sum()  # a graph of x that lives on
    pos, f = torch.arange(50, device="cuda"), torch.rand(32, device="cuda")
    g = torch.randn((50, 4, 64), device="cuda")
    out = torch.empty_like(g)
    assert not attn.awq_rope(x, pos, f).requires_grad
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        attn.awq_rope_backward(g, pos, f, out=out)
    for _ in range(3):
        g.copy_(torch.randn(g.shape, device="cuda"))
        want = attn.awq_rope_backward(g, pos, f)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    eager.backward()
    assert bool((x.grad == 2).all())


def _beside(call, workspace_bytes):
    """call(stream) on a side stream that has some milliseconds of other work first, while the current stream overwrites all the
    new memory it can get of the workspace's and outputs' sizes."""
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


def test_on_a_side_stream(attn):
    rng = np.random.default_rng(4)
    table, codes, params, row = _decode_state(attn, rng, 4, 16, 4, 128, 64, 5000)
    q = row[:, :16].contiguous()
    lens = torch.tensor([5000, 1, 3333, 200], dtype=torch.int32, device="cuda")
    nb = attn.awq_kv4_attention_workspace_bytes(4, 4, False, 16, 4, 128, True, 0, 5000)
    assert nb > 0
    want = attn.awq_kv4_attention(q, codes, params, table, lens, max_kv=5000, lse=True)
    got = _beside(lambda s: attn.awq_kv4_attention(q, codes, params, table, lens, max_kv=5000, lse=True, stream=s), [nb, q.numel() * 2, 4 * 64])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    pos, f = torch.arange(4, device="cuda"), torch.rand(64, device="cuda")
    for call in (attn.awq_rope, attn.awq_rope_backward):
        assert torch.equal(_beside(lambda s: call(q, pos, f, stream=s), [q.numel() * 2]), call(q, pos, f))
    slots = torch.tensor([3, 70, -1, 200], device="cuda")
    a, b = (codes.clone(), params.clone()), (codes.clone(), params.clone())
    attn.awq_kv4_write(row[:, 16:20], row[:, 20:], *a, slots)
    _beside(lambda s: attn.awq_kv4_write(row[:, 16:20], row[:, 20:], *b, slots, stream=s), [1 << 16])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    got = _beside(lambda s: attn.awq_kv4_read(*a, slots, stream=s), [4 * 4 * 128 * 2])
    assert all(torch.equal(x, y) for x, y in zip(got, attn.awq_kv4_read(*a, slots)))


def test_two_calls_at_once(attn):
    rng = np.random.default_rng(5)
    table, codes, params, row = _decode_state(attn, rng, 4, 16, 4, 128, 64, 20000)
    q = row[:, :16].contiguous()
    prompt = torch.randn((4 * 600, 16, 128), device="cuda").bfloat16()
    lens = torch.tensor([20000, 700, 3333, 9000], dtype=torch.int32, device="cuda")
    calls = [lambda s: attn.awq_kv4_attention(q, codes, params, table, lens, max_kv=20000, stream=s),
             lambda s: attn.awq_kv4_attention(prompt, codes, params, table, lens, max_kv=20000, stream=s)]
    want = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[c(s) for c, s in zip(calls, streams)] for _ in range(5)]
    torch.cuda.synchronize()
    for pair in got:
        assert all(torch.equal(a, b) for a, b in zip(pair, want))


def test_refusals_of_the_binding(attn):
    codes, params = attn.kv4_cache(4, 2, 64, 16)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.zeros((2, 3), dtype=torch.int32, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    k, slots = torch.zeros((2, 2, 64), device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    f = torch.zeros(32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    bad = [
        (ValueError, lambda: attn.awq_kv4_attention(q[..., :32], codes, params, table, lens)),
        (TypeError, lambda: attn.awq_kv4_attention(q, codes, params, table.long(), lens)),
        (TypeError, lambda: attn.awq_kv4_attention(q, codes, params, table, lens.long())),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes, params, table, lens[:1])),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes, params, table.t(), lens)),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes, params, table[:, ::2], lens)),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes, params, table, lens, q_offsets=lens)),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes.transpose(2, 3).contiguous().transpose(2, 3), params, table, lens)),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes.cpu(), params, table, lens)),
        (ValueError, lambda: attn.awq_kv4_attention(q, codes, params, table, lens, lse=torch.zeros(4, 2, device="cuda"))),
        (TypeError, lambda: attn.awq_kv4_attention(q, codes, params, table, lens, out=torch.zeros((2, 4, 64), dtype=torch.float16, device="cuda"))),
        (attn.AwqError, lambda: attn.awq_kv4_attention(torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"), codes, params, table, lens)),
        (attn.AwqError, lambda: attn.awq_kv4_attention(q[:, :3], codes, params, table, lens)),
        (ValueError, lambda: attn.awq_kv4_write(k, k[:1], codes, params, slots)),
        (TypeError, lambda: attn.awq_kv4_write(k, k.half(), codes, params, slots)),
        (TypeError, lambda: attn.awq_kv4_write(k, k, codes, params, slots.float())),
        (ValueError, lambda: attn.awq_kv4_write(k, k, codes, params, slots[:1])),
        (ValueError, lambda: attn.awq_kv4_read(codes, params, slots, out=(None, None))),
        (TypeError, lambda: attn.awq_kv4_read(codes, params, slots, dtype=torch.int32)),
        (ValueError, lambda: attn.awq_rope(q, pos[:1], f)), (TypeError, lambda: attn.awq_rope(q, pos.float()[None], f)),
        (TypeError, lambda: attn.awq_rope(q, pos, f.double())), (ValueError, lambda: attn.awq_rope(q, pos, f, axis=pos)),
        (ValueError, lambda: attn.awq_rope(q, pos, f, style="other")), (ValueError, lambda: attn.awq_rope(q.transpose(1, 2), pos, f)),
        (attn.AwqError, lambda: attn.awq_rope(q, pos, torch.zeros(33, device="cuda"))),
        (attn.AwqError, lambda: attn.awq_rope(q[:0], pos[:0], f)),
        (attn.AwqError, lambda: attn.awq_rope(q, pos, f, out=q.expand(2, 4, 64).as_strided((2, 4, 64), (64, 64, 1)))),
    ]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")
