"""The mixture-of-experts block as it is used: experts quantized on their own tokens by the search (awq_layer,
awq_export_fp16), then the block run with the exports: norm, sort, gather with 1 / s, the gated product, the down
product, combine, and the norm after it; its gradient; the same captured in a HIP graph, on a side stream and twice
at once.

Bounds. The forward bound carries every stage's rounding (half a step of its value) through the stages behind it
with the magnitudes of the weights. The gradient is compared in the 2-norm: it passes nine 16-bit roundings of
at most 2^-8 each; a later stage enlarges a relative error by at most |W| |g| / |W g|, which is the ratio of two random
sums and is taken as 2: 9 * 2 * 2^-8 = 0.07."""
import numpy as np
import pytest

from oracle import awq_moe as M

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from moe_cases import U, host, within  # noqa: E402

N, K, E, D, FF = 200, 2, 4, 256, 128
EPS = float(np.float32(1e-6))
H = 2.0 ** -8  # half a step of bfloat16


@pytest.fixture(scope="module")
def libs():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from post_quantization_mean_amd import binding, moe
    moe._load()
    return moe, binding


def _stacked(B, xs, ws):
    """Each expert quantized on its own rows: the stacked export and the searched scales."""
    parts, scales = [], []
    for x, w in zip(xs, ws):
        res = B.awq_layer(x, w, n_grid=4)
        ex = B.awq_export_fp16(res["qscales"], res["zeros"])
        parts.append((res["codes"], ex["steps_f16"], ex["zeros_u4"]))
        scales.append(res["best_scales"])
    return [torch.stack(t).contiguous() for t in zip(*parts)], torch.stack(scales)


@pytest.fixture(scope="module")
def block(libs):
    """Inputs, and the two stacked exports of a block whose experts were quantized on the tokens they see."""
    moe, B = libs
    g = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).bfloat16()  # noqa: E731
    v = {"y": rnd(N, D), "residual": rnd(N, D), "gate": rnd(D), "w_post": 1 + rnd(D, k=0.2), "w_pre": 1 + rnd(D, k=0.2),
         "w_last": 1 + rnd(D, k=0.2)}
    ids = torch.topk(torch.rand((N, E), generator=g, device="cuda"), K, dim=1).indices
    ids[::17, 1] = -1
    v["ids"] = ids
    v["weights"] = torch.softmax(torch.randn((N, K), generator=g, device="cuda"), 1)
    first = moe.awq_block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], 0.5, EPS)
    plan = moe.awq_moe_sort(ids, E)
    rows = moe.awq_moe_gather(first["h"], plan["position"])
    ends = plan["offsets"].tolist()
    xs = [rows[a:b] for a, b in zip(ends, ends[1:])]
    v["gate_up"], s = _stacked(B, xs, [rnd(2 * FF, D, k=D ** -0.5) for _ in range(E)])
    v["in_scales"] = (1.0 / s).float()
    hs = [moe.awq_w4a16_grouped_gemm(x.contiguous() * i.bfloat16(), *[t[e:e + 1] for t in v["gate_up"]],
                                     torch.tensor([0, len(x)], dtype=torch.int32, device="cuda"), act="silu")
          for e, (x, i) in enumerate(zip(xs, v["in_scales"]))]
    v["down"], s = _stacked(B, hs, [rnd(D, FF, k=FF ** -0.5) for _ in range(E)])
    v["mid_scales"] = (1.0 / s).float()  # kept apart here, so that the export's own weights are what is multiplied
    return v


def _scale_rows(x, scales, offsets):
    """Rows times their expert's scales (a program folds these into the up rows; here the chain stays explicit)."""
    at = torch.arange(x.shape[0], device=x.device, dtype=torch.int32)
    e = torch.searchsorted(offsets[1:].contiguous(), at, right=True).clamp(max=E - 1)
    return (x.float() * scales[e]).bfloat16()


def _forward(moe, v, keep=None):
    first = moe.awq_block_norm(v["y"], v["residual"], v["w_pre"], v["w_post"], v["gate"], 0.5, EPS)
    plan = moe.awq_moe_sort(v["ids"], E)
    zeros = lambda w: torch.zeros((N * K, w), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rows = moe.awq_moe_gather(first["h"], plan["position"], expert_ids=v["ids"], in_scales=v["in_scales"], out=zeros(D))
    h = moe.awq_w4a16_grouped_gemm(rows, *v["gate_up"], plan["offsets"], act="silu", y=zeros(FF))
    h = _scale_rows(h, v["mid_scales"], plan["offsets"])
    o = moe.awq_w4a16_grouped_gemm(h, *v["down"], plan["offsets"], y=zeros(D))
    out = moe.awq_moe_combine(o, plan["position"], v["weights"])
    last = moe.awq_block_norm(out, first["residual"], v["w_last"], v["w_post"], None, 1.0, EPS)
    if keep is not None:
        keep.update(first=first, plan=plan, rows=rows, o=o, out=out)
    return last


def _weights(t):
    return [torch.from_numpy(w) for w in M.expert_weights(host(t[0]), host(t[1]).view(np.uint16), host(t[2]), "bf16")]


def _reference(v, d=None):
    """The block in float64 (torch on the CPU, so that its gradient can be asked for)."""
    f = lambda k: d[k] if d is not None and k in d else torch.from_numpy(host(v[k]))  # noqa: E731
    norm = lambda x, w: x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w  # noqa: E731
    r = f("residual") + 0.5 * f("gate") * norm(f("y"), f("w_post"))
    h = norm(r, f("w_pre"))
    ids = host(v["ids"])
    W1, W2, s1, s2 = _weights(v["gate_up"]), _weights(v["down"]), f("in_scales"), f("mid_scales")
    out = torch.zeros((N, D), dtype=torch.float64)
    mag = torch.zeros((N, D), dtype=torch.float64)  # the forward bound of the combined rows
    for e in range(E):
        t, j = np.nonzero(ids == e)
        x = h[t] * s1[e]
        ex = 3 * H * x.abs()  # the residual's, h's and the row's rounding
        gu, dgu = x @ W1[e].T, ex @ W1[e].abs().T
        g, u, dg, du = gu[:, :FF], gu[:, FF:], dgu[:, :FF], dgu[:, FF:]
        a = g * torch.sigmoid(g) * u * s2[e]
        da = (1.1 * dg * (u.abs() + du) + (g.abs() + dg) * du) * s2[e] + 2 * H * a.abs()
        w = f("weights")[t, j][:, None]
        out = out.index_add(0, torch.from_numpy(t), a @ W2[e].T * w)
        mag = mag.index_add(0, torch.from_numpy(t), (da @ W2[e].abs().T + H * (a @ W2[e].T).abs()) * w)
    mag = mag + H * out.abs()
    r2 = r + norm(out, f("w_post"))
    return {"residual": r2, "h": norm(r2, f("w_last")), "out": out, "mag": mag, "r": r}


def test_forward(libs, block):
    moe, _ = libs
    keep = {}
    last = _forward(moe, block, keep)
    ref = _reference(block)
    within(host(keep["out"]), ref["out"].numpy(), ref["mag"].numpy() * 1.05 + 64 * U, "out")  # 5 %: products of two bounds
    want, h = M.block_norm(host(keep["out"]), host(keep["first"]["residual"]), host(block["w_last"]), host(block["w_post"]), None,
                           1.0, EPS)
    within(host(last["residual"]), want, H * np.abs(want) + 256 * U * (1 + np.abs(want)), "residual")
    within(host(last["h"]), h, H * np.abs(h) + 1024 * U * (1 + np.abs(h)), "h")


def test_gradient_of_the_block(libs, block):
    """Through combine, the down product, the gated activation (by its formula, in float32), the gate/up product,
    gather and the norm, from a gradient of `out`."""
    moe, _ = libs
    v, keep = block, {}
    _forward(moe, v, keep)
    plan, zeros = keep["plan"], lambda w: torch.zeros((N * K, w), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    G = torch.randn((N, D), generator=g, device="cuda").bfloat16()
    b = moe.awq_moe_combine_backward(G, keep["o"], plan["position"], v["weights"], out={"d_rows": zeros(D)})
    d_h = moe.awq_w4a16_grouped_gemm_backward(b["d_rows"], *v["down"], plan["offsets"], dx=zeros(FF))
    gu = moe.awq_w4a16_grouped_gemm(keep["rows"], *v["gate_up"], plan["offsets"],
                                    y=torch.zeros((N * K, 2 * FF), device="cuda"))
    d_a = _scale_rows(d_h, v["mid_scales"], plan["offsets"]).float()
    gt, up = gu[:, :FF], gu[:, FF:]
    s = torch.sigmoid(gt)
    d_gu = torch.cat([d_a * up * s * (1 + gt * (1 - s)), d_a * gt * s], 1).bfloat16()
    d_rows = moe.awq_w4a16_grouped_gemm_backward(d_gu, *v["gate_up"], plan["offsets"], dx=zeros(D))
    d_hn = moe.awq_moe_gather_backward(d_rows, plan["position"], expert_ids=v["ids"], in_scales=v["in_scales"])
    n = moe.awq_block_norm_backward(v["y"], v["residual"], None, d_hn, v["w_pre"], v["w_post"], v["gate"], 0.5, EPS)
    got = {"weights": b["d_weights"], "y": n["d_y"], "residual": n["d_residual"], "w_pre": n["d_w_pre"], "w_post": n["d_w_post"],
           "gate": n["d_gate"]}
    leaves = {k: torch.from_numpy(host(v[k])).requires_grad_() for k in got}
    want = torch.autograd.grad(torch.sum(_reference(v, leaves)["out"] * torch.from_numpy(host(G))), list(leaves.values()))
    kept = host(plan["position"]) >= 0
    for (k, a), w in zip(got.items(), want):
        a, w = host(a), w.numpy()
        if k == "weights":
            assert np.all(a[~kept] == 0) and np.all(w[~kept] == 0)
        off = np.linalg.norm(a - w) / np.linalg.norm(w)
        print(f"  d_{k}: {off:.2e}", flush=True)
        assert off < 9 * 2 * H, k


def test_captured_replayed_and_on_a_side_stream(libs, block):
    """A capture of the block gives the eager result on every replay, with new inputs and eager work in between; the
    same on a side stream, and twice at once on two streams."""
    moe, _ = libs
    v = dict(block)
    for k in ("y", "residual", "ids"):
        v[k] = block[k].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _forward(moe, v)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _forward(moe, v)
    g = torch.Generator(device="cuda").manual_seed(13)
    for i in range(4):
        v["y"].copy_(torch.randn((N, D), generator=g, device="cuda").bfloat16())
        ids = torch.topk(torch.rand((N, E), generator=g, device="cuda"), K, dim=1).indices
        ids[i::5, 0] = -1
        v["ids"].copy_(ids)
        graph.replay()
        want = _forward(moe, v)
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), (i, k)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    res = []
    for s in (a, b, a, b):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            res.append(_forward(moe, v))
    torch.cuda.synchronize()
    for r in res:
        assert all(torch.equal(r[k], want[k]) for k in want)


def test_gradients_captured_and_replayed(libs, block):
    """The gradients are bitwise the same eager and replayed (no atomics), with a caller's workspace."""
    moe, _ = libs
    v, keep = block, {}
    _forward(moe, v, keep)
    plan = keep["plan"]
    G = torch.randn((N, D), device="cuda").bfloat16()
    ws = torch.empty(moe.awq_block_norm_backward_workspace_bytes(N, D), dtype=torch.uint8, device="cuda")
    rows = torch.zeros((N * K, D), dtype=torch.bfloat16, device="cuda")

    def step():
        b = moe.awq_moe_combine_backward(G, keep["o"], plan["position"], v["weights"], out={"d_rows": rows})
        dx = moe.awq_w4a16_grouped_gemm_backward(b["d_rows"], *v["down"], plan["offsets"])
        d = moe.awq_moe_gather_backward(b["d_rows"], plan["position"], expert_ids=v["ids"], in_scales=v["in_scales"])
        n = moe.awq_block_norm_backward(v["y"], v["residual"], G, d, v["w_pre"], v["w_post"], v["gate"], 0.5, EPS, workspace=ws)
        return {**b, **n, "dx": dx[:int(N * K * 0.9)]}

    kept = int(plan["offsets"][-1])
    assert kept >= int(N * K * 0.9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        G.copy_(torch.randn((N, D), device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got_now = {k: t.clone() for k, t in got.items()}
        want = step()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got_now[k], want[k]), k
