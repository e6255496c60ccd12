"""Thin Python binding of the 4-bit mixture-of-experts block (include/awq_moe.h, in libawq_mi355x.so).

As in `binding`, every function has the name of the C entry point it calls and only marshals arguments;
outputs are allocated unless given. Work goes to torch's current stream of the tensors' device. With `stream`
(a stream of that device) a call does what it does inside `torch.cuda.stream(stream)`: outputs and workspaces
are allocated there too, and what is passed has to be ready on that stream and to outlive its work; an output that
is used on another stream has to wait for it. No call records a graph for autograd: outputs do not require a
gradient even where inputs do, and the *_backward functions are the gradients, for a program that calls them itself;
the quantized weights and the input multipliers are constants.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import AwqError, _HALF_BITS, _buf, _c_i64, _c_int, _c_size, _on_stream, _vp, _workspace  # noqa: F401

AWQ_MAX_EXPERTS = 1024
AWQ_MAX_TOP_K = 64
AWQ_MAX_SLOTS = 1 << 23
AWQ_MAX_NORM_WIDTH = 32768
AWQ_GROUPED_PLAIN = 0
AWQ_GROUPED_GATED_SILU = 1
AWQ_GROUPED_GATED_RELU = 2

_c_float = ctypes.c_float
_SIGNATURES = {
    "awq_block_norm": (_c_int, [_vp, _c_i64, _vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_float, _vp,
                                _c_float, _vp, _c_i64, _vp, _c_i64, _vp]),
    "awq_block_norm_backward_workspace_bytes": (_c_size, [_c_i64, _c_i64]),
    "awq_block_norm_backward": (_c_int, [_vp, _c_i64, _vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_float,
                                         _vp, _c_float, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _vp,
                                         _vp, _c_i64, _vp, _c_size, _vp]),
    "awq_moe_sort_workspace_bytes": (_c_size, [_c_i64, _c_int, _c_int]),
    "awq_moe_sort": (_c_int, [_vp, _c_int, _c_i64, _c_int, _c_int, _vp, _vp, _vp, _vp, _c_size, _vp]),
    "awq_moe_gather": (_c_int, [_vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _c_int, _vp, _c_int, _vp, _c_int, _vp,
                                _c_i64, _c_i64, _vp]),
    "awq_moe_gather_backward": (_c_int, [_vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _c_i64, _c_int, _vp, _c_int, _vp,
                                         _c_int, _vp, _c_i64, _vp]),
    "awq_moe_combine": (_c_int, [_vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_int, _vp, _c_i64, _vp]),
    "awq_moe_combine_backward": (_c_int, [_vp, _c_i64, _vp, _c_i64, _c_int, _c_i64, _c_i64, _vp, _vp, _c_i64, _c_int,
                                          _vp, _c_i64, _vp, _vp]),
    "awq_w4a16_grouped_gemm": (_c_int, [_vp, _c_i64, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_i64, _c_i64, _c_i64,
                                        _c_int, _vp, _c_i64, _c_int, _vp]),
    "awq_w4a16_grouped_gemm_backward": (_c_int, [_vp, _c_i64, _c_int, _vp, _vp, _vp, _vp, _c_int, _c_i64, _c_i64,
                                                 _c_i64, _vp, _c_i64, _c_int, _vp]),
}
_DTYPES = {torch.float32: binding.AWQ_DTYPE_F32, torch.bfloat16: binding.AWQ_DTYPE_BF16,
           torch.float16: binding.AWQ_DTYPE_F16}
_MODES = {None: AWQ_GROUPED_PLAIN, "silu": AWQ_GROUPED_GATED_SILU, "relu": AWQ_GROUPED_GATED_RELU}

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = binding.load_library()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_symbols() -> list[str]:
    return list(_SIGNATURES)


# the raw handle of a device's current stream; the public call builds a Stream object, which costs a small call as much
# as its launch
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, dev, *args) -> None:
    """Enqueues on the current stream of the tensors' device, with that device current."""
    index = dev.index
    if index == torch.cuda.current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status:
        binding._check(status)


def _matrix(t, name: str, shape=None, dtype=None, device=None) -> tuple[int, int]:
    """(pointer, row pitch) of a device matrix with unit stride along its rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    rows, cols = t.shape
    if shape is not None and (rows, cols) != shape:
        raise ValueError(f"{name} must be a {list(shape)} matrix, not {[rows, cols]}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return t.data_ptr(), row if rows > 1 else cols  # (the stride of a single row means nothing)


def _output(t, name: str, shape, dtype, device):
    """A caller's output or a new one, with its pointer and pitch."""
    if t is None:
        t = torch.empty(*shape, dtype=dtype, device=device)  # sizes one by one: a tuple costs almost a microsecond more
        return t, t.data_ptr(), shape[1]
    p, ld = _matrix(t, name, shape, dtype, device)
    if ld < shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    return t, p, ld


def _vector(t, name: str, dtype, n: int, device) -> int:
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == (n,) and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must be a vector of {n} elements")
    return _buf(t, name, dtype, n, device)


def _data_dtype(t, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be a torch.bfloat16, torch.float16 or torch.float32 tensor")
    return _DTYPES[t.dtype]


# ------------------------------------------------------------------ norms around a block


def _norm_args(y, residual, w_pre, w_post, gate, res_scale, eps):
    """The arguments that both directions share: (dtype, n, d, device, arguments)."""
    dt = _data_dtype(residual, "residual")
    t, dev = residual.dtype, residual.device
    pr, ldr = _matrix(residual, "residual")
    n, d = residual.shape
    py, ldy = (None, 0) if y is None else _matrix(y, "y", (n, d), t, dev)
    p1 = None if w_post is None else _vector(w_post, "w_post", t, d, dev)
    p2 = None if w_pre is None else _vector(w_pre, "w_pre", t, d, dev)
    pg, ldg = None, 0
    if gate is not None:
        if isinstance(gate, torch.Tensor) and gate.dim() == 2:
            pg, ldg = _matrix(gate, "gate", (n, d), t, dev)
            if ldg == 0:
                raise ValueError("a gate that is one row for all tokens is a vector")
        else:
            pg = _vector(gate, "gate", t, d, dev)
    return t, n, d, dev, (py, ldy, pr, ldr, dt, n, d, p1, pg, ldg, res_scale, p2, eps)


def awq_block_norm(y, residual: torch.Tensor, w_pre=None, w_post=None, gate=None, res_scale: float = 1.0,
                   eps: float = 1e-6, out=None, stream=None) -> dict:
    """{"residual": r', "h": h} with r' = residual + res_scale * gate * norm(y) * w_post (without w_post: y
    itself; y None: r' = residual, not returned) and h = norm(r') * w_pre (only with w_pre). gate is a
    vector [d] or a matrix [n_tokens, d]. `out` may hold "residual" (also residual itself) and "h"."""
    if stream is not None:
        return _on_stream(stream, awq_block_norm, y, residual, w_pre, w_post, gate, res_scale, eps, out)
    lib = _load()
    t, n, d, dev, args = _norm_args(y, residual, w_pre, w_post, gate, res_scale, eps)
    out = out or {}
    res, po, ldo, ph, ldh = {}, None, 0, None, 0
    if y is not None:
        res["residual"], po, ldo = _output(out.get("residual"), "residual (output)", (n, d), t, dev)
    if w_pre is not None:
        res["h"], ph, ldh = _output(out.get("h"), "h", (n, d), t, dev)
    _call(lib.awq_block_norm, dev, *args, po, ldo, ph, ldh)
    return res


def awq_block_norm_backward_workspace_bytes(n_tokens: int, d: int) -> int:
    return _load().awq_block_norm_backward_workspace_bytes(n_tokens, d)


def awq_block_norm_backward(y, residual: torch.Tensor, d_res_out, d_h, w_pre=None, w_post=None, gate=None,
                            res_scale: float = 1.0, eps: float = 1e-6, workspace=None, out=None, wanted=None,
                            stream=None) -> dict:
    """The gradients of awq_block_norm from those of its outputs (d_res_out may be None, d_h is None without
    w_pre): "d_residual", and where the input is there "d_y", "d_w_pre", "d_w_post" and "d_gate" (float32
    for vectors). `wanted` limits them to the names it holds."""
    if stream is not None:
        return _on_stream(stream, awq_block_norm_backward, y, residual, d_res_out, d_h, w_pre, w_post, gate, res_scale,
                          eps, workspace, out, wanted)
    lib = _load()
    t, n, d, dev, args = _norm_args(y, residual, w_pre, w_post, gate, res_scale, eps)
    pr, ldr = (None, 0) if d_res_out is None else _matrix(d_res_out, "d_res_out", (n, d), t, dev)
    ph, ldh = (None, 0) if d_h is None else _matrix(d_h, "d_h", (n, d), t, dev)
    there = {"d_residual": residual, "d_y": y, "d_w_pre": w_pre, "d_w_post": w_post, "d_gate": gate}
    if wanted is not None:
        for name in wanted:
            if there.get(name) is None:
                raise ValueError(f"there is no {name} to compute")
    out = out or {}
    res, ptr = {}, {}
    for name, of in there.items():
        ptr[name] = (None, 0)
        if of is None or (wanted is not None and name not in wanted):
            continue
        if of.dim() == 2:
            res[name], *ptr[name] = _output(out.get(name), name, (n, d), t, dev)
        else:
            o = out.get(name)
            o = torch.empty(d, dtype=torch.float32, device=dev) if o is None else o
            res[name], ptr[name] = o, (_vector(o, name, torch.float32, d, dev), 0)
    workspace = _workspace(lib.awq_block_norm_backward_workspace_bytes(n, d), dev, workspace)
    _call(lib.awq_block_norm_backward, dev, *args, pr, ldr, ph, ldh, *ptr["d_y"], *ptr["d_residual"],
          ptr["d_w_post"][0], ptr["d_w_pre"][0], *ptr["d_gate"], workspace.data_ptr(),
          workspace.numel() * workspace.element_size())
    return res


# ------------------------------------------------------------------ tokens by expert and back


def _slots(t, name: str, dtype, n=None, k=None, device=None) -> int:
    """Pointer of a contiguous [n_tokens, top_k] tensor."""
    if isinstance(t, torch.Tensor) and t.is_cuda and (t.dim() == 2 if n is None else t.shape == (n, k)) \
            and (t.dtype in dtype if type(dtype) is tuple else t.dtype == dtype) \
            and (device is None or t.device == device) and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or (n is not None and tuple(t.shape) != (n, k)):
        raise ValueError(f"{name} must be a [n_tokens, top_k] matrix" + ("" if n is None else f", here [{n}, {k}]"))
    return _buf(t, name, dtype, t.numel(), device)


def awq_moe_sort_workspace_bytes(n_tokens: int, top_k: int, n_experts: int) -> int:
    return _load().awq_moe_sort_workspace_bytes(n_tokens, top_k, n_experts)


def awq_moe_sort(expert_ids: torch.Tensor, n_experts: int, workspace=None, out=None, stream=None) -> dict:
    """The stable order by expert of the slots of expert_ids ([n_tokens, top_k] int32 or int64; ids outside
    [0, n_experts) are dropped): int32 "offsets" [n_experts + 1], "order" [slots], "position" [n_tokens, top_k]."""
    if stream is not None:
        return _on_stream(stream, awq_moe_sort, expert_ids, n_experts, workspace, out)
    lib = _load()
    pi = _slots(expert_ids, "expert_ids", (torch.int32, torch.int64))
    n, k = expert_ids.shape
    dev = expert_ids.device
    out = out or {}
    res, ptrs = {}, []
    for name, shape in (("offsets", (n_experts + 1,)), ("order", (n * k,)), ("position", (n, k))):
        o = out.get(name)
        if o is None:
            o = torch.empty(*(shape if n_experts > 0 else (0,)), dtype=torch.int32, device=dev)
            ptrs.append(o.data_ptr())
        elif not isinstance(o, torch.Tensor) or o.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}")
        else:
            ptrs.append(_buf(o, name, torch.int32, 0, dev))
        res[name] = o
    nb, pw = lib.awq_moe_sort_workspace_bytes(n, k, n_experts), None
    if nb:
        workspace = _workspace(nb, dev, workspace)
        pw, nb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(lib.awq_moe_sort, dev, pi, expert_ids.element_size(), n, k, n_experts, *ptrs, pw, nb)
    return res


def _scale_args(in_scales, expert_ids, n, k, d, dev):
    """(expert_ids pointer, id bytes, in_scales pointer, n_experts)."""
    if in_scales is None:
        return None, 4, None, 0
    if expert_ids is None:
        raise ValueError("in_scales needs expert_ids")
    pi = _slots(expert_ids, "expert_ids", (torch.int32, torch.int64), n, k, dev)
    if not isinstance(in_scales, torch.Tensor) or in_scales.dim() != 2 or in_scales.shape[1] != d:
        raise ValueError(f"in_scales must be a [n_experts, {d}] matrix")
    return pi, expert_ids.element_size(), _buf(in_scales, "in_scales", torch.float32, in_scales.numel(), dev), \
        in_scales.shape[0]


def awq_moe_gather(x: torch.Tensor, position: torch.Tensor, expert_ids=None, in_scales=None, n_rows=None, out=None,
                   stream=None) -> torch.Tensor:
    """rows [n_rows, d] with rows[position[t, j]] = x[t] * in_scales[expert_ids[t, j]] (in_scales: float32
    [n_experts, d], usually 1 / the scales searched for each expert). n_rows is the slots' count unless given,
    or that of `out`; rows that no slot names are left as they were."""
    if stream is not None:
        return _on_stream(stream, awq_moe_gather, x, position, expert_ids, in_scales, n_rows, out)
    lib = _load()
    dt = _data_dtype(x, "x")
    px, ldx = _matrix(x, "x")
    n, d = x.shape
    dev = x.device
    k = position.shape[1] if isinstance(position, torch.Tensor) and position.dim() == 2 else 0
    pp = _slots(position, "position", torch.int32, n, k, dev)
    ids = _scale_args(in_scales, expert_ids, n, k, d, dev)
    if n_rows is None:
        n_rows = n * k if out is None else out.shape[0]
    rows, po, ldo = _output(out, "rows", (n_rows, d), x.dtype, dev)
    _call(lib.awq_moe_gather, dev, px, ldx, dt, n, d, pp, k, *ids, po, ldo, n_rows)
    return rows


def awq_moe_gather_backward(d_rows: torch.Tensor, position: torch.Tensor, expert_ids=None, in_scales=None, out=None,
                            stream=None) -> torch.Tensor:
    """d_x [n_tokens, d]: the sum of each token's rows of d_rows, times in_scales."""
    if stream is not None:
        return _on_stream(stream, awq_moe_gather_backward, d_rows, position, expert_ids, in_scales, out)
    lib = _load()
    dt = _data_dtype(d_rows, "d_rows")
    pr, ldr = _matrix(d_rows, "d_rows")
    n_rows, d = d_rows.shape
    dev = d_rows.device
    pp = _slots(position, "position", torch.int32, device=dev)
    n, k = position.shape
    ids = _scale_args(in_scales, expert_ids, n, k, d, dev)
    d_x, po, ldo = _output(out, "d_x", (n, d), d_rows.dtype, dev)
    _call(lib.awq_moe_gather_backward, dev, pr, ldr, dt, n_rows, d, pp, n, k, *ids, po, ldo)
    return d_x


def awq_moe_combine(rows: torch.Tensor, position: torch.Tensor, weights: torch.Tensor, out=None,
                    stream=None) -> torch.Tensor:
    """out [n_tokens, d]: the sum over j of weights[t, j] (float32) * rows[position[t, j]]."""
    if stream is not None:
        return _on_stream(stream, awq_moe_combine, rows, position, weights, out)
    lib = _load()
    dt = _data_dtype(rows, "rows")
    pr, ldr = _matrix(rows, "rows")
    n_rows, d = rows.shape
    dev = rows.device
    pp = _slots(position, "position", torch.int32, device=dev)
    n, k = position.shape
    pw = _slots(weights, "weights", torch.float32, n, k, dev)
    res, po, ldo = _output(out, "out", (n, d), rows.dtype, dev)
    _call(lib.awq_moe_combine, dev, pr, ldr, dt, n_rows, d, pp, pw, n, k, po, ldo)
    return res


def awq_moe_combine_backward(d_out: torch.Tensor, rows: torch.Tensor, position: torch.Tensor, weights: torch.Tensor,
                             out=None, stream=None) -> dict:
    """{"d_rows": weights[t, j] * d_out[t] at position[t, j], "d_weights": <d_out[t], rows[position[t, j]]>}.
    `out` may hold either (d_rows also rows itself, where no two slots name the same row); rows of d_rows that no slot
    names are left as they were."""
    if stream is not None:
        return _on_stream(stream, awq_moe_combine_backward, d_out, rows, position, weights, out)
    lib = _load()
    dt = _data_dtype(rows, "rows")
    pr, ldr = _matrix(rows, "rows")
    n_rows, d = rows.shape
    dev = rows.device
    pp = _slots(position, "position", torch.int32, device=dev)
    n, k = position.shape
    pw = _slots(weights, "weights", torch.float32, n, k, dev)
    pd, ldd = _matrix(d_out, "d_out", (n, d), rows.dtype, dev)
    out = out or {}
    d_rows, po, ldo = _output(out.get("d_rows"), "d_rows", (n_rows, d), rows.dtype, dev)
    d_weights = out.get("d_weights")
    if d_weights is None:
        d_weights = torch.empty(n, k, dtype=torch.float32, device=dev)
    pdw = _slots(d_weights, "d_weights", torch.float32, n, k, dev)
    _call(lib.awq_moe_combine_backward, dev, pd, ldd, pr, ldr, dt, n_rows, d, pp, pw, n, k, po, ldo, pdw)
    return {"d_rows": d_rows, "d_weights": d_weights}


# ------------------------------------------------------------------ the experts' products


def _export_args(x, codes, steps_f16, zeros_u4, offsets):
    """(pointers of the export and the offsets, n_experts, d_in, d_out) of stacked experts."""
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("the rows must be torch.bfloat16 or torch.float16")
    dev = x.device
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
        raise ValueError("codes must be a [n_experts, d_out, d_in / 2] tensor")
    e, d_out, half = codes.shape
    d_in = 2 * half
    g = d_in // binding.GROUP_SIZE
    for t, name, shape in ((steps_f16, "steps_f16", (e, d_out, g)), (zeros_u4, "zeros_u4", (e, d_out, (g + 1) // 2))):
        if not isinstance(t, torch.Tensor) or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be a {list(shape)} tensor")
    ptrs = (_buf(codes, "codes", torch.uint8, codes.numel(), dev),
            _buf(steps_f16, "steps_f16", _HALF_BITS, steps_f16.numel(), dev),
            _buf(zeros_u4, "zeros_u4", torch.uint8, zeros_u4.numel(), dev),
            _vector(offsets, "offsets", torch.int32, e + 1, dev))
    return ptrs, e, d_in, d_out


def _grouped_output(x, y, name, shape, out_dtype):
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    if out_dtype not in (torch.float32, x.dtype):
        raise TypeError(f"{name} must be torch.float32 or the rows' dtype")
    y, p, ld = _output(y, name, shape, out_dtype, x.device)
    return y, p, ld, _DTYPES[out_dtype]


def awq_w4a16_grouped_gemm(x: torch.Tensor, codes: torch.Tensor, steps_f16: torch.Tensor, zeros_u4: torch.Tensor,
                           offsets: torch.Tensor, act=None, out_dtype=None, y=None, stream=None) -> torch.Tensor:
    """Row i of x ([n_rows, d_in], sorted by expert: offsets from awq_moe_sort) times its expert's dequantized
    weights (the exports of the experts stacked: codes [n_experts, d_out, d_in/2], steps_f16
    [n_experts, d_out, d_in/128], zeros_u4 [n_experts, d_out, ceil(d_in/256)]). act "silu" or "relu": the
    weights stack a gate and an up matrix, and y = act(x gate^T) * (x up^T). y is x's dtype or float32; rows from
    offsets[n_experts] on are left as they were."""
    if stream is not None:
        return _on_stream(stream, awq_w4a16_grouped_gemm, x, codes, steps_f16, zeros_u4, offsets, act, out_dtype, y)
    lib = _load()
    if act not in _MODES:
        raise ValueError(f"act {act!r} is none of None, 'silu', 'relu'")
    ptrs, e, d_in, d_out = _export_args(x, codes, steps_f16, zeros_u4, offsets)
    px, ldx = _matrix(x, "x", (x.shape[0], d_in) if x.dim() == 2 else None)
    n = x.shape[0]
    if act is not None and d_out % 2:
        raise ValueError(f"d_out {d_out} of a gate/up pair is odd")
    y, py, ldy, yd = _grouped_output(x, y, "y", (n, d_out if act is None else d_out // 2), out_dtype)
    _call(lib.awq_w4a16_grouped_gemm, x.device, px, ldx, _DTYPES[x.dtype], *ptrs, e, n, d_in, d_out, _MODES[act],
          py, ldy, yd)
    return y


def awq_w4a16_grouped_gemm_backward(d_y: torch.Tensor, codes: torch.Tensor, steps_f16: torch.Tensor,
                                    zeros_u4: torch.Tensor, offsets: torch.Tensor, out_dtype=None, dx=None,
                                    stream=None) -> torch.Tensor:
    """d_x [n_rows, d_in]: row i of d_y ([n_rows, d_out]) times its expert's dequantized weights, not
    transposed: the gradient of the plain product with respect to x. The kernels take rows that start at 16-byte
    boundaries: a d_y whose rows do not (a contiguous one where d_out is no multiple of 8) is copied to ones that do."""
    if stream is not None:
        return _on_stream(stream, awq_w4a16_grouped_gemm_backward, d_y, codes, steps_f16, zeros_u4, offsets, out_dtype,
                          dx)
    lib = _load()
    ptrs, e, d_in, d_out = _export_args(d_y, codes, steps_f16, zeros_u4, offsets)
    pd, ldd = _matrix(d_y, "d_y", (d_y.shape[0], d_out) if d_y.dim() == 2 else None)
    n = d_y.shape[0]
    if pd % 16 or (ldd % 8 and n > 1):
        ldd = (d_out + 7) // 8 * 8
        rows = torch.empty(n, ldd, dtype=d_y.dtype, device=d_y.device)
        rows[:, :d_out].copy_(d_y)
        pd = rows.data_ptr()
    dx, px, ldx, xd = _grouped_output(d_y, dx, "dx", (n, d_in), out_dtype)
    _call(lib.awq_w4a16_grouped_gemm_backward, d_y.device, pd, ldd, _DTYPES[d_y.dtype], *ptrs, e, n, d_in, d_out,
          px, ldx, xd)
    return dx
