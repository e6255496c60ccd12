"""Thin Python binding of attention over a cache of 4-bit keys and values (include/awq_attn.h, in libawq_mi355x.so).

As in `moe`, every awq_* function has the name of the C entry point it calls and only marshals arguments; outputs are
allocated unless given. Work goes to torch's current stream of the tensors' device. With `stream` (a stream of that device)
a call does what it does inside `torch.cuda.stream(stream)`: outputs and workspaces are allocated there too, and what is
passed has to be ready on that stream and to outlive its work; an output that is used on another stream has to wait for it.
No call records a graph for autograd: outputs do not require a gradient even where inputs do; awq_rope_backward is
awq_rope's gradient, for a program that calls it itself, and the cache is a constant.

A cache is two tensors, `codes` uint8 [n_pages, 2, n_kv, page_size, head_dim / 2] and `params` float16
[n_pages, 2, n_kv, n_groups, page_size, 2] (keys and values; step and offset), which kv4_cache makes. Pages are contiguous and
may be further apart than they are large (one layer's part of a tensor whose pages hold several layers).
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .binding import AwqError, _c_i64, _c_int, _c_size, _on_stream, _vp, _workspace  # noqa: F401
from .moe import _DTYPES, _call, _data_dtype

AWQ_KV4_MAX_HEAD_DIM = 256
AWQ_KV4_MIN_PAGE = 16
AWQ_KV4_MAX_PAGE = 1024
AWQ_KV4_LARGEST = 65024.0
AWQ_MAX_ROPE_DIM = 512
AWQ_ROPE_HALF = 0
AWQ_ROPE_PAIRS = 1

_c_float = ctypes.c_float
_HEADS = [_vp, _c_i64, _c_i64]
_ROPE = _HEADS + [_c_int, _c_i64, _c_i64, _c_i64, _vp, _c_i64, _c_int, _c_int, _vp, _vp, _c_i64, _c_int, _c_float] + _HEADS + [_vp]
_SIGNATURES = {
    "awq_rope": (_c_int, _ROPE),
    "awq_rope_backward": (_c_int, _ROPE),
    "awq_kv4_write": (_c_int, _HEADS + _HEADS + [_c_int, _c_i64, _c_i64, _c_i64, _vp, _c_int, _vp, _c_i64, _vp, _c_i64, _c_i64,
                                                 _c_int, _vp]),
    "awq_kv4_read": (_c_int, [_vp, _c_i64, _vp, _c_i64, _c_i64, _c_int, _c_i64, _c_i64, _vp, _c_int, _c_i64, _c_int] + _HEADS +
                     _HEADS + [_vp]),
    "awq_kv4_attention_workspace_bytes": (_c_size, [_c_i64, _c_i64, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_i64, _c_i64]),
    "awq_kv4_attention": (_c_int, _HEADS + [_c_int, _c_i64, _c_i64, _c_i64, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _c_int, _vp,
                                            _c_i64, _c_i64, _vp, _vp, _c_i64, _c_float, _c_int, _c_i64, _c_i64] + _HEADS +
                          [_c_int, _vp, _vp, _c_size, _vp]),
}
_STYLES = {"half": AWQ_ROPE_HALF, "pairs": AWQ_ROPE_PAIRS}
_INTS = (torch.int32, torch.int64)

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


def _heads(t, name: str, shape=None, dtype=None, device=None) -> tuple[int, int, int]:
    """(pointer, pitch of tokens, pitch of heads) of a device tensor [n_tokens, n_heads, head_dim]."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [n_tokens, n_heads, head_dim] tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the other operands on {device}")
    token, head, channel = t.stride()
    if channel != 1 and t.shape[2] > 1:
        raise ValueError(f"the channels of {name} must be consecutive")
    return t.data_ptr(), token, head


def _ints(t, name: str, n: int, dtypes, device) -> int:
    """Pointer of a contiguous vector of n integers."""
    if isinstance(t, torch.Tensor) and t.shape == (n,) and t.dtype in dtypes and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.shape != (n,):
        raise ValueError(f"{name} must be a vector of {n} elements")
    return binding._buf(t, name, dtypes, n, device)


# ------------------------------------------------------------------ rotary positions


def _rope(fn, names, x, positions, inv_freq, axis, style, scale, out):
    dt = _data_dtype(x, names[0])
    px = _heads(x, names[0])
    dev = x.device
    n, heads, d = x.shape
    if style not in _STYLES:
        raise ValueError(f"style {style!r} is neither 'half' nor 'pairs'")
    if isinstance(positions, torch.Tensor) and positions.dim() == 1:
        pp, ldp, axes = _ints(positions, "positions", n, _INTS, dev), n, 1
    else:
        if not isinstance(positions, torch.Tensor) or positions.dim() != 2 or positions.shape[1] != n:
            raise ValueError(f"positions must be a vector of {n} or a [n_axes, {n}] matrix")
        if positions.dtype not in _INTS:
            raise TypeError(f"positions must be torch.int32 or torch.int64, not {positions.dtype}")
        if positions.device != dev:
            raise ValueError(f"positions is on {positions.device}, the other operands on {dev}")
        if n > 1 and positions.stride(1) != 1:
            raise ValueError("positions must have unit stride along the tokens")
        axes = positions.shape[0]
        pp, ldp = positions.data_ptr(), positions.stride(0) if axes > 1 else n
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a vector")
    half = inv_freq.shape[0]
    pf = binding._buf(inv_freq, "inv_freq", torch.float32, half, dev)
    pa = None if axis is None else _ints(axis, "axis", half, (torch.int32,), dev)
    if out is None:
        out = torch.empty(n, heads, d, dtype=x.dtype, device=dev)
        po = out.data_ptr(), heads * d, d
    else:
        po = _heads(out, names[1], x.shape, x.dtype, dev)
    _call(fn, dev, *px, dt, n, heads, d, pp, ldp, positions.element_size(), axes, pf, pa, 2 * half, _STYLES[style], scale, *po)
    return out


def awq_rope(x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, axis=None, style: str = "half",
             scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """x ([n_tokens, n_heads, head_dim]) with the pairs of its first 2 * len(inv_freq) channels turned by positions[axis[i], t] *
    inv_freq[i] and multiplied by scale; the other channels are copied. positions: int32 or int64 [n_axes, n_tokens] (or
    [n_tokens]); inv_freq float32; axis int32, one per pair (None: axis 0). style "half": pair i is channels
    (i, i + len(inv_freq)); "pairs": (2 i, 2 i + 1). `out` may be x itself."""
    if stream is not None:
        return _on_stream(stream, awq_rope, x, positions, inv_freq, axis, style, scale, out)
    return _rope(_load().awq_rope, ("x", "out"), x, positions, inv_freq, axis, style, scale, out)


def awq_rope_backward(d_out: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, axis=None, style: str = "half",
                      scale: float = 1.0, out=None, stream=None) -> torch.Tensor:
    """The gradient of awq_rope with respect to x from that of its output. `out` may be d_out itself."""
    if stream is not None:
        return _on_stream(stream, awq_rope_backward, d_out, positions, inv_freq, axis, style, scale, out)
    return _rope(_load().awq_rope_backward, ("d_out", "d_x"), d_out, positions, inv_freq, axis, style, scale, out)


# ------------------------------------------------------------------ the cache


def kv4_cache(n_pages: int, n_kv: int, head_dim: int, page_size: int = 64, device="cuda"):
    """(codes, params) of an empty cache (zeros)."""
    groups = (head_dim + binding.GROUP_SIZE - 1) // binding.GROUP_SIZE
    return (torch.zeros((n_pages, 2, n_kv, page_size, head_dim // 2), dtype=torch.uint8, device=device),
            torch.zeros((n_pages, 2, n_kv, groups, page_size, 2), dtype=torch.float16, device=device))


def _packed(shape, stride) -> bool:
    """Are the elements of a page (all but the first dimension) consecutive?"""
    n = 1
    for size, step in zip(reversed(shape[1:]), reversed(stride[1:])):
        if size != 1 and step != n:
            return False
        n *= size
    return True


def _cache(codes, params, device=None):
    """((codes, page_codes, params, page_params, n_pages, page_size), n_kv, head_dim) of a cache."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != 5 or codes.shape[1] != 2:
        raise ValueError("codes must be a [n_pages, 2, n_kv, page_size, head_dim / 2] tensor")
    pages, _, kv, page, half = codes.shape
    groups = (2 * half + binding.GROUP_SIZE - 1) // binding.GROUP_SIZE
    if not isinstance(params, torch.Tensor) or params.shape != (pages, 2, kv, groups, page, 2):
        raise ValueError(f"params must be a {[pages, 2, kv, groups, page, 2]} tensor")
    if codes.dtype != torch.uint8 or params.dtype != torch.float16:
        raise TypeError(f"codes must be torch.uint8 and params torch.float16, not {codes.dtype} and {params.dtype}")
    if not codes.is_cuda or not params.is_cuda:
        raise ValueError("codes and params must be device tensors")
    device = device or codes.device
    if codes.device != device or params.device != device:
        raise ValueError(f"codes are on {codes.device} and params on {params.device}, the other operands on {device}")
    if not _packed(codes.shape, codes.stride()) or not _packed(params.shape, params.stride()):
        raise ValueError("the pages of codes and params must be contiguous")
    one = pages == 1  # (the stride of a single page means nothing)
    to_codes = 2 * kv * page * half if one else codes.stride(0)
    to_params = 4 * kv * groups * page if one else params.stride(0)
    if to_params % 2:
        raise ValueError("the pages of params must lie an even number of elements apart")
    return (codes.data_ptr(), to_codes, params.data_ptr(), to_params // 2, pages, page), kv, 2 * half


def awq_kv4_write(k: torch.Tensor, v: torch.Tensor, codes: torch.Tensor, params: torch.Tensor, slots: torch.Tensor,
                  stream=None) -> None:
    """Quantizes the keys and values of new tokens ([n_tokens, n_kv, head_dim], one type) into the cache: token i into slot
    slots[i] = page * page_size + place (int32 or int64; one outside the cache: not written)."""
    if stream is not None:
        return _on_stream(stream, awq_kv4_write, k, v, codes, params, slots)
    lib = _load()
    dt = _data_dtype(k, "k")
    dev = k.device
    cache, kv, d = _cache(codes, params, dev)
    pk = _heads(k, "k")
    n = k.shape[0]
    if k.shape != (n, kv, d):
        raise ValueError(f"k must have shape [n_tokens, {kv}, {d}], not {list(k.shape)}")
    pv = _heads(v, "v", k.shape, k.dtype, dev)
    ps = _ints(slots, "slots", n, _INTS, dev)
    pc, to_codes, pp, to_params, pages, page = cache
    _call(lib.awq_kv4_write, dev, *pk, *pv, dt, n, kv, d, ps, slots.element_size(), pc, to_codes, pp, to_params, pages, page)


def awq_kv4_read(codes: torch.Tensor, params: torch.Tensor, slots: torch.Tensor, dtype=torch.bfloat16, out=None,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(k, v), each [n_tokens, n_kv, head_dim] of dtype (or that of `out`, a pair of which either may be None: not wanted):
    the cached numbers of slots. Rows whose slot is outside the cache are left as they were (zeros in new tensors)."""
    if stream is not None:
        return _on_stream(stream, awq_kv4_read, codes, params, slots, dtype, out)
    lib = _load()
    cache, kv, d = _cache(codes, params)
    dev = codes.device
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a vector")
    n = slots.shape[0]
    ps = _ints(slots, "slots", n, _INTS, dev)
    if out is None:
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be torch.bfloat16, torch.float16 or torch.float32, not {dtype}")
        k, v = (torch.zeros(n, kv, d, dtype=dtype, device=dev) for _ in range(2))
    else:
        k, v = out
    given = [t for t in (k, v) if t is not None]
    if not given:
        raise ValueError("neither k nor v is wanted")
    dt = _data_dtype(given[0], "out")
    pk, pv = ((None, 0, 0) if t is None else _heads(t, name, (n, kv, d), given[0].dtype, dev) for t, name in ((k, "k"), (v, "v")))
    _call(lib.awq_kv4_read, dev, *cache, kv, d, ps, slots.element_size(), n, dt, *pk, *pv)
    return k, v


# ------------------------------------------------------------------ attention over the cache


def awq_kv4_attention_workspace_bytes(n_tokens: int, n_seqs: int, ragged: bool, n_heads: int, n_kv: int, head_dim: int,
                                      causal: bool, window: int, max_kv: int) -> int:
    """max_kv 0: enough for any table."""
    return _load().awq_kv4_attention_workspace_bytes(n_tokens, n_seqs, ragged, n_heads, n_kv, head_dim, causal, window, max_kv)


def awq_kv4_attention(q: torch.Tensor, codes: torch.Tensor, params: torch.Tensor, table: torch.Tensor, kv_len: torch.Tensor,
                      q_offsets=None, scale=None, causal: bool = True, window: int = 0, max_kv: int = 0, out_dtype=None, out=None,
                      lse=None, workspace=None, stream=None):
    """Attention of new tokens over the cache: out [n_tokens, n_heads, head_dim] of q's type (or float32).

    q [n_tokens, n_heads, head_dim] (bfloat16 or float16) holds the new tokens of all sequences: those of sequence s are
    q_offsets[s] .. q_offsets[s + 1] - 1 (int32 [n_seqs + 1]; None: equally many for each). Its cached tokens, the new ones
    usually the last of them, are kv_len[s] (int32) in the pages table[s] (int32 [n_seqs, width]). New token i stands at
    p = kv_len - q_len + i and sees cached tokens j <= p (causal) and j > p - window (window > 0). scale: head_dim ** -0.5
    unless given. max_kv: the largest kv_len, by which the work is split (0: what the table can hold). A token that sees
    nothing gets zeros; rows that belong to no sequence are left as they were (zeros in a new tensor). `out` may be q. One kernel takes
    all sequences of a call: single tokens and long prompts are faster in calls of their own.
    lse: a float32 [n_tokens, n_heads] tensor that receives the logarithm of each row's sum, or True for a new one; then
    (out, lse) is returned."""
    if stream is not None:
        return _on_stream(stream, awq_kv4_attention, q, codes, params, table, kv_len, q_offsets, scale, causal, window, max_kv,
                          out_dtype, out, lse, workspace)
    lib = _load()
    if not isinstance(q, torch.Tensor) or q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be a torch.bfloat16 or torch.float16 tensor")
    dev = q.device
    pq = _heads(q, "q")
    n, heads, d = q.shape
    cache, kv, cached_d = _cache(codes, params, dev)
    if d != cached_d:
        raise ValueError(f"q has heads of {d} channels, the cache of {cached_d}")
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be a [n_seqs, pages] matrix")
    seqs, width = table.shape
    if table.dtype != torch.int32:
        raise TypeError(f"table must be torch.int32, not {table.dtype}")
    if table.device != dev:
        raise ValueError(f"table is on {table.device}, the other operands on {dev}")
    if width > 1 and table.stride(1) != 1:
        raise ValueError("table must have unit stride along the pages")
    pl = _ints(kv_len, "kv_len", seqs, (torch.int32,), dev)
    po = None if q_offsets is None else _ints(q_offsets, "q_offsets", seqs + 1, (torch.int32,), dev)
    if out_dtype is None:
        out_dtype = q.dtype if out is None else out.dtype
    if out_dtype not in (q.dtype, torch.float32):
        raise TypeError(f"out must be {q.dtype} or torch.float32, not {out_dtype}")
    if out is None:
        out = (torch.empty if po is None else torch.zeros)(n, heads, d, dtype=out_dtype, device=dev)
        pout = out.data_ptr(), heads * d, d
    else:
        pout = _heads(out, "out", (n, heads, d), out_dtype, dev)
    ps = None
    if lse is not None and lse is not False:
        if lse is True:
            lse = torch.full((n, heads), -float("inf"), dtype=torch.float32, device=dev)
        if not isinstance(lse, torch.Tensor) or lse.shape != (n, heads):
            raise ValueError(f"lse must be a [{n}, {heads}] matrix")
        ps = binding._buf(lse, "lse", torch.float32, n * heads, dev)
    most = max_kv if max_kv > 0 else width * cache[5]
    nb, pw = lib.awq_kv4_attention_workspace_bytes(n, seqs, po is not None, heads, kv, d, causal, window, most), None
    if nb:
        workspace = _workspace(nb, dev, workspace)
        pw, nb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _call(lib.awq_kv4_attention, dev, *pq, _DTYPES[q.dtype], n, heads, kv, d, *cache, table.data_ptr(),
          table.stride(0) if seqs > 1 else width, width, pl, po, seqs, d ** -0.5 if scale is None else scale, causal, window,
          max_kv, *pout, _DTYPES[out_dtype], ps, pw, nb)
    return out if ps is None else (out, lse)
