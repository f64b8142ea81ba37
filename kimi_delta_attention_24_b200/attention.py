"""Softmax attention beside the KDA layers: Python binding of the kda_qk_norm_rope, kda_kv_append,
kda_kv_read and kda_attn_decode entry points of libkda_b200.so (include/kda.h has the contract).

    qk_norm_rope(q, k, ...) -> (q_out, k_out)        per-head RMS norm, then the position rotation
    qk_norm_rope_bwd(d_q_out, d_k_out, q, k, ...)    its gradients
    kv_append(k, v, k_cache, v_cache, slots, ...)    the same, keys and values into a paged cache
    kv_read(k_cache, v_cache, page_table, ...)       cached rows read back
    attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, ...)   attention over the cache

Argument marshalling only.  Caches are [num_pages, num_kv_heads, page_size, D], bf16 or
float8_e4m3fn with fp32 scales [num_pages, num_kv_heads, page_size]; pages may lie apart (any stride of
the first dimension).  Every call runs on ``stream`` (the current stream when None) of the tensors'
device; what a call allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

__all__ = ["qk_norm_rope", "qk_norm_rope_bwd", "kv_append", "kv_read", "attn_decode", "attn_decode_workspace_size",
           "new_attn_decode_workspace"]

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_E4M3 = torch.float8_e4m3fn

_FUNCTIONS = ("kda_qk_norm_rope", "kda_qk_norm_rope_bwd", "kda_kv_append", "kda_kv_read", "kda_attn_decode")


def _declare(lib):
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.kda_qk_norm_rope.argtypes = [vp, vp, i64, i64, vp, vp, f32, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.kda_qk_norm_rope_bwd.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, f32, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                         i32, i32, vp, sz, vp]
    lib.kda_qk_norm_rope_bwd_workspace_size.argtypes = []
    lib.kda_qk_norm_rope_bwd_workspace_size.restype = sz
    lib.kda_kv_append.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                  i32, i32, i32, i32, i64, i64, vp, vp]
    lib.kda_kv_read.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, i64, i64, vp, vp]
    lib.kda_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.kda_attn_decode_workspace_size.restype = sz
    lib.kda_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, f32, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                    i64, i64, vp, sz, vp]
    for name in _FUNCTIONS:
        getattr(lib, name).restype = ctypes.c_int


# A call of a few microseconds on the GPU costs more on the host, so the checks below are flat and
# read each property of a tensor once.
_raw_stream = torch._C._cuda_getCurrentRawStream
_fns = None


def _functions():
    """The library's functions, looked up once."""
    global _fns
    from . import load
    lib = load()
    _fns = {name: getattr(lib, name) for name in _FUNCTIONS}
    _fns["bwd_size"] = lib.kda_qk_norm_rope_bwd_workspace_size
    _fns["decode_size"] = lib.kda_attn_decode_workspace_size
    return _fns


def _device(t):
    index = t.get_device()
    if index < 0:
        raise ValueError("the tensors must be CUDA tensors")
    return index


def _empty(like, shape, dtype, index, stream):
    """An allocation that belongs to the call's stream."""
    if stream is None or stream == _raw_stream(index):
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)):
        return like.new_empty(shape, dtype=dtype)


def _empty_like(t, index, stream):
    if stream is None or stream == _raw_stream(index):
        return torch.empty_like(t, memory_format=torch.contiguous_format)
    return _empty(t, t.shape, t.dtype, index, stream)


def _run(name, index, stream, *args):
    fn = (_fns or _functions())[name]
    if stream is None:
        stream = _raw_stream(index)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            st = fn(*args, stream)
    if st != 0:
        from . import KDAError
        raise KDAError(st, name)


def _at(t, name, dtype, index):
    """The address of a contiguous tensor of the given type on the call's device."""
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _shaped(t, name, dtype, index, shape):
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return _at(t, name, dtype, index)


def _rows(t, name, index):
    """A bf16 tensor [..., heads, D] whose heads are contiguous and whose tokens lie one stride apart:
    (address, token stride, tokens, heads, D)."""
    if t.dtype is not _BF16:
        raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        tokens, heads, d = shape
        if tokens > 1 and heads > 1 and stride[2] == 1 and stride[1] == d:
            return t.data_ptr(), stride[0], tokens, heads, d
    elif len(shape) < 3:
        raise ValueError(f"{name} must be [..., heads, D]")
    heads, d = shape[-2], shape[-1]
    tokens = 1
    for n in shape[:-2]:
        tokens *= n
    if tokens * heads * d == 0:
        return t.data_ptr(), heads * d, tokens, heads, d
    if (d > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    token, span = None, 1  # the step between tokens; dimensions of size one have none
    for n, s in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if n == 1:
            continue
        if token is None:
            token = s
        elif s != token * span:
            raise ValueError(f"{name}: the tokens must lie one stride apart")
        span *= n
    return t.data_ptr(), heads * d if token is None else token, tokens, heads, d


def _cache(k_cache, v_cache, k_scale, v_scale, index):
    """The addresses of a paged cache and its scales, and its sizes: (k, v, k scales, v scales, pages,
    heads, page size, D, page strides)."""
    if (k_scale is None) != (v_scale is None):
        raise ValueError("k_scale and v_scale go together")
    dtype = _BF16 if k_scale is None else _E4M3
    shape = k_cache.shape
    if len(shape) != 4 or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must be [num_pages, num_kv_heads, page_size, D], both alike")
    pages, heads, page, d = shape
    steps = []
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dtype is not dtype:
            raise ValueError(f"{name} must be {dtype} {'without' if k_scale is None else 'with'} scales, got {t.dtype}")
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}")
        step = t.stride()
        if not t.is_contiguous() and (step[3] != 1 or (page > 1 and step[2] != d) or (heads > 1 and step[1] != page * d)):
            raise ValueError(f"the pages of {name} must be contiguous")
        steps.append(step[0] if pages > 1 else heads * page * d)
    if k_scale is None:
        return k_cache.data_ptr(), v_cache.data_ptr(), None, None, pages, heads, page, d, *steps
    lines = (pages, heads, page)
    return (k_cache.data_ptr(), v_cache.data_ptr(), _shaped(k_scale, "k_scale", _F32, index, lines),
            _shaped(v_scale, "v_scale", _F32, index, lines), pages, heads, page, d, *steps)


def _status(workspace, index):
    """The address of an optional workspace (its status word)."""
    if workspace is None:
        return None
    if workspace.numel() < 256:
        raise ValueError("workspace must have at least 256 bytes")
    return _at(workspace, "workspace", torch.uint8, index)


def _rotation(cos_sin, positions, tokens, index):
    """The addresses of the rotation's table and positions, rot_dim and the table's length."""
    if cos_sin is None:
        return None, None, 0, 0
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [max_positions, rot_dim]")
    if positions is None:
        raise ValueError("positions are needed with cos_sin")
    if positions.numel() != tokens:
        raise ValueError(f"positions must have {tokens} entries, got {positions.numel()}")
    most, rot = cos_sin.shape
    return _at(cos_sin, "cos_sin", _F32, index), _at(positions, "positions", _I32, index), rot, most


def _qk(q, k, index):
    """Queries and keys of the same tokens, either of which may be None: their addresses, strides and
    heads, then tokens and D."""
    if q is None:
        kp, ks, tokens, hk, d = _rows(k, "k", index)
        return None, 0, 0, kp, ks, hk, tokens, d
    qp, qs, tokens, hq, d = _rows(q, "q", index)
    if k is None:
        return qp, qs, hq, None, 0, 0, tokens, d
    kp, ks, kt, hk, kd = _rows(k, "k", index)
    if kt != tokens or kd != d:
        raise ValueError("q and k must have the same tokens and head size")
    return qp, qs, hq, kp, ks, hk, tokens, d


def qk_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None, interleaved=False, q_out=None,
                 k_out=None, workspace=None, stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """RMS norm of every head of ``q`` and ``k`` (bf16 [..., heads, D], heads contiguous, tokens any one
    stride apart), then the rotation by the tokens' ``positions`` (int32) in ``cos_sin`` (fp32
    [max_positions, rot_dim]: cosines, then sines).  A weight (fp32 [D]) of None leaves its norm out, a
    ``cos_sin`` of None the rotation; ``q`` or ``k`` may be None.  Returns (q_out, k_out), contiguous."""
    index = _device(k if q is None else q)
    qp, qs, hq, kp, ks, hk, tokens, d = _qk(q, k, index)
    table, pos, rot, most = _rotation(cos_sin, positions, tokens, index)
    wq = _shaped(q_weight, "q_weight", _F32, index, (d,))
    wk = _shaped(k_weight, "k_weight", _F32, index, (d,))
    qo = ko = None
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = _empty_like(q, index, stream)
        qo = q_out.data_ptr()
    else:
        qo = _shaped(q_out, "q_out", _BF16, index, q.shape)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = _empty_like(k, index, stream)
        ko = k_out.data_ptr()
    else:
        ko = _shaped(k_out, "k_out", _BF16, index, k.shape)
    _run("kda_qk_norm_rope", index, stream, qp, kp, qs, ks, wq, wk, eps, table, pos, qo, ko, tokens, hq, hk, d, rot, most,
         1 if interleaved else 0, _status(workspace, index))
    return q_out, k_out


def qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None,
                     interleaved=False, workspace=None, stream=None):
    """Gradients of sum(d_q_out * q_out) + sum(d_k_out * k_out) of ``qk_norm_rope``: a dict of dq, dk
    (bf16, contiguous) and dq_weight, dk_weight (fp32 [D]; None where the weight is None).  ``q`` or
    ``k`` may be None, with its gradient."""
    index = _device(k if q is None else q)
    qp, qs, hq, kp, ks, hk, tokens, d = _qk(q, k, index)
    table, pos, rot, most = _rotation(cos_sin, positions, tokens, index)
    if (d_q_out is None) != (q is None) or (d_k_out is None) != (k is None):
        raise ValueError("a gradient goes with each of q and k")
    gq = None if q is None else _shaped(d_q_out, "d_q_out", _BF16, index, q.shape)
    gk = None if k is None else _shaped(d_k_out, "d_k_out", _BF16, index, k.shape)
    wq = _shaped(q_weight, "q_weight", _F32, index, (d,))
    wk = _shaped(k_weight, "k_weight", _F32, index, (d,))
    if workspace is None:
        workspace = _empty(k if q is None else q, ((_fns or _functions())["bwd_size"](),), torch.uint8, index, stream)
    ws = _at(workspace, "workspace", torch.uint8, index)
    dq = None if q is None else _empty_like(q, index, stream)
    dk = None if k is None else _empty_like(k, index, stream)
    dwq = None if q_weight is None else _empty_like(q_weight, index, stream)
    dwk = None if k_weight is None else _empty_like(k_weight, index, stream)
    _run("kda_qk_norm_rope_bwd", index, stream, gq, gk, qp, kp, qs, ks, wq, wk, eps, table, pos,
         None if dq is None else dq.data_ptr(), None if dk is None else dk.data_ptr(), None if dwq is None else dwq.data_ptr(),
         None if dwk is None else dwk.data_ptr(), tokens, hq, hk, d, rot, most, 1 if interleaved else 0, ws, workspace.numel())
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, q=None, q_out=None, q_weight=None, k_weight=None,
              eps=1e-6, cos_sin=None, positions=None, interleaved=False, workspace=None, stream=None) -> Optional[torch.Tensor]:
    """Norm and rotation as ``qk_norm_rope``; the keys, and ``v`` as it is, go to rows ``slots`` (int32,
    one per token, page * page_size + row; negative: the token is skipped) of the paged cache, quantised
    with a scale per row where the cache is float8_e4m3fn.  Returns q_out (None without ``q``); skipped
    tokens' rows of a given ``q_out`` stay as they were."""
    index = _device(k)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = _cache(k_cache, v_cache, k_scale, v_scale, index)
    qp, qs, hq, kp, ks, hk, tokens, kd = _qk(q, k, index)
    vp, vs, vt, vh, vd = _rows(v, "v", index)
    if hk != heads or kd != d or vt != tokens or vh != heads or vd != d:
        raise ValueError("k and v must have the cache's heads and head size, and the same tokens")
    if slots.numel() != tokens:
        raise ValueError(f"slots must have {tokens} entries, got {slots.numel()}")
    sl = _at(slots, "slots", _I32, index)
    table, pos, rot, most = _rotation(cos_sin, positions, tokens, index)
    wq = _shaped(q_weight, "q_weight", _F32, index, (d,))
    wk = _shaped(k_weight, "k_weight", _F32, index, (d,))
    qo = None
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = _empty_like(q, index, stream)
        qo = q_out.data_ptr()
    else:
        qo = _shaped(q_out, "q_out", _BF16, index, q.shape)
    _run("kda_kv_append", index, stream, qp, kp, vp, qs, ks, vs, wq, wk, eps, table, pos, qo, kc, vc, ksc, vsc, sl, tokens, hq,
         heads, d, rot, most, 1 if interleaved else 0, pages, page, kstep, vstep, _status(workspace, index))
    return q_out


def kv_read(k_cache, v_cache, page_table, cu_seqlens, k_out, v_out, k_scale=None, v_scale=None, workspace=None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows cu_seqlens[n] .. cu_seqlens[n + 1] of ``k_out`` and ``v_out`` (bf16 [total, num_kv_heads, D])
    from tokens 0, 1, .. of sequence n in the cache (``page_table`` int32 [N, max_pages], ``cu_seqlens``
    int32 [N + 1]); rows behind the last sequence stay as they were."""
    index = _device(k_cache)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = _cache(k_cache, v_cache, k_scale, v_scale, index)
    if page_table.dim() != 2 or cu_seqlens.numel() != page_table.shape[0] + 1:
        raise ValueError("page_table must be [N, max_pages] and cu_seqlens [N + 1]")
    n, wide = page_table.shape
    shape = k_out.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != d:
        raise ValueError("k_out must be [total, num_kv_heads, D] of the cache")
    _run("kda_kv_read", index, stream, kc, vc, ksc, vsc, _at(page_table, "page_table", _I32, index),
         _at(cu_seqlens, "cu_seqlens", _I32, index), _at(k_out, "k_out", _BF16, index), _shaped(v_out, "v_out", _BF16, index, shape),
         n, shape[0], heads, d, pages, page, wide, kstep, vstep, _status(workspace, index))
    return k_out, v_out


def attn_decode_workspace_size(new_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace ``attn_decode`` needs (independent of the batch and the lengths)."""
    from . import load
    return int(load().kda_attn_decode_workspace_size(int(new_tokens), int(num_q_heads), int(num_kv_heads), int(head_dim)))


def new_attn_decode_workspace(new_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """A workspace for ``attn_decode``, its 256-byte header (the status word) zeroed."""
    ws = torch.empty(attn_decode_workspace_size(new_tokens, num_q_heads, num_kv_heads, head_dim), dtype=torch.uint8, device=device)
    ws[:256].zero_()
    return ws


def attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, out=None, lse=None, k_scale=None, v_scale=None, softcap=0.0,
                window=0, workspace=None, stream=None) -> torch.Tensor:
    """Attention of each sequence's last T tokens (``q`` bf16 [B, T, Hq, D], or [B, Hq, D] for one) over
    its ``seq_lens`` (int32 [B]) cached tokens, the new ones included, through ``page_table`` (int32
    [B, max_pages]).  ``softcap`` > 0 caps the scores, ``window`` > 0 limits each query to that many keys,
    its own the last.  ``lse`` (fp32, q's shape without D) receives the log of the sums.  Returns ``out``."""
    index = _device(q)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = _cache(k_cache, v_cache, k_scale, v_scale, index)
    shape = q.shape
    if len(shape) == 4:
        b, new, hq, qd = shape
    elif len(shape) == 3:
        b, hq, qd = shape
        new = 1
    else:
        raise ValueError("q must be [B, T, Hq, D] or [B, Hq, D]")
    if qd != d:
        raise ValueError("q must have the cache's head size")
    if page_table.dim() != 2 or page_table.shape[0] != b:
        raise ValueError("page_table must be [B, max_pages]")
    qp = _at(q, "q", _BF16, index)
    pt = _at(page_table, "page_table", _I32, index)
    sl = _shaped(seq_lens, "seq_lens", _I32, index, (b,))
    if out is None:
        out = _empty_like(q, index, stream)
        op = out.data_ptr()
    else:
        op = _shaped(out, "out", _BF16, index, shape)
    lp = _shaped(lse, "lse", _F32, index, shape[:-1])
    if workspace is None:
        workspace = _empty(q, ((_fns or _functions())["decode_size"](new, hq, heads, d),), torch.uint8, index, stream)
    ws = _at(workspace, "workspace", torch.uint8, index)
    _run("kda_attn_decode", index, stream, qp, kc, vc, ksc, vsc, pt, sl, scale, softcap, window, op, lp, b, new, hq, heads, d,
         pages, page, page_table.shape[1], kstep, vstep, ws, workspace.numel())
    return out
