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


class _Call:
    """The device, stream and library of one call, and its errors."""

    __slots__ = ("lib", "dev", "index", "stream", "side")

    def __init__(self, t: torch.Tensor, stream):
        from . import load
        self.lib = load()
        if not t.is_cuda:
            raise ValueError("the tensors must be CUDA tensors")
        self.dev = t.device
        self.index = self.dev.index
        current = torch.cuda.current_stream(self.dev).cuda_stream
        self.stream = current if stream is None else stream
        self.side = self.stream != current

    def empty(self, shape, dtype):
        """An allocation that belongs to the call's stream."""
        if not self.side:
            return torch.empty(shape, dtype=dtype, device=self.dev)
        with torch.cuda.stream(torch.cuda.ExternalStream(self.stream, device=self.dev)):
            return torch.empty(shape, dtype=dtype, device=self.dev)

    def run(self, name, *args):
        fn = getattr(self.lib, name)
        if torch.cuda.current_device() == self.index:
            st = fn(*args, self.stream)
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, self.stream)
        if st != 0:
            from . import KDAError
            raise KDAError(st, name)

    def check(self, t, name, dtype, shape=None):
        """A contiguous tensor of the given type (and shape); its address, None for None."""
        if t is None:
            return None
        if t.device != self.dev:
            raise ValueError(f"{name} must be on {self.dev}")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        return t.data_ptr()

    def rows(self, t, name):
        """A bf16 tensor [..., heads, D] whose heads are contiguous and whose tokens lie one stride
        apart: (address, token stride, tokens)."""
        if t.device != self.dev:
            raise ValueError(f"{name} must be on {self.dev}")
        if t.dtype != _BF16:
            raise ValueError(f"{name} must be {_BF16}, got {t.dtype}")
        shape, stride = t.shape, t.stride()
        if len(shape) < 3:
            raise ValueError(f"{name} must be [..., heads, D]")
        heads, d = shape[-2], shape[-1]
        tokens = 1
        for n in shape[:-2]:
            tokens *= n
        if tokens * heads * d == 0:
            return t.data_ptr(), heads * d, tokens
        if (d > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != d):
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        token = None  # the step between tokens; size-one dimensions have none
        span = 1
        for n, s in zip(reversed(shape[:-2]), reversed(stride[:-2])):
            if n == 1:
                continue
            if token is None:
                token = s
            elif s != token * span:
                raise ValueError(f"{name}: the tokens must lie one stride apart")
            span *= n
        return t.data_ptr(), heads * d if token is None else token, tokens

    def cache(self, k_cache, v_cache, k_scale, v_scale):
        """The addresses of a paged cache and its scales, and its sizes."""
        quant = k_scale is not None
        if quant != (v_scale is not None):
            raise ValueError("k_scale and v_scale go together")
        dtype = _E4M3 if quant else _BF16
        for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
            if t.device != self.dev:
                raise ValueError(f"{name} must be on {self.dev}")
            if t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype} {'with' if quant else 'without'} scales, got {t.dtype}")
            if t.dim() != 4 or not (t.numel() == 0 or t[0].is_contiguous()):
                raise ValueError(f"{name} must be [num_pages, num_kv_heads, page_size, D] with contiguous pages")
        if v_cache.shape != k_cache.shape:
            raise ValueError("k_cache and v_cache must have the same shape")
        pages, heads, page, d = k_cache.shape
        ks = self.check(k_scale, "k_scale", _F32, (pages, heads, page))
        vs = self.check(v_scale, "v_scale", _F32, (pages, heads, page))
        step = [t.stride(0) if pages > 1 else heads * page * d for t in (k_cache, v_cache)]
        return k_cache.data_ptr(), v_cache.data_ptr(), ks, vs, pages, heads, page, d, step[0], step[1]

    def workspace(self, t):
        if t is None:
            return None
        at = self.check(t, "workspace", torch.uint8)
        if t.numel() < 256:
            raise ValueError("workspace must have at least 256 bytes")
        return at

    def rotation(self, cos_sin, positions, tokens):
        """The addresses of the rotation's table and positions, rot_dim and the table's length."""
        if cos_sin is None:
            return None, None, 0, 0
        if cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_positions, rot_dim]")
        table = self.check(cos_sin, "cos_sin", _F32)
        if positions is None:
            raise ValueError("positions are needed with cos_sin")
        at = self.check(positions, "positions", _I32)
        if positions.numel() != tokens:
            raise ValueError(f"positions must have {tokens} entries, got {positions.numel()}")
        return table, at, cos_sin.shape[1], cos_sin.shape[0]


def _qk(c: _Call, q, k):
    """Queries and keys of the same tokens, either of which may be None."""
    if q is not None:
        qp, qs, tokens = c.rows(q, "q")
        hq, d = q.shape[-2:]
    if k is not None:
        kp, ks, kt = c.rows(k, "k")
        hk, kd = k.shape[-2:]
        if q is None:
            return None, 0, 0, kp, ks, hk, kt, kd
        if kt != tokens or kd != d:
            raise ValueError("q and k must have the same tokens and head size")
        return qp, qs, hq, kp, ks, hk, tokens, d
    return qp, qs, hq, None, 0, 0, tokens, d


def qk_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None, interleaved=False, q_out=None,
                 k_out=None, workspace=None, stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """RMS norm of every head of ``q`` and ``k`` (bf16 [..., heads, D], heads contiguous, tokens any one
    stride apart), then the rotation by the tokens' ``positions`` (int32) in ``cos_sin`` (fp32
    [max_positions, rot_dim]: cosines, then sines).  A weight (fp32 [D]) of None leaves its norm out, a
    ``cos_sin`` of None the rotation; ``q`` or ``k`` may be None.  Returns (q_out, k_out), contiguous."""
    c = _Call(k if q is None else q, stream)
    qp, qs, hq, kp, ks, hk, tokens, d = _qk(c, q, k)
    table, pos, rot, most = c.rotation(cos_sin, positions, tokens)
    wq = c.check(q_weight, "q_weight", _F32, (d,))
    wk = c.check(k_weight, "k_weight", _F32, (d,))
    if q is not None and q_out is None:
        q_out = c.empty(q.shape, _BF16)
    if k is not None and k_out is None:
        k_out = c.empty(k.shape, _BF16)
    qo = c.check(q_out, "q_out", _BF16, q.shape) if q is not None else None
    ko = c.check(k_out, "k_out", _BF16, k.shape) if k is not None else None
    c.run("kda_qk_norm_rope", qp, kp, qs, ks, wq, wk, eps, table, pos, qo, ko, tokens, hq, hk, d, rot, most,
          1 if interleaved else 0, c.workspace(workspace))
    return q_out if q is not None else None, k_out if k is not None else None


def qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None,
                     interleaved=False, workspace=None, stream=None):
    """Gradients of sum(d_q_out * q_out) + sum(d_k_out * k_out) of ``qk_norm_rope``: a dict of dq, dk
    (bf16, contiguous) and dq_weight, dk_weight (fp32 [D]; None where the weight is None).  ``q`` or
    ``k`` may be None, with its gradient."""
    c = _Call(k if q is None else q, stream)
    qp, qs, hq, kp, ks, hk, tokens, d = _qk(c, q, k)
    table, pos, rot, most = c.rotation(cos_sin, positions, tokens)
    if (d_q_out is None) != (q is None) or (d_k_out is None) != (k is None):
        raise ValueError("a gradient goes with each of q and k")
    gq = c.check(d_q_out, "d_q_out", _BF16, None if q is None else q.shape)
    gk = c.check(d_k_out, "d_k_out", _BF16, None if k is None else k.shape)
    wq = c.check(q_weight, "q_weight", _F32, (d,))
    wk = c.check(k_weight, "k_weight", _F32, (d,))
    size = c.lib.kda_qk_norm_rope_bwd_workspace_size()
    if workspace is None:
        workspace = c.empty((size,), torch.uint8)
    ws = c.check(workspace, "workspace", torch.uint8)
    r = {"dq": None if q is None else c.empty(q.shape, _BF16), "dk": None if k is None else c.empty(k.shape, _BF16),
         "dq_weight": None if q_weight is None else c.empty((d,), _F32),
         "dk_weight": None if k_weight is None else c.empty((d,), _F32)}
    at = [None if t is None else t.data_ptr() for t in r.values()]
    c.run("kda_qk_norm_rope_bwd", gq, gk, qp, kp, qs, ks, wq, wk, eps, table, pos, *at, tokens, hq, hk, d, rot, most,
          1 if interleaved else 0, ws, workspace.numel())
    return r


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, q=None, q_out=None, q_weight=None, k_weight=None,
              eps=1e-6, cos_sin=None, positions=None, interleaved=False, workspace=None, stream=None) -> Optional[torch.Tensor]:
    """Norm and rotation as ``qk_norm_rope``; the keys, and ``v`` as it is, go to rows ``slots`` (int32,
    one per token, page * page_size + row; negative: the token is skipped) of the paged cache, quantised
    with a scale per row where the cache is float8_e4m3fn.  Returns q_out (None without ``q``); skipped
    tokens' rows of a given ``q_out`` stay as they were."""
    c = _Call(k, stream)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = c.cache(k_cache, v_cache, k_scale, v_scale)
    qp, qs, hq, kp, ks, hk, tokens, kd = _qk(c, q, k)
    vp, vs, vt = c.rows(v, "v")
    if hk != heads or kd != d or vt != tokens or v.shape[-2] != heads or v.shape[-1] != d:
        raise ValueError("k and v must have the cache's heads and head size, and the same tokens")
    sl = c.check(slots, "slots", _I32)
    if slots.numel() != tokens:
        raise ValueError(f"slots must have {tokens} entries, got {slots.numel()}")
    table, pos, rot, most = c.rotation(cos_sin, positions, tokens)
    wq = c.check(q_weight, "q_weight", _F32, (d,))
    wk = c.check(k_weight, "k_weight", _F32, (d,))
    qo = None
    if q is not None:
        if q_out is None:
            q_out = c.empty(q.shape, _BF16)
        qo = c.check(q_out, "q_out", _BF16, q.shape)
    c.run("kda_kv_append", qp, kp, vp, qs, ks, vs, wq, wk, eps, table, pos, qo, kc, vc, ksc, vsc, sl, tokens, hq, heads, d, rot,
          most, 1 if interleaved else 0, pages, page, kstep, vstep, c.workspace(workspace))
    return q_out if q is not None else None


def kv_read(k_cache, v_cache, page_table, cu_seqlens, k_out, v_out, k_scale=None, v_scale=None, workspace=None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows cu_seqlens[n] .. cu_seqlens[n + 1] of ``k_out`` and ``v_out`` (bf16 [total, num_kv_heads, D])
    from tokens 0, 1, .. of sequence n in the cache (``page_table`` int32 [N, max_pages], ``cu_seqlens``
    int32 [N + 1]); rows behind the last sequence stay as they were."""
    c = _Call(k_cache, stream)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = c.cache(k_cache, v_cache, k_scale, v_scale)
    if page_table.dim() != 2 or cu_seqlens.numel() != page_table.shape[0] + 1:
        raise ValueError("page_table must be [N, max_pages] and cu_seqlens [N + 1]")
    n, wide = page_table.shape
    pt = c.check(page_table, "page_table", _I32)
    cu = c.check(cu_seqlens, "cu_seqlens", _I32)
    total = k_out.shape[0]
    ko = c.check(k_out, "k_out", _BF16, (total, heads, d))
    vo = c.check(v_out, "v_out", _BF16, (total, heads, d))
    c.run("kda_kv_read", kc, vc, ksc, vsc, pt, cu, ko, vo, n, total, heads, d, pages, page, wide, kstep, vstep,
          c.workspace(workspace))
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
    c = _Call(q, stream)
    kc, vc, ksc, vsc, pages, heads, page, d, kstep, vstep = c.cache(k_cache, v_cache, k_scale, v_scale)
    shape = q.shape
    if len(shape) == 3:
        b, hq, qd = shape
        new = 1
    elif len(shape) == 4:
        b, new, hq, qd = shape
    else:
        raise ValueError("q must be [B, T, Hq, D] or [B, Hq, D]")
    qp = c.check(q, "q", _BF16)
    if qd != d:
        raise ValueError("q must have the cache's head size")
    if page_table.dim() != 2 or page_table.shape[0] != b:
        raise ValueError("page_table must be [B, max_pages]")
    pt = c.check(page_table, "page_table", _I32)
    sl = c.check(seq_lens, "seq_lens", _I32, (b,))
    if out is None:
        out = c.empty(shape, _BF16)
    op = c.check(out, "out", _BF16, shape)
    lp = c.check(lse, "lse", _F32, shape[:-1])
    if workspace is None:
        workspace = c.empty((c.lib.kda_attn_decode_workspace_size(new, hq, heads, d),), torch.uint8)
    ws = c.check(workspace, "workspace", torch.uint8)
    c.run("kda_attn_decode", qp, kc, vc, ksc, vsc, pt, sl, scale, softcap, window, op, lp, b, new, hq, heads, d, pages, page,
          page_table.shape[1], kstep, vstep, ws, workspace.numel())
    return out
