"""Softmax attention beside the KDA layers: Python binding of the kda_qk_norm_rope, kda_kv_append,
kda_kv_read and kda_attn_decode entry points of libkda_b200.so (include/kda.h has the contract).

    qk_norm_rope(q, k, ...) -> (q_out, k_out)        per-head RMS norm, then the position rotation
    qk_norm_rope_bwd(d_q_out, d_k_out, q, k, ...)    its gradients
    kv_append(k, v, k_cache, v_cache, slots, ...)    the same, keys and values into a paged cache
    kv_read(k_cache, v_cache, page_table, ...)       cached rows read back
    attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, ...)   attention over the cache

Argument marshalling only, in lib/attn_binding.*.so (csrc/attn_binding.cpp: a call of a few microseconds on
the GPU would spend several times that in Python).  Caches are [num_pages, num_kv_heads, page_size,
D], bf16 or float8_e4m3fn with fp32 scales [num_pages, num_kv_heads, page_size]; pages may lie apart (any
stride of the first dimension).  Every call runs on ``stream`` (the current stream when None) of the
tensors' device; what a call allocates belongs to that stream.  Wrong tensors raise ValueError, what the
library refuses KDAError.  No call is recorded by autograd: its results have no grad_fn, also where an input
requires a gradient (for training, qk_norm_rope_bwd is the gradient to call).
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Tuple

import torch

__all__ = ["qk_norm_rope", "qk_norm_rope_bwd", "kv_append", "kv_read", "attn_decode", "attn_decode_workspace_size",
           "new_attn_decode_workspace"]

# in the order attn_binding.init takes their addresses
_FUNCTIONS = ("kda_qk_norm_rope", "kda_qk_norm_rope_bwd", "kda_qk_norm_rope_bwd_workspace_size", "kda_kv_append", "kda_kv_read",
              "kda_attn_decode", "kda_attn_decode_workspace_size")
_binding = None


def _declare(lib):
    vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.kda_qk_norm_rope.argtypes = [vp, vp, i64, i64, vp, vp, f32, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, vp, vp]
    lib.kda_qk_norm_rope_bwd.argtypes = [vp, vp, vp, vp, i64, i64, vp, vp, f32, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                         i32, i32, vp, sz, vp]
    lib.kda_qk_norm_rope_bwd_workspace_size.argtypes = []
    lib.kda_kv_append.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, f32, vp, vp, vp, vp, vp, vp, vp, vp, i64, i32, i32, i32, i32,
                                  i32, i32, i32, i32, i64, i64, vp, vp]
    lib.kda_kv_read.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, i32, i32, i32, i64, i64, vp, vp]
    lib.kda_attn_decode_workspace_size.argtypes = [i32, i32, i32, i32]
    lib.kda_attn_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, f32, f32, i32, vp, vp, i32, i32, i32, i32, i32, i32, i32, i32,
                                    i64, i64, vp, sz, vp]
    for name in _FUNCTIONS:
        getattr(lib, name).restype = sz if name.endswith("_size") else ctypes.c_int


def _load():
    """Loads the binding and gives it the library's functions.  Raises if it has not been built for this torch
    and this Python."""
    global _binding
    from . import KDAError, build, load
    lib = load()
    path = build.binding_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m kimi_delta_attention_24_b200.build`")
    spec = importlib.util.spec_from_file_location("attn_binding", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.init(KDAError, *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _FUNCTIONS))
    _binding = module
    return module


def qk_norm_rope(q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None, interleaved=False, q_out=None,
                 k_out=None, workspace=None, stream=None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """RMS norm of every head of ``q`` and ``k`` (bf16 [..., heads, D], heads contiguous, tokens any one
    stride apart), then the rotation by the tokens' ``positions`` (int32) in ``cos_sin`` (fp32
    [max_positions, rot_dim]: cosines, then sines).  A weight (fp32 [D]) of None leaves its norm out, a
    ``cos_sin`` of None the rotation; ``q`` or ``k`` may be None.  Returns (q_out, k_out), contiguous; the rows
    of a token whose position is out of range are not written (where the call allocates them, they hold
    anything).  Not recorded by autograd."""
    return (_binding or _load()).qk_norm_rope(q, k, q_weight, k_weight, eps, cos_sin, positions, interleaved, q_out, k_out,
                                                workspace, stream)


def qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight=None, k_weight=None, eps=1e-6, cos_sin=None, positions=None,
                     interleaved=False, workspace=None, stream=None):
    """Gradients of sum(d_q_out * q_out) + sum(d_k_out * k_out) of ``qk_norm_rope``: a dict of dq, dk
    (bf16, contiguous) and dq_weight, dk_weight (fp32 [D]; None where the weight is None).  ``q`` or
    ``k`` may be None, with its gradient.  A token whose position is out of range has gradients of zero."""
    return (_binding or _load()).qk_norm_rope_bwd(d_q_out, d_k_out, q, k, q_weight, k_weight, eps, cos_sin, positions,
                                                    interleaved, workspace, stream)


def kv_append(k, v, k_cache, v_cache, slots, k_scale=None, v_scale=None, q=None, q_out=None, q_weight=None, k_weight=None,
              eps=1e-6, cos_sin=None, positions=None, interleaved=False, workspace=None, stream=None) -> Optional[torch.Tensor]:
    """Norm and rotation as ``qk_norm_rope``; the keys, and ``v`` as it is, go to rows ``slots`` (int32,
    one per token, page * page_size + row; negative: the token is skipped) of the paged cache, quantised
    with a scale per row where the cache is float8_e4m3fn.  Returns q_out (None without ``q``); skipped
    tokens' rows of a given ``q_out`` stay as they were (of one that the call allocates, they hold anything)."""
    return (_binding or _load()).kv_append(k, v, k_cache, v_cache, slots, k_scale, v_scale, q, q_out, q_weight, k_weight, eps,
                                             cos_sin, positions, interleaved, workspace, stream)


def kv_read(k_cache, v_cache, page_table, cu_seqlens, k_out, v_out, k_scale=None, v_scale=None, workspace=None,
            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Rows cu_seqlens[n] .. cu_seqlens[n + 1] of ``k_out`` and ``v_out`` (bf16 [total, num_kv_heads, D])
    from tokens 0, 1, .. of sequence n in the cache (``page_table`` int32 [N, max_pages], ``cu_seqlens``
    int32 [N + 1]); rows behind the last sequence stay as they were."""
    return (_binding or _load()).kv_read(k_cache, v_cache, page_table, cu_seqlens, k_out, v_out, k_scale, v_scale, workspace,
                                           stream)


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
    return (_binding or _load()).attn_decode(q, k_cache, v_cache, page_table, seq_lens, scale, out, lse, k_scale, v_scale,
                                               softcap, window, workspace, stream)
