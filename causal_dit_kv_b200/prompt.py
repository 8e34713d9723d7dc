"""Attention over whole packed prompts: the first pass of a clip or a text.

A thin wrapper over sdv2_prompt_attention (include/sdv2.h): it checks the tensors'
shapes, types, layouts and device and names the stream.
"""
from __future__ import annotations

import math

import torch

from . import binding as B

_DTYPE = {torch.bfloat16: B.DT_BF16, torch.float16: B.DT_FP16}


def rows_3d(x, name, heads, dim, dtype, device):
    """Check x [tokens, heads, dim] on CUDA device `device` (its index), a token's heads and channels
    contiguous, no two tokens overlapping; returns (pointer, token stride, tokens)."""
    shape, stride = x.shape, x.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], got {tuple(shape)}")
    if x.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.get_device() != device:
        raise ValueError(f"{name} is on {x.device}, expected cuda:{device}")
    tokens = shape[0]
    if stride[2] != 1 or (stride[1] != dim and heads > 1):
        raise ValueError(f"{name}: a token's heads and channels must be contiguous")
    # (the stride of a single token is arbitrary; 0, as of a broadcast tensor, would be "contiguous" to the library)
    if tokens > 1 and stride[0] < heads * dim:
        raise ValueError(f"{name}: tokens must not overlap or share their memory")
    return x.data_ptr(), (stride[0] if tokens > 1 else heads * dim), tokens


def prompt_attention(q, k, v, out, offsets, block_tokens=1, softmax_scale=None, stream=None):
    """Causal attention (by blocks of ``block_tokens`` tokens) within each packed sequence.

    q, out: [tokens, heads, d]; k, v: [tokens, kv_heads, d]; bf16 or fp16, d 64 or 128; a token's
    heads contiguous, tokens at any stride that is a multiple of 8 elements; all on the current CUDA
    device.  offsets: host integers, sequence s being rows offsets[s] .. offsets[s + 1] - 1; other rows
    of ``out`` stay.
    """
    dtype, dev = q.dtype, q.get_device()
    if dtype not in _DTYPE:
        raise ValueError(f"q must be bfloat16 or float16, got {dtype}")
    if dev < 0 or dev != B.current_device():
        raise ValueError(f"q is on {q.device}, the current device is cuda:{B.current_device()}")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    _, heads, d = q.shape
    kv_heads = k.shape[1]
    qp, qs, tokens = rows_3d(q, "q", heads, d, dtype, dev)
    kp, ks, k_tokens = rows_3d(k, "k", kv_heads, d, dtype, dev)
    vp, vs, v_tokens = rows_3d(v, "v", kv_heads, d, dtype, dev)
    op, os_, out_tokens = rows_3d(out, "out", heads, d, dtype, dev)
    if k_tokens != tokens or v_tokens != tokens or out_tokens != tokens:
        raise ValueError("q, k, v and out must have the same number of tokens")
    if tokens == 0:
        if any(int(x) != 0 for x in offsets):
            raise ValueError("offsets must lie in 0..tokens")
        return
    cfg = B.sdv2_prompt_config(heads, kv_heads, d, B._int32(min(block_tokens, (1 << 31) - 1)), _DTYPE[dtype], tokens, qs, ks, vs, os_)
    B.sdv2_prompt_attention(cfg, qp, kp, vp, op, offsets, 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale,
                            stream)


def prompt_check():
    """Synchronise and return SDV2_OK, or SDV2_E_DEVICE if a prompt kernel's wait ran out."""
    return B.sdv2_prompt_check()
