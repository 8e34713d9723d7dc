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
    """Check x [tokens, heads, dim], heads and channels contiguous; returns (pointer, token stride)."""
    if x.dim() != 3 or (heads is not None and x.shape[1] != heads) or (dim is not None and x.shape[2] != dim):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, "
                         f"{'head_dim' if dim is None else dim}], got {tuple(x.shape)}")
    if x.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {x.dtype}")
    if x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    st, sh, sd = x.stride()
    tokens, h, d = x.shape
    if sd != 1 or (sh != d and h > 1):
        raise ValueError(f"{name}: a token's heads and channels must be contiguous")
    # (the stride of a single token is arbitrary)
    return x.data_ptr(), (st if tokens > 1 else h * d)


def current_device(x, name):
    """x's device, which must be the current CUDA device (the library launches there)."""
    if not x.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if x.device.index != torch.cuda.current_device():
        raise ValueError(f"{name} is on {x.device}, the current device is {torch.cuda.current_device()}")
    return x.device


def prompt_attention(q, k, v, out, offsets, block_tokens=1, softmax_scale=None, stream=None):
    """Causal attention (by blocks of ``block_tokens`` tokens) within each packed sequence.

    q, out: [tokens, heads, d]; k, v: [tokens, kv_heads, d]; bf16 or fp16, d 64 or 128; a token's
    heads contiguous, tokens at any stride that is a multiple of 8 elements.  offsets: host
    integers, sequence s being rows offsets[s] .. offsets[s + 1] - 1; other rows of ``out`` stay.
    """
    dev = current_device(q, "q")
    if q.dtype not in _DTYPE:
        raise ValueError(f"q must be bfloat16 or float16, got {q.dtype}")
    qp, qs = rows_3d(q, "q", None, None, q.dtype, dev)
    tokens, heads, d = q.shape
    kp, ks = rows_3d(k, "k", None, d, q.dtype, dev)
    kv_heads = k.shape[1]
    vp, vs = rows_3d(v, "v", kv_heads, d, q.dtype, dev)
    op, os_ = rows_3d(out, "out", heads, d, q.dtype, dev)
    if k.shape[0] != tokens or v.shape[0] != tokens or out.shape[0] != tokens:
        raise ValueError("q, k, v and out must have the same number of tokens")
    if tokens == 0:
        if any(int(x) != 0 for x in offsets):
            raise ValueError("offsets must lie in 0..tokens")
        return
    cfg = B.sdv2_prompt_config(heads, kv_heads, d, min(int(block_tokens), (1 << 31) - 1), _DTYPE[q.dtype], tokens, qs,
                               ks, vs, os_)
    scale = 1.0 / math.sqrt(d) if softmax_scale is None else softmax_scale
    B.sdv2_prompt_attention(cfg, qp, kp, vp, op, offsets, scale, stream)


def prompt_check():
    """Synchronise and return SDV2_OK, or SDV2_E_DEVICE if a prompt kernel's wait ran out."""
    return B.sdv2_prompt_check()
