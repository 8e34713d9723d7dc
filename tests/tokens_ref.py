"""Plain 64-bit implementations of the token-sequence operators, and the tolerance of a
16-bit attention output against them.  Test infrastructure only; any device."""
from __future__ import annotations

import math

import torch


def visible_keys(place: int, total: int, block: int) -> int:
    """Keys 0 .. n-1 that the token at `place` of a sequence of `total` tokens sees."""
    return min(total, (place // block + 1) * block)


def attention_rows(q, k, v, places, block, scale):
    """q [n, Hq, d] at `places` of a sequence with keys k, v [total, Hkv, d]: the output in 64 bits,
    the same product with |v| (the weight of each rounding of a probability), and the largest
    scale * sum |q_i k_i| of a row and key."""
    n, hq, d = q.shape
    total, hkv = k.shape[0], k.shape[1]
    g = hq // hkv
    q, k, v = q.double(), k.double(), v.double()
    i = torch.as_tensor(places, device=q.device).view(-1, 1)
    seen = torch.clamp((i // block + 1) * block, max=total)
    hidden = torch.arange(total, device=q.device).view(1, -1) >= seen
    out, weight = torch.empty_like(q), torch.empty_like(q)
    largest = 0.0
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        s = (q[:, h] @ kh.T * scale).masked_fill(hidden, -math.inf)
        p = torch.softmax(s, 1)
        out[:, h], weight[:, h] = p @ vh, p @ vh.abs()
        largest = max(largest, float((q[:, h].abs() @ kh.abs().T).max()) * scale)
    return out, weight, largest


def prompt_reference(q, k, v, offsets, block, scale):
    """(out, weight, largest) of attention_rows for every sequence; rows outside all are NaN."""
    out, weight = (torch.full(q.shape, math.nan, dtype=torch.float64, device=q.device) for _ in range(2))
    largest = 0.0
    for a, b in zip(offsets, offsets[1:]):
        if b > a:
            out[a:b], weight[a:b], top = attention_rows(q[a:b], k[a:b], v[a:b], range(b - a), block, scale)
            largest = max(largest, top)
    return out, weight, largest


def attention_tolerance(out, weight, largest, dtype, d, keys, v_max):
    """Elementwise bound of |kernel - out|, from the kernel's roundings alone (u: half a step of the type).

    Each probability is rounded once to 16 bits: u * weight.  The output is rounded once: u * |out|
    (and u * the error so far).  fp32: a score is a sum of d exact products, off by at most
    d 2^-24 sum |q_i k_i|, which moves its probability and the row sum by that much each; the row
    sum and the output are sums over the keys, off by at most keys 2^-24 each; the exponential
    is off by 2^-22 and its argument (below 2^7 in magnitude where the probability is not 0) by
    2^-17.  fp16 probabilities below 2^-14 and outputs below that are off by half a step of the
    subnormals, 2^-25; the row sum is at least 1.
    """
    u = torch.finfo(dtype).eps / 2
    fp32 = 2 * d * 2.0 ** -24 * largest + 2 * keys * 2.0 ** -24 + 2.0 ** -22 + 2 * 2.0 ** -17
    tol = (u + fp32) * (1 + u) * weight + u * out.abs()
    if dtype == torch.float16:
        tol = tol + keys * 2.0 ** -25 * v_max + 2.0 ** -25
    return tol


def assert_attention(got, want, tol):
    """Every element of `got` that `want` has a value for (not NaN) lies within `tol`."""
    there = ~torch.isnan(want)
    err = (got.double() - want)[there].abs()
    bad = ~(err <= tol[there])                       # (a NaN in `got` is bad)
    assert not bool(bad.any()), (int(bad.sum()), float((err / tol[there]).max()), float(err.max()))
