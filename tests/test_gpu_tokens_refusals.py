"""Tensors that the token-sequence operators turn down before any launch (B200)."""
import pytest
import torch

from test_gpu_pages import Model, cfg

pytestmark = pytest.mark.gpu


def _bad(x):
    """x's shape over memory that its tokens share, or share in part."""
    n, h, d = x.shape
    return [x[:1].expand(n, h, d), x.as_strided((n, h, d), ((h - 1) * d, d, 1))]


def test_prompt_tokens_that_share_memory():
    from causal_dit_kv_b200 import prompt_attention
    x = {name: torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda") for name in ("q", "k", "v", "out")}
    for name in x:
        for bad in _bad(x[name]):
            with pytest.raises(ValueError, match=f"{name}: .*overlap"):
                prompt_attention(**{**x, name: bad}, offsets=[0, 6])


def test_paged_tokens_that_share_memory():
    m = Model(**cfg(heads=4, kv_heads=2, max_queries=8))
    m.grow([6, 0, 9, 0])
    q, kv = m.normal(7, 4, 64), m.normal(7, 2, 64)
    counts = [3, 0, 4, 0]
    for bad in _bad(kv):
        with pytest.raises(ValueError, match="k: .*overlap"):
            m.c.write(0, bad, kv, counts)
        with pytest.raises(ValueError, match="v: .*overlap"):
            m.c.write(0, kv, bad, counts)
    for bad in _bad(q):
        with pytest.raises(ValueError, match="q: .*overlap"):
            m.c.attention(0, bad, torch.empty_like(q), counts)
        with pytest.raises(ValueError, match="out: .*overlap"):
            m.c.attention(0, q, bad, counts)
    m.check()
