"""Refusals of the token-sequence operators' C ABI and their host-side logic, no GPU
needed: every bad argument is turned down before the device is touched."""
import os

import pytest


@pytest.fixture(scope="module")
def B():
    from causal_dit_kv_b200 import binding
    if not os.path.exists(binding.LIB_PATH):
        from causal_dit_kv_b200 import build
        build.build()
    binding.lib()
    return binding


def _prompt(B, offsets=(0, 8), scale=0.1, q=16, k=16, v=16, out=16, **kw):
    cfg = dict(heads=4, kv_heads=2, head_dim=64, block_tokens=1, dtype=0, tokens=8, q_stride=0, k_stride=0, v_stride=0,
               out_stride=0)
    cfg.update(kw)
    B.sdv2_prompt_attention(B.sdv2_prompt_config(**cfg), q, k, v, out, list(offsets), scale, stream=0)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=96), "SHAPE"), (dict(heads=3), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(kv_heads=0), "SHAPE"),
    (dict(heads=2048, kv_heads=2048), "SHAPE"), (dict(block_tokens=0), "SHAPE"), (dict(dtype=2), "SHAPE"),
    (dict(tokens=-1), "SHAPE"), (dict(tokens=1 << 30), "SHAPE"), (dict(scale=0.0), "ARG"),
    (dict(scale=float("nan")), "ARG"), (dict(scale=float("inf")), "ARG"), (dict(q=8), "ALIGN"), (dict(out=24), "ALIGN"),
    (dict(q=None), "ARG"), (dict(out=None), "ARG"), (dict(q_stride=255), "SHAPE"), (dict(k_stride=120), "SHAPE"),
    (dict(q_stride=260), "ALIGN"), (dict(out_stride=1 << 40), "SHAPE"), (dict(offsets=(0, 9)), "ARG"),
    (dict(offsets=(-1, 8)), "ARG"), (dict(offsets=(0, 5, 4, 8)), "ARG")])
def test_prompt_refusals(B, kw, status):
    with pytest.raises(B.SDV2Error) as e:
        _prompt(B, **kw)
    assert e.value.status == getattr(B, "SDV2_E_" + status)


def test_prompt_without_work(B):
    _prompt(B, offsets=(0,))
    _prompt(B, offsets=(3, 3, 3))
    with pytest.raises(ValueError):
        _prompt(B, offsets=())
