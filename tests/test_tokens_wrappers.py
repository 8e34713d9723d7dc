"""What the token-sequence operators' wrappers make of tensors and host numbers before the library is
called, no GPU needed."""
from array import array

import numpy as np
import pytest
import torch

from causal_dit_kv_b200.prompt import rows_3d

H, D = 3, 64


def _rows(x):
    return rows_3d(x, "x", H, D, torch.bfloat16, -1)          # (a CPU tensor's device index)


def _wide(tokens=7, width=5):
    return torch.zeros((tokens, width, D), dtype=torch.bfloat16)


@pytest.mark.parametrize("x,stride,tokens", [
    (_wide(7, H), H * D, 7), (_wide()[:, 1:4], 5 * D, 7), (_wide()[::2, 2:], 10 * D, 4), (_wide()[:0, :H], H * D, 0),
    (_wide()[:1, :H], H * D, 1), (_wide(1, H).expand(1, H, D), H * D, 1)])
def test_token_strides(x, stride, tokens):
    assert _rows(x)[1:] == (stride, tokens)


@pytest.mark.parametrize("x", [
    _wide(1, H).expand(7, H, D),                              # every token the same row: stride 0
    _wide(1, H).expand(2, H, D),
    _wide().as_strided((4, H, D), (D, D, 1)),                 # rows that overlap
    _wide().as_strided((4, H, D), (H * D - 8, D, 1))])
def test_tokens_that_share_memory_are_refused(x):
    """A token stride of 0 means contiguous to the library, which would read and write past the tensor."""
    with pytest.raises(ValueError, match="overlap"):
        _rows(x)


def _pool(monkeypatch, calls):
    """A PagedKVCache without a device, whose library calls are recorded."""
    from causal_dit_kv_b200 import PagedKVCache, binding as B
    for name in ("sdv2_pages_write", "sdv2_pages_attention"):
        monkeypatch.setattr(B, name, lambda *args: calls.append(args))
    c = PagedKVCache.__new__(PagedKVCache)
    c.handle, c.device, c.dtype, c._any, c._scale = None, -1, torch.bfloat16, 16, 0.125
    c.streams, c.heads, c.kv_heads, c.head_dim = 2, H, H, D
    return c


@pytest.mark.parametrize("make", [
    list, tuple, lambda x: np.array(x, np.int8), lambda x: np.array(x, np.int64), torch.tensor,
    lambda x: torch.tensor(x, dtype=torch.int8), lambda x: array("b", x)])
def test_counts_of_any_width_add_up(monkeypatch, make):
    """Counts whose sum does not fit their own type."""
    calls = []
    c = _pool(monkeypatch, calls)
    x = torch.zeros((200, H, D), dtype=torch.bfloat16)
    c.write(0, x, x, make([100, 100]))
    c.attention(0, x, x.clone(), make([100, 100]))
    assert list(calls[0][6]) == [100, 100] and list(calls[1][6]) == [100, 100]
    with pytest.raises(ValueError, match="199 tokens"):
        c.write(0, x[:199], x, make([100, 100]))


@pytest.mark.parametrize("name", ["streams", "layers", "heads", "kv_heads", "head_dim", "pages", "page_tokens",
                                  "stream_pages", "max_queries"])
def test_numbers_past_32_bits_are_refused(name):
    """Not taken modulo 2^32."""
    from causal_dit_kv_b200 import binding as B
    good = dict(streams=4, layers=2, heads=8, kv_heads=2, head_dim=64, pages=100, page_tokens=64, stream_pages=50,
                max_queries=16)
    assert B.sdv2_pages_bytes(B.make_pages_config(**good)) > 0
    with pytest.raises(OverflowError):
        B.make_pages_config(**{**good, name: good[name] + (1 << 32)})
    with pytest.raises(OverflowError):
        B.make_pages_config(**good, block_tokens=1 - (1 << 32))
    assert B.make_pages_config(**good, block_tokens=1 << 40).block_tokens == (1 << 31) - 1


def test_arguments_past_32_bits_are_refused():
    from causal_dit_kv_b200 import binding as B
    for call in (lambda: B.sdv2_pages_write(None, 1 << 32, 16, 16, 0, 0, [1], 0),
                 lambda: B.sdv2_pages_attention(None, 1 << 32, 16, 16, 0, 0, [1], 1.0, 0),
                 lambda: B.sdv2_pages_fork(None, 1 << 32, [1], False, 0), lambda: B.sdv2_pages_share(None, 1 << 32),
                 lambda: B.sdv2_pages_query(None, 1 << 32)):
        with pytest.raises(OverflowError):
            call()
