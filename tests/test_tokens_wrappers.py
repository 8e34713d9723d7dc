"""What the token-sequence operators' wrappers make of tensors and host numbers before the library is
called, no GPU needed."""
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
