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
    (dict(offsets=(-1, 8)), "ARG"), (dict(offsets=(0, (1 << 25) + 1), tokens=1 << 26), "SHAPE"), (dict(offsets=(0, 5, 4, 8)), "ARG")])
def test_prompt_refusals(B, kw, status):
    with pytest.raises(B.SDV2Error) as e:
        _prompt(B, **kw)
    assert e.value.status == getattr(B, "SDV2_E_" + status)


def test_prompt_without_work(B):
    _prompt(B, offsets=(0,))
    _prompt(B, offsets=(3, 3, 3))
    with pytest.raises(ValueError):
        _prompt(B, offsets=())


def _pages(B, **kw):
    cfg = dict(streams=4, layers=2, heads=8, kv_heads=2, head_dim=64, pages=100, page_tokens=64, stream_pages=50,
               max_queries=16, block_tokens=1)
    cfg.update(kw)
    return B.make_pages_config(**cfg)


@pytest.mark.parametrize("kw", [
    dict(streams=0), dict(streams=257), dict(layers=0), dict(heads=7), dict(heads=129, kv_heads=1), dict(kv_heads=0),
    dict(heads=2048, kv_heads=2048), dict(head_dim=32), dict(page_tokens=48), dict(pages=0),
    dict(pages=1 << 30, kv_heads=2), dict(stream_pages=0), dict(stream_pages=1 << 24), dict(stream_pages=(1 << 19) + 1),
    dict(max_queries=0),
    dict(max_queries=1 << 28), dict(block_tokens=0), dict(dtype=3)])
def test_pages_config_refusals(B, kw):
    with pytest.raises(B.SDV2Error):
        B.sdv2_pages_bytes(_pages(B, **kw))
    with pytest.raises(B.SDV2Error):
        B.sdv2_pages_layout_of(_pages(B, **kw))


def test_pages_layout(B):
    cfg = _pages(B, layers=30, kv_heads=8, head_dim=128, page_tokens=32)
    lay = B.sdv2_pages_layout_of(cfg)
    assert lay.layer_stride == 100 * 8 * 32 * 128 * 2
    offs = [lay.k_offset, lay.v_offset, lay.table_offset, lay.length_offset, lay.version_offset, lay.status_offset,
            lay.scratch_offset]
    assert offs == sorted(offs) and all(o % 256 == 0 for o in offs)
    assert lay.v_offset >= lay.k_offset + 30 * lay.layer_stride and lay.table_offset >= lay.v_offset + 30 * lay.layer_stride
    assert lay.scratch_offset + lay.scratch_bytes == lay.total_bytes == B.sdv2_pages_bytes(cfg)


def test_pages_null_handles(B):
    lib = B.lib()
    one = B.int32_array([0]).buffer_info()[0]
    assert lib.sdv2_pages_extend(None, one, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_write(None, 0, 16, 16, 0, 0, one, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_attention(None, 0, 16, 16, 0, 0, one, 1.0, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_fork(None, 0, one, 1, 0, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_free(None, one, 1, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_compact(None, None, None) == B.SDV2_E_ARG
    assert lib.sdv2_pages_share(None, 1) == B.SDV2_E_ARG
    assert lib.sdv2_pages_check(None) == B.SDV2_E_ARG and lib.sdv2_pages_used(None) == -1
    assert lib.sdv2_pages_destroy(None) == B.SDV2_OK
    with pytest.raises(B.SDV2Error) as e:
        B.sdv2_pages_create(_pages(B), 256 * 1000 + 16, 1 << 40)       # unaligned buffer
    assert e.value.status == B.SDV2_E_ALIGN
    with pytest.raises(B.SDV2Error) as e:
        B.sdv2_pages_create(_pages(B), 256 * 1000, 1000)               # too small
    assert e.value.status == B.SDV2_E_ALIGN


@pytest.mark.parametrize("code", ["b", "h", "i", "q", "I"])
def test_host_integers_of_any_width(B, code):
    from array import array
    got = B.int32_array(array(code, [3, 0, 5]))
    assert got.typecode == "i" and got.itemsize == 4 and list(got) == [3, 0, 5]


def test_host_integers_refused(B):
    with pytest.raises(OverflowError):
        B.int32_array([1 << 31])
    with pytest.raises(TypeError):
        B.int32_array([1.5])
