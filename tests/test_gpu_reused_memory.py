"""Handles on memory that work of another stream still writes (B200): torch gives a freed block back to
the stream that it was freed on, with that stream's work on it pending."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _on_a_busy_block(nbytes, make):
    """make() on a side stream whose allocator reuses a block that a pending kernel fills with ones."""
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        block = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        block.fill_(0)                                # (the kernel is loaded before the wait)
        ptr = block.data_ptr()
        torch.cuda._sleep(200_000_000)                # a tenth of a second
        block.fill_(0x3f)
        del block
        made = make()
        assert made.buffer.data_ptr() == ptr
    torch.cuda.synchronize()
    return made


def test_paged_cache():
    from causal_dit_kv_b200 import PagedKVCache, binding as B
    kw = dict(streams=4, layers=2, heads=4, kv_heads=2, head_dim=64, pages=50)
    n = B.sdv2_pages_bytes(B.make_pages_config(**kw))
    c = _on_a_busy_block(n, lambda: PagedKVCache(**kw))
    assert bool((c.page_table() == -1).all()) and bool((c.lengths() == 0).all())
    assert not bool(c.k_pages().any()) and not bool(c.v_pages().any()) and c.check() == 0
    c.extend([5, 0, 0, 0])
    assert c.lengths().tolist() == [5, 0, 0, 0] and c.page_table()[0, :2].tolist() == [0, -1]


def test_ring_cache():
    from causal_dit_kv_b200 import KVCache, binding as B
    kw = dict(batch=2, layers=2, heads=2, head_dim=64, frame_h=4, frame_w=4, chunk_frames=1, sink_frames=1, window_frames=2)
    n = B.sdv2_cache_bytes(B.make_cache_config(**kw))
    c = _on_a_busy_block(n, lambda: KVCache(**kw))
    assert not bool(c.k_cache(1).any()) and c.check() == 0


def test_motion_state():
    from causal_dit_kv_b200 import MotionState, binding as B
    kw = dict(batch=2, chunk_frames=1, channels=16, height=8, width=8)
    n = B.sdv2_motion_bytes(B.make_motion_config(**kw))
    m = _on_a_busy_block(n, lambda: MotionState(**kw))
    fresh = MotionState(**kw)
    assert torch.equal(m.buffer, fresh.buffer) and m.check() == 0
