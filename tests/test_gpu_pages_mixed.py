"""Paged attention calls whose streams bring different numbers of queries (B200): viewers on their
next token, in a group that reads its common pages once, beside streams of many queries."""
import pytest
import torch

from test_gpu_pages import Model, cfg

pytestmark = pytest.mark.gpu


def _session(mode, heads, dim, dtype, prefix, alone, members=8, page=64):
    """Stream 0 and its forks, one query each, then a stream of its own with `alone` queries."""
    m = Model(share=mode, **cfg(streams=members + 2, heads=heads[0], kv_heads=heads[1], head_dim=dim, dtype=dtype,
                                page_tokens=page, pages=prefix // page + 20 + 4 * members, max_queries=members + alone + 8))
    m.grow([prefix] + [0] * members + [40])
    m.fork(0, list(range(1, members)))
    m.grow([1 + 5 * b for b in range(members)] + [0, alone])
    return m, [1] * members + [0, alone]


@pytest.mark.parametrize("mode", ["auto", "always", "never"])
@pytest.mark.parametrize("alone", [16, 17, 64, 300])
@pytest.mark.parametrize("heads,dim,dtype", [((12, 12), 128, "bf16"), ((12, 12), 64, "fp16"), ((4, 2), 64, "bf16"),
                                             ((8, 8), 128, "fp16")])
def test_a_group_of_few_rows_beside_a_stream_of_many(mode, alone, heads, dim, dtype):
    m, counts = _session(mode, heads, dim, dtype, 4096, alone)
    m.attend(0, counts)
    m.attend(0, counts[:-1] + [1])                    # and all of them few


@pytest.mark.parametrize("alone", [17, 200])
def test_a_group_beside_one_that_is_left_apart(alone):
    """Two groups, of which the automatic rule shares the first only; the second has many queries."""
    m = Model(share="auto", **cfg(streams=9, heads=8, kv_heads=8, head_dim=128, page_tokens=64, pages=200, max_queries=2 * alone + 8))
    m.grow([5000, 0, 0, 0, 0, 0, 70, 0, 0])
    m.fork(0, [1, 2, 3, 4, 5])
    m.fork(6, [7])
    m.grow([1, 2, 3, 1, 1, 1, alone, alone, 0])
    m.attend(0, [1] * 6 + [alone, alone, 0])
    m.attend(0, [1] * 6 + [alone, 1, 0])


@pytest.mark.parametrize("mode", ["auto", "always"])
def test_a_replay_of_a_mixed_call(mode):
    m, counts = _session(mode, (8, 8), 128, "bf16", 5000, 40)
    n = sum(counts)
    q = m.normal(n, 8, 128)
    out = torch.zeros_like(q)
    m.c.attention(0, q, out, counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.c.attention(0, q, out, counts)
    for step in range(4):
        m.grow([3, 70, 1, 0, 64, 1, 1, 1, 5, 90])
        q.copy_(m.normal(n, 8, 128))
        graph.replay()
        m.attend(0, counts, q=q, run=lambda layer, q, o, c, s: o.copy_(out))
