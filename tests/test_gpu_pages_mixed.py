"""Paged attention calls whose streams bring different numbers of queries (B200): viewers on their
next token, in a group that reads its common pages once, beside streams of many queries."""
import random

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


def test_the_same_bits_again():
    """Calls of every combination of kernels repeat themselves exactly."""
    m, counts = _session("always", (8, 8), 128, "bf16", 5000, 40)
    for call in (counts, [1] * 8 + [0, 1], [3, 1, 1, 1, 4, 6, 1, 1, 0, 2], [0] * 8 + [0, 40]):
        q = m.normal(sum(call), 8, 128)
        first = m.attend(0, call, q=q)
        for _ in range(5):
            again = torch.empty_like(q)
            m.c.attention(0, q, again, call)
            assert torch.equal(first, again)


@pytest.mark.parametrize("seed", range(10))
def test_random_sessions(seed):
    """Extends, forks, forks of forks, frees and compactions in any order, any mix of queries."""
    r = random.Random(seed)
    heads, kv_heads = r.choice([(4, 2), (10, 2), (8, 1), (12, 12), (6, 3)])
    streams, page = r.randint(3, 10), r.choice([16, 32, 64, 128])
    m = Model(seed=seed, share=r.choice(["auto", "always", "never"]),
              **cfg(streams=streams, heads=heads, kv_heads=kv_heads, head_dim=r.choice([64, 128]), page_tokens=page,
                    dtype=r.choice(["bf16", "fp16"]), pages=12000 // page, max_queries=2000, layers=r.randint(1, 2),
                    block_tokens=r.choice([1, 1, 7, 64])))
    for _ in range(14):
        what = r.choice(["grow", "grow", "grow", "fork", "fork", "free", "compact"])
        if what == "grow":
            counts = [r.choice([0, 1, r.randint(1, 3 * page), r.randint(1, 900)]) for _ in range(streams)]
            need = sum(-(-(m.tokens(b) + x) // page) - len(m.lists[b]) for b, x in enumerate(counts))
            if need <= m.users.count(0):
                m.grow(counts)
        elif what == "fork":
            src = r.randrange(streams)
            dst = [b for b in range(streams) if b != src and m.tokens(b) == 0 and r.random() < 0.7]
            deep = r.random() < 0.15
            copied = len(m.lists[src]) - (0 if deep else m.tokens(src) // page)
            if m.tokens(src) and copied * len(dst) <= m.users.count(0):
                m.fork(src, dst, deep)
        elif what == "free":
            m.free([r.randrange(streams)])
        else:
            m.compact()
        m.check()
        most = r.choice([1, 3, 20, 200])
        counts = [min(m.tokens(b), r.choice([0, 1, 1, r.randint(1, most)])) for b in range(streams)]
        if sum(counts):
            m.attend(r.randrange(m.kw["layers"]), counts)
