"""The paged cache (sdv2_pages_*) against plain forms (B200): page lists and contents bit
for bit against a host model, the attention within the derived tolerance of the 64-bit form;
shared prefixes, grouped heads, every page size, blocks, dirty pages, captured calls, and a
session from prompt to compaction."""
import math

import pytest
import torch

import tokens_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


class Model:
    """The streams' tokens as plain tensors, page lists by the documented rule, beside the cache."""

    def __init__(self, seed=1, dirty=True, share="always", **kw):
        from causal_dit_kv_b200 import PagedKVCache
        self.kw = kw
        self.c = PagedKVCache(**kw)
        self.c.share(share)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype = DT[kw.get("dtype", "bf16")]
        if dirty:                                     # what pages hold before they are written
            self.c.k_pages().fill_(math.nan)
            self.c.v_pages().fill_(math.inf)
        shape = (0, kw["kv_heads"], kw["head_dim"])
        self.k, self.v = ([[torch.zeros(shape, dtype=self.dtype, device="cuda") for _ in range(kw["layers"])]
                           for _ in range(kw["streams"])] for _ in range(2))
        self.users = [0] * kw["pages"]
        self.lists = [[] for _ in range(kw["streams"])]

    def normal(self, *shape):
        return torch.randn(shape, generator=self.gen, device="cuda").to(self.dtype)

    def take(self, n):
        got = [p for p, u in enumerate(self.users) if u == 0][:n]
        for p in got:
            self.users[p] = 1
        return got

    def tokens(self, b):
        return self.k[b][0].shape[0]

    def grow(self, counts):
        """extend, then write every layer from a fused projection's output."""
        self.c.extend(counts)
        hkv, n, pt = self.kw["kv_heads"], sum(counts), self.c.page_tokens
        for b, x in enumerate(counts):
            self.lists[b] += self.take(-(-(self.tokens(b) + x) // pt) - len(self.lists[b]))
        for layer in range(self.kw["layers"]):
            kv = self.normal(n, 2 * hkv, self.kw["head_dim"])
            self.c.write(layer, kv[:, :hkv], kv[:, hkv:], counts)
            at = 0
            for b, x in enumerate(counts):
                self.k[b][layer] = torch.cat([self.k[b][layer], kv[at:at + x, :hkv]])
                self.v[b][layer] = torch.cat([self.v[b][layer], kv[at:at + x, hkv:]])
                at += x

    def fork(self, src, dst, deep=False):
        self.c.fork(src, dst, deep)
        full = 0 if deep else self.tokens(src) // self.c.page_tokens
        for b in dst:
            new = self.take(len(self.lists[src]) - full)
            for p in self.lists[src][:full]:
                self.users[p] += 1
            self.lists[b] = self.lists[src][:full] + new
            self.k[b], self.v[b] = list(self.k[src]), list(self.v[src])

    def free(self, streams):
        self.c.free(streams)
        for b in streams:
            for p in self.lists[b]:
                self.users[p] -= 1
            self.lists[b] = []
            self.k[b], self.v[b] = [x[:0] for x in self.k[b]], [x[:0] for x in self.v[b]]

    def compact(self):
        used = sum(u > 0 for u in self.users)
        src = [p for p in range(used, len(self.users)) if self.users[p]]
        to = dict(zip(src, [p for p in range(used) if not self.users[p]]))
        for p, q in to.items():
            self.users[q], self.users[p] = self.users[p], 0
        self.lists = [[to.get(p, p) for p in pages] for pages in self.lists]
        assert self.c.compact() == used

    def check(self):
        """Tables, lengths and every token's keys and values, bit for bit."""
        table, lengths = self.c.page_table().tolist(), self.c.lengths().tolist()
        assert self.c.used() == sum(u > 0 for u in self.users)
        for b, pages in enumerate(self.lists):
            n = self.tokens(b)
            assert lengths[b] == n and self.c.query(b)[:2] == (n, pages)
            assert table[b] == pages + [-1] * (self.c.stream_pages - len(pages))
            for layer in range(self.kw["layers"]):
                if n == 0:
                    continue
                for pool, want in ((self.c.k_pages(layer), self.k[b][layer]), (self.c.v_pages(layer), self.v[b][layer])):
                    got = pool[pages].permute(0, 2, 1, 3).reshape(-1, *want.shape[1:])[:n]
                    assert torch.equal(got.view(torch.int16), want.contiguous().view(torch.int16)), (b, layer)
        assert self.c.check() == 0

    def attend(self, layer, counts, gain=1.0, scale=None, q=None, run=None):
        """One attention call, checked; returns its output."""
        n, hq, d = sum(counts), self.kw["heads"], self.kw["head_dim"]
        if q is None:
            q = self.normal(n, hq, d) * gain
        out = torch.full((n + 3, hq, d), 7.0, dtype=self.dtype, device="cuda")
        (run or self.c.attention)(layer, q, out[:n], counts, scale)
        assert bool((out[n:] == 7).all())
        at = 0
        for b, x in enumerate(counts):
            if x:
                total = self.tokens(b)
                want, weight, largest = R.attention_rows(q[at:at + x], self.k[b][layer], self.v[b][layer],
                                                         range(total - x, total), self.kw.get("block_tokens", 1),
                                                         d ** -0.5 if scale is None else scale)
                tol = R.attention_tolerance(want, weight, largest, self.dtype, d, total, 6.0)
                R.assert_attention(out[at:at + x], want, tol)
            at += x
        assert self.c.check() == 0
        return out[:n]


def cfg(**kw):
    base = dict(streams=4, layers=1, heads=4, kv_heads=2, head_dim=64, pages=64, page_tokens=16)
    base.update(kw)
    return base


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (128, "bf16")])
def test_tables_and_contents(page, dim, dtype):
    """Extends, writes, forks (shared and deep), frees and compactions, bit for bit."""
    m = Model(**cfg(streams=6, layers=3, heads=6, kv_heads=3, head_dim=dim, page_tokens=page, dtype=dtype, pages=40))
    m.grow([5, 0, page, 2 * page + 1, 0, 0])
    m.check()
    m.grow([page - 5, 1, 0, page, 0, 0])
    m.fork(3, [4, 5])
    m.check()
    m.grow([1, 0, 0, 1, 2, page])
    m.check()
    m.free([0, 3])
    m.check()
    m.compact()
    m.check()
    m.fork(5, [0, 3], deep=True)
    m.grow([1] * 6)
    m.check()
    m.free([4, 1])
    m.compact()
    m.compact()
    m.grow([0, 3, 0, 0, 2 * page, 0])
    m.check()
    m.free(list(range(6)))
    m.compact()
    m.check()
    assert m.c.used() == 0


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 700])
@pytest.mark.parametrize("heads,dim,page,dtype", [((1, 1), 128, 64, "bf16"), ((12, 12), 64, 16, "fp16"),
                                                  ((10, 2), 128, 32, "fp16"), ((128, 1), 64, 128, "bf16")])
def test_one_token(length, heads, dim, page, dtype):
    m = Model(**cfg(streams=2, heads=heads[0], kv_heads=heads[1], head_dim=dim, page_tokens=page, dtype=dtype))
    m.grow([length, 0])
    m.attend(0, [1, 0])


@pytest.mark.parametrize("new", [1, 3, 60, 200])
@pytest.mark.parametrize("block", [1, 7, 64, 1 << 31])
def test_several_tokens_and_blocks(new, block):
    """More query rows than a tile holds, rows that see none of a tile's keys, blocks."""
    m = Model(**cfg(streams=3, heads=6, kv_heads=2, head_dim=128, page_tokens=32, block_tokens=block, max_queries=600))
    m.grow([new, 300 + new, 77 + new])
    m.attend(0, [new, new, new])
    m.attend(0, [new, 0, 1])


@pytest.mark.parametrize("streams", [1, 3, 30, 100, 256])
def test_batches(streams):
    """Ragged streams, some of them idle; both sizes of the parameter block."""
    m = Model(**cfg(streams=streams, heads=8, kv_heads=2, head_dim=64, pages=streams * 40, max_queries=streams))
    m.grow([(37 * b) % 600 + 1 for b in range(streams)])
    m.attend(0, [0 if streams > 1 and b % 5 == 3 else 1 for b in range(streams)])


@pytest.mark.parametrize("prefix", [16, 100, 128, 1000, 4100])
@pytest.mark.parametrize("heads,dim,dtype", [((4, 4), 128, "bf16"), ((10, 2), 64, "fp16")])
@pytest.mark.parametrize("new", [1, 20])
def test_shared_prefix(prefix, heads, dim, dtype, new):
    """Twelve streams forked off one, their tails of different lengths, two idle ones and one of its
    own in between."""
    m = Model(**cfg(streams=14, heads=heads[0], kv_heads=heads[1], head_dim=dim, dtype=dtype, pages=1200,
                    max_queries=14 * new))
    m.grow([0, prefix] + [0] * 12)
    m.fork(1, [0, 2, 3, 4, 5, 6, 8, 9, 10, 11, 12])
    m.grow([new + (29 * b) % 150 for b in range(14)])
    assert m.c.query(2)[2] == prefix // 16 and m.c.query(7)[2] == 0
    counts = [new] * 14
    counts[4] = counts[11] = 0
    m.attend(0, counts)
    m.attend(0, [new if b in (7, 8) else 0 for b in range(14)])       # one of the group alone


@pytest.mark.parametrize("mode", ["auto", "never", "always"])
@pytest.mark.parametrize("prefix,new", [(64, 1), (5000, 1), (5000, 9)])
def test_sharing_modes(mode, prefix, new):
    """Read once or apart, few rows and many: right either way; with more than 16 rows in common the
    common keys are a launch of their own."""
    from causal_dit_kv_b200 import binding as B
    m = Model(share=mode, **cfg(streams=16, heads=8, kv_heads=8, head_dim=128, page_tokens=64, pages=200, max_queries=16 * new))
    m.grow([prefix] + [0] * 15)
    m.fork(0, list(range(1, 16)))
    m.grow([new] * 16)
    before = B.sdv2_launch_count()
    m.attend(0, [new] * 16)
    launches = B.sdv2_launch_count() - before
    once = mode == "always" or (mode == "auto" and prefix == 5000)
    # tiles for the common keys, rows for the streams' own, merge; otherwise rows and, if units are cut, merge
    rows_in_common = 16 * new
    assert launches == 3 if once and rows_in_common > 16 else launches <= 2


def test_two_groups_and_a_fork_of_a_fork():
    m = Model(**cfg(streams=9, heads=4, kv_heads=1, head_dim=128, pages=300, page_tokens=32))
    m.grow([200, 0, 0, 0, 333, 0, 0, 0, 50])
    m.fork(0, [2, 6])
    m.fork(4, [1, 5])
    m.grow([1, 1, 70, 0, 1, 1, 1, 0, 1])
    m.fork(2, [3])                                    # shares more with 2 than with 0 and 6
    m.fork(5, [7])
    m.grow([1] * 9)
    assert m.c.query(3)[2] == 6 and m.c.query(7)[2] == 10
    m.attend(0, [1] * 9)
    m.free([0, 6])
    m.grow([3, 1, 1, 1, 1, 1, 2, 1, 1])
    assert m.c.query(3)[2] == 8                       # 270 tokens of 2 at the fork
    m.attend(0, [1] * 9)
    m.compact()
    m.attend(0, [1] * 9)
    m.check()


@pytest.mark.parametrize("page,dim,dtype", [(16, 128, "fp16"), (128, 64, "bf16"), (64, 128, "bf16")])
def test_many_rows_over_long_and_short_keys(page, dim, dtype):
    """The tile kernel's work cut inside units, units of one tile beside units of many, several row
    tiles, and streams with different numbers of queries in one group."""
    m = Model(**cfg(streams=9, heads=9, kv_heads=3, head_dim=dim, dtype=dtype, page_tokens=page, pages=900,
                    max_queries=400))
    m.grow([3000, 0, 0, 0, 40, 0, 700, 0, 0])
    m.fork(0, [1, 2, 5])
    m.fork(6, [7])
    counts = [70, 1, 33, 0, 40, 129, 7, 18, 0]
    m.grow([70, 1, 200, 0, 7, 129, 300, 18, 0])
    m.attend(0, counts)
    m.attend(0, [17, 17, 17, 0, 17, 17, 17, 17, 0])
    m.grow([1] * 9)
    m.attend(0, [2, 5, 1, 1, 3, 1, 1, 4, 1])          # few rows of their own, many in common
    m.attend(0, [1, 1, 0, 1, 0, 1, 1, 0, 1])          # few rows both


@pytest.mark.parametrize("streams,tokens", [(1, 30000), (2, 9000)])
def test_long_keys_of_one_head(streams, tokens):
    """One or two units over all workers: hundreds of pieces to merge."""
    m = Model(**cfg(streams=streams, heads=4, kv_heads=1, head_dim=64, page_tokens=16, pages=streams * 1900,
                    max_queries=64))
    m.grow([tokens - 37 * b for b in range(streams)])
    m.attend(0, [1] * streams)
    m.attend(0, [30] * streams)


def test_edits_and_moves_of_several_launches():
    """More table entries, page copies and copies of one page than one launch's list holds."""
    m = Model(**cfg(streams=120, layers=2, heads=1, kv_heads=1, head_dim=64, page_tokens=16, pages=9000))
    m.grow([16 * 2100 if b == 0 else 0 for b in range(120)])
    m.check()
    m.fork(0, [5, 7], deep=True)                      # 2100 sources, 4200 copies
    m.check()
    m.grow([3 if b in (0, 5) else 0 for b in range(120)])
    m.fork(5, [b for b in range(120) if b not in (0, 5, 7)])   # 117 copies of one page
    m.check()
    m.free([0, 7, 11])
    m.compact()
    m.check()
    m.attend(0, [1 if b in (5, 6, 119) else 0 for b in range(120)])


def test_two_caches_on_two_streams():
    """Two handles' calls at once, each on a stream of its own."""
    ms = [Model(seed=s, **cfg(streams=4, heads=4, kv_heads=2, head_dim=128, pages=400, max_queries=80))
          for s in (1, 2)]
    for m in ms:
        m.grow([900, 0, 400, 1])
        m.fork(0, [1])
        m.grow([20, 20, 20, 20])
    qs = [m.normal(80, 4, 128) for m in ms]
    outs = [torch.empty_like(q) for q in qs]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, q, out, stream in zip(ms, qs, outs, streams):
            m.c.attention(0, q, out, [20] * 4, stream=stream)
    torch.cuda.synchronize()
    for m, q, out in zip(ms, qs, outs):
        assert torch.equal(m.attend(0, [20] * 4, q=q), out)


@pytest.mark.parametrize("dim,dtype", [(64, "fp16"), (128, "bf16")])
def test_every_row_and_no_other_is_written(dim, dtype):
    """Rows of partly filled tiles, written whole and as pieces; what lies between strided rows stays."""
    m = Model(seed=7, **cfg(streams=5, heads=6, kv_heads=2, head_dim=dim, pages=400, max_queries=400, dtype=dtype))
    m.grow([1500, 0, 0, 300, 40])
    m.fork(0, [1, 2])
    m.grow([50, 43, 1, 11, 6])
    counts = [50, 43, 1, 11, 6]
    q = m.normal(sum(counts), 6, dim)
    room = torch.full((sum(counts) + 3, 8, dim), 5.0, dtype=q.dtype, device="cuda")
    out = room[:sum(counts), :6]
    m.c.attention(0, q, out, counts)
    assert bool((room[:, 6:] == 5).all()) and bool((room[sum(counts):] == 5).all())
    assert torch.equal(out, m.attend(0, counts, q=q))


def test_graph_of_the_tile_kernel_follows_the_streams():
    """A captured attention of many rows with a common prefix, replayed after its streams have grown
    across pages and KV tiles."""
    m = Model(**cfg(streams=3, heads=4, kv_heads=2, head_dim=64, pages=300, max_queries=60, block_tokens=20))
    m.grow([500, 0, 0])
    m.fork(0, [1, 2])
    m.grow([20, 40, 160])
    counts = [20, 20, 20]
    q = m.normal(60, 4, 64)
    out = torch.zeros_like(q)
    m.c.attention(0, q, out, counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.c.attention(0, q, out, counts)
    for step in range(12):
        m.grow([20, 20, 60])
        q.copy_(m.normal(60, 4, 64))
        graph.replay()
        m.attend(0, counts, q=q, run=lambda layer, q, o, c, s: o.copy_(out))
    m.fork(0, [])                                     # nothing forked: the captured call stays good
    graph.replay()
    assert m.c.check() == 0


def test_fork_whose_queries_reach_into_the_prefix():
    """Streams with nothing, or little, of their own: the common keys end before the first query."""
    m = Model(**cfg(streams=3, heads=4, kv_heads=2, head_dim=64, pages=60, max_queries=300))
    m.grow([160, 0, 0])
    m.fork(0, [1, 2])
    m.attend(0, [1, 1, 1])
    m.attend(0, [60, 1, 3])
    m.attend(0, [100, 100, 100])


def test_climbing_scores_and_gain():
    m = Model(**cfg(streams=2, heads=2, kv_heads=2, head_dim=64, pages=200, dtype="fp16"), dirty=False)
    m.grow([1500, 700])
    for b, n in ((0, 1500), (1, 700)):
        ramp = (torch.linspace(0, 8, n, device="cuda")[:, None].expand(n, 64)).half()
        m.k[b][0][:, 0] = ramp
    kv = torch.cat([m.k[0][0], m.k[1][0]]), torch.cat([m.v[0][0], m.v[1][0]])
    m.c.write(0, kv[0], kv[1], [1500, 700])
    q = m.normal(2, 2, 64)
    q[:, 0] = 1.0
    q[:, 1] *= 8
    m.attend(0, [1, 1], q=q)
    m.attend(0, [1, 1], scale=0.31)


def test_strided_queries_and_output():
    m = Model(**cfg(streams=2, heads=4, kv_heads=2, head_dim=64))
    m.grow([40, 300])
    qkv = m.normal(2, 9, 64)
    wide = torch.full((2, 11, 64), 3.0, dtype=m.dtype, device="cuda")

    def run(layer, q, out, counts, scale):
        m.c.attention(layer, q, wide[:, 3:7], counts, scale)
        out.copy_(wide[:, 3:7])

    m.attend(0, [1, 1], q=qkv[:, 2:6], run=run)
    assert bool((wide[:, :3] == 3).all()) and bool((wide[:, 7:] == 3).all())


def test_captured_calls_follow_the_streams():
    """A captured write and attention, replayed as the streams grow (page borders and KV tiles are
    crossed), match; after a fork they touch nothing and say so."""
    from causal_dit_kv_b200 import binding as B
    m = Model(**cfg(streams=3, heads=4, kv_heads=2, head_dim=128, pages=200))
    m.grow([100, 0, 250])
    m.fork(0, [1])
    m.grow([1, 1, 1])
    counts = [1, 1, 1]
    kv, q = m.normal(3, 4, 128), m.normal(3, 4, 128)
    out = torch.zeros((3, 4, 128), dtype=m.dtype, device="cuda")
    m.c.attention(0, q, out, counts)                  # (kernels loaded before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.c.write(0, kv[:, :2], kv[:, 2:], counts)
        m.c.attention(0, q, out, counts)
    for step in range(140):
        m.c.extend(counts)
        for b in range(3):
            m.lists[b] += m.take(-(-(m.tokens(b) + 1) // 16) - len(m.lists[b]))
        kv.copy_(m.normal(3, 4, 128))
        q.copy_(m.normal(3, 4, 128))
        graph.replay()
        for b in range(3):
            m.k[b][0] = torch.cat([m.k[b][0], kv[b:b + 1, :2]])
            m.v[b][0] = torch.cat([m.v[b][0], kv[b:b + 1, 2:]])
        if step % 20 == 19 or step < 3:
            m.check()
            m.attend(0, counts, q=q, run=lambda layer, q, o, c, s: o.copy_(out))
    m.free([2])
    before = m.c.buffer.clone()
    out.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert m.c.check() == B.SDV2_E_DEVICE and "replayed" in B.sdv2_last_error()
    assert bool((out == 5).all()) and m.c.check() == 0
    k0, v0 = int(m.c.layout.k_offset), int(m.c.layout.table_offset)
    assert torch.equal(before[k0:v0], m.c.buffer[k0:v0])


def test_changes_are_refused_in_capture():
    from causal_dit_kv_b200 import binding as B
    m = Model(**cfg())
    m.grow([20, 30, 0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (lambda: m.c.extend([1, 0, 0, 0]), lambda: m.c.fork(0, [2]), lambda: m.c.free([0])):
            with pytest.raises(B.SDV2Error) as e:
                call()
            assert e.value.status == B.SDV2_E_STATE
        m.c.k_pages().mul_(1)                         # (a capture holds something)
    m.check()


def test_state_refusals():
    from causal_dit_kv_b200 import binding as B
    m = Model(**cfg(pages=8, stream_pages=5, max_queries=4))

    def refused(status, call, *args, **kw):
        with pytest.raises(B.SDV2Error) as e:
            call(*args, **kw)
        assert e.value.status == status, e.value
    m.grow([40, 0, 0, 0])
    refused(B.SDV2_E_STATE, m.c.extend, [41, 0, 0, 0])                 # 81 tokens: 6 pages
    refused(B.SDV2_E_STATE, m.c.extend, [0, 48, 48, 0])                # 6 pages, 5 free
    refused(B.SDV2_E_ARG, m.c.extend, [-1, 0, 0, 0])
    refused(B.SDV2_E_STATE, m.c.fork, 0, [1, 2], True)                 # 6 pages
    refused(B.SDV2_E_ARG, m.c.fork, 0, [0])
    refused(B.SDV2_E_ARG, m.c.fork, 0, [1, 1])
    refused(B.SDV2_E_ARG, m.c.fork, 4, [1])
    refused(B.SDV2_E_ARG, m.c.fork, 0, [4])
    refused(B.SDV2_E_ARG, m.c.free, [4])
    refused(B.SDV2_E_ARG, m.c.free, [1, 1])
    m.fork(0, [1])
    refused(B.SDV2_E_STATE, m.c.fork, 0, [1])                          # not empty
    kv = m.normal(9, 2, 64)
    refused(B.SDV2_E_STATE, m.c.write, 0, kv, kv, [9, 0, 0, 0])        # token 31 lies in a shared page
    m.c.write(0, m.k[0][0][32:], m.v[0][0][32:], [8, 0, 0, 0])
    refused(B.SDV2_E_STATE, m.c.write, 0, kv[:1], kv[:1], [0, 0, 1, 0])
    refused(B.SDV2_E_ARG, m.c.write, 1, kv[:1], kv[:1], [1, 0, 0, 0])
    q = m.normal(5, 4, 64)
    refused(B.SDV2_E_STATE, m.c.attention, 0, q[:1], q[:1].clone(), [0, 0, 0, 1])
    refused(B.SDV2_E_SHAPE, m.c.attention, 0, q, q.clone(), [3, 2, 0, 0])
    refused(B.SDV2_E_ARG, m.c.attention, 0, q[:1], q[:1].clone(), [1, 0, 0, 0], 0.0)
    for bad in (lambda: m.c.extend([1]), lambda: m.c.attention(0, q[:1].float(), q[:1], [1, 0, 0, 0]),
                lambda: m.c.attention(0, q[:2], q[:2].clone(), [1, 0, 0, 0]),
                lambda: m.c.write(0, kv[:1], kv[:1, :1], [1, 0, 0, 0]),
                lambda: m.c.write(0, kv[:1].cpu(), kv[:1], [1, 0, 0, 0])):
        with pytest.raises(ValueError):
            bad()
    m.c.attention(0, q[:0], q[:0].clone(), [0, 0, 0, 0])
    m.check()


def test_pages_past_32_bit_offsets():
    """A pool whose layer is over 4 GB: pages at its far end are written, read and copied."""
    m = Model(dirty=False, **cfg(streams=3, heads=8, kv_heads=8, head_dim=128, page_tokens=128, pages=17000, layers=1))
    filler = 16900
    m.c.extend([filler * 128, 0, 0])                  # (its contents do not matter)
    m.users[:filler] = [1] * filler
    m.grow([0, 300, 0])
    m.fork(1, [2])
    m.grow([0, 1, 200])
    m.attend(0, [0, 1, 1])
    got = m.c.k_pages(0)[m.lists[2]].permute(0, 2, 1, 3).reshape(-1, 8, 128)[:500]
    assert min(m.lists[1]) >= filler and torch.equal(got, m.k[2][0])


def test_session_from_prompt_to_compaction():
    """A run as a service makes it: prompts attended and written, viewers forked, steps with shared
    prefixes, viewers leaving, the pool compacted, and the steps after that."""
    from causal_dit_kv_b200 import prompt_attention
    L, hq, hkv, d = 2, 8, 2, 128
    m = Model(**cfg(streams=8, layers=L, heads=hq, kv_heads=hkv, head_dim=d, pages=400, block_tokens=64,
                    max_queries=8 * 64))
    lengths = [640, 0, 0, 0, 192, 0, 0, 0]
    m.c.extend(lengths)
    for b, n in enumerate(lengths):
        m.lists[b] += m.take(-(-n // 16))
    offsets = [0, 640, 832]
    for layer in range(L):
        qkv = m.normal(832, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        out = torch.empty((832, hq, d), dtype=m.dtype, device="cuda")
        prompt_attention(q, k, v, out, offsets, block_tokens=64)
        m.c.write(layer, k, v, lengths)
        want, weight, largest = R.prompt_reference(q, k, v, offsets, 64, d ** -0.5)
        R.assert_attention(out, want, R.attention_tolerance(want, weight, largest, m.dtype, d, 640, 6.0))
        # the same queries over the pages give the prompt's result too
        paged = torch.empty((192, hq, d), dtype=m.dtype, device="cuda")
        for b, (lo, hi) in ((0, (448, 640)), (4, (640, 832))):
            m.c.attention(layer, q[lo:hi], paged, [192 if x == b else 0 for x in range(8)])
            R.assert_attention(paged, want[lo:hi], R.attention_tolerance(want, weight, largest, m.dtype, d, 640, 6.0)[lo:hi])
        for b, lo, hi in ((0, 0, 640), (4, 640, 832)):
            m.k[b][layer], m.v[b][layer] = k[lo:hi], v[lo:hi]
    m.check()
    m.fork(0, [1, 2, 3])
    m.fork(4, [5])
    for step in range(3):
        m.grow([64, 64, 64, 64, 64, 64, 0, 0])
        for layer in range(L):
            m.attend(layer, [64] * 6 + [0, 0])
    m.free([0, 4])
    m.compact()
    m.fork(2, [7])
    m.grow([0, 64, 64, 64, 0, 64, 0, 64])
    for layer in range(L):
        m.attend(layer, [0, 64, 64, 64, 0, 64, 0, 64])
    m.check()
