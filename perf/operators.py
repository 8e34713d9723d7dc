"""Cases of the prompt and page operators: what a streaming service calls when a clip or a text prompt
comes in, when viewers branch off it, and at every step after that.

Four operators, each with its plain form in elementary torch operations:

  prompt  attention over whole packed prompts, causal by blocks of tokens, grouped heads
  paged   attention of the newest tokens of every stream over its pages; streams that were forked
          from one another read the pages they share once
  pages   forking streams, freeing them, compacting the pool
  write   new tokens' keys and values into the pages

``run`` computes the plain form, or with ``own`` makes the framework's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # prompts: a handful of short texts before a session starts (latency)
        {"name": "prompt short", "op": "prompt", "lengths": "37,1,128,200,64,90", "heads": 12, "kv_heads": 12,
         "dim": 128, "block": 1, "dtype": "bf16"},
        # prompts: ragged texts of several requests, grouped heads
        {"name": "prompt ragged grouped", "op": "prompt", "lengths": "2311,1024,517,4096,77", "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 1, "dtype": "bf16"},
        # prompts: an opening clip of eight 1024-token frames, each frame's tokens see one another, 40 heads
        {"name": "prompt clip", "op": "prompt", "lengths": "8192", "heads": 40, "kv_heads": 40, "dim": 128,
         "block": 1024, "dtype": "bf16"},
        # prompts: narrow heads in half precision, sizes off every tile
        {"name": "prompt odd fp16", "op": "prompt", "lengths": "1000,3001,511,1777", "heads": 16, "kv_heads": 2,
         "dim": 64, "block": 1, "dtype": "fp16"},
        # one viewer's next token after a short history (latency)
        {"name": "paged one stream", "op": "paged", "streams": 1, "prefix": 0, "low": 1000, "high": 1000, "new": 1,
         "heads": 12, "kv_heads": 12, "dim": 128, "page": 64, "block": 1, "dtype": "bf16", "salt": 1},
        # a batch of unrelated streams of very different lengths, one token each
        {"name": "paged batch", "op": "paged", "streams": 32, "prefix": 0, "low": 500, "high": 8000, "new": 1,
         "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "block": 1, "dtype": "bf16", "salt": 2},
        # 64 viewers branched off one long clip, one token each
        {"name": "paged shared prefix", "op": "paged", "streams": 64, "prefix": 16384, "low": 1, "high": 600,
         "new": 1, "heads": 40, "kv_heads": 8, "dim": 128, "page": 64, "block": 1, "dtype": "bf16", "salt": 3},
        # 16 viewers branched off one clip, the 64 tokens of one frame each, 12 heads, half precision
        {"name": "paged frame chunk fp16", "op": "paged", "streams": 16, "prefix": 4000, "low": 64, "high": 900,
         "new": 64, "heads": 12, "kv_heads": 12, "dim": 64, "page": 32, "block": 64, "dtype": "fp16", "salt": 4},
        # 16 viewers branch off a clip, in place of the 16 before them: shared pages, the last page copied
        {"name": "pages fork", "op": "pages", "what": "fork", "deep": False, "streams": 17, "tokens": 4100,
         "layers": 30, "kv_heads": 12, "dim": 128, "page": 64, "dtype": "bf16"},
        # sessions end in turn, the pool is closed up, others start
        {"name": "pages turnover", "op": "pages", "what": "compact", "deep": False, "streams": 2, "tokens": 2000,
         "layers": 30, "kv_heads": 12, "dim": 128, "page": 64, "dtype": "bf16"},
        # a step's keys and values of 64 streams in one layer (latency)
        {"name": "write step", "op": "write", "streams": 64, "low": 100, "high": 2000, "new": 1, "kv_heads": 8,
         "dim": 128, "page": 64, "dtype": "bf16", "salt": 5},
        # the keys and values of prompts in one layer
        {"name": "write prompts", "op": "write", "streams": 4, "low": 2048, "high": 4097, "new": 2048,
         "kv_heads": 40, "dim": 128, "page": 64, "dtype": "bf16", "salt": 6},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "paged", "paged", "paged", "pages", "write"])
    dim, dtype, page = rng.choice([64, 128]), rng.choice(["bf16", "fp16"]), rng.choice([16, 32, 64, 128])
    if op == "prompt":
        heads, kv_heads = rng.choice([(12, 12), (40, 40), (32, 8), (16, 2), (8, 1), (6, 3), (10, 2), (40, 8)])
        longest = _log(rng, 16, 8192)
        lengths = [longest] + [_log(rng, 1, longest) for _ in range(rng.randint(0, 7))]
        while len(lengths) * heads * longest ** 2 > 40 * 8192 ** 2:      # the padded plain form's size
            lengths.pop()
        rng.shuffle(lengths)
        return {"op": op, "lengths": ",".join(map(str, lengths)), "heads": heads, "kv_heads": kv_heads, "dim": dim,
                "block": rng.choice([1, 1, 64, 100, 256, 1024]), "dtype": dtype}
    if op == "paged":
        heads, kv_heads = rng.choice([(12, 12), (32, 8), (16, 2), (8, 1), (10, 2), (40, 8), (6, 3)])
        streams = _log(rng, 1, 64)
        new = rng.choice([1, 1, 1, 2, 5, 16, 64])
        high = _log(rng, new, max(new, min(8000, 300000 // streams)))
        prefix = rng.choice([0, _log(rng, 64, 16384)])
        while streams > 1 and streams * new * heads * (prefix + high) > 1 << 30:      # the largest listed case's products
            streams //= 2
        return {"op": op, "streams": streams, "prefix": prefix,
                "low": _log(rng, new, high), "high": high, "new": new, "heads": heads, "kv_heads": kv_heads,
                "dim": dim, "page": page, "block": rng.choice([1, 1, 64]), "dtype": dtype,
                "salt": rng.randrange(1 << 20)}
    if op == "pages":
        what = rng.choice(["fork", "fork", "compact"])
        kv_heads, layers = rng.choice([1, 2, 8, 12]), _log(rng, 1, 30)
        tokens = _log(rng, 1, 4000)
        return {"op": op, "what": what, "deep": what == "fork" and tokens < 600 and rng.random() < 0.5,
                "streams": 2 if what == "compact" else rng.randint(2, 17), "tokens": tokens, "layers": layers,
                "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype}
    new = _log(rng, 1, 2048)
    high = _log(rng, new, 4097)
    return {"op": op, "streams": _log(rng, 1, 64) if new < 64 else rng.randint(1, 4), "low": _log(rng, new, high),
            "high": high, "new": new, "kv_heads": rng.choice([1, 3, 8, 12, 40]), "dim": dim, "page": page,
            "dtype": dtype, "salt": rng.randrange(1 << 20)}


def _own_tokens(case):
    """Tokens of each stream past the shared prefix (the newest ones included)."""
    r = random.Random(case["salt"])
    return [r.randint(case["low"], case["high"]) for _ in range(case["streams"])]


def _pages_of(tokens, page):
    return -(-tokens // page)


def _visible(first, n, total, block):
    """Keys that queries at positions first .. first + n - 1 of a sequence of `total` tokens see, summed."""
    return sum(min(total, (i // block + 1) * block) for i in range(first, first + n))


def work(case):
    d = case["dim"]
    if case["op"] == "prompt":
        lengths = [int(x) for x in case["lengths"].split(",")]
        rows = sum(lengths)
        pairs = sum(_visible(0, n, n, case["block"]) for n in lengths)
        return {"bytes": 2 * d * rows * (2 * case["heads"] + 2 * case["kv_heads"]), "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "paged":
        mine, new, prefix = _own_tokens(case), case["new"], case["prefix"]
        pairs = sum(_visible(prefix + m - new, new, prefix + m, case["block"]) for m in mine)
        rows = new * case["streams"]
        return {"bytes": 4 * d * case["kv_heads"] * (prefix + sum(mine)) + 4 * d * case["heads"] * rows,
                "flops": 4 * d * case["heads"] * pairs}
    if case["op"] == "pages":
        page_bytes = case["layers"] * 2 * case["kv_heads"] * case["page"] * d * 2
        pages = _pages_of(case["tokens"], case["page"])
        if case["what"] == "compact":
            return {"bytes": 2 * 2 * pages * page_bytes, "flops": 0}
        copied = pages if case["deep"] else (1 if case["tokens"] % case["page"] else 0)
        table = 4 * 2 * pages * (case["streams"] - 1)
        # (a source page is read once for all its copies)
        return {"bytes": copied * page_bytes * case["streams"] + table, "flops": 0}
    return {"bytes": 2 * 2 * case["streams"] * case["new"] * case["kv_heads"] * d * 2, "flops": 0}


# ---------------------------------------------------------------- the inputs

def _normal(gen, *shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


class _Pool:
    """The plain form's pool: page lists on the host, tables, lengths and pages on the GPU."""

    def __init__(self, streams, layers, kv_heads, dim, page, pages, width, dtype):
        self.page, self.width = page, width
        self.k = torch.zeros((layers, pages, kv_heads, page, dim), dtype=dtype, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = torch.full((streams, width), -1, dtype=torch.int32, device="cuda")
        self.lengths = torch.zeros(streams, dtype=torch.int32, device="cuda")
        self.lists = [[] for _ in range(streams)]
        self.tokens = [0] * streams
        self.users = [0] * pages

    def take(self, n):
        got = [p for p, u in enumerate(self.users) if u == 0][:n]
        for p in got:
            self.users[p] = 1
        return got

    def put(self, b):
        """Stream b's table row and length on the GPU."""
        self.table[b] = torch.tensor(self.lists[b] + [-1] * (self.width - len(self.lists[b])), dtype=torch.int32)
        self.lengths[b] = self.tokens[b]

    def extend(self, counts):
        for b, n in enumerate(counts):
            if n:
                self.tokens[b] += n
                self.lists[b] += self.take(_pages_of(self.tokens[b], self.page) - len(self.lists[b]))
                self.put(b)

    def free(self, streams):
        for b in streams:
            for p in self.lists[b]:
                self.users[p] -= 1
            self.lists[b], self.tokens[b] = [], 0
            self.put(b)

    def fork(self, source, to, deep):
        full = 0 if deep else self.tokens[source] // self.page
        src, dst = [], []
        for b in to:
            new = self.take(len(self.lists[source]) - full)
            src += self.lists[source][full:]
            dst += new
            for p in self.lists[source][:full]:
                self.users[p] += 1
            self.lists[b], self.tokens[b] = self.lists[source][:full] + new, self.tokens[source]
            self.put(b)
        self.move(src, dst)

    def compact(self):
        live = sum(u > 0 for u in self.users)
        src = [p for p in range(live, len(self.users)) if self.users[p]]
        dst = [p for p in range(live) if not self.users[p]]
        to = dict(zip(src, dst))
        self.move(src, dst)
        for p, q in to.items():
            self.users[q], self.users[p] = self.users[p], 0
        for b, pages in enumerate(self.lists):
            self.lists[b] = [to.get(p, p) for p in pages]
            self.put(b)

    def move(self, src, dst):
        if src:
            s, t = torch.tensor(src, device="cuda"), torch.tensor(dst, device="cuda")
            self.k[:, t] = self.k[:, s]
            self.v[:, t] = self.v[:, s]

    def write(self, layer, k, v, counts):
        n = torch.tensor(counts, device="cuda")
        stream = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), n)
        nth = torch.arange(k.shape[0], device="cuda") - (n.cumsum(0) - n)[stream]
        at = (self.lengths.long() - n)[stream] + nth
        page = self.table[stream, at // self.page].long()
        self.k[layer][page, :, at % self.page] = k
        self.v[layer][page, :, at % self.page] = v


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, d = DTYPES[case["dtype"]], case["dim"]
    if case["op"] == "prompt":
        lengths = [int(x) for x in case["lengths"].split(",")]
        rows, heads, kv_heads = sum(lengths), case["heads"], case["kv_heads"]
        # queries, keys and values as a fused projection leaves them: one row of all heads per token
        qkv = _normal(gen, rows, (heads + 2 * kv_heads), d, dtype=dtype)
        offsets = [0]
        for n in lengths:
            offsets.append(offsets[-1] + n)
        return {"case": case, "q": qkv[:, :heads], "k": qkv[:, heads:heads + kv_heads], "v": qkv[:, heads + kv_heads:],
                "offsets": offsets, "out": torch.empty((rows, heads, d), dtype=dtype, device="cuda")}

    page, kv_heads = case["page"], case["kv_heads"]
    if case["op"] == "pages":
        layers, streams, tokens = case["layers"], case["streams"], case["tokens"]
        each = _pages_of(tokens, page)
        pages = each * streams if case["deep"] or case["what"] == "compact" else each + streams
        pool = _make_pool(streams, layers, case.get("heads", kv_heads), kv_heads, d, page, pages, each, 1, 1, case["dtype"])
        first = [tokens] + [tokens if case["what"] == "compact" else 0] * (streams - 1)
        pool.extend(first)
        for layer in range(layers):
            rows = sum(first)
            pool.write(layer, _normal(gen, rows, kv_heads, d, dtype=dtype), _normal(gen, rows, kv_heads, d, dtype=dtype), first)
        if case["what"] == "fork":
            pool.fork(0, list(range(1, streams)), case["deep"])
        return {"case": case, "pool": pool}

    mine, new, prefix, streams = _own_tokens(case), case["new"], case.get("prefix", 0), case["streams"]
    pages = _pages_of(prefix, page) + sum(_pages_of(m + page, page) for m in mine) + streams
    width = _pages_of(prefix + max(mine), page)
    heads = case.get("heads", kv_heads)
    pool = _make_pool(streams, 1, heads, kv_heads, d, page, pages, width, streams * new, case.get("block", 1), case["dtype"])
    if prefix:
        first = [prefix] + [0] * (streams - 1)
        pool.extend(first)
        pool.write(0, _normal(gen, prefix, kv_heads, d, dtype=dtype), _normal(gen, prefix, kv_heads, d, dtype=dtype), first)
        if streams > 1:
            pool.fork(0, list(range(1, streams)), False)
    pool.extend(mine)
    rows = sum(mine)
    pool.write(0, _normal(gen, rows, kv_heads, d, dtype=dtype), _normal(gen, rows, kv_heads, d, dtype=dtype), mine)
    counts = [new] * streams
    state = {"case": case, "pool": pool, "counts": counts}
    if case["op"] == "paged":
        state["q"] = _normal(gen, streams * new, heads, d, dtype=dtype)
        state["out"] = torch.empty_like(state["q"])
    else:
        # a step's projection again: keys and values side by side
        kv = _normal(gen, streams * new, 2 * kv_heads, d, dtype=dtype)
        state["k"], state["v"] = kv[:, :kv_heads], kv[:, kv_heads:]
    return state


def _make_pool(streams, layers, heads, kv_heads, dim, page, pages, width, queries, block, dtype):
    if own:
        from causal_dit_kv_b200 import PagedKVCache
        return PagedKVCache(streams, layers, heads, kv_heads, dim, pages, page_tokens=page, stream_pages=width,
                            max_queries=queries, block_tokens=block, dtype=dtype)
    return _Pool(streams, layers, kv_heads, dim, page, pages, width, DTYPES[dtype])


# ---------------------------------------------------------------- one pass

def run(state):
    case, op = state["case"], state["case"]["op"]
    if op == "prompt":
        if own:
            from causal_dit_kv_b200 import prompt_attention
            prompt_attention(state["q"], state["k"], state["v"], state["out"], state["offsets"], block_tokens=case["block"])
            return state["out"]
        return _plain_prompt(state["q"], state["k"], state["v"], state["offsets"], case["block"])
    pool = state["pool"]
    if op == "paged":
        if own:
            pool.attention(0, state["q"], state["out"], state["counts"])
            return state["out"]
        return _plain_paged(pool, state["q"], state["counts"], case["new"], case["block"])
    if op == "write":
        pool.write(0, state["k"], state["v"], state["counts"])
    elif case["what"] == "fork":
        pool.free(list(range(1, case["streams"])))
        pool.fork(0, list(range(1, case["streams"])), case["deep"])
    else:
        for b in (0, 1):
            pool.free([b])
            pool.compact()
            pool.extend([case["tokens"] if s == b else 0 for s in (0, 1)])
    if own:
        return {"table": pool.page_table(), "lengths": pool.lengths(), "k": pool.k_pages(), "v": pool.v_pages()}
    return {"table": pool.table, "lengths": pool.lengths, "k": pool.k, "v": pool.v}


def _softmax_product(q, k, v, visible):
    """q [n, h, g, r, d], k and v [n, h, l, d] in 32 bits, visible [n, r, l]: [n, h, g, r, d]."""
    n, h, g, r, d = q.shape
    s = torch.matmul(q.reshape(n, h, g * r, d), k.transpose(2, 3)).view(n, h, g, r, -1)
    s.mul_(1.0 / math.sqrt(d)).masked_fill_(~visible[:, None, None], -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.matmul(s.view(n, h, g * r, -1), v).view(n, h, g, r, d) / total


def _plain_prompt(q, k, v, offsets, block):
    lengths = torch.tensor(offsets[1:], device="cuda") - torch.tensor(offsets[:-1], device="cuda")
    first = torch.tensor(offsets[:-1], device="cuda")
    longest = max(b - a for a, b in zip(offsets, offsets[1:]))
    at = torch.arange(longest, device="cuda")
    there = at[None] < lengths[:, None]                                   # [n, longest]
    index = torch.where(there, first[:, None] + at[None], first[:, None].clamp(max=q.shape[0] - 1))
    heads, kv_heads, d = q.shape[1], k.shape[1], q.shape[2]
    qf = q[index].float().view(len(offsets) - 1, longest, kv_heads, heads // kv_heads, d).permute(0, 2, 3, 1, 4)
    kf, vf = (x[index].float().permute(0, 2, 1, 3) for x in (k, v))
    last = torch.minimum(lengths[:, None].clamp(min=1), (at[None] // block + 1) * block)
    out = _softmax_product(qf, kf, vf, at[None, None] < last[..., None])
    return out.permute(0, 3, 1, 2, 4)[there].reshape(q.shape).to(q.dtype)


def _plain_paged(pool, q, counts, new, block):
    streams, heads, d = len(counts), q.shape[1], q.shape[2]
    kv_heads = pool.k.shape[2]
    table = pool.table.long().clamp(min=0)
    kf, vf = (x[0][table].permute(0, 2, 1, 3, 4).reshape(streams, kv_heads, -1, d).float() for x in (pool.k, pool.v))
    qf = q.float().view(streams, new, kv_heads, heads // kv_heads, d).permute(0, 2, 3, 1, 4)
    at = pool.lengths.long()[:, None] - new + torch.arange(new, device="cuda")
    last = torch.minimum(pool.lengths.long()[:, None], (at // block + 1) * block)
    visible = torch.arange(kf.shape[2], device="cuda")[None, None] < last[..., None]
    return _softmax_product(qf, kf, vf, visible).permute(0, 3, 1, 2, 4).reshape(q.shape).to(q.dtype)


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Row by row of the definition: sequences and heads one after another, everything in 64 bits."""
    if case["op"] not in ("prompt", "paged"):
        return None                                                       # copies: nothing is computed
    global own
    kept, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = kept
    block, d = case["block"], case["dim"]
    group = case["heads"] // case["kv_heads"]
    out = torch.empty(state["out"].shape, dtype=torch.float64, device="cuda")
    if case["op"] == "prompt":
        spans = [(a, b - a, b - a) for a, b in zip(state["offsets"], state["offsets"][1:])]
    else:
        pool, new = state["pool"], case["new"]
        spans = [(b * new, new, pool.tokens[b]) for b in range(case["streams"])]
    for b, (row, n, total) in enumerate(spans):
        if case["op"] == "prompt":
            k, v = (state[x][row:row + n].double().transpose(0, 1) for x in ("k", "v"))
        else:
            k, v = (torch.cat([x[0, p] for p in pool.lists[b]], 1)[:, :total].double() for x in (pool.k, pool.v))
        for r in range(0, n, 2048):
            m = min(2048, n - r)
            i = torch.arange(total - n + r, total - n + r + m, device="cuda")
            hidden = torch.arange(total, device="cuda")[None] // block > i[:, None] // block
            for h in range(case["heads"]):
                s = state["q"][row + r:row + r + m, h].double() @ k[h // group].T / d ** 0.5
                out[row + r:row + r + m, h] = torch.softmax(s.masked_fill(hidden, -math.inf), 1) @ v[h // group]
    return out
