"""Prompt attention (sdv2_prompt_attention) against the plain 64-bit form (B200): packed
sequences of one token to several tiles, grouped heads, blocks, strides, what lies between
the sequences, and calls that take several launches."""
import math

import pytest
import torch

import tokens_ref as R

pytestmark = pytest.mark.gpu


def _inputs(seed, tokens, hq, hkv, d, dtype, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn((tokens, hq + 2 * hkv, d), generator=g, device="cuda")
    qkv[:, :hq] *= gain
    qkv = qkv.to(dtype)
    return qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]


def _check(q, k, v, offsets, block, scale=None, out=None):
    from causal_dit_kv_b200 import prompt_attention, prompt_check
    d = q.shape[2]
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda") if out is None else out
    prompt_attention(q, k, v, out, offsets, block_tokens=block, softmax_scale=scale)
    want, weight, largest = R.prompt_reference(q, k, v, offsets, block, 1 / math.sqrt(d) if scale is None else scale)
    keys = max(b - a for a, b in zip(offsets, offsets[1:]))
    inside = v[~torch.isnan(want[:, 0, 0])]
    tol = R.attention_tolerance(want, weight, largest, q.dtype, d, keys, float(inside.abs().max()))
    R.assert_attention(out, want, tol)
    assert prompt_check() == 0
    return out


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


@pytest.mark.parametrize("lengths", [[1], [2], [127], [128], [129], [255], [256], [257], [513],
                                     [1, 1, 1], [0, 5, 0, 0, 300, 0], [130, 1, 127, 640, 64]])
@pytest.mark.parametrize("heads,d,dtype", [((1, 1), 128, torch.bfloat16), ((4, 2), 64, torch.float16),
                                           ((3, 1), 128, torch.float16), ((10, 2), 64, torch.bfloat16)])
def test_lengths(lengths, heads, d, dtype):
    q, k, v = _inputs(1, sum(lengths), *heads, d, dtype)
    _check(q, k, v, _offsets(lengths), 1)


@pytest.mark.parametrize("block", [1, 2, 63, 64, 100, 128, 129, 256, 600, 1 << 31])
@pytest.mark.parametrize("heads", [(2, 2), (8, 1)])
def test_blocks(block, heads):
    q, k, v = _inputs(2, 1100, *heads, 128, torch.bfloat16)
    _check(q, k, v, [0, 600, 1100], block)


@pytest.mark.parametrize("heads,d", [((4, 4), 128), ((4, 2), 64)])
@pytest.mark.parametrize("a,b", [(123, 77), (500, 700), (900, 1), (1030, 2050)])
def test_other_tokens_have_no_part(heads, d, a, b):
    """Gaps between the sequences hold NaN and infinities, a sequence between two others too: no
    row of another sequence sees them, and rows of out in the gaps stay."""
    offsets = [10, 10, 10 + a, 77 + a, 77 + a + b]
    n = offsets[-1] + 9
    q, k, v = _inputs(3, n, *heads, d, torch.bfloat16)
    for x in (q, k, v):
        x[:10] = math.nan
        x[n - 9:] = math.inf
    k[10 + a:77 + a] = -math.inf                      # a whole sequence without a finite key or value
    v[10 + a:77 + a] = math.nan
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    from causal_dit_kv_b200 import prompt_attention
    prompt_attention(q, k, v, out, offsets)
    for part in (offsets[1:3], offsets[3:]):
        want, weight, largest = R.prompt_reference(q, k, v, part, 1, d ** -0.5)
        R.assert_attention(out, want, R.attention_tolerance(want, weight, largest, q.dtype, d, part[1] - part[0], 6.0))
    assert bool((out[:10] == 7).all()) and bool((out[n - 9:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_scores_that_climb(dtype):
    """Scores that grow by far more than 2^8 from tile to tile (the accumulator is rescaled in
    every one), and a row whose first key outweighs all others."""
    n, d = 900, 64
    q, k, v = _inputs(4, n, 2, 2, d, dtype)
    ramp = torch.linspace(0, 60, n, device="cuda")[:, None]
    q[:, 0], k[:, 0] = 1.0, (ramp / 8).to(dtype).expand(n, d)     # scores up to 64 * 60 / 8 / 8
    k[0, 1] = 0
    k[0, 1, 0], q[:, 1, 0] = 100.0, 20.0
    _check(q, k, v, [0, n], 1)


def test_scale_and_large_gain():
    q, k, v = _inputs(5, 400, 6, 3, 128, torch.float16, gain=6.0)
    _check(q, k, v, [0, 150, 400], 1, scale=0.3)


def test_strided_out_and_contiguous_inputs():
    q, k, v = (x.contiguous() for x in _inputs(6, 300, 5, 5, 64, torch.bfloat16))
    wide = torch.full((300, 9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    _check(q, k, v, [0, 300], 1, out=wide[:, 2:7])
    assert bool((wide[:, :2] == 3).all()) and bool((wide[:, 7:] == 3).all())


def test_many_sequences_and_items():
    """More sequences than one launch takes, and more row tiles than one launch's list holds."""
    from causal_dit_kv_b200 import binding as B
    lengths = [(7 * i) % 200 + 1 for i in range(600)]
    q, k, v = _inputs(7, sum(lengths), 2, 1, 64, torch.bfloat16)
    before = B.sdv2_launch_count()
    _check(q, k, v, _offsets(lengths), 1)
    assert B.sdv2_launch_count() - before == 3
    lengths = [7000] * 120                            # 6600 tiles of 128 rows
    offsets = _offsets(lengths)
    q, k, v = _inputs(8, sum(lengths), 2, 1, 64, torch.bfloat16)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    from causal_dit_kv_b200 import prompt_attention, prompt_check
    before = B.sdv2_launch_count()
    prompt_attention(q, k, v, out, offsets, block_tokens=16)
    assert B.sdv2_launch_count() - before == 2 and prompt_check() == 0
    for s in (0, 59, 119):
        a, b = offsets[s], offsets[s + 1]
        want, weight, largest = R.attention_rows(q[a:b], k[a:b], v[a:b], range(7000), 16, 0.125)
        R.assert_attention(out[a:b], want, R.attention_tolerance(want, weight, largest, q.dtype, 64, 7000, 6.0))


def test_no_tokens():
    from causal_dit_kv_b200 import prompt_attention
    q, k, v = _inputs(9, 4, 2, 2, 64, torch.bfloat16)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    prompt_attention(q, k, v, out, [0])
    prompt_attention(q, k, v, out, [2, 2, 2])
    assert bool((out == 7).all())
    prompt_attention(q[:0], k[:0], v[:0], out[:0], [0, 0])


def test_same_bits_again_on_another_stream_and_from_a_graph():
    q, k, v = _inputs(10, 1500, 8, 2, 128, torch.bfloat16)
    from causal_dit_kv_b200 import prompt_attention
    offsets = [0, 900, 1500]
    first = _check(q, k, v, offsets, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = torch.empty_like(first)
        prompt_attention(q, k, v, again, offsets)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, again)
    graph, graphed = torch.cuda.CUDAGraph(), torch.zeros_like(first)
    with torch.cuda.graph(graph):
        prompt_attention(q, k, v, graphed, offsets)
    for _ in range(2):
        graphed.zero_()
        graph.replay()
        assert torch.equal(first, graphed)


def test_calls_and_replays_at_once():
    """Calls that run beside one another, each with more units than the device has SMs, take over
    none but their own; the same for replays of their graphs."""
    from causal_dit_kv_b200 import prompt_attention, prompt_check
    cases = [(_inputs(20, 2600, 16, 4, 128, torch.bfloat16), [0, 2500, 2501, 2600]),
             (_inputs(21, 3000, 12, 12, 64, torch.float16), [0, 1000, 3000]),
             (_inputs(22, 1800, 24, 8, 128, torch.float16), [0, 1800])]
    alone = [_check(*x, offsets, 1) for x, offsets in cases]
    outs = [[torch.zeros_like(a) for _ in range(6)] for a in alone]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(6):
        for (x, offsets), out, stream in zip(cases, outs, streams):
            prompt_attention(*x, out[i], offsets, stream=stream)
    torch.cuda.synchronize()
    for a, out in zip(alone, outs):
        assert all(torch.equal(a, o) for o in out)
    graphs = [torch.cuda.CUDAGraph() for _ in cases]
    for (x, offsets), out, graph in zip(cases, outs, graphs):
        with torch.cuda.graph(graph):
            for o in out[:3]:
                prompt_attention(*x, o, offsets)
    for out in outs:
        for o in out:
            o.zero_()
    torch.cuda.synchronize()
    for graph, stream in zip(graphs, streams):
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for a, out in zip(alone, outs):
        assert all(torch.equal(a, o) for o in out[:3])
    assert prompt_check() == 0


def test_rows_behind_the_last_sequence_stay():
    """Ends inside a tile, inside a warp's 32 rows and after a single row, both ways of pairing tiles."""
    from causal_dit_kv_b200 import prompt_attention
    for heads, d, dtype in [((4, 2), 128, torch.bfloat16), ((3, 3), 64, torch.float16)]:
        for n in (1, 31, 33, 129, 200, 255):
            q, k, v = _inputs(23, 400, *heads, d, dtype)
            out = torch.full(q.shape, 5.0, dtype=dtype, device="cuda")
            prompt_attention(q, k, v, out, [3, 3 + n])
            assert bool((out[:3] == 5).all()) and bool((out[3 + n:] == 5).all())
            short = torch.empty((n, heads[0], d), dtype=dtype, device="cuda")
            prompt_attention(q[3:3 + n], k[3:3 + n], v[3:3 + n], short, [0, n])
            assert torch.equal(out[3:3 + n], short)


def test_wrapper_refusals():
    from causal_dit_kv_b200 import prompt_attention
    q, k, v = _inputs(11, 8, 4, 2, 64, torch.bfloat16)
    out = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    bad = [(q.float(), k, v, out), (q, k.half(), v, out), (q, k, v.cpu(), out), (q.cpu(), k, v, out),
           (q, k[:7], v, out), (q, k, v[:, :1], out), (q, k, v, out[:, :3]), (q[:, :, :32], k, v, out),
           (q.transpose(0, 1), k, v, out), (q[0], k, v, out)]
    for args in bad:
        with pytest.raises(ValueError):
            prompt_attention(*args, [0, 8])
