"""A sliding window with first tokens that stay visible: decode (16-bit, INT8) and prefill against 64-bit references."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests._gpu_helpers import check_no_device_flags, device
from tests._operator_refs import HALF_STEP, rounded_close

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _seen(n, pos, window, sinks):
    t = torch.arange(n)[None]
    return (t <= pos[:, None]) & ((t < sinks) | (t > pos[:, None] - window))


def _forget(tables, lens, first, window, sinks, bs):
    """Bad entries for the blocks that lie between the first tokens and the window of the first query."""
    for i, n in enumerate(lens):
        lo = max(0, first[i] + 1 - window)
        for b in range(-(-sinks // bs), lo // bs):
            tables[i, b] = -5 - b


def _decode(dev, dtype, hq, hkv, d, bs, lens, window, sinks, part=0, int8=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    tables, blocks = refs.place(lens, bs, g)
    q = (torch.randn((len(lens), hq, d), generator=g) * 2).to(dtype)
    if int8:
        kv = torch.randint(-127, 128, (blocks, 2, hkv, bs, d), generator=g, dtype=torch.int8)
        scales = [(torch.rand((hkv, d), generator=g) + 0.5) / 64 for _ in range(2)]
        vals = kv.double() * torch.stack(scales).double()[:, :, None]
    else:
        kv = torch.randn((blocks, 2, hkv, bs, d), generator=g).to(dtype)
        vals = kv.double()
    seen = [_seen(n, torch.tensor([n - 1]), window, sinks) for n in lens]
    ctx = [refs.context(vals, tables[i], n) for i, n in enumerate(lens)]
    if not int8:
        refs.poison(kv, tables, [s[0].nonzero()[:, 0].tolist() for s in seen])
    _forget(tables, lens, [n - 1 for n in lens], window, sinks, bs)
    put = lambda t: t.to(dev)  # noqa: E731
    args = (put(q), *pkv.split_pool(put(kv)))
    rest = (put(tables), torch.tensor(lens, dtype=torch.int32, device=dev), d ** -0.5)
    kw = dict(window=window, sinks=sinks, max_context_len=max(lens + [1]), partition_size=part)
    if int8:
        out = pkv.paged_attention_decode_sinks_int8(*args, put(scales[0]), put(scales[1]), *rest, **kw)
    else:
        out = pkv.paged_attention_decode_sinks(*args, *rest, **kw)
    check_no_device_flags(dev)
    out = out.cpu()
    for i, n in enumerate(lens):
        want, mag, most = refs.attend(q[i:i + 1], *ctx[i], d ** -0.5, seen[i])
        # the lane forms (one or two heads) keep 32-bit weights over a 16-bit cache; INT8 ones are rounded to fp16
        half = 2.0 ** -11 if int8 else HALF_STEP[dtype]
        rounded_close(out[i], want[0], refs.attention_bound(mag, most, d, half, 2.0 ** -10 if int8 else 0.0)[0],
                      f"sequence {i} of {n} tokens")


LENS = [0, 1, 5, 16, 17, 63, 64, 130, 255, 400]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 128), (3, 1, 64), (8, 1, 64), (16, 1, 128), (20, 1, 128), (128, 8, 64)])
@pytest.mark.parametrize("bs,window,sinks", [(16, 50, 4), (8, 33, 20), (32, 64, 33), (16, 1, 1), (16, 100, 0), (8, 1000, 3)])
def test_decode(hq, hkv, d, bs, window, sinks, dtype):
    _decode(device(), dtype, hq, hkv, d, bs, LENS, window, sinks, seed=hq + d + bs)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d", [(2, 2, 64), (4, 2, 128), (8, 2, 128), (5, 1, 64), (8, 1, 128), (20, 1, 128)])
@pytest.mark.parametrize("bs,window,sinks", [(16, 50, 4), (8, 33, 20), (32, 70, 33), (16, 1, 40)])
def test_decode_int8(hq, hkv, d, bs, window, sinks, dtype):
    _decode(device(), dtype, hq, hkv, d, bs, LENS, window, sinks, int8=True, seed=hq + d + bs)


@pytest.mark.parametrize("part", [32, 64, 96])
@pytest.mark.parametrize("window,sinks", [(40, 6), (150, 33), (300, 70), (7, 250)])
def test_decode_in_partitions_that_cut_the_gap(part, window, sinks):
    _decode(device(), BF16, 8, 2, 128, 32, [500, 90, 33, 299], window, sinks, part=part, seed=part)
    _decode(device(), F16, 2, 2, 64, 16, [500, 90, 33, 299], window, sinks, part=part, seed=part)
    _decode(device(), F16, 4, 1, 128, 16, [500, 90, 33, 299], window, sinks, part=part, int8=True, seed=part)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("hq,hkv,d,seqs", [(8, 8, 64, 64), (16, 4, 128, 64), (8, 8, 64, 9), (64, 8, 64, 30)])
def test_decode_of_batches_that_fill_the_machine(hq, hkv, d, seqs, int8):
    """Spans whole in one block, or in few partitions: contexts from none to several spans, most of them full."""
    lens = [0, 1, 19, 20, 21, 170] + [160 + i * 97 % 700 for i in range(seqs - 6)]
    _decode(device(), F16, hq, hkv, d, 16, lens, 150, 20, int8=int8, seed=seqs + hq)


def test_decode_equals_the_windowed_one_without_first_tokens():
    dev, g = device(), torch.Generator().manual_seed(4)
    lens, bs = [700, 64, 3], 16
    tables, blocks = refs.place(lens, bs, g)
    q = torch.randn((3, 8, 128), generator=g).to(BF16).to(dev)
    kv = torch.randn((blocks, 2, 2, bs, 128), generator=g).to(BF16).to(dev)
    n, t = torch.tensor(lens, dtype=torch.int32, device=dev), tables.to(dev)
    a = pkv.paged_attention_decode_sinks(q, *pkv.split_pool(kv), t, n, window=100, sinks=0, max_context_len=700, partition_size=64)
    b = pkv.paged_attention_decode_scored(q, *pkv.split_pool(kv), t, n, window=100, max_context_len=700, partition_size=64)
    assert torch.equal(a, b)
    a = pkv.paged_attention_decode_sinks(q, *pkv.split_pool(kv), t, n, window=2 ** 31 - 1, sinks=2 ** 31 - 1, max_context_len=700)
    b = pkv.paged_attention_decode_scored(q, *pkv.split_pool(kv), t, n, max_context_len=700)
    assert torch.equal(a, b)


def _prefill(dev, dtype, hq, hkv, bs, cached, chunks, window, sinks, splits=0, seed=0, extra=0):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(cached, chunks)]
    tables, blocks = refs.place(lens, bs, g)
    rows = sum(chunks)
    q = (torch.randn((rows + extra, hq, 128), generator=g) * 2).to(dtype)
    kv = torch.randn((blocks, 2, hkv, bs, 128), generator=g).to(dtype)
    vals = kv.double()
    seen = [_seen(n, torch.arange(n - c, n), window, sinks) for n, c in zip(lens, chunks)]
    ctx = [refs.context(vals, tables[i], n) for i, n in enumerate(lens)]
    refs.poison(kv, tables, [s.any(0).nonzero()[:, 0].tolist() for s in seen])
    _forget(tables, lens, [n - c for n, c in zip(lens, chunks)], window, sinks, bs)
    out = torch.full_like(q, 3.0).to(dev)
    start = torch.tensor([0] + chunks, dtype=torch.int32).cumsum(0).to(torch.int32)
    pkv.paged_attention_prefill_sinks(q.to(dev), *pkv.split_pool(kv.to(dev)), tables.to(dev), start.to(dev),
                                      torch.tensor(lens, dtype=torch.int32, device=dev), 128 ** -0.5, out,
                                      max_query_len=max(chunks), max_context_len=max(lens), window=window, sinks=sinks,
                                      kv_splits=splits)
    check_no_device_flags(dev)
    out = out.cpu()
    assert (out[rows:] == 3.0).all()
    at = 0
    for i, c in enumerate(chunks):
        want, mag, most = refs.attend(q[at:at + c], *ctx[i], 128 ** -0.5, seen[i])
        rounded_close(out[at:at + c], want, refs.attention_bound(mag, most, 128, HALF_STEP[dtype]), f"sequence {i}")
        at += c


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 1), (3, 1), (40, 2), (128, 1)])
@pytest.mark.parametrize("bs,window,sinks", [(16, 50, 4), (8, 133, 20), (32, 64, 33), (16, 1, 1), (16, 300, 0), (32, 90, 200)])
@pytest.mark.parametrize("splits", [1, 3])
def test_prefill(hq, hkv, bs, window, sinks, splits, dtype):
    _prefill(device(), dtype, hq, hkv, bs, [0, 300, 1, 17, 511], [1, 37, 150, 64, 3], window, sinks, splits, seed=hq + bs, extra=2)


def test_prefill_of_many_sequences_and_row_tiles():
    _prefill(device(), BF16, 4, 2, 16, [i * 13 % 200 for i in range(70)], [i * 7 % 40 + 1 for i in range(70)], 30, 5, 1, seed=1)
    _prefill(device(), F16, 2, 1, 32, [640], [900], 256, 100, 1, seed=2)
    _prefill(device(), F16, 2, 1, 32, [640], [900], 256, 100, 0, seed=3)


def test_an_endless_stream_step_by_step():
    """A prompt and decode steps whose past blocks are freed as the window leaves them: what the steps return is what a
    prefill of the whole stream gives its rows."""
    dev, g = device(), torch.Generator().manual_seed(12)
    bs, window, sinks, n, total, hq, hkv = 8, 20, 5, 30, 75, 4, 2
    rows = lambda t, h: torch.randn((t, h, 128), generator=g).to(BF16).to(dev)  # noqa: E731
    k, v, q = rows(total, hkv), rows(total, hkv), rows(total, hq)
    whole = torch.zeros((10, 2, hkv, bs, 128), dtype=BF16, device=dev)
    full = torch.arange(10, dtype=torch.int32, device=dev)[None]
    pkv.reshape_and_cache(k, v, torch.arange(total, device=dev), *pkv.split_pool(whole))
    lens = torch.tensor([total], dtype=torch.int32, device=dev)
    want = pkv.paged_attention_prefill_sinks(q, *pkv.split_pool(whole), full, torch.tensor([0, total], dtype=torch.int32, device=dev),
                                             lens, max_query_len=total, max_context_len=total, window=window, sinks=sinks)
    # a pool of six blocks serves the stream: one for the first tokens, at most four for the window, one to go on
    pool = torch.full((6, 2, hkv, bs, 128), float("nan"), dtype=BF16, device=dev)
    free, table = list(range(6)), torch.full((1, 10), -1, dtype=torch.int32)
    for t in range(total):
        if t % bs == 0:
            table[0, t // bs] = free.pop()
        if t >= n:  # the steps' table only; the prompt is written whole above
            for b in range(1, max(0, t + 1 - window) // bs):
                if table[0, b] >= 0:
                    free.append(int(table[0, b]))
                    pool[int(table[0, b])] = float("nan")
                    table[0, b] = -1
        elif t // bs > 3:
            raise AssertionError("the prompt fits four blocks")
        slot = torch.tensor([int(table[0, t // bs]) * bs + t % bs], device=dev)
        pkv.reshape_and_cache(k[t:t + 1], v[t:t + 1], slot, *pkv.split_pool(pool))
        if t >= n:
            got = pkv.paged_attention_decode_sinks(q[t:t + 1], *pkv.split_pool(pool), table.to(dev),
                                                   torch.tensor([t + 1], dtype=torch.int32, device=dev), window=window,
                                                   sinks=sinks, max_context_len=t + 1)
            # both round their weights to bf16 (2^-8 each way) and their outputs (below 4)
            assert (got.float() - want[t:t + 1].float()).abs().max() < 4 * 4 * 2.0 ** -8
    check_no_device_flags(dev)


def test_in_a_graph_on_another_stream():
    dev, g = device(), torch.Generator().manual_seed(13)
    lens, bs = [300, 40], 16
    tables, blocks = refs.place(lens, bs, g)
    kv = torch.randn((blocks, 2, 2, bs, 128), generator=g).to(F16).to(dev)
    n, t = torch.tensor(lens, dtype=torch.int32, device=dev), tables.to(dev)
    q = torch.randn((2, 8, 128), generator=g).to(F16).to(dev)
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=dev)
    dec = pkv.prepare_paged_attention_decode_sinks(q, *pkv.split_pool(kv), t, n, window=70, sinks=3, max_context_len=300, partition_size=32)
    pre = pkv.prepare_paged_attention_prefill_sinks(q, *pkv.split_pool(kv), t, start, n, window=70, sinks=3, max_query_len=1,
                                                    max_context_len=300)
    a, b = dec().clone(), pre().clone()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dec()
        pre()
    dec.result.zero_()
    pre.result.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dec.result, a) and torch.equal(pre.result, b)
    assert (a.float() - b.float()).abs().max() < 8 * 4 * 2.0 ** -11
