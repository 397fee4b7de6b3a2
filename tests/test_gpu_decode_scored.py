"""The scored decode on the GPU against the 64-bit reference: caps, slopes, windows, starts, weights; what lies outside the
visible tokens (blocks, table entries, NaN and infinities) is never read."""
import math

import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _operator_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def make(lens, hq, hkv, d, bs, dtype, seed, int8=False, q_std=2.0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)     # entries past a context are not read
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    shape = (nb, 2, hkv, bs, d)
    c = dict(lens=lens, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, tables=tables, scale=1 / math.sqrt(d),
             q=(torch.randn((len(lens), hq, d), generator=g) * q_std).to(dtype))
    if int8:
        c["kv"] = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8)
        c["scales"] = [(torch.rand((hkv, d), generator=g) + 0.5) / 60 for _ in range(2)]
    else:
        c["kv"] = torch.randn(shape, generator=g).to(dtype)
    return c


def rows_of(c, i, half, h):
    n, bs = c["lens"][i], c["bs"]
    t = torch.arange(n)
    x = c["kv"][c["tables"][i][t // bs].long(), half, h, t % bs]
    return x.double() * c["scales"][half][h].double() if "scales" in c else x


def lo_of(c, i, window, starts):
    lo = max(0, c["lens"][i] - window) if window else 0
    return min(max(lo, int(starts[i]) if starts is not None else 0), c["lens"][i])


def poison(c, window, starts):
    """NaN / Inf into every slot that no sequence sees, and bad entries into tables before the first visible block."""
    bs, seen = c["bs"], torch.zeros(c["kv"].shape[0], c["bs"], dtype=torch.bool)
    for i, n in enumerate(c["lens"]):
        lo = lo_of(c, i, window, starts)
        for t in range(lo, n):
            seen[c["tables"][i, t // bs], t % bs] = True
        c["tables"][i, :(lo if lo < n else n) // bs] = -3 - i
    kv = c["kv"].clone()
    bad = torch.tensor([math.nan, math.inf, -math.inf], dtype=c["dtype"])
    for k, (b, o) in enumerate((~seen).nonzero().tolist()):
        kv[b, :, :, o] = bad[k % 3]
    return kv


def run(dev, c, softcap=0.0, slopes=None, window=0, starts=None, weights=None, want=False, part=0, kv=None, in_place=False):
    on = (c["kv"] if kv is None else kv).to(dev)
    put = lambda t: None if t is None else t.to(dev)
    kw = dict(softcap=softcap, slopes=put(slopes), window=window, starts=put(starts), max_context_len=max(c["lens"] + [0]),
              partition_size=part)
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=dev)
    args = (c["q"].to(dev), *pkv.split_pool(on))
    if "scales" in c:
        out = pkv.paged_attention_decode_scored_int8(*args, *[s.to(dev) for s in c["scales"]], c["tables"].to(dev), lens,
                                                     c["scale"], **kw)
        wout = None
    else:
        win = put(weights)
        wout = win if in_place else torch.full((len(c["lens"]), c["hkv"], max(c["lens"] + [1]) + 3), 5.0, device=dev) if want \
            else None
        out = pkv.paged_attention_decode_scored(*args, c["tables"].to(dev), lens, c["scale"], weights=win, weights_out=wout,
                                                **kw)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    return out.cpu(), None if wout is None else wout.cpu()


def check(c, out, wout=None, softcap=0.0, slopes=None, window=0, starts=None, weights=None, rest=5.0):
    g = c["hq"] // c["hkv"]
    int8 = "scales" in c
    p_half = 2.0 ** -11 if int8 or c["dtype"] == F16 else 2.0 ** -8
    for i, n in enumerate(c["lens"]):
        lo = lo_of(c, i, window, starts)
        for h in range(c["hkv"]):
            k, v = rows_of(c, i, 0, h), rows_of(c, i, 1, h)
            acc, err = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
            for hq in range(h * g, (h + 1) * g):
                slope = float(slopes[hq]) if slopes is not None else 0.0
                ref, w, absref = refs.attend_row(c["q"][i, hq], k, v, c["scale"], softcap, slope, n - 1, lo, n)
                slack = refs.score_slack(c["q"][i, hq], k[lo:], c["scale"], softcap, slope, n, int8)
                refs.check_attention(out[i, hq], ref, absref, slack, p_half, f"seq {i} head {hq}")
                acc += w
                err += w * (2 * slack + 2.0 ** -19)
            if wout is not None:
                base = weights[i, h, :n].double() if weights is not None else 0.0
                diff = (wout[i, h, :n].double() - base - acc).abs()
                # masked tokens keep their weight exactly: acc and err are 0 there.  A weight (or the exponential
                # before its quotient with a sum of at least 1) below fp32's smallest normal 2^-126 is flushed to 0,
                # so each head may lose up to 2^-125
                assert (diff <= err + (acc > 0) * ((base + acc) * 2.0 ** -23 + g * 2.0 ** -125)).all(), f"weights, seq {i} head {h}"
                assert (wout[i, h, n:] == (weights[i, h, n:] if rest is None else rest)).all()


SLOPES = lambda hq: torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float()
SHAPES = [  # hq, hkv, d, bs: one, two, four, eight, sixteen and odd heads per KV head
    (4, 4, 64, 16), (6, 2, 128, 8), (4, 2, 128, 32), (8, 2, 128, 16), (8, 1, 128, 8), (32, 2, 128, 32), (16, 1, 128, 8),
    (8, 2, 64, 32), (16, 2, 64, 8), (10, 5, 64, 32),
    # groups that fill no whole block: three, five, six, twelve, twenty, thirty-four heads
    (6, 2, 128, 16), (10, 2, 128, 16), (15, 3, 64, 8), (12, 2, 128, 8), (24, 2, 64, 16), (24, 2, 128, 32), (20, 1, 128, 16),
    (40, 2, 64, 32), (34, 1, 128, 8), (16, 1, 64, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("part", [0, 64])
def test_all_forms_together(hq, hkv, d, bs, dtype, part):
    dev = device()
    c = make([1, 0, 33, 300, 129, 16], hq, hkv, d, bs, dtype, seed=hq + d + bs)
    slopes, starts = SLOPES(hq), torch.tensor([0, 0, 40, 250, 31, 15], dtype=torch.int32)
    w = torch.rand((6, hkv, 303), generator=torch.Generator().manual_seed(1))
    kv = poison(c, 200, starts)
    out, wout = run(dev, c, 5.0, slopes, 200, starts, w, True, part, kv)
    check(c, out, wout, 5.0, slopes, 200, starts, w)
    assert (out[1] == 0).all() and (out[2] == 0).all()                           # nothing visible


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("form", ["plain", "cap", "slopes", "window", "starts"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(3, 3, 128, 16), (8, 2, 128, 16), (32, 2, 128, 16), (8, 2, 64, 8)])
def test_each_form_alone(hq, hkv, d, bs, form, dtype):
    dev = device()
    c = make([700, 5, 1025], hq, hkv, d, bs, dtype, seed=11)
    kw = dict(plain={}, cap=dict(softcap=2.0), slopes=dict(slopes=SLOPES(hq)), window=dict(window=130),
              starts=dict(starts=torch.tensor([699, -4, 513], dtype=torch.int32)))[form]
    kv = poison(c, kw.get("window", 0), kw.get("starts"))
    out, wout = run(dev, c, want=True, kv=kv, **kw)
    check(c, out, wout, **kw)
    alone, _ = run(dev, c, kv=kv, **kw)
    check(c, alone, **kw)


@pytest.mark.parametrize("window", [1, 7, 8, 16, 17, 64, 1000, 5000])
@pytest.mark.parametrize("hq,hkv,d,bs,int8", [(2, 2, 128, 32, False), (8, 2, 128, 32, False), (8, 2, 128, 32, True),
                                              (2, 2, 128, 32, True), (4, 1, 64, 16, False), (16, 1, 128, 8, False)])
def test_window_borders(hq, hkv, d, bs, int8, window):
    dev = device()
    c = make([1000, 1001, 1015, 1016, 1, 8], hq, hkv, d, bs, BF16, seed=window, int8=int8)
    kv = None if int8 else poison(c, window, None)
    out, wout = run(dev, c, window=window, want=True, kv=kv, part=bs * 2)
    check(c, out, wout, window=window)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_int8_cache(hq, hkv, d, bs, dtype):
    dev = device()
    c = make([1, 0, 33, 300, 129], hq, hkv, d, bs, dtype, seed=hq + bs, int8=True)
    slopes, starts = SLOPES(hq), torch.tensor([0, 0, 40, 250, 31], dtype=torch.int32)
    for part in (0, 64):
        out, _ = run(dev, c, 5.0, slopes, 200, starts, part=part)
        check(c, out, None, 5.0, slopes, 200, starts)
    out, _ = run(dev, c, 0.5)
    check(c, out, None, 0.5)


@pytest.mark.parametrize("scale,softcap", [(0.001, 1.0), (3.0, 1.0), (30.0, 50.0), (-2.0, 3.0), (0.0, 2.0), (1.0, 1e-3),
                                           (1.0, 1e6)])
def test_caps_from_linear_to_saturated(scale, softcap):
    dev = device()
    for hq, hkv in ((4, 1), (2, 2)):
        c = make([200, 65], hq, hkv, 128, 16, F16, seed=3)
        c["scale"] = scale
        out, wout = run(dev, c, softcap, want=True)
        check(c, out, wout, softcap)


def test_weights_accumulate_in_place_over_steps_and_feed_eviction():
    """Decode steps accumulate into one array; the heaviest tokens stay; the next step decodes the compacted context."""
    dev = device()
    c = make([150, 90], 8, 2, 128, 16, BF16, seed=21)
    w = torch.zeros((2, 2, 160))
    on, total = w.to(dev), torch.zeros((2, 2, 160), dtype=torch.float64)
    kv = c["kv"].to(dev)
    k_cache, v_cache = pkv.split_pool(kv)
    lens, tables = torch.tensor(c["lens"], dtype=torch.int32, device=dev), c["tables"].clamp(min=0).to(dev)
    g = torch.Generator().manual_seed(4)
    for _ in range(3):
        q = torch.randn((2, 8, 128), generator=g).to(BF16)
        pkv.paged_attention_decode_scored(q.to(dev), k_cache, v_cache, tables, lens, weights=on, weights_out=on,
                                          max_context_len=150)
        for i, n in enumerate(c["lens"]):
            for h in range(8):
                total[i, h // 4, :n] += refs.attend_row(q[i, h], rows_of(c, i, 0, h // 4), rows_of(c, i, 1, h // 4),
                                                        128 ** -0.5, 0, 0, n - 1, 0, n)[1]
    torch.cuda.synchronize()
    # three steps of four heads, no weight over 0.1, each off by twice the score slack (below 1.3e-4 for these rows)
    assert (on.cpu().double() - total).abs().max() <= 3 * 4 * 0.1 * 2.6e-4 and (on.cpu()[1, :, 90:] == 0).all()
    kept, kept_lens = pkv.evict_select(on, lens, 64, sinks=2, recent=8, max_context_len=150, weights_out=on)
    before = [[(rows_of(c, i, 0, h)[kept.cpu()[i, h].long()], rows_of(c, i, 1, h)[kept.cpu()[i, h].long()])
               for h in range(2)] for i in range(2)]
    pkv.evict_compact(k_cache, v_cache, tables, lens, kept, kept_lens)
    q = torch.randn((2, 8, 128), generator=g).to(BF16)
    out = pkv.paged_attention_decode_scored(q.to(dev), k_cache, v_cache, tables, kept_lens, weights=on, weights_out=on,
                                            max_context_len=64)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert kept_lens.cpu().tolist() == [64, 64]
    for i in range(2):
        for h in range(8):
            k, v = before[i][h // 4]
            ref, _, absref = refs.attend_row(q[i, h], k, v, 128 ** -0.5, 0, 0, 63, 0, 64)
            refs.check_attention(out.cpu()[i, h], ref, absref, refs.score_slack(q[i, h], k, 128 ** -0.5, 0, 0, 0), 2.0 ** -8,
                                 "after eviction")


def test_a_long_context_split_many_ways_and_its_weights():
    dev = device()
    c = make([20011], 4, 1, 128, 16, F16, seed=31)
    out, wout = run(dev, c, 20.0, SLOPES(4) / 64, 0, None, None, True, 16 * 16)
    check(c, out, wout, 20.0, SLOPES(4) / 64)


@pytest.mark.parametrize("odd", [0, 1], ids=["vectors", "odd_stride"])
def test_weights_of_a_large_batch(odd):
    """Enough tokens for several steps per block of the weights; the first and last sequences are checked in full, the others'
    weights by their sums (each query head's weights sum to 1)."""
    dev = device()
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(1, 2600, (64,), generator=g).tolist()
    lens[0], lens[-1] = 2600, 2599
    c = make(lens, 16, 8, 64, 16, F16, seed=9)
    kv = c["kv"].to(dev)
    w = torch.full((64, 8, 2600 + odd), 5.0, device=dev)
    old = torch.rand((64, 8, 2600 + odd), generator=g).to(dev)
    dl = torch.tensor(lens, dtype=torch.int32, device=dev)
    out = pkv.paged_attention_decode_scored(c["q"].to(dev), *pkv.split_pool(kv), c["tables"].to(dev), dl, c["scale"], weights=old,
                                            weights_out=w, max_context_len=2600)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    inside = torch.arange(2600 + odd, device=dev) < dl[:, None]
    assert (w[~inside[:, None].expand_as(w)] == 5.0).all()
    added = torch.where(inside[:, None], w.double() - old.double(), 0.0).sum(2).cpu()
    assert (added - 2.0).abs().max() <= 2600 * 2.0 ** -23 + 1e-3          # roundings of w + the scores' slack (below 5e-4)
    ends = dict(c, lens=[lens[0], lens[-1]], tables=c["tables"][[0, -1]], q=c["q"][[0, -1]])
    check(ends, out.cpu()[[0, -1]], w.cpu()[[0, -1]], weights=old.cpu()[[0, -1]])


def test_bad_lengths_and_entries_are_flagged():
    dev = device()
    c = make([40, 40], 4, 2, 128, 16, F16, seed=5)
    c["tables"][0, 1] = 10 ** 6
    kv = c["kv"].to(dev)
    out = pkv.paged_attention_decode_scored(c["q"].to(dev), *pkv.split_pool(kv), c["tables"].to(dev),
                                            torch.tensor([40, 41], dtype=torch.int32, device=dev), softcap=3.0,
                                            max_context_len=40)
    assert sorted(pkv.get_device_error(dev)[1]) == ["block_table", "context_len"]
    c["lens"] = [40, 40]
    ref, _, absref = refs.attend_row(c["q"][1, 0], rows_of(c, 1, 0, 0), rows_of(c, 1, 1, 0), c["scale"], 3.0, 0, 39, 0, 40)
    refs.check_attention(out.cpu()[1, 0], ref, absref, refs.score_slack(c["q"][1, 0], rows_of(c, 1, 0, 0), c["scale"], 3.0, 0, 0),
                         2.0 ** -11, "clamped to the bound")
    w = torch.full((2, 2, 40), 7.0, device=dev)
    for hq in (4, 2):                                        # the MMA and the lane form
        pkv.paged_attention_decode_scored(c["q"][:, :hq].contiguous().to(dev), *pkv.split_pool(kv), c["tables"].to(dev),
                                          torch.tensor([40, 40], dtype=torch.int32, device=dev), weights_out=w,
                                          max_context_len=40)
        assert pkv.get_device_error(dev)[1] == ["block_table"]
        assert (w[0, :, 16:32] == 0).all() and ((w[0].sum(1) - hq / 2).abs() < 1e-3).all()   # the bad block's tokens weigh nothing


def test_two_graphs_and_two_streams_do_not_share_a_workspace():
    dev = device()
    calls, refs_ = [], []
    for seed in (1, 2):
        c = make([3000, 1777], 8, 2, 128, 16, BF16, seed=seed)
        kv = c["kv"].to(dev)
        lens = torch.tensor(c["lens"], dtype=torch.int32, device=dev)
        w = torch.zeros((2, 2, 3008), device=dev)
        call = pkv.prepare_paged_attention_decode_scored(c["q"].to(dev), *pkv.split_pool(kv), c["tables"].clamp(min=0).to(dev),
                                                         lens, softcap=9.0, weights_out=w, max_context_len=3000,
                                                         partition_size=256)
        call()
        torch.cuda.synchronize()
        refs_.append((call.result.clone(), w.clone()))
        calls.append((call, w))
    streams = [torch.cuda.Stream(dev) for _ in calls]
    graphs = []
    for call, _ in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append(graph)
    for replay in (False, True):
        for call, w in calls:
            call.result.zero_()
            w.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for s, (call, _), graph in zip(streams, calls, graphs):
                with torch.cuda.stream(s):
                    graph.replay() if replay else call()
        torch.cuda.synchronize()
        for (call, w), (out, ref_w) in zip(calls, refs_):
            assert torch.equal(call.result, out) and torch.equal(w, ref_w)
    check_no_device_flags(dev)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 4, 64, 16), (4, 2, 128, 32), (8, 2, 128, 16), (8, 1, 128, 8), (32, 2, 128, 32),
                                         (15, 3, 64, 8), (24, 2, 128, 32)])
def test_outputs_do_not_change_when_the_weights_are_wanted(hq, hkv, d, bs, dtype):
    """Bit for bit; and where every visible token has one value, the output is that value (the weights' roundings are divided
    out again: off by a few 2^-24 of itself, which rounds back)."""
    dev = device()
    c = make([1, 2, 3, 5, 40, 700], hq, hkv, d, bs, dtype, seed=23)
    value = torch.randn((hkv, d), generator=torch.Generator().manual_seed(2)).to(dtype)
    for same in (True, False):
        if same:
            kv = c["kv"].clone()
            kv[:, 1] = value[None, :, None]
        else:
            kv = c["kv"]
        for kw in (dict(), dict(softcap=3.0), dict(window=4)):
            plain, _ = run(dev, c, kv=kv, **kw)
            out, _ = run(dev, c, kv=kv, want=True, **kw)
            assert torch.equal(out, plain)
            if same:
                assert torch.equal(out, value.repeat_interleave(hq // hkv, 0).expand(6, hq, d))
