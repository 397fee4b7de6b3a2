"""The scored prefill on the GPU against the 64-bit reference, row by row: caps, slopes, windows, document starts, prefixes,
rows that see nothing, key ranges that begin and end inside a block or a tile, splits and every item order."""
import math

import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _operator_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
SLOPES = lambda hq: torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float()


def make(cached, chunks, hq, hkv, bs, dtype, seed, extra_rows=0):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(cached, chunks)]
    need = [-(-n // bs) for n in lens]
    nb = sum(need) + 3
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    tables = torch.full((len(lens), max(need + [1])), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    rows = sum(chunks)
    return dict(lens=lens, chunks=chunks, hq=hq, hkv=hkv, bs=bs, dtype=dtype, tables=tables, scale=128 ** -0.5, rows=rows,
                q=(torch.randn((rows + extra_rows, hq, 128), generator=g) * 2).to(dtype),
                kv=torch.randn((nb, 2, hkv, bs, 128), generator=g).to(dtype))


def bounds(c, i, j, window, starts, prefix):
    n = c["lens"][i]
    pos = n - c["chunks"][i] + j
    row = sum(c["chunks"][:i]) + j
    lo = max(0, pos + 1 - window) if window else 0
    if starts is not None:
        lo = max(lo, int(starts[row]))
    hi = pos + 1
    if prefix is not None:
        hi = max(hi, min(n, int(prefix[i])))
    return row, pos, lo, hi


def poison(c, window, starts, prefix):
    """NaN / Inf into what no row of a sequence sees (its tokens before the first visible one and past the context, unused
    blocks), and bad entries into the tables before the first visible block."""
    bs, seen = c["bs"], torch.zeros(c["kv"].shape[0], c["bs"], dtype=torch.bool)
    for i, n in enumerate(c["lens"]):
        lows = [bounds(c, i, j, window, starts, prefix) for j in range(c["chunks"][i])]
        lows = [b[2] for b in lows if b[2] < b[3]]
        lo = min(lows) if lows else max(0, n - 1)
        for t in range(lo, n):
            seen[c["tables"][i, t // bs], t % bs] = True
        c["tables"][i, :lo // bs] = -3 - i
    bad = torch.tensor([math.nan, math.inf, -math.inf], dtype=c["dtype"])
    for k, (b, o) in enumerate((~seen).nonzero().tolist()):
        c["kv"][b, :, :, o] = bad[k % 3]


def run(dev, c, softcap=0.0, slopes=None, window=0, starts=None, prefix=None, splits=0):
    put = lambda t: None if t is None else t.to(dev)
    out = torch.full_like(c["q"], 3.0).to(dev)
    qs = torch.tensor([0] + c["chunks"], dtype=torch.int32).cumsum(0).to(torch.int32)
    if starts is not None and len(starts) < len(c["q"]):
        starts = torch.cat([starts, torch.zeros(len(c["q"]) - len(starts), dtype=torch.int32)])
    pkv.paged_attention_prefill_scored(
        c["q"].to(dev), *pkv.split_pool(c["kv"].to(dev)), c["tables"].to(dev), qs.to(dev),
        torch.tensor(c["lens"], dtype=torch.int32, device=dev), c["scale"], out, max_query_len=max(c["chunks"]),
        max_context_len=max(c["lens"]), softcap=softcap, slopes=put(slopes), window=window, starts=put(starts),
        prefix_lens=put(prefix), kv_splits=splits)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    out = out.cpu()
    assert (out[c["rows"]:] == 3.0).all()                                        # rows behind the last sequence
    return out


def check(c, out, softcap=0.0, slopes=None, window=0, starts=None, prefix=None, step=1):
    g, bs = c["hq"] // c["hkv"], c["bs"]
    p_half = 2.0 ** -11 if c["dtype"] == F16 else 2.0 ** -8
    for i, n in enumerate(c["lens"]):
        t = torch.arange(n)
        kv = c["kv"][c["tables"][i][t // bs].long(), :, :, t % bs]               # [n, 2, Hkv, d]
        js = sorted(set(range(0, c["chunks"][i], step)) | {c["chunks"][i] - 1} - {-1})
        for j in js:
            row, pos, lo, hi = bounds(c, i, j, window, starts, prefix)
            for hq in {0, g - 1, c["hq"] - 1, (j * 7) % c["hq"]}:
                k, v = kv[:, 0, hq // g], kv[:, 1, hq // g]
                slope = float(slopes[hq]) if slopes is not None else 0.0
                ref, _, absref = refs.attend_row(c["q"][row, hq], k, v, c["scale"], softcap, slope, pos, lo, hi)
                slack = refs.score_slack(c["q"][row, hq], k[lo:hi], c["scale"], softcap, slope, n)
                refs.check_attention(out[row, hq], ref, absref, slack, p_half, f"seq {i} row {j} head {hq}")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("splits", [0, 3])
@pytest.mark.parametrize("hq,hkv,bs", [(4, 4, 16), (8, 2, 32), (6, 2, 8), (16, 2, 16), (20, 1, 32)])
def test_all_forms_together(hq, hkv, bs, splits, dtype):
    dev = device()
    c = make([0, 300, 17, 130], [70, 45, 1, 200], hq, hkv, bs, dtype, seed=hq, extra_rows=3)
    g = torch.Generator().manual_seed(2)
    starts = torch.cat([torch.randint(0, n, (k,), generator=g) for n, k in zip(c["lens"], c["chunks"])]).to(torch.int32)
    starts[::5] = 0
    starts[3::11] = 10 ** 6                                                      # sees nothing
    starts[1::13] = -9
    prefix = torch.tensor([64, 310, 0, 1000], dtype=torch.int32)
    kw = dict(softcap=4.0, slopes=SLOPES(hq), window=150, starts=starts, prefix=prefix)
    out = run(dev, c, splits=splits, **kw)
    check(c, out, step=3, **kw)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("form", ["plain", "cap", "hard_cap", "slopes", "window", "starts", "prefix", "nothing"])
@pytest.mark.parametrize("hq,hkv,bs,cached,chunks", [
    (2, 2, 16, [0, 0], [257, 257]), (8, 2, 8, [513, 0, 100], [64, 129, 7]), (32, 1, 32, [40], [33])],
    ids=["whole", "ragged", "wide"])
def test_each_form_alone(hq, hkv, bs, cached, chunks, form, dtype):
    dev = device()
    c = make(cached, chunks, hq, hkv, bs, dtype, seed=5)
    rows = c["rows"]
    docs = torch.cat([torch.arange(a, a + k) // 50 * 50 for a, k in zip(cached, chunks)]).to(torch.int32)
    kw = dict(plain={}, cap=dict(softcap=30.0), hard_cap=dict(softcap=0.7), slopes=dict(slopes=SLOPES(hq)),
              window=dict(window=37), starts=dict(starts=docs), nothing=dict(starts=torch.full((rows,), 9999, dtype=torch.int32)),
              prefix=dict(prefix=torch.tensor([130, 60, 5][:len(chunks)], dtype=torch.int32)))[form]
    poison(c, kw.get("window", 0), kw.get("starts"), kw.get("prefix"))
    out = run(dev, c, **kw)
    if form == "nothing":
        assert (out == 0).all()
    else:
        check(c, out, step=5, **kw)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 127, 128, 129, 300])
@pytest.mark.parametrize("hq,hkv,bs,splits", [(2, 2, 32, 0), (8, 2, 16, 2), (12, 1, 8, 1)])
def test_window_borders(hq, hkv, bs, splits, window):
    dev = device()
    c = make([250, 251, 0], [70, 1, 140], hq, hkv, bs, BF16, seed=window)
    poison(c, window, None, None)
    check(c, run(dev, c, window=window, splits=splits), window=window, step=7)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("softcap,biased", [(5.0, False), (50.0, False), (100.0, False), (50.0, True), (0.0, True)])
@pytest.mark.parametrize("splits", [0, 2])
def test_one_visible_token_returns_its_value(splits, softcap, biased, dtype):
    """The weight's rounding is divided out again: P V / P, off by 2^-22 of itself at most, rounds back to V."""
    dev = device()
    c = make([0, 130, 37], [150, 3, 64], 8, 2, 16, dtype, 7)
    out = run(dev, c, softcap, SLOPES(8) if biased else None, 1, splits=splits).cpu()
    for i in range(3):
        for j in range(c["chunks"][i]):
            row, pos, _, _ = bounds(c, i, j, 1, None, None)
            v = c["kv"][c["tables"][i, pos // 16], 1, :, pos % 16]
            assert torch.equal(out[row], v.repeat_interleave(4, 0))


def test_documents_with_poison_before_them():
    """One sequence's rows all in its last document, whose start lies inside a block and a tile."""
    dev = device()
    for start in (1, 127, 128, 200, 255, 299):
        c = make([300], [64], 8, 2, 16, F16, seed=start)
        starts = torch.full((64,), start, dtype=torch.int32)
        poison(c, 0, starts, None)
        for splits in (0, 2):
            check(c, run(dev, c, starts=starts, splits=splits), starts=starts, step=9)


def test_a_single_token_equals_the_scored_decode():
    dev = device()
    c = make([700, 33, 0], [1, 1, 1], 8, 2, 16, BF16, seed=8)
    kw = dict(softcap=6.0, slopes=SLOPES(8), window=300)
    out = run(dev, c, **kw)
    check(c, out, **kw)
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=dev)
    dec = pkv.paged_attention_decode_scored(c["q"].to(dev), *pkv.split_pool(c["kv"].to(dev)), c["tables"].to(dev), lens,
                                            c["scale"], softcap=6.0, slopes=kw["slopes"].to(dev), window=300,
                                            max_context_len=701).cpu()
    # both are within the reference's bound: twice one side's for each, and the final roundings of both
    assert (out.float() - dec.float()).abs().max() <= 4 * 2.0 ** -8 * 4


def test_many_sequences_and_a_long_chunk():
    """More than 32 sequences (the row-tile order), and a chunk of many row tiles behind a long context (sorted groups)."""
    dev = device()
    c = make([5 * i for i in range(37)], [3 + i % 7 for i in range(37)], 4, 2, 16, BF16, seed=9)
    kw = dict(softcap=20.0, window=90)
    check(c, run(dev, c, **kw), step=2, **kw)
    c = make([1500, 200], [700, 911], 16, 2, 16, F16, seed=10)
    kw = dict(softcap=50.0, slopes=SLOPES(16), window=600, prefix=torch.tensor([0, 300], dtype=torch.int32))
    check(c, run(dev, c, **kw), step=41, **kw)


def test_bad_lengths_and_entries_are_flagged():
    dev = device()
    c = make([40, 40], [10, 10], 4, 2, 16, F16, seed=5)
    c["tables"][0, 2] = 10 ** 6
    qs = torch.tensor([0, 10, 20], dtype=torch.int32, device=dev)
    out = torch.full_like(c["q"], 3.0).to(dev)
    call = lambda lens, qs: pkv.paged_attention_prefill_scored(
        c["q"].to(dev), *pkv.split_pool(c["kv"].to(dev)), c["tables"].to(dev), qs, lens, c["scale"], out, max_query_len=10,
        max_context_len=50, softcap=3.0)
    call(torch.tensor([50, 50], dtype=torch.int32, device=dev), qs)
    assert pkv.get_device_error(dev)[1] == ["block_table"]
    out.fill_(3.0)
    call(torch.tensor([51, 9], dtype=torch.int32, device=dev), qs)
    assert pkv.get_device_error(dev)[1] == ["context_len"] and (out == 3.0).all()


@pytest.mark.parametrize("splits", [0, 2])
def test_captured_and_replayed(splits):
    dev = device()
    c = make([100, 0], [50, 130], 8, 2, 16, BF16, seed=6)
    qs = torch.tensor([0, 50, 180], dtype=torch.int32, device=dev)
    q = c["q"].to(dev)
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=dev)
    call = pkv.prepare_paged_attention_prefill_scored(
        q, *pkv.split_pool(c["kv"].to(dev)), c["tables"].to(dev), qs, lens, max_query_len=130, max_context_len=150,
        softcap=8.0, window=77, kv_splits=splits)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    c["q"] = (c["q"].float() * 0.5).to(BF16)
    c["lens"], c["chunks"] = [149, 130], [50, 130]                      # other lengths at replay
    q.copy_(c["q"])
    lens.copy_(torch.tensor(c["lens"], dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    check(c, call.result.cpu(), softcap=8.0, window=77, step=7)


def test_two_streams_at_once():
    """Two prepared calls on two streams, each with its own item table."""
    dev = device()
    calls, want = [], []
    for seed, kw in ((1, dict(softcap=20.0)), (2, dict(window=300))):
        c = make([400, 0, 77], [300, 211, 64], 8, 2, 16, BF16, seed=seed)
        qs = torch.tensor([0, 300, 511, 575], dtype=torch.int32, device=dev)
        call = pkv.prepare_paged_attention_prefill_scored(
            c["q"].to(dev), *pkv.split_pool(c["kv"].to(dev)), c["tables"].clamp(min=0).to(dev), qs,
            torch.tensor(c["lens"], dtype=torch.int32, device=dev), max_query_len=300, max_context_len=700, **kw)
        call()
        torch.cuda.synchronize()
        check(c, call.result.cpu(), step=50, **kw)
        want.append(call.result.clone())
        calls.append(call)
    streams = [torch.cuda.Stream(dev) for _ in calls]
    for call in calls:
        call.result.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, call in zip(streams, calls):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    for call, w in zip(calls, want):
        assert torch.equal(call.result, w)


def test_more_row_tiles_than_the_item_table_holds():
    dev = device()
    n = 70
    c = make([3 * i for i in range(n)], [1 + i % 9 for i in range(n)], 2, 2, 16, F16, seed=12)
    wide = torch.full((n, 512), -7, dtype=torch.int32)
    wide[:, :c["tables"].shape[1]] = c["tables"]
    qs = torch.tensor([0] + c["chunks"], dtype=torch.int32).cumsum(0).to(torch.int32)
    kw = dict(softcap=20.0, window=50)
    args = (c["q"].to(dev), *pkv.split_pool(c["kv"].to(dev)), wide.to(dev), qs.to(dev),
            torch.tensor(c["lens"], dtype=torch.int32, device=dev), c["scale"])
    assert pkv.prefill_scored_workspace_bytes(c["rows"], n, 2, 2, 128, 16, 8192, 8192, 50) == 0
    out = pkv.paged_attention_prefill_scored(*args, max_query_len=8192, max_context_len=8192, **kw)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    check(c, out.cpu(), **kw)


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("softcap", [55.0, 60.0])
def test_every_score_at_the_cap(sign, softcap):
    """All scores at +cap or -cap (the weights' extremes for a fixed reference, and just past it), and large values."""
    dev = device()
    c = make([200], [150], 4, 2, 16, BF16, seed=3)
    c["kv"][:, 0] = torch.rand_like(c["kv"][:, 0].float()).add(1).mul(3).to(BF16)
    c["q"] = (torch.rand_like(c["q"].float()).add(1) * 20 * sign).to(BF16)
    c["kv"][:, 1] = (c["kv"][:, 1].float() * 1e18).to(BF16)
    for splits in (0, 2):
        check(c, run(dev, c, softcap=softcap, splits=splits), softcap=softcap, step=11)


def _alone(c):
    """The first sequence of a case by itself, over the same pool."""
    return dict(c, lens=c["lens"][:1], chunks=c["chunks"][:1], tables=c["tables"][:1], rows=c["chunks"][0],
                q=c["q"][:c["chunks"][0]])


@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("softcap", [8.0, 30.0, 1e3, 1e4])
def test_capped_rows_do_not_depend_on_their_neighbours(softcap, dtype):
    """Bit for bit: a sequence whose chunk ends inside a row tile, alone and packed before one whose queries are 100 times
    larger; rows beside a row with large queries; rows before a token with large keys."""
    dev = device()
    c = make([200, 0], [37, 64], 8, 2, 16, dtype, seed=13)
    first = run(dev, _alone(c), softcap=softcap, splits=1)
    packed = dict(c, q=torch.cat([c["q"][:37], (c["q"][37:].float() * 100).to(dtype)]))
    assert torch.equal(run(dev, packed, softcap=softcap, splits=1)[:37], first)
    loud = c["q"].clone()
    loud[11:20:4] = (loud[11:20:4].float() * 100).to(dtype)
    others = [j for j in range(37) if j not in range(11, 20, 4)]
    assert torch.equal(run(dev, _alone(dict(c, q=loud)), softcap=softcap, splits=1)[others], first[others])
    kv = c["kv"].clone()
    for t in (215, 230):
        kv[c["tables"][0, t // 16], 0, :, t % 16] *= 200
    got = run(dev, _alone(dict(c, kv=kv)), softcap=softcap, splits=1)
    assert torch.equal(got[:15], first[:15])                                     # positions 200 .. 214
    check(_alone(dict(c, kv=kv)), got, softcap=softcap, step=5)


@pytest.mark.parametrize("scale,softcap", [(-2.0, 0.0), (0.0, 0.0), (8.0, 0.0), (-2.0, 3.0), (0.0, 2.0), (8.0, 3.0), (0.3, 1e6)])
@pytest.mark.parametrize("biased", [False, True])
def test_scales_of_any_sign_and_size(scale, softcap, biased):
    dev = device()
    kw = dict(softcap=softcap, slopes=SLOPES(4) if biased else None)
    for dtype in (F16, BF16):
        c = make([130, 0], [40, 70], 4, 2, 16, dtype, seed=17)
        c["scale"] = scale
        check(c, run(dev, c, **kw), step=7, **kw)


@pytest.mark.parametrize("part", [0.2, 0.4, 0.6, 0.74, 3.0])
@pytest.mark.parametrize("scale,softcap", [(8.0, 1e-3), (-8.0, 1e-3), (60.0, 1e-2), (-2.0, 1e-3), (1e-6, 1e6)])
def test_scores_at_every_part_of_extreme_caps(scale, softcap, part):
    """The largest |score / softcap| before the cap is `part`, for caps whose ratio to the scale is extreme."""
    dev = device()
    c = make([100], [150], 4, 2, 16, BF16, seed=19)
    c["scale"] = scale
    k = c["kv"][c["tables"][0].long()][:, 0].double().permute(1, 0, 2, 3).reshape(2, -1, 128)[:, :250]
    most = torch.einsum("rhgd,htd->rhgt", c["q"].double().view(150, 2, 2, 128), k).abs().max().item()
    c["q"] = (c["q"].double() * (part * softcap / abs(scale) / most)).to(BF16)
    check(c, run(dev, c, softcap=softcap), softcap=softcap, step=9)


@pytest.mark.parametrize("softcap,sign,size", [(c, *x) for c in (30.0, 50.0, 55.0) for x in (
    (-1, 1.0), (-1, 1e-4), (-1, 1e-8), (1, 1.0), (1, 1e18))] + [(51.9, -1, 1e-6), (51.9, 1, 1e17)])
def test_every_score_at_a_cap_and_values_of_any_size(softcap, sign, size):
    """All scores at -cap: the smallest weights of a fixed reference, whose products with small values still count in full; at
    +cap the largest, whose products with large values stay finite.  Every token has the same value, and so has the output: the
    weights' roundings are divided out, and the sums' (350 of 2^-23) round back."""
    dev = device()
    c = make([200], [150], 4, 2, 16, BF16, seed=3)
    c["kv"][:, 0] = torch.rand_like(c["kv"][:, 0].float()).add(1).mul(3).to(BF16)
    c["q"] = (torch.rand_like(c["q"].float()).add(1) * 20 * sign).to(BF16)
    value = torch.randn((2, 128), generator=torch.Generator().manual_seed(2))
    value = (value.sign() * value.abs().clamp(0.5, 2.0) * size).to(BF16)
    c["kv"][:, 1] = value[None, :, None]
    for splits in (0, 2):
        out = run(dev, c, softcap=softcap, splits=splits)
        assert torch.equal(out[:150], value.repeat_interleave(2, 0).expand(150, 4, 128))
