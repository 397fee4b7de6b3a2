"""Rotary positions with the cache write, on the GPU, against the 64-bit reference.

Tolerance: the fraction of a turn (at most 1/2) is rounded to fp32, 2^-25 turns, times 2 pi
below 2^-22.3; sincospif adds less than 2^-23, so sine and cosine are off by less than 2^-21.5.
The two products and the sum add three roundings of 2^-24.  A value (|a| + |b| its pair's
magnitudes) is off by at most (|a| + |b|) * 2^-20 before its one rounding to 16 bits."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _operator_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -20


def _case(dev, tokens, hq, hkv, d, bs, dtype, axes, rot, seed, far=5000, packed=True, int8=False):
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * d + (16 if packed else 0)
    rows = torch.randn((tokens, width), generator=g).to(dtype)
    on = rows.to(dev)
    cut = lambda r: (r[:, :hq * d].unflatten(1, (hq, d)), r[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                     r[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d)))
    q, k, v = cut(on)
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (axes, tokens), generator=g)
    axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    nb = (tokens + bs - 1) // bs + 2
    slots = torch.randperm(nb * bs, generator=g)[:tokens]
    shape = (nb, 2, hkv, bs, d)
    kv = torch.randint(-127, 128, shape, generator=g, dtype=torch.int8) if int8 else torch.randn(shape, generator=g).to(dtype)
    return dict(q=q, k=k, v=v, host=cut(rows), pos=pos, axis=axis, inv=inv, slots=slots, kv=kv)


def _check(c, dev, interleaved, pos=None, axis=None, slots=None, in_place=False):
    pos = c["pos"] if pos is None else pos
    slots = c["slots"] if slots is None else slots
    kv = c["kv"].to(dev)
    before = kv.clone()
    k_cache, v_cache = pkv.split_pool(kv)
    q = c["q"].clone() if in_place else c["q"]
    out = pkv.rope_reshape_and_cache(q, c["k"], c["v"], pos.to(dev), c["inv"].to(dev), slots.to(dev), k_cache, v_cache,
                                     q if in_place else None, axis_of_pair=None if axis is None else axis.to(dev),
                                     interleaved=interleaved)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    ax = torch.zeros_like(c["axis"]) if axis is None else axis
    p2 = pos if pos.dim() == 2 else pos[None]
    hq, hk, hv = c["host"]
    ref, mag = refs.rotate(hq, p2, ax, c["inv"], interleaved)
    refs.rounded_close(out.cpu(), ref, mag * SLACK, "q")
    ref, mag = refs.rotate(hk, p2, ax, c["inv"], interleaved)
    bs = kv.shape[3]
    keep = slots >= 0
    blk, off = slots[keep] // bs, slots[keep] % bs
    got = kv.cpu()
    refs.rounded_close(got[blk, 0, :, off], ref[keep], mag[keep] * SLACK, "k")
    assert torch.equal(got[blk, 1, :, off], hv[keep])
    rest = torch.ones(kv.shape[0], bs, dtype=torch.bool)
    rest[blk, off] = False
    untouched = before.cpu().permute(0, 3, 1, 2, 4)[rest]
    assert torch.equal(got.permute(0, 3, 1, 2, 4)[rest], untouched)
    rot = 2 * len(c["inv"])
    assert torch.equal(out.cpu()[..., rot:], hq[..., rot:])      # copied, not rounded again
    return out


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens,hq,hkv,d,bs,axes,rot", [
    (1, 32, 8, 128, 16, 1, 128), (7, 32, 32, 64, 8, 2, 64), (37, 64, 8, 128, 32, 3, 128), (5, 4, 4, 64, 16, 4, 16),
    (65, 20, 4, 128, 16, 3, 96), (3, 1, 1, 128, 8, 2, 48), (11, 128, 2, 64, 32, 3, 32), (2, 129, 43, 128, 16, 2, 128)])
def test_rope_matches_the_reference(tokens, hq, hkv, d, bs, axes, rot, dtype, interleaved):
    dev = device()
    c = _case(dev, tokens, hq, hkv, d, bs, dtype, axes, rot, seed=tokens + rot)
    _check(c, dev, interleaved, axis=c["axis"])


def test_far_and_negative_positions_keep_their_angles():
    dev = device()
    c = _case(dev, 9, 8, 2, 128, 16, torch.bfloat16, 1, 128, seed=3, packed=False)
    pos = torch.tensor([0, -1, 1, 2 ** 20 + 1, 2 ** 24 + 3, -2 ** 24 - 1, 2 ** 30 + 7, 99999999, 2 ** 31 + 5])
    # angles up to 2^31 rad: inv_freq / 2 pi in 64 bits leaves 2^31 * 2^-53 turns, and so does the reference's product
    _check(c, dev, False, pos=pos)
    _check(c, dev, True, pos=pos[None].contiguous(), axis=torch.zeros(64, dtype=torch.int32))


def test_one_axis_in_place_and_skipped_tokens():
    dev = device()
    c = _case(dev, 12, 16, 4, 128, 16, torch.float16, 1, 128, seed=5, packed=False)
    slots = c["slots"].clone()
    slots[::3] = -1
    a = _check(c, dev, False, pos=c["pos"][0], slots=slots)
    b = _check(c, dev, False, pos=c["pos"][0], slots=slots, in_place=True)
    assert torch.equal(a, b)


@pytest.mark.parametrize("int8", [False, True], ids=["16bit", "int8"])
@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True)])
@pytest.mark.parametrize("tokens", [1300, 2049])
def test_an_odd_chunk_of_many_tokens(tokens, d, interleaved, int8):
    """Enough tokens for narrow blocks, and for two tokens per block with one in the last."""
    dev = device()
    c = _case(dev, tokens, 3, 1, d, 16, torch.bfloat16, 2, d, seed=10, int8=int8)
    if not int8:
        slots = c["slots"].clone()
        slots[5::11] = -1
        _check(c, dev, interleaved, axis=c["axis"], slots=slots)
        return
    sc = torch.full((1, d), 0.03)
    kv = c["kv"].to(dev)
    out = pkv.rope_reshape_and_cache_int8(c["q"], c["k"], c["v"], c["pos"].to(dev), c["inv"].to(dev), c["slots"].to(dev),
                                          *pkv.split_pool(kv), sc.to(dev), sc.to(dev), axis_of_pair=c["axis"].to(dev),
                                          interleaved=interleaved)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    ref, mag = refs.rotate(c["host"][0], c["pos"], c["axis"], c["inv"], interleaved)
    refs.rounded_close(out.cpu(), ref, mag * SLACK, "q")
    ref, mag = refs.rotate(c["host"][1], c["pos"], c["axis"], c["inv"], interleaved)
    code = kv.cpu()[c["slots"] // 16, 0, :, c["slots"] % 16].double()
    assert ((code - (ref / 0.03).clamp(-127, 127)).abs() <= 0.5 + mag * SLACK / 0.03 + 127 * 2.0 ** -22).all()


def test_rows_longer_than_one_step_and_no_tokens():
    dev = device()
    c = _case(dev, 3, 200, 100, 128, 8, torch.bfloat16, 2, 64, seed=6)
    _check(c, dev, True, axis=c["axis"])
    empty = _case(dev, 0, 4, 2, 64, 16, torch.float16, 1, 64, seed=7, packed=False)
    kv = empty["kv"].to(dev)
    out = pkv.rope_reshape_and_cache(empty["q"], empty["k"], empty["v"], empty["pos"].to(dev), empty["inv"].to(dev),
                                     empty["slots"].to(dev), *pkv.split_pool(kv))
    assert out.shape == (0, 4, 64)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
@pytest.mark.parametrize("tokens,hq,hkv,d,bs,rot", [(33, 8, 4, 128, 16, 128), (5, 4, 4, 64, 8, 32)])
def test_rope_int8_codes(tokens, hq, hkv, d, bs, rot, dtype, interleaved):
    """code * scale is within half a step of the exact value, or the code is clamped; the quotient carries the
    rotation's error and two fp32 roundings (division, |quotient| <= 127 near the clamp)."""
    dev = device()
    c = _case(dev, tokens, hq, hkv, d, bs, dtype, 2, rot, seed=tokens, int8=True)
    g = torch.Generator().manual_seed(1)
    ks, vs = ((torch.rand((hkv, d), generator=g) + 0.5) / 40 for _ in range(2))
    kv = c["kv"].to(dev)
    before = kv.cpu().clone()
    out = pkv.rope_reshape_and_cache_int8(c["q"], c["k"], c["v"], c["pos"].to(dev), c["inv"].to(dev),
                                          c["slots"].to(dev), *pkv.split_pool(kv), ks.to(dev), vs.to(dev),
                                          axis_of_pair=c["axis"].to(dev), interleaved=interleaved)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    ref, mag = refs.rotate(c["host"][0], c["pos"], c["axis"], c["inv"], interleaved)
    refs.rounded_close(out.cpu(), ref, mag * SLACK, "q")
    blk, off = c["slots"] // bs, c["slots"] % bs
    got = kv.cpu()
    kref, kmag = refs.rotate(c["host"][1], c["pos"], c["axis"], c["inv"], interleaved)
    vref = c["host"][2].double()
    for half, (ref, mag, sc) in enumerate(((kref, kmag, ks.double()), (vref, torch.zeros_like(vref), vs.double()))):
        code = got[blk, half, :, off].double()
        exact = (ref / sc).clamp(-127, 127)
        slack = mag * SLACK / sc + 127 * 2.0 ** -23
        assert ((code - exact).abs() <= 0.5 + slack).all()
    mask = torch.ones(kv.shape[0], bs, dtype=torch.bool)
    mask[blk, off] = False
    assert torch.equal(got.permute(0, 3, 1, 2, 4)[mask], before.permute(0, 3, 1, 2, 4)[mask])


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_int8_v_codes_are_the_plain_writes(dtype):
    """The V rows, and K rows at position 0, get reshape_and_cache_int8's codes exactly: ties, clamped values, infinities, NaN
    and extreme scales among them."""
    dev = device()
    t, hkv, d, bs = 64, 4, 64, 16
    g = torch.Generator().manual_seed(2)
    scale = (torch.rand((hkv, d), generator=g) + 0.5) / 20
    scale[0] = 0.125                                                 # exact quotients: every multiple of 1/16 a tie
    scale[1, ::3], scale[1, 1::3] = 1e-38, 3e38
    x = torch.randn((t, hkv, d), generator=g)
    x[:, 0] = torch.randint(-300, 300, (t, d), generator=g) / 16
    x[::5, 2], x[1::5, 2], x[2::7, 3] = float("inf"), -float("inf"), float("nan")
    x[3::7, 1] = 0.0
    if dtype == torch.bfloat16:
        x[4::7, 1] = 3e38
    x = x.to(dtype).to(dev)
    slots = torch.randperm(5 * bs, generator=g)[:t].to(dev)
    pools = [torch.zeros((5, 2, hkv, bs, d), dtype=torch.int8, device=dev) for _ in range(2)]
    sc = scale.to(dev)
    pkv.reshape_and_cache_int8(x, x, slots, *pkv.split_pool(pools[0]), sc, sc)
    fin = torch.nan_to_num(x.float(), nan=0.0, posinf=1.0, neginf=-1.0).to(dtype)      # a rotation mixes infinities into NaN
    pkv.rope_reshape_and_cache_int8(x[:, :1].contiguous(), x, x, torch.zeros(t, dtype=torch.int64, device=dev),
                                    torch.ones(16, dtype=torch.float64, device=dev), slots, *pkv.split_pool(pools[1]), sc, sc)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert torch.equal(pools[0][:, 1], pools[1][:, 1])
    kpools = [torch.zeros((5, 2, hkv, bs, d), dtype=torch.int8, device=dev) for _ in range(2)]
    pkv.reshape_and_cache_int8(fin, fin, slots, *pkv.split_pool(kpools[0]), sc, sc)
    pkv.rope_reshape_and_cache_int8(fin[:, :1].contiguous(), fin, fin, torch.zeros(t, dtype=torch.int64, device=dev),
                                    torch.ones(16, dtype=torch.float64, device=dev), slots, *pkv.split_pool(kpools[1]), sc, sc)
    torch.cuda.synchronize()
    assert torch.equal(kpools[0], kpools[1])


def test_bad_slots_and_axes_are_flagged_and_skipped():
    dev = device()
    c = _case(dev, 4, 4, 2, 64, 16, torch.float16, 2, 64, seed=8, packed=False)
    kv = c["kv"].to(dev)
    before = kv.clone()
    k_cache, v_cache = pkv.split_pool(kv)
    slots = torch.full((4,), kv.shape[0] * 16, dtype=torch.int64, device=dev)
    out = pkv.rope_reshape_and_cache(c["q"], c["k"], c["v"], c["pos"].to(dev), c["inv"].to(dev), slots, k_cache, v_cache,
                                     axis_of_pair=c["axis"].to(dev))
    _, names = pkv.get_device_error(dev)
    assert names == ["slot"] and torch.equal(kv, before)
    ref, mag = refs.rotate(c["host"][0], c["pos"], c["axis"], c["inv"], False)
    refs.rounded_close(out.cpu(), ref, mag * SLACK, "q")
    axis = torch.full((32,), 2, dtype=torch.int32, device=dev)
    out = pkv.rope_reshape_and_cache(c["q"], c["k"], c["v"], c["pos"].to(dev), c["inv"].to(dev), c["slots"].to(dev),
                                     k_cache, v_cache, axis_of_pair=axis)
    _, names = pkv.get_device_error(dev)
    assert names == ["rope_axis"] and torch.equal(out, c["q"])


def test_the_rotated_cache_serves_decode_on_a_side_stream_and_in_a_graph():
    """Rotate and write, then decode, captured once and replayed with new rows: the same as eager calls."""
    dev = device()
    c = _case(dev, 4, 8, 2, 128, 16, torch.bfloat16, 3, 128, seed=9, packed=False)
    kv = c["kv"].to(dev)
    k_cache, v_cache = pkv.split_pool(kv)
    tables = torch.arange(kv.shape[0], dtype=torch.int32, device=dev)[:1].expand(4, 1).contiguous()
    tables[:, 0] = torch.tensor([0, 1, 2, 0], dtype=torch.int32)
    lens = torch.tensor([5, 16, 1, 3], dtype=torch.int32, device=dev)
    slots = pkv.slot_mapping(tables, lens.long() - 1, 16, num_blocks=kv.shape[0])
    q, k, v = (c[n].clone() for n in "qkv")
    pos, inv, axis = c["pos"].to(dev), c["inv"].to(dev), c["axis"].to(dev)
    rope = pkv.prepare_rope_reshape_and_cache(q, k, v, pos, inv, slots, k_cache, v_cache, axis_of_pair=axis)
    attend = pkv.prepare_paged_attention_decode(rope.result, k_cache, v_cache, tables, lens, max_context_len=16)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        rope()
        attend()
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope()
        attend()
    for t in (q, k, v):
        t.copy_(torch.randn(t.shape, device=dev).to(t.dtype))
    graph.replay()
    torch.cuda.synchronize()
    replayed = attend.result.clone()
    rope()
    attend()
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert torch.equal(replayed, attend.result)
