"""The operators around plain attention refuse what their contracts exclude, on the host: the C ABI before any CUDA
call, the binding before the library."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from paged_kv_cache_155_gb300 import _build
from paged_kv_cache_155_gb300.block_manager import BlockManager, OutOfBlocks

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    _build.build()
    from paged_kv_cache_155_gb300._lib import lib as load
    return load()


def _rope(lib, int8=False, **kw):
    a = dict(q=16, qs=512, k=16, ks=128, v=16, vs=128, pos=16, axes=1, axis=None, inv=16, rot=64, inter=0, slots=16, t=4,
             out=16, outs=512, kc=16, vc=16, nb=8, stride=2 * 2 * 16 * 64, hq=8, hkv=2, d=64, bs=16, sk=16, sv=16, dt=0)
    a.update(kw)
    head = [a[n] for n in ("q", "qs", "k", "ks", "v", "vs", "pos", "axes", "axis", "inv", "rot", "inter", "slots", "t", "out",
                           "outs", "kc", "vc", "nb", "stride", "hq", "hkv", "d", "bs")]
    if int8:
        return lib.pkv_rope_reshape_and_cache_int8(*head, a["sk"], a["sv"], a["dt"], None)
    return lib.pkv_rope_reshape_and_cache(*head, a["dt"], None)


@pytest.mark.parametrize("int8", [False, True])
def test_rope_refusals(lib, int8):
    call = lambda **kw: _rope(lib, int8, **kw)
    assert call(t=0) == 0
    for kw in (dict(d=96), dict(bs=4), dict(dt=2), dict(rot=24), dict(rot=8)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(rot=0), dict(rot=128), dict(axes=0), dict(axes=5), dict(t=-1), dict(hq=0), dict(hkv=0), dict(nb=0),
               dict(qs=504), dict(qs=516), dict(ks=120), dict(vs=132), dict(outs=0), dict(q=8), dict(out=24), dict(k=None),
               dict(pos=12), dict(inv=None), dict(slots=4), dict(axis=2), dict(kc=None), dict(vc=8), dict(stride=100),
               dict(stride=2 * 2 * 16 * 64 + 4)):
        assert call(**kw) == INVALID, kw
    if int8:
        assert call(sk=None) == INVALID and call(sv=8) == INVALID and call(stride=2 * 2 * 16 * 64 + 8) == INVALID


def _scored(lib, int8=False, **kw):
    a = dict(q=16, k=16, v=16, ks=16, vs=16, nb=64, stride=2 * 4 * 16 * 64, bt=16, mb=8, cl=16, maxl=100, b=4, hq=4, hkv=4, d=64,
             bs=16, scale=0.125, cap=0.0, slopes=None, window=0, starts=None, w=None, wo=None, ws=0, out=16, wk=None, wkb=0,
             part=128, dt=0)
    a.update(kw)
    head = [a[n] for n in ("nb", "stride", "bt", "mb", "cl", "maxl", "b", "hq", "hkv", "d", "bs", "scale", "cap", "slopes",
                           "window", "starts")]
    tail = [a[n] for n in ("out", "wk", "wkb", "part", "dt")] + [None]
    if int8:
        return lib.pkv_paged_attention_decode_scored_int8(a["q"], a["k"], a["v"], a["ks"], a["vs"], *head, *tail)
    return lib.pkv_paged_attention_decode_scored(a["q"], a["k"], a["v"], *head, a["w"], a["wo"], a["ws"], *tail)


@pytest.mark.parametrize("int8", [False, True])
def test_scored_decode_refusals(lib, int8):
    call = lambda **kw: _scored(lib, int8, **kw)
    assert call(b=0) == 0
    for kw in (dict(d=96), dict(bs=64), dict(dt=7)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(cap=-1.0), dict(cap=1e-9), dict(cap=1e9), dict(cap=float("nan")), dict(cap=float("inf")), dict(window=-1),
               dict(slopes=2), dict(starts=1), dict(hq=6), dict(maxl=129), dict(q=None), dict(out=8), dict(cl=None),
               dict(scale=float("inf")), dict(part=24), dict(part=64)):     # 64: two partitions and no workspace
        assert call(**kw) == INVALID, kw
    if not int8:
        for kw in (dict(w=16), dict(wo=16, ws=99), dict(wo=2, ws=100), dict(w=2, wo=16, ws=100), dict(wo=16, ws=100)):
            assert call(**kw) == INVALID, kw                                # the last: the weights need a workspace
        assert call(wo=16, ws=100, hq=4 * 129) == UNSUPPORTED
    size = lib.pkv_decode_scored_workspace_bytes
    assert size(4, 4, 4, 64, 16, 100, 0, 0, 0, 128) == 0
    assert size(4, 4, 4, 64, 16, 100, 40, 0, 0, 64) == 0                    # the window's 55 tokens fit one partition
    assert size(4, 4, 4, 64, 16, 100, 0, 1, 0, 128) == 4 * (4 * 4 * 66 + 4 * 4 * 128)
    assert size(4, 4, 4, 64, 16, 100, -1, 0, 0, 128) == 2 ** 64 - 1


def test_scored_decode_binding_refusals():
    kv = torch.zeros((8, 2, 2, 16, 64), dtype=torch.float16)
    k, v = pkv.split_pool(kv)
    q, bt, n = torch.zeros((2, 4, 64), dtype=torch.float16), torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    call = lambda *a, **kw: pkv.paged_attention_decode_scored(*a, max_context_len=64, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        call(q, k, v, bt, n)
    w = torch.zeros((2, 2, 64))
    for kw in (dict(softcap=-2.0), dict(window=-1), dict(slopes=torch.zeros(3)), dict(slopes=torch.zeros(4).double()),
               dict(starts=n[:1]), dict(starts=n.long()), dict(weights=w), dict(weights_out=w[:, :, :63]),
               dict(weights_out=w.double()), dict(weights=w, weights_out=torch.zeros((2, 2, 65))), dict(out=q.float())):
        with pytest.raises(ValueError):
            call(q, k, v, bt, n, **kw)
    for a in ((q.bfloat16(), k, v, bt, n), (q, k, v, bt.long(), n), (q, k, v, bt[:1], n), (q, k, v, bt, n.long())):
        with pytest.raises(ValueError):
            call(*a)


def test_scored_prefill_refusals(lib):
    def call(**kw):
        a = dict(q=16, k=16, v=16, nb=64, stride=2 * 4 * 16 * 128, bt=16, mb=8, qs=16, cl=16, rows=10, maxq=10, maxl=100, b=2,
                 hq=4, hkv=4, d=128, bs=16, scale=0.1, cap=0.0, slopes=None, window=0, starts=None, prefix=None, out=16, wk=None,
                 wkb=0, splits=1, dt=0)
        a.update(kw)
        names = ("q", "k", "v", "nb", "stride", "bt", "mb", "qs", "cl", "rows", "maxq", "maxl", "b", "hq", "hkv", "d", "bs",
                 "scale", "cap", "slopes", "window", "starts", "prefix", "out", "wk", "wkb", "splits", "dt")
        return lib.pkv_paged_attention_prefill_scored(*[a[n] for n in names], None)

    assert call(b=0) == 0 and call(rows=0) == 0
    for kw in (dict(d=64), dict(bs=64), dict(dt=2)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(cap=-1.0), dict(cap=1e-9), dict(cap=float("nan")), dict(window=-1), dict(slopes=2), dict(starts=1),
               dict(prefix=3), dict(hq=6), dict(maxl=129), dict(maxq=101), dict(q=None), dict(out=8), dict(qs=None),
               dict(scale=float("nan")), dict(splits=-1), dict(mb=64, maxl=1000, splits=2)):  # the last: no workspace
        assert call(**kw) == INVALID, kw
    size = lib.pkv_prefill_scored_workspace_bytes
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 0, 0, 2) == 10 * 4 * 2 * 130 * 4
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 0, 0, 1) == 16 + 2 * 32          # an item table of one row tile a sequence
    assert size(10 ** 6, 100, 4, 4, 128, 16, 10000, 10000, 0, 0, 1) == 0         # too many row tiles for a table
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 100, 0, 8) == 10 * 4 * 2 * 130 * 4   # 100 + 127 + 15 tokens: two tiles
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 100, 1, 8) == 10 * 4 * 8 * 130 * 4
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, -1, 0, 1) == 2 ** 64 - 1


def test_scored_prefill_binding_refusals():
    kv = torch.zeros((8, 2, 2, 16, 128), dtype=torch.float16)
    k, v = pkv.split_pool(kv)
    q, bt = torch.zeros((6, 4, 128), dtype=torch.float16), torch.zeros((2, 4), dtype=torch.int32)
    qs, n = torch.tensor([0, 3, 6], dtype=torch.int32), torch.tensor([3, 3], dtype=torch.int32)
    call = lambda *a, **kw: pkv.paged_attention_prefill_scored(*a, max_query_len=3, max_context_len=64, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        call(q, k, v, bt, qs, n)
    for kw in (dict(softcap=-2.0), dict(window=-1), dict(slopes=torch.zeros(3)), dict(starts=n), dict(prefix_lens=qs),
               dict(starts=torch.zeros(6)), dict(out=q.float())):
        with pytest.raises(ValueError):
            call(q, k, v, bt, qs, n, **kw)
    for a in ((q.bfloat16(), k, v, bt, qs, n), (q, k, v, bt, n, n), (q, k, v, bt[:1], qs, n), (q, k, v, bt, qs, n.long())):
        with pytest.raises(ValueError):
            call(*a)


def test_evict_refusals(lib):
    def select(**kw):
        a = dict(w=16, ws=64, cl=16, maxl=64, b=2, hkv=2, budget=8, sinks=1, recent=2, wo=None, kept=16, kl=16)
        a.update(kw)
        return lib.pkv_evict_select(a["w"], a["ws"], a["cl"], a["maxl"], a["b"], a["hkv"], a["budget"], a["sinks"],
                                    a["recent"], a["wo"], a["kept"], a["kl"], None)

    assert select(b=0) == 0
    for kw in (dict(budget=0), dict(sinks=7), dict(sinks=-1), dict(recent=-1), dict(recent=2 ** 31 - 1, budget=2 ** 31 - 1),
               dict(ws=63), dict(budget=2 ** 30 + 1), dict(ws=2 ** 31, maxl=2 ** 30 + 1), dict(b=-1), dict(b=70000), dict(hkv=0), dict(maxl=-1), dict(w=None), dict(kept=2), dict(kl=None),
               dict(wo=2)):
        assert select(**kw) == INVALID, kw

    def compact(**kw):
        a = dict(kc=16, vc=16, nb=8, stride=2 * 2 * 16 * 64, hkv=2, d=64, bs=16, bt=16, mb=4, cl=16, b=2, kept=16, kl=16,
                 budget=8, dst=32, dmb=2, dt=0)
        a.update(kw)
        return lib.pkv_evict_compact(a["kc"], a["vc"], a["nb"], a["stride"], a["hkv"], a["d"], a["bs"], a["bt"], a["mb"],
                                     a["cl"], a["b"], a["kept"], a["kl"], a["budget"], a["dst"], a["dmb"], a["dt"], None)

    assert compact(b=0) == 0
    for kw in (dict(d=80), dict(bs=12), dict(dt=3)):
        assert compact(**kw) == UNSUPPORTED, kw
    for kw in (dict(nb=0), dict(mb=0), dict(budget=0), dict(budget=2 ** 30 + 1), dict(dmb=0), dict(bt=None), dict(cl=2), dict(kept=None), dict(kl=1),
               dict(dst=18), dict(kc=8), dict(vc=None), dict(stride=64), dict(hkv=0), dict(b=-1), dict(b=70000),
               dict(dst=16, dmb=3)):
        assert compact(**kw) == INVALID, kw


def test_binding_refuses_before_the_library():
    kv = torch.zeros((4, 2, 2, 16, 64), dtype=torch.float16)
    k, v = pkv.split_pool(kv)
    q, kn = torch.zeros((3, 4, 64), dtype=torch.float16), torch.zeros((3, 2, 64), dtype=torch.float16)
    good = dict(positions=torch.zeros(3, dtype=torch.int64), inv_freq=torch.ones(32, dtype=torch.float64),
                slot_mapping=torch.zeros(3, dtype=torch.int64))

    def rope(q=q, kn=kn, vn=kn, **kw):
        a = dict(good)
        extra = {n: kw.pop(n) for n in list(kw) if n not in a}
        a.update(kw)
        return pkv.rope_reshape_and_cache(q, kn, vn, a["positions"], a["inv_freq"], a["slot_mapping"], k, v, **extra)

    with pytest.raises(ValueError, match="CUDA"):
        rope()                                              # host tensors
    for kw in (dict(q=q.float()), dict(q=q[:2]), dict(q=q.transpose(1, 2)), dict(kn=kn[:, :1]), dict(vn=kn.bfloat16()),
               dict(positions=torch.zeros(3)), dict(positions=torch.zeros((2, 4), dtype=torch.int64)),
               dict(inv_freq=torch.ones(32)), dict(slot_mapping=torch.zeros(2, dtype=torch.int64)),
               dict(axis_of_pair=torch.zeros(32)), dict(axis_of_pair=torch.zeros(31, dtype=torch.int32)),
               dict(q_out=torch.zeros((3, 4, 64)))):
        with pytest.raises(ValueError):
            rope(**kw)
    w, n = torch.zeros((2, 2, 64)), torch.tensor([5, 64], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.evict_select(w, n, 8)
    for kw in (dict(budget=0), dict(budget=4, sinks=3, recent=2), dict(budget=8, max_context_len=65),
               dict(budget=8, weights_out=torch.zeros((2, 2, 63))), dict(budget=8, kept=torch.zeros((2, 2, 7)))):
        with pytest.raises(ValueError):
            pkv.evict_select(w, n, **kw)
    with pytest.raises(ValueError):
        pkv.evict_select(w.double(), n, 8)
    kept = torch.zeros((2, 2, 8), dtype=torch.int32)
    bt = torch.zeros((2, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.evict_compact(k, v, bt, n, kept, n)
    for args in ((bt.long(), n, kept, n), (bt, n[:1], kept, n), (bt, n, kept[:, :1], n), (bt, n, kept, n.long())):
        with pytest.raises(ValueError):
            pkv.evict_compact(k, v, *args)
    with pytest.raises(ValueError):
        pkv.evict_compact(k, v, bt, n, kept, n, dst_block_tables=bt[:1])


def test_new_lengths_over_the_old_ones_are_refused(lib):
    """One KV head writes a sequence's new length while the others may still read the old one."""
    buf = np.zeros(64, dtype=np.int32)
    at = buf.ctypes.data
    call = lambda cl, kl, b=4: lib.pkv_evict_select(at, 64, cl, 64, b, 2, 8, 1, 2, None, at + 128, kl, None)
    for cl, kl in ((at, at), (at, at + 12), (at + 12, at)):
        assert call(cl, kl) == INVALID
    assert call(at, at, b=0) == 0
    w, n = torch.zeros((2, 2, 64)), torch.tensor([5, 64, 7], dtype=torch.int32)
    for lens, kept_lens in ((n[:2], n[:2]), (n[:2], n[1:])):
        with pytest.raises(ValueError, match="overlap"):
            pkv.evict_select(w, lens, 8, kept_lens=kept_lens)


def test_integers_past_32_bits_are_refused_not_cut():
    k, v = pkv.split_pool(torch.zeros((8, 2, 2, 16, 128), dtype=torch.float16))
    q, bt, n = torch.zeros((2, 4, 128), dtype=torch.float16), torch.zeros((2, 4), dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    qs = torch.tensor([0, 1, 2], dtype=torch.int32)
    far = 2 ** 32 + 5
    for kw in (dict(window=far), dict(partition_size=2 ** 32), dict(max_context_len=far)):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_attention_decode_scored(q, k, v, bt, n, **{"max_context_len": 64, **kw})
    for kw in (dict(window=far), dict(kv_splits=2 ** 32 + 1), dict(max_context_len=far), dict(max_query_len=far)):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.paged_attention_prefill_scored(q, k, v, bt, qs, n, **{"max_context_len": 64, "max_query_len": 1, **kw})
    for kw in (dict(budget=far), dict(budget=8, max_context_len=far)):
        with pytest.raises(ValueError, match="32 bits"):
            pkv.evict_select(torch.zeros((2, 2, 64)), n, **kw)


def test_block_manager_make_private_and_truncate():
    bm = BlockManager(10, 4, 8)
    bm.add_sequence(1)
    for _ in range(18):
        bm.append_token(1)
    old = bm.block_table(1)
    assert len(bm.make_private(1, 18)) == 0                 # nothing shared
    bm.fork(1, 2)
    with pytest.raises(ValueError):
        BlockManager(0, 4, 8)
    pairs = bm.make_private(1, 9)                           # three of the five shared blocks
    assert pairs[:, 0].tolist() == old[:3]
    assert bm.block_table(1) == pairs[:, 1].tolist() + old[3:]
    assert [bm.refcount(b) for b in old] == [1, 1, 1, 2, 2] and bm.num_free == 2
    assert len(bm.make_private(1, 9)) == 0
    bm.fork(2, 3)
    with pytest.raises(OutOfBlocks):
        bm.make_private(2, 18)                              # five copies, two blocks free
    assert bm.block_table(2) == old and bm.num_free == 2    # nothing changed
    bm.truncate(1, 9)
    assert bm.seq_len(1) == 9 and len(bm.block_table(1)) == 3 and bm.refcount(old[4]) == 2
    bm.truncate(1, 9)
    bm.truncate(1, 8)
    assert len(bm.block_table(1)) == 2 and bm.num_free == 3
    slot, pair = bm.append_token(1)                         # grows again from the cut
    assert pair == (-1, -1) and slot % 4 == 0 and bm.seq_len(1) == 9
    bm.truncate(1, 0)
    assert bm.block_table(1) == [] and bm.num_free == 5
    for bad in (-1, 1):
        with pytest.raises(Exception):
            bm.truncate(1, bad)
        with pytest.raises(Exception):
            bm.make_private(1, bad)
    with pytest.raises(Exception):
        bm.truncate(99, 0)
    n = ctypes.c_int64()
    assert bm._lib.pkv_bm_make_private(bm._h, 2, 4, None, ctypes.byref(n)) == INVALID
    assert bm._lib.pkv_bm_make_private(bm._h, 2, 0, None, ctypes.byref(n)) == 0 and n.value == 0
    bm.free_sequence(2)
    bm.free_sequence(3)
    bm.free_sequence(1)
    assert bm.num_free == 10
    assert isinstance(pairs, np.ndarray)


def test_a_prepared_call_passes_the_same_values_converted(lib):
    """From its second call on a prepared call passes the ctypes values of its arguments: a call of no tokens, by both."""
    args = (1 << 20, 4096, 1 << 21, 1024, 1 << 40, 1024, 1 << 23, 3, None, 1 << 25, 128, True, 1 << 26, 0, 1 << 27, 4096,
            1 << 28, 1 << 29, 100, 65536, 32, 8, 128, 16, 0)
    call = pkv.ops.PreparedCall("pkv_rope_reshape_and_cache", args, torch.device("cuda", 0), ())
    typed = call._typed_args()
    assert [t.value for t in typed] == list(args)
    assert lib.pkv_rope_reshape_and_cache(*args, 0) == lib.pkv_rope_reshape_and_cache(*typed, 0) == 0
