"""The 4-bit cache, windows with first tokens and drafted trees refuse what their contracts exclude, on the host: the C ABI
before any CUDA call, the binding before the library."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from paged_kv_cache_155_gb300 import _build

INVALID, UNSUPPORTED, NONE = 1, 2, 2 ** 64 - 1
I32 = torch.int32


@pytest.fixture(scope="module")
def lib():
    _build.build()
    from paged_kv_cache_155_gb300._lib import lib as load
    return load()


def caller(fn, names, good):
    def call(**kw):
        a = {**good, **kw}
        assert set(a) == set(names.split())
        return fn(*[a[n] for n in names.split()], None)
    return call


def refuses(call, unsupported, invalid):
    for kw in unsupported:
        assert call(**kw) == UNSUPPORTED, kw
    for kw in invalid:
        assert call(**kw) == INVALID, kw


def test_int4_write(lib):
    rec = 4 * 16 * 40                                            # four heads' records of blocks of 16, head_dim 64
    call = caller(lib.pkv_reshape_and_cache_int4, "k v slots t kc vc nb stride hkv d bs dt",
                  dict(k=16, v=16, slots=16, t=3, kc=16, vc=16, nb=8, stride=2 * rec, hkv=4, d=64, bs=16, dt=0))
    assert call(t=0) == 0
    refuses(call, [dict(d=96), dict(d=256), dict(bs=4), dict(bs=64), dict(dt=2), dict(dt=pkv.INT4)],
            [dict(t=-1), dict(t=2 ** 40), dict(t=2 ** 29), dict(hkv=0), dict(hkv=65536, stride=2 ** 30), dict(nb=0), dict(k=None),
             dict(v=8), dict(slots=12), dict(slots=None), dict(kc=None), dict(vc=24), dict(stride=rec - 16), dict(stride=rec + 8)])


def test_int4_read_back(lib):
    rec, half = 4 * 16 * 80, 4 * 16 * 128
    call = caller(lib.pkv_dequantise_blocks_int4, "k4 v4 nb4 s4 pairs n kc vc nb stride hkv d bs dt",
                  dict(k4=16, v4=16, nb4=8, s4=2 * rec, pairs=16, n=2, kc=16, vc=16, nb=8, stride=2 * half, hkv=4, d=128, bs=16, dt=1))
    assert call(n=0) == 0
    refuses(call, [dict(d=80), dict(bs=12), dict(dt=2)],
            [dict(n=-1), dict(n=2 ** 31), dict(hkv=0), dict(nb4=0), dict(nb=0), dict(k4=None), dict(v4=8), dict(kc=8), dict(vc=None),
             dict(pairs=None), dict(pairs=20), dict(s4=rec - 16), dict(s4=2 * rec + 8), dict(stride=half - 8), dict(stride=2 * half + 4)])


def test_int4_decode(lib):
    rec = 2 * 16 * 80
    call = caller(lib.pkv_paged_attention_decode_int4, "q k v nb stride bt mb cl maxl b hq hkv d bs scale out wk wkb dt",
                  dict(q=16, k=16, v=16, nb=64, stride=2 * rec, bt=16, mb=8, cl=16, maxl=100, b=4, hq=8, hkv=2, d=128, bs=16,
                       scale=0.1, out=16, wk=16, wkb=1 << 40, dt=0))
    assert call(b=0) == 0
    refuses(call, [dict(d=96), dict(bs=64), dict(dt=2), dict(dt=pkv.INT4)],
            [dict(b=-1), dict(hq=7), dict(hq=0), dict(hkv=0), dict(nb=0), dict(nb=2 ** 31), dict(mb=0), dict(maxl=-1), dict(maxl=129),
             dict(scale=float("nan")), dict(stride=rec - 16), dict(stride=2 * rec + 8), dict(q=None), dict(out=8), dict(k=8),
             dict(v=None), dict(bt=None), dict(cl=2), dict(wk=None), dict(wk=8), dict(b=2 ** 30, mb=2 ** 20, maxl=2 ** 20)])
    size = lib.pkv_decode_int4_workspace_bytes
    assert size(4, 7, 2, 128, 16, 100) == NONE and size(4, 8, 2, 100, 16, 100) == NONE and size(-1, 8, 2, 128, 16, 100) == NONE


def test_copy_blocks_of_a_4_bit_cache(lib):
    rec = 3 * 8 * 40
    call = caller(lib.pkv_copy_blocks, "k v nb stride hkv d bs pairs n dt",
                  dict(k=16, v=16, nb=8, stride=2 * rec, hkv=3, d=64, bs=8, pairs=16, n=1, dt=pkv.INT4))
    assert call(n=0) == 0 and call(n=0, stride=rec) == 0
    refuses(call, [dict(dt=3), dict(dt=5), dict(dt=-1), dict(d=80)], [dict(stride=rec - 16), dict(stride=rec + 8), dict(pairs=None)])
    # the other calls on caches know no 4-bit one
    assert lib.pkv_reshape_and_cache(16, 16, 16, 1, 16, 16, 8, 2048, 1, 64, 8, pkv.INT4, None) == UNSUPPORTED
    assert lib.pkv_evict_compact(16, 16, 8, 4096, 1, 64, 8, 16, 4, 16, 2, 16, 16, 8, None, 0, pkv.INT4, None) == UNSUPPORTED


@pytest.mark.parametrize("int8", [False, True])
def test_sinks_decode(lib, int8):
    names = ("q k v ks vs" if int8 else "q k v") + " nb stride bt mb cl maxl b hq hkv d bs scale window sinks out wk wkb part dt"
    good = dict(q=16, k=16, v=16, nb=64, stride=2 * 4 * 16 * 64, bt=16, mb=8, cl=16, maxl=100, b=4, hq=4, hkv=4, d=64, bs=16,
                scale=0.125, window=20, sinks=4, out=16, wk=None, wkb=0, part=128, dt=0)
    if int8:
        good.update(ks=16, vs=16)
    call = caller(lib.pkv_paged_attention_decode_sinks_int8 if int8 else lib.pkv_paged_attention_decode_sinks, names, good)
    assert call(b=0) == 0
    refuses(call, [dict(d=96), dict(bs=64), dict(dt=7)],
            [dict(window=0), dict(window=-5), dict(sinks=-1), dict(hq=6), dict(maxl=129), dict(q=None), dict(out=8), dict(cl=None),
             dict(scale=float("inf")), dict(part=24), dict(part=32)])          # 32: two partitions and no workspace
    if int8:
        refuses(call, [], [dict(ks=None), dict(vs=8), dict(stride=2 * 4 * 16 * 64 + 8)])
    size = lib.pkv_decode_sinks_workspace_bytes
    assert size(4, 4, 4, 64, 16, 100, 20, 4, int(int8), 128) == 0
    assert size(4, 4, 4, 64, 16, 100, 20, 4, int(int8), 32) == 4 * 4 * 2 * 66 * 4  # 20 + 15 + 16 counted tokens
    assert size(4, 4, 4, 64, 16, 100, 0, 4, int(int8), 128) == NONE and size(4, 4, 4, 64, 16, 100, 20, -1, int(int8), 128) == NONE
    assert size(4, 4, 4, 64, 16, 100, 2 ** 31 - 1, 2 ** 31 - 1, int(int8), 128) == 0


def test_sinks_prefill(lib):
    call = caller(lib.pkv_paged_attention_prefill_sinks,
                  "q k v nb stride bt mb qs cl rows maxq maxl b hq hkv d bs scale window sinks out wk wkb splits dt",
                  dict(q=16, k=16, v=16, nb=64, stride=2 * 4 * 16 * 128, bt=16, mb=8, qs=16, cl=16, rows=10, maxq=10, maxl=100, b=2,
                       hq=4, hkv=4, d=128, bs=16, scale=0.1, window=9, sinks=3, out=16, wk=None, wkb=0, splits=1, dt=0))
    assert call(b=0) == 0 and call(rows=0) == 0
    refuses(call, [dict(d=64), dict(bs=64), dict(dt=2)],
            [dict(window=0), dict(sinks=-1), dict(hq=6), dict(maxl=129), dict(maxq=101), dict(q=None), dict(out=8), dict(qs=None),
             dict(scale=float("nan")), dict(splits=-1), dict()])                 # the last: the item table needs a workspace
    size = lib.pkv_prefill_sinks_workspace_bytes
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 100, 4, 1) == 16 + 2 * 32
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 100, 4, 8) == 10 * 4 * 3 * 130 * 4   # 100 + 127 + 15 + 16 tokens: three tiles
    assert size(10, 2, 4, 4, 128, 16, 10, 1000, 0, 4, 1) == NONE and size(10, 2, 4, 4, 128, 16, 10, 1000, 9, -1, 1) == NONE


def test_tree(lib):
    names = "q k v nb stride bt mb qs cl mask words rows maxq maxl b hq hkv d bs scale out wk wkb dt"
    call = caller(lib.pkv_paged_attention_tree, names,
                  dict(q=16, k=16, v=16, nb=64, stride=2 * 4 * 16 * 128, bt=16, mb=8, qs=16, cl=16, mask=16, words=1, rows=10, maxq=10,
                       maxl=100, b=2, hq=4, hkv=4, d=128, bs=16, scale=0.1, out=16, wk=16, wkb=1 << 40, dt=0))
    assert call(b=0) == 0 and call(rows=0) == 0 and call(maxq=0) == 0
    refuses(call, [dict(d=64), dict(bs=64), dict(dt=2), dict(hq=4 * 129)],
            [dict(hq=6), dict(maxl=129), dict(maxq=101), dict(maxq=65, words=1), dict(words=-1), dict(words=2 ** 21), dict(q=None),
             dict(out=8), dict(qs=None), dict(cl=18), dict(mask=None), dict(mask=12), dict(wk=None), dict(wk=24),
             dict(scale=float("nan")), dict(nb=2 ** 31), dict(stride=4 * 16 * 128 - 8), dict(rows=-1), dict(k=None), dict(v=8),
             dict(b=2 ** 28, mb=64, maxl=1024)])


def test_tree_commit(lib):
    call = caller(lib.pkv_tree_commit, "k v nb stride hkv d bs bt mb qs cl maxq maxl b path n most new dt",
                  dict(k=16, v=16, nb=64, stride=2 * 4 * 16 * 64, hkv=4, d=64, bs=16, bt=16, mb=8, qs=16, cl=64, maxq=10, maxl=100,
                       b=4, path=16, n=16, most=5, new=128, dt=2))
    assert call(b=0) == 0
    refuses(call, [dict(d=96), dict(bs=4), dict(dt=pkv.INT4)],
            [dict(b=-1), dict(b=65536), dict(hkv=0), dict(nb=0), dict(mb=0), dict(maxq=-1), dict(maxl=5), dict(maxl=129), dict(most=-1),
             dict(k=None), dict(v=8), dict(stride=100), dict(stride=2 * 4 * 16 * 64 + 8), dict(bt=None), dict(qs=2), dict(cl=None),
             dict(path=None), dict(n=None), dict(new=64), dict(new=76), dict(new=52), dict(new=129)])


def test_bindings():
    f16 = torch.float16
    q = torch.zeros((2, 4, 128), dtype=f16)
    bt, n, qs = torch.zeros((2, 4), dtype=I32), torch.ones(2, dtype=I32), torch.tensor([0, 1, 2], dtype=I32)
    k, v = pkv.split_pool(torch.zeros((8, 2, 2, 16, 128), dtype=f16))
    pool = pkv.int4_pool(8, 2, 16, 128)
    assert pool.shape == (8, 2, 2, 16, 80) and pool.dtype == torch.uint8
    with pytest.raises(ValueError):
        pkv.int4_pool(8, 2, 16, 96)
    k4, v4 = pkv.split_pool(pool)
    rows, slots, pairs = torch.zeros((3, 2, 128), dtype=f16), torch.zeros(3, dtype=torch.int64), torch.zeros((1, 2), dtype=torch.int64)
    far = 2 ** 32 + 5
    bound = dict(max_query_len=1, max_context_len=64)
    mask = torch.ones((2, 1), dtype=torch.int64)
    good = [
        lambda **kw: pkv.reshape_and_cache_int4(**{**dict(k_new=rows, v_new=rows, slot_mapping=slots, k_cache=k4, v_cache=v4), **kw}),
        lambda **kw: pkv.dequantise_blocks_int4(**{**dict(k_cache4=k4, v_cache4=v4, src_dst_pairs=pairs, k_cache=k, v_cache=v), **kw}),
        lambda **kw: pkv.paged_attention_decode_int4(**{**dict(q=q, k_cache=k4, v_cache=v4, block_tables=bt, context_lens=n,
                                                               max_context_len=64), **kw}),
        lambda **kw: pkv.paged_attention_decode_sinks(**{**dict(q=q, k_cache=k, v_cache=v, block_tables=bt, context_lens=n, window=5,
                                                                sinks=2, max_context_len=64), **kw}),
        lambda **kw: pkv.paged_attention_prefill_sinks(**{**dict(q=q, k_cache=k, v_cache=v, block_tables=bt, query_start=qs,
                                                                 context_lens=n, window=5, sinks=2), **bound, **kw}),
        lambda **kw: pkv.paged_attention_tree(**{**dict(q=q, k_cache=k, v_cache=v, block_tables=bt, query_start=qs, context_lens=n,
                                                        tree_mask=mask), **bound, **kw}),
        lambda **kw: pkv.tree_commit(**{**dict(k_cache=k, v_cache=v, block_tables=bt, query_start=qs, context_lens=n,
                                               accepted=torch.zeros((2, 3), dtype=I32), accepted_lens=n.clone()), **bound, **kw}),
    ]
    for call in good:                       # everything is in contract but the device
        with pytest.raises(ValueError, match="CUDA"):
            call()
    bad = [
        [dict(k_new=rows[:, :1]), dict(v_new=rows.bfloat16()), dict(slot_mapping=slots.int()), dict(slot_mapping=slots[:2]),
         dict(k_cache=k, v_cache=v), dict(k_new=rows[:, :, :64], v_new=rows[:, :, :64])],
        [dict(src_dst_pairs=pairs.int()), dict(src_dst_pairs=pairs[0]), dict(k_cache=k[:, :1], v_cache=v[:, :1]), dict(k_cache4=k, v_cache4=v)],
        [dict(q=q[:, :, :64]), dict(block_tables=bt.long()), dict(block_tables=bt[:1]), dict(context_lens=n.long()), dict(out=q.bfloat16()),
         dict(k_cache=k, v_cache=v), dict(max_context_len=far)],
        [dict(window=0), dict(sinks=-1), dict(window=far), dict(sinks=far), dict(partition_size=far), dict(q=q.bfloat16()),
         dict(context_lens=n[:1]), dict(max_context_len=far)],
        [dict(window=0), dict(sinks=-1), dict(window=far), dict(sinks=far), dict(kv_splits=far), dict(max_query_len=far),
         dict(query_start=qs[:2]), dict(out=q[:1]), dict(q=q.bfloat16())],
        [dict(tree_mask=mask.int()), dict(tree_mask=mask[:1]), dict(tree_mask=mask[:, 0]), dict(max_query_len=65), dict(max_query_len=far),
         dict(query_start=qs.long()), dict(out=q.float())],
        [dict(accepted=torch.zeros((2, 3))), dict(accepted=torch.zeros((1, 3), dtype=I32)), dict(accepted_lens=n[:1]),
         dict(new_context_lens=n), dict(new_context_lens=n.long()), dict(max_context_len=far)],
    ]
    for call, cases in zip(good, bad):
        for kw in cases:
            with pytest.raises((ValueError, TypeError)) as e:
                call(**kw)
            assert "CUDA" not in str(e.value), kw
