"""Eviction on the GPU: the choice of the kept tokens and the move of their rows, exactly the reference's."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _operator_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu


def _weights(kind, shape, g):
    w = torch.rand(shape, generator=g)
    if kind == "tail":
        w = w ** 12
    elif kind == "ties":
        w = (w * 4).floor() / 4
    elif kind == "equal":
        w = torch.full(shape, 0.25)
    elif kind == "signed":
        w = torch.randn(shape, generator=g).round(decimals=1)
        w[w == 0] = -0.0
        w[..., ::5] = 0.0
    elif kind == "odd":
        w[..., 3::7] = float("nan")
        w[..., 4::11] = float("inf")
        w[..., 5::13] = -float("inf")
        w[..., 6::17] = 1e-42
    return w


def _select(dev, w, lens, budget, sinks, recent, max_len=None, in_place=False):
    ref, ref_lens = refs.select(w, lens, budget, sinks, recent)
    on = w.to(dev)
    out = on if in_place else torch.full_like(on, 7.0)
    kept, kept_lens = pkv.evict_select(on, torch.tensor(lens, dtype=torch.int32, device=dev), budget, sinks=sinks,
                                       recent=recent, max_context_len=max_len, weights_out=out)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert torch.equal(kept.cpu(), ref)
    assert torch.equal(kept_lens.cpu(), ref_lens)
    want = w.clone() if in_place else torch.full_like(w, 7.0)
    for i, n in enumerate(lens):
        m = int(ref_lens[i])
        want[i, :, :n] = 0.0
        want[i, :, :m] = w[i].gather(1, ref[i, :, :m].long())
    assert torch.equal(out.cpu().view(torch.int32), want.view(torch.int32))     # bits: NaN and -0 move too


@pytest.mark.parametrize("in_place", [False, True], ids=["out", "in_place"])
@pytest.mark.parametrize("kind", ["plain", "tail", "ties", "equal", "signed", "odd"])
@pytest.mark.parametrize("lens,budget,sinks,recent", [
    ([0, 1, 17, 100], 16, 2, 5), ([1024, 1023, 513], 256, 0, 0), ([300, 40, 299], 40, 40, 0), ([300, 77], 50, 10, 40),
    ([1025, 5000, 8192], 1000, 4, 100), ([8193, 1, 20000], 4097, 1, 64)])
def test_select_matches_the_reference(lens, budget, sinks, recent, kind, in_place):
    dev = device()
    g = torch.Generator().manual_seed(budget)
    w = _weights(kind, (len(lens), 3, max(lens) + 5), g)
    _select(dev, w, lens, budget, sinks, recent, in_place=in_place)


@pytest.mark.parametrize("kind", ["tail", "ties"])
def test_select_over_rows_longer_than_the_registers_hold(kind):
    dev = device()
    g = torch.Generator().manual_seed(1)
    lens = [70001, 32769, 5]
    w = _weights(kind, (3, 2, 70016), g)
    _select(dev, w, lens, 9000, 16, 1000, in_place=kind == "ties")


@pytest.mark.parametrize("budget,sinks,recent", [(40000, 3, 100), (39999, 0, 0), (12000, 5000, 7000), (12000, 0, 12000)])
@pytest.mark.parametrize("width", [40000, 40003])
def test_select_of_long_rows_that_stay_whole_or_leave_no_choice(budget, sinks, recent, width):
    dev = device()
    lens = [40000, 39999, 33000, 3]
    w = _weights("tail", (4, 2, width), torch.Generator().manual_seed(budget))
    for in_place in (False, True):
        _select(dev, w, lens, budget, sinks, recent, in_place=in_place)


@pytest.mark.parametrize("n", [9, 1000, 5001, 20000])
def test_select_of_weights_at_any_alignment(n):
    dev = device()
    flat = _weights("signed", (3 * n + 4,), torch.Generator().manual_seed(n)).to(dev)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    for at in range(4):
        w = flat[at:at + 3 * n].view(1, 3, n)
        kept, _ = pkv.evict_select(w, lens, n // 2, sinks=1, recent=2)
        torch.cuda.synchronize()
        ref, _ = refs.select(w.cpu(), [n], n // 2, 1, 2)
        assert torch.equal(kept.cpu(), ref)
    check_no_device_flags(dev)


@pytest.mark.parametrize("rows", [40, 60, 100, 200])
def test_select_of_many_long_rows(rows):
    """Enough rows past 8192 tokens for clusters of four and two and for one block each; a few rows are checked."""
    dev = device()
    g = torch.Generator().manual_seed(rows)
    lens = [9000 + 7 * i for i in range(rows // 4)]
    w = _weights("tail", (len(lens), 4, max(lens)), g)
    on = w.to(dev)
    kept, kept_lens = pkv.evict_select(on, torch.tensor(lens, dtype=torch.int32, device=dev), 3000, sinks=2, recent=50,
                                       weights_out=on)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert (kept_lens.cpu() == 3000).all()
    for i in (0, len(lens) // 2, len(lens) - 1):
        ref, _ = refs.select(w[i:i + 1], lens[i:i + 1], 3000, 2, 50)
        assert torch.equal(kept.cpu()[i], ref[0])
        assert torch.equal(on.cpu()[i, :, :3000], w[i].gather(1, ref[0].long())) and (on.cpu()[i, :, 3000:lens[i]] == 0).all()


@pytest.mark.parametrize("kind", ["tail", "ties"])
@pytest.mark.parametrize("seqs,heads,longest", [(10, 4, 41000), (10, 6, 33500), (20, 4, 25000), (50, 3, 17000)])
def test_select_in_place_of_rows_that_clusters_read_again(seqs, heads, longest, kind):
    """Clusters of four hold 32768 tokens of a row in registers, clusters of two 16384: longer rows, whose later batches are
    read again in each pass and as they are written; equal weights on both sides of the batches' borders."""
    dev = device()
    lens = [longest - 37 * i for i in range(seqs)]
    w = _weights(kind, (seqs, heads, longest), torch.Generator().manual_seed(longest))
    on = w.to(dev)
    kept, kept_lens = pkv.evict_select(on, torch.tensor(lens, dtype=torch.int32, device=dev), 12000, sinks=4, recent=300,
                                       weights_out=on)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert (kept_lens.cpu() == 12000).all()
    for i in (0, seqs // 2, seqs - 1):
        ref, _ = refs.select(w[i:i + 1], lens[i:i + 1], 12000, 4, 300)
        assert torch.equal(kept.cpu()[i], ref[0])
        assert torch.equal(on.cpu()[i, :, :12000], w[i].gather(1, ref[0].long())) and (on.cpu()[i, :, 12000:lens[i]] == 0).all()


def test_select_clamps_and_flags_bad_lengths():
    dev = device()
    w = torch.rand((2, 1, 64))
    kept, n = pkv.evict_select(w.to(dev), torch.tensor([-3, 90], dtype=torch.int32, device=dev), 8, max_context_len=64)
    _, names = pkv.get_device_error(dev)
    assert names == ["context_len"]
    ref, ref_n = refs.select(w, [0, 64], 8, 0, 0)
    assert torch.equal(kept.cpu(), ref) and torch.equal(n.cpu(), ref_n)


def _pool(g, nb, hkv, bs, d, dtype):
    shape = (nb, 2, hkv, bs, d)
    if dtype == torch.int8:
        return torch.randint(-127, 128, shape, generator=g, dtype=dtype)
    return torch.randn(shape, generator=g).to(dtype)


def _case(g, lens, budget, hkv, bs, d, dtype, spare=3):
    need = [-(-n // bs) for n in lens]
    fresh = [-(-min(n, budget) // bs) for n in lens]
    total = sum(need) + sum(fresh) + spare
    perm = torch.randperm(total, generator=g).to(torch.int32)
    tables = torch.zeros((len(lens), max(need + [1])), dtype=torch.int32)
    dst = torch.zeros((len(lens), max(fresh + [1])), dtype=torch.int32)
    at = 0
    for i in range(len(lens)):
        tables[i, :need[i]] = perm[at:at + need[i]]
        at += need[i]
        dst[i, :fresh[i]] = perm[at:at + fresh[i]]
        at += fresh[i]
    kv = _pool(g, total, hkv, bs, d, dtype)
    kept, kept_lens = refs.select(torch.rand((len(lens), hkv, max(lens) + 1), generator=g), lens, budget, min(2, budget), 0)
    return kv, tables, dst, kept, kept_lens


@pytest.mark.parametrize("in_place", [False, True], ids=["fresh", "in_place"])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.int8], ids=["f16", "bf16", "i8"])
@pytest.mark.parametrize("lens,budget,hkv,bs,d", [
    ([1, 0, 9, 40], 8, 2, 8, 64), ([700, 333, 1], 257, 3, 16, 128), ([1500], 700, 1, 32, 128), ([100, 130], 99, 4, 16, 64)])
def test_compact_moves_the_kept_rows(lens, budget, hkv, bs, d, dtype, in_place):
    dev = device()
    g = torch.Generator().manual_seed(budget + d)
    kv, tables, dst, kept, kept_lens = _case(g, lens, budget, hkv, bs, d, dtype)
    want = refs.compact(kv, tables, kept, kept_lens, tables if in_place else dst)
    on = kv.to(dev)
    pkv.evict_compact(*pkv.split_pool(on), tables.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), kept.to(dev),
                      kept_lens.to(dev), dst_block_tables=None if in_place else dst.to(dev))
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    assert torch.equal(on.cpu().view(torch.int8), want.view(torch.int8))


def test_compact_flags_bad_inputs_and_skips_their_rows():
    dev = device()
    g = torch.Generator().manual_seed(2)
    kv, tables, dst, kept, kept_lens = _case(g, [64, 64], 16, 2, 16, 64, torch.float16)
    lens = torch.tensor([64, 64], dtype=torch.int32, device=dev)
    call = lambda on, t, k, n, d: pkv.evict_compact(*pkv.split_pool(on), t.to(dev), lens, k.to(dev), n.to(dev),
                                                    dst_block_tables=None if d is None else d.to(dev))
    bad = kept.clone()
    bad[0, 0, 15], bad[1, 1, 0] = 64, -5
    on = kv.to(dev)
    call(on, tables, bad, kept_lens, dst)
    assert pkv.get_device_error(dev)[1] == ["kept"]
    want = refs.compact(kv, tables, kept, kept_lens, dst)
    want[dst[0, 0], :, 0, 15] = kv[dst[0, 0], :, 0, 15]
    want[dst[1, 0], :, 1, 0] = kv[dst[1, 0], :, 1, 0]
    assert torch.equal(on.cpu(), want)
    below = kept.clone()
    below[0, 0, 15] = 14                                   # in place, a row below its rank
    on = kv.to(dev)
    call(on, tables, below, kept_lens, None)
    assert pkv.get_device_error(dev)[1] == ["kept"]
    t = tables.clone()
    t[0, :] = 10 ** 6
    on = kv.to(dev)
    call(on, t, kept, kept_lens, dst)
    assert pkv.get_device_error(dev)[1] == ["block_table"]
    want = refs.compact(kv, tables, kept, torch.tensor([0, 16]), dst)
    assert torch.equal(on.cpu(), want)
    on = kv.to(dev)
    call(on, tables, kept, torch.tensor([17, -1], dtype=torch.int32), dst)
    assert pkv.get_device_error(dev)[1] == ["context_len"]
    assert torch.equal(on.cpu(), kv)


def test_eviction_with_the_block_manager():
    """A forked sequence is cut back in place: its shared blocks are copied first, the fork keeps every token."""
    dev = device()
    bs, hkv, d = 8, 2, 64
    g = torch.Generator().manual_seed(3)
    bm = pkv_block_manager(24, bs)
    bm.add_sequence(1)
    for _ in range(61):
        bm.append_token(1)
    bm.fork(1, 2)
    kv = _pool(g, 24, hkv, bs, d, torch.bfloat16)
    before = kv.clone()
    old = bm.block_table(1)
    on = kv.to(dev)
    k_cache, v_cache = pkv.split_pool(on)
    lens = torch.tensor([61], dtype=torch.int32, device=dev)
    weights = torch.rand((1, hkv, 64), generator=g)
    kept, kept_lens = pkv.evict_select(weights.to(dev), lens, 20, sinks=1, recent=4, max_context_len=61)
    pairs = bm.make_private(1, 20)
    assert len(pairs) == 3
    pkv.copy_blocks(k_cache, v_cache, torch.from_numpy(pairs).to(dev))
    table = torch.tensor([bm.block_table(1)], dtype=torch.int32)
    pkv.evict_compact(k_cache, v_cache, table.to(dev), lens, kept, kept_lens)
    bm.truncate(1, 20)
    torch.cuda.synchronize()
    check_no_device_flags(dev)
    got, ref = on.cpu(), refs.select(weights, [61], 20, 1, 4)[0]
    assert torch.equal(kept.cpu(), ref)
    for h in range(hkv):
        for j in range(20):
            t = int(ref[0, h, j])
            assert torch.equal(got[table[0, j // bs], :, h, j % bs], before[old[t // bs], :, h, t % bs])
    assert torch.equal(got[old], before[old])               # the fork's tokens
    assert bm.block_table(2) == old and bm.seq_len(1) == 20 and len(bm.block_table(1)) == 3


def pkv_block_manager(num_blocks, bs):
    from paged_kv_cache_155_gb300.block_manager import BlockManager
    return BlockManager(num_blocks, bs, 16)
