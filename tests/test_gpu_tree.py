"""A tree of drafted tokens over the paged cache: the verification's attention and the accepted path's move."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from paged_kv_cache_155_gb300.block_manager import BlockManager
from tests import _cache_refs as refs
from tests._gpu_helpers import check_no_device_flags, device
from tests._operator_refs import HALF_STEP, rounded_close

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def ancestors(n, g):
    """[n, n] bool: each node sees itself and its ancestors, for random parents among the nodes before it."""
    seen = torch.eye(n, dtype=torch.bool)
    for i in range(1, n):
        seen[i] |= seen[int(torch.randint(0, i, (1,), generator=g))]
    return seen


def words_of(seen, words):
    """bool [n, m] -> int64 [n, words]."""
    out = torch.zeros((seen.shape[0], words), dtype=torch.int64)
    for c in range(seen.shape[1]):
        out[:, c // 64] |= seen[:, c].to(torch.int64) << (c % 64)
    return out


def run(dev, dtype, hq, hkv, bs, cached, nodes, seed=0, words=None, masks=None, extra=0, scale=128 ** -0.5):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(cached, nodes)]
    tables, blocks = refs.place(lens, bs, g)
    rows, most = sum(nodes), max(nodes)
    words = words or -(-most // 64)
    q = (torch.randn((rows + extra, hq, 128), generator=g) * 2).to(dtype)
    kv = torch.randn((blocks, 2, hkv, bs, 128), generator=g).to(dtype)
    masks = masks or [ancestors(n, g) for n in nodes]
    mask = torch.cat([words_of(m, words) for m in masks] + [torch.full((extra, words), -1, dtype=torch.int64)])
    # bits behind a chunk's tokens are ignored
    at = 0
    for n in nodes:
        for c in range(n, 64 * words, 3):
            bit = 1 << (c % 64)
            mask[at:at + n, c // 64] |= bit - (bit >> 63 << 64)
        at += n
    ctx = [refs.context(kv.double(), tables[i], n) for i, n in enumerate(lens)]
    refs.poison(kv, tables, [range(n) for n in lens])
    out = torch.full_like(q, 3.0).to(dev)
    start = torch.tensor([0] + nodes, dtype=torch.int32).cumsum(0).to(torch.int32)
    pkv.paged_attention_tree(q.to(dev), *pkv.split_pool(kv.to(dev)), tables.to(dev), start.to(dev),
                             torch.tensor(lens, dtype=torch.int32, device=dev), mask.to(dev), scale, out,
                             max_query_len=most, max_context_len=max(lens))
    check_no_device_flags(dev)
    out = out.cpu()
    assert (out[rows:] == 3.0).all()
    at = 0
    for i, n in enumerate(nodes):
        seen = torch.cat([torch.ones((n, cached[i]), dtype=torch.bool), masks[i]], 1)
        want, mag, size = refs.attend(q[at:at + n], *ctx[i], scale, seen)
        rounded_close(out[at:at + n], want, refs.attention_bound(mag, size, 128, HALF_STEP[dtype]), f"sequence {i}")
        at += n


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,bs", [(2, 2, 8), (8, 1, 16), (12, 4, 32), (40, 2, 16), (32, 2, 8), (128, 1, 32)])
def test_trees(hq, hkv, bs, dtype):
    run(device(), dtype, hq, hkv, bs, [0, 1, 127, 128, 129, 300, 1000], [1, 7, 16, 63, 64, 65, 2], seed=hq + bs, extra=3)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_one_long_context(dtype):
    """One unit per KV head cut into many pieces, and a draft of one token."""
    run(device(), dtype, 8, 2, 16, [5000], [13], seed=1)
    run(device(), dtype, 4, 1, 32, [4095], [1], seed=2)


def test_many_sequences_of_every_length():
    run(device(), BF16, 4, 2, 16, [i * 37 % 500 for i in range(75)], [i * 11 % 23 for i in range(74)] + [9], seed=3)
    run(device(), F16, 16, 4, 8, [0] * 40 + [900], [1] * 40 + [100], seed=4)


@pytest.mark.parametrize("hkv", [2, 3, 4])
@pytest.mark.parametrize("seqs", [6, 60])
def test_drafts_of_one_to_eight_row_tiles(hkv, seqs):
    """Row tiles side by side and alone, their units whole and cut, with sequences that draft nothing between."""
    cached = [i * 211 % 700 for i in range(seqs)]
    run(device(), BF16, 16 * hkv, hkv, 16, cached, [i * 13 % 62 + (i == seqs - 1) for i in range(seqs)], seed=seqs + hkv)


def test_wide_masks_and_any_bits():
    g = torch.Generator().manual_seed(5)
    masks = [torch.rand((n, n), generator=g) < 0.4 for n in (200, 130, 90, 5)]  # not only ancestors: any bits
    masks[3][:] = False                                                         # ... and rows that see nothing
    masks[0][7] = False
    run(device(), F16, 4, 2, 16, [10, 0, 257, 0], [200, 130, 90, 5], seed=5, masks=masks)
    run(device(), BF16, 8, 2, 8, [33], [70], seed=6, words=4)
    run(device(), BF16, 8, 2, 8, [33], [70], seed=7, scale=-0.05)


def test_a_chain_is_the_causal_prefill():
    dev, g = device(), torch.Generator().manual_seed(8)
    cached, nodes, bs = [100, 513], [20, 40], 16
    lens = [a + b for a, b in zip(cached, nodes)]
    tables, blocks = refs.place(lens, bs, g)
    q = torch.randn((60, 8, 128), generator=g).to(F16).to(dev)
    kv = torch.randn((blocks, 2, 2, bs, 128), generator=g).to(F16).to(dev)
    start = torch.tensor([0, 20, 60], dtype=torch.int32, device=dev)
    n, t = torch.tensor(lens, dtype=torch.int32, device=dev), tables.to(dev)
    mask = torch.cat([words_of(torch.ones(c, c).tril().bool(), 1) for c in nodes]).to(dev)
    a = pkv.paged_attention_tree(q, *pkv.split_pool(kv), t, start, n, mask, max_query_len=40, max_context_len=553)
    b = pkv.paged_attention_prefill(q, *pkv.split_pool(kv), t, start, n, max_query_len=40, max_context_len=553)
    assert (a.float() - b.float()).abs().max() < 4 * 4 * 2.0 ** -11  # outputs below 4; both round weights and outputs


def test_bad_sequences_are_flagged_and_left_out():
    dev, g = device(), torch.Generator().manual_seed(9)
    lens, nodes, bs = [40, 3, 70, 500], [4, 5, 6, 7], 16     # the second is shorter than its chunk, the last past the bound
    tables, blocks = refs.place([64, 16, 80, 512], bs, g)
    q = torch.randn((22, 4, 128), generator=g).to(F16)
    kv = torch.randn((blocks, 2, 2, bs, 128), generator=g).to(F16)
    tables[2, 1] = blocks  # a bad entry: its tokens do not count
    out = torch.full_like(q, 3.0).to(dev)
    start = torch.tensor([0] + nodes).cumsum(0).to(torch.int32)
    masks = [ancestors(c, g) for c in nodes]
    pkv.paged_attention_tree(q.to(dev), *pkv.split_pool(kv.to(dev)), tables.to(dev), start.to(dev),
                             torch.tensor(lens, dtype=torch.int32, device=dev), torch.cat([words_of(m, 1) for m in masks]).to(dev),
                             out=out, max_query_len=7, max_context_len=200)
    assert sorted(pkv.get_device_error(dev)[1]) == ["block_table", "context_len"]
    out = out.cpu()
    assert (out[4:9] == 3.0).all() and (out[15:] == 3.0).all()
    k, v = refs.context(kv.double(), tables[0], 40)
    seen = torch.cat([torch.ones((4, 36), dtype=torch.bool), masks[0]], 1)
    assert (out[:4].double() - refs.attend(q[:4], k, v, 128 ** -0.5, seen)[0]).abs().max() < 1e-2


def test_two_prepared_calls_in_graphs_on_two_streams():
    dev, g = device(), torch.Generator().manual_seed(10)
    cached, nodes, bs = [900, 77], [12, 30], 16
    lens = [a + b for a, b in zip(cached, nodes)]
    tables, blocks = refs.place(lens, bs, g)
    q = torch.randn((42, 8, 128), generator=g).to(BF16).to(dev)
    kv = torch.randn((blocks, 2, 2, bs, 128), generator=g).to(BF16).to(dev)
    start = torch.tensor([0, 12, 42], dtype=torch.int32, device=dev)
    n, t = torch.tensor(lens, dtype=torch.int32, device=dev), tables.to(dev)
    mask = torch.cat([words_of(ancestors(c, g), 1) for c in nodes]).to(dev)
    calls = [pkv.prepare_paged_attention_tree(q, *pkv.split_pool(kv), t, start, n, mask, max_query_len=30, max_context_len=920)
             for _ in range(2)]
    want = calls[0]().clone()
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
        c.result.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(calls[0].result, want) and torch.equal(calls[1].result, want)


@pytest.mark.parametrize("kind", [F16, BF16, torch.int8])
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (5, 128, 16), (32, 128, 32), (33, 64, 16)])
def test_commit(hkv, d, bs, kind):
    dev, g = device(), torch.Generator().manual_seed(hkv)
    cached, nodes = [0, 3, 30, 77, 16, 5], [1, 40, 12, 25, 6, 0]
    lens = [a + b for a, b in zip(cached, nodes)]
    tables, blocks = refs.place(lens, bs, g)
    kv = torch.randint(-30000, 30000, (blocks, 2, hkv, bs, d), generator=g)
    kv = kv.to(torch.int8) if kind is torch.int8 else kv.to(torch.int16).view(kind)
    paths = [sorted(torch.randperm(n, generator=g)[:m].tolist()) for n, m in zip(nodes, [1, 19, 12, 0, 3, 0])]
    path = torch.full((6, 20), 9999, dtype=torch.int32)
    for i, p in enumerate(paths):
        path[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    want = kv.clone()
    for i, p in enumerate(paths):
        for j, c in enumerate(p):
            a, b = cached[i] + c, cached[i] + j
            want[tables[i, b // bs], :, :, b % bs] = kv[tables[i, a // bs], :, :, a % bs]
    dk = kv.to(dev)
    start = torch.tensor([0] + nodes).cumsum(0).to(torch.int32).to(dev)
    got = pkv.tree_commit(*pkv.split_pool(dk), tables.to(dev), start, torch.tensor(lens, dtype=torch.int32, device=dev),
                          path.to(dev), torch.tensor([len(p) for p in paths], dtype=torch.int32, device=dev),
                          max_query_len=40, max_context_len=max(lens))
    check_no_device_flags(dev)
    assert got.tolist() == [a + len(p) for a, p in zip(cached, paths)]
    bits = lambda t: t if kind is torch.int8 else t.view(torch.int16)  # noqa: E731
    assert torch.equal(bits(dk.cpu()), bits(want))


def test_commit_flags_what_does_not_fit():
    dev = device()
    kv = torch.randn((8, 2, 1, 8, 64), generator=torch.Generator().manual_seed(1)).to(F16).to(dev)
    before = kv.clone()
    t = torch.arange(8, dtype=torch.int32, device=dev).view(4, 2)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    start, n = i32(0, 5, 10, 15, 20), i32(9, 3, 17, 10)
    path = i32(2, 1, 3, 5, -1, 3, 0, 1, 2, 3, 4, 5).view(4, 3)
    new = pkv.tree_commit(*pkv.split_pool(kv), t, start, n, path, i32(2, 2, 2, 4), max_query_len=5, max_context_len=16)
    # the second's length is below its chunk, the third's past the bound, the fourth's path longer than its room
    assert sorted(pkv.get_device_error(dev)[1]) == ["context_len", "kept"]
    before[0, :, :, 4] = before[0, :, :, 6]  # the first node of the first path; the second does not ascend
    assert torch.equal(kv, before) and new[3] == 5


def test_drafts_verified_and_committed_are_the_plain_steps():
    """Three verification steps with a block manager: drafts written, attended and committed; the rows of the accepted nodes
    are those of plain decode steps over the accepted tokens, and so is the cache afterwards."""
    dev, g = device(), torch.Generator().manual_seed(14)
    hq, hkv, bs, nodes = 8, 2, 8, 11
    rows = lambda t, h: torch.randn((t, h, 128), generator=g).to(BF16).to(dev)  # noqa: E731
    bm = BlockManager(64, bs, 16)
    pools = [torch.zeros((64, 2, hkv, bs, 128), dtype=BF16, device=dev) for _ in range(2)]
    plain_table = torch.arange(32, 48, dtype=torch.int32, device=dev)[None]
    bm.add_sequence(1)
    length = 21
    k, v = rows(length, hkv), rows(length, hkv)
    slots = torch.tensor([bm.append_token(1)[0] for _ in range(length)], device=dev)
    pkv.reshape_and_cache(k, v, slots, *pkv.split_pool(pools[0]))
    at = lambda ts: torch.tensor([32 * bs + t for t in ts], device=dev)  # noqa: E731
    pkv.reshape_and_cache(k, v, at(range(length)), *pkv.split_pool(pools[1]))
    for step in range(3):
        k, v, q = rows(nodes, hkv), rows(nodes, hkv), rows(nodes, hq)
        seen = ancestors(nodes, g)
        slots = torch.tensor([bm.append_token(1)[0] for _ in range(nodes)], device=dev)
        pkv.reshape_and_cache(k, v, slots, *pkv.split_pool(pools[0]))
        used = bm.block_table(1)
        table = torch.tensor([list(used) + [0] * (16 - len(used))], dtype=torch.int32, device=dev)
        lens = torch.tensor([length + nodes], dtype=torch.int32, device=dev)
        start = torch.tensor([0, nodes], dtype=torch.int32, device=dev)
        out = pkv.paged_attention_tree(q, *pkv.split_pool(pools[0]), table, start, lens, words_of(seen, 1).to(dev),
                                       max_query_len=nodes, max_context_len=16 * bs)
        path = seen[int(torch.randint(0, nodes, (1,), generator=g))].nonzero()[:, 0].tolist()
        new = pkv.tree_commit(*pkv.split_pool(pools[0]), table, start, lens, torch.tensor([path], dtype=torch.int32, device=dev),
                              torch.tensor([len(path)], dtype=torch.int32, device=dev), max_query_len=nodes,
                              max_context_len=16 * bs)
        for j, c in enumerate(path):
            pkv.reshape_and_cache(k[c:c + 1], v[c:c + 1], at([length + j]), *pkv.split_pool(pools[1]))
            want = pkv.paged_attention_decode(q[c:c + 1], *pkv.split_pool(pools[1]), plain_table,
                                              torch.tensor([length + j + 1], dtype=torch.int32, device=dev), max_context_len=16 * bs)
            assert (out[c:c + 1].float() - want.float()).abs().max() < 4 * 4 * 2.0 ** -8  # outputs below 4
        length += len(path)
        assert new.tolist() == [length]
        bm.truncate(1, length)
        for t in range(length):
            assert torch.equal(pools[0][int(used[t // bs]), :, :, t % bs], pools[1][32 + t // bs, :, :, t % bs])
    check_no_device_flags(dev)
