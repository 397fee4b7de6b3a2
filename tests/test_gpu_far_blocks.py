"""Pools whose blocks lie far apart (offsets past 32 bits) give what a dense pool gives, bit for bit; workspaces that are
too small are refused."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests._gpu_helpers import check_no_device_flags, device
from tests.test_gpu_tree import ancestors, words_of

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
APART = 128 << 20  # bytes from block to block: block 17 and those behind it start past 2^31 bytes, block 33 past 2^32


def _far(pool):
    """The K and V halves of a pool like this one, its blocks APART bytes from each other."""
    step = APART // pool.element_size()
    buf = torch.empty(pool.shape[0] * step, dtype=pool.dtype, device=pool.device)
    far = buf.as_strided(pool.shape, (step, *pool.stride()[1:]))
    far.copy_(pool)
    return far[:, 0], far[:, 1]


def _context(lens, bs, blocks=40):
    """Tables whose sequences use the pool's last blocks first."""
    need = [-(-n // bs) for n in lens]
    assert sum(need) <= blocks
    tables, at = torch.zeros((len(lens), max(need)), dtype=torch.int32), blocks
    for i, n in enumerate(need):
        tables[i, :n] = torch.arange(at - 1, at - 1 - n, -1)
        at -= n
    return tables


def test_four_bit_cache():
    dev, g = device(), torch.Generator().manual_seed(1)
    for hq, hkv, d, bs in ((8, 2, 128, 16), (16, 2, 64, 8), (20, 1, 128, 32)):
        lens = [9 * bs + 3, 14 * bs - 1, bs]
        tables = _context(lens, bs).to(dev)
        n = torch.tensor(lens, dtype=torch.int32, device=dev)
        slots = torch.cat([tables[i].cpu()[torch.arange(c) // bs].long() * bs + torch.arange(c) % bs
                           for i, c in enumerate(lens)]).to(dev)
        k, v = (torch.randn((sum(lens), hkv, d), generator=g).to(BF16).to(dev) for _ in range(2))
        q = torch.randn((3, hq, d), generator=g).to(BF16).to(dev)
        near = pkv.int4_pool(40, hkv, bs, d, dev).zero_()
        far = _far(near)
        pkv.reshape_and_cache_int4(k, v, slots, *pkv.split_pool(near))
        pkv.reshape_and_cache_int4(k, v, slots, *far)
        assert torch.equal(far[0], near[:, 0]) and torch.equal(far[1], near[:, 1])
        outs = [pkv.paged_attention_decode_int4(q, *halves, tables, n, max_context_len=max(lens))
                for halves in (pkv.split_pool(near), far)]
        assert torch.equal(*outs)
        pairs = torch.tensor([[39, 1], [20, 39]], device=dev)
        back = [torch.zeros((40, 2, hkv, bs, d), dtype=BF16, device=dev) for _ in range(2)]
        pkv.dequantise_blocks_int4(*pkv.split_pool(near), pairs, *pkv.split_pool(back[0]))
        there = _far(back[1])
        pkv.dequantise_blocks_int4(*far, pairs, *there)
        assert torch.equal(there[0], back[0][:, 0]) and torch.equal(there[1], back[0][:, 1])
        pkv.copy_blocks(*pkv.split_pool(near), pairs)
        pkv.copy_blocks(*far, pairs)
        assert torch.equal(far[0], near[:, 0]) and torch.equal(far[1], near[:, 1])
        check_no_device_flags(dev)


def test_trees_and_their_commit():
    dev, g = device(), torch.Generator().manual_seed(2)
    bs, cached, nodes = 16, [200, 31], [20, 65]
    lens = [a + b for a, b in zip(cached, nodes)]
    tables = _context(lens, bs).to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    start = torch.tensor([0, 20, 85], dtype=torch.int32, device=dev)
    q = torch.randn((85, 8, 128), generator=g).to(BF16).to(dev)
    near = torch.randn((40, 2, 2, bs, 128), generator=g).to(BF16).to(dev)
    far = _far(near)
    mask = torch.cat([words_of(ancestors(c, g), 2) for c in nodes]).to(dev)
    kw = dict(max_query_len=65, max_context_len=220)
    outs = [pkv.paged_attention_tree(q, *halves, tables, start, n, mask, **kw) for halves in (pkv.split_pool(near), far)]
    assert torch.equal(*outs)
    path = torch.tensor([[0, 3, 9, 19, 0], [1, 2, 30, 63, 64]], dtype=torch.int32, device=dev)
    taken = torch.tensor([4, 5], dtype=torch.int32, device=dev)
    new = [pkv.tree_commit(*halves, tables, start, n, path, taken, **kw) for halves in (pkv.split_pool(near), far)]
    assert torch.equal(*new) and torch.equal(far[0], near[:, 0]) and torch.equal(far[1], near[:, 1])
    check_no_device_flags(dev)


def test_windows_with_first_tokens():
    dev, g = device(), torch.Generator().manual_seed(3)
    bs, lens = 16, [333, 250]
    tables = _context(lens, bs).to(dev)
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    kw = dict(window=100, sinks=20, max_context_len=333)
    q = torch.randn((2, 8, 128), generator=g).to(BF16).to(dev)
    near = torch.randn((40, 2, 2, bs, 128), generator=g).to(BF16).to(dev)
    far = _far(near)
    assert torch.equal(*(pkv.paged_attention_decode_sinks(q, *h, tables, n, **kw) for h in (pkv.split_pool(near), far)))
    rows = torch.randn((50, 8, 128), generator=g).to(BF16).to(dev)
    start = torch.tensor([0, 40, 50], dtype=torch.int32, device=dev)
    assert torch.equal(*(pkv.paged_attention_prefill_sinks(rows, *h, tables, start, n, max_query_len=40, **kw)
                         for h in (pkv.split_pool(near), far)))
    codes = torch.randint(-127, 128, (40, 2, 2, bs, 128), generator=g).to(torch.int8).to(dev)
    scales = [torch.rand((2, 128), generator=g).to(dev) / 64 for _ in range(2)]
    assert torch.equal(*(pkv.paged_attention_decode_sinks_int8(q, *h, *scales, tables, n, **kw)
                         for h in (pkv.split_pool(codes), _far(codes))))
    check_no_device_flags(dev)


def test_workspaces_that_are_too_small():
    dev = device()
    tables, n = torch.zeros((1, 64), dtype=torch.int32, device=dev), torch.ones(1, dtype=torch.int32, device=dev)
    q = torch.zeros((1, 8, 128), dtype=BF16, device=dev)
    pool = torch.zeros((4, 2, 2, 16, 128), dtype=BF16, device=dev)
    four = pkv.int4_pool(4, 2, 16, 128, dev).zero_()
    start, mask = torch.tensor([0, 1], dtype=torch.int32, device=dev), torch.ones((1, 1), dtype=torch.int64, device=dev)
    short = lambda nbytes: torch.empty(nbytes - 16, dtype=torch.uint8, device=dev)
    for call in (
            lambda: pkv.paged_attention_decode_int4(q, *pkv.split_pool(four), tables, n, max_context_len=1024,
                                                    workspace=short(pkv.decode_int4_workspace_bytes(1, 8, 2, 128, 16, 1024))),
            lambda: pkv.paged_attention_tree(q, *pkv.split_pool(pool), tables, start, n, mask, max_query_len=1,
                                             max_context_len=1024, workspace=short(pkv.tree_workspace_bytes())),
            lambda: pkv.paged_attention_decode_sinks(q, *pkv.split_pool(pool), tables, n, window=900, sinks=4, max_context_len=1024,
                                                     partition_size=64,
                                                     workspace=short(pkv.decode_sinks_workspace_bytes(1, 8, 2, 128, 16, 1024, 900,
                                                                                                      4, partition_size=64))),
            lambda: pkv.paged_attention_prefill_sinks(q, *pkv.split_pool(pool), tables, start, n, max_query_len=1,
                                                      max_context_len=1024, window=900, sinks=4, kv_splits=4,
                                                      workspace=short(pkv.prefill_sinks_workspace_bytes(1, 1, 8, 2, 128, 16, 1, 1024,
                                                                                                        900, 4, 4)))):
        with pytest.raises(pkv.PagedKVError):
            call()
