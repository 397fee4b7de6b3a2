"""The new lengths of a commit stand apart from everything that its thread blocks read: an overlap is refused on the host."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from paged_kv_cache_155_gb300 import _build

I32 = torch.int32


def test_c_abi():
    _build.build()
    from paged_kv_cache_155_gb300._lib import lib
    good = dict(k=16, v=16, nb=64, stride=2 * 4 * 16 * 64, hkv=4, d=64, bs=16, bt=4096, mb=8, qs=8192, cl=12288, maxq=10, maxl=100, b=4,
                path=16384, n=20480, most=5, new=24576, dt=1)
    call = lambda **kw: lib().pkv_tree_commit(*{**good, **kw}.values(), None)  # noqa: E731
    for first, count in ((4096, 4 * 8), (8192, 4 + 1), (12288, 4), (16384, 4 * 5), (20480, 4)):
        for new in (first - 12, first, first + 4 * count - 4):
            assert call(new=new) == 1, (first, new)


def test_binding():
    k, v = pkv.split_pool(torch.zeros((8, 2, 2, 16, 128), dtype=torch.float16))
    both = torch.zeros(100, dtype=I32)
    args = dict(k_cache=k, v_cache=v, block_tables=both[:8].view(2, 4), query_start=both[10:13], context_lens=both[20:22],
                accepted=both[30:36].view(2, 3), accepted_lens=both[40:42], max_query_len=1, max_context_len=64)
    for at in (0, 7, 9, 12, 19, 21, 29, 35, 39, 41):
        with pytest.raises(ValueError, match="overlap"):
            pkv.tree_commit(**args, new_context_lens=both[at:at + 2])
    for at in (8, 13, 18, 22, 28, 36, 38, 42):  # beside them
        with pytest.raises(ValueError, match="CUDA"):
            pkv.tree_commit(**args, new_context_lens=both[at:at + 2])
