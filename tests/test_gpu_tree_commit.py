"""What a commit of drafted paths leaves behind for sequences that it refuses."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests._gpu_helpers import device

pytestmark = pytest.mark.gpu
I32 = torch.int32


def _commit(lens, starts, path, taken, new=None, dtype=torch.float16, **bound):
    dev = device()
    b = len(lens)
    kv = torch.randn((2 * b, 2, 1, 8, 64), generator=torch.Generator().manual_seed(1)).to(dtype).to(dev)
    table = torch.arange(2 * b, dtype=I32, device=dev).view(b, 2)
    put = lambda v: torch.tensor(v, dtype=I32, device=dev)  # noqa: E731
    before = kv.clone()
    got = pkv.tree_commit(*pkv.split_pool(kv), table, put(starts), put(lens), put(path), put(taken), new,
                          **{**dict(max_query_len=5, max_context_len=16), **bound})
    return got, kv, before


def test_every_sequence_gets_a_length():
    """Of a sequence that is out of contract the one it came with, of a path that does not fit none of its nodes."""
    for new in (None, torch.full((5,), 77, dtype=I32, device=device())):
        got, kv, before = _commit([9, 3, 17, 10, 6], [0, 5, 10, 15, 20, 25], [[2, 3, 1]] * 5, [2, 2, 2, 4, 0], new)
        assert sorted(pkv.get_device_error(device())[1]) == ["context_len", "kept"]
        assert got.tolist() == [6, 3, 17, 5, 1]
        before[0, :, :, 4], before[0, :, :, 5] = before[0, :, :, 6], before[0, :, :, 7]
        assert torch.equal(kv, before)


def test_lengths_and_starts_of_any_value():
    """Differences of what the arrays hold that do not fit 32 bits are refused like any other."""
    low, high = -2 ** 31, 2 ** 31 - 1
    for lens, starts, good in (([low, low + 3, -1, high, 9], [0, 5, 10, 15, 20, 25], [4]),
                               ([9, 9, 9, 9, 9], [0, 5, low, high, 0, 5], [0, 4]),
                               ([low, high, 16, low + 5, 9], [-5, 0, 0, low, high, 5], [])):
        new, kv, before = _commit(lens, starts, [[2, 3, 1]] * 5, [2] * 5)
        assert pkv.get_device_error(device())[1] == ["context_len"]
        want = list(lens)
        for i in good:
            want[i] = 6  # four cached tokens and two nodes
            before[2 * i, :, :, 4], before[2 * i, :, :, 5] = before[2 * i, :, :, 6], before[2 * i, :, :, 7]
        assert new.tolist() == want and torch.equal(kv, before)
