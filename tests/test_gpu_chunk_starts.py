"""Chunk starts of any value: sequences whose start and end do not make a chunk are flagged and left out by every call over
chunks, differences that wrap around 32 bits among them."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
I32 = torch.int32
CALLS = {
    "plain": (pkv.paged_attention_prefill, {}),
    "scored": (pkv.paged_attention_prefill_scored, dict(window=7)),
    "sinks": (pkv.paged_attention_prefill_sinks, dict(window=7, sinks=1)),
    "sinks split": (pkv.paged_attention_prefill_sinks, dict(window=500, sinks=1, kv_splits=2)),
    "tree": (pkv.paged_attention_tree, {}),
}


@pytest.mark.parametrize("name", CALLS)
def test_starts_of_any_value(name):
    dev, g = device(), torch.Generator().manual_seed(3)
    call, kw = CALLS[name]
    low, high = -2 ** 31, 2 ** 31 - 1
    kv = torch.randn((16, 2, 2, 16, 128), generator=g).to(torch.float16).to(dev)
    tables = torch.arange(16, dtype=I32, device=dev).view(4, 4)
    q = torch.randn((8, 8, 128), generator=g).to(torch.float16).to(dev)
    lens = torch.tensor([9, 9, 9, 9], dtype=I32, device=dev)
    if name == "tree":
        kw = dict(kw, tree_mask=torch.full((8, 1), 15, dtype=torch.int64, device=dev))
    bound = dict(max_query_len=8, max_context_len=64, **kw)
    outs = []
    for starts in ([0, 4, 4, 4, 4], [0, 4, high, low, 8], [0, 4, low, high, 4]):
        out = torch.full_like(q, 3.0)
        call(q, *pkv.split_pool(kv), tables, torch.tensor(starts, dtype=I32, device=dev), lens, out=out, **bound)
        if outs:
            assert pkv.get_device_error(dev)[1] == ["context_len"], starts
        else:
            check_no_device_flags(dev)
        assert (out[4:] == 3.0).all(), starts
        outs.append(out[:4])
    assert not (outs[0] == 3.0).all(1).any() and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
