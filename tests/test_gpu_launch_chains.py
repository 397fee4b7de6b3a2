"""Calls launched ahead of the end of the one before them, directly behind a kernel of the library that lets them start early and
writes what they read (nothing between the two, which a copy or another library's kernel would order), and before one that
overwrites it."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests._gpu_helpers import check_no_device_flags, device
from tests.test_gpu_tree import ancestors, words_of

pytestmark = pytest.mark.gpu
BF16, BS, LENS, ROWS = torch.bfloat16, 16, [3333, 410, 5000], [40, 23, 64]
TIMES = 25


def _tensors(dev):
    g = torch.Generator().manual_seed(11)
    need = [-(-n // BS) for n in LENS]
    tables = torch.zeros((3, max(need)), dtype=torch.int32)
    perm, at = torch.randperm(sum(need), generator=g).to(torch.int32), 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    rn = lambda *shape: torch.randn(shape, generator=g).to(BF16)  # noqa: E731
    rows = sum(ROWS)
    tokens = torch.arange(at * BS)
    x = dict(q=rn(3, 8, 128), rows=rn(rows, 8, 128), kv=rn(at, 2, 2, BS, 128), k=rn(at * BS, 2, 128), v=rn(at * BS, 2, 128),
             tables=tables, lens=torch.tensor(LENS, dtype=torch.int32), start=torch.tensor([0, 40, 63, 127], dtype=torch.int32),
             slots=tokens, mask=torch.cat([words_of(ancestors(n, g), 1) for n in ROWS]),
             pairs=torch.arange(at).repeat_interleave(2).reshape(-1, 2),
             codes=torch.randint(0, 256, (at, 2, 2, BS, 80), generator=g).to(torch.uint8) & 0x3f,  # finite scales
             i8=torch.randint(-127, 128, (at, 2, 2, BS, 128), generator=g).to(torch.int8), scales=torch.rand((2, 2, 128), generator=g) / 64,
             path=torch.stack([torch.arange(1, 23, dtype=torch.int32)] * 3), taken=torch.tensor([22, 7, 20], dtype=torch.int32),
             after=torch.zeros(3, dtype=torch.int32), later=torch.zeros(3, dtype=torch.int32))
    return {k: t.to(dev) for k, t in x.items()}


def _consumers(x, lens):
    """name -> (call, the tensor it writes), with these context lengths."""
    halves, codes, i8 = pkv.split_pool(x["kv"]), pkv.split_pool(x["codes"]), pkv.split_pool(x["i8"])
    chunk, size = (x["tables"], x["start"], lens), dict(max_query_len=64, max_context_len=max(LENS))
    own = lambda c: (c, c.result)  # noqa: E731
    return {
        "int4_decode": own(pkv.prepare_paged_attention_decode_int4(x["q"], *codes, x["tables"], lens, max_context_len=max(LENS))),
        "tree": own(pkv.prepare_paged_attention_tree(x["rows"], *halves, *chunk, x["mask"], **size)),
        "sinks": own(pkv.prepare_paged_attention_decode_sinks(x["q"], *halves, x["tables"], lens, window=999, sinks=5, max_context_len=max(LENS))),
        "sinks_int8": own(pkv.prepare_paged_attention_decode_sinks_int8(x["q"], *i8, *x["scales"], x["tables"], lens, window=999, sinks=5,
                                                                        max_context_len=max(LENS))),
        "sinks_prefill": own(pkv.prepare_paged_attention_prefill_sinks(x["rows"], *halves, *chunk, window=999, sinks=5, **size)),
        "sinks_prefill_split": own(pkv.prepare_paged_attention_prefill_sinks(x["rows"], *halves, *chunk, window=999, sinks=5, kv_splits=3, **size)),
        "int4_read": (pkv.prepare_dequantise_blocks_int4(*codes, x["pairs"], *halves), x["kv"]),
        "commit": (pkv.prepare_tree_commit(*halves, *chunk, x["path"], x["taken"], x["later"], **size), x["kv"]),
    }


def _producers(x):
    halves, codes = pkv.split_pool(x["kv"]), pkv.split_pool(x["codes"])
    return {
        "int4_write": pkv.prepare_reshape_and_cache_int4(x["k"], x["v"], x["slots"], *codes),
        "int4_read": pkv.prepare_dequantise_blocks_int4(*codes, x["pairs"], *halves),
        "commit": pkv.prepare_tree_commit(*halves, x["tables"], x["start"], x["lens"], x["path"], x["taken"], x["after"], max_query_len=64,
                                          max_context_len=max(LENS)),
    }


READS = ["tree", "sinks", "sinks_prefill", "sinks_prefill_split"]
PAIRS = [("int4_write", "int4_decode"), ("int4_write", "int4_read"), ("int4_read", "commit"),
         *[("int4_read", n) for n in READS], ("commit", "int4_decode"), ("commit", "sinks_int8"), ("commit", "commit"),
         *[("commit", n) for n in READS]]


@pytest.mark.parametrize("first,second", PAIRS)
def test_behind_a_kernel_that_lets_it_start_early(first, second):
    dev = device()
    x = _tensors(dev)
    held = {k: t.clone() for k, t in x.items()}
    call, result = _consumers(x, x["after"] if first == "commit" else x["lens"])[second]
    produce = _producers(x)[first]

    def reset():
        for k, t in x.items():
            t.copy_(held[k])
        if result is not x["kv"]:
            result.zero_()
        torch.cuda.synchronize()

    reset()
    produce()
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    want, want_later = result.clone(), x["later"].clone()
    for _ in range(TIMES):
        reset()
        produce()
        call()
        torch.cuda.synchronize()
        assert torch.equal(result, want) and torch.equal(x["later"], want_later)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        produce()
        call()
    for _ in range(TIMES):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(result, want) and torch.equal(x["later"], want_later)
    check_no_device_flags(dev)


@pytest.mark.parametrize("first,second", [("int4_decode", "int4_write"), ("int4_read", "int4_write"), *[(n, "int4_read") for n in READS],
                                          *[(n, "commit") for n in READS], ("sinks_int8", "commit"), ("int4_decode", "commit")])
def test_before_a_kernel_that_overwrites_what_it_reads(first, second):
    """... launched while the reading kernel, or its merge, still runs."""
    dev = device()
    x = _tensors(dev)
    held = {k: t.clone() for k, t in x.items()}
    x["after"].copy_(x["lens"])
    held["after"].copy_(x["lens"])
    call, result = _consumers(x, x["after"])[first]  # a commit writes the lengths it reads
    over = _producers(x)[second]
    call()
    torch.cuda.synchronize()
    want = result.clone()
    for _ in range(TIMES):
        for k, t in x.items():
            t.copy_(held[k])
        torch.cuda.synchronize()
        call()
        over()
        torch.cuda.synchronize()
        assert torch.equal(result, want)
    check_no_device_flags(dev)
