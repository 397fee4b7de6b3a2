"""Calls see what the work before them on their stream wrote, however late it ends: behind a kernel, behind an event of another
stream, and in captured graphs that fork and join; and what comes behind them sees what they wrote."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests._gpu_helpers import check_no_device_flags, device
from tests.test_gpu_tree import ancestors, words_of

pytestmark = pytest.mark.gpu
BF16, BS, LENS = torch.bfloat16, 16, [333, 41, 500]
ROWS = [20, 3, 37]


def _inputs(g):
    need = [-(-n // BS) for n in LENS]
    tables = torch.zeros((3, max(need)), dtype=torch.int32)
    perm, at = torch.randperm(sum(need), generator=g).to(torch.int32), 0
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    rn = lambda *shape: torch.randn(shape, generator=g).to(BF16)
    return dict(q=rn(3, 8, 128), rows=rn(60, 8, 128), kv=rn(at, 2, 2, BS, 128), new=rn(2, 60, 2, 128), tables=tables,
                lens=torch.tensor(LENS, dtype=torch.int32), start=torch.tensor([0, 20, 23, 60], dtype=torch.int32),
                slots=torch.randperm(at * BS, generator=g)[:60],
                mask=torch.cat([words_of(ancestors(n, g), 1) for n in ROWS]),
                pairs=torch.arange(at).repeat_interleave(2).reshape(-1, 2),
                codes=torch.randint(0, 256, (at, 2, 2, BS, 80), generator=g).to(torch.uint8) & 0x3f,  # finite scales
                i8=torch.randint(-127, 128, (at, 2, 2, BS, 128), generator=g).to(torch.int8),
                scales=torch.rand((2, 2, 128), generator=g) / 64,
                path=torch.tensor([[0, 5, 19], [2, 0, 0], [1, 30, 36]], dtype=torch.int32),
                taken=torch.tensor([3, 1, 2], dtype=torch.int32))


def _calls(x):
    """name -> (call, what it writes) over the tensors x."""
    halves, codes, i8 = pkv.split_pool(x["kv"]), pkv.split_pool(x["codes"]), pkv.split_pool(x["i8"])
    over = (x["tables"], x["lens"])
    chunk = (x["tables"], x["start"], x["lens"])
    most, size = max(LENS), dict(max_query_len=37, max_context_len=max(LENS))
    wrap = lambda c: (c, c.result)
    after = torch.zeros(3, dtype=torch.int32, device=x["kv"].device)
    return {
        "int4_write": (pkv.prepare_reshape_and_cache_int4(*x["new"], x["slots"], *codes), x["codes"]),
        "int4_read": (pkv.prepare_dequantise_blocks_int4(*codes, x["pairs"], *halves), x["kv"]),
        "int4_decode": wrap(pkv.prepare_paged_attention_decode_int4(x["q"], *codes, *over, max_context_len=most)),
        "tree": wrap(pkv.prepare_paged_attention_tree(x["rows"], *halves, *chunk, x["mask"], **size)),
        "commit": (pkv.prepare_tree_commit(*halves, *chunk, x["path"], x["taken"], after, **size), x["kv"]),
        "sinks": wrap(pkv.prepare_paged_attention_decode_sinks(x["q"], *halves, *over, window=99, sinks=5, max_context_len=most)),
        "sinks_int8": wrap(pkv.prepare_paged_attention_decode_sinks_int8(x["q"], *i8, *x["scales"], *over, window=99, sinks=5,
                                                                         max_context_len=most)),
        "sinks_prefill": wrap(pkv.prepare_paged_attention_prefill_sinks(x["rows"], *halves, *chunk, window=99, sinks=5, **size)),
    }


NAMES = ["int4_write", "int4_read", "int4_decode", "tree", "commit", "sinks", "sinks_int8", "sinks_prefill"]


@pytest.mark.parametrize("name", NAMES)
def test_behind_late_writes_of_the_inputs(name):
    dev, host = device(), _inputs(torch.Generator().manual_seed(1))
    real = {k: v.to(dev) for k, v in host.items()}
    x = {k: v.clone() for k, v in real.items()}
    call, result = _calls(x)[name]
    call()
    torch.cuda.synchronize()
    want = result.clone()
    blank = {k: torch.zeros_like(v) for k, v in real.items()}
    side = torch.cuda.Stream()

    def late():  # the inputs arrive behind some 0.2 ms of work
        torch.cuda._sleep(400_000)
        for k in x:
            x[k].copy_(real[k])

    def clear():
        for k in x:
            x[k].copy_(blank[k])
        result.zero_()
        torch.cuda.synchronize()

    def check():
        seen = result.clone()  # (on the call's stream, behind it)
        torch.cuda.synchronize()
        assert torch.equal(seen, want)

    clear()
    late()
    call()
    check()
    # behind an event of another stream
    clear()
    with torch.cuda.stream(side):
        late()
    torch.cuda.current_stream().wait_stream(side)
    call()
    check()
    # captured: behind the copies alone, then behind two branches that join, one of them the work before the fork
    for fork in (False, True):
        graph, copy = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            if fork:
                copy.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(copy):
                    late()
                result.add_(0)
                torch.cuda.current_stream().wait_stream(copy)
            else:
                late()
            call()
            seen = result.clone()
        for _ in range(2):
            clear()
            seen.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(seen, want), f"fork {fork}"
    check_no_device_flags(dev)


def test_a_run_of_calls_that_read_each_others_results():
    """Write, read back, draft's attention and commit, decode: again and again on one workspace, against the same with a
    synchronisation behind every call."""
    dev, host = device(), _inputs(torch.Generator().manual_seed(2))
    results = []
    for wait in (True, False):
        x = {k: v.to(dev) for k, v in host.items()}
        calls = _calls(x)
        for _ in range(8):
            for name in NAMES:
                call, result = calls[name]
                call()
                if wait:
                    torch.cuda.synchronize()
                if result.dtype == BF16 and result is not x["kv"]:
                    x["new"][0].view(-1)[:result.numel()].add_(result.view(-1)[:x["new"][0].numel()])
        torch.cuda.synchronize()
        results.append({k: v.clone() for k, v in x.items()} | {k: calls[k][1].clone() for k in NAMES})
    for k in results[0]:
        assert torch.equal(results[0][k], results[1][k]), k
    check_no_device_flags(dev)


def test_drafts_behind_the_commit_that_gives_their_lengths():
    """A tree's attention whose context lengths the commit right before it writes, at the end of long moves."""
    dev, g = device(), torch.Generator().manual_seed(3)
    seqs, hkv, nodes, cached = 4, 8, 64, 900
    blocks = -(-(cached + 2 * nodes) // BS)
    tables = torch.randperm(seqs * blocks, generator=g).to(torch.int32).reshape(seqs, blocks).to(dev)
    kv = torch.randn((seqs * blocks, 2, hkv, BS, 128), generator=g).to(BF16).to(dev)
    start = (torch.arange(seqs + 1) * nodes).to(torch.int32).to(dev)
    lens = torch.full((seqs,), cached + nodes, dtype=torch.int32, device=dev)
    path = torch.arange(1, nodes, dtype=torch.int32).repeat(seqs, 1).to(dev)
    taken = torch.full((seqs,), nodes - 1, dtype=torch.int32, device=dev)
    after = torch.zeros(seqs, dtype=torch.int32, device=dev)
    mask = torch.cat([words_of(ancestors(8, g), 1) for _ in range(seqs)]).to(dev)
    few = (torch.arange(seqs + 1) * 8).to(torch.int32).to(dev)
    q = torch.randn((seqs * 8, 4 * hkv, 128), generator=g).to(BF16).to(dev)
    commit = pkv.prepare_tree_commit(*pkv.split_pool(kv), tables, start, lens, path, taken, after, max_query_len=nodes,
                                     max_context_len=cached + nodes)
    attend = pkv.prepare_paged_attention_tree(q, *pkv.split_pool(kv), tables, few, after, mask, max_query_len=8,
                                              max_context_len=cached + nodes)
    for _ in range(50):
        after.zero_()
        attend.result.zero_()
        commit()
        got = attend().clone()
        torch.cuda.synchronize()
        assert torch.equal(got, attend())
    check_no_device_flags(dev)
