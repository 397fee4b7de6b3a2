"""The operators around plain attention on pools with a wider block stride, and on blocks whose offsets pass 32 bits."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _operator_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu


def _chain(dev, k_cache, v_cache, blocks, dtype, seed):
    """Rotate and write 40 tokens of one sequence, decode with weights, prefill the last 20, evict to 16 tokens into fresh
    blocks, decode again; each step against the reference.  blocks: three for the sequence, two fresh ones."""
    bs, hkv, d, hq = 16, 2, 128, 8
    g = torch.Generator().manual_seed(seed)
    q, k, v = ((torch.randn((40, h, d), generator=g)).to(dtype) for h in (hq, hkv, hkv))
    pos = torch.arange(40)
    inv = 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    table = torch.tensor([blocks[:3]], dtype=torch.int32)
    slots = pkv.slot_mapping(table, pos, bs, token_rows=torch.zeros(40, dtype=torch.int64))
    on = lambda t: t.to(dev)
    qr = pkv.rope_reshape_and_cache(on(q), on(k), on(v), on(pos), on(inv), on(slots), k_cache, v_cache)
    torch.cuda.synchronize()
    rows = lambda cache, tab, n: torch.stack([cache[int(tab[t // bs]), :, t % bs] for t in range(n)]).cpu()
    kr, vr = rows(k_cache, blocks, 40), rows(v_cache, blocks, 40)
    axis = torch.zeros(64, dtype=torch.int32)
    ref, mag = refs.rotate(k, pos[None], axis, inv, False)
    refs.rounded_close(kr, ref, mag * 2.0 ** -20, "k")
    assert torch.equal(vr, v)
    half = refs.HALF_STEP[dtype]
    lens = torch.tensor([40], dtype=torch.int32, device=dev)
    qd = qr[39:40].contiguous()
    w = torch.zeros((1, hkv, 48), device=dev)
    out = pkv.paged_attention_decode_scored(qd, k_cache, v_cache, on(table), lens, softcap=7.0, weights_out=w, max_context_len=40)

    def attention(got, query, keys, values, p, n, softcap):
        for h in range(hq):
            kk, vv = keys[:, h // 4], values[:, h // 4]
            r, _, a = refs.attend_row(query[h].cpu(), kk, vv, d ** -0.5, softcap, 0, p, 0, n)
            refs.check_attention(got[h].cpu(), r, a, refs.score_slack(query[h].cpu(), kk, d ** -0.5, softcap, 0, 0), half, "out")

    attention(out[0], qd[0], kr, vr, 39, 40, 7.0)
    qp = qr[20:].contiguous()
    outp = pkv.paged_attention_prefill_scored(qp, k_cache, v_cache, on(table), torch.tensor([0, 20], dtype=torch.int32, device=dev),
                                              lens, max_query_len=20, max_context_len=40, softcap=7.0)
    for j in (0, 7, 19):
        attention(outp[j], qp[j], kr, vr, 20 + j, 21 + j, 7.0)
    kept, kept_lens = pkv.evict_select(w, lens, 16, sinks=1, recent=3, max_context_len=40)
    fresh = torch.tensor([blocks[3:]], dtype=torch.int32, device=dev)
    pkv.evict_compact(k_cache, v_cache, on(table), lens, kept, kept_lens, dst_block_tables=fresh)
    torch.cuda.synchronize()
    at = kept.cpu()[0].long()
    kc = torch.stack([kr[at[h], h] for h in range(hkv)], 1)
    vc = torch.stack([vr[at[h], h] for h in range(hkv)], 1)
    assert torch.equal(rows(k_cache, blocks[3:], 16), kc) and torch.equal(rows(v_cache, blocks[3:], 16), vc)
    out = pkv.paged_attention_decode_scored(qd, k_cache, v_cache, fresh, kept_lens, max_context_len=16)
    attention(out[0], qd[0], kc, vc, 15, 16, 0)
    check_no_device_flags(dev)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["f16", "bf16"])
def test_a_wider_block_stride(dtype):
    dev = device()
    pool = torch.full((9, 5, 2, 16, 128), float("nan"), dtype=dtype, device=dev)     # K and V are two of five planes
    before = pool[:, [0, 2, 4]].clone()
    _chain(dev, pool[:, 1], pool[:, 3], [7, 0, 3, 8, 1], dtype, 1)
    assert torch.equal(pool[:, [0, 2, 4]].view(torch.int16), before.view(torch.int16))


def test_blocks_past_32_bit_offsets():
    """A pool of more than 2^32 elements (and 2^33 bytes): the sequence's and the fresh blocks lie at its end."""
    dev = device()
    nb = 2 ** 32 // (2 * 2 * 16 * 128) + 64
    kv = torch.empty((nb, 2, 2, 16, 128), dtype=torch.bfloat16, device=dev)
    _chain(dev, kv[:, 0], kv[:, 1], [nb - 1, nb - 40, nb - 3, nb - 60, nb - 2], torch.bfloat16, 2)
    del kv
    torch.cuda.empty_cache()
