"""The sink decode over an INT8 cache: its mean error is that of the weights' and the output's roundings."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hkv,d,bs", [(8, 8, 64, 8), (8, 8, 64, 32), (4, 2, 64, 16), (16, 4, 128, 16), (8, 1, 128, 16), (20, 2, 64, 16)])
def test_a_score_is_as_exact_as_the_codes(hq, hkv, d, bs):
    """Few visible tokens and large scores, so that an error of a score shows.  The weights are rounded to fp16 (a relative 2^-11
    at most), the output once: each uniform over half a step to either side, a mean square of 0.541 / 3 of the relative half
    step's over a binade; a quarter more for what the few samples and fp32 add.  A query held in one fp16 number would add
    2^-11 |q| |k| to every score, which nearly doubles the error."""
    dtype = torch.float16
    dev, g = device(), torch.Generator().manual_seed(hq + d + bs)
    seqs, window, sinks, scale = 64, 14, 2, 4 * d ** -0.5
    lens = [30 + i % 40 for i in range(seqs)]
    tables, blocks = refs.place(lens, bs, g)
    q = (torch.randn((seqs, hq, d), generator=g) * 2).to(dtype)
    kv = torch.randint(-127, 128, (blocks, 2, hkv, bs, d), generator=g, dtype=torch.int8)
    scales = [(torch.rand((hkv, d), generator=g) + 0.5) / 64 for _ in range(2)]
    got = pkv.paged_attention_decode_sinks_int8(
        q.to(dev), *pkv.split_pool(kv.to(dev)), scales[0].to(dev), scales[1].to(dev), tables.to(dev),
        torch.tensor(lens, dtype=torch.int32, device=dev), scale, window=window, sinks=sinks, max_context_len=max(lens)).cpu().double()
    check_no_device_flags(dev)
    vals = kv.double() * torch.stack(scales).double()[:, :, None]
    err = torch.zeros((seqs, hq, d), dtype=torch.float64)
    var = torch.zeros_like(err)
    half = torch.finfo(dtype).eps / 2
    for i, n in enumerate(lens):
        k, v = refs.context(vals, tables[i], n)
        use = [t for t in range(n) if t < sinks or t >= n - window]
        k, v = k[use].transpose(0, 1).repeat_interleave(hq // hkv, 0), v[use].transpose(0, 1).repeat_interleave(hq // hkv, 0)
        p = torch.softmax((k @ q[i].double()[..., None])[..., 0] * scale, -1)
        want = (p[:, None] @ v)[:, 0]
        err[i] = got[i] - want
        step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -20)))) * half
        var[i] = step ** 2 / 3 + (p[:, None] ** 2 @ v ** 2)[:, 0] * 2.0 ** -22 * 0.541 / 3
    rms, bound = err.square().sum().sqrt().item(), var.sum().sqrt().item()
    assert rms <= 1.25 * bound, f"{rms / bound:.3f}"
