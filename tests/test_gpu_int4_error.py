"""Decode over a 4-bit cache: every output within the bound of the roundings that the kernel makes, and their mean."""
import math

import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests import _int4_bounds as bounds
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def _run(dtype, hq, hkv, d, bs, lens, seed, scale):
    dev, g = device(), torch.Generator().manual_seed(seed)
    tables, blocks = refs.place(lens, bs, g)
    x = (torch.randn((blocks, 2, hkv, bs, d), generator=g) * 0.8 + torch.randn((1, 2, hkv, 1, d), generator=g) * 0.5).to(dtype)
    parts = refs.quantise(x)
    q = (torch.randn((len(lens), hq, d), generator=g) * 2).to(dtype)
    got = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(refs.pack(*parts).to(dev)), tables.to(dev),
                                          torch.tensor(lens, dtype=torch.int32, device=dev), scale,
                                          max_context_len=max(lens)).cpu().double()
    check_no_device_flags(dev)
    err, var = [], []
    for i, n in enumerate(lens):
        want, bound, v = bounds.decode(q[i], parts, tables[i], n, dtype, scale)
        off = (got[i] - want).abs()
        assert (off <= bound).all(), f"sequence {i} of {n}: {(off / bound.clamp(min=1e-300)).max():.2f} of the bound"
        err.append(off.square().sum())
        var.append(v.sum())
    return math.sqrt(sum(err)), math.sqrt(sum(var))


SHAPES = [(2, 2, 64, 8), (4, 1, 128, 16), (8, 1, 64, 32), (14, 2, 128, 8), (16, 1, 128, 16), (40, 2, 64, 16)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_outputs_within_their_roundings(hq, hkv, d, bs, dtype):
    _run(dtype, hq, hkv, d, bs, [0, 1, 2, 31, 33, 100, 257, 1300], hq + d, d ** -0.5)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
def test_mean_error_is_that_of_two_roundings(hq, hkv, d, bs, dtype):
    """Short contexts, where a rounding of a weight shows: a weight that counted for its whole code in fp16 rows, or had fewer
    bits, would exceed the quarter that is left for a few hundred samples and fp32."""
    err, want = _run(dtype, hq, hkv, d, bs, [1 + i % 12 for i in range(96)], hq + d + 1, d ** -0.5)
    assert err <= 1.25 * want, f"{err / want:.3f}"


def test_mean_error_over_long_contexts():
    for dtype in (F16, BF16):
        err, want = _run(dtype, 8, 2, 128, 16, [700 + 97 * i for i in range(8)], 5, 128 ** -0.5)
        assert err <= 1.25 * want, f"{err / want:.3f}"
