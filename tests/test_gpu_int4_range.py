"""4-bit cache at the ends of its types' range: every finite row is within half a step, and no finite row reads back as
anything but a finite one."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


def far_rows(dtype, d, g):
    """[40, 3, d] finite rows whose groups spread over up to twice the type's range, between ordinary and tiny ones."""
    most = torch.finfo(dtype).max
    x = (torch.rand((40, 3, d // 32, 32), generator=g).double() * 2 - 1) * most
    n = torch.arange(40)
    x[n % 5 == 1] *= 2.0 ** -3
    x[n % 5 == 2, :, 0] /= most                       # one ordinary group beside far ones
    x[n % 5 == 3] = x[n % 5 == 3].abs()
    x[n % 5 == 4, 1] *= 2.0 ** -8 if dtype is F16 else 2.0 ** -240  # one head of tiny rows
    x[:8, :, :, 3], x[:8, :, :, 30] = -most, most     # the whole range
    x[8:16, :, :, 7], x[8:16, :, :, 9] = -most / 2, most / 2  # a spread of one range
    x[16:20] = most
    x[20:24] = -most
    x[24:28] = x[24:28].clamp(min=0)
    x[24:28, :, :, 5] = 0
    x[24:28, :, :, 6] = most
    x = x.clamp(-most, most).to(dtype).flatten(2)
    assert x.isfinite().all()
    return x


def written(x, bs, dev):
    """K and V pools of blocks 0 .. that hold the rows in order."""
    t, hkv, d = x.shape
    pool = pkv.int4_pool(t // bs, hkv, bs, d, dev)
    pkv.reshape_and_cache_int4(x.to(dev), x.flip(0).contiguous().to(dev), torch.arange(t).to(dev), *pkv.split_pool(pool))
    check_no_device_flags(dev)
    return pool


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_write_of_rows_that_span_the_range(dtype, d):
    x = far_rows(dtype, d, torch.Generator().manual_seed(d))
    pool = written(x, 8, device()).cpu()
    want = torch.stack([x, x.flip(0)]).unflatten(1, (5, 8)).permute(1, 0, 3, 2, 4)  # [5, 2, 3, 8, d]
    codes, scale, zero = refs.unpack(pool, dtype)
    c, s, z = refs.quantise(want)
    assert scale.isfinite().all() and torch.equal(scale, s) and torch.equal(zero, z) and torch.equal(codes, c)
    step = scale.double().repeat_interleave(32, -1)
    assert (refs.values(pool, dtype) - want.double()).abs().le(step / 2).all()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
def test_finite_rows_read_back_finite(dtype, d):
    """A scale rounded up can put the largest code past the type's range: it stands for the largest finite value."""
    dev, most = device(), torch.finfo(dtype).max
    x = far_rows(dtype, d, torch.Generator().manual_seed(d + 1))
    pool = written(x, 8, dev)
    kv = torch.zeros((5, 2, 3, 8, d), dtype=dtype, device=dev)
    pkv.dequantise_blocks_int4(*pkv.split_pool(pool), torch.arange(5, device=dev)[:, None].expand(5, 2).contiguous(), *pkv.split_pool(kv))
    check_no_device_flags(dev)
    want = refs.values(pool.cpu(), dtype)
    assert (want.abs() > most).any()
    # c s is exact in fp32 (15 bits), the sum is rounded there and then to the type
    assert torch.equal(kv.cpu(), (want / 4).float().double().mul(4).clamp(-most, most).to(dtype))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_an_infinity_reads_back_as_nan(dtype):
    dev = device()
    x = torch.randn((8, 1, 64), generator=torch.Generator().manual_seed(2)).to(dtype)
    x[1, 0, 3], x[2, 0, 40], x[3, 0, :32] = float("inf"), -float("inf"), float("inf")
    pool, kv = written(x, 8, dev), torch.zeros((1, 2, 1, 8, 64), dtype=dtype, device=dev)
    pkv.dequantise_blocks_int4(*pkv.split_pool(pool), torch.zeros((1, 2), dtype=torch.int64, device=dev), *pkv.split_pool(kv))
    got = kv.cpu()[0, 0, 0].isnan().unflatten(-1, (2, 32))
    want = torch.zeros((8, 2, 32), dtype=torch.bool)
    want[1, 0], want[2, 1], want[3, 0] = True, True, True
    assert torch.equal(got, want)


def heads(hq, hkv):
    return [h // (hq // hkv) for h in range(hq)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d", [(3, 3, 64), (12, 3, 128), (24, 3, 128), (48, 3, 64)])
def test_decode_over_far_rows_is_finite(hq, hkv, d, dtype):
    """Contexts of one token return its V row, at the ends of the type's range too."""
    dev, most, g = device(), torch.finfo(dtype).max, torch.Generator().manual_seed(d + 2)
    v = far_rows(dtype, d, g)
    k, q = torch.randn((40, 3, d), generator=g).to(dtype), torch.randn((40, hq, d), generator=g).to(dtype)
    pool = pkv.int4_pool(40, hkv, 8, d, dev)
    pkv.reshape_and_cache_int4(k.to(dev), v.to(dev), torch.arange(40).to(dev) * 8, *pkv.split_pool(pool))
    got = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool), torch.arange(40, dtype=torch.int32, device=dev)[:, None],
                                          torch.ones(40, dtype=torch.int32, device=dev), max_context_len=1).cpu()
    check_no_device_flags(dev)
    _, s, z = refs.unpack(pool.cpu(), dtype)
    spread = lambda t: t[:, 1, :, 0].double().repeat_interleave(32, -1)[:, heads(hq, hkv)]  # noqa: E731
    want = refs.values(pool.cpu(), dtype)[:, 1, :, 0][:, heads(hq, hkv)]
    assert (want.abs() > most).any() and got.isfinite().all()
    # p s is rounded once to fp16 (15 codes), the sums a few times in fp32, the output once
    slack = 15 * spread(s) * 2.0 ** -11 + (15 * spread(s) + spread(z).abs()) * 2.0 ** -18
    half = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype is F16 else 0.0
    assert (got.double() - want.clamp(-most, most)).abs().le(want.abs() * half + slack * (1 + half) + tiny).all()
