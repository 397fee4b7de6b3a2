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
