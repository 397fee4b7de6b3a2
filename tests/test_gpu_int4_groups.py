"""Decode over a 4-bit cache whose V rows hold groups of very different scales: each is as exact as alone."""
import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests import _int4_bounds as bounds
from tests._gpu_helpers import check_no_device_flags, device

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
# powers of two of a row's four groups (two at head_dim 64: the first and the last)
APART = [[0, -12, -17, -20], [10, 0, -8, -14], [0, -6, -7, -9]]
FAR = {F16: [[13, 2, -9, -22]], BF16: [[0, -18, -26, -40], [120, 60, 0, -60], [-20, -40, -60, -90]]}


def _v(n, hkv, d, powers, kind, dtype, g):
    x = torch.randn((n, hkv, d // 32, 32), generator=g).double()
    p = torch.tensor(powers if d == 128 else [powers[0], powers[3]]).double()
    t = torch.arange(n)
    at = (torch.arange(len(p))[None] + (t[:, None] if kind == "turns" else 0)) % len(p)
    factor = torch.exp2(p[at]).expand(n, -1).clone()
    if kind == "late":  # ordinary rows but for a few
        factor[(t != n // 2) & (t != n - 1)] = 2.0 ** powers[0]
    if kind == "offsets":  # zeros much larger than the scales, of either sign
        x = (2 + x.clamp(-1, 1) / 8) * (1 - 2 * (t % 2))[:, None, None, None]
    x *= factor[:, None, :, None]
    if kind == "zeros":  # whole groups, and whole rows, of one value
        x[t % 3 == 0, :, 0] = 0
        x[t % 3 == 1, :, -1] = x[t % 3 == 1, :, -1, :1]
        x[t % 5 == 0] = 0
    return x.flatten(2).to(dtype)


def run(dtype, hq, hkv, d, bs, lens, powers, kind, seed, spread=1.0):
    dev, g = device(), torch.Generator().manual_seed(seed)
    tables, blocks = refs.place(lens, bs, g)
    k = (torch.randn((sum(lens), hkv, d), generator=g) * spread).to(dtype)
    q = torch.randn((len(lens), hq, d), generator=g).to(dtype)
    v = torch.cat([_v(n, hkv, d, powers, kind, dtype, g) for n in lens])
    if kind == "zeros":  # the zero rows weigh the most
        at = 0
        for i, n in enumerate(lens):
            k[at:at + n:5] = (2 * q[i].view(hkv, -1, d)[:, 0].sign()).to(dtype)
            at += n
    slots = torch.cat([tables[i, torch.arange(n) // bs].long() * bs + torch.arange(n) % bs for i, n in enumerate(lens)])
    pool = torch.full((blocks, 2, hkv, bs, d * 5 // 8), 0xff, dtype=torch.uint8, device=dev)
    pkv.reshape_and_cache_int4(k.to(dev), v.to(dev), slots.to(dev), *pkv.split_pool(pool))
    got = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool), tables.to(dev),
                                          torch.tensor(lens, dtype=torch.int32, device=dev), max_context_len=max(lens)).cpu().double()
    check_no_device_flags(dev)
    parts, err, var = refs.unpack(pool.cpu(), dtype), [], []
    for i, n in enumerate(lens):
        want, bound, v2 = bounds.decode(q[i], parts, tables[i], n, dtype, d ** -0.5)
        off = (got[i] - want).abs()
        assert got[i].isfinite().all() and (off <= bound).all(), f"sequence {i} of {n}: {(off / bound.clamp(min=1e-300)).max():.2f} of the bound"
        err.append(off.unflatten(-1, (-1, 32)))
        var.append(v2.unflatten(-1, (-1, 32)))
    return torch.stack(err), torch.stack(var)


SHAPES = [(3, 3, 64, 8), (4, 1, 128, 16), (6, 2, 128, 32), (8, 1, 128, 8), (14, 2, 64, 16), (16, 1, 128, 16), (40, 2, 64, 32), (20, 1, 128, 8)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d,bs", SHAPES)
@pytest.mark.parametrize("kind", ["apart", "turns", "late", "zeros", "offsets"])
def test_groups_of_different_scales(hq, hkv, d, bs, kind, dtype):
    for i, powers in enumerate(APART + FAR[dtype]):
        run(dtype, hq, hkv, d, bs, [1, 2, 17, 33, 150, 64, 400], powers, kind, seed=hq + d + i)


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_groups_of_different_scales_in_cut_contexts(dtype):
    """Contexts cut into pieces whose references differ."""
    for kind in ("turns", "late", "zeros"):
        run(dtype, 8, 2, 128, 16, [3000, 5, 1111], APART[0], kind, seed=3, spread=3.0)


@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (40, 8, 128), (72, 8, 64)])
def test_groups_of_different_scales_in_many_contexts(hq, hkv, d):
    """Several units to a worker, whole ones behind one whose last rows differ."""
    lens = [i * 29 % 70 for i in range(400)]
    for dtype in (F16, BF16):
        run(dtype, hq, hkv, d, 16, lens, APART[0], "late", seed=4)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("hq,hkv,d,bs", [(4, 1, 128, 16), (8, 1, 64, 8), (32, 2, 128, 16)])
def test_each_group_is_as_exact_as_alone(hq, hkv, d, bs, dtype):
    """The mean error of each group over many short contexts is that of its two roundings (a quarter more, for a few hundred
    samples whose groups share theirs)."""
    for powers in ([0, 0, 0, 0], [0, -6, -7, -9], [0, -12, -17, -20]):
        err, var = run(dtype, hq, hkv, d, bs, [1 + i % 9 for i in range(64)], powers, "apart", seed=7)
        for j in range(d // 32):
            rms, want = err[:, :, j].square().sum().sqrt(), var[:, :, j].sum().sqrt()
            assert rms <= 1.25 * want, f"{powers}, group {j}: {rms / want:.3f}"
