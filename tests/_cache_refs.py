"""Plain 64-bit references of the 4-bit cache and of attention over an explicit set of visible tokens, on CPU tensors."""
from __future__ import annotations

import torch


def round_up(x, dtype):
    """x >= 0 (64 bits) -> the smallest value of dtype that is at least x."""
    r = x.float().to(dtype)
    low = r.double() < x
    return (r.view(torch.int16) + low.to(torch.int16)).view(dtype)


def quantise(x):
    """Rows [..., d] of a 16-bit type -> (codes [..., d / 32, 32] int64, scale, zero [..., d / 32] of that type)."""
    g = x.double().unflatten(-1, (-1, 32))
    low, high = g.amin(-1), g.amax(-1)
    scale = round_up((high - low) / 15, x.dtype)
    s = scale.double()[..., None]
    codes = torch.where(s > 0, (g - low[..., None]) / s, torch.zeros_like(g)).round().clamp(0, 15)
    return codes.to(torch.int64), scale, low.to(x.dtype)


def pack(codes, scale, zero):
    """Codes and parameters of blocks [..., bs, NG, 32] / [..., bs, NG] -> records [..., bs, 5 d / 8] as the pool holds them."""
    *lead, bs, ng, _ = codes.shape
    nib = torch.zeros((*lead, bs, ng * 32), dtype=torch.int64)
    for j in range(ng):
        for u in range(8):
            for e in range(4):
                nib[..., 4 * (u * ng + j) + e] = codes[..., j, 4 * u + e]
    code_bytes = (nib[..., 0::2] | (nib[..., 1::2] << 4)).to(torch.uint8)
    params = torch.stack([scale, zero], -1).contiguous().view(torch.uint8).reshape(*lead, bs, 4 * ng)
    rec = torch.cat([code_bytes.flatten(-2), params.flatten(-2)], -1)
    return rec.unflatten(-1, (bs, rec.shape[-1] // bs))


def unpack(pool, dtype):
    """Records [..., bs, 5 d / 8] -> (codes [..., bs, NG, 32] int64, scale, zero [..., bs, NG])."""
    bs, width = pool.shape[-2:]
    d = width * 8 // 5
    ng = d // 32
    rec = pool.flatten(-2)
    b = rec[..., :bs * d // 2].unflatten(-1, (bs, d // 2)).to(torch.int64)
    nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    codes = torch.zeros((*nib.shape[:-1], ng, 32), dtype=torch.int64)
    for j in range(ng):
        for u in range(8):
            for e in range(4):
                codes[..., j, 4 * u + e] = nib[..., 4 * (u * ng + j) + e]
    params = rec[..., bs * d // 2:].unflatten(-1, (bs, d // 8)).contiguous().view(dtype).unflatten(-1, (ng, 2))
    return codes, params[..., 0], params[..., 1]


def values(pool, dtype):
    """What a 4-bit pool's codes stand for, [..., bs, d] in 64 bits."""
    codes, scale, zero = unpack(pool, dtype)
    return (codes.double() * scale.double()[..., None] + zero.double()[..., None]).flatten(-2)


def context(pool, table, n):
    """K, V [n, Hkv, d] of a sequence: pool [NB, 2, Hkv, bs, d], table its block ids."""
    bs = pool.shape[3]
    blocks = pool[table[:-(-n // bs)].long()].transpose(2, 3).reshape(-1, 2, bs, pool.shape[2], pool.shape[4])
    kv = blocks.transpose(0, 1).reshape(2, -1, pool.shape[2], pool.shape[4])[:, :n]
    return kv[0], kv[1]


def attend(q, k, v, scale, seen):
    """q [R, Hq, d] over k, v [n, Hkv, d] where seen [R, n]: (out [R, Hq, d], sum of weight * |v|, largest sum of
    |q||k| of a visible token per row and head), in 64 bits; hidden rows of k and v are not read."""
    r, hq, d = q.shape
    g = hq // k.shape[1]
    use = seen.any(0)
    k, v, seen = k[use].double(), v[use].double(), seen[:, use]
    out, mag = torch.zeros((r, hq, d), dtype=torch.float64), torch.zeros((r, hq, d), dtype=torch.float64)
    most = torch.zeros((r, hq, 1), dtype=torch.float64)
    for h in range(hq):
        x = q[:, h].double() @ k[:, h // g].T * scale
        x[~seen] = -torch.inf
        w = torch.softmax(x, 1).nan_to_num(nan=0.0)
        out[:, h], mag[:, h] = w @ v[:, h // g], w @ v[:, h // g].abs()
        size = (q[:, h].double().abs() @ k[:, h // g].abs().T).masked_fill(~seen, 0.0)
        if size.shape[1]:
            most[:, h, 0] = size.amax(1) * abs(scale)
    return out, mag, most


def place(lens, bs, g, spare=2):
    """Random tables for contexts of these lengths (entries past a context are bad ones), and the pool's blocks."""
    need = [-(-n // bs) for n in lens]
    perm, at = torch.randperm(sum(need) + spare, generator=g).to(torch.int32), 0
    tables = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)
    for i, n in enumerate(need):
        tables[i, :n] = perm[at:at + n]
        at += n
    return tables, len(perm)


def poison(kv, tables, tokens):
    """NaN and infinities into every row of the pool but the given tokens (a list per sequence)."""
    bs = kv.shape[3]
    covered = torch.zeros(kv.shape[0], bs, dtype=torch.bool)
    for i, ts in enumerate(tokens):
        for t in ts:
            covered[tables[i, t // bs], t % bs] = True
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=kv.dtype)
    for k, (b, o) in enumerate((~covered).nonzero().tolist()):
        kv[b, :, :, o] = bad[k % 3]


def attention_bound(mag, most, d, p_half, int8_q=0.0):
    """How far an output may be from exact before its last rounding: every product and partial sum of a score rounds once at
    2^-23 (tensor cores truncate) of the summed magnitudes, scaling adds a few of its size; both sides of the softmax's
    quotient carry that; each weight is rounded once to the MMA's type, as is the row sum (p_half each).  int8_q: the
    relative error of an INT8 cache's fp16 query."""
    slack = most * ((d + 8) * 2.0 ** -23 + 2.0 ** -20 + int8_q)
    return mag * (2 * slack + 2 * p_half + 2.0 ** -18)
