"""How far a decode over a 4-bit cache may be from its definition, from the arithmetic of its roundings."""
from __future__ import annotations

import torch

from tests._operator_refs import HALF_STEP, TINY


def decode(q, parts, table, n, dtype, scale):
    """One sequence: q [Hq, d], its pool's codes, scales and zeros (unpack), its block ids, n tokens -> (out [Hq, d], bound,
    variance), in 64 bits.

    bound: a score's products and partial sums round at 2^-23 (tensor cores truncate) of the summed magnitudes |q| (s c + |z|),
    32 in a group, then a few per group, and its scaling a few times more (2^-20); both sides of the softmax's quotient carry
    that, a weight's exponential and the sums of p and of p z another 2^-18.  The product p s is rounded once to fp16, 2^-11, which
    counts for c, or for |c - 8| in fp16 rows.  Below 2^-14 it is rounded at 2^-25, where the largest p s of the token's row
    have 2^6 or more and the group's own are within 2^-8 of them, or at less where they are not.
    variance: of the roundings of p s and of the output alone: uniform over half a step to either side, whose mean
    square over a binade's mantissas is 0.541 / 3 of the relative half step's."""
    hq, d = q.shape
    codes, s, z = parts
    hkv, bs, ng = codes.shape[2:5]
    at = table[:-(-n // bs)].long()
    # [blocks, 2, hkv, bs, ...] -> [2, n, hkv, ...]
    take = lambda t: t[at].double().transpose(2, 3).transpose(0, 1).flatten(1, 2)[:, :n]  # noqa: E731
    c, s, z = take(codes), take(s)[..., None], take(z)[..., None]
    # channel 32 j + i of a token: code i of group j
    flat = lambda t: t.expand(2, n, hkv, ng, 32).flatten(-2)  # noqa: E731
    value, size = flat(s * c + z), flat(s * c + z.abs())
    mid = 8.0 if dtype is torch.float16 else 0.0
    coded = flat(s * (c - mid).abs())
    held = flat(s * (c - mid).abs() + z.abs() + mid * s)
    one = flat(s)
    out, bound, var = (torch.zeros((hq, d), dtype=torch.float64) for _ in range(3))
    if n == 0:
        return out, bound, var
    for h in range(hq):
        g = h // (hq // hkv)
        x = value[0, :, g] @ q[h].double() * scale
        p = torch.softmax(x, 0)
        most = (size[0, :, g] @ q[h].double().abs()).max() * abs(scale)
        slack = most * ((32 + 2 * ng + 8) * 2.0 ** -23 + 2.0 ** -20)
        out[h] = p @ value[1, :, g]
        ps = p[:, None] * one[1, :, g]
        bound[h] = p @ coded[1, :, g] * 2.0 ** -11 + (p @ held[1, :, g]) * (2 * slack + 2.0 ** -18) + 16 * n * 2.0 ** -23 * ps.amax(0)
        var[h] = (p[:, None] ** 2 * coded[1, :, g] ** 2).sum(0) * 2.0 ** -22 * 0.541 / 3
    most = torch.finfo(dtype).max
    clipped = out.clamp(-most, most)
    step = torch.exp2(torch.floor(torch.log2(clipped.abs().clamp(min=torch.finfo(dtype).smallest_normal)))) * HALF_STEP[dtype]
    return clipped, (clipped.abs() + bound) * HALF_STEP[dtype] + bound + TINY[dtype], var + step ** 2 / 3
