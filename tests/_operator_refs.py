"""Plain 64-bit references of the operators around plain attention (rotary write, scored
attention, eviction), on CPU tensors and one row at a time, and the arithmetic behind the
tests' tolerances."""
from __future__ import annotations

import math

import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}   # relative, of one rounding
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}              # half a subnormal step of fp16


def rotate(x, positions, axis, inv_freq, interleaved):
    """x [T, H, d] -> the rotated rows in 64 bits, and |a| + |b| of each value's pair."""
    y = x.double().clone()
    mag = y.abs().clone()
    pairs = len(inv_freq)
    for i in range(pairs):
        angle = positions[int(axis[i])].double() * float(inv_freq[i])
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        a, b = x[..., ia].double(), x[..., ib].double()
        y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
        mag[..., ia] = mag[..., ib] = a.abs() + b.abs()
    return y, mag


def rounded_close(got, ref, slack, what):
    """got (16-bit) is ref rounded once, where ref itself may be off by `slack`."""
    half, tiny = HALF_STEP[got.dtype], TINY[got.dtype]
    bound = (ref.abs() + slack) * half + slack + tiny
    err = (got.double() - ref).abs()
    assert torch.isfinite(got).all(), what
    worst = (err / bound.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound, max abs err {err.max().item():.3e}"


def select(weights, lens, budget, sinks, recent):
    """kept [B, Hkv, budget] and kept_lens by sorting (-weight, position); NaN ranks last."""
    b, hkv, _ = weights.shape
    kept = torch.full((b, hkv, budget), -1, dtype=torch.int32)
    for i in range(b):
        n = int(lens[i])
        m = min(n, budget)
        fixed = set(range(n)) if n <= budget else set(range(sinks)) | set(range(n - recent, n))
        for h in range(hkv):
            w = weights[i, h, :n].tolist()
            rest = sorted((t for t in range(n) if t not in fixed),
                          key=lambda t: (math.isnan(w[t]), 0.0 if math.isnan(w[t]) else -w[t], t))
            kept[i, h, :m] = torch.tensor(sorted(fixed | set(rest[:m - len(fixed)])), dtype=torch.int32)
    return kept, torch.tensor([min(int(n), budget) for n in lens], dtype=torch.int32)


def compact(kv, tables, kept, kept_lens, dst):
    """A copy of the pool [NB, 2, Hkv, bs, d] with the kept rows moved into `dst`'s blocks."""
    src, out, bs = kv, kv.clone(), kv.shape[3]
    for i, n in enumerate(kept_lens.tolist()):
        for h in range(kv.shape[2]):
            for j in range(n):
                t = int(kept[i, h, j])
                out[dst[i, j // bs], :, h, j % bs] = src[tables[i, t // bs], :, h, t % bs]
    return out


def score_row(q, k, scale, softcap, slope, pos, lo, hi):
    """Scores of one query [d] (64 bits) against k [n, d]; -inf outside [lo, hi)."""
    x = (k.double() @ q.double()) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    t = torch.arange(k.shape[0], dtype=torch.float64)
    x = x + slope * (t - pos)
    x[(t < lo) | (t >= hi)] = -math.inf
    return x


def attend_row(q, k, v, scale, softcap, slope, pos, lo, hi):
    """(output [d], weights [n], sum of weight * |v| [d]) of one query row; an empty row gives zeros.
    Only the visible rows of v are read."""
    x = score_row(q, k, scale, softcap, slope, pos, lo, hi)
    seen = torch.isfinite(x)
    w = torch.zeros_like(x)
    if seen.any():
        w[seen] = torch.softmax(x[seen], 0)
    vs = v[seen].double()
    return w[seen] @ vs, w, w[seen] @ vs.abs()


def score_slack(q, k, scale, softcap, slope, span, int8=False):
    """How far a kernel's fp32 score of q [d] against rows k [n, d] may be from exact: every product of the dot product and
    every partial sum rounds once at 2^-23 (tensor cores truncate) of the summed magnitudes; an INT8 cache's query is first
    rounded to fp16 after scaling by a power of two (2^-11 of each product, or 2^-24 of the largest query channel);
    capping and the bias add a few roundings of the score's and the bias's size."""
    mag = (k.double().abs() @ q.double().abs()).max().item() * abs(scale) if k.shape[0] else 0.0
    d = q.shape[0]
    slack = mag * (d + 8) * 2.0 ** -23
    if int8 and k.shape[0]:
        slack += mag * 2.0 ** -11 + abs(scale) * d * 2.0 ** -24 * q.abs().max().item() * k.abs().max().item()
    return slack + (mag + min(softcap, mag) + abs(slope) * span) * 2.0 ** -21


def check_attention(got, ref, absref, slack, p_half, what):
    """An attention output row [d] against exact `ref`: each weight is off by the score slack on both sides of the quotient
    (factor 2) and by one rounding of the weights to the MMA's type, which the row sum shares (factor 2)."""
    rounded_close(got, ref, absref * (2 * slack + 2 * p_half + 2.0 ** -18), what)
