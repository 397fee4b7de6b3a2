"""Timed cases of the operators around the paged KV cache that a decoding or prefilling
model calls next to plain attention:

  rope    rotary positions with up to four axes on the queries and the new keys, and the
          write of the rotated keys and the values into their cache slots
  decode  one query token per sequence over its paged context, with capped scores, a
          distance bias, a window, a first visible token, and accumulated attention weights
  prefill a chunk of new tokens per sequence over its paged context, with the same score
          forms, document starts and a prefix that every row sees
  evict   the choice of the tokens to keep by accumulated weight, per KV head, and the move
          of their rows into fresh blocks

``own`` selects the library's calls; otherwise every operator runs in its plain form.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the new token of 64 sequences, three-axis positions: the write before a decode step
        dict(name="rope_step", op="rope", tokens=64, hq=32, hkv=8, d=128, bs=16, dtype="f16", int8=False,
             axes=3, rot=128, interleaved=False, far=40000),
        # a video's patches and their text as one chunk: time, height and width positions
        dict(name="rope_video_chunk", op="rope", tokens=8192, hq=64, hkv=8, d=128, bs=16, dtype="bf16", int8=False,
             axes=3, rot=128, interleaved=False, far=1000000),
        # a quantised cache and a partial rotation in adjacent pairs, an odd chunk
        dict(name="rope_int8_partial", op="rope", tokens=1777, hq=32, hkv=32, d=64, bs=32, dtype="bf16", int8=True,
             axes=2, rot=32, interleaved=True, far=8000),
        # local layers of a grouped model: capped scores over the last 1024 tokens
        dict(name="decode_cap_window", op="decode", seqs=64, lo=128, hi=8192, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16", cap=30.0, slopes=False, window=1024, starts=False, weights=False),
        # distance bias over full contexts, a query head per KV head
        dict(name="decode_slopes", op="decode", seqs=32, lo=4096, hi=4096, hq=32, hkv=32, d=128, bs=16,
             dtype="f16", cap=0.0, slopes=True, window=0, starts=False, weights=False),
        # ragged contexts whose weights are accumulated for eviction
        dict(name="decode_weights", op="decode", seqs=64, lo=128, hi=8192, hq=32, hkv=8, d=128, bs=16,
             dtype="f16", cap=0.0, slopes=False, window=0, starts=False, weights=True),
        # two long contexts, capped, with their weights
        dict(name="decode_weights_long", op="decode", seqs=2, lo=30000, hi=32768, hq=64, hkv=8, d=128, bs=32,
             dtype="bf16", cap=50.0, slopes=False, window=0, starts=False, weights=True),
        # chunks behind cached tokens in a local layer with capped scores
        dict(name="prefill_cap_window", op="prefill", seqs=8, chunk=512, ragged=False, cached=7680, hq=64, hkv=8, bs=16,
             dtype="bf16", cap=50.0, slopes=False, window=2048, docs=0, prefix=0),
        # whole prompts with a distance bias
        dict(name="prefill_slopes", op="prefill", seqs=2, chunk=2048, ragged=False, cached=0, hq=32, hkv=32, bs=16,
             dtype="f16", cap=0.0, slopes=True, window=0, docs=0, prefix=0),
        # packed documents in ragged prompts, and images in front that every row sees whole
        dict(name="prefill_docs_prefix", op="prefill", seqs=9, chunk=777, ragged=True, cached=0, hq=32, hkv=8, bs=32,
             dtype="bf16", cap=0.0, slopes=False, window=0, docs=3, prefix=256),
        # a batch cut back to a quarter of its tokens
        dict(name="evict_batch", op="evict", seqs=32, lo=2048, hi=4096, hkv=8, d=128, bs=16, dtype="f16",
             budget=1024, sinks=4, recent=128),
        # long contexts cut back to 8192 tokens
        dict(name="evict_long", op="evict", seqs=3, lo=30001, hi=32768, hkv=8, d=128, bs=32, dtype="bf16",
             budget=8192, sinks=16, recent=2048),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill", "evict"])
    bs = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    hq, hkv = rng.choice([(32, 32), (32, 8), (64, 8), (128, 8), (32, 16), (20, 4), (12, 12)])
    d = rng.choice([64, 128, 128])
    cap = rng.choice([0.0, 20.0, 50.0])
    if op == "rope":
        tokens = min(_log(rng, 1, 8192), 8192 * 80 * 128 // ((hq + 2 * hkv) * d))
        return dict(op=op, tokens=tokens, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype, int8=rng.random() < 0.3,
                    axes=rng.randint(1, 4), rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4,
                    far=_log(rng, 100, 1000000))
    if op == "decode":
        hi = _log(rng, 16, 32768)
        seqs = max(1, min(_log(rng, 1, 64), 32 * 4096 * 32 * 128 // (hi * hkv * d)))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs,
                    dtype=dtype, cap=cap, slopes=rng.random() < 0.4, window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    starts=rng.random() < 0.3, weights=rng.random() < 0.5)
    if op == "prefill":
        chunk, cached = _log(rng, 2, 2048), rng.choice([0, _log(rng, 1, 7680)])
        most = 8 * 512 * 64 * 4352
        seqs = max(1, min(rng.randint(1, 9), most // (chunk * hq * (chunk // 2 + cached))))
        return dict(op=op, seqs=seqs, chunk=chunk, ragged=rng.random() < 0.5, cached=cached, hq=hq, hkv=hkv, bs=bs,
                    dtype=dtype, cap=cap, slopes=rng.random() < 0.4, window=rng.choice([0, 0, _log(rng, 1, 4096)]),
                    docs=rng.choice([0, 0, rng.randint(1, 6)]), prefix=rng.choice([0, 0, _log(rng, 1, 512)]))
    hi = _log(rng, 64, 32768)
    seqs = max(1, min(_log(rng, 1, 64), 32 * 4096 * 8 * 128 // (hi * hkv * d)))
    budget = max(2, int(hi * rng.uniform(0.1, 0.9)))
    return dict(op=op, seqs=seqs, lo=hi // 2 + 1, hi=hi, hkv=hkv, d=d, bs=bs, dtype=dtype, budget=budget,
                sinks=rng.randint(0, min(16, budget // 2)), recent=rng.randint(0, budget // 2))


# ---------------------------------------------------------------------------- inputs
def _gens(seed):
    return torch.Generator(device="cuda").manual_seed(seed), torch.Generator().manual_seed(seed)


def _randn(shape, dtype, gen, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _lens(n, lo, hi, host):
    lens = torch.randint(max(1, lo), hi + 1, (n,), generator=host)
    lens[0] = hi
    return lens


def _tables(lens, bs, gen, spare=0):
    """Seeded random placement of every sequence's blocks; unused entries 0."""
    need = (lens + bs - 1) // bs
    mb, total = int(need.max()), int(need.sum())
    perm = torch.randperm(total + spare, generator=gen, device="cuda").to(torch.int32)
    used = torch.arange(mb)[None, :] < need[:, None]
    tables = torch.zeros((len(lens), mb), dtype=torch.int32, device="cuda")
    tables[used.cuda()] = perm[:total]
    return tables, perm[total:], total + spare


def _slopes(hq):
    """The geometric ladder 2^(-8 (h + 1) / heads)."""
    return torch.exp2(-8.0 * torch.arange(1, hq + 1, dtype=torch.float64) / hq).float().cuda()


def _pool(c, blocks, gen):
    dtype = DTYPES[c["dtype"]]
    return torch.randn((blocks, 2, c["hkv"], c["bs"], c["d"]), generator=gen, device="cuda", dtype=dtype)


def _prepare_rope(c, seed):
    gen, host = _gens(seed)
    dtype, t, hq, hkv, d = DTYPES[c["dtype"]], c["tokens"], c["hq"], c["hkv"], c["d"]
    qkv = _randn((t, (hq + 2 * hkv) * d), dtype, gen)  # the projection's rows: q, k and v side by side
    pairs = c["rot"] // 2
    inv_freq = (1e6 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).cuda()
    # images of 24 x 24 patches over time behind some text; further axes as the first
    at = torch.arange(t, dtype=torch.int64) + int(torch.randint(0, c["far"], (1,), generator=host))
    grid = [at, at // 24 % 24 + at[0], at % 24 + at[0], at - at[0]]
    positions = torch.stack(grid[:c["axes"]]).cuda()
    share = [pairs * (a + 1) // c["axes"] for a in range(c["axes"])]
    axis = torch.tensor([next(a for a in range(c["axes"]) if i < share[a]) for i in range(pairs)], dtype=torch.int32)
    blocks = (t + c["bs"] - 1) // c["bs"] + 3
    if t <= 256:  # decode steps: each token in a block of its own sequence
        slots = torch.randperm(blocks * c["bs"], generator=gen, device="cuda")[:t].contiguous()
    else:  # a chunk fills the blocks of its table
        table = torch.randperm(blocks, generator=gen, device="cuda")
        i = torch.arange(t, device="cuda")
        slots = table[i // c["bs"]] * c["bs"] + i % c["bs"]
    s = dict(case=c, q=qkv[:, :hq * d].view(t, hq, d), k=qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d),
             v=qkv[:, (hq + hkv) * d:].view(t, hkv, d), positions=positions, axis=axis.cuda(), inv_freq=inv_freq,
             slots=slots, q_out=torch.zeros((t, hq, d), dtype=dtype, device="cuda"))
    shape = (blocks, 2, hkv, c["bs"], d)
    if c["int8"]:
        s["kv"] = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
        s["k_scale"], s["v_scale"] = (
            (torch.rand((hkv, d), generator=gen, device="cuda") + 0.5) / 32 for _ in range(2))
        s["scales"] = torch.stack([s["k_scale"], s["v_scale"]])[:, :, None]
        s["values"] = torch.zeros(shape, dtype=dtype, device="cuda")
    else:
        s["kv"] = torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return s


def _prepare_decode(c, seed):
    gen, host = _gens(seed)
    lens = _lens(c["seqs"], c["lo"], c["hi"], host)
    tables, _, blocks = _tables(lens, c["bs"], gen, spare=2)
    q = _randn((c["seqs"], c["hq"], c["d"]), DTYPES[c["dtype"]], gen, 2.0)
    s = dict(case=c, q=q, kv=_pool(c, blocks, gen), tables=tables, lens=lens.to(torch.int32).cuda(),
             max_len=int(lens.max()), scale=1 / math.sqrt(c["d"]), out=torch.zeros_like(q),
             slopes=_slopes(c["hq"]) if c["slopes"] else None, starts=None, weights=None, weights_out=None)
    if c["starts"]:  # the first visible token of each sequence, the last one among them
        s["starts"] = torch.minimum(torch.randint(0, c["hi"], (c["seqs"],), generator=host), lens - 1).to(torch.int32).cuda()
    if c["weights"]:
        shape = (c["seqs"], c["hkv"], tables.shape[1] * c["bs"])
        s["weights"] = torch.rand(shape, generator=gen, device="cuda") * 0.01
        s["weights_out"] = torch.zeros(shape, device="cuda")
    return s


def _prepare_prefill(c, seed):
    gen, host = _gens(seed)
    b, c = c["seqs"], dict(c, d=128)
    share = torch.arange(b) * 5 % b + 1 if c["ragged"] else b  # ragged: each share of the longest chunk once
    chunk = (c["chunk"] * share + b - 1) // b * torch.ones(b, dtype=torch.int64)
    lens = chunk + torch.randint(0, c["cached"] + 1, (b,), generator=host)
    tables, _, blocks = _tables(lens, c["bs"], gen, spare=2)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), chunk.cumsum(0)])
    rows = int(start[-1])
    q = _randn((rows, c["hq"], 128), DTYPES[c["dtype"]], gen, 2.0)
    s = dict(case=c, q=q, kv=_pool(c, blocks, gen), tables=tables, lens=lens.to(torch.int32).cuda(),
             query_start=start.to(torch.int32).cuda(), max_chunk=int(chunk.max()), max_len=int(lens.max()),
             scale=1 / math.sqrt(128), out=torch.zeros_like(q), slopes=_slopes(c["hq"]) if c["slopes"] else None,
             starts=None, prefix=None)
    if c["docs"]:  # document borders in each sequence; a row's document starts at the last one before it
        edges = (torch.rand((b, c["docs"]), generator=host) * lens[:, None]).long()
        seq = torch.repeat_interleave(torch.arange(b), chunk)
        pos = torch.arange(rows) - start[seq] + (lens - chunk)[seq]
        e = edges[seq]
        s["starts"] = torch.where(e <= pos[:, None], e, 0).amax(1).to(torch.int32).cuda()
    if c["prefix"]:
        s["prefix"] = torch.randint(0, c["prefix"] + 1, (b,), generator=host).to(torch.int32).cuda()
    return s


def _prepare_evict(c, seed):
    gen, host = _gens(seed)
    lens = _lens(c["seqs"], c["lo"], c["hi"], host)
    kept = torch.minimum(lens, torch.tensor(c["budget"]))
    fresh = (kept + c["bs"] - 1) // c["bs"]
    most = c["seqs"] * (-(-c["hi"] // c["bs"]) + -(-c["budget"] // c["bs"]))  # the pool's size, whatever the lengths
    used = int(((lens + c["bs"] - 1) // c["bs"]).sum())
    tables, free, blocks = _tables(lens, c["bs"], gen, spare=most - used)
    dst = torch.zeros((c["seqs"], int(fresh.max())), dtype=torch.int32, device="cuda")
    dst[(torch.arange(dst.shape[1])[None, :] < fresh[:, None]).cuda()] = free[:int(fresh.sum())]
    shape = (c["seqs"], c["hkv"], tables.shape[1] * c["bs"])
    # a few heavy tokens in a long tail; equal weights happen (2^-11 steps relative)
    weights = torch.rand(shape, generator=gen, device="cuda").pow_(8).half().float()
    return dict(case=c, kv=_pool(c, blocks, gen), tables=tables, dst=dst, lens=lens.to(torch.int32).cuda(),
                max_len=int(lens.max()), weights=weights, weights_out=torch.zeros(shape, device="cuda"))


def prepare(case, seed):
    made = dict(rope=_prepare_rope, decode=_prepare_decode, prefill=_prepare_prefill, evict=_prepare_evict)
    state = made[case["op"]](case, seed)
    state["handle"] = []  # a call prepared on the first pass, as a serving loop keeps it
    return state


# ---------------------------------------------------------------------------- the library's calls
def _handle(s, make):
    if not s["handle"]:
        s["handle"].append(make())
    return s["handle"][0]


def _own_rope(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]

    def make():
        args = (s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"], s["kv"][:, 0], s["kv"][:, 1])
        kw = dict(axis_of_pair=s["axis"], interleaved=c["interleaved"])
        if c["int8"]:
            return pkv.prepare_rope_reshape_and_cache_int8(*args, s["k_scale"], s["v_scale"], s["q_out"], **kw)
        return pkv.prepare_rope_reshape_and_cache(*args, s["q_out"], **kw)

    q = _handle(s, make)()
    return dict(q=q, kv=_dequantised(s) if c["int8"] else s["kv"])


def _own_decode(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]
    call = _handle(s, lambda: pkv.prepare_paged_attention_decode_scored(
        s["q"], s["kv"][:, 0], s["kv"][:, 1], s["tables"], s["lens"], s["scale"], s["out"], softcap=c["cap"],
        slopes=s["slopes"], window=c["window"], starts=s["starts"], weights=s["weights"],
        weights_out=s["weights_out"], max_context_len=s["max_len"]))
    out = call()
    return dict(out=out, weights=s["weights_out"]) if c["weights"] else dict(out=out)


def _own_prefill(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]
    call = _handle(s, lambda: pkv.prepare_paged_attention_prefill_scored(
        s["q"], s["kv"][:, 0], s["kv"][:, 1], s["tables"], s["query_start"], s["lens"], s["scale"], s["out"],
        max_query_len=s["max_chunk"], max_context_len=s["max_len"], softcap=c["cap"], slopes=s["slopes"],
        window=c["window"], starts=s["starts"], prefix_lens=s["prefix"]))
    return dict(out=call())


def _own_evict(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]

    def make():
        select = pkv.prepare_evict_select(s["weights"], s["lens"], c["budget"], sinks=c["sinks"], recent=c["recent"],
                                          max_context_len=s["max_len"], weights_out=s["weights_out"])
        kept, kept_lens = select.result
        return select, pkv.prepare_evict_compact(s["kv"][:, 0], s["kv"][:, 1], s["tables"], s["lens"], kept, kept_lens,
                                                 dst_block_tables=s["dst"])

    select, compact = _handle(s, make)
    kept, kept_lens = select()
    compact()
    return dict(kept=kept, lens=kept_lens, weights=s["weights_out"], kv=s["kv"])


# ---------------------------------------------------------------------------- the plain forms
def _rotate(x, cos, sin, interleaved):
    """The first 2 * pairs channels of x [T, H, d] (fp32) turned by the pairs' angles."""
    rot = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _dequantised(s):
    """The values that the cache's codes stand for, in the model's type."""
    return torch.mul(s["kv"], s["scales"], out=s["values"])


def _plain_rope(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    angle = s["positions"][s["axis"].long()].T.double() * s["inv_freq"]  # [T, pairs], 64 bits: far positions
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(dtype)
    k, v = _rotate(s["k"].float(), cos, sin, c["interleaved"]), s["v"].float()
    blk, off = s["slots"] // c["bs"], s["slots"] % c["bs"]
    if c["int8"]:
        k, v = (torch.round((x / sc).clamp(-127, 127)) for x, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
    s["kv"][blk, 0, :, off] = k.to(s["kv"].dtype)
    s["kv"][blk, 1, :, off] = v.to(s["kv"].dtype)
    return dict(q=q, kv=_dequantised(s) if c["int8"] else s["kv"])


def _gather(s):
    """K and V of every sequence as [B, Hkv, tokens, d] in fp32."""
    kv = s["kv"][s["tables"].long()]  # [B, blocks, 2, Hkv, bs, d]
    b, mb, _, hkv, bs, d = kv.shape
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hkv, mb * bs, d).float()
    return kv[0], kv[1]


def _scored(s, q, k, v, pos, lo, hi):
    """q [B, R, Hq, d] at positions pos [B, R], row r sees tokens lo <= t < hi ([B, R]):
    the output and the softmax weights [B, Hkv, G, R, tokens]."""
    c = s["case"]
    b, r, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    q = q.float().view(b, r, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * r, d)
    x = (torch.matmul(q, k.transpose(2, 3)) * s["scale"]).view(b, hkv, g, r, -1)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    t = torch.arange(k.shape[2], device="cuda")
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, hkv, g, 1, 1) * (t - pos[:, None, None, :, None])
    seen = (t >= lo[..., None]) & (t < hi[..., None])
    x = x.masked_fill(~seen[:, None, None], -torch.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -torch.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    p = p / l.masked_fill(l == 0, 1.0)
    out = torch.matmul(p.view(b, hkv, g * r, -1), v).view(b, hkv, g, r, d)
    return out.permute(0, 3, 1, 2, 4).reshape(b, r, hq, d), p


def _plain_decode(s):
    c = s["case"]
    k, v = _gather(s)
    hi = s["lens"].long()[:, None]
    lo = torch.zeros_like(hi) if not c["window"] else (hi - c["window"]).clamp(min=0)
    if s["starts"] is not None:
        lo = torch.maximum(lo, s["starts"].long()[:, None])
    out, p = _scored(s, s["q"][:, None], k, v, hi - 1, lo, hi)
    out = out[:, 0].to(s["q"].dtype)
    if not c["weights"]:
        return dict(out=out)
    inside = torch.arange(k.shape[2], device="cuda") < hi
    return dict(out=out, weights=torch.where(inside[:, None], s["weights"] + p.sum((2, 3)), s["weights_out"]))


def _row_bounds(s):
    """Per padded chunk row [B, max chunk]: its row of q, whether there is one, its position and what it sees."""
    c, qs, lens = s["case"], s["query_start"].long(), s["lens"].long()
    j = torch.arange(s["max_chunk"], device="cuda")[None]
    chunk = (qs[1:] - qs[:-1])[:, None]
    there = j < chunk
    row = torch.where(there, qs[:-1, None] + j, 0)
    pos = lens[:, None] - chunk + j
    hi = pos + 1
    if s["prefix"] is not None:
        hi = torch.minimum(torch.maximum(hi, s["prefix"].long()[:, None]), lens[:, None])
    lo = torch.zeros_like(pos) if not c["window"] else (pos + 1 - c["window"]).clamp(min=0)
    if s["starts"] is not None:
        lo = torch.maximum(lo, s["starts"].long()[row])
    return row, there, pos, lo, hi


def _plain_prefill(s):
    k, v = _gather(s)
    row, there, pos, lo, hi = _row_bounds(s)
    out, _ = _scored(s, s["q"][row], k, v, pos, lo, torch.where(there, hi, 0))
    return dict(out=out[there].to(s["q"].dtype))  # the chunks back to back


def _plain_evict(s):
    c = s["case"]
    lens = s["lens"].long()[:, None, None]
    w = s["weights"]
    t = torch.arange(w.shape[2], device="cuda")
    first, last = t < c["sinks"], t >= lens - c["recent"]
    key = torch.where(first | last, torch.inf, w).masked_fill(t >= lens, -torch.inf)
    order = torch.sort(key, dim=2, descending=True, stable=True).indices[..., :c["budget"]]
    n = lens.clamp(max=c["budget"])
    i = torch.arange(order.shape[2], device="cuda")
    kept = torch.where(i < n, order, w.shape[2]).sort(2).values
    there = kept < w.shape[2]
    src = kept.clamp(max=w.shape[2] - 1)
    weights = s["weights_out"].clone()
    weights[..., :i.numel()] = torch.where(there, w.gather(2, src), weights[..., :i.numel()])
    weights.masked_fill_((t >= n) & (t < lens), 0.0)
    seq = torch.arange(w.shape[0], device="cuda")[:, None, None].expand_as(src)[there]
    head = torch.arange(w.shape[1], device="cuda")[None, :, None].expand_as(src)[there]
    to, at = i.expand_as(src)[there], src[there]
    bs = c["bs"]
    s["kv"][s["dst"].long()[seq, to // bs], :, head, to % bs] = \
        s["kv"][s["tables"].long()[seq, at // bs], :, head, at % bs]
    pad = torch.full((w.shape[0], w.shape[1], c["budget"]), -1, dtype=torch.int32, device="cuda")
    pad[..., :i.numel()] = torch.where(there, kept, -1).to(torch.int32)
    return dict(kept=pad, lens=n.view(-1).to(torch.int32), weights=weights, kv=s["kv"])


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(rope=_own_rope, decode=_own_decode, prefill=_own_prefill, evict=_own_evict)[op](state)
    return dict(rope=_plain_rope, decode=_plain_decode, prefill=_plain_prefill, evict=_plain_evict)[op](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        t, d = c["tokens"], c["d"]
        each = t * d * (2 * c["hq"] * 2 + 2 * c["hkv"] * (2 + (1 if c["int8"] else 2)))
        return dict(bytes=each + t * 8 * (c["axes"] + 1) + c["rot"] // 2 * 12 + (c["int8"] and 2 * c["hkv"] * d * 4),
                    flops=t * (c["hq"] + c["hkv"]) * c["rot"] * 3)
    if c["op"] == "decode":
        mean = (max(1, c["lo"]) + c["hi"]) / 2
        total = mean * (c["seqs"] - 1) + c["hi"]
        seen = total
        if c["window"] and c["hi"] > 0:
            seen = min(total, c["seqs"] * c["window"])
        if c["starts"]:
            seen = seen / 2
        moved = seen * 2 * c["hkv"] * c["d"] * 2 + 2 * c["seqs"] * c["hq"] * c["d"] * 2 + total / c["bs"] * 4
        if c["weights"]:
            moved += 2 * total * c["hkv"] * 4
        return dict(bytes=int(moved), flops=int(4 * seen * c["hq"] * c["d"]))
    if c["op"] == "prefill":
        b = c["seqs"]
        chunks = [-(-c["chunk"] * (i * 5 % b + 1 if c["ragged"] else b) // b) for i in range(b)]
        pairs = tokens = 0.0
        for n in chunks:
            full = n * (c["cached"] / 2 + n / 2)
            if c["window"]:
                full = min(full, n * c["window"])
            pairs += full / (c["docs"] + 1) * 2 if c["docs"] else full
            tokens += n + min(c["cached"] / 2, c["window"] or c["cached"])
        rows = sum(chunks)
        return dict(bytes=int(tokens * 2 * c["hkv"] * 128 * 2 + rows * c["hq"] * 128 * 4),
                    flops=int(4 * min(pairs, rows * (c["cached"] + c["chunk"])) * c["hq"] * 128))
    mean = (c["lo"] + c["hi"]) / 2
    total = mean * (c["seqs"] - 1) + c["hi"]
    kept = min(c["budget"], mean) * c["seqs"]
    return dict(bytes=int(total * c["hkv"] * 8 + kept * c["hkv"] * (4 + 4 * 2 * c["d"])), flops=int(total * c["hkv"]))


# ---------------------------------------------------------------------------- the definitions in 64 bits
def _exact_rope(c, s):
    f = s["inv_freq"].cpu().tolist()
    axis = s["axis"].cpu().tolist()
    pos = s["positions"].cpu()
    tau = 2 * math.pi
    phase = torch.stack([(pos[a].double() * w).remainder(tau) for a, w in zip(axis, f)], 1)
    turn = torch.polar(torch.ones_like(phase), phase).cuda()  # e^(i angle), [T, pairs]
    n = len(f)

    def rotate(x):
        y = x.double().clone()
        re, im = (y[..., 0:2 * n:2], y[..., 1:2 * n:2]) if c["interleaved"] else (y[..., :n], y[..., n:2 * n])
        z = torch.complex(re, im) * turn[:, None]
        re.copy_(z.real)
        im.copy_(z.imag)
        return y

    kv = s["kv"].double()
    k, v = rotate(s["k"]), s["v"].double()
    if c["int8"]:
        scales = torch.stack([s["k_scale"], s["v_scale"]]).double()
        kv = kv * scales[:, :, None, :]
        k, v = (torch.round((x / sc).clamp(-127, 127)) * sc for x, sc in ((k, scales[0]), (v, scales[1])))
    flat = kv.permute(0, 3, 1, 2, 4).reshape(-1, 2, c["hkv"], c["d"])
    flat[s["slots"]] = torch.stack([k, v], 1)
    return dict(q=rotate(s["q"]), kv=flat.view(-1, c["bs"], 2, c["hkv"], c["d"]).permute(0, 2, 3, 1, 4).contiguous())


def _exact_rows(c, s, seq, n, q, pos, lo, hi):
    """One sequence's rows q [R, Hq, d] over its n tokens, in 64 bits: (out, weights [Hq, R, n])."""
    bs, d = c["bs"], s["kv"].shape[-1]
    blocks = s["tables"][seq, :(n + bs - 1) // bs].long()
    kv = s["kv"].index_select(0, blocks).double().transpose(2, 3).reshape(len(blocks), 2, bs, c["hkv"], d)
    k, v = (kv[:, i].reshape(-1, c["hkv"], d)[:n].permute(1, 0, 2) for i in (0, 1))
    t = torch.arange(n, device="cuda")
    hidden = (t[None] < lo[:, None]) | (t[None] >= hi[:, None])
    outs, weights = [], []
    g = c["hq"] // c["hkv"]
    for h in range(c["hq"]):
        x = q[:, h].double() @ k[h // g].T / math.sqrt(d)
        if c["cap"]:
            x = torch.tanh(x / c["cap"]) * c["cap"]
        if c["slopes"]:
            x = x - float(s["slopes"][h]) * (pos[:, None] - t[None]).double()
        x[hidden] = -math.inf
        w = torch.softmax(x, 1).nan_to_num(nan=0.0)
        outs.append(w @ v[h // g])
        weights.append(w)
    return torch.stack(outs, 1), weights


def _exact_decode(c, s):
    outs, acc = [], s["weights_out"].double() if c["weights"] else None
    for i, n in enumerate(s["lens"].tolist()):
        lo = max(0, n - c["window"]) if c["window"] else 0
        if c["starts"]:
            lo = max(lo, int(s["starts"][i]))
        at = lambda x: torch.tensor([x], device="cuda")  # noqa: E731
        out, w = _exact_rows(c, s, i, n, s["q"][i:i + 1], at(n - 1), at(lo), at(n))
        outs.append(out[0])
        if c["weights"]:
            acc[i, :, :n] = s["weights"][i, :, :n].double() + torch.cat(w).view(c["hkv"], -1, n).sum(1)
    return dict(out=torch.stack(outs), weights=acc) if c["weights"] else dict(out=torch.stack(outs))


def _exact_prefill(c, s):
    outs, qs = [], s["query_start"].tolist()
    for i, n in enumerate(s["lens"].tolist()):
        a, b = qs[i], qs[i + 1]
        pos = torch.arange(n - (b - a), n, device="cuda")
        lo, hi = torch.zeros_like(pos), pos + 1
        if c["window"]:
            lo = (hi - c["window"]).clamp(min=0)
        if c["docs"]:
            lo = torch.maximum(lo, s["starts"][a:b].long())
        if c["prefix"]:
            hi = hi.clamp(min=min(n, int(s["prefix"][i])))
        outs.append(_exact_rows(c, s, i, n, s["q"][a:b], pos, lo, hi)[0])
    return dict(out=torch.cat(outs))


def _exact_evict(c, s):
    # nothing is rounded: the kept positions and the rows by index, one head at a time
    kv, weights = s["kv"].clone(), s["weights_out"].clone()
    kept = torch.full((c["seqs"], c["hkv"], c["budget"]), -1, dtype=torch.int32)
    lens = s["lens"].tolist()
    for i, n in enumerate(lens):
        m = min(n, c["budget"])
        fixed = set(range(min(c["sinks"], n))) | set(range(max(0, n - c["recent"]), n))
        for h in range(c["hkv"]):
            w = s["weights"][i, h, :n]
            if m < n:
                vals = w.tolist()
                rest = sorted((t for t in range(n) if t not in fixed), key=lambda t: (-vals[t], t))
                at = torch.tensor(sorted(fixed | set(rest[:m - len(fixed)])))
            else:
                at = torch.arange(n)
            kept[i, h, :m] = at.to(torch.int32)
            at, to = at.cuda(), torch.arange(m, device="cuda")
            weights[i, h, :n] = 0
            weights[i, h, :m] = w[at]
            kv[s["dst"][i, to // c["bs"]].long(), :, h, to % c["bs"]] = \
                s["kv"][s["tables"][i, at // c["bs"]].long(), :, h, at % c["bs"]]
    lens = torch.tensor([min(n, c["budget"]) for n in lens], dtype=torch.int32)
    return dict(kept=kept, lens=lens, weights=weights.double(), kv=kv.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, s)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    return (_exact_decode if case["op"] == "decode" else _exact_prefill)(case, s)
