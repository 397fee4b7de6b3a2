"""Timed cases of three further operators around the paged KV cache:

  int4    a cache of 4-bit codes with a scale and a zero per 32 channels of each row: new rows
          quantised as they are written, and blocks read back into a 16-bit cache
  decode4 one query token per sequence over its context in such a cache
  tree    the verification of a tree of drafted tokens: their rows written behind the context,
          their attention (each sees the context and its own ancestors), and the accepted
          path's rows moved together
  sinks   one query token per sequence over the last tokens of its context and a few first
          ones, in a 16-bit or an INT8 cache
  sinks_prefill   a chunk of new tokens per sequence with the same mask

``own`` selects the library's calls; otherwise every operator runs in its plain form.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # the new token of 64 sequences, each in a block of its own
        dict(name="int4_step", op="int4", tokens=64, hkv=8, d=128, bs=16, dtype="f16"),
        # a long prompt's chunk, its blocks read back for a prefill over 16-bit rows
        dict(name="int4_chunk", op="int4", tokens=8192, hkv=8, d=128, bs=16, dtype="bf16"),
        # an odd chunk of a model with a KV head per query head
        dict(name="int4_odd", op="int4", tokens=1777, hkv=32, d=64, bs=32, dtype="f16"),
        # a full batch of grouped heads
        dict(name="decode4_batch", op="decode4", seqs=64, lo=4096, hi=4096, hq=32, hkv=8, d=128, bs=16, dtype="f16"),
        # a few long contexts
        dict(name="decode4_long", op="decode4", seqs=4, lo=30001, hi=32768, hq=64, hkv=8, d=128, bs=32, dtype="bf16"),
        # ragged contexts, a KV head per query head, small blocks
        dict(name="decode4_mha", op="decode4", seqs=24, lo=100, hi=2048, hq=32, hkv=32, d=64, bs=8, dtype="bf16"),
        # a small tree per sequence: a verification step where latency counts
        dict(name="tree_step", op="tree", seqs=8, lo=1024, hi=4096, nodes=16, ragged=False, hq=32, hkv=8, bs=16, dtype="bf16"),
        # wide trees of several sizes behind long contexts
        dict(name="tree_wide", op="tree", seqs=16, lo=4096, hi=8192, nodes=63, ragged=True, hq=64, hkv=8, bs=32, dtype="f16"),
        # an endless stream's step: the last 1024 tokens and the first 4
        dict(name="sinks_step", op="sinks", seqs=64, lo=128, hi=8192, hq=32, hkv=8, d=128, bs=16, dtype="bf16", int8=False,
             window=1024, sinks=4),
        # a longer window over a quantised cache, a KV head per query head
        dict(name="sinks_int8", op="sinks", seqs=16, lo=8000, hi=16384, hq=32, hkv=32, d=64, bs=16, dtype="f16", int8=True,
             window=4096, sinks=16),
        # chunks behind cached tokens
        dict(name="sinks_chunk", op="sinks_prefill", seqs=8, chunk=512, ragged=False, cached=7680, hq=64, hkv=8, bs=16,
             dtype="bf16", window=2048, sinks=4),
        # ragged whole prompts, a short window, and first tokens that fill blocks of their own
        dict(name="sinks_prompts", op="sinks_prefill", seqs=5, chunk=1999, ragged=True, cached=0, hq=32, hkv=32, bs=32,
             dtype="f16", window=333, sinks=70),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int4", "decode4", "tree", "sinks", "sinks_prefill"])
    bs = rng.choice([8, 16, 32])
    dtype = rng.choice(["f16", "bf16"])
    hq, hkv = rng.choice([(32, 32), (32, 8), (64, 8), (128, 8), (32, 16), (20, 4), (12, 12)])
    d = rng.choice([64, 128, 128])
    if op == "int4":
        return dict(op=op, tokens=min(_log(rng, 1, 8192), 8192 * 8 * 128 // (hkv * d)), hkv=hkv, d=d, bs=bs, dtype=dtype)
    if op == "decode4":
        hi = _log(rng, 16, 32768)
        seqs = max(1, min(_log(rng, 1, 64), 64 * 4096 * 8 * 128 // (hi * hkv * d)))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype)
    if op == "tree":
        hi, nodes = _log(rng, 16, 16384), _log(rng, 1, 100)
        seqs = max(1, min(_log(rng, 1, 64), 16 * 8192 * 64 * 40 // (hi * hq * nodes), 16 * 8192 * 8 // (hi * hkv)))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, nodes=nodes, ragged=rng.random() < 0.5,
                    hq=hq, hkv=hkv, bs=bs, dtype=dtype)
    window, sinks = _log(rng, 1, 4096), rng.choice([1, 4, 4, 16, _log(rng, 1, 200)])
    if op == "sinks":
        hi = _log(rng, 16, 16384)
        seqs = max(1, min(_log(rng, 1, 64), 16 * 16384 * 32 * 64 // (hi * hkv * d)))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, hi // 2 + 1, hi]), hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype,
                    int8=rng.random() < 0.4, window=window, sinks=sinks)
    chunk, cached = _log(rng, 2, 2048), rng.choice([0, _log(rng, 1, 7680)])
    most = 8 * 512 * 64 * 2048
    seqs = max(1, min(rng.randint(1, 9), most // (chunk * hq * min(window, chunk // 2 + cached + 1))))
    return dict(op=op, seqs=seqs, chunk=chunk, ragged=rng.random() < 0.5, cached=cached, hq=hq, hkv=hkv, bs=bs, dtype=dtype,
                window=window, sinks=sinks)


# ---------------------------------------------------------------------------- 4-bit rows
# A block's rows of one KV head, as bytes: the codes of its tokens, d / 2 bytes each, then a
# (scale, zero) pair in the rows' type per token and group of 32 channels.  Channel 32 j + 4 u + e
# of a token is nibble e of the token's 16-bit word u * (d / 32) + j.
def _up(x, dtype):
    """x >= 0 (64 bits) rounded up to dtype."""
    r = x.float().to(dtype)
    return (r.view(torch.int16) + (r.double() < x).to(torch.int16)).view(dtype)


def _quantise(x):
    """Rows [..., d] -> (codes [..., d / 32, 32], scale, zero [..., d / 32] of the rows' type); in 64 bits, as
    16-bit values often lie halfway between two codes."""
    g = x.double().unflatten(-1, (-1, 32))
    zero = g.amin(-1)
    scale = _up((g.amax(-1) - zero) / 15, x.dtype)
    codes = torch.round((g - zero[..., None]) / scale.double()[..., None]).nan_to_num(nan=0.0).clamp(0, 15)
    return codes, scale, zero.to(x.dtype)


def _pack(codes, scale, zero):
    """-> (code bytes [..., d / 2], parameter bytes [..., d / 8])."""
    c = codes.to(torch.uint8).unflatten(-1, (8, 2, 2)).transpose(-4, -3)  # [..., u, j, byte, nibble]
    params = torch.stack([scale, zero], -1).flatten(-2).view(torch.uint8)
    return (c[..., 0] | (c[..., 1] << 4)).flatten(-3), params


def _parts(pool, d):
    """Views of a pool [..., bs, 5 d / 8]: code bytes [..., bs, d / 2] and parameter bytes [..., bs, d / 8]."""
    bs = pool.shape[-2]
    flat = pool.flatten(-2)
    return flat[..., :bs * d // 2].unflatten(-1, (bs, d // 2)), flat[..., bs * d // 2:].unflatten(-1, (bs, d // 8))


def _unpack(pool, d, dtype):
    """The codes [..., bs, d / 32, 32] and (scale, zero) [..., bs, d / 32, 2] of a pool [..., bs, 5 d / 8], fp32."""
    b, params = _parts(pool, d)
    c = torch.stack([b & 15, b >> 4], -1).flatten(-2).unflatten(-1, (8, d // 32, 4)).transpose(-3, -2).flatten(-2)
    return c.float(), params.contiguous().view(dtype).float().unflatten(-1, (-1, 2))


def _values(pool, d, dtype):
    c, p = _unpack(pool, d, dtype)
    return (c * p[..., 0:1] + p[..., 1:2]).flatten(-2)


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
    return tables, total + spare


def _pool(c, blocks, gen):
    return torch.randn((blocks, 2, c["hkv"], c["bs"], c["d"]), generator=gen, device="cuda", dtype=DTYPES[c["dtype"]])


def _pool4(c, blocks, gen):
    """A pool of quantised normal rows whose channels have several means and widths."""
    d, dtype = c["d"], DTYPES[c["dtype"]]
    pool = torch.empty((blocks, 2, c["hkv"], c["bs"], d * 5 // 8), dtype=torch.uint8, device="cuda")
    width = torch.rand((2, c["hkv"], 1, d), generator=gen, device="cuda") + 0.5
    mean = torch.randn((2, c["hkv"], 1, d), generator=gen, device="cuda") * 0.5
    step = max(1, 2 ** 26 // (2 * c["hkv"] * c["bs"] * d))
    for at in range(0, blocks, step):
        part = pool[at:at + step]
        x = torch.randn((len(part), 2, c["hkv"], c["bs"], d), generator=gen, device="cuda")
        codes, params = _parts(part, d)
        codes[:], params[:] = _pack(*_quantise((x * width + mean).to(dtype)))
    return pool


def _prepare_int4(c, seed):
    gen, _ = _gens(seed)
    dtype, t, hkv, d, bs = DTYPES[c["dtype"]], c["tokens"], c["hkv"], c["d"], c["bs"]
    i = torch.arange(t, device="cuda")
    if t <= 256:  # decode steps: each token in a block of its own sequence
        blocks = t + 3
        table = torch.randperm(blocks, generator=gen, device="cuda")[:t]
        slots = table * bs + torch.randint(0, bs, (t,), generator=gen, device="cuda")
    else:  # a chunk fills the blocks of its table
        blocks = (t + bs - 1) // bs + 3
        table = torch.randperm(blocks, generator=gen, device="cuda")[:blocks - 3]
        slots = table[i // bs] * bs + i % bs
    to = torch.randperm(len(table), generator=gen, device="cuda")
    return dict(case=c, k=_randn((t, hkv, d), dtype, gen), v=_randn((t, hkv, d), dtype, gen, 0.5), slots=slots,
                pool=_pool4(c, blocks, gen), pairs=torch.stack([table, to], 1).contiguous(),
                kv=torch.zeros((len(table), 2, hkv, bs, d), dtype=dtype, device="cuda"))


def _prepare_decode4(c, seed):
    gen, host = _gens(seed)
    lens = _lens(c["seqs"], c["lo"], c["hi"], host)
    tables, blocks = _tables(lens, c["bs"], gen, spare=2)
    q = _randn((c["seqs"], c["hq"], c["d"]), DTYPES[c["dtype"]], gen, 2.0)
    return dict(case=c, q=q, pool=_pool4(c, blocks, gen), tables=tables, lens=lens.to(torch.int32).cuda(),
                max_len=int(lens.max()), scale=1 / math.sqrt(c["d"]), out=torch.zeros_like(q))


def _prepare_tree(c, seed):
    gen, host = _gens(seed)
    b, c = c["seqs"], dict(c, d=128)
    share = torch.arange(b) * 5 % b + 1 if c["ragged"] else torch.full((b,), b)
    chunk = (c["nodes"] * share + b - 1) // b
    lens = _lens(b, c["lo"], c["hi"], host) + chunk
    most = b * -(-(c["hi"] + int(chunk.max())) // c["bs"])  # the pool's size, whatever the lengths
    tables, blocks = _tables(lens, c["bs"], gen, spare=most - int(((lens + c["bs"] - 1) // c["bs"]).sum()))
    start = torch.cat([torch.zeros(1, dtype=torch.int64), chunk.cumsum(0)])
    rows, words, most = int(start[-1]), (int(chunk.max()) + 63) // 64, int(chunk.max())
    pick = torch.rand((rows,), generator=host).tolist()
    seen, path, path_lens = [], torch.full((b, most), -1, dtype=torch.int32), []
    for i in range(b):
        ancestors = []  # bit sets: a node's parent is one of the nodes before it, the last ones more often
        for n in range(int(chunk[i])):
            parent = int(n * pick[int(start[i]) + n] ** 0.5)
            ancestors.append((ancestors[parent] if n else 0) | 1 << n)
        seen += ancestors
        kept = ancestors[int(len(ancestors) * pick[int(start[i])])] if i % 7 != 6 else 0  # the accepted path; some accept nothing
        nodes = [n for n in range(len(ancestors)) if kept >> n & 1]
        path[i, :len(nodes)] = torch.tensor(nodes, dtype=torch.int32)
        path_lens.append(len(nodes))
    low = (1 << 64) - 1
    signed = [[(m >> 64 * w & low) - ((m >> 64 * w & low) >> 63 << 64) for w in range(words)] for m in seen]
    dtype = DTYPES[c["dtype"]]
    q = _randn((rows, c["hq"], 128), dtype, gen, 2.0)
    seq = torch.repeat_interleave(torch.arange(b), chunk)
    pos = (torch.arange(rows) - start[seq] + (lens - chunk)[seq]).cuda()
    slots = tables[seq.cuda(), pos // c["bs"]].long() * c["bs"] + pos % c["bs"]
    return dict(case=c, q=q, k=_randn((rows, c["hkv"], 128), dtype, gen), v=_randn((rows, c["hkv"], 128), dtype, gen),
                slots=slots, kv=_pool(c, blocks, gen), tables=tables, lens=lens.to(torch.int32).cuda(),
                query_start=start.to(torch.int32).cuda(), max_chunk=most, max_len=int(lens.max()), scale=1 / math.sqrt(128),
                mask=torch.tensor(signed, dtype=torch.int64).cuda(), path=path.cuda(),
                path_lens=torch.tensor(path_lens, dtype=torch.int32).cuda(), out=torch.zeros_like(q),
                new_lens=torch.zeros(b, dtype=torch.int32, device="cuda"))


def _prepare_sinks(c, seed):
    gen, host = _gens(seed)
    lens = _lens(c["seqs"], c["lo"], c["hi"], host)
    tables, blocks = _tables(lens, c["bs"], gen, spare=2)
    q = _randn((c["seqs"], c["hq"], c["d"]), DTYPES[c["dtype"]], gen, 2.0)
    s = dict(case=c, q=q, tables=tables, lens=lens.to(torch.int32).cuda(), max_len=int(lens.max()),
             scale=1 / math.sqrt(c["d"]), out=torch.zeros_like(q))
    if c["int8"]:
        shape = (blocks, 2, c["hkv"], c["bs"], c["d"])
        s["kv"] = torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)
        s["scales"] = [(torch.rand((c["hkv"], c["d"]), generator=gen, device="cuda") + 0.5) / 64 for _ in range(2)]
    else:
        s["kv"] = _pool(c, blocks, gen)
    return s


def _prepare_sinks_prefill(c, seed):
    gen, host = _gens(seed)
    b, c = c["seqs"], dict(c, d=128)
    share = torch.arange(b) * 5 % b + 1 if c["ragged"] else torch.full((b,), b)
    chunk = (c["chunk"] * share + b - 1) // b
    lens = chunk + torch.randint(0, c["cached"] + 1, (b,), generator=host)
    tables, blocks = _tables(lens, c["bs"], gen, spare=2)
    start = torch.cat([torch.zeros(1, dtype=torch.int64), chunk.cumsum(0)])
    q = _randn((int(start[-1]), c["hq"], 128), DTYPES[c["dtype"]], gen, 2.0)
    return dict(case=c, q=q, kv=_pool(c, blocks, gen), tables=tables, lens=lens.to(torch.int32).cuda(),
                query_start=start.to(torch.int32).cuda(), max_chunk=int(chunk.max()), max_len=int(lens.max()),
                scale=1 / math.sqrt(128), out=torch.zeros_like(q))


def prepare(case, seed):
    made = dict(int4=_prepare_int4, decode4=_prepare_decode4, tree=_prepare_tree, sinks=_prepare_sinks,
                sinks_prefill=_prepare_sinks_prefill)
    state = made[case["op"]](case, seed)
    state["handle"] = []  # calls prepared on the first pass, as a serving loop keeps them
    return state


# ---------------------------------------------------------------------------- the library's calls
def _handle(s, make):
    if not s["handle"]:
        s["handle"].extend(make())
    return s["handle"]


def _own_int4(s):
    import paged_kv_cache_155_gb300 as pkv

    def make():  # the halves are cut once, when the calls are prepared
        k4, v4 = s["pool"][:, 0], s["pool"][:, 1]
        return (pkv.prepare_reshape_and_cache_int4(s["k"], s["v"], s["slots"], k4, v4),
                pkv.prepare_dequantise_blocks_int4(k4, v4, s["pairs"], s["kv"][:, 0], s["kv"][:, 1]))

    write, read = _handle(s, make)
    write()
    read()
    return dict(kv=s["kv"])


def _own_decode4(s):
    import paged_kv_cache_155_gb300 as pkv
    call, = _handle(s, lambda: (pkv.prepare_paged_attention_decode_int4(
        s["q"], s["pool"][:, 0], s["pool"][:, 1], s["tables"], s["lens"], s["scale"], s["out"],
        max_context_len=s["max_len"]),))
    return dict(out=call())


def _own_tree(s):
    import paged_kv_cache_155_gb300 as pkv

    def make():
        k, v = s["kv"][:, 0], s["kv"][:, 1]
        rest = (s["tables"], s["query_start"], s["lens"])
        bound = dict(max_query_len=s["max_chunk"], max_context_len=s["max_len"])
        return (pkv.prepare_reshape_and_cache(s["k"], s["v"], s["slots"], k, v),
                pkv.prepare_paged_attention_tree(s["q"], k, v, *rest, s["mask"], s["scale"], s["out"], **bound),
                pkv.prepare_tree_commit(k, v, *rest, s["path"], s["path_lens"], s["new_lens"], **bound))

    write, attend, commit = _handle(s, make)
    write()
    out = attend()
    commit()
    return dict(out=out, kv=s["kv"], lens=s["new_lens"])


def _own_sinks(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]

    def make():
        cache = (s["kv"][:, 0], s["kv"][:, 1])
        rest = (s["tables"], s["lens"], s["scale"], s["out"])
        kw = dict(window=c["window"], sinks=c["sinks"], max_context_len=s["max_len"])
        if c["int8"]:
            return pkv.prepare_paged_attention_decode_sinks_int8(s["q"], *cache, *s["scales"], *rest, **kw),
        return pkv.prepare_paged_attention_decode_sinks(s["q"], *cache, *rest, **kw),

    call, = _handle(s, make)
    return dict(out=call())


def _own_sinks_prefill(s):
    import paged_kv_cache_155_gb300 as pkv
    c = s["case"]
    call, = _handle(s, lambda: (pkv.prepare_paged_attention_prefill_sinks(
        s["q"], s["kv"][:, 0], s["kv"][:, 1], s["tables"], s["query_start"], s["lens"], s["scale"], s["out"],
        max_query_len=s["max_chunk"], max_context_len=s["max_len"], window=c["window"], sinks=c["sinks"]),))
    return dict(out=call())


# ---------------------------------------------------------------------------- the plain forms
def _plain_int4(s):
    c = s["case"]
    codes, params = _parts(s["pool"], c["d"])
    blk, off = s["slots"] // c["bs"], s["slots"] % c["bs"]
    codes[blk, :, :, off], params[blk, :, :, off] = _pack(*_quantise(torch.stack([s["k"], s["v"]], 1)))
    s["kv"][s["pairs"][:, 1]] = _values(s["pool"][s["pairs"][:, 0]], c["d"], s["kv"].dtype).to(s["kv"].dtype)
    return dict(kv=s["kv"])


def _contexts(kv):
    """Gathered blocks [B, blocks, 2, Hkv, bs, d] -> K and V as [B, Hkv, tokens, d]."""
    b, mb, _, hkv, bs, d = kv.shape
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, b, hkv, mb * bs, d)
    return kv[0], kv[1]


def _attend(q, k, v, scale, seen):
    """q [B, R, Hq, d] over k, v [B, Hkv, tokens, d] where seen [B, R, tokens], fp32: [B, R, Hq, d]."""
    b, r, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    q = q.float().view(b, r, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * r, d)
    x = (torch.matmul(q, k.transpose(2, 3)) * scale).view(b, hkv, g, r, -1)
    x = x.masked_fill(~seen[:, None, None], -torch.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.masked_fill(m == -torch.inf, 0.0))
    l = p.sum(-1, keepdim=True)
    p = p / l.masked_fill(l == 0, 1.0)
    out = torch.matmul(p.view(b, hkv, g * r, -1), v).view(b, hkv, g, r, d)
    return out.permute(0, 3, 1, 2, 4).reshape(b, r, hq, d)


def _plain_decode4(s):
    k, v = _contexts(_values(s["pool"][s["tables"].long()], s["case"]["d"], s["q"].dtype))
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"].long()[:, None, None]
    return dict(out=_attend(s["q"][:, None], k, v, s["scale"], seen)[:, 0].to(s["q"].dtype))


def _rows(s):
    """Per padded chunk row [B, max chunk]: its row of q, whether there is one, its position; the chunks' first positions."""
    qs, lens = s["query_start"].long(), s["lens"].long()
    j = torch.arange(s["max_chunk"], device="cuda")[None]
    chunk = (qs[1:] - qs[:-1])[:, None]
    there = j < chunk
    base = lens[:, None] - chunk
    return torch.where(there, qs[:-1, None] + j, 0), there, base + j, base


def _plain_tree(s):
    c, kv, bs = s["case"], s["kv"], s["case"]["bs"]
    kv[s["slots"] // bs, :, :, s["slots"] % bs] = torch.stack([s["k"], s["v"]], 1)
    k, v = _contexts(kv[s["tables"].long()].float())
    row, there, _, base = _rows(s)
    node = torch.arange(k.shape[2], device="cuda") - base  # [B, tokens]: the chunk token, negative in the context
    inside = (node >= 0) & (node < there.sum(1, keepdim=True))
    at = node.clamp(0, s["mask"].shape[1] * 64 - 1)
    word = s["mask"][row].gather(2, (at // 64)[:, None].expand(-1, row.shape[1], -1))
    bit = (word >> (at % 64)[:, None] & 1).bool()
    seen = (node < 0)[:, None] | (inside[:, None] & bit)
    out = _attend(s["q"][row], k, v, s["scale"], seen)[there].to(s["q"].dtype)
    # the accepted path's rows move together
    j = torch.arange(s["path"].shape[1], device="cuda")
    move = j < s["path_lens"][:, None]
    seq, to = move.nonzero(as_tuple=True)
    src = (base[seq, 0] + s["path"][seq, to].long())
    dst = (base[seq, 0] + to)
    t = s["tables"].long()
    kv[t[seq, dst // bs], :, :, dst % bs] = kv[t[seq, src // bs], :, :, src % bs]
    return dict(out=out, kv=kv, lens=(base[:, 0] + s["path_lens"]).to(torch.int32))


def _plain_sinks(s):
    c = s["case"]
    kv = s["kv"][s["tables"].long()].float()
    if c["int8"]:
        kv = kv * torch.stack(s["scales"])[:, :, None]
    k, v = _contexts(kv)
    t, n = torch.arange(k.shape[2], device="cuda"), s["lens"].long()[:, None, None]
    seen = (t < n) & ((t < c["sinks"]) | (t >= n - c["window"]))
    return dict(out=_attend(s["q"][:, None], k, v, s["scale"], seen)[:, 0].to(s["q"].dtype))


def _plain_sinks_prefill(s):
    c = s["case"]
    k, v = _contexts(s["kv"][s["tables"].long()].float())
    row, there, pos, _ = _rows(s)
    t, pos = torch.arange(k.shape[2], device="cuda"), pos[..., None]
    seen = (t <= pos) & ((t < c["sinks"]) | (t > pos - c["window"]))
    return dict(out=_attend(s["q"][row], k, v, s["scale"], seen)[there].to(s["q"].dtype))  # the chunks back to back


def run(state):
    op = state["case"]["op"]
    if own:
        return dict(int4=_own_int4, decode4=_own_decode4, tree=_own_tree, sinks=_own_sinks,
                    sinks_prefill=_own_sinks_prefill)[op](state)
    return dict(int4=_plain_int4, decode4=_plain_decode4, tree=_plain_tree, sinks=_plain_sinks,
                sinks_prefill=_plain_sinks_prefill)[op](state)


# ---------------------------------------------------------------------------- what a pass cannot do without
def _chunks(c, longest):
    b = c["seqs"]
    return [-(-longest * (i * 5 % b + 1 if c["ragged"] else b) // b) for i in range(b)]


def work(case):
    c = case
    if c["op"] == "int4":
        t, row = c["tokens"], c["hkv"] * c["d"]
        read = t * c["bs"] if t <= 256 else t  # rows of the blocks read back
        return dict(bytes=int(2 * t * row * (2 + 0.625) + 2 * read * row * (2 + 0.625) + t * 8), flops=2 * (t * 4 + read * 2) * row)
    if c["op"] == "decode4":
        total = (max(1, c["lo"]) + c["hi"]) / 2 * (c["seqs"] - 1) + c["hi"]
        return dict(bytes=int(total * 2 * c["hkv"] * c["d"] * 0.625 + 2 * c["seqs"] * c["hq"] * c["d"] * 2 + total / c["bs"] * 4),
                    flops=int(4 * total * c["hq"] * c["d"]))
    if c["op"] == "tree":
        mean, nodes = (max(1, c["lo"]) + c["hi"]) / 2, _chunks(c, c["nodes"])
        rows = sum(nodes)
        total = mean * (c["seqs"] - 1) + c["hi"] + rows
        each = 2 * c["hkv"] * 128 * 2  # a token's K and V
        pairs = sum(n * (mean + n / 4) for n in nodes)
        return dict(bytes=int(total * each + rows * (c["hq"] * 128 * 2 * 2 + 2 * each) + rows * 8), flops=int(4 * pairs * c["hq"] * 128))
    if c["op"] == "sinks":
        total = (max(1, c["lo"]) + c["hi"]) / 2 * (c["seqs"] - 1) + c["hi"]
        seen = min(total, c["seqs"] * (c["window"] + c["sinks"]))
        return dict(bytes=int(seen * 2 * c["hkv"] * c["d"] * (1 if c["int8"] else 2) + 2 * c["seqs"] * c["hq"] * c["d"] * 2 + seen / c["bs"] * 4),
                    flops=int(4 * seen * c["hq"] * c["d"]))
    chunks, reach = _chunks(c, c["chunk"]), c["window"] + c["sinks"]
    pairs = sum(min(n * (c["cached"] / 2 + n / 2), n * reach) for n in chunks)
    tokens = sum(n + min(c["cached"] / 2, reach) for n in chunks)
    rows = sum(chunks)
    return dict(bytes=int(tokens * 2 * c["hkv"] * 128 * 2 + rows * c["hq"] * 128 * 4), flops=int(4 * pairs * c["hq"] * 128))


# ---------------------------------------------------------------------------- the definitions in 64 bits
def _exact_int4(c, s):
    """Row groups one after the other: smallest and largest value, the rounded-up step, the nearest multiple."""
    d, bs = c["d"], c["bs"]
    x = torch.stack([s["k"], s["v"]], 1).double().reshape(-1, 32)
    low, high = x.min(1).values, x.max(1).values
    want = (high - low) / 15
    half = want.to(s["k"].dtype)
    bits = half.view(torch.int16).clone()
    bits[half.double() < want] += 1
    step = bits.view(s["k"].dtype).double()
    n = torch.where(step[:, None] > 0, (x - low[:, None]) / step[:, None], 0.0).round().clamp(0, 15)
    rows = (low[:, None] + n * step[:, None]).view(c["tokens"], 2, c["hkv"], d)
    # what the blocks held before: byte by byte
    old = s["pool"][s["pairs"][:, 0]]
    held = torch.empty((len(old), 2, c["hkv"], bs, d), dtype=torch.float64, device="cuda")
    flat = old.reshape(len(old), 2, c["hkv"], -1)
    for ch in range(d):
        j, u, e = ch // 32, ch % 32 // 4, ch % 4
        at = torch.arange(bs, device="cuda") * (d // 2) + 2 * (u * (d // 32) + j) + e // 2
        code = (flat[..., at] >> (4 * (e % 2))) & 15
        p = bs * d // 2 + torch.arange(bs, device="cuda") * (d // 8) + 4 * j
        pair = torch.stack([flat[..., p + i] for i in range(4)], -1).contiguous().view(s["k"].dtype).double()
        held[..., ch] = code.double() * pair[..., 0] + pair[..., 1]
    place = torch.full((len(s["pool"]),), -1, dtype=torch.int64, device="cuda")
    place[s["pairs"][:, 0]] = torch.arange(len(old), device="cuda")
    held[place[s["slots"] // bs], :, :, s["slots"] % bs] = rows
    kv = torch.zeros(s["kv"].shape, dtype=torch.float64, device="cuda")
    kv[s["pairs"][:, 1]] = held
    return dict(kv=kv)


def _exact_rows(q, k, v, seen):
    """One sequence's rows q [R, Hq, d] over its tokens k, v [n, Hkv, d] where seen [R, n], in 64 bits."""
    g = q.shape[1] // k.shape[1]
    outs = []
    for h in range(q.shape[1]):
        x = q[:, h].double() @ k[:, h // g].T / math.sqrt(q.shape[2])
        x[~seen] = -math.inf
        outs.append(torch.softmax(x, 1).nan_to_num(nan=0.0) @ v[:, h // g])
    return torch.stack(outs, 1)


def _exact_context(c, s, seq, n):
    """K and V of one sequence's first n tokens, [n, Hkv, d] in 64 bits."""
    bs = c["bs"]
    blocks = s["tables"][seq, :(n + bs - 1) // bs].long()
    if c["op"] == "decode4":
        codes, params = _unpack(s["pool"][blocks], c["d"], s["q"].dtype)
        kv = (codes.double() * params[..., 0:1].double() + params[..., 1:2].double()).flatten(-2)
    else:
        kv = s["kv"][blocks].double()
        if c.get("int8"):
            kv = kv * torch.stack(s["scales"]).double()[:, :, None]
    kv = kv.transpose(2, 3).reshape(len(blocks), 2, bs, c["hkv"], -1)
    return [kv[:, i].reshape(-1, c["hkv"], kv.shape[-1])[:n] for i in (0, 1)]


def _exact_attention(c, s):
    outs = []
    rows = s["query_start"].tolist() if "query_start" in s else list(range(c["seqs"] + 1))
    for i, n in enumerate(s["lens"].tolist()):
        q = s["q"][rows[i]:rows[i + 1]]
        pos = torch.arange(n - len(q), n, device="cuda")[:, None]
        t = torch.arange(n, device="cuda")[None]
        if c["op"] == "decode4":
            seen = t <= pos
        elif c["op"] == "tree":
            base = n - len(q)
            seen = (t < base).expand(len(q), n).clone()
            for m in range(len(q)):
                seen[:, base + m] = (s["mask"][rows[i]:rows[i + 1], m // 64] >> (m % 64) & 1).bool()
        else:
            seen = (t <= pos) & ((t < c["sinks"]) | (pos - t < c["window"]))
        outs.append(_exact_rows(q, *_exact_context(c, s, i, n), seen))
    return torch.cat(outs)


def _exact_tree(c, s):
    bs, rows = c["bs"], s["query_start"].tolist()
    lens, table = s["lens"].tolist(), s["tables"].tolist()
    slots = s["slots"].tolist()
    for r, slot in enumerate(slots):
        s["kv"][slot // bs, 0, :, slot % bs] = s["k"][r]
        s["kv"][slot // bs, 1, :, slot % bs] = s["v"][r]
    out = _exact_attention(c, s)
    after = []
    for i, n in enumerate(lens):
        base, kept = n - (rows[i + 1] - rows[i]), int(s["path_lens"][i])
        for j, m in enumerate(s["path"][i, :kept].tolist()):
            slot, r = (base + j), rows[i] + m
            s["kv"][table[i][slot // bs], 0, :, slot % bs] = s["k"][r]
            s["kv"][table[i][slot // bs], 1, :, slot % bs] = s["v"][r]
        after.append(base + kept)
    return dict(out=out, kv=s["kv"].double(), lens=torch.tensor(after, dtype=torch.int32))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "int4":
        return _exact_int4(c, s)
    return _exact_tree(c, s) if c["op"] == "tree" else dict(out=_exact_attention(c, s))
