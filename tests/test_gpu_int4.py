"""4-bit cache: the quantising write, the read-back and the decode against 64-bit references."""
import math

import pytest
import torch

import paged_kv_cache_155_gb300 as pkv
from tests import _cache_refs as refs
from tests._gpu_helpers import check_no_device_flags, device
from tests._operator_refs import rounded_close

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16]


def _rows(t, hkv, d, dtype, g):
    """Normal rows, and in turn constant, tiny, wide and small-integer ones (whose values often lie between two codes)."""
    x = torch.randn((t, hkv, d), generator=g)
    kind = torch.arange(t) % 7
    x[kind == 1] = 0.375
    x[kind == 2] *= 2.0 ** -22
    x[kind == 3] *= 2000.0
    x[kind == 4] = torch.randint(-15, 16, (int((kind == 4).sum()), hkv, d), generator=g).float()
    x[kind == 5] = x[kind == 5].abs() + 100.0
    return x.to(dtype)


def _shuffled_pool(blocks, hkv, bs, d, g):
    return torch.randint(0, 256, (blocks, 2, hkv, bs, d * 5 // 8), generator=g, dtype=torch.uint8)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,hkv,d,bs", [(1, 1, 64, 8), (5, 3, 64, 32), (64, 8, 128, 16), (33, 12, 128, 8), (70, 2, 128, 32),
                                        (9, 33, 64, 16)])
def test_write_is_the_reference_bit_for_bit(t, hkv, d, bs, dtype):
    dev, g = device(), torch.Generator().manual_seed(t + hkv)
    blocks = -(-t // bs) + 2
    pool = _shuffled_pool(blocks, hkv, bs, d, g)
    k, v = _rows(t, hkv, d, dtype, g), _rows(t, hkv, d, dtype, g).flip(0).contiguous()
    slots = torch.randperm(blocks * bs, generator=g)[:t]
    slots[t // 2] = -1 if t > 1 else slots[0]
    dp = pool.to(dev)
    pkv.reshape_and_cache_int4(k.to(dev), v.to(dev), slots.to(dev), *pkv.split_pool(dp))
    check_no_device_flags(dev)
    codes, scale, zero = refs.unpack(pool, dtype)
    for n, s in enumerate(slots.tolist()):
        if s >= 0:
            for half, x in enumerate((k, v)):
                c, sc, z = refs.quantise(x[n])
                codes[s // bs, half, :, s % bs], scale[s // bs, half, :, s % bs], zero[s // bs, half, :, s % bs] = c, sc, z
    assert torch.equal(dp.cpu(), refs.pack(codes, scale, zero))


@pytest.mark.parametrize("dtype", DTYPES)
def test_values_are_half_a_step_off_at_most(dtype):
    dev, g = device(), torch.Generator().manual_seed(3)
    x = _rows(256, 2, 128, dtype, g)
    pool = pkv.int4_pool(16, 2, 16, 128, dev)
    pkv.reshape_and_cache_int4(x.to(dev), x.to(dev), torch.arange(256).to(dev), *pkv.split_pool(pool))
    got = refs.values(pool.cpu(), dtype)[:, 0].transpose(1, 2).reshape(256, 2, 128)
    grp = x.double().unflatten(-1, (4, 32))
    step = refs.round_up((grp.amax(-1) - grp.amin(-1)) / 15, dtype).double().repeat_interleave(32, -1)
    assert (got - x.double()).abs().le(step / 2).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_write_of_values_halfway_between_codes(dtype):
    """Groups of z + m s / 2, m in 0 .. 30 with both ends: every odd m is a tie, which goes to the even code."""
    dev, g = device(), torch.Generator().manual_seed(4)
    t, hkv, d = 200, 2, 64
    m = torch.randint(0, 31, (t, 2 * hkv, 2, 32), generator=g)
    m[..., 3], m[..., 17] = 0, 30
    unit = 2.0 ** torch.randint(-12, 4, (t, 2 * hkv, 2, 1), generator=g)
    s = torch.randint(1, 5, (t, 2 * hkv, 2, 1), generator=g)  # 30 s + 60 <= 256: exact in eight bits
    z = torch.randint(-60, 61, (t, 2 * hkv, 2, 1), generator=g)
    x = ((z + m * s) * unit).flatten(2).to(dtype)
    assert (x.double().unflatten(-1, (2, 32)) == (z + m * s) * unit.double()).all()
    slots = torch.arange(t)
    dp = pkv.int4_pool(13, hkv, 16, d, dev)
    pkv.reshape_and_cache_int4(x[:, :hkv].contiguous().to(dev), x[:, hkv:].contiguous().to(dev), slots.to(dev), *pkv.split_pool(dp))
    codes, scale, zero = refs.unpack(dp.cpu(), dtype)
    want = torch.where(m % 4 == 1, m // 2, (m + 1) // 2)  # m / 2, ties to even
    for half in range(2):
        got = codes[:, half].transpose(1, 2).reshape(208, hkv, 2, 32)[:t]
        assert torch.equal(got, want[:, half * hkv:(half + 1) * hkv])


def test_write_of_nan_and_of_the_smallest_values():
    dev = device()
    for dtype in DTYPES:
        x = torch.randn((4, 1, 64), generator=torch.Generator().manual_seed(1)).to(dtype)
        x[0, 0, 5] = math.nan
        x[1] = 0.0
        x[1, 0, 7] = torch.finfo(dtype).smallest_normal if dtype is torch.bfloat16 else 2.0 ** -24
        x[2, 0, :32] = torch.finfo(dtype).max
        x[2, 0, 3] = -torch.finfo(dtype).max if dtype is torch.float16 else 0.0
        pool = torch.zeros((1, 2, 1, 8, 40), dtype=torch.uint8, device=dev)
        pkv.reshape_and_cache_int4(x.to(dev), x.to(dev), torch.arange(4).to(dev), *pkv.split_pool(pool))
        codes, scale, zero = refs.unpack(pool.cpu(), dtype)
        assert codes[0, 0, 0, 0, 0, 5] == 0 and torch.isfinite(scale).all() and torch.isfinite(zero).all()
        for n in (1, 2, 3):
            c, s, z = refs.quantise(x[n])
            assert torch.equal(codes[0, 0, :, n], c) and torch.equal(scale[0, 0, :, n], s) and torch.equal(zero[0, 0, :, n], z)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hkv,d,bs", [(1, 64, 8), (3, 128, 8), (8, 128, 16), (5, 64, 32), (32, 128, 32)])
def test_read_back(hkv, d, bs, dtype):
    dev, g = device(), torch.Generator().manual_seed(hkv)
    x = _rows(9 * bs, 2 * hkv, d, dtype, g)
    pool = pkv.int4_pool(9, hkv, bs, d, dev)
    slots = torch.arange(9 * bs).to(dev)
    pkv.reshape_and_cache_int4(x[:, :hkv].contiguous().to(dev), x[:, hkv:].contiguous().to(dev), slots, *pkv.split_pool(pool))
    kv = torch.full((7, 2, hkv, bs, d), 3.0, dtype=dtype, device=dev)
    pairs = torch.tensor([[8, 0], [2, 5], [0, 6]])
    pkv.dequantise_blocks_int4(*pkv.split_pool(pool), pairs.to(dev), *pkv.split_pool(kv))
    check_no_device_flags(dev)
    codes, scale, zero = refs.unpack(pool.cpu(), dtype)
    # the products and sums in fp32, rounded once more: c s is exact there
    want32 = (codes.float() * scale.float()[..., None] + zero.float()[..., None]).flatten(-2).to(dtype)
    want = torch.full((7, 2, hkv, bs, d), 3.0, dtype=dtype)
    for a, b in pairs.tolist():
        want[b] = want32[a]
    assert torch.equal(kv.cpu().view(torch.int16), want.view(torch.int16))


def test_bad_slots_and_pairs_are_skipped_and_flagged():
    dev = device()
    x = torch.ones((3, 2, 64), dtype=torch.float16, device=dev)
    pool = torch.zeros((2, 2, 2, 8, 40), dtype=torch.uint8, device=dev)
    k4, v4 = pkv.split_pool(pool)
    pkv.reshape_and_cache_int4(x, x, torch.tensor([16, 2 ** 40, -3], device=dev), k4, v4)
    assert pkv.get_device_error(dev)[1] == ["slot"] and not pool.any()
    kv = torch.zeros((2, 2, 2, 8, 64), dtype=torch.float16, device=dev)
    pkv.dequantise_blocks_int4(k4, v4, torch.tensor([[2, 0], [0, -1], [-5, 0], [0, 2]], device=dev), *pkv.split_pool(kv))
    assert pkv.get_device_error(dev)[1] == ["copy_pair"] and not kv.any()


def _pool_of(lens, hkv, bs, d, dtype, g, spread=1.0):
    """(pool, tables): a quantised pool whose contexts are placed at random; bytes that no context covers are 0xff (NaN scales)."""
    need = [-(-n // bs) for n in lens]
    blocks = sum(need) + 2
    perm, at = torch.randperm(blocks, generator=g).to(torch.int32), 0
    tables = torch.full((len(lens), max(need + [1]) + 1), -7, dtype=torch.int32)  # entries past a context are never read
    x = (torch.randn((blocks, 2, hkv, bs, d), generator=g) * spread + torch.randn((1, 2, hkv, 1, d), generator=g)).to(dtype)
    codes, scale, zero = refs.quantise(x)
    covered = torch.zeros((blocks, bs), dtype=torch.bool)
    for i, n in enumerate(lens):
        tables[i, :need[i]] = perm[at:at + need[i]]
        at += need[i]
        for t in range(n):
            covered[tables[i, t // bs], t % bs] = True
    hide = ~covered[:, None, None, :].expand(blocks, 2, hkv, bs)
    codes[hide] = 15
    bad = torch.full((1,), -1, dtype=torch.int16).view(dtype)[0]
    scale[hide], zero[hide] = bad, bad
    return refs.pack(codes, scale, zero), tables


def _check_decode(got, q, pool, tables, lens, dtype, scale, what):
    vals, d = refs.values(pool, dtype), q.shape[2]
    for i, n in enumerate(lens):
        k, v = refs.context(vals, tables[i], n)
        seen = torch.ones((1, n), dtype=torch.bool)
        out, mag, most = refs.attend(q[i:i + 1], k, v, scale, seen)
        # a score: 34 roundings of 2^-23 of a group's largest partial sum, |q'| (1024 + 64 c) <= 496 |q| after the factor
        # 1/4, times the group's scale; and the query's 2^-24 of its largest channel
        if n:
            _, s, _ = refs.unpack(pool, dtype)
            big = s[tables[i, :-(-n // pool.shape[3])].long()].double().nan_to_num(nan=0.0).max().item()
            sum_q = q[i].double().abs().sum(-1, keepdim=True)[None]
            slack = 34 * 496 * 2.0 ** -23 * big * sum_q * abs(scale) + most * (2.0 ** -20 + d * 2.0 ** -24)
        else:
            slack = torch.zeros((1, q.shape[1], 1), dtype=torch.float64)
        # an output: the weights' score error on both sides of the quotient, their fp16 rounding (2^-11), and the offset's
        # share of the sums (1024 per largest value 4 * 15 + ..: 17 times, 2^-23 a step, one per 16 tokens and merge)
        wide = s_max(pool, tables[i], n, dtype) * 16
        steps = n / 64 + 40
        rounded_close(got[i], out[0], (mag * (2 * slack + 2.0 ** -11 + 2.0 ** -18) + wide * (2.0 ** -11 + 17 * steps * 2.0 ** -23))[0], f"{what}, sequence {i}")


def s_max(pool, table, n, dtype):
    if n == 0:
        return 0.0
    _, s, _ = refs.unpack(pool[table[:-(-n // pool.shape[3])].long()][:, 1], dtype)
    return s.double().nan_to_num(nan=0.0).max().item()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("hq,hkv,d,bs", [(1, 1, 64, 8), (4, 4, 128, 16), (8, 1, 128, 8), (32, 4, 128, 32), (12, 4, 64, 16),
                                         (16, 1, 128, 16), (40, 2, 64, 32), (36, 1, 128, 8), (13, 1, 64, 8), (128, 8, 128, 16),
                                         (32, 8, 128, 16), (6, 3, 128, 8), (3, 1, 128, 32)])
@pytest.mark.parametrize("more", [0, 1500])
def test_decode(hq, hkv, d, bs, dtype, more):
    dev, g = device(), torch.Generator().manual_seed(hq * 7 + d + bs)
    lens = [0, 1, 31, 32, 33, 65, 200, 311] + [more] * (more > 0)  # a long context's units are cut by several workers
    pool, tables = _pool_of(lens, hkv, bs, d, dtype, g)
    q = (torch.randn((len(lens), hq, d), generator=g) * 2).to(dtype)
    out = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool.to(dev)), tables.to(dev),
                                          torch.tensor(lens, dtype=torch.int32, device=dev), max_context_len=max(lens))
    check_no_device_flags(dev)
    _check_decode(out.cpu(), q, pool, tables, lens, dtype, 1 / math.sqrt(d), f"more {more}")


def test_decode_of_many_and_of_few_tokens():
    """More sequences than a warp reads at once, and batches whose workers outnumber their chunks."""
    dev = device()
    for hq, hkv, lens in ((4, 2, [i * 53 % 300 for i in range(100)]), (8, 8, [3]), (16, 1, [0, 0]), (1, 1, [4000, 0, 1])):
        g = torch.Generator().manual_seed(len(lens))
        pool, tables = _pool_of(lens, hkv, 16, 64, torch.float16, g)
        q = (torch.randn((len(lens), hq, 64), generator=g) * 2).to(torch.float16)
        out = torch.full_like(q, 7.0).to(dev)
        pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool.to(dev)), tables.to(dev),
                                        torch.tensor(lens, dtype=torch.int32, device=dev), out=out, max_context_len=max(lens))
        check_no_device_flags(dev)
        _check_decode(out.cpu(), q, pool, tables, lens, torch.float16, 0.125, f"{len(lens)} sequences")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [2.0 ** -12, 2.0 ** 8])
def test_decode_of_small_and_large_values(dtype, spread):
    """Scales far from 1 on either side, and a query of one sharp row."""
    dev, g = device(), torch.Generator().manual_seed(5)
    lens = [40, 513]
    pool, tables = _pool_of(lens, 2, 16, 128, dtype, g, spread)
    q = (torch.randn((2, 8, 128), generator=g) * 0.5 / max(1.0, spread)).to(dtype)
    out = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool.to(dev)), tables.to(dev),
                                          torch.tensor(lens, dtype=torch.int32, device=dev), 0.3, max_context_len=540)
    check_no_device_flags(dev)
    _check_decode(out.cpu(), q, pool, tables, lens, dtype, 0.3, f"spread {spread}")


def test_decode_flags_bad_entries_and_lengths():
    dev, g = device(), torch.Generator().manual_seed(6)
    lens = [70, 20]
    pool, tables = _pool_of(lens, 1, 16, 64, torch.float16, g)
    q = torch.randn((2, 4, 64), generator=g).to(torch.float16)
    bad = tables.clone()
    bad[0, 1] = 10 ** 6
    out = pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool.to(dev)), bad.to(dev),
                                          torch.tensor(lens, dtype=torch.int32, device=dev), max_context_len=70)
    assert pkv.get_device_error(dev)[1] == ["block_table"]
    vals = refs.values(pool, torch.float16)
    k, v = refs.context(vals, tables[0], 70)
    seen = torch.ones((1, 70), dtype=torch.bool)
    seen[:, 16:32] = False  # the flagged block's tokens do not count
    want = refs.attend(q[:1], k, v, 0.125, seen)[0][0]
    assert (out[0].cpu().double() - want).abs().max() < 2e-2
    pkv.paged_attention_decode_int4(q.to(dev), *pkv.split_pool(pool.to(dev)), tables.clamp(min=0).to(dev),
                                    torch.tensor([71, -2], dtype=torch.int32, device=dev), max_context_len=70)
    assert pkv.get_device_error(dev)[1] == ["context_len"]


def test_prepared_calls_on_another_stream_and_in_a_graph():
    dev, g = device(), torch.Generator().manual_seed(8)
    lens = [5, 900, 64]
    pool, tables = _pool_of(lens, 2, 16, 128, torch.bfloat16, g)
    q = torch.randn((3, 8, 128), generator=g).to(torch.bfloat16).to(dev)
    dl, dt, dp = torch.tensor(lens, dtype=torch.int32, device=dev), tables.to(dev), pool.to(dev)
    calls = [pkv.prepare_paged_attention_decode_int4(q, *pkv.split_pool(dp), dt, dl, max_context_len=910)
             for _ in range(2)]  # two workspaces: their graphs may run together
    want = calls[0]().clone()
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for c in calls:
        c.result.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(calls[0].result, want) and torch.equal(calls[1].result, want)


def test_placement_does_not_change_a_bit():
    dev, g = device(), torch.Generator().manual_seed(9)
    pool, tables = _pool_of([333], 2, 8, 64, torch.float16, g)
    q = torch.randn((1, 6, 64), generator=g).to(torch.float16).to(dev)
    n = torch.tensor([333], dtype=torch.int32, device=dev)
    perm = torch.randperm(pool.shape[0], generator=g)
    moved = torch.empty_like(pool)
    moved[perm] = pool
    there = torch.where(tables >= 0, perm[tables.clamp(min=0).long()].to(torch.int32), tables)
    a = pkv.paged_attention_decode_int4(q, *pkv.split_pool(pool.to(dev)), tables.to(dev), n, max_context_len=333)
    b = pkv.paged_attention_decode_int4(q, *pkv.split_pool(moved.to(dev)), there.to(dev), n, max_context_len=333)
    assert torch.equal(a, b)


def test_copy_of_shared_blocks():
    dev, g = device(), torch.Generator().manual_seed(10)
    for d in (64, 128):
        pool = _shuffled_pool(6, 3, 16, d, g)
        dp = pool.to(dev)
        pkv.copy_blocks(*pkv.split_pool(dp), torch.tensor([[4, 0], [1, 5]], device=dev))
        pool[0], pool[5] = pool[4], pool[1]
        assert torch.equal(dp.cpu(), pool)


@pytest.mark.parametrize("dtype", DTYPES)
def test_prompt_then_steps_over_a_quantised_cache(dtype):
    """A prompt quantised as it is written, its next chunk prefilled over the read-back blocks, then decode steps over the
    codes: each step equals the 16-bit decode over the read-back blocks but for the roundings."""
    dev, g = device(), torch.Generator().manual_seed(11)
    hq, hkv, d, bs, n, chunk = 8, 2, 128, 16, 75, 9
    table = torch.randperm(12, generator=g).to(torch.int32)[None].to(dev)
    pool, kv = torch.zeros((12, 2, hkv, bs, d * 5 // 8), dtype=torch.uint8, device=dev), torch.zeros((12, 2, hkv, bs, d), dtype=dtype, device=dev)
    rows = lambda t, h: torch.randn((t, h, d), generator=g).to(dtype).to(dev)  # noqa: E731
    pairs = torch.arange(12, device=dev)[:, None].expand(12, 2).contiguous()
    halves4, halves = pkv.split_pool(pool), pkv.split_pool(kv)
    slots = pkv.slot_mapping(table, torch.arange(n, device=dev), bs, token_rows=torch.zeros(n, dtype=torch.int64, device=dev), num_blocks=12)
    pkv.reshape_and_cache_int4(rows(n, hkv), rows(n, hkv), slots, *halves4)
    pkv.dequantise_blocks_int4(*halves4, pairs, *halves)
    lens = torch.tensor([n], dtype=torch.int32, device=dev)
    q = rows(chunk, hq)
    pre = pkv.paged_attention_prefill(q, *halves, table, torch.tensor([0, chunk], dtype=torch.int32, device=dev), lens,
                                      max_query_len=chunk, max_context_len=n)
    last = pkv.paged_attention_decode_int4(q[-1:], *halves4, table, lens, max_context_len=n)
    tol = 3 * (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -11) * 8  # outputs below 8; roundings of V, P and the result
    assert (pre[-1:].float() - last.float()).abs().max() < tol
    for step in range(3):
        lens += 1
        k, v, q = rows(1, hkv), rows(1, hkv), rows(1, hq)
        slot = pkv.slot_mapping(table, lens.long() - 1, bs, num_blocks=12)
        pkv.reshape_and_cache_int4(k, v, slot, *halves4)
        pkv.dequantise_blocks_int4(*halves4, pairs, *halves)
        a = pkv.paged_attention_decode_int4(q, *halves4, table, lens, max_context_len=n + 3)
        b = pkv.paged_attention_decode(q, *halves, table, lens, max_context_len=n + 3)
        assert (a.float() - b.float()).abs().max() < tol
    check_no_device_flags(dev)
