// decode_int4_kernel.cuh -- paged decode attention over the 4-bit cache (format: int4.cuh).
//
// What it computes: the decode's softmax attention (decode_kernel.cuh) with the values that the
// codes stand for, K_t = sK c + zK and V_t = sV c + zV per group j of 32 channels:
//     s_t = scale * sum_j ( sK[t,j] (q_j . c[t,j]) + zK[t,j] sum(q_j) ),
//     o   = sum_t p_t ( sV[t,j] c[t,j] + zV[t,j] ),       p_t = exp(s_t - ref).
// The codes meet the query and the weights as exact small integers, and a token's scales
// enter once per group: q_j . c is one group's MMA accumulator, the V scale multiplies the
// weight (p_t sV[t,j], rounded once to fp16); the zeros are one more MMA for K (against sum(q_j),
// split in two or three 16-bit numbers) and plain fp32 sums for V.
//
// What bounds it: 5/8 byte a value, a quarter of what a 16-bit cache reads, against the same
// number of codes to widen; so per code the kernel spends 0.75 integer operations and half an
// MMA slot, and little else.
//  * Both products run as warp-level MMAs (m16n8k16, fp16 operands, fp32 accumulators) with the
//    tokens (S^T = K Q^T) or the channels (O^T = V^T P^T) as the 16 rows and eight query heads as the
//    columns, for any group of heads: unused columns are zero.  Groups of more than eight heads take
//    two column tiles on the same K and V fragments, so their codes are widened once.
//  * Up to four heads take their columns twice (NT = 0, "paired"): a code word's two halves are groups
//    2 i and 2 i + 1 of one unit, and as a fragment's pair of k indices they meet four columns that are zero in
//    the odd k (group 2 i) and four that are zero in the even k (group 2 i + 1).  So words enter the MMAs
//    as they lie, without the byte permutes that sort them by group, and a lane scales two groups instead of four:
//    half the scales, weights and accumulators.  (64 x 4096 tokens of 32 / 8 heads 69 us, sorted words 78; 64 x 100 to
//    2048 tokens of 32 heads of 64 61 and 65; both without a test of V's scales.)
//  * Widening costs a mask: a nibble at bits 0 .. 3 or 4 .. 7 of a 16-bit word is a subnormal fp16
//    number, exactly c 2^-24 or c 2^-20, and MMAs take those as they are (codes_f16).  K's factor 16
//    between the two is in the query, V's is applied to the output channel, whose accumulator holds
//    one nibble position only.  (With the exponent of 1024.0 set above the nibbles, as an offset to be
//    taken away again, and 16 tokens a step, 64 x 4096 tokens of 32 / 8 heads took 106 us; so 83.)
//  * The weights' reference is the running maximum of s_t + log2(max_j sV[t,j]), not of s_t, so that
//    p_t sV[t,j], what fp16 has to hold, is at most 2^12 and 2^6 or more where it counts, whatever V's scale is:
//    as long as a token's groups have scales within 2^8 of its largest one.  From the first chunk on that holds another
//    token (or scales or zeros near the ends of bf16's range), a worker weighs the rest of its share with exponents per
//    chunk, head and group (int4_work_own), so that a small group next to a large one is as exact as alone.  Measured, all
//    rows alike / a zero group in every row: 64 x 4096 tokens, 32 / 8 heads 70 / 86 us, 128 / 8 heads 120 / 180; without
//    the test and the other form 68.7 and 120.
//  * Every warp is a worker of its own: the 32-token chunks of all (sequence, KV head) units stand in one
//    row and are cut into equal shares, so that any mix of lengths keeps all warps busy to the end and
//    none waits for another (CTAs as workers, whose warps join their sums, measured the same on long contexts
//    and 1.5 us slower on a few).  A worker holds at most two pieces of cut units (its first and last);
//    their partials are merged by paged_decode_int4_merge_kernel, whole units are written at once.
//  * A worker streams its share through its own ring of stages by bulk copies (a block's record of one head
//    is contiguous: codes and scales arrive together), one copy per lane, the table entries read a chunk
//    ahead; the ring runs on from one unit to the next.  A stage is one softmax step.
//  * The token of an MMA row is chosen so that V's four token rows of a load lie side by side
//    (token_of_row): two-way instead of four-way shared-memory conflicts.
// Measured: 64 x 4096 tokens of 32 / 8 heads of 128, fp16: 70 us (0.71 of measured HBM; 59 us, 0.84, per
// 64 x 4096 further tokens, so 11 fixed); with eight columns and sorted words, and without a test of V's
// scales, it was 55 us without the arithmetic and 68 without the copies.
#pragma once

#include "decode_kernel.cuh"
#include "int4.cuh"

namespace pkv {

template <int D, int BS, int NT>
struct DecodeInt4Geom {
    static constexpr int kWarps = 4;
    static constexpr int kGroups = D / 32;
    static constexpr int kStageTokens = 32;
    static constexpr int kBlocks = kStageTokens / BS;              // blocks per stage
    static constexpr int kRecord = int4_record_bytes(D, BS);       // a block's K (or V) rows of one head
    static constexpr int kHalfBytes = kBlocks * kRecord;           // 2560 at head_dim 128
    static constexpr int kStageBytes = 2 * kHalfBytes;
    static constexpr int kResident = NT <= 1 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);  // CTAs per SM, by registers
    // about 180 KB of stages per SM: several times the bytes that cover the memory latency
    static constexpr int kStages = 46080 / kResident / kStageBytes;
    static constexpr int kHeads = NT == 0 ? 4 : 8 * NT;
    static constexpr int kTiles = NT == 0 ? 1 : NT;               // column tiles
    static constexpr int kLaneGroups = NT == 0 ? kGroups / 2 : kGroups;  // groups whose sums a lane holds
    static constexpr int kSmemBytes = kWarps * kStages * (kStageBytes + 8 + 4);
};

// A cut unit.  The table of them is indexed by unit (seq * units + unit) when there are no more units
// than workers, else by the worker in whose share it begins (at most one goes on past a share).
struct Int4Split {
    int pieces;  // workers that hold pieces of it; 0: not cut, or none begins in this share
    int worker;  // the first of them, whose piece is in its slot `slot` (the others' in slot 0)
    int slot;
    int seq, unit;
};
struct Int4Params {
    const void *q;                // [num_seqs][num_q_heads][D]
    const void *k_cache, *v_cache;
    void *out;
    float *seg_o, *seg_m, *seg_l; // partials [2 worker + slot][heads of a block][D], [..][heads]
    Int4Split *splits;            // [min(workers, num_seqs * units)]
    int by_unit, seg_workers;     // its index; workers that the partials have room for
    const int32_t *block_tables, *context_lens;
    unsigned int *status;
    int64_t num_blocks, block_stride;  // bytes
    int max_blocks_per_seq, len_cap, num_seqs, num_q_heads, group;
    int blocks;                   // blocks of heads per KV head
    int units;                    // units of a sequence: num_kv_heads * blocks
    float scale_log2;
};
constexpr int kInt4MinShare = 2;  // chunks of a share, at least
// V's rows that a chunk weighs as they are: the largest scale in 2^kInt4Low .. 2^kInt4High, the others within kInt4Ratio
// of it (fp16 holds p sV in full down to 2^-14, and the reference's tokens have 2^kInt4Head or more), zeros up to
// 2^kInt4Zero.  Beyond, the reference is taken from the clamped scale, or from the zero / 2^kInt4ZeroLift, so that
// p <= 2^42, p sV <= 2^97 and p zV <= 2^102: their sums over any context stay in fp32's range.
constexpr float kInt4Ratio = 1.f / 256.f;  // 2^-8
constexpr int kInt4Low = -30, kInt4High = 40, kInt4Zero = 60, kInt4ZeroLift = 90;
constexpr float kInt4Head = 6.f;
// bf16 (scale, zero) words: 2^kInt4High, 2^kInt4Zero, and -2^kInt4Low kInt4Ratio, 2^kInt4Zero
constexpr uint32_t kInt4Most = ((kInt4High + 127) << 7) | ((kInt4Zero + 127) << 23);
constexpr uint32_t kInt4Least = 0x8000u | ((kInt4Low - 8 + 127) << 7) | ((kInt4Zero + 127) << 23);

// The token (0 .. 7) of MMA row r: rows 2 t, which one lane load of V takes for t = 0 .. 3, are
// tokens 0 .. 3, and rows 2 t + 1 tokens 5, 4, 7, 6.
__host__ __device__ constexpr int token_of_row(int r) { return r & 1 ? 4 + ((r >> 1) ^ 1) : r >> 1; }

// Four codes in each half of a word -> fp16 pairs: r[0], r[2] = c 2^-24, r[1], r[3] = c 2^-20.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&r)[4]) {
    const uint32_t y = x >> 8;
    r[0] = x & 0x000f000fu;
    r[1] = x & 0x00f000f0u;
    r[2] = y & 0x000f000fu;
    r[3] = y & 0x00f000f0u;
}

// ... for V, whose output channels have accumulators of their own: r[2] is the whole byte, c + 16 c' with the
// next code c', whose channel's accumulator takes its share away at the end (one operation less).
__device__ __forceinline__ void codes_f16_bytes(uint32_t x, uint32_t (&r)[4]) {
    r[0] = x & 0x000f000fu;
    r[1] = x & 0x00f000f0u;
    r[2] = __byte_perm(x, 0u, 0x4341);
    r[3] = r[2] & 0x00f000f0u;
}

// The words of two units (of one token, or of one unit in two tokens) -> per group j the four
// codes of the first in the low half and of the second in the high half.
template <int NG>
__device__ __forceinline__ uint32_t group_word(const uint32_t (&a)[NG / 2], const uint32_t (&b)[NG / 2], int j) {
    return __byte_perm(a[j / 2], b[j / 2], j & 1 ? 0x7632 : 0x5410);
}

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a * b + c of two halves of the type
template <typename T>
__device__ __forceinline__ uint32_t fma_halves(uint32_t a, float b, uint32_t c) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 d = __hfma2(*reinterpret_cast<const __half2 *>(&a), __float2half2_rn(b), *reinterpret_cast<const __half2 *>(&c));
        return *reinterpret_cast<const uint32_t *>(&d);
    } else {
        const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&a), __float2bfloat162_rn(b),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&c));
        return *reinterpret_cast<const uint32_t *>(&d);
    }
}

// The larger and the smaller halves of two (scale, zero) words: the scale's in the low half.
template <typename T>
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 m = __hmax2(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}
template <typename T>
__device__ __forceinline__ uint32_t min_halves(uint32_t a, uint32_t b) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 m = __hmin2(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// A sequence's length as the kernels take it, and its chunks (at least one, possibly empty: an
// empty context's zeros are written too).
__device__ __forceinline__ int int4_len(const Int4Params &p, int seq) {
    return min(max(p.context_lens[seq], 0), p.len_cap);
}
__device__ __forceinline__ int int4_chunks(int len) { return max(1, (len + 31) / 32); }

// The chunks of every worker's share, and of all units together (total); by one warp.
__device__ __forceinline__ int int4_share(const Int4Params &p, int workers, int &total) {
    const int lane = threadIdx.x & 31;
    total = 0;
#pragma unroll 8
    for (int seq = lane; seq < p.num_seqs; seq += 32) total += int4_chunks(int4_len(p, seq));
    total = __reduce_add_sync(0xffffffffu, total) * p.units;
    return max(kInt4MinShare, (total + workers - 1) / workers);
}

// Where a worker goes on: its piece and the piece's next chunk, the chunks that are left of its share from the piece's first
// on, its ring's next stage, and what it has summed.
template <int N, int GL>
struct Int4At {
    int seq, unit, chunk, c, left, s;
    uint32_t phase;
    bool first_piece;
    Int4Split split;
    float oacc[N][GL][2][4], zacc[N][GL][2], m[N][2], l[N][2];
};
template <int D, int BS, int NT>
using Int4AtOf = Int4At<DecodeInt4Geom<D, BS, NT>::kTiles, DecodeInt4Geom<D, BS, NT>::kLaneGroups>;

// A worker's pieces from `at` on.  Without kOwn it stops at the first chunk with a row that wants exponents of its own, with
// no copy in flight: false, and `at` is there.  With kOwn it goes on there, and takes all that is left.
template <typename T, int D, int BS, int NT, bool kOwn>
__device__ __forceinline__ bool int4_work(const Int4Params &p, const int worker, const int share, Int4AtOf<D, BS, NT> &at) {
    using G = DecodeInt4Geom<D, BS, NT>;
    constexpr int NW = G::kWarps, S = G::kStages, NG = G::kGroups, SB = G::kBlocks, HEADS = G::kHeads;
    constexpr int N = G::kTiles, GL = G::kLaneGroups;
    constexpr bool kPaired = NT == 0;
    constexpr int ROW = int4_row_bytes(D), PAR = int4_param_bytes(D);
    constexpr bool kBF16 = !std::is_same<T, __half>::value;

    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mg = lane >> 2, mt = lane & 3;
    const int par = mt >> 1;  // paired: a lane's groups are 2 i + par; else group i
    auto head_of = [&](int n, int e) { return kPaired ? 2 * (mt & 1) + e : 8 * n + 2 * mt + e; };  // of a lane's columns
    auto group_of = [&](int i) { return kPaired ? 2 * i + par : i; };
    unsigned char *my_stages = smem + warp * S * G::kStageBytes;
    uint64_t *my_bars = reinterpret_cast<uint64_t *>(smem + NW * S * G::kStageBytes) + warp * S;
    uint32_t *my_good = reinterpret_cast<uint32_t *>(smem + NW * S * (G::kStageBytes + 8)) + warp * S;  // blocks of a stage that were copied
    int seq = at.seq, unit = at.unit, chunk = at.chunk, left = at.left;

    // ---- the copies' walk, up to S chunks ahead: lanes 2 i and 2 i + 1 copy block i's K and V records of
    //      a chunk.  A lane's table entry of the next chunk is read while the one before it is copied.
    const uint64_t policy = l2_policy_evict_first();
    const char *const cache0 = static_cast<const char *>(lane & 1 ? p.v_cache : p.k_cache);
    const char *cache = cache0 + static_cast<int64_t>(unit / p.blocks) * G::kRecord;  // of the unit's KV head
    int i_seq = seq, i_unit = unit, i_chunk = at.c, i_left = left - (at.c - chunk), i_len = int4_len(p, seq), i_entry = -1;
    auto fetch = [&]() {
        i_entry = -1;
        const int at = i_chunk * SB + (lane >> 1);
        if (i_left > 0 && lane < 2 * SB && at * BS < i_len) {
            i_entry = p.block_tables[static_cast<int64_t>(i_seq) * p.max_blocks_per_seq + at];
            if (i_entry < 0 || i_entry >= p.num_blocks) {
                raise_flag(p.status, PKV_DEVERR_BLOCK_TABLE);
                i_entry = -1;
            }
        }
    };
    auto issue = [&](int s) {
        const uint32_t good = __ballot_sync(0xffffffffu, i_entry >= 0);
        if (lane == 0) {
            my_good[s] = good;
            if (good) mbar_arrive_expect_tx(&my_bars[s], __popc(good) * G::kRecord);
            else mbar_arrive(&my_bars[s]);
        }
        __syncwarp();
        if (i_entry >= 0)
            bulk_copy_g2s(my_stages + s * G::kStageBytes + (lane & 1) * G::kHalfBytes + (lane >> 1) * G::kRecord,
                          cache + i_entry * p.block_stride, G::kRecord, &my_bars[s], policy);
        --i_left;
        if (++i_chunk == int4_chunks(i_len)) {
            i_chunk = 0;
            if (++i_unit == p.units) {
                i_unit = 0;
                ++i_seq;
                if (i_left > 0) i_len = int4_len(p, i_seq);
            }
            cache = cache0 + static_cast<int64_t>(i_unit / p.blocks) * G::kRecord;
        }
        fetch();
    };
    fetch();
    int s = at.s;  // the next chunk's stage and its barrier's phase
    uint32_t phase = at.phase;
    for (int k = 0; k < S && i_left > 0; ++k) issue(s + k < S ? s + k : s + k - S);

    constexpr float kGrow = kInt4Head + 6.f;  // the reference, kInt4Head below a maximum, moves when one exceeds it by more
    const int tau = token_of_row(mg);
    const int va = mt, vb = 4 + (mt ^ 1);  // V's tokens of a lane: rows 2 mt and 2 mt + 1
    // paired: the low and the high weight of a transposed word, in the half of this column's groups
    const uint32_t sel0 = mg >> 2 ? 0x1044u : 0x4410u, sel1 = mg >> 2 ? 0x3244u : 0x4432u;
    auto load_units = [](const unsigned char *src, uint32_t (&u0)[NG / 2], uint32_t (&u1)[NG / 2]) {
        if constexpr (NG == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src);
            u0[0] = u.x;
            u0[1] = u.y;
            u1[0] = u.z;
            u1[1] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            u0[0] = u.x;
            u1[0] = u.y;
        }
    };
    auto load_params = [&](const unsigned char *src, uint32_t (&w)[GL]) {
        if constexpr (kPaired) {
#pragma unroll
            for (int j = 0; j < GL; ++j) w[j] = *reinterpret_cast<const uint32_t *>(src + 8 * j + 4 * par);
        } else if constexpr (NG == 4) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src);
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2 *>(src);
            w[0] = u.x;
            w[1] = u.y;
        }
    };
    // A lane's weights of a token times its group's scale, as a fp16 pair, and the group's zero added to their sums.
    // fp16 rows: the pair's rounding counts for the code's distance from 8 only, since 8 of it go with the zero,
    // unrounded (p s c + p z = w (c - 8) + p (z + 8 s) with w for p s): codes stand for values around zero, so that the
    // error is that of one more rounding of the output, where it was twice that in contexts of a few tokens.
    // kOwn: the pair is taken times down (powers of two), whose inverses are up.
    auto weigh = [](const float (&p)[2], float2 sz, float (&z)[2], const float (&down)[2], const float (&up)[2]) {
        const __half2 w = kOwn ? __floats2half2_rn(p[0] * sz.x * down[0], p[1] * sz.x * down[1]) : __floats2half2_rn(p[0] * sz.x, p[1] * sz.x);
        const uint32_t bits = *reinterpret_cast<const uint32_t *>(&w);
        if constexpr (!kBF16) {
            if constexpr (kOwn) {
                z[0] = fmaf(__low2float(w), -8.f * up[0], z[0]);
                z[1] = fmaf(__high2float(w), -8.f * up[1], z[1]);
            } else {
                const __half2 less = __hmul2(w, __float2half2_rn(-8.f));  // exact
                add_f16x2(z[0], z[1], *reinterpret_cast<const uint32_t *>(&less));
            }
            sz.y = fmaf(8.f, sz.x, sz.y);
        }
        z[0] = fmaf(p[0], sz.y, z[0]);
        z[1] = fmaf(p[1], sz.y, z[1]);
        return bits;
    };
    // Waits for the copies in flight from chunk c + k on (chunk c's stage is s); by any lane.
    auto drain = [&](int c, int k) {
        bool done = true;
        for (; k < S && k < left - (c - chunk); ++k)
            done &= mbar_wait_bounded(&my_bars[s + k < S ? s + k : s + k - S], s + k < S ? phase : phase ^ 1u, kDrainTimeoutNs);
        return done;
    };
    // Whether one of four tokens' rows wants exponents of its own, from their largest and smallest (scale, zero) words: the
    // sign of a difference.
    auto wants_own = [](const uint32_t (&top)[4], const uint32_t (&least)[4]) {
        uint32_t below = 0;
#pragma unroll
        for (int i = 0; i < 4; i += 2)
            below |= fma_halves<T>(__byte_perm(top[i], top[i + 1], 0x5410), -kInt4Ratio, __byte_perm(least[i], least[i + 1], 0x5410));
        if constexpr (kBF16) {
            const uint32_t high = max_halves<T>(max_halves<T>(top[0], top[1]), max_halves<T>(top[2], top[3]));
            const uint32_t low = min_halves<T>(min_halves<T>(least[0], least[1]), min_halves<T>(least[2], least[3]));
            below |= fma_halves<T>(high, -1.f, kInt4Most) | fma_halves<T>(low, 1.f, kInt4Least);
        }
        return (below & 0x80008000u) != 0;
    };
    // The exponent, per column of this lane, of its tokens' largest |w|; the power of two that brings it into [2^11, 2^12), and
    // that one's inverse.
    auto exponents = [](float w0, float w1) {
        uint32_t x = (__float_as_uint(w0) >> 23) | ((__float_as_uint(w1) >> 23) << 16);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) x = __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, o));
        return x;
    };
    auto powers = [](uint32_t x, float (&down)[2], float (&up)[2]) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = max(static_cast<int>(x >> (16 * e) & 0xffffu) - 127 - 11, -100);
            down[e] = exp2_int(-k);
            up[e] = exp2_int(k);
        }
    };
    auto add_back = [](float (&to)[2][4], const float (&sum)[2][4], const float (&up)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) to[h][e] = fmaf(sum[h][e], up[e & 1], to[h][e]);
    };
    // the eight tokens 8 i .. 8 i + 7 of a stage's half: their block's record and their first row in it
    auto octet = [](const unsigned char *half, int i) { return half + 8 * i / BS * G::kRecord; };
    auto first_row = [](int i) { return 8 * i % BS; };

    Int4Split split = at.split;
    bool resume = kOwn;
    for (bool first_piece = at.first_piece; left > 0; first_piece = false) {
        const int ctx = p.context_lens[seq], len = min(max(ctx, 0), p.len_cap);
        const int chunks = int4_chunks(len), end = min(chunks, chunk + left);
        if (chunk == 0 && unit == 0 && ctx != len && lane == 0) raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        const int kvh = unit / p.blocks, sub = unit - kvh * p.blocks;
        const int hq0 = kvh * p.group + sub * HEADS;
        const int nheads = min(HEADS, p.group - sub * HEADS);

        // ---- the query: lane (mg, mt) holds column mg of every column tile (paired: head mg % 4 in the groups
        //      2 i + mg / 4) at channels 32 j + 8 mt + 0 .. 7, the channels of a K row's units 2 mt and 2 mt + 1.
        //      Scaled by a power of two (a head's largest magnitude into [2^9, 2^10)), then odd nibbles' by 1/16.
        uint32_t qb[N][NG][4], zb[N][2];  // zb: sum(q) per group, in 16-bit pieces along k
        float hs[N][2];                    // score scale of heads 2 mt, 2 mt + 1, log2 units
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float f[GL][8];
            const int h = kPaired ? mg & 3 : 8 * n + mg;
            const int col_par = mg >> 2;  // paired: this column's groups
            const T *qrow = static_cast<const T *>(p.q) + (static_cast<int64_t>(seq) * p.num_q_heads + hq0 + h) * D + 8 * mt;
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < GL; ++j) {
                const uint4 u = h < nheads ? *reinterpret_cast<const uint4 *>(qrow + 32 * (kPaired ? 2 * j + col_par : j)) : make_uint4(0, 0, 0, 0);
                Elem<T>::to_f32x8(u, f[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[j][e]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            if constexpr (kPaired) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 16));
            const int qe = row_exponent(amax);
            const float down = exp2_int(-qe) * 1024.f;
            const float up = exp2_int(qe) * (p.scale_log2 / 1024.f);
            float sum[NG];
#pragma unroll
            for (int j = 0; j < GL; ++j) {
                float t = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float fe = e & 1 ? 0.0625f : 1.f;
                    const float a = f[j][e] * down, b = f[j][4 + e] * down;
                    float ra, rb;
                    if constexpr (kPaired) {
                        // the other groups' k index stays zero
                        qb[n][2 * j][e] = col_par ? pack_mma2<false>(0.f, a * fe, ra, rb) : pack_mma2<false>(a * fe, 0.f, ra, rb);
                        qb[n][2 * j + 1][e] = col_par ? pack_mma2<false>(0.f, b * fe, ra, rb) : pack_mma2<false>(b * fe, 0.f, ra, rb);
                    } else {
                        qb[n][j][e] = pack_mma2<false>(a * fe, b * fe, ra, rb);
                    }
                    t += a + b;
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                if constexpr (kPaired) {
                    // the zeros' sums go into the first four columns, all groups' (the halves are added later)
                    const float u = __shfl_xor_sync(0xffffffffu, t, 16);
                    sum[2 * j] = col_par ? 0.f : t;
                    sum[2 * j + 1] = col_par ? 0.f : u;
                } else {
                    sum[j] = t;
                }
            }
            // k of the zeros' MMA: group pair (k / 2) % (NG / 2) of piece k / NG; the pieces of a sum are its
            // rounding to the MMA's type, that of the remainder, and (bf16) of what then remains
            const int pair = NG == 4 ? mt & 1 : 0, piece = NG == 4 ? mt >> 1 : mt;
            float a = pair ? sum[NG - 2] : sum[0], b = pair ? sum[NG - 1] : sum[1];
            constexpr int PIECES = kBF16 ? 3 : 2;
            zb[n][0] = zb[n][1] = 0u;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                float ra, rb;
                const uint32_t w = pack_mma2<kBF16>(a, b, ra, rb);
                if (piece == k) zb[n][0] = w;
                if (NG == 4 && k == 2 && piece == 0) zb[n][1] = w;
                a -= ra;
                b -= rb;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) hs[n][e] = __shfl_sync(0xffffffffu, up, 4 * (kPaired ? 2 * (mt & 1) + e : 2 * mt + e));
        }

        // ---- accumulators: O^T m-tile (j, half) holds channels 32 group_of(j) + 4 mg + 2 half (d0, d1) and + 1
        //      (d2, d3) of heads head_of(n, 0) (d0, d2) and head_of(n, 1)
        float oacc[N][GL][2][4], zacc[N][GL][2], m[N][2], l[N][2];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int j = 0; j < GL; ++j) {
                zacc[n][j][0] = zacc[n][j][1] = 0.f;
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[n][j][0][e] = oacc[n][j][1][e] = 0.f;
            }
        }
        int c = chunk;
        if constexpr (kOwn) {
            if (resume) {
                c = at.c;
#pragma unroll
                for (int n = 0; n < N; ++n) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) m[n][e] = at.m[n][e], l[n][e] = at.l[n][e];
#pragma unroll
                    for (int j = 0; j < GL; ++j) {
                        zacc[n][j][0] = at.zacc[n][j][0], zacc[n][j][1] = at.zacc[n][j][1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) oacc[n][j][0][e] = at.oacc[n][j][0][e], oacc[n][j][1][e] = at.oacc[n][j][1][e];
                    }
                }
            }
            resume = false;
        }
        for (; c < end; ++c) {
            const bool ok = mbar_wait_bounded(&my_bars[s], phase, kWaitTimeoutNs);
            if (__any_sync(0xffffffffu, !ok)) {
                // give up: flag it, let this warp's copies still in flight land, stop
                if (lane == 0) {
                    raise_flag(p.status, PKV_DEVERR_TIMEOUT);
                    drain(c, 0);
                    if (!p.by_unit) p.splits[worker].pieces = 0;
                }
                __syncwarp();
                return true;
            }
            // tokens of the stage that count: in the context, and their block copied
            const int valid = len - c * 32;  // >= 1, but 0 for an empty context
            const uint32_t good = my_good[s];
            uint32_t vis = valid < 32 ? (1u << valid) - 1u : 0xffffffffu;
            if (good != (SB == 4 ? 0xffu : SB == 2 ? 0xfu : 0x3u)) {
#pragma unroll
                for (int b = 0; b < SB; ++b)
                    if (!(good >> (2 * b) & 1u)) vis &= BS == 32 ? 0u : ~(((1u << (BS & 31)) - 1u) << (b * BS & 31));
            }
            const bool partial = vis != 0xffffffffu;
            const unsigned char *kst = my_stages + s * G::kStageBytes, *vst = kst + G::kHalfBytes;
            // ---- S^T = K Q^T, tokens 8 i + tau (octets i): per group its own accumulator, then the scales
            float sc[4][N][2];  // [octet][column tile][heads head_of(n, 0 and 1)]
#pragma unroll
            for (int i2 = 0; i2 < 4; i2 += 2) {
                uint32_t u0[2][NG / 2], u1[2][NG / 2], kp[2][GL];  // words of units 2 mt, 2 mt + 1; (scale, zero)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const unsigned char *rec = octet(kst, i2 + r);
                    load_units(rec + (first_row(i2 + r) + tau) * ROW + mt * (ROW / 4), u0[r], u1[r]);
                    load_params(rec + BS * ROW + (first_row(i2 + r) + tau) * PAR, kp[r]);
                }
                // the zeros of this lane's group pair
                uint32_t z[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(octet(kst, i2 + r) + BS * ROW + (first_row(i2 + r) + tau) * PAR +
                                                                     (NG == 4 ? 8 * (mt & 1) : 0));
                    z[r] = __byte_perm(w.x, w.y, 0x7632);
                }
                float sz[N][4];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    sz[n][0] = sz[n][1] = sz[n][2] = sz[n][3] = 0.f;
                    mma_16816<kBF16>(sz[n], z[0], z[1], z[0], z[1], zb[n][0], zb[n][1]);
                }
                float ss[N][4];
#pragma unroll
                for (int j = 0; j < GL; ++j) {
                    const float pa = Int4Param<T>::unpack(kp[0][j]).x, pb = Int4Param<T>::unpack(kp[1][j]).x;
                    float a[N][4];
#pragma unroll
                    for (int n = 0; n < N; ++n) a[n][0] = a[n][1] = a[n][2] = a[n][3] = 0.f;
#pragma unroll
                    for (int x = 0; x < (kPaired ? 2 : 1); ++x) {
                        uint32_t ra[4], rb[4];
                        codes_f16(kPaired ? (x ? u1[0][j] : u0[0][j]) : group_word<NG>(u0[0], u1[0], j), ra);
                        codes_f16(kPaired ? (x ? u1[1][j] : u0[1][j]) : group_word<NG>(u0[1], u1[1], j), rb);
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            const uint32_t(&q)[4] = qb[n][kPaired ? 2 * j + x : j];
                            mma_16816<false>(a[n], ra[0], rb[0], ra[1], rb[1], q[0], q[1]);
                            mma_16816<false>(a[n], ra[2], rb[2], ra[3], rb[3], q[2], q[3]);
                        }
                    }
                    // (scalar products here and below: packed ones would take a second copy of the scale, a
                    // move on the busier integer pipe each)
#pragma unroll
                    for (int n = 0; n < N; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float by = e < 2 ? pa : pb;
                            ss[n][e] = j == 0 ? a[n][e] * by : fmaf(a[n][e], by, ss[n][e]);
                        }
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    constexpr float kUnit = 16777216.f;  // 2^24: the codes' unit
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = fmaf(ss[n][e], kUnit, sz[n][e]);
                        if constexpr (kPaired) x += __shfl_xor_sync(0xffffffffu, x, 2);  // the other groups'
                        sc[i2 + e / 2][n][e & 1] = x;
                    }
                }
            }
            // ---- V's (scale, zero) pairs; hidden tokens' do not count, whatever their rows hold (stale
            //      bytes, NaN scales)
            uint32_t vp[4][GL];
#pragma unroll
            for (int i = 0; i < 4; ++i) load_params(octet(vst, i) + BS * ROW + (first_row(i) + tau) * PAR, vp[i]);
            // log2 of each token's largest V scale; the clamps keep p (about 2^-e) in range
            float ev[4];
            uint32_t top[4], least[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                top[i] = least[i] = vp[i][0];
#pragma unroll
                for (int j = 1; j < GL; ++j) top[i] = max_halves<T>(top[i], vp[i][j]), least[i] = min_halves<T>(least[i], vp[i][j]);
                if constexpr (kPaired) top[i] = max_halves<T>(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
                ev[i] = fmaxf(fast_log2(Int4Param<T>::unpack(top[i]).x), static_cast<float>(kInt4Low));
            }
            if constexpr (kOwn && kBF16) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float z = 0.f;
#pragma unroll
                    for (int j = 0; j < GL; ++j) z = fmaxf(z, fabsf(Int4Param<T>::unpack(vp[i][j]).y));
                    if constexpr (kPaired) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 2));
                    ev[i] = fmaxf(fminf(ev[i], static_cast<float>(kInt4High)), fast_log2(z) - static_cast<float>(kInt4ZeroLift));
                }
            }
            bool odd = !kOwn && wants_own(top, least);  // one of this lane's rows
            if (partial) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if ((vis >> (8 * i + tau)) & 1u) continue;
                    ev[i] = -INFINITY;
                    top[i] = least[i] = kBF16 ? 0x3f80u : 0x3c00u;  // as one that wants none
#pragma unroll
                    for (int j = 0; j < GL; ++j) vp[i][j] = 0u;
#pragma unroll
                    for (int n = 0; n < N; ++n) sc[i][n][0] = sc[i][n][1] = 0.f;
                }
                odd = !kOwn && wants_own(top, least);
            }
            float mx[N][2];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < N; ++n) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 4; ++i) v = fmaxf(v, fmaf(sc[i][n][e], hs[n][e], ev[i]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                    mx[n][e] = v;
                    grow |= v > m[n][e] + kGrow;  // from -inf at the first visible token
                }
            }
            if (__any_sync(0xffffffffu, grow || odd)) {
                if (!kOwn && __any_sync(0xffffffffu, odd)) {
                    // the ring goes on behind the copies in flight, whose chunks are read again
                    if (!__all_sync(0xffffffffu, drain(c, 1))) {
                        if (lane == 0) {
                            raise_flag(p.status, PKV_DEVERR_TIMEOUT);
                            if (!p.by_unit) p.splits[worker].pieces = 0;
                        }
                        return true;
                    }
                    fence_proxy_async_smem();
                    const int next = s + min(S, left - (c - chunk));
                    at.seq = seq, at.unit = unit, at.chunk = chunk, at.c = c, at.left = left;
                    at.s = next < S ? next : next - S;
                    at.phase = next < S ? phase : phase ^ 1u;
                    at.first_piece = first_piece;
                    at.split = split;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) at.m[n][e] = m[n][e], at.l[n][e] = l[n][e];
#pragma unroll
                        for (int j = 0; j < GL; ++j) {
                            at.zacc[n][j][0] = zacc[n][j][0], at.zacc[n][j][1] = zacc[n][j][1];
#pragma unroll
                            for (int e = 0; e < 4; ++e) at.oacc[n][j][0][e] = oacc[n][j][0][e], at.oacc[n][j][1][e] = oacc[n][j][1][e];
                        }
                    }
                    return false;
                }
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[e] = 1.f;
                        if (mx[n][e] > m[n][e] + kGrow) {
                            a[e] = fast_exp2(m[n][e] - (mx[n][e] - kInt4Head));  // 0 when m = -inf
                            m[n][e] = mx[n][e] - kInt4Head;
                        }
                        l[n][e] *= a[e];
                    }
#pragma unroll
                    for (int j = 0; j < GL; ++j) {
                        zacc[n][j][0] *= a[0];
                        zacc[n][j][1] *= a[1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            oacc[n][j][0][e] *= a[e & 1];
                            oacc[n][j][1][e] *= a[e & 1];
                        }
                    }
                }
            }
            // ---- weights
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float ref = m[n][e] == -INFINITY ? 0.f : m[n][e];
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[i][n][e] = fast_exp2(fmaf(sc[i][n][e], hs[n][e], -ref));
                }
            if (partial) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (!((vis >> (8 * i + tau)) & 1u)) {
#pragma unroll
                        for (int n = 0; n < N; ++n) sc[i][n][0] = sc[i][n][1] = 0.f;
                    }
            }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) l[n][e] += (sc[0][n][e] + sc[1][n][e]) + (sc[2][n][e] + sc[3][n][e]);
            // ---- O^T += V^T P^T, 16 tokens at a time: the weights times a group's scales in the B layout,
            //      unit mg of tokens va, vb of both octets as the A fragments.  kOwn: each head's weights of a group are
            //      brought to 2^12 at most by a power of two before they are rounded, and their sums back.
            uint32_t ex[kOwn ? N : 1][kOwn ? GL : 1];
            if constexpr (kOwn) {
#pragma unroll
                for (int n = 0; n < N; ++n)
#pragma unroll
                    for (int j = 0; j < GL; ++j) {
                        float w[2] = {0.f, 0.f};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int e = 0; e < 2; ++e) w[e] = fmaxf(w[e], fabsf(sc[i][n][e] * Int4Param<T>::unpack(vp[i][j]).x));
                        ex[n][j] = exponents(w[0], w[1]);
                    }
            }
#pragma unroll
            for (int i2 = 0; i2 < 4; i2 += 2) {
                uint32_t v[4][NG / 2];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = i2 + r / 2;
                    const unsigned char *src = octet(vst, i) + (first_row(i) + (r & 1 ? vb : va)) * ROW + mg * (ROW / 8);
                    if constexpr (NG == 4) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src);
                        v[r][0] = u.x;
                        v[r][1] = u.y;
                    } else {
                        v[r][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                }
                if constexpr (kPaired) {
                    // an octet per MMA: its tokens take two k indices each, one per group of the word
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < GL; ++j) {
                            const float(&p)[2] = sc[i2 + r][0];
                            const float2 sz = Int4Param<T>::unpack(vp[i2 + r][j]);
                            uint32_t ra[4], rb[4];
                            codes_f16_bytes(v[2 * r][j], ra);
                            codes_f16_bytes(v[2 * r + 1][j], rb);
                            float down[2], up[2], sum[2][4] = {};
                            if constexpr (kOwn) powers(ex[0][j], down, up);
                            const uint32_t w = movmatrix_trans(weigh(p, sz, zacc[0][j], down, up));
                            const uint32_t b0 = __byte_perm(w, 0u, sel0), b1 = __byte_perm(w, 0u, sel1);
                            float(&to)[2][4] = kOwn ? sum : oacc[0][j];
                            mma_16816<false>(to[0], ra[0], ra[1], rb[0], rb[1], b0, b1);
                            mma_16816<false>(to[1], ra[2], ra[3], rb[2], rb[3], b0, b1);
                            if constexpr (kOwn) add_back(oacc[0][j], sum, up);
                        }
                } else {
#pragma unroll
                    for (int j = 0; j < GL; ++j) {
                        uint32_t ra[4], rb[4];
                        codes_f16_bytes(group_word<NG>(v[0], v[1], j), ra);
                        codes_f16_bytes(group_word<NG>(v[2], v[3], j), rb);
                        const float2 s0 = Int4Param<T>::unpack(vp[i2][j]), s1 = Int4Param<T>::unpack(vp[i2 + 1][j]);
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            const float(&p0)[2] = sc[i2][n], (&p1)[2] = sc[i2 + 1][n];
                            float down[2], up[2], sum[2][4] = {};
                            if constexpr (kOwn) powers(ex[n][j], down, up);
                            const uint32_t b0 = movmatrix_trans(weigh(p0, s0, zacc[n][j], down, up));
                            const uint32_t b1 = movmatrix_trans(weigh(p1, s1, zacc[n][j], down, up));
                            float(&to)[2][4] = kOwn ? sum : oacc[n][j];
                            mma_16816<false>(to[0], ra[0], ra[1], rb[0], rb[1], b0, b1);
                            mma_16816<false>(to[1], ra[2], ra[3], rb[2], rb[3], b0, b1);
                            if constexpr (kOwn) add_back(oacc[n][j], sum, up);
                        }
                    }
                }
            }
            __syncwarp();
            if (i_left > 0) {
                fence_proxy_async_smem();
                issue(s);
            }
            if (++s == S) {
                s = 0;
                phase ^= 1u;
            }
        }

        // ---- the unit's piece is done: a head's sums over its lanes, then out or into its slot
        const bool whole = chunk == 0 && end == chunks;
        const int64_t slot = (2 * static_cast<int64_t>(worker) + (first_piece ? 0 : 1)) * HEADS;
#pragma unroll
        for (int n = 0; n < N; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = head_of(n, e);
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
                const float norm = !whole ? 1.f : l[n][e] > 0.f ? 1.f / l[n][e] : 0.f;
                const int64_t row = static_cast<int64_t>(seq) * p.num_q_heads + hq0 + h;
#pragma unroll
                for (int j = 0; j < GL; ++j) {
                    float z = zacc[n][j][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                    constexpr float kEven = 16777216.f, kOdd = 1048576.f;  // 2^24, 2^20: the nibbles' places
                    const float r0 = fmaf(oacc[n][j][0][e], kEven, z) * norm, r1 = fmaf(oacc[n][j][0][2 + e], kOdd, z) * norm;
                    // (the third nibble's accumulator holds the fourth's too)
                    const float r2 = fmaf(oacc[n][j][1][e] - oacc[n][j][1][2 + e], kEven, z) * norm, r3 = fmaf(oacc[n][j][1][2 + e], kOdd, z) * norm;
                    if (h >= nheads) continue;
                    if (whole)
                        *reinterpret_cast<uint2 *>(static_cast<T *>(p.out) + row * D + 32 * group_of(j) + 4 * mg) =
                            make_uint2(Int4Param<T>::pack2_finite(r0, r1), Int4Param<T>::pack2_finite(r2, r3));
                    else
                        *reinterpret_cast<float4 *>(p.seg_o + (slot + h) * D + 32 * group_of(j) + 4 * mg) = make_float4(r0, r1, r2, r3);
                }
                if (!whole && mg == 0 && h < nheads) {
                    p.seg_m[slot + h] = m[n][e];
                    p.seg_l[slot + h] = l[n][e];
                }
            }
        }
        left -= end - chunk;
        if (chunk == 0) {  // (end < chunks: left is 0, and the pieces behind are those of the next workers)
            split = Int4Split{end < chunks ? 1 + (chunks - end + share - 1) / share : 0, worker, first_piece ? 0 : 1, seq, unit};
            if (p.by_unit && lane == 0) p.splits[seq * p.units + unit] = split;
        }
        chunk = 0;
        if (++unit == p.units) {
            unit = 0;
            ++seq;
        }
    }
    if (lane == 0 && !p.by_unit) p.splits[worker] = split;
    return true;
}

// Apart from the kernel, so that its registers are not spent on it.
template <typename T, int D, int BS, int NT>
__device__ __noinline__ void int4_work_own(const Int4Params &p, const int worker, const int share, Int4AtOf<D, BS, NT> &at) {
    int4_work<T, D, BS, NT, true>(p, worker, share, at);
}


template <typename T, int D, int BS, int NT>
__global__ void __launch_bounds__(128, DecodeInt4Geom<D, BS, NT>::kResident) paged_decode_int4_kernel(const __grid_constant__ Int4Params p) {
    using G = DecodeInt4Geom<D, BS, NT>;
    constexpr int NW = G::kWarps, S = G::kStages;
    pdl_trigger();  // the merge behind this grid may be placed
    pdl_wait();     // launched ahead of the end of the kernel before it

    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t *my_bars = reinterpret_cast<uint64_t *>(smem + NW * S * G::kStageBytes) + warp * S;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&my_bars[s], 1);
        fence_mbar_init();
    }
    __syncwarp();

    // ---- this worker's share: chunks [first, first + left) of the row
    const int worker = blockIdx.x * NW + warp;
    int total;
    const int share = int4_share(p, gridDim.x * NW, total);
    const int64_t first = static_cast<int64_t>(worker) * share;
    int left = first < total ? min(share, total - static_cast<int>(first)) : 0;
    if (left == 0) {
        if (lane == 0 && !p.by_unit) p.splits[worker].pieces = 0;
        return;
    }
    int seq = 0, unit = 0, chunk = 0;  // where the share begins
    for (int s0 = 0, before = 0;; s0 += 32) {
        const int mine = s0 + lane < p.num_seqs ? int4_chunks(int4_len(p, s0 + lane)) : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, static_cast<int64_t>(before + incl) * p.units > first);
        if (past) {
            const int l = __ffs(past) - 1;
            const int n = __shfl_sync(0xffffffffu, mine, l);
            const int pos = static_cast<int>(first - static_cast<int64_t>(before + __shfl_sync(0xffffffffu, incl - mine, l)) * p.units);
            seq = s0 + l;
            unit = pos / n;
            chunk = pos - unit * n;
            break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }

    Int4AtOf<D, BS, NT> at;
    at.seq = seq, at.unit = unit, at.chunk = at.c = chunk, at.left = left, at.s = 0;
    at.phase = 0u;
    at.first_piece = true;
    at.split = Int4Split{0, 0, 0, 0, 0};
    if (!int4_work<T, D, BS, NT, false>(p, worker, share, at)) int4_work_own<T, D, BS, NT>(p, worker, share, at);
}

// Log-sum-exp merge of the cut units: entry blockIdx.x of their table.  WPH warps share a head's pieces:
// four where units are few and cut into many (grid.y: the heads), else one (grid.y: the heads' fours, or
// all in turn).
template <typename T, int D, int WPH>
__global__ void __launch_bounds__(128) paged_decode_int4_merge_kernel(const Int4Params p, int heads) {
    static_assert(WPH == 1 || WPH == 4, "one or four warps per head");
    constexpr int PER = D / 32;
    using Part = typename std::conditional<PER == 4, float4, float2>::type;
    __shared__ float comb[WPH == 4 ? 4 : 1][D + 2];  // the four warps' (o, m, l) of a head
    pdl_trigger();
    pdl_wait();
    Int4Split s = p.splits[blockIdx.x];
    if (p.by_unit) {
        s.seq = blockIdx.x / p.units;
        s.unit = blockIdx.x - s.seq * p.units;
    }
    // (a kernel that gave up on a wait leaves entries unwritten)
    if (s.pieces <= 0 || s.worker < 0 || s.worker >= p.seg_workers || s.pieces > p.seg_workers - s.worker || (s.slot & ~1)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int kvh = s.unit / p.blocks, sub = s.unit - kvh * p.blocks;
    const int nheads = min(heads, p.group - sub * heads);
    auto slot = [&](int i, int h) { return (2 * static_cast<int64_t>(s.worker + i) + (i == 0 ? s.slot : 0)) * heads + h; };
    const int share = WPH == 4 ? warp : 0;
    const int mine = s.pieces > share ? (s.pieces - share + WPH - 1) / WPH : 0;  // pieces share, share + WPH, ...
    for (int h = WPH == 4 ? blockIdx.y : blockIdx.y * 4 + warp; h < nheads; h += WPH == 4 ? gridDim.y : 4 * gridDim.y) {
        // the first pieces' rows are on their way while the maxima are compared
        Part v[8];
        auto rows = [&](int i0) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (i0 + u < mine) v[u] = reinterpret_cast<const Part *>(p.seg_o + slot(share + WPH * (i0 + u), h) * D)[lane];
        };
        rows(0);
        float mmax = -INFINITY;
        for (int i = lane; i < mine; i += 32) mmax = fmaxf(mmax, p.seg_m[slot(share + WPH * i, h)]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mmax = fmaxf(mmax, __shfl_xor_sync(0xffffffffu, mmax, o));
        float lsum = 0.f, o[PER] = {};
        for (int i0 = 0; i0 < mine; i0 += 32) {
            const int cnt = min(32, mine - i0);
            float w = 0.f;  // this lane's piece
            if (lane < cnt) {
                const int64_t at = slot(share + WPH * (i0 + lane), h);
                const float mi = p.seg_m[at];
                w = mi == -INFINITY ? 0.f : fast_exp2(mi - mmax);
                lsum = fmaf(w, p.seg_l[at], lsum);
            }
            for (int j0 = 0; j0 < cnt; j0 += 8) {
                if (i0 + j0 > 0) rows(i0 + j0);
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float wu = __shfl_sync(0xffffffffu, w, (j0 + u) & 31);
                    if (j0 + u < cnt) {
                        const float *f = reinterpret_cast<const float *>(&v[u]);
#pragma unroll
                        for (int e = 0; e < PER; ++e) o[e] = fmaf(wu, f[e], o[e]);
                    }
                }
            }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, off);
        if constexpr (WPH == 4) {
            // the four warps' results, relative to their own maxima, combined in warp 0
            __syncthreads();  // (the head before is read)
#pragma unroll
            for (int e = 0; e < PER; ++e) comb[warp][lane * PER + e] = o[e];
            if (lane == 0) {
                comb[warp][D] = mmax;
                comb[warp][D + 1] = lsum;
            }
            __syncthreads();
            if (warp != 0) continue;
            float mall = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) mall = fmaxf(mall, comb[w][D]);
            lsum = 0.f;
#pragma unroll
            for (int e = 0; e < PER; ++e) o[e] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float sw = comb[w][D] == -INFINITY ? 0.f : fast_exp2(comb[w][D] - mall);
                lsum = fmaf(sw, comb[w][D + 1], lsum);
#pragma unroll
                for (int e = 0; e < PER; ++e) o[e] = fmaf(sw, comb[w][lane * PER + e], o[e]);
            }
        }
        const float norm = lsum > 0.f ? 1.f / lsum : 0.f;
        T *dst = static_cast<T *>(p.out) + (static_cast<int64_t>(s.seq) * p.num_q_heads + kvh * p.group + sub * heads + h) * D + PER * lane;
#pragma unroll
        for (int e = 0; e < PER; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = Int4Param<T>::pack2_finite(o[e] * norm, o[e + 1] * norm);
    }
}

}  // namespace pkv
