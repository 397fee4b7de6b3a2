// decode_int4_kernel.cuh -- paged decode attention over the 4-bit cache (format: int4.cuh),
// one CTA per (partition of the context, KV head [x block of query heads], sequence).
//
// What it computes: the decode's softmax attention (decode_kernel.cuh) with the values that the
// codes stand for, K_t = sK c + zK and V_t = sV c + zV per group j of 32 channels:
//     s_t = scale * sum_j ( sK[t,j] (q_j . c[t,j]) + zK[t,j] sum(q_j) ),
//     o   = sum_t p_t ( sV[t,j] c[t,j] + zV[t,j] ),       p_t = exp(s_t - ref).
// The codes meet the query and the weights as exact small integers, and a token's scales
// enter once per group: q_j . c is one group's MMA accumulator, the V scale multiplies the
// weight (p_t sV[t,j], rounded once to fp16), and the zeros are plain fp32 sums.
//
// What bounds it: 5/8 byte a value, a quarter of what a 16-bit cache reads, against the same
// number of codes to widen; so per code the kernel spends 0.9 integer operations and half an
// MMA slot, and little else.
//  * Both products run as warp-level MMAs (m16n8k16, fp16 operands, fp32 accumulators) with the
//    tokens (S^T = K Q^T) or the channels (O^T = V^T P^T) as the 16 rows and eight query heads as the
//    columns, for any group of heads: unused columns are zero.  Groups of more than eight heads take
//    two column tiles on the same K and V fragments, so their codes are widened once.
//  * Widening: four codes of a 16-bit word become fp16 numbers without a conversion: shifted so
//    that a nibble falls on mantissa bits 2 .. 5 or 6 .. 9 of 1024.0, it reads 1024 + 4 c or
//    1024 + 64 c (codes_f16).  (At bits 0 .. 3, without a shift, the offset would be 68 times the
//    largest code and cost the sums that many roundings; here it is 17 times at most.)  K's factor 1/4
//    or 1/64 is in the query, V's is applied to the output channel, whose accumulator holds one nibble
//    position only.  K's offset is the accumulator's start, -1024 sum(q); V's is 1024 times the sum of
//    the weights as they were rounded, which one more MMA against ones makes.
//  * The weights' reference is the running maximum of s_t + log2(max_j sV[t,j]), not of s_t, so that
//    p_t sV[t,j], what fp16 has to hold, is at most 2^6 and near 1 where it counts, whatever V's scale is.
//  * Each warp streams its own ring of 32-token stages by bulk copies (a block's record of one head is
//    contiguous: codes and scales arrive together) and shares nothing with the other warps until the end.
//  * The token of an MMA row is chosen so that V's four token rows of a load lie side by side
//    (token_of_row): two-way instead of four-way shared-memory conflicts.
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
    static constexpr int kResident = NT == 1 ? 3 : 2;              // CTAs per SM, by registers
    // about 180 KB of stages per SM: several times the bytes that cover the memory latency
    static constexpr int kStages = (NT == 1 ? 15360 : 20480) / kStageBytes;
    static constexpr int kMaxTableEntries = 1024;
    static constexpr int kHeads = 8 * NT;
    static constexpr int kSmemBytes = kWarps * kStages * (kStageBytes + 8) + kMaxTableEntries * 4;
    static_assert(kHeads * (D + 4) * 4 <= kStages * kStageBytes, "merge scratch must fit a warp's stages");
};

// The token (0 .. 7) of MMA row r: rows 2 t, which one lane load of V takes for t = 0 .. 3, are
// tokens 0 .. 3, and rows 2 t + 1 tokens 5, 4, 7, 6.
__host__ __device__ constexpr int token_of_row(int r) { return r & 1 ? 4 + ((r >> 1) ^ 1) : r >> 1; }

// Four codes in each half of a word -> fp16 pairs: r[0], r[2] = 1024 + 4 c, r[1], r[3] = 1024 + 64 c.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t (&r)[4]) {
    const uint32_t a = x << 2, b = x >> 6;
    r[0] = (a & 0x003c003cu) | 0x64006400u;
    r[1] = (a & 0x03c003c0u) | 0x64006400u;
    r[2] = (b & 0x003c003cu) | 0x64006400u;
    r[3] = (b & 0x03c003c0u) | 0x64006400u;
}
constexpr float kInt4Offset = 1024.f;

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

template <typename T, int D, int BS, int NT>
__global__ void __launch_bounds__(128, DecodeInt4Geom<D, BS, NT>::kResident) paged_decode_int4_kernel(const DecodeParams p) {
    using G = DecodeInt4Geom<D, BS, NT>;
    constexpr int NW = G::kWarps, S = G::kStages, NG = G::kGroups, ST = G::kStageTokens, SB = G::kBlocks;
    constexpr int ROW = int4_row_bytes(D), PAR = int4_param_bytes(D);
    if (p.trigger_dependents) pdl_trigger();

    extern __shared__ __align__(128) unsigned char smem[];
    unsigned char *stages = smem;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + NW * S * G::kStageBytes);
    int32_t *tbl = reinterpret_cast<int32_t *>(smem + NW * S * (G::kStageBytes + 8));

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int part = blockIdx.x, seq = blockIdx.z;
    const int kvh = blockIdx.y / p.subgroups, sub = blockIdx.y - kvh * p.subgroups;
    const int hq0 = kvh * p.group + sub * G::kHeads;
    const int nheads = min(G::kHeads, p.group - sub * G::kHeads);

    // ---- the partition's table entries, fetched together with the context length
    const int tok0 = part * p.partition_size;
    const int32_t *trow = p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + tok0 / BS;
    int first_entry = 0;
    if (static_cast<int>(threadIdx.x) < min(p.max_blocks_per_seq - tok0 / BS, p.partition_size / BS))
        first_entry = trow[threadIdx.x];
    int len = p.context_lens[seq];
    if (len < 0 || len > p.len_cap) {
        if (threadIdx.x == 0 && part == 0 && blockIdx.y == 0) raise_flag(p.status, PKV_DEVERR_CONTEXT_LEN);
        len = len < 0 ? 0 : p.len_cap;
    }
    const int nparts = partitions_of(p, len);
    if (part >= nparts) return;  // uniform over the CTA
    const int ntok = max(0, min(len, tok0 + p.partition_size) - tok0);
    const int nchunks = (ntok + ST - 1) / ST;
    const int nblk = (ntok + BS - 1) / BS;
    for (int i = threadIdx.x; i < nblk; i += blockDim.x) {
        int b = i < static_cast<int>(blockDim.x) ? first_entry : trow[i];
        if (b < 0 || b >= p.num_blocks) {
            raise_flag(p.status, PKV_DEVERR_BLOCK_TABLE);
            b = -1;
        }
        tbl[i] = b;
    }
    unsigned char *my_stages = stages + warp * S * G::kStageBytes;
    uint64_t *my_bars = bars + warp * S;
    if (lane == 0) {
        for (int s = 0; s < S; ++s) mbar_init(&my_bars[s], 1);
        fence_mbar_init();
    }
    __syncthreads();

    // chunk c (32 tokens) -> stage s of this warp; flagged blocks are not copied
    const uint64_t policy = l2_policy_evict_first();
    const char *kc = static_cast<const char *>(p.k_cache) + static_cast<int64_t>(kvh) * G::kRecord;
    const char *vc = static_cast<const char *>(p.v_cache) + static_cast<int64_t>(kvh) * G::kRecord;
    auto issue = [&](int c, int s) {
        const int b0 = c * SB, nb = min(SB, nblk - b0);
        uint32_t bytes = 0;
#pragma unroll
        for (int i = 0; i < SB; ++i)
            if (i < nb && tbl[b0 + i] >= 0) bytes += 2 * G::kRecord;
        if (bytes == 0) {
            mbar_arrive(&my_bars[s]);
            return;
        }
        mbar_arrive_expect_tx(&my_bars[s], bytes);
        unsigned char *dst = my_stages + s * G::kStageBytes;
#pragma unroll
        for (int i = 0; i < SB; ++i) {
            if (i >= nb || tbl[b0 + i] < 0) continue;
            const int64_t at = static_cast<int64_t>(tbl[b0 + i]) * p.block_stride;
            bulk_copy_g2s(dst + i * G::kRecord, kc + at, G::kRecord, &my_bars[s], policy);
            bulk_copy_g2s(dst + G::kHalfBytes + i * G::kRecord, vc + at, G::kRecord, &my_bars[s], policy);
        }
    };
    const int my_chunks = nchunks > warp ? (nchunks - warp + NW - 1) / NW : 0;
    if (lane == 0) {
        for (int i = 0; i < S && i < my_chunks; ++i) issue(warp + i * NW, i);
    }

    // ---- the query: lane (mg, mt) holds column (head) mg of every column tile at channels
    //      32 j + 8 mt + 0 .. 7, the channels of a K row's units 2 mt and 2 mt + 1.  Scaled by a
    //      power of two (its largest magnitude into [2^5, 2^6)), then nibble e's by 1/4 or 1/64.
    const int mg = lane >> 2, mt = lane & 3;
    uint32_t qb[NT][NG][4];
    float off[NT][NG][2], qs[NT][NG][2];  // -1024 sum(q'), sum(q) of heads 2 mt, 2 mt + 1 per group
    float hs[NT][2];                      // their score scale, log2 units
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float f[NG][8];
        const int h = 8 * n + mg;
        const T *qrow = static_cast<const T *>(p.q) + (static_cast<int64_t>(seq) * p.num_q_heads + hq0 + h) * D + 8 * mt;
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            const uint4 u = h < nheads ? *reinterpret_cast<const uint4 *>(qrow + 32 * j) : make_uint4(0, 0, 0, 0);
            Elem<T>::to_f32x8(u, f[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[j][e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int qe = row_exponent(amax);
        const float down = exp2_int(-qe) * 64.f;
        const float up = exp2_int(qe) * (p.scale_log2 / 64.f);
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            float sum_q = 0.f, sum_r = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float fe = e & 1 ? 1.f / 64.f : 0.25f;
                const float a = f[j][e] * down, b = f[j][4 + e] * down;
                float ra, rb;
                qb[n][j][e] = pack_mma2<false>(a * fe, b * fe, ra, rb);
                sum_q += a + b;
                sum_r += ra + rb;
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                sum_q += __shfl_xor_sync(0xffffffffu, sum_q, o);
                sum_r += __shfl_xor_sync(0xffffffffu, sum_r, o);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                qs[n][j][e] = __shfl_sync(0xffffffffu, sum_q, 4 * (2 * mt + e));
                off[n][j][e] = -kInt4Offset * __shfl_sync(0xffffffffu, sum_r, 4 * (2 * mt + e));
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) hs[n][e] = __shfl_sync(0xffffffffu, up, 4 * (2 * mt + e));
    }

    // ---- accumulators: O^T m-tile (j, half) holds channels 32 j + 4 mg + 2 half (d0, d1) and + 1
    //      (d2, d3) of heads 2 mt (d0, d2) and 2 mt + 1; ones: 1024 times the sums of the rounded weights
    float oacc[NT][NG][2][4], ones[NT][NG][4], zacc[NT][NG][2], m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) {
            zacc[n][j][0] = zacc[n][j][1] = 0.f;
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[n][j][0][e] = oacc[n][j][1][e] = ones[n][j][e] = 0.f;
        }
    }
    constexpr float kGrow = 6.f;  // the reference moves when a maximum exceeds it by more (log2 units)
    const int tau = token_of_row(mg);
    const int va = mt, vb = 4 + (mt ^ 1);  // V's tokens of a lane: rows 2 mt and 2 mt + 1

    bool aborted = false;
    for (int i = 0; i < my_chunks; ++i) {
        const int s = i % S;
        const bool ok = mbar_wait_bounded(&my_bars[s], (i / S) & 1, kWaitTimeoutNs);
        if (__any_sync(0xffffffffu, !ok)) {
            // give up: flag it, let this warp's copies still in flight land, stop
            if (lane == 0) {
                raise_flag(p.status, PKV_DEVERR_TIMEOUT);
                for (int k = i; k < my_chunks && k < i + S; ++k)
                    mbar_wait_bounded(&my_bars[k % S], (k / S) & 1, kDrainTimeoutNs);
            }
            __syncwarp();
            aborted = true;
            break;
        }
        const int c = warp + i * NW;
        const int valid = min(ST, ntok - c * ST);  // >= 1
        // tokens of the stage that count: in the context, and their block's entry not flagged
        uint32_t vis = valid < 32 ? (1u << valid) - 1u : 0xffffffffu;
#pragma unroll
        for (int b = 0; b < SB; ++b) {
            if (b * BS < valid && tbl[c * SB + b] < 0) vis &= BS == 32 ? 0u : ~(((1u << (BS & 31)) - 1u) << (b * BS & 31));
        }
        const unsigned char *kst = my_stages + s * G::kStageBytes, *vst = kst + G::kHalfBytes;
#pragma unroll
        for (int tb = 0; tb < ST; tb += 16) {
            if (tb >= valid) break;  // warp-uniform: the step holds no context token
            const bool partial = ((vis >> tb) & 0xffffu) != 0xffffu;
            // rows mg and mg + 8 of the tile: tokens tb + tau and tb + 8 + tau
            constexpr int B = BS;
            const int ba = tb / B, oa = tb % B, bb = (tb + 8) / B, ob = (tb + 8) % B;
            const unsigned char *ka = kst + ba * G::kRecord, *kb = kst + bb * G::kRecord;
            const unsigned char *wa = vst + ba * G::kRecord, *wb = vst + bb * G::kRecord;
            // ---- S^T = K Q^T: per group its own accumulator, from the offset on
            uint32_t k0[2][NG / 2], k1[2][NG / 2];  // [row half][words of units 2 mt, 2 mt + 1]
            uint32_t kp[2][NG], vp[2][NG];          // (scale, zero) words of the two tokens
            auto load_units = [&](const unsigned char *src, uint32_t (&u0)[NG / 2], uint32_t (&u1)[NG / 2]) {
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
            auto load_params = [&](const unsigned char *src, uint32_t (&w)[NG]) {
                if constexpr (NG == 4) {
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
            load_units(ka + (oa + tau) * ROW + mt * (ROW / 4), k0[0], k1[0]);
            load_units(kb + (ob + tau) * ROW + mt * (ROW / 4), k0[1], k1[1]);
            load_params(ka + B * ROW + (oa + tau) * PAR, kp[0]);
            load_params(kb + B * ROW + (ob + tau) * PAR, kp[1]);
            load_params(wa + B * ROW + (oa + tau) * PAR, vp[0]);
            load_params(wb + B * ROW + (ob + tau) * PAR, vp[1]);
            float sc[NT][4];  // tokens (0, 1: tau, 2, 3: 8 + tau) x heads 2 mt, 2 mt + 1
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t ra[4], rb[4];
                codes_f16(group_word<NG>(k0[0], k1[0], j), ra);
                codes_f16(group_word<NG>(k0[1], k1[1], j), rb);
                const float2 pa = Int4Param<T>::unpack(kp[0][j]), pb = Int4Param<T>::unpack(kp[1][j]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float a[4] = {off[n][j][0], off[n][j][1], off[n][j][0], off[n][j][1]};
                    mma_16816<false>(a, ra[0], rb[0], ra[1], rb[1], qb[n][j][0], qb[n][j][1]);
                    mma_16816<false>(a, ra[2], rb[2], ra[3], rb[3], qb[n][j][2], qb[n][j][3]);
                    fma_f32x2(sc[n][0], sc[n][1], a[0], a[1], pa.x, pa.x);
                    fma_f32x2(sc[n][2], sc[n][3], a[2], a[3], pb.x, pb.x);
                    fma_f32x2(sc[n][0], sc[n][1], qs[n][j][0], qs[n][j][1], pa.y, pa.y);
                    fma_f32x2(sc[n][2], sc[n][3], qs[n][j][0], qs[n][j][1], pb.y, pb.y);
                }
            }
            float2 sv[2][NG];  // V's (scale, zero)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int j = 0; j < NG; ++j) sv[r][j] = Int4Param<T>::unpack(vp[r][j]);
            bool seen[2] = {true, true};
            if (partial) {
                // hidden tokens: what their rows hold (stale bytes, NaN scales) does not count
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    seen[r] = (vis >> (tb + 8 * r + tau)) & 1u;
#pragma unroll
                    for (int j = 0; j < NG; ++j)
                        if (!seen[r]) sv[r][j] = make_float2(0.f, 0.f);
                }
            }
            // log2 of the token's largest V scale; the clamp keeps p (at most 2^-e) in range
            float ev[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float most = sv[r][0].x;
#pragma unroll
                for (int j = 1; j < NG; ++j) most = fmaxf(most, sv[r][j].x);
                ev[r] = fmaxf(fast_log2(most), -40.f);
            }
            float mx[NT][2];
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[n][e] *= hs[n][e & 1];
                    if (partial && !seen[e >> 1]) sc[n][e] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float v = fmaxf(sc[n][e] + ev[0], sc[n][2 + e] + ev[1]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
                    mx[n][e] = v;
                    grow |= v > m[n][e] + kGrow;  // from -inf at the first visible token
                }
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float a[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        a[e] = 1.f;
                        if (mx[n][e] > m[n][e] + kGrow) {
                            a[e] = fast_exp2(m[n][e] - mx[n][e]);  // 0 when m = -inf
                            m[n][e] = mx[n][e];
                        }
                        l[n][e] *= a[e];
                    }
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        zacc[n][j][0] *= a[0];
                        zacc[n][j][1] *= a[1];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            ones[n][j][e] *= a[e & 1];
                            oacc[n][j][0][e] *= a[e & 1];
                            oacc[n][j][1][e] *= a[e & 1];
                        }
                    }
                }
            }
            // ---- weights, and their products with V's scales in the B layout of O^T
            uint32_t pb0[NT][NG], pb1[NT][NG];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
                const float w[4] = {fast_exp2(sc[n][0] - r0), fast_exp2(sc[n][1] - r1), fast_exp2(sc[n][2] - r0),
                                    fast_exp2(sc[n][3] - r1)};
                l[n][0] += w[0] + w[2];
                l[n][1] += w[1] + w[3];
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    const __half2 ha = __floats2half2_rn(w[0] * sv[0][j].x, w[1] * sv[0][j].x);
                    const __half2 hb = __floats2half2_rn(w[2] * sv[1][j].x, w[3] * sv[1][j].x);
                    pb0[n][j] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&ha));
                    pb1[n][j] = movmatrix_trans(*reinterpret_cast<const uint32_t *>(&hb));
                    fma_f32x2(zacc[n][j][0], zacc[n][j][1], w[0], w[1], sv[0][j].y, sv[0][j].y);
                    fma_f32x2(zacc[n][j][0], zacc[n][j][1], w[2], w[3], sv[1][j].y, sv[1][j].y);
                }
            }
            // ---- O^T += V^T P^T: unit mg of tokens va, vb and 8 + va, 8 + vb
            uint32_t v[4][NG / 2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const unsigned char *src = (r < 2 ? wa + oa * ROW : wb + ob * ROW) + (r & 1 ? vb : va) * ROW + mg * (ROW / 8);
                if constexpr (NG == 4) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(src);
                    v[r][0] = u.x;
                    v[r][1] = u.y;
                } else {
                    v[r][0] = *reinterpret_cast<const uint32_t *>(src);
                }
            }
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                uint32_t ra[4], rb[4];
                codes_f16(group_word<NG>(v[0], v[1], j), ra);
                codes_f16(group_word<NG>(v[2], v[3], j), rb);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    mma_16816<false>(oacc[n][j][0], ra[0], ra[1], rb[0], rb[1], pb0[n][j], pb1[n][j]);
                    mma_16816<false>(oacc[n][j][1], ra[2], ra[3], rb[2], rb[3], pb0[n][j], pb1[n][j]);
                    mma_16816<false>(ones[n][j], 0x64006400u, 0x64006400u, 0x64006400u, 0x64006400u, pb0[n][j], pb1[n][j]);
                }
            }
        }
        __syncwarp();
        if (lane == 0 && i + S < my_chunks) {
            fence_proxy_async_smem();
            issue(warp + (i + S) * NW, s);
        }
    }

    // ---- a head's row sums over its lanes, then the warps merged through shared memory (each
    //      warp reuses its own stages: all of its copies have landed)
    float *mine = reinterpret_cast<float *>(my_stages);  // [heads][D + 4]
    __syncwarp();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], o);
            float *row = mine + (8 * n + 2 * mt + e) * (D + 4);
#pragma unroll
            for (int j = 0; j < NG; ++j) {
                float z = zacc[n][j][e];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
                const float w = ones[n][j][e];
                *reinterpret_cast<float4 *>(row + 32 * j + 4 * mg) =
                    make_float4(fmaf(oacc[n][j][0][e] - w, 0.25f, z), fmaf(oacc[n][j][0][2 + e] - w, 1.f / 64.f, z),
                                fmaf(oacc[n][j][1][e] - w, 0.25f, z), fmaf(oacc[n][j][1][2 + e] - w, 1.f / 64.f, z));
            }
            if (mg == 0) {
                row[D] = aborted ? -INFINITY : m[n][e];
                row[D + 1] = aborted ? 0.f : l[n][e];
            }
        }
    }
    __syncthreads();
    const bool single = nparts == 1;
    for (int idx = threadIdx.x; idx < nheads * D; idx += blockDim.x) {
        const int h = idx / D, j = idx - h * D;
        float mw[NW], mmax = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            mw[w] = reinterpret_cast<const float *>(stages + w * S * G::kStageBytes)[h * (D + 4) + D];
            mmax = fmaxf(mmax, mw[w]);
        }
        float lsum = 0.f, osum = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float *src = reinterpret_cast<const float *>(stages + w * S * G::kStageBytes) + h * (D + 4);
            if (mw[w] == -INFINITY) continue;
            const float wgt = fast_exp2(mw[w] - mmax);
            lsum += wgt * src[D + 1];
            osum += wgt * src[j];
        }
        const int64_t row = static_cast<int64_t>(seq) * p.num_q_heads + hq0 + h;
        if (single) {
            static_cast<T *>(p.out)[row * D + j] = Elem<T>::from_f32(lsum > 0.f ? osum / lsum : 0.f);
        } else {
            const int64_t pr = row * p.num_partitions + part;
            p.ws_o[pr * D + j] = osum;
            if (j == 0) {
                p.ws_m[pr] = mmax;
                p.ws_l[pr] = lsum;
            }
        }
    }
}

}  // namespace pkv
