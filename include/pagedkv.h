/*
 * pagedkv.h -- C ABI of libpagedkv, a GB300 (sm_103a) library for the decode
 * hot path of paged KV-cache attention.
 *
 * Pages the operations follow (title and section):
 *   P1 = "KV Cache与PagedAttention深度解析：vLLM内存管理革命" (iopencloud.com)
 *   P2 = "KV Cache从原理到实战：大模型推理内存管理演进与优化" (xnwp.cn/news/16711)
 *   P3 = PagedAttention + prefix caching via nano-vllm (zwxr.cn/news/317362)
 *   P4 = "大模型 (LLM) 推理加速核心技术解析：从 KV Cache 到 PagedAttention 实战"
 *        (jsqmd.com/news/745991)
 *
 * Conventions shared by every call
 * --------------------------------
 * Layout.  The KV pool is [num_blocks][2][num_kv_heads][block_size][head_dim]
 *   (P1 §4.3 and §5.1, with num_kv_heads for grouped-query models, P2 §5.3).
 *   Calls take the K half and the V half as two base pointers plus the stride,
 *   in elements, between consecutive physical blocks: for the packed pool
 *   k_cache = pool, v_cache = pool + num_kv_heads*block_size*head_dim and
 *   block_stride_elems = 2*num_kv_heads*block_size*head_dim.  Within a block,
 *   row (h, offset) of K starts at k_cache + blk*block_stride_elems +
 *   (h*block_size + offset)*head_dim.
 * Slots.  Slot s names block s / block_size, offset s % block_size (P1 §5.3).
 * Heads.  Query head hq reads KV head hq / (num_q_heads / num_kv_heads).
 * Types.  dtype is fp16 or bf16 for q, K, V and out; accumulation is fp32.
 *   head_dim is 64 or 128; block_size is 8, 16 or 32.  Others: PKV_ERR_UNSUPPORTED.
 * Memory.  Every pointer argument is a DEVICE pointer owned by the caller,
 *   except where a call says HOST (pkv_slot_mapping_host, the outputs of
 *   pkv_get_device_error and the block manager's arrays).  Tensor base
 *   pointers must be 16-byte aligned and block strides a multiple of 8
 *   elements.  No call allocates memory; the library's only state is one
 *   device status word per device (see pkv_get_device_error), the fixed
 *   scratch array of pkv_paged_attention_decode_static_scratch, and cached
 *   device attributes.
 * Streams.  `stream` is a cudaStream_t (NULL = legacy default stream).  Every
 *   call only enqueues work on it and returns; results are ready when the
 *   stream reaches that point.
 * Errors.  Arguments that can be checked on the host are checked before any
 *   launch: PKV_ERR_INVALID_ARG (nothing enqueued).  Values that live in device
 *   memory (slots, block-table entries, context lengths, copy pairs) are
 *   checked by the kernels: a bad value is skipped, never dereferenced, and
 *   raises a flag in the device status word.  A failed launch returns
 *   PKV_ERR_CUDA.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

typedef enum pkv_status {
    PKV_OK = 0,
    PKV_ERR_INVALID_ARG = 1,   /* host-checkable argument out of contract      */
    PKV_ERR_UNSUPPORTED = 2,   /* valid but not built (dtype, head_dim, bs)    */
    PKV_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed         */
    PKV_ERR_DEVICE = 4,        /* pkv_get_device_error found flags raised      */
    PKV_ERR_SCRATCH_LIMIT = 5, /* split-context scratch needed exceeds
                                  PKV_STATIC_SCRATCH_BYTES (static-scratch decode) */
    PKV_ERR_OUT_OF_BLOCKS = 6  /* block manager: the free pool cannot cover the request */
} pkv_status;

/* PKV_INT8 names an INT8 cache, PKV_INT4 a 4-bit one; only pkv_copy_blocks takes
 * PKV_INT4 as `dtype`, and it, pkv_evict_compact and pkv_tree_commit PKV_INT8 (3 is no type; the entry points of
 * these caches below take the query / new-row dtype, fp16 or bf16). */
typedef enum pkv_dtype { PKV_F16 = 0, PKV_BF16 = 1, PKV_INT8 = 2, PKV_INT4 = 4 } pkv_dtype;

/* Flags of the device status word (bitwise OR of what the kernels saw). */
#define PKV_DEVERR_SLOT        0x1u  /* slot_mapping entry >= num_blocks*block_size  */
#define PKV_DEVERR_BLOCK_TABLE 0x2u  /* block_tables entry outside [0, num_blocks)    */
#define PKV_DEVERR_CONTEXT_LEN 0x4u  /* context_lens entry < 0, > max_context_len or
                                        > max_blocks_per_seq*block_size (clamped)      */
#define PKV_DEVERR_COPY_PAIR   0x8u  /* copy pair entry outside [0, num_blocks)       */
#define PKV_DEVERR_TIMEOUT     0x10u /* a bounded wait on an async copy gave up       */
#define PKV_DEVERR_ROPE_AXIS   0x20u /* axis_of_pair entry outside [0, num_axes)      */
#define PKV_DEVERR_KEPT        0x40u /* kept position outside the context, or (in place) below its rank */

/*
 * pkv_reshape_and_cache -- write each new token's K and V rows into its slot.
 * (P1 §2.2: compute only K_t, V_t and append them; P1 §5.3: the write goes to
 * offset t % block_size of the sequence's last block.)
 *
 *   k_new, v_new   [num_tokens][num_kv_heads][head_dim], contiguous, dtype.
 *   slot_mapping   [num_tokens] int64; slot < 0 means "skip this token"
 *                  (padding); slot >= num_blocks*block_size raises
 *                  PKV_DEVERR_SLOT and the token is skipped.  Two tokens must
 *                  not share a slot (the result would be either row).
 *   k_cache/v_cache, num_blocks, block_stride_elems: the pool, as above.
 * The copy is bit-exact.  num_tokens == 0 is a no-op.
 */
PKV_API pkv_status pkv_reshape_and_cache(const void *k_new, const void *v_new,
                                         const int64_t *slot_mapping, int64_t num_tokens,
                                         void *k_cache, void *v_cache, int64_t num_blocks,
                                         int64_t block_stride_elems, int num_kv_heads,
                                         int head_dim, int block_size, pkv_dtype dtype,
                                         void *stream);

/*
 * pkv_slot_mapping -- the slot each new token's K/V rows are written to, i.e.
 * the slot_mapping input of pkv_reshape_and_cache (P1 §5.3: logical position t
 * of a sequence lies in its table entry t / block_size at offset
 * t % block_size; the flat slot is entry * block_size + offset; P1 §4.2's worked
 * table [7, 2, 9, 1, 5, 8, 3] puts position 99 in slot 3*16 + 3).
 *
 *   block_tables   [num_table_rows][max_blocks_per_seq] int32, device.
 *   token_rows     [num_tokens] int64, device: the table row of each token's
 *                  sequence; NULL means token i uses row i (then
 *                  num_table_rows >= num_tokens).
 *   positions      [num_tokens] int64, device: each token's logical position;
 *                  a negative position is padding and gets slot -1.
 *   num_blocks     pool size, for the range check of table entries.
 *   slot_mapping   [num_tokens] int64, device output.
 * A position past the table (>= max_blocks_per_seq * block_size) or a token row
 * outside the table raises PKV_DEVERR_SLOT, a table entry outside
 * [0, num_blocks) raises PKV_DEVERR_BLOCK_TABLE; such a token gets slot -1.
 * Enqueued on `stream`; num_tokens == 0 is a no-op.
 */
PKV_API pkv_status pkv_slot_mapping(const int32_t *block_tables, int64_t num_table_rows,
                                    int max_blocks_per_seq, const int64_t *token_rows,
                                    const int64_t *positions, int64_t num_tokens, int block_size,
                                    int64_t num_blocks, int64_t *slot_mapping, void *stream);

/*
 * pkv_slot_mapping_host -- pkv_slot_mapping on HOST arrays, computed on the
 * calling thread (no CUDA call), for callers that keep their block tables in
 * host memory.  Same rule and outputs; instead of device flags it returns
 * PKV_ERR_INVALID_ARG when any token had a bad position, row or table entry
 * (every slot is still written, those tokens' as -1).
 */
PKV_API pkv_status pkv_slot_mapping_host(const int32_t *block_tables, int64_t num_table_rows,
                                         int max_blocks_per_seq, const int64_t *token_rows,
                                         const int64_t *positions, int64_t num_tokens,
                                         int block_size, int64_t num_blocks,
                                         int64_t *slot_mapping);

/*
 * pkv_decode_workspace_bytes -- device scratch that pkv_paged_attention_decode
 * needs for a split-context (partitioned) call: fp32 partial outputs plus the
 * running maximum and sum of every (sequence, query head, partition).
 * partition_size 0 means "the library's choice" and returns the size for the
 * partition count that choice gives on the current device.  Returns 0 when
 * no split is needed and (size_t)-1 for arguments out of contract.
 */
PKV_API size_t pkv_decode_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                          int head_dim, int block_size, int max_context_len,
                                          int partition_size);

/*
 * pkv_paged_attention_decode -- one query token per sequence attends over its
 * paged KV cache:  out[i, hq] = softmax(scale * q[i, hq] . K_i^T) V_i
 * (P1 §2.1), where K_i, V_i are the first context_lens[i] tokens of sequence i
 * reached through block_tables[i] (P1 §4.2-4.3), accumulated with the running
 * maximum / running sum rescaling of P1 §7.2 in fp32.
 *
 *   q             [num_seqs][num_q_heads][head_dim], contiguous, dtype.
 *   block_tables  [num_seqs][max_blocks_per_seq] int32, physical block ids.
 *   context_lens  [num_seqs] int32, tokens to attend over (the new token
 *                 included); 0 gives a zero output row.
 *   max_context_len  host-side upper bound of context_lens (sizes the grid; a
 *                 larger device value raises PKV_DEVERR_CONTEXT_LEN and is
 *                 clamped).
 *   scale         softmax scale, normally 1/sqrt(head_dim).
 *   out           [num_seqs][num_q_heads][head_dim], contiguous, dtype; each
 *                 value rounded once (to nearest even) from fp32.
 *   workspace     device scratch of workspace_bytes (>= the value of
 *                 pkv_decode_workspace_bytes for the same arguments); may be
 *                 NULL when that value is 0.  Contents need no initialisation.
 *   partition_size  tokens per split-context partition, a multiple of
 *                 block_size; 0 = library's choice.  Each (sequence, KV head,
 *                 partition) is processed independently and merged by a second
 *                 kernel (log-sum-exp merge) when a sequence spans >1 partition.
 * The reduction order depends only on logical positions, so the result is
 * bitwise independent of where blocks sit in the pool.
 */
PKV_API pkv_status pkv_paged_attention_decode(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float scale, void *out, void *workspace,
    size_t workspace_bytes, int partition_size, pkv_dtype dtype, void *stream);

/*
 * pkv_copy_blocks -- copy-on-write block copies (P1 §8.3; P3 §2.3 and §5.5).
 * For each pair p, the K half and the V half of block src_dst_pairs[2p] are
 * copied bit-exactly over those of block src_dst_pairs[2p+1].  dtype is the
 * cache's: PKV_F16, PKV_BF16, PKV_INT8 or PKV_INT4 (whose block_stride_elems counts
 * bytes).
 *
 *   src_dst_pairs  [num_pairs][2] int64, device.  Destinations must be
 *                  distinct and must not also appear as sources (otherwise the
 *                  result depends on the order the GPU runs the copies).  An
 *                  entry outside [0, num_blocks) raises PKV_DEVERR_COPY_PAIR
 *                  and that pair is skipped.
 * num_pairs == 0 is a no-op.
 */
PKV_API pkv_status pkv_copy_blocks(void *k_cache, void *v_cache, int64_t num_blocks,
                                   int64_t block_stride_elems, int num_kv_heads, int head_dim,
                                   int block_size, const int64_t *src_dst_pairs,
                                   int64_t num_pairs, pkv_dtype dtype, void *stream);

/* ------------------------------------------------------------------------
 * INT8 KV cache with per-channel scales (P2 §5.2: storing the cache in INT8
 * halves its bytes, and with it the bytes a decode step reads; per-channel
 * scales, computed separately for K and V, are the variant that page
 * recommends).  The pool keeps the layout above with one signed byte per
 * element: [num_blocks][2][num_kv_heads][block_size][head_dim] int8, block
 * strides and offsets counted in elements (= bytes) and a multiple of 16.
 * Scales are caller-owned device arrays k_scale, v_scale of
 * [num_kv_heads][head_dim] fp32, each > 0 and finite (calibrated offline;
 * the library never changes them), 16-byte aligned.
 * A value x (fp16 / bf16) of KV head h, channel c is stored as
 *     code = round_half_even(clamp(x / s[h][c], -127, 127))
 * with the division in IEEE single precision (a NaN input stores -127), and
 * read back as code * s[h][c].
 * ------------------------------------------------------------------------ */

/*
 * pkv_reshape_and_cache_int8 -- pkv_reshape_and_cache into an INT8 cache:
 * each element of the new rows k_new / v_new ([num_tokens][num_kv_heads]
 * [head_dim], dtype = fp16 or bf16) is quantised with its channel's scale and
 * stored at its slot.  Slot rules and errors as pkv_reshape_and_cache.
 */
PKV_API pkv_status pkv_reshape_and_cache_int8(const void *k_new, const void *v_new,
                                              const int64_t *slot_mapping, int64_t num_tokens,
                                              int8_t *k_cache, int8_t *v_cache, int64_t num_blocks,
                                              int64_t block_stride_elems, int num_kv_heads,
                                              int head_dim, int block_size, const float *k_scale,
                                              const float *v_scale, pkv_dtype dtype, void *stream);

/* Workspace of pkv_paged_attention_decode_int8 (same contract as
 * pkv_decode_workspace_bytes). */
PKV_API size_t pkv_decode_int8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                               int head_dim, int block_size, int max_context_len,
                                               int partition_size);

/*
 * pkv_paged_attention_decode_int8 -- pkv_paged_attention_decode over an INT8
 * cache: the same softmax attention with K_i[t][c] = code * k_scale[h][c] and
 * V_i[t][c] = code * v_scale[h][c].  q and out are `dtype` (fp16 or bf16);
 * accumulation is fp32.  The K scales are folded into the query and the V
 * scales applied once per output channel, so the kernel reads only the codes.
 * Every other argument and the errors are those of pkv_paged_attention_decode;
 * the automatic split is pkv_decode_int8_plan's.
 */
PKV_API pkv_status pkv_paged_attention_decode_int8(
    const void *q, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale,
    const float *v_scale, int64_t num_blocks, int64_t block_stride_elems,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, void *out, void *workspace, size_t workspace_bytes,
    int partition_size, pkv_dtype dtype, void *stream);

/* ------------------------------------------------------------------------
 * 4-bit KV cache with scales of its own: every row carries them, so nothing is
 * calibrated.  The 32 channels of group j of one token and KV head are stored as
 *     zero z  = their smallest value (exact in the rows' type),
 *     scale s = (largest - smallest) / 15, rounded up to the rows' type,
 *     codes c = the integer nearest to (x - z) / s (x - z in fp32), ties to even, 0 when s = 0,
 * and read back as s * c + z: a value is off by s / 2 at most.  Values must be
 * finite (a NaN gets code 0, a group with an infinity reads back as NaN); one past the
 * type's range, as the rounded-up scale can make of the largest code, counts as its largest
 * finite value, when it is read back and in the decode's outputs.
 * The pool is bytes, [num_blocks][2][num_kv_heads][block_size * head_dim * 5 / 8]:
 * a head's record of a block holds the codes of its tokens, head_dim / 2 bytes
 * each, then head_dim / 32 (scale, zero) pairs for each of its tokens.  With
 * NG = head_dim / 32, channel 32 j + 4 u + e of a token is nibble e (low first) of
 * its 16-bit word u * NG + j.  Block strides count bytes, a multiple of 16.
 * dtype is the rows' type, fp16 or bf16, the same in every call on a pool.
 * ------------------------------------------------------------------------ */

/*
 * pkv_reshape_and_cache_int4 -- pkv_reshape_and_cache into a 4-bit cache: the rows
 * k_new, v_new ([num_tokens][num_kv_heads][head_dim], dtype) quantised as above
 * and stored at their slots.  Slot rules and errors as pkv_reshape_and_cache (two
 * tokens that share a slot may leave codes of one and scales of the other);
 * num_kv_heads <= 65535, num_tokens * num_kv_heads <= 2^31 - 256.
 */
PKV_API pkv_status pkv_reshape_and_cache_int4(const void *k_new, const void *v_new,
                                              const int64_t *slot_mapping, int64_t num_tokens,
                                              void *k_cache, void *v_cache, int64_t num_blocks,
                                              int64_t block_stride_bytes, int num_kv_heads,
                                              int head_dim, int block_size, pkv_dtype dtype,
                                              void *stream);

/*
 * pkv_dequantise_blocks_int4 -- read blocks back: for each pair p, block
 * src_dst_pairs[2p] of the 4-bit pool is written as 16-bit values (s * c + z, one
 * rounding) over block src_dst_pairs[2p+1] of a 16-bit pool of the same shape, e.g.
 * for a chunked prefill behind a cached context.  Every row of the block is read,
 * unwritten ones included.
 *   src_dst_pairs  [num_pairs][2] int64, device; destinations must be distinct.  An
 *                  entry outside its pool raises PKV_DEVERR_COPY_PAIR and its pair
 *                  is skipped.
 */
PKV_API pkv_status pkv_dequantise_blocks_int4(const void *k_cache4, const void *v_cache4,
                                              int64_t num_blocks4, int64_t block_stride_bytes4,
                                              const int64_t *src_dst_pairs, int64_t num_pairs,
                                              void *k_cache, void *v_cache, int64_t num_blocks,
                                              int64_t block_stride_elems, int num_kv_heads,
                                              int head_dim, int block_size, pkv_dtype dtype,
                                              void *stream);

/* Workspace of pkv_paged_attention_decode_int4 on the current device: it depends on its
 * SMs, the head counts and head_dim ((size_t)-1 for arguments out of contract). */
PKV_API size_t pkv_decode_int4_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                               int head_dim, int block_size, int max_context_len);

/*
 * pkv_paged_attention_decode_int4 -- pkv_paged_attention_decode over a 4-bit cache.
 * The contexts' work is cut evenly on the device, whatever their lengths, so there is
 * no partition size; workspace >= pkv_decode_int4_workspace_bytes(...) is always
 * needed, and calls that may overlap need one each.  Tokens past a context, in its last
 * block, may hold anything.  A query is held to 2^-24 of its largest channel.  Each
 * group of a V row is as exact as if all had its scale, down to 2^-90 of the row's largest (rows
 * whose scales lie 2^8 or more apart, 0 among them, take up to twice the time).  Other arguments and errors as
 * pkv_paged_attention_decode; the result depends on the batch's lengths within the
 * roundings (they decide where a context is cut), not on the blocks' places.
 */
PKV_API pkv_status pkv_paged_attention_decode_int4(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_bytes, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float scale, void *out, void *workspace,
    size_t workspace_bytes, pkv_dtype dtype, void *stream);

/*
 * pkv_shared_prefix_workspace_bytes -- workspace of
 * pkv_paged_attention_decode_shared_prefix for these arguments on the current
 * device ((size_t)-1 if they are out of contract).
 */
PKV_API size_t pkv_shared_prefix_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                                 int head_dim, int block_size, int prefix_len,
                                                 int max_context_len, int partition_size);

/*
 * pkv_paged_attention_decode_shared_prefix -- the same result as
 * pkv_paged_attention_decode for a batch whose sequences all start with the
 * same prefix_len tokens held in the blocks prefix_block_table[0 ..
 * prefix_len/block_size) (prefix caching: P1 §8.2, P3 §2.3 / §3), computed as
 * a cascade: (1) all num_seqs * G query rows of each KV head attend to the
 * prefix together as dense tensor-core tiles, so each prefix block is read once
 * per 128 query rows instead of once per sequence; (2) each sequence attends
 * to its own tokens [prefix_len, context_len); (3) a log-sum-exp merge.
 *
 *   prefix_block_table  [prefix_len / block_size] int32, device.
 *   prefix_len          > 0, a multiple of block_size, <= max_context_len.
 *                       Every context_lens[i] must be >= prefix_len (a shorter
 *                       one raises PKV_DEVERR_CONTEXT_LEN), and every
 *                       block_tables[i] must start with the prefix's blocks
 *                       (or blocks holding the same data).
 *   workspace           >= pkv_shared_prefix_workspace_bytes(...); required.
 * Other arguments as pkv_paged_attention_decode.  head_dim 128 only (else
 * PKV_ERR_UNSUPPORTED).
 */
PKV_API pkv_status pkv_paged_attention_decode_shared_prefix(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *prefix_block_table, int prefix_len,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, void *out, void *workspace, size_t workspace_bytes,
    int partition_size, pkv_dtype dtype, void *stream);

/* ------------------------------------------------------------------------
 * Operators that a model's layers run around plain attention.  The pages have
 * no counterpart for them: rotary positions, score forms and masks belong to
 * the model, and eviction bounds a context that the pages let grow.
 *
 * Token t and position p of a score (distance bias, window, starts,
 * prefix_lens) are rows of the cached context.  After
 * pkv_evict_compact they are no longer the tokens' positions: the kept tokens
 * have moved together, each KV head its own.  A distance bias then measures the
 * shortened distance, a window counts kept tokens, and starts and prefix_lens
 * have to be given anew.  Rotary positions are not affected: K is stored
 * rotated by the position that the caller gave, and the next token's is still
 * the caller's to count.
 * ------------------------------------------------------------------------ */

/*
 * pkv_rope_reshape_and_cache -- rotary positions with one to four axes on the
 * queries and the new keys, and the cache write: q_out gets the rotated
 * queries, the slot of each token its rotated K row and its V row.  For token
 * n, pair i = 0 .. rotary_dim/2 - 1 of a head's channels turns by
 *     angle = positions[axis_of_pair[i]][n] * inv_freq[i]:
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * where pair i is channels (i, i + rotary_dim/2), or (2i, 2i + 1) with
 * interleaved != 0; the channels from rotary_dim on are copied.  Several axes
 * serve tokens with several positions (time, height and width of a video's
 * patches); axis_of_pair may assign them in sections or in turn.
 *
 *   q, k_new, v_new   rows of [num_tokens] tokens, [heads][head_dim] dense
 *                  within a token and q_stride / k_stride / v_stride elements
 *                  from token to token (multiples of 8, at least a row): the
 *                  parts of a fused projection's output are taken in place.
 *   positions      [num_axes][num_tokens] int64, device; any value (negative
 *                  ones turn backwards).
 *   axis_of_pair   [rotary_dim/2] int32, device; NULL: axis 0 for every pair.
 *                  An entry outside [0, num_axes) raises PKV_DEVERR_ROPE_AXIS
 *                  and leaves its pair unrotated.
 *   inv_freq       [rotary_dim/2] double, device: radians per position.
 *   rotary_dim     a multiple of 16 up to head_dim (else PKV_ERR_UNSUPPORTED
 *                  / PKV_ERR_INVALID_ARG).
 *   slot_mapping   as pkv_reshape_and_cache; a token whose slot is negative or
 *                  out of range writes no cache row, its q_out row is written.
 *   q_out          q_out_stride elements from token to token; may be q itself
 *                  (same pointer and stride), else must not overlap the inputs.
 * The angle is reduced modulo one turn in 64-bit integers, so positions in
 * the millions keep their angles (error |position| * 2^-53 turns); sine,
 * cosine and the rotation are fp32, rounded once to the stored type.
 */
PKV_API pkv_status pkv_rope_reshape_and_cache(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
    int64_t v_stride, const int64_t *positions, int num_axes, const int32_t *axis_of_pair,
    const double *inv_freq, int rotary_dim, int interleaved, const int64_t *slot_mapping,
    int64_t num_tokens, void *q_out, int64_t q_out_stride, void *k_cache, void *v_cache,
    int64_t num_blocks, int64_t block_stride_elems, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, pkv_dtype dtype, void *stream);

/* pkv_rope_reshape_and_cache into an INT8 cache: the rotated K row (fp32) and
 * the V row are quantised as by pkv_reshape_and_cache_int8. */
PKV_API pkv_status pkv_rope_reshape_and_cache_int8(
    const void *q, int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
    int64_t v_stride, const int64_t *positions, int num_axes, const int32_t *axis_of_pair,
    const double *inv_freq, int rotary_dim, int interleaved, const int64_t *slot_mapping,
    int64_t num_tokens, void *q_out, int64_t q_out_stride, int8_t *k_cache, int8_t *v_cache,
    int64_t num_blocks, int64_t block_stride_elems, int num_q_heads, int num_kv_heads,
    int head_dim, int block_size, const float *k_scale, const float *v_scale, pkv_dtype dtype,
    void *stream);

/*
 * pkv_decode_scored_workspace_bytes -- workspace of
 * pkv_paged_attention_decode_scored (int8_cache 0) or its INT8-cache form for
 * these arguments on the current device; want_weights != 0 when weights_out is
 * given.  0 when none is needed, (size_t)-1 for arguments out of contract.
 */
PKV_API size_t pkv_decode_scored_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                                 int head_dim, int block_size, int max_context_len,
                                                 int window, int want_weights, int int8_cache,
                                                 int partition_size);

/*
 * pkv_paged_attention_decode_scored -- pkv_paged_attention_decode with the
 * score forms and masks of a model's layers, and the attention weights for
 * eviction.  The query of sequence i sits at position p = context_lens[i] - 1;
 * head hq's score of token t is
 *     x = scale * q . k_t;   x = softcap * tanh(x / softcap)   (softcap > 0);
 *     x = x + slopes[hq] * (t - p)                             (slopes given)
 * and the softmax runs over the tokens lo <= t <= p with
 *     lo = max(0, p + 1 - window  (window > 0),  starts[i]  (starts given)).
 *
 *   softcap        0 (none) or in [1e-3, 1e6].
 *   slopes         [num_q_heads] fp32, finite, device, or NULL.
 *   window         0: the whole context.
 *   starts         [num_seqs] int32, device, or NULL: the first visible token,
 *                  e.g. of the sequence's last document.  A sequence that sees
 *                  nothing (starts[i] >= context_lens[i]) gets a zero row.
 *   weights, weights_out   fp32 [num_seqs][num_kv_heads][weights_stride],
 *                  device: for every token t of the context
 *                      weights_out[i][h][t] = weights[i][h][t] + sum over KV
 *                      head h's query heads of their softmax weight of t
 *                  (weights NULL: plus nothing); columns past the context are
 *                  left as they are.  The same array may be both; else they
 *                  must not overlap.  weights_stride >= max_context_len.
 *                  weights_out NULL: not wanted.  At most 128 query heads per
 *                  KV head (else PKV_ERR_UNSUPPORTED).
 *   workspace      >= pkv_decode_scored_workspace_bytes(...).  With weights_out
 *                  it holds every score in fp32, for each sequence as many as
 *                  the bound allows: 4 * num_seqs * num_q_heads * (the smaller
 *                  of max_context_len and window + block_size - 1) bytes and a
 *                  few per cent (256 sequences of 64 heads bounded by 131072
 *                  tokens: 8.6 GB), however short the contexts are.
 * Tokens before lo are not read: table entries of blocks that lie before lo
 * are never dereferenced (a window's past blocks may be freed), and what lo's
 * block holds before it does not matter, NaN or infinities included.  Other
 * arguments and errors as pkv_paged_attention_decode.
 */
PKV_API pkv_status pkv_paged_attention_decode_scored(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float scale, float softcap,
    const float *slopes, int window, const int32_t *starts, const float *weights,
    float *weights_out, int64_t weights_stride, void *out, void *workspace,
    size_t workspace_bytes, int partition_size, pkv_dtype dtype, void *stream);

/* pkv_paged_attention_decode_scored over an INT8 cache (the score forms and
 * masks; no weights: its scores carry the fp16 rounding of the folded query). */
PKV_API pkv_status pkv_paged_attention_decode_scored_int8(
    const void *q, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale,
    const float *v_scale, int64_t num_blocks, int64_t block_stride_elems,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, float softcap, const float *slopes, int window,
    const int32_t *starts, void *out, void *workspace, size_t workspace_bytes,
    int partition_size, pkv_dtype dtype, void *stream);

/* ------------------------------------------------------------------------
 * A sliding window with a few first tokens that stay visible (attention sinks): a
 * query at position p sees the tokens t <= p with
 *     t < sinks   or   t > p - window        (window >= 1, sinks >= 0).
 * Blocks that lie wholly between the first tokens and the window are not read and
 * their table entries are never dereferenced, so a caller who places blocks itself may
 * give them to others, and an endless stream then needs a bounded number of blocks
 * (its table still has an entry per block of the whole stream).  pkv_bm_* gives back whole
 * sequences and tails only.  What the remaining rows between hold does not matter
 * for the decode (NaN and infinities included).
 * ------------------------------------------------------------------------ */

/* Workspace of pkv_paged_attention_decode_sinks (int8_cache 0) or its INT8-cache
 * form; the contract of pkv_decode_scored_workspace_bytes. */
PKV_API size_t pkv_decode_sinks_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads,
                                                int head_dim, int block_size, int max_context_len,
                                                int window, int sinks, int int8_cache,
                                                int partition_size);

/* pkv_paged_attention_decode_sinks -- pkv_paged_attention_decode with that mask: the
 * query of sequence i sits at position context_lens[i] - 1.  Other arguments and
 * errors as pkv_paged_attention_decode. */
PKV_API pkv_status pkv_paged_attention_decode_sinks(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float scale, int window, int sinks, void *out,
    void *workspace, size_t workspace_bytes, int partition_size, pkv_dtype dtype, void *stream);

/* pkv_paged_attention_decode_sinks over an INT8 cache (pkv_paged_attention_decode_int8). */
PKV_API pkv_status pkv_paged_attention_decode_sinks_int8(
    const void *q, const int8_t *k_cache, const int8_t *v_cache, const float *k_scale,
    const float *v_scale, int64_t num_blocks, int64_t block_stride_elems,
    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, int window, int sinks, void *out, void *workspace,
    size_t workspace_bytes, int partition_size, pkv_dtype dtype, void *stream);

/* Workspace of pkv_paged_attention_prefill_sinks; the contract of
 * pkv_prefill_scored_workspace_bytes. */
PKV_API size_t pkv_prefill_sinks_workspace_bytes(int num_rows, int num_seqs, int num_q_heads,
                                                 int num_kv_heads, int head_dim, int block_size,
                                                 int max_query_len, int max_context_len, int window,
                                                 int sinks, int kv_splits);

/* pkv_paged_attention_prefill_sinks -- pkv_paged_attention_prefill with that mask, each
 * chunk row at its own position.  The V rows that some of a row tile's rows see and
 * others do not must be finite.  workspace >= pkv_prefill_sinks_workspace_bytes(...).
 * Other arguments and errors as pkv_paged_attention_prefill. */
PKV_API pkv_status pkv_paged_attention_prefill_sinks(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, int window, int sinks, void *out, void *workspace,
    size_t workspace_bytes, int kv_splits, pkv_dtype dtype, void *stream);

/* ------------------------------------------------------------------------
 * A tree of drafted tokens (speculative decoding): the drafted tokens of a sequence
 * are its chunk, written behind its context like any chunk; the verification's
 * attention lets each see the context and its own ancestors, and the path that is
 * accepted is then moved together.
 * ------------------------------------------------------------------------ */

/* Workspace of pkv_paged_attention_tree on the current device: it depends on its SMs
 * alone ((size_t)-1 without a device). */
PKV_API size_t pkv_tree_workspace_bytes(void);

/*
 * pkv_paged_attention_tree -- attention of the chunk rows of pkv_paged_attention_prefill
 * with a mask of their own: row j of sequence i's chunk (C tokens behind L - C context
 * tokens) sees every token t < L - C, and chunk token c where bit c is set in the
 * row's words of tree_mask (c < C; bit c % 64 of word c / 64).  A row usually sees
 * itself and its ancestors, but any bits will do; a row that sees nothing gets zeros.
 *
 *   tree_mask     [num_rows][mask_words] int64, device; 64 * mask_words >=
 *                 max_query_len.
 *   workspace     >= pkv_tree_workspace_bytes(); calls that may overlap need one
 *                 each.  Contents need no initialisation.
 * Every chunk token's V row must be finite.  All other arguments and errors as
 * pkv_paged_attention_prefill (head_dim 128, up to 128 query heads per KV head).
 */
PKV_API pkv_status pkv_paged_attention_tree(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, const int64_t *tree_mask,
    int mask_words, int num_rows, int max_query_len, int max_context_len, int num_seqs,
    int num_q_heads, int num_kv_heads, int head_dim, int block_size, float scale, void *out,
    void *workspace, size_t workspace_bytes, pkv_dtype dtype, void *stream);

/*
 * pkv_tree_commit -- keep the accepted path of each sequence's drafted tokens: with
 * base = L - C, the K and V rows of chunk token accepted[i][j] move to position
 * base + j, for j < accepted_lens[i] (bit-exact, in place).  Afterwards the context
 * is base + accepted_lens[i] tokens long, and the blocks past it can be freed
 * (pkv_bm_truncate).  dtype is the cache's: PKV_F16, PKV_BF16 or PKV_INT8.
 *
 *   accepted       [num_seqs][max_accepted] int32, device: chunk tokens in ascending
 *                  order.  One that does not ascend or lies outside the chunk raises
 *                  PKV_DEVERR_KEPT and is skipped (the rows behind it are then
 *                  unspecified); a length that does not fit raises it too and counts as 0.
 *   query_start, context_lens, max_query_len, max_context_len   as
 *                  pkv_paged_attention_tree; a sequence out of contract raises
 *                  PKV_DEVERR_CONTEXT_LEN and is left as it is.
 *   new_context_lens   [num_seqs] int32, device, or NULL: the lengths afterwards, of a
 *                  sequence out of contract the length that it came with; must not
 *                  overlap the other index arrays (PKV_ERR_INVALID_ARG).
 * The blocks that get rows must belong to their sequence alone (pkv_bm_make_private).
 */
PKV_API pkv_status pkv_tree_commit(void *k_cache, void *v_cache, int64_t num_blocks,
                                   int64_t block_stride_elems, int num_kv_heads, int head_dim,
                                   int block_size, const int32_t *block_tables,
                                   int max_blocks_per_seq, const int32_t *query_start,
                                   const int32_t *context_lens, int max_query_len,
                                   int max_context_len, int num_seqs, const int32_t *accepted,
                                   const int32_t *accepted_lens, int max_accepted,
                                   int32_t *new_context_lens, pkv_dtype dtype, void *stream);

/*
 * pkv_evict_select -- which tokens of each (sequence, KV head) stay in the
 * cache.  A context of L = context_lens[i] tokens keeps n = min(L, budget):
 * all of them when L <= budget, else the first `sinks`, the last `recent` and
 * the budget - sinks - recent heaviest of those between (equal weights: the
 * lower position; a NaN weight ranks below every number).
 *
 *   weights        [num_seqs][num_kv_heads][weights_stride] fp32, device: the
 *                  weight of each cached token, as
 *                  pkv_paged_attention_decode_scored accumulates it.
 *   context_lens   [num_seqs] int32, device; max_context_len bounds them on
 *                  the host (a value outside raises PKV_DEVERR_CONTEXT_LEN and
 *                  is clamped) and must not exceed weights_stride.
 *   sinks + recent <= budget, 0 < budget <= 2^30, max_context_len <= 2^30.
 *   weights_out    NULL, or a buffer of the same shape that gets the kept
 *                  tokens' weights in their new places [0, n) and zeros in
 *                  [n, L); the rest of a row is left as it is.  May be
 *                  `weights` itself, else must not overlap it.
 *   kept           [num_seqs][num_kv_heads][budget] int32: the kept positions,
 *                  ascending, then -1.
 *   kept_lens      [num_seqs] int32: n, the context lengths after eviction; must
 *                  not overlap context_lens (PKV_ERR_INVALID_ARG).
 */
PKV_API pkv_status pkv_evict_select(const float *weights, int64_t weights_stride,
                                    const int32_t *context_lens, int max_context_len,
                                    int num_seqs, int num_kv_heads, int budget, int sinks,
                                    int recent, float *weights_out, int32_t *kept,
                                    int32_t *kept_lens, void *stream);

/*
 * pkv_evict_compact -- move the K and V rows of the kept tokens to the front of
 * each sequence's context (bit-exact): row kept[i][h][j] of head h becomes row
 * j, for j < kept_lens[i].  dtype is the cache's: PKV_F16, PKV_BF16 or PKV_INT8.
 *
 *   block_tables, context_lens   the contexts before eviction.
 *   kept, kept_lens, budget      as pkv_evict_select writes them.
 *   dst_block_tables  [num_seqs][dst_max_blocks_per_seq] int32, device: fresh
 *                  blocks for the compacted contexts, none of which belongs to
 *                  any of the source contexts; the sources are left as they
 *                  are.  NULL (or block_tables itself) compacts in place: then
 *                  kept must ascend, and every block that gets rows must belong
 *                  to its sequence alone (pkv_bm_make_private).
 * Rows of the destination past kept_lens[i] are left as they are.  A kept
 * position outside its context (or, in place, below its rank) raises
 * PKV_DEVERR_KEPT, a bad table entry PKV_DEVERR_BLOCK_TABLE, and that row is
 * skipped; lengths that do not fit raise PKV_DEVERR_CONTEXT_LEN and skip the
 * sequence.  Afterwards the context lengths are kept_lens, and the blocks past
 * them can be freed (pkv_bm_truncate).
 */
PKV_API pkv_status pkv_evict_compact(void *k_cache, void *v_cache, int64_t num_blocks,
                                     int64_t block_stride_elems, int num_kv_heads, int head_dim,
                                     int block_size, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *context_lens,
                                     int num_seqs, const int32_t *kept, const int32_t *kept_lens,
                                     int budget, const int32_t *dst_block_tables,
                                     int dst_max_blocks_per_seq, pkv_dtype dtype, void *stream);

/*
 * pkv_prefill_workspace_bytes -- workspace of pkv_paged_attention_prefill for
 * these arguments on the current device: 0 when the KV range is not split,
 * (size_t)-1 for arguments out of contract.  kv_splits as in
 * pkv_paged_attention_prefill.
 */
PKV_API size_t pkv_prefill_workspace_bytes(int num_rows, int num_seqs, int num_q_heads,
                                           int num_kv_heads, int head_dim, int block_size,
                                           int max_query_len, int max_context_len, int kv_splits);

/*
 * pkv_paged_attention_prefill -- chunked prefill attention over the paged
 * cache (P4 §2: with a cache, the new tokens' queries attend to the cached
 * tokens and causally to each other; P2 §2.3 / §5.4: a whole prompt, or a long
 * prompt in chunks).  Sequence i has context_lens[i] = L_i tokens in the
 * cache, the last C_i = query_start[i+1] - query_start[i] of which are its
 * chunk (already written, e.g. by pkv_reshape_and_cache with the chunk's
 * slots).  Chunk row j -- global query row query_start[i] + j, at position
 * p = L_i - C_i + j -- attends to tokens 0 .. p (the causal rule on absolute
 * positions):
 *     out[row, hq] = softmax_t<=p(scale * q[row, hq] . k_t) V,
 * accumulated in fp32 on the tensor cores (tcgen05, 128 query rows x 128
 * tokens per tile; the group's heads of each token share the K/V tiles).
 *
 *   q, out         [num_rows][num_q_heads][head_dim], contiguous, dtype; the
 *                  chunks of all sequences back to back.
 *   query_start    [num_seqs + 1] int32, device: non-decreasing chunk offsets,
 *                  query_start[num_seqs] <= num_rows.
 *   context_lens   [num_seqs] int32, device: L_i >= C_i.
 *   max_query_len, max_context_len   host bounds of C_i and L_i (size the grid;
 *                  a sequence outside them, or with query_start out of order,
 *                  raises PKV_DEVERR_CONTEXT_LEN and its rows are not written).
 *   kv_splits      0 = library's choice; n > 0 splits each row tile's KV range
 *                  into about n pieces of whole 128-token tiles, merged by a
 *                  log-sum-exp pass (workspace needed when the plan splits).
 * Other arguments as pkv_paged_attention_decode; head_dim 128 only (else
 * PKV_ERR_UNSUPPORTED).  A chunk of one token per sequence computes the same
 * attention as pkv_paged_attention_decode.
 */
PKV_API pkv_status pkv_paged_attention_prefill(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, void *out, void *workspace, size_t workspace_bytes,
    int kv_splits, pkv_dtype dtype, void *stream);

/*
 * pkv_prefill_scored_workspace_bytes -- workspace of
 * pkv_paged_attention_prefill_scored, as pkv_prefill_workspace_bytes (an item
 * table of 32 bytes per row tile when the KV range is not split);
 * has_prefix != 0 when prefix_lens is given.
 */
PKV_API size_t pkv_prefill_scored_workspace_bytes(int num_rows, int num_seqs, int num_q_heads,
                                                  int num_kv_heads, int head_dim, int block_size,
                                                  int max_query_len, int max_context_len, int window,
                                                  int has_prefix, int kv_splits);

/*
 * pkv_paged_attention_prefill_scored -- pkv_paged_attention_prefill with the
 * score forms of pkv_paged_attention_decode_scored (softcap, slopes) and an
 * interval of visible tokens per row: the chunk row at position p of sequence i
 * attends to the tokens lo <= t < hi with
 *     lo = max(0, p + 1 - window  (window > 0),  starts[row]  (starts given))
 *     hi = max(p + 1, min(context_lens[i], prefix_lens[i])  (prefix_lens given))
 *   starts         [num_rows] int32, device, or NULL: each query row's first
 *                  visible token (the start of its document in a packed
 *                  sequence).  A row with lo >= hi gets zeros.
 *   prefix_lens    [num_seqs] int32, device, or NULL: the first tokens of each
 *                  sequence that every one of its rows sees, also before its
 *                  own position (a prefix mask, e.g. over an image).
 *   workspace      >= pkv_prefill_scored_workspace_bytes(...) when that is > 0.
 * The key range of 128 query rows runs from the smallest lo among them to the
 * largest hi; blocks outside it are not read, so a window's past blocks may be
 * freed.  Inside it, the V rows that some of the 128 rows do not see must be
 * finite.  A bf16 call with 0 < softcap < 52 and no slopes keeps no maximum per
 * row (its scores cannot leave [-softcap, softcap]): there |V| times the tokens
 * that a row sees must stay below 2^78, and where a row's scores all lie near
 * -softcap, values below 2^-26 count with an absolute error of up to 2^-26.
 * Other arguments and errors as pkv_paged_attention_prefill.
 */
PKV_API pkv_status pkv_paged_attention_prefill_scored(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *query_start, const int32_t *context_lens, int num_rows, int max_query_len,
    int max_context_len, int num_seqs, int num_q_heads, int num_kv_heads, int head_dim,
    int block_size, float scale, float softcap, const float *slopes, int window,
    const int32_t *starts, const int32_t *prefix_lens, void *out, void *workspace,
    size_t workspace_bytes, int kv_splits, pkv_dtype dtype, void *stream);

/* Size of the library's built-in decode scratch array (per device). */
#define PKV_STATIC_SCRATCH_BYTES (32u << 20) /* 32 MiB */

/*
 * pkv_paged_attention_decode_static_scratch -- pkv_paged_attention_decode for
 * callers that cannot allocate device memory.  The pages have no counterpart:
 * this is a deployment convenience, not part of the method.
 *
 * Who needs it: a caller that has no device memory to give the decode call
 * its split-context workspace -- e.g. a serving engine that reserved nearly
 * all free device memory for its KV block pool up front, or a plug-in whose
 * host framework hands it tensor pointers but no allocator it may call.
 *
 * Arguments and results are those of pkv_paged_attention_decode without the
 * workspace pair; the scratch comes from a PKV_STATIC_SCRATCH_BYTES array
 * inside the library that every device loading the library keeps until the
 * process exits.  The call allocates nothing (no cudaMalloc/cudaFree, no
 * allocating library routine).
 *   - A plan whose scratch (pkv_decode_workspace_bytes for the same
 *     arguments) exceeds PKV_STATIC_SCRATCH_BYTES is rejected with
 *     PKV_ERR_SCRATCH_LIMIT before anything is enqueued; pass a larger
 *     partition_size (fewer partitions) or use the workspace entry point.
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - All calls on a device share the array, which keeps the last call's
 *     contents.  Nothing in it needs clearing (every value is written before
 *     it is read), but calls that overlap on the GPU -- e.g. on two streams
 *     with no ordering between them -- race on it and must be serialised by
 *     the caller.
 */
PKV_API pkv_status pkv_paged_attention_decode_static_scratch(
    const void *q, const void *k_cache, const void *v_cache, int64_t num_blocks,
    int64_t block_stride_elems, const int32_t *block_tables, int max_blocks_per_seq,
    const int32_t *context_lens, int max_context_len, int num_seqs, int num_q_heads,
    int num_kv_heads, int head_dim, int block_size, float scale, void *out, int partition_size,
    pkv_dtype dtype, void *stream);

/*
 * pkv_get_device_error -- synchronise `stream`, read the current device's
 * status word into *flags (PKV_DEVERR_* bits; may be NULL) and clear it.
 * Returns PKV_OK when no flag was set, PKV_ERR_DEVICE when one was, and
 * PKV_ERR_CUDA if the read failed.
 */
PKV_API pkv_status pkv_get_device_error(void *stream, uint32_t *flags);

/* Static description of a status code. */
PKV_API const char *pkv_status_string(pkv_status status);

/* Kernel launches this process has made through the library (all calls). */
PKV_API uint64_t pkv_launch_count(void);

/*
 * pkv_decode_plan -- the launch decision pkv_paged_attention_decode makes,
 * as a pure host function (no CUDA call): given the shape and the SM count it
 * writes the partition size, partitions per sequence, query heads handled per
 * block and whether the merge kernel runs.  Returns PKV_OK or the status the
 * decode call would return for these arguments.  A block serves the largest
 * of 16 (head_dim 128), 8, 4, 2, 1 query heads dividing the group.  With
 * partition_size 0 the split aims at eight waves of the kernel form's resident
 * blocks per SM (two for the per-lane form and for 16 heads per block, three
 * for the warp-MMA form of 4 or 8 heads per block), with partitions of at
 * least 256 tokens whose K/V bytes are at least 32 times their partial
 * outputs.  For the forms with two resident blocks per SM, when those floors
 * leave fewer than eight waves, the partition count per max_context_len
 * sequence is the smallest in [n/2, n] (n: the floors' count) whose blocks
 * fill whole waves within 0.15 of the best count in that range.
 */
PKV_API pkv_status pkv_decode_plan(int num_seqs, int num_q_heads, int num_kv_heads,
                                   int head_dim, int block_size, int max_context_len,
                                   int partition_size, int sm_count, int *out_partition_size,
                                   int *out_num_partitions, int *out_heads_per_block,
                                   int *out_needs_merge);

/*
 * pkv_decode_int8_plan -- pkv_decode_plan for pkv_paged_attention_decode_int8
 * (the same rules, with at most 8 heads per block; the INT8 forms keep six
 * (per-lane) or four (warp MMAs) blocks resident per SM, and a token's K/V is
 * half the bytes).
 */
PKV_API pkv_status pkv_decode_int8_plan(int num_seqs, int num_q_heads, int num_kv_heads,
                                        int head_dim, int block_size, int max_context_len,
                                        int partition_size, int sm_count, int *out_partition_size,
                                        int *out_num_partitions, int *out_heads_per_block,
                                        int *out_needs_merge);

/*
 * pkv_debug_wait_timeout -- failure-detection self test.  Launches one block
 * that waits, with the library's bounded wait, on an mbarrier that nothing
 * completes; after timeout_ns nanoseconds the wait gives up, raises
 * PKV_DEVERR_TIMEOUT in the status word and the kernel returns normally.
 * timeout_ns must be in (0, 10^10].
 */
PKV_API pkv_status pkv_debug_wait_timeout(uint64_t timeout_ns, void *stream);

/* ------------------------------------------------------------------------
 * Host block manager (no GPU involved): the bookkeeping that produces the
 * inputs of the calls above -- block tables, context lengths, slot mappings
 * and copy-on-write pairs.  P1 §5.2-5.3: a free pool of physical blocks; when
 * token t is appended the sequence needs ceil((t+1)/block_size) blocks, a new
 * block comes from the pool when its table is short, and the token's slot is
 * offset t % block_size of the last block.  P1 §6.2 / §8.2-8.3: finished
 * sequences return their blocks; shared blocks carry a reference count and are
 * freed at zero.  P3 §2.3 / §5.5: a sequence about to write into a block that
 * another sequence references first gets a private copy (a copy-on-write pair
 * for pkv_copy_blocks).  Blocks are handed out 0, 1, 2, ... from a fresh pool
 * and reused last-freed-first.  One manager per thread (not thread-safe).
 * ------------------------------------------------------------------------ */
typedef struct pkv_block_manager pkv_block_manager;

/* NULL on bad sizes (num_blocks in [1, 2^31), block_size >= 1, max_blocks_per_seq >= 1). */
PKV_API pkv_block_manager *pkv_bm_create(int64_t num_blocks, int block_size,
                                         int max_blocks_per_seq);
PKV_API void pkv_bm_destroy(pkv_block_manager *bm);
PKV_API int64_t pkv_bm_num_free(const pkv_block_manager *bm);
/* Reference count of a physical block (0 = free); -1 for a bad block id. */
PKV_API int32_t pkv_bm_refcount(const pkv_block_manager *bm, int64_t block);
/* New empty sequence; PKV_ERR_INVALID_ARG if the id exists. */
PKV_API pkv_status pkv_bm_add_sequence(pkv_block_manager *bm, int64_t seq_id);
/* New sequence child_id sharing every block of parent_id (reference counts +1),
 * e.g. a beam-search branch. */
PKV_API pkv_status pkv_bm_fork(pkv_block_manager *bm, int64_t parent_id, int64_t child_id);
/* Prefix caching: the empty sequence dst_id starts with src_id's first
 * num_tokens tokens (a multiple of block_size) by sharing their blocks. */
PKV_API pkv_status pkv_bm_share_prefix(pkv_block_manager *bm, int64_t src_id, int64_t dst_id,
                                       int64_t num_tokens);
/* Append one token: *slot receives its slot.  If the sequence's last block was
 * shared, it is replaced by a fresh copy and (*cow_src, *cow_dst) name the copy
 * to perform before the cache write; otherwise both are -1.
 * PKV_ERR_OUT_OF_BLOCKS when a block is needed and the pool is empty (nothing
 * changes); PKV_ERR_INVALID_ARG for an unknown id or a full table. */
PKV_API pkv_status pkv_bm_append_token(pkv_block_manager *bm, int64_t seq_id, int64_t *slot,
                                       int64_t *cow_src, int64_t *cow_dst);
/* Make the blocks that hold a sequence's first num_tokens tokens its own, so that
 * they can be rewritten in place: each one that another sequence references is
 * replaced by a fresh block, and cow_pairs[*num_cow_pairs][2] (host) names the
 * copies to perform (pkv_copy_blocks) before the write.  cow_pairs has room for
 * ceil(num_tokens / block_size) pairs (may be NULL when that is 0).  num_tokens
 * in [0, length]; PKV_ERR_OUT_OF_BLOCKS when the pool cannot cover the copies
 * (nothing changes). */
PKV_API pkv_status pkv_bm_make_private(pkv_block_manager *bm, int64_t seq_id, int64_t num_tokens,
                                       int64_t *cow_pairs, int64_t *num_cow_pairs);
/* Cut a sequence to its first num_tokens tokens (in [0, length]): the blocks past
 * them lose this sequence's reference, and return to the pool at zero. */
PKV_API pkv_status pkv_bm_truncate(pkv_block_manager *bm, int64_t seq_id, int64_t num_tokens);
/* Drop a sequence; its blocks' reference counts fall and blocks at zero return
 * to the pool. */
PKV_API pkv_status pkv_bm_free_sequence(pkv_block_manager *bm, int64_t seq_id);
/* Tokens held by a sequence (-1 if unknown). */
PKV_API int64_t pkv_bm_seq_len(const pkv_block_manager *bm, int64_t seq_id);
/* Copy a sequence's block table (host int32) into out[capacity]; *num_entries
 * gets its length (also when capacity is too small, which returns
 * PKV_ERR_INVALID_ARG). */
PKV_API pkv_status pkv_bm_block_table(const pkv_block_manager *bm, int64_t seq_id, int32_t *out,
                                      int capacity, int *num_entries);
/* One decode step for a batch of distinct sequences, all host buffers: appends
 * one token to each and writes slot_mapping[num_seqs], block_tables
 * [num_seqs][max_blocks_per_seq] (unused entries 0), context_lens[num_seqs]
 * (the new token included) and up to num_seqs copy-on-write pairs
 * cow_pairs[*num_cow_pairs][2] -- exactly the inputs of pkv_copy_blocks,
 * pkv_reshape_and_cache and pkv_paged_attention_decode for this step, run in
 * that order.  The pool is checked for the whole step first: on
 * PKV_ERR_OUT_OF_BLOCKS nothing changes. */
PKV_API pkv_status pkv_bm_decode_step(pkv_block_manager *bm, const int64_t *seq_ids,
                                      int num_seqs, int64_t *slot_mapping,
                                      int32_t *block_tables, int32_t *context_lens,
                                      int64_t *cow_pairs, int64_t *num_cow_pairs);

#ifdef __cplusplus
}
#endif
#endif /* PAGEDKV_H */
