/*
 * paged_kv.h -- C ABI of the paged KV cache on MI355X (gfx950): what fills a
 * cache whose layer tensors the exponent codec (splitzip.h) compresses, what
 * attends over it, and what moves layer tensors between its pages and the
 * contiguous [tokens, KV heads, head dim] form that the codec codes.
 *
 * ---- The cache -----------------------------------------------------------
 *   One layer's keys and values, each in a pool of num_pages pages of
 *   page_size tokens.  Position p of a sequence lives in page
 *   table[p / page_size] at slot p % page_size.  Element (page, slot, head,
 *   i) of a pool is at page * page_stride + slot * token_stride +
 *   head * head_stride + i, in elements: token-major and head-major pages
 *   and views into larger pools are all the same call.
 *   dtype: BF16, or FP8 E5M2 (IEEE-style, Inf and NaN kept).
 *
 * ---- The batch -----------------------------------------------------------
 *   num_seqs sequences with n_s new tokens each, packed: sequence s has the
 *   rows cu[s] .. cu[s+1] - 1 of every per-token tensor (cu[0] >= 0,
 *   ascending, cu[num_seqs] <= total_tokens; rows that no sequence has are
 *   padding and are left as they were).  kv_len_s counts the sequence's
 *   tokens with the new ones, so new token i has position
 *   p = kv_len_s - n_s + i.  A token with p < 0 has no place: append and
 *   scatter drop it, gather gives zeros, its attention row is empty.  The
 *   same descriptor serves all four calls.
 *
 *   Tables and lengths are device data, so the host cannot check them: the
 *   kernels do.  A page id outside [0, num_pages) or past pages_per_seq, a
 *   kv_len outside [0, max_kv_len], a token range that is not ascending
 *   inside [0, total_tokens] or longer than max_tokens never leads to an
 *   access outside the pools: the page's positions are treated as masked
 *   (gather: zeros; append, scatter: dropped), a sequence with a bad length
 *   or range as having none of its new tokens (its rows are left as they
 *   were), and *d_status is set to SZ_ERR_INVALID_ARGUMENT.
 *
 * ---- Conventions ---------------------------------------------------------
 *   Those of splitzip.h: d_* pointers are HIP device memory owned by the
 *   caller; calls are asynchronous on `stream`; the library never allocates,
 *   frees or synchronises, and keeps nothing between calls; argument errors
 *   detectable on the host are returned before anything is enqueued.  The
 *   descriptors are host memory, read during the call.  Pools, per-token
 *   tensors and workspaces are 16-byte aligned and their strides multiples
 *   of 16 bytes; int32 and float arrays are 4-byte aligned (cos/sin tables
 *   16).  d_status (device int32, may be NULL) is only ever written on an
 *   error, never cleared: the caller zeroes it once and looks when it likes.
 *   Calls sharing a workspace or an output must not overlap in time.
 *   total_tokens = 0 or num_seqs = 0 is a call that does nothing.
 */
#ifndef PAGED_KV_H
#define PAGED_KV_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "splitzip.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void* d_k;               /* element (0, 0, 0, 0) of the key pool */
    void* d_v;               /* ... of the value pool */
    uint64_t page_stride;    /* elements, for both pools */
    uint64_t token_stride;
    uint64_t head_stride;
    uint32_t num_pages;      /* 1 .. 2^31 - 1 */
    uint32_t page_size;      /* tokens: a power of two, 1 .. 65536 */
    uint32_t kv_heads;       /* 1 .. 1024 */
    uint32_t head_dim;       /* 64, 80, 96, 128 or 256 */
    sz_dtype dtype;          /* of both pools */
    uint32_t reserved;       /* must be 0 */
} kv_cache;

typedef struct {
    const int32_t* d_pages;      /* page ids, sequence s from d_pages + s * pages_stride */
    const int32_t* d_cu_tokens;  /* num_seqs + 1 */
    const int32_t* d_kv_lens;    /* num_seqs */
    uint64_t pages_stride;       /* entries, >= pages_per_seq */
    uint32_t pages_per_seq;      /* >= 1 */
    uint32_t num_seqs;           /* < 2^20 */
    uint32_t total_tokens;       /* rows of the per-token tensors, < 2^24 */
    uint32_t max_tokens;         /* >= 1; no n_s is larger */
    uint32_t max_kv_len;         /* no kv_len_s is larger; < 2^31 - 2^17 */
    uint32_t reserved;           /* must be 0 */
} kv_batch;

/* ---- Append: keys and values of the new tokens into their pages, with the
 * per-head RMS norm and the position rotation applied on the way, and the
 * queries normed and rotated in the same pass.
 *
 * For each head vector x of head_dim elements of k (and q):
 *   y = x * w / sqrt(mean(x^2) + eps)                 if its norm weight w is given
 *   the first rotary_dim elements of y are rotated by row p of cos_sin
 *   (cos for pairs 0 .. rotary_dim/2 - 1, then their sin):
 *     pair i = (y_i, y_{i + rotary_dim/2}), or (y_{2i}, y_{2i+1}) if interleaved,
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * and is rounded once, to the cache's dtype (k) or BF16 (q), to nearest
 * even (x^2 and their mean are held in 32 bits, with their range); E5M2 does not saturate (61440 and more give Inf).  Values take no
 * norm and no rotation.  A BF16 key without norm and rotation, and a BF16
 * value, is copied bit for bit.  A position at or past max_positions is
 * treated like a bad page: nothing of that token is written, and *d_status
 * is set.  Two tokens of one call with the same page and slot: which of
 * them stays is undefined.
 * q_out may be q itself (same stride); other outputs must not overlap
 * inputs.  d_q = NULL: no queries (q_heads, strides and q_norm unused). ---- */
typedef struct {
    const void* d_k;          /* BF16, [total_tokens, kv_heads, head_dim] */
    const void* d_v;
    const void* d_q;          /* BF16, [total_tokens, q_heads, head_dim], or NULL */
    void* d_q_out;            /* BF16, the same shape */
    uint64_t k_stride;        /* elements from token to token; heads are contiguous */
    uint64_t v_stride;
    uint64_t q_stride;
    uint64_t q_out_stride;
    const float* d_cos_sin;   /* [max_positions, rotary_dim], or NULL: no rotation */
    const void* d_q_norm;     /* BF16 [head_dim], or NULL: no norm */
    const void* d_k_norm;
    float eps;                /* >= 0, finite */
    uint32_t q_heads;         /* 1 .. 65536 */
    uint32_t rotary_dim;      /* a multiple of 16, 16 .. head_dim */
    uint32_t max_positions;   /* >= 1 */
    uint32_t interleaved;     /* 0 or 1 */
    uint32_t reserved;        /* must be 0 */
} kv_append_args;

sz_status kv_append(const kv_cache* cache, const kv_batch* batch, const kv_append_args* args, int32_t* d_status,
                    hipStream_t stream);

/* ---- Attention of the new tokens over the cache (appended before):
 *   o = sum_j softmax_j(scale * q . k_j) v_j     over the positions j with
 *   p - window < j <= p (causal; window 0: all j <= p), or all j < kv_len.
 * Query head h reads KV head h / (q_heads / kv_heads).  A row that sees no
 * position, or only scores of -Inf, is empty: o = 0, lse = -Inf.  What a
 * row does not see never reaches it, NaN and Inf included.
 * d_lse (may be NULL): float [total_tokens, q_heads], ln of the sum of
 * exp(scale * q . k_j).
 * Scores, softmax statistics and the sum over j are held in 32 bits; the
 * weights are rounded to 16 bits before they multiply the values (BF16 for a
 * BF16 cache, FP16 for an E5M2 one).
 * d_out may be d_q itself (same stride); other outputs must not overlap inputs.
 * d_workspace: >= kv_attention_workspace_bytes of the same arguments, need
 * not be initialised, clobbered (may be NULL when that is 0). ---- */
typedef struct {
    const void* d_q;          /* BF16, [total_tokens, q_heads, head_dim] */
    void* d_out;              /* BF16, the same shape */
    float* d_lse;
    uint64_t q_stride;        /* elements from token to token; heads are contiguous */
    uint64_t out_stride;
    float scale;              /* > 0, finite */
    uint32_t q_heads;         /* a multiple of kv_heads, at most 64 times it */
    uint32_t causal;          /* 0 or 1 */
    uint32_t window;          /* 0: none; needs causal */
} kv_attention_args;

/* A call whose launch would have too many workgroups is refused: the rows of
 * a KV head, total_tokens * q_heads / kv_heads, make tiles of 16 (where
 * max_tokens * q_heads / kv_heads <= 16: one a sequence), or of 128 or 256
 * rows, and tiles * kv_heads stays below 2^23. */

/* Depends on the shapes and limits in the descriptors alone.  Pure host
 * function; 0 for arguments that kv_attention refuses. */
uint64_t kv_attention_workspace_bytes(const kv_cache* cache, const kv_batch* batch, const kv_attention_args* args);

sz_status kv_attention(const kv_cache* cache, const kv_batch* batch, const kv_attention_args* args,
                       void* d_workspace, uint64_t workspace_bytes, int32_t* d_status, hipStream_t stream);

/* ---- Gather and scatter: the batch's token rows out of the pages into
 * contiguous layer tensors [total_tokens, kv_heads, head_dim] of the cache's
 * dtype (what sz_compress takes), and back.  Bits are copied.  The strides
 * are in elements from token to token.  Neither tensor may overlap a pool
 * or the other. ---- */
sz_status kv_gather(const kv_cache* cache, const kv_batch* batch, void* d_k, uint64_t k_stride, void* d_v,
                    uint64_t v_stride, int32_t* d_status, hipStream_t stream);

sz_status kv_scatter(const kv_cache* cache, const kv_batch* batch, const void* d_k, uint64_t k_stride,
                     const void* d_v, uint64_t v_stride, int32_t* d_status, hipStream_t stream);

/* KV_ABI_VERSION as the library was compiled, as sz_abi_version. */
#define KV_ABI_VERSION 1u
uint32_t kv_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_H */
