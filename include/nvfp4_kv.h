/*
 * nvfp4_kv.h - C ABI of the serving step around the NVFP4 products for AMD
 * Instinct MI355X (gfx950): a paged key/value cache held in NVFP4, what
 * fills it, reads it and shrinks it, and the choice of the next token.
 *
 * The cache.  A page holds NVFP4_KV_PAGE (64) slots; `data` is
 * [pages][kv_heads] records of 72 * head_dim bytes (nvfp4_kv_record_bytes):
 *   0       K codes   [64 slots][D/2]     low nibble = even dim
 *   32 D    V codes   [8 blocks][D][4]    nibble i of the dword is slot
 *                                         8 * block + i at that dim
 *   64 D    K scales  [4 a][4 r][4 b][2 h][2 t][D/64 j]
 *                     slot = 32 h + 8 a + 4 t + r, group = b * D/64 + j
 *   68 D    V scales  [8 blocks][D/16 groups][8 slots]
 * with e2m1 codes, one e4m3 scale byte per 16 dims of a row (0x00..0x7E) and
 * one fp32 tensor scale for K and one for V: a stored value is
 * tensor_scale * e4m3 * e2m1, as everywhere in nvfp4_w4a16.h.  The orders
 * inside a record are those in which the attention kernels' lanes take their
 * matrix operands, so a page is read with wide loads and decoded in place.
 *
 * Sequences.  All calls take one block of sequences: `table`
 * [seqs][table_pitch] int32 page numbers, `kv_lens` [seqs] int32 slots in
 * use, the new tokens included, and `q_starts` [seqs + 1] int32: sequence
 * s's new tokens are rows q_starts[s] .. q_starts[s+1] - 1 of the packed
 * tensors and take its last slots: token j sits at slot
 * kv_lens[s] - (q_starts[s+1] - q_starts[s]) + j.  These arrays live on the
 * device and are not read by the host; a length is held to
 * [0, 64 * table_pitch], a start to [0, total], and a page number outside
 * [0, pages) stands for slots that nothing is written to and nothing sees.
 * Starts ascend; where they do not, nothing beyond the arrays is read or
 * written, but which of the rows are computed is not defined.
 *
 * Conventions are nvfp4_w4a16.h's: int status codes (nvfp4_strerror),
 * arguments checked before any launch, nothing launched and nothing written
 * on error, asynchronous on `stream` (a hipStream_t; NULL = the null
 * stream), no allocation and no host synchronisation, capturable into a HIP
 * graph after nvfp4_init().  A call's result depends on its inputs alone:
 * sums run in a fixed order or are exact, so repeated calls give the same
 * bits (which may differ in the last place between batches of another size).
 */
#ifndef NVFP4_KV_H
#define NVFP4_KV_H

#include <stdint.h>

#include "nvfp4_w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Slots of a page. */
#define NVFP4_KV_PAGE 64

/* A cache; the caller owns `data` (device, 16-byte aligned). */
typedef struct {
    uint8_t* data;
    int64_t pages;
    int32_t kv_heads;   /* 1..1024 */
    int32_t head_dim;   /* 64, 128 or 256 */
    float k_scale;      /* tensor scales, positive and finite */
    float v_scale;
} nvfp4_kv_cache_t;

/* A block of sequences, as above (device pointers, 4-byte aligned). */
typedef struct {
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* q_starts;
    int64_t table_pitch;   /* pages a table row holds, 1..2^23 */
    int64_t seqs;          /* 0..65535 */
    int64_t total;         /* rows of the packed tensors, 0..2^24 */
} nvfp4_kv_seqs_t;

/* Logit types of nvfp4_sample. */
enum {
    NVFP4_LOGITS_BF16 = 0,
    NVFP4_LOGITS_F32 = 1
};

/*
 * Host, pure.  *bytes = the bytes of one (page, head) record of this head
 * dimension: 72 * head_dim.  Errors: NULL, SHAPE.
 */
int nvfp4_kv_record_bytes(int64_t head_dim, int64_t* bytes);

/*
 * Device.  Quantises the new tokens' K and V rows into the cache.
 * k, v: bf16 [total][kv_heads][head_dim]; k_pitch and v_pitch are the
 * elements from token to token, k_head_pitch and v_head_pitch from head to
 * head (so a view of a fused projection's output can be passed), all
 * multiples of 8 and at least 0; k and v 16-byte aligned.
 * Rule (nvfp4_pack's with the tensor scale t given): per 16 dims
 * u = (amax / 6) / t rounded to the nearest e4m3 (ties to even, saturating at
 * 448); e2m1 code of x / (e4m3 * t) rounded to nearest (ties to even,
 * saturating at 6), all-zero codes when the scale is 0.  A NaN is stored as
 * 0 and an infinity as the largest magnitude, so that one bad row cannot
 * reach queries that do not see it.  Rows whose slot is negative are dropped.
 * Two sequences must not share a page that this call writes to.
 * Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_append(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const void* k, int64_t k_pitch,
                    int64_t k_head_pitch, const void* v, int64_t v_pitch, int64_t v_head_pitch, void* stream);

/*
 * Device.  The values that the sequences' last slots stand for, packed as
 * nvfp4_kv_append takes them: k_out, v_out bf16 [total][kv_heads][head_dim],
 * contiguous, 16-byte aligned; the fp32 product t * (e4m3 * e2m1) rounded to
 * bf16.  Rows without a slot (a negative one, or a page outside the cache)
 * are zeros; rows that no sequence owns are not written.
 * Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_read(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, void* k_out, void* v_out, void* stream);

/* What a query sees of its sequence, and how scores are formed. */
typedef struct {
    const void* q;          /* bf16 [total][heads][head_dim], 16-byte aligned */
    int64_t q_pitch;        /* elements from token to token, a multiple of 8 */
    int64_t q_head_pitch;   /* elements from head to head, a multiple of 8 */
    int64_t heads;          /* a multiple of kv_heads; heads / kv_heads <= 256 */
    int64_t max_q;          /* no sequence has more new tokens, 0..2^24 */
    int64_t max_kv;         /* no sequence is longer, 0..64 * table_pitch (the
                               launch is sized by both: one that is more is
                               taken for one of that size) */
    int64_t window;         /* slots a query sees at most, 0: no limit */
    float scale;            /* finite, and its product with k_scale too */
    float softcap;          /* scores become softcap * tanh(score / softcap); 0: not */
    int32_t causal;         /* 1: a query sees its own slot and those before it */
} nvfp4_kv_queries_t;

/*
 * Host, pure.  *bytes = the workspace nvfp4_kv_attention needs for these
 * arguments (0 where it needs none): the partial results of sequences whose
 * slots are split over workgroups.  Errors: NULL, SHAPE.
 */
int nvfp4_kv_attention_workspace(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                 const nvfp4_kv_queries_t* queries, int64_t* bytes);

/*
 * Device.  Attention of the new tokens over the cache.  For query token i of
 * a sequence of n slots and nq new tokens, at slot p = n - nq + i, head h
 * reading kv head h / (heads / kv_heads):
 *   z_j = scale * q . k_j, then softcap * tanh(z_j / softcap) if softcap > 0,
 *   over slots j < n with j <= p if causal and j > p - window if window > 0;
 *   out = sum_j softmax(z)_j v_j, bf16 [total][heads][head_dim] contiguous;
 *   lse = log sum_j exp z_j, fp32 [total][heads], may be NULL.
 * A query that sees nothing has out 0 and lse -inf.  Rows that no sequence
 * owns are not written.  Scores, softmax statistics and sums are fp32 (rows
 * with scores beyond its range are not defined); the
 * weights exp(z - max) are rounded to f16 for the second product.
 * out: 16-byte aligned.  workspace: device, 16-byte aligned, not shared by
 * calls that overlap in time.  Errors: NULL, SHAPE, ALIGN, SCRATCH (the
 * workspace is too small), HIP, DEVICE.
 */
int nvfp4_kv_attention(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries,
                       void* out, float* lse, void* workspace, int64_t workspace_bytes, void* stream);

/*
 * Device.  The attention weight that each slot got from the new tokens:
 *   weights[s][h][j] = prior[s][h][j] + sum exp(z_j - lse)
 * over the new tokens of sequence s and the query heads of kv head h, with
 * z and what a query sees as in nvfp4_kv_attention and lse [total][heads]
 * as it wrote it (queries with lse -inf give nothing).  weights, prior: fp32
 * [seqs][kv_heads][max_kv]; prior may be NULL (zeros) or equal to weights.
 * Slots from kv_lens[s] on get 0.  Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_weights(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries,
                     const float* lse, const float* prior, float* weights, void* stream);

/*
 * Device.  Cuts every sequence to at most `keep` slots by their accumulated
 * weights, each kv head on its own, into other pages.  Of n slots (n <= keep:
 * all of them) the first `sink`, the last `recent` and the
 * keep - sink - recent of the rest with the largest weights stay (ties: the
 * lower slot; a NaN counts as -inf), in slot order.
 *   weights      fp32 [seqs][kv_heads][weights_pitch]
 *   dst          a cache of the same geometry and tensor scales (codes are
 *                copied as they are; may be the same data), whose pages in
 *                dst_table [seqs][dst_pitch] are none that `seqs` still reads;
 *                dst_pitch * 64 >= keep
 *   kept         int32 [seqs][kv_heads][keep], slots ascending, then -1
 *   kept_weights fp32 [seqs][kv_heads][keep], their weights, then 0
 *   new_lens     int32 [seqs], min(n, keep)
 * Slots after the last kept one of a page hold zeros.  seqs->q_starts and
 * seqs->total are not used.  Errors: NULL, SHAPE (also sink + recent > keep,
 * keep < 1, 64 * table_pitch or a length beyond weights_pitch is held to
 * weights_pitch), ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_evict(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const float* weights,
                   int64_t weights_pitch, int64_t keep, int64_t sink, int64_t recent, const nvfp4_kv_cache_t* dst,
                   const int32_t* dst_table, int64_t dst_pitch, int32_t* kept, float* kept_weights, int32_t* new_lens,
                   void* stream);

/*
 * Device.  Draws one token a row from logits [rows][vocab] (row pitch
 * `pitch` elements, type NVFP4_LOGITS_*), the row's random number u in [0, 1)
 * and its parameters:
 *   d_i = (l_i - max l) * (1 / temperature), w_i = floor(2^30 exp d_i), and
 *   2^30 where l_i = max l; temperature <= 0 keeps the first maximum only;
 *   in the order of w descending, then index ascending,
 *   top_k:  the first top_k stay (<= 0: all),
 *   top_p:  of those, the ones before which less than top_p of their mass lies,
 *   min_p:  of those, the ones with w >= min_p * 2^30; the first always stays;
 *   with R the mass that stays, the token is the lowest index at which the
 *   running mass exceeds floor(u * R) (held to R - 1).
 * token int32 [rows]; logprob fp32 [rows] = log(w_token / R), may be NULL.
 * Masses are integers, so no order of summation changes a token.  A NaN
 * logit counts as -inf; a row with none above -inf gives token -1 and
 * logprob -inf.  Parameter arrays (device): temperature, top_p, min_p fp32
 * [rows], top_k int32 [rows]; NULL stands for 1, 1, 0 and 0.
 * workspace: device, 16-byte aligned, nvfp4_sample_workspace's bytes.
 * Shape: 0 <= rows <= 65535, 1 <= vocab <= 2^22, pitch >= vocab.
 * Errors: NULL, SHAPE, ALIGN (logits to their element size), DTYPE, SCRATCH,
 * HIP, DEVICE.
 */
int nvfp4_sample(const void* logits, int logits_type, int64_t rows, int64_t vocab, int64_t pitch, const float* u,
                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                 int32_t* token, float* logprob, void* workspace, int64_t workspace_bytes, void* stream);

/* Host, pure.  *bytes = the workspace nvfp4_sample needs.  Errors: NULL, SHAPE. */
int nvfp4_sample_workspace(int64_t rows, int64_t vocab, int64_t* bytes);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_KV_H */
