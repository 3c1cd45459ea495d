/*
 * nvfp4_draft.h - C ABI of the verify round over drafted tokens for AMD
 * Instinct MI355X (gfx950), beside the cache and the sampler of nvfp4_kv.h:
 * the page tables and slot maps of a step made on the device, what the nodes
 * of a drafted tree see and their attention over the cache, penalties, biases
 * and grammar masks on their logits, the branch that the model accepts, and
 * that branch's move to the front of its sequence.
 *
 * Trees.  A sequence's new tokens (nvfp4_kv.h) are the nodes of its tree, in
 * an order in which a node comes after its parent: node 0 is the root, the
 * last token that is settled; parents[row] is the node (counted from the
 * sequence's first row) that the row's node continues, and a value outside
 * [0, node) stands for none.  A node sees the slots before the tree, its
 * ancestors and itself.  A chain of tokens is a tree too (parents -1, 0, 1,
 * ...), a tree has at most NVFP4_TREE_MAX nodes, and `max_q` bounds the nodes
 * of every sequence of a call: one that has more is taken for its first max_q,
 * which then take its last slots.
 *
 * A round: nvfp4_kv_pages (tables), nvfp4_kv_tree (masks, positions), in each
 * layer nvfp4_kv_append and nvfp4_kv_tree_attention, nvfp4_adjust_logits and
 * nvfp4_sample on the nodes' logits, nvfp4_tree_accept, nvfp4_kv_move.  None
 * reads a device array on the host, so a round can be captured in one graph.
 *
 * Conventions are nvfp4_kv.h's.  Starts ascend in every call; where they do
 * not, or where a table, path, mask or parent holds anything at all, nothing
 * beyond the arrays is read or written, but which rows are computed is not
 * defined.
 */
#ifndef NVFP4_DRAFT_H
#define NVFP4_DRAFT_H

#include <stdint.h>

#include "nvfp4_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Nodes of a tree at most, and 64-bit words of a node's mask at most. */
#define NVFP4_TREE_MAX 256
#define NVFP4_TREE_WORDS 4

/* Entries of a sequence's bias list at most. */
#define NVFP4_BIAS_MAX 1024

/* The pages of a pool and of its sequences (device pointers, 4-byte aligned). */
typedef struct {
    int32_t* pool;          /* [capacity]: entry (head + i) % capacity, i < count, is a free page */
    const int32_t* state;   /* [2]: head, count */
    int64_t capacity;       /* 1..2^30, at least the pages that there are */
    int32_t* table;         /* [seqs][table_pitch] */
    int64_t table_pitch;    /* 1..2^23, times min(seqs, 1024) at most 2^30 */
    const int32_t* held;    /* [seqs] entries of a table row that the sequence owns */
    const int32_t* keep;    /* [seqs] slots that stay */
    const int32_t* fresh;   /* [seqs] new tokens that are asked for */
    int64_t seqs;           /* 0..65535 */
    int64_t total;          /* rows of the packed tensors, 0..2^24 */
} nvfp4_kv_pages_t;

/*
 * Device.  A step's tables.  held is taken into [0, table_pitch], keep into
 * [0, 64 held], a negative fresh as 0, head into [0, capacity) and count into
 * [0, capacity].  Sequence s wants keep + fresh slots, in ceil(want / 64)
 * pages.  It is granted if these fit a table row and, counting what the
 * sequences up to s ask for (those that do not fit a row apart): its new pages,
 * if it needs any, are within the count of free pages, and its new tokens, if
 * any, within `total`.  Granted:
 * pages beyond those it holds come from the pool's front, in order, into its
 * table row; pages that it holds and does not need any more go to the pool's
 * back (they are not given out again by the same call; what has no room in the
 * ring is dropped).  Not granted: it keeps its pages and `keep` slots and has
 * no new tokens.  Written:
 *   state_out  [2]         the pool's head and count after the call
 *   held_out   [seqs]      pages held after it
 *   kv_lens    [seqs]      slots in use, the new tokens included
 *   q_starts   [seqs + 1]  as nvfp4_kv.h has it
 *   slots      [total]     64 * page + slot in page of each new token; -1 behind
 *                          the last one and for a page outside [0, 2^25)
 *   positions  [total]     its slot's number within the sequence; -1 behind the last
 * slots are for callers that write a step's rows elsewhere by other means
 * (nvfp4_kv_append finds them from the table), positions for rotary angles and
 * the like; either may be NULL.  state_out may be state, held_out held and
 * kv_lens keep: a captured step then carries its own state on.  With other
 * outputs a call repeated on the same inputs gives the same again.  Table
 * entries that no new page takes stay as they were.
 * Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_pages(const nvfp4_kv_pages_t* pages, int32_t* state_out, int32_t* held_out, int32_t* kv_lens,
                   int32_t* q_starts, int32_t* slots, int32_t* positions, void* stream);

/*
 * Device.  What each node sees of its tree and where it stands:
 *   masks     uint64 [total][ceil(max_q / 64)]: bit a of a node's words is set
 *             where node a is one of its ancestors or itself
 *   positions int32 [total]: slots before the tree + the node's depth (a root's is 0)
 * kv_lens, q_starts as in nvfp4_kv.h; parents int32 [total].  1 <= max_q <=
 * NVFP4_TREE_MAX; masks 8-byte aligned.  Rows of no sequence are not written.
 * Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_tree(const int32_t* parents, const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs, int64_t total,
                  int64_t max_q, uint64_t* masks, int32_t* positions, void* stream);

/* What the nodes see, as nvfp4_kv_tree writes it or otherwise made. */
typedef struct {
    const uint64_t* masks;      /* [total][words], 8-byte aligned */
    const int32_t* positions;   /* [total]; NULL where there is no window */
    int64_t words;              /* ceil(max_q / 64)..NVFP4_TREE_WORDS */
    int32_t whole_tree;         /* 1: the window counts before the tree alone, and the masks
                                   say all that is seen of the tree itself; else 0 */
} nvfp4_kv_tree_t;

/*
 * Host, pure.  nvfp4_kv_attention_workspace for nvfp4_kv_tree_attention.
 * Errors: NULL, SHAPE, ALIGN.
 */
int nvfp4_kv_tree_attention_workspace(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                      const nvfp4_kv_queries_t* queries, int64_t* bytes);

/*
 * Device.  nvfp4_kv_attention for the nodes of trees: of n slots and nq new
 * tokens, row i sees
 *   the slots j < n - nq, with j > its position - window if window > 0, and
 *   the slots n - nq + a for which bit a of its mask is set (a < nq), with node
 *   a's position > its own - window if window > 0 and whole_tree is 0,
 * so a chain of tokens sees what it sees in nvfp4_kv_attention under the same
 * window.  A mask need not be a tree's, and one without bits leaves a row with the
 * slots before alone (or with nothing: out 0, lse -inf).  A position is taken
 * into [n - nq, n).  queries->causal is not used, queries->max_q is at most
 * NVFP4_TREE_MAX; all else, outputs and workspace are nvfp4_kv_attention's.
 * max_q and max_kv also choose between kernels: bounds far above the trees and
 * caches (a capacity, in a captured round) change last bits, and cost short
 * caches up to three times the time.
 * Errors: NULL, SHAPE, ALIGN, SCRATCH, HIP, DEVICE.
 */
int nvfp4_kv_tree_attention(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                            const nvfp4_kv_queries_t* queries, const nvfp4_kv_tree_t* tree, void* out, float* lse,
                            void* workspace, int64_t workspace_bytes, void* stream);

/* Logits and what they are adjusted by (device pointers; NULL where a field may be left out). */
typedef struct {
    const void* logits;            /* [rows][vocab], type NVFP4_LOGITS_* */
    int64_t rows, vocab, pitch;    /* rows 0..65535, vocab 1..2^22, pitch >= vocab elements from row to row */
    int64_t out_pitch;             /* >= vocab */
    int32_t logits_type, out_type; /* NVFP4_LOGITS_* */
    const int32_t* q_starts;       /* [seqs + 1] rows of each sequence; NULL: row r is sequence r, and seqs = rows */
    int64_t seqs;                  /* 0..65535 */
    const int32_t* history;        /* [seqs][history_pitch] tokens said so far, or NULL */
    const int32_t* history_lens;   /* [seqs], with history */
    const int32_t* prompt_lens;    /* [seqs] of those, the first ones that are the prompt; NULL: none */
    int64_t history_pitch;         /* 0..2^19; lengths are held to it */
    const float* repetition;       /* [seqs] r; NULL or a value not above 0: 1 */
    const float* presence;         /* [seqs] p; NULL: 0 */
    const float* frequency;        /* [seqs] f; NULL: 0 */
    const int32_t* bias_tokens;    /* [seqs][bias_width], or NULL; a token outside the vocabulary is none */
    const float* bias_values;      /* [seqs][bias_width], with bias_tokens */
    int64_t bias_width;            /* 0..NVFP4_BIAS_MAX */
    const uint32_t* allowed;       /* [states][allowed_pitch] bit v % 32 of word v / 32: token v may come; or NULL */
    const int32_t* allowed_rows;   /* [rows] the state of each row, outside [0, states): no mask; NULL: state r */
    int64_t allowed_pitch;         /* >= ceil(vocab / 32) */
    int64_t states;
    const int32_t* drafted;        /* [rows] a tree's tokens, or NULL */
    const uint64_t* masks;         /* [rows][mask_words], with drafted */
    int64_t mask_words;            /* 1..NVFP4_TREE_WORDS */
} nvfp4_adjust_t;

/*
 * Device.  out[r][v] of logit x = logits[r][v], with n the times that token v
 * stands in its sequence's history after the prompt, and among the drafted
 * tokens that the row's mask names (bit a: row q_starts[s] + a):
 *   if r != 1 and v stands in the history or n > 0:  x = x > 0 ? x / r : x * r
 *   if n > 0:  x = x - p - f * n
 *   if v is in the bias list:  x = x + its value (the last one's, if several)
 *   if the row's state does not allow v:  x = -inf
 * in fp32, rounded once (ties to even) where out is bf16.  A NaN stays one
 * where it is allowed.  out may be logits (with the same type and pitch), and
 * must not overlap them otherwise.
 * Rows of no sequence are not written.  Alignment: logits and out to their element
 * size, masks to 8 bytes, the rest to 4.
 * Errors: NULL, SHAPE, ALIGN, DTYPE, HIP, DEVICE.
 */
int nvfp4_adjust_logits(const nvfp4_adjust_t* adjust, void* out, void* stream);

/*
 * Device.  The branch that the model goes along: from node 0 on to the node's
 * continuation whose drafted token is `chosen` at the node (the lowest, where
 * several are; negative tokens are none), until there is none.
 *   drafted, parents, chosen int32 [total]; kv_lens, q_starts as in nvfp4_kv.h
 *   path     int32 [seqs][max_q]: the nodes taken, ascending, then -1
 *   counts   int32 [seqs]: how many
 *   token    int32 [seqs]: chosen at the last of them, which no draft carries;
 *            -1 for a sequence without rows
 *   new_lens int32 [seqs]: slots before the tree + counts, at least 0; may be kv_lens
 * 1 <= max_q <= NVFP4_TREE_MAX.  Errors: NULL, SHAPE, ALIGN, HIP, DEVICE.
 */
int nvfp4_tree_accept(const int32_t* drafted, const int32_t* parents, const int32_t* chosen, const int32_t* kv_lens,
                      const int32_t* q_starts, int64_t seqs, int64_t total, int64_t max_q, int32_t* path,
                      int32_t* counts, int32_t* token, int32_t* new_lens, void* stream);

/*
 * Device.  Moves the slots of a path to the front of their tree, in every one
 * of `count` caches of one geometry (the layers of a model, 1..1024, none of
 * whose data overlap, all under the same table): slot n - nq + j becomes what slot n - nq + path[s][j] was,
 * codes and scales as they are, for j = 0, 1, ... up to the first entry outside
 * [0, nq).  Paths ascend strictly, as nvfp4_tree_accept's do; where they do
 * not, which rows the moved slots hold is not defined.  All other slots, and
 * ones whose source or place is negative or on a page outside the cache, stay as they
 * were.  kv_lens and q_starts are those of the tree (before new_lens takes
 * their place), path int32 [seqs][max_q], 1 <= max_q <= NVFP4_TREE_MAX.  Two
 * sequences must not share a page that this call writes to.
 * Errors: NULL, SHAPE (also caches of different geometry or overlapping data), ALIGN, HIP, DEVICE.
 */
int nvfp4_kv_move(const nvfp4_kv_cache_t* caches, int64_t count, const nvfp4_kv_seqs_t* seqs, const int32_t* path,
                  int64_t max_q, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_DRAFT_H */
