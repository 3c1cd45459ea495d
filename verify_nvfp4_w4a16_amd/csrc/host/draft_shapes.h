// Argument checks of the verify round over drafted tokens.
#pragma once

#include <cstdint>

#include "nvfp4_draft.h"

namespace nvfp4 {

constexpr int64_t kPoolMax = int64_t(1) << 30;        // pages of a pool: head + count + new ones stay below 2^31
constexpr int kPagesBlock = 1024;                      // sequences whose pages are added up at a time
constexpr int64_t kHistoryMax = int64_t(1) << 19;     // a count and the drafted tokens stay below 2^20
constexpr int64_t kMoveCaches = 1024;

// Each returns an NVFP4_* status.
int check_kv_pages(const nvfp4_kv_pages_t* p, const int32_t* state_out, const int32_t* held_out, const int32_t* kv_lens,
                   const int32_t* q_starts, const int32_t* slots, const int32_t* positions);
// Sequences of trees without tables: seqs, total, max_q and the two arrays.
int check_trees(const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs, int64_t total, int64_t max_q);
// Of checked sequences and queries.
int check_kv_tree(const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q, const nvfp4_kv_tree_t* t);
int check_adjust(const nvfp4_adjust_t* a, const void* out);
int check_kv_move(const nvfp4_kv_cache_t* caches, int64_t count, const nvfp4_kv_seqs_t* s, const int32_t* path, int64_t max_q);

// A required array of 4-byte elements.
int check_words(const void* p);

}  // namespace nvfp4
