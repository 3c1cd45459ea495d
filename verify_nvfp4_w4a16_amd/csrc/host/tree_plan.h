// How a call of nvfp4_kv_tree_attention is laid out over workgroups, and the
// workspace that this takes: host arithmetic, free of HIP.
#pragma once

#include <cstdint>

#include "nvfp4_draft.h"

namespace nvfp4 {

constexpr int kTreeWaves = 4;
constexpr int64_t kTreeWork = 36 * 1024;   // 16 rows x pages from which tiles of 64 and 128 rows pay
constexpr int kTreeLanes = 64;   // sequences whose pages a wavefront adds up by itself

struct TreePlan {
    int rows;         // of a workgroup's tile; 0: few rows, nvfp4_kv_attention's kernel for such
    bool whole;       // a workgroup takes a whole segment
    int ranges;       // else what a range of the pages holds of one: at most this many ranges,
    int least;        // of at least so many pages
    int64_t workgroups;
    bool added;       // more than kTreeLanes sequences: their pages are added up by a kernel before
};

// Of checked arguments.
TreePlan tree_plan(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q);

// Bytes of the sequences' sums, ahead of the parts.
int64_t tree_sum_bytes(const nvfp4_kv_seqs_t* s);

int64_t tree_workspace_bytes(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q);

}  // namespace nvfp4
