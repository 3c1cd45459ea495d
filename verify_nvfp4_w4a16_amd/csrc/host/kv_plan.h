// How a call of nvfp4_kv_attention is laid out over workgroups, and the
// workspace that this takes: host arithmetic, free of HIP.
#pragma once

#include <cstdint>

#include "nvfp4_kv.h"

namespace nvfp4 {

constexpr int kKvWaves = 4;
constexpr int kKvRowTile = 16;               // few rows: of one workgroup
constexpr int kKvTileRows = 32 * kKvWaves;   // many rows
constexpr int kKvMaxSplits = 1024;
constexpr int kKvItems = 2048;               // whole chunks of a plan (1280 to 3584 took the same within 3 %)

// 16-row or 128-row workgroups, and over how many workgroups each sequence's
// pages are split.
struct KvPlan {
    int tile;            // rows of a many-row workgroup, 0: few rows
    int64_t row_tiles;
    int splits, chunk;   // tile
    bool planned;        // else
    int items;
    int64_t part_rows;   // rows of partial results
};

// The window as the kernels take it: 0 (no limit) where no sequence of the
// call is longer, so that a window of any size can be added to a slot.
int kv_window(const nvfp4_kv_queries_t* q);

// Of checked arguments.
KvPlan kv_plan(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q);

// Bytes of the planned items, ahead of the partial results.
int64_t kv_plan_bytes(const nvfp4_kv_seqs_t* s);

int64_t kv_workspace_bytes(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q);

}  // namespace nvfp4
