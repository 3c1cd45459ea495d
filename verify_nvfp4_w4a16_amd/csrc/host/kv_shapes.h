// Argument checks shared by the calls on the paged NVFP4 cache.
#pragma once

#include <cstdint>

#include "nvfp4_kv.h"

namespace nvfp4 {

constexpr int64_t kKvMaxTotal = int64_t(1) << 24;        // rows of a packed tensor
constexpr int64_t kKvMaxTablePitch = int64_t(1) << 23;   // pages of a table row: slots stay below 2^29
constexpr int64_t kKvMaxPitch = int64_t(1) << 31;        // elements from token to token
constexpr int64_t kKvMaxGroup = 256;                     // query heads of one kv head

// Each returns an NVFP4_* status.
int check_kv_cache(const nvfp4_kv_cache_t* c);
int check_kv_seqs(const nvfp4_kv_seqs_t* s, bool starts);
int check_kv_rows(const void* p, int64_t pitch, int64_t head_pitch, int64_t total);
int check_kv_queries(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q);

}  // namespace nvfp4
