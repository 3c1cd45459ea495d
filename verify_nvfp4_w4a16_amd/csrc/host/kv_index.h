// Which page or row of a sequence a workgroup works on, where the sequence is
// found by its start alone: used by the kernels, and by host checks that take
// starts in any order (constexpr functions serve both sides).
#pragma once

#include "nvfp4_kv.h"

namespace nvfp4 {

// Appending: sequence s's workgroups are numbered from here, enough for every
// page its rows touch, wherever they begin.
constexpr int kv_append_unit(int start, int s) { return start / NVFP4_KV_PAGE + 2 * s; }

// The page that workgroup `unit` fills, of a sequence whose first new token
// takes slot `first`; -1 if the workgroup is not one of the sequence's, as
// happens where starts descend.
constexpr int kv_append_page(int unit, int start, int s, int first) {
    const int own = unit - kv_append_unit(start, s);
    return own < 0 ? -1 : (first < 0 ? 0 : first / NVFP4_KV_PAGE) + own;
}

// The row of a token and a head of the group among a sequence's `count`; -1 if none.
constexpr int kv_row_of(int token, int first_token, int group, int head, int count) {
    if (token < first_token) return -1;
    const long long r = static_cast<long long>(token - first_token) * group + head;
    return r < count ? static_cast<int>(r) : -1;
}

}  // namespace nvfp4
