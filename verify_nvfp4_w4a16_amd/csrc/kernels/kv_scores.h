// Which slots a query row of the paged cache sees, and its scores: shared by
// the attention kernels and by the one that sums the weights of slots.
#pragma once

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "../host/kv_plan.h"
#include "kv_common.h"

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

struct KvScores {
    const uint16_t* q;
    int64_t q_pitch, q_head_pitch;
    int heads, group;      // query heads, and those of one kv head
    uint32_t inverse;      // floor((2^32 - 1) / group)
    int window;            // 0: no limit
    int max_q, max_kv;     // what the launch was sized for: sequences are held to it
    int causal;
    float scale;           // of q . (e4m3 * e2m1): the caller's times K's tensor scale is scale * 2^(exponent + 14),
    int exponent;          // apart because the product may be too small for fp32 where scores are not
    float cap, cap_inv;    // softcap (0: none) and its inverse

    // r / group for r in [0, 2^31): the product with the inverse is at most one short (a division takes 30 operations).
    __device__ __forceinline__ int over_group(int r) const {
        const int i = int(__umulhi(uint32_t(r), inverse));
        return r - i * group >= group ? i + 1 : i;
    }

    // z * log2(e) of products' sums x, whose row was scaled by its own power
    // of two (f is scale over that power, times log2(e) where there is no cap).
    template <int N>
    __device__ __forceinline__ void shape(float (&x)[N], float f) const {
        if (cap == 0.0f) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] *= f;
            return;
        }
        // cap * tanh(z / cap).  From y = z / cap = 1/4 on as 1 - 2 / (1 + exp(2 y)), with exact limits at
        // both ends; below that the difference would lose what is small beside the cap, and y's power
        // series to the seventh has it to 2^-21 of itself (the next term is y^8 * 62 / 2835).
        const float c = cap * kLog2e;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float y = x[i] * f * cap_inv, y2 = y * y;
            const float e = __builtin_amdgcn_exp2f(y * (2.0f * kLog2e));
            const float far = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + e);
            const float near = y + y * (y2 * (-1.0f / 3.0f + y2 * (2.0f / 15.0f - y2 * (17.0f / 315.0f))));
            x[i] = c * (fabsf(y) < 0.25f ? near : far);
        }
    }
};

inline KvScores kv_scores(const nvfp4_kv_cache_t* c, const nvfp4_kv_queries_t* q) {
    KvScores s;
    s.q = static_cast<const uint16_t*>(q->q);
    s.q_pitch = q->q_pitch;
    s.q_head_pitch = q->q_head_pitch;
    s.heads = static_cast<int>(q->heads);
    s.group = static_cast<int>(q->heads / c->kv_heads);
    s.inverse = 0xffffffffu / uint32_t(s.group);
    s.window = nvfp4::kv_window(q);
    s.max_q = static_cast<int>(q->max_q);
    s.max_kv = static_cast<int>(q->max_kv);
    s.causal = q->causal;
    s.scale = static_cast<float>(std::frexp(double(q->scale) * double(c->k_scale), &s.exponent));
    s.exponent -= 14;   // of the row's own power of two (convert_query)
    s.cap = std::min(q->softcap, 0x1p126f);   // more changes no score below 2^100, and its product with log2(e) is in range
    s.cap_inv = s.cap > 0.0f ? std::min(1.0f / s.cap, FLT_MAX) : 0.0f;
    return s;
}

// Slots [lo, hi) that some row of a set sees and [lo_all, hi_all) that all see.
struct Span {
    int lo, hi, lo_all, hi_all;
};

// One query row: its packed token, its query head within the group, and its slots [lo, hi).
struct QueryRow {
    int token, g, lo, hi;
};

// The rows of one sequence and kv head: row r is new token r / group, query
// head r % group of the group.
struct QueryRows {
    int first_token, new_tokens, len, count, group;

    __device__ __forceinline__ QueryRows(int first, int count_new, int length, int of_kv_head)
        : first_token(first), new_tokens(count_new), len(length), count(count_new * of_kv_head), group(of_kv_head) {}
    __device__ __forceinline__ QueryRows(const KvView& v, const KvScores& sc, int s) {
        first_token = v.start(s);
        new_tokens = min(max(v.start(s + 1) - first_token, 0), sc.max_q);
        len = min(v.len(s), sc.max_kv);
        group = sc.group;
        count = new_tokens * group;
    }
    __device__ __forceinline__ int see_lo(const KvScores& sc, int i) const {
        return sc.window > 0 ? max(len - new_tokens + i - sc.window + 1, 0) : 0;
    }
    __device__ __forceinline__ int see_hi(const KvScores& sc, int i) const {
        return sc.causal ? max(min(len, len - new_tokens + i + 1), 0) : len;
    }
    // For rows first .. last (both below count).
    __device__ __forceinline__ Span span(const KvScores& sc, int first, int last) const {
        const int i0 = sc.over_group(first), i1 = sc.over_group(last);
        return Span{see_lo(sc, i0), see_hi(sc, i1), see_lo(sc, i1), see_hi(sc, i0)};
    }
    // A row at or beyond count stands in for the last one (its result is dropped).
    __device__ __forceinline__ QueryRow row(const KvScores& sc, int r) const {
        r = min(r, count - 1);
        const int i = sc.over_group(r);
        return QueryRow{first_token + i, r - i * group, see_lo(sc, i), see_hi(sc, i)};
    }
    // Index of a row in [total][heads].
    __device__ __forceinline__ int64_t place(const KvScores& sc, int r, int hk) const {
        return place(sc, row(sc, r), hk);
    }
    static __device__ __forceinline__ int64_t place(const KvScores& sc, const QueryRow& r, int hk) {
        return int64_t(r.token) * sc.heads + hk * sc.group + r.g;
    }
};

// A query row as f16 operands: N pieces of 8 dims, piece i at p + i * STEP.
// bf16 reaches further than f16, so the row is scaled by the power of two that
// puts its largest magnitude into [2^14, 2^15): every element within 2^-28 of
// it keeps all its bits.  The lanes that share the row (those whose numbers
// differ in the bits FIRST .. LAST / 2) agree on the power.  Returns the factor that turns
// a sum of products into the score (times log2(e) where scores are not capped).
template <int N, int FIRST, int LAST>
__device__ __forceinline__ float convert_query(const KvScores& sc, const u32x4 (&raw)[N], f16x8 (&q)[N]) {
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            top = fmaxf(top, fabsf(bits_f32(raw[i][j] << 16)));
            top = fmaxf(top, fabsf(bits_f32(raw[i][j] & 0xffff0000u)));
        }
#pragma unroll
    for (int d = FIRST; d < LAST; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    // the power from the exponent field, held to what 2^14 / 2^e needs to stay finite
    const int e = min(max(int(f32_bits(top) >> 23) - 127, -100), 126);
    const float up = ldexpf(1.0f, 14 - e);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            q[i][2 * j] = static_cast<_Float16>(bits_f32(raw[i][j] << 16) * up);
            q[i][2 * j + 1] = static_cast<_Float16>(bits_f32(raw[i][j] & 0xffff0000u) * up);
        }
    const float f = __builtin_amdgcn_ldexpf(sc.scale, sc.exponent + e);
    return sc.cap == 0.0f ? f * kLog2e : f;
}

template <int N, int STEP, int FIRST>
__device__ __forceinline__ float load_query(const KvScores& sc, const uint16_t* p, f16x8 (&q)[N]) {
    u32x4 raw[N];
#pragma unroll
    for (int i = 0; i < N; ++i) raw[i] = load16(p + STEP * i);
    return convert_query<N, FIRST, 64>(sc, raw, q);
}

__device__ __forceinline__ const uint16_t* query_at(const KvScores& sc, const QueryRow& r, int hk) {
    return sc.q + int64_t(r.token) * sc.q_pitch + int64_t(hk * sc.group + r.g) * sc.q_head_pitch;
}

}  // namespace
