// Device helpers shared by the kernels on the paged NVFP4 cache: the record's
// layout (include/nvfp4_kv.h), the sequence arrays held to their ranges, and
// the exact decode of e2m1 x e4m3 to f16 matrix operands.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "nvfp4_kv.h"
#include "../host/kv_plan.h"
#include "nvfp4_common.h"

namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kPage = NVFP4_KV_PAGE;

// One (page, kv head) record.
template <int D>
struct KvRecord {
    static constexpr int kBytes = 72 * D;
    static constexpr int kVCodes = 32 * D;
    static constexpr int kKScales = 64 * D;
    static constexpr int kVScales = 68 * D;
    static constexpr int kGroups = D / 16;

    static __device__ __forceinline__ int k_code(int slot) { return slot * (D / 2); }
    static __device__ __forceinline__ int v_code(int block, int dim) { return kVCodes + (block * D + dim) * 4; }
    static __device__ __forceinline__ int k_scale(int slot, int group) {
        const int h = slot >> 5, a = (slot >> 3) & 3, t = (slot >> 2) & 1, r = slot & 3;
        constexpr int per = D / 64;
        const int b = group / per, j = group % per;
        return kKScales + ((((a * 4 + r) * 4 + b) * 2 + h) * 2 + t) * per + j;
    }
    static __device__ __forceinline__ int v_scale(int block, int group) {
        return kVScales + (block * kGroups + group) * 8;
    }
};

// The cache and the sequences as the kernels take them.
struct KvView {
    uint8_t* data;
    int64_t pages;
    int kv_heads;
    const int32_t* table;
    const int32_t* kv_lens;
    const int32_t* q_starts;
    int64_t table_pitch;
    int seqs;
    int total;

    __device__ __forceinline__ int len(int s) const {
        const int n = kv_lens[s];
        const int most = static_cast<int>(table_pitch * kPage);   // below 2^29
        return n < 0 ? 0 : (n > most ? most : n);
    }
    __device__ __forceinline__ int start(int s) const {
        const int t = q_starts[s];
        return t < 0 ? 0 : (t > total ? total : t);
    }
    // Number of logical page p (below table_pitch) of sequence s.
    __device__ __forceinline__ int page_id(int s, int p) const { return table[int64_t(s) * table_pitch + p]; }
    __device__ __forceinline__ bool has(int page) const { return page >= 0 && page < pages; }
    // Record of (page, head h); nullptr for a page outside the cache.
    template <int D>
    __device__ __forceinline__ uint8_t* record_of(int page, int h) const {
        return has(page) ? data + (int64_t(page) * kv_heads + h) * KvRecord<D>::kBytes : nullptr;
    }
    // The same for loads ahead of use, which are made whether the page is
    // there or not (a load under a condition would make every wait for loads
    // assume that it was not made): the cache's first page stands in.
    template <int D>
    __device__ __forceinline__ const uint8_t* record_or_first(int page, int h) const {
        return data + (int64_t(has(page) ? page : 0) * kv_heads + h) * KvRecord<D>::kBytes;
    }
    template <int D>
    __device__ __forceinline__ uint8_t* record(int s, int p, int h) const {
        return record_of<D>(page_id(s, p), h);
    }
};

// `count` workgroups in as many launches as hold them: launch(first, how many).
template <class Launch>
int launch_sliced(int64_t count, int threads, Launch launch) {
    const int64_t most = nvfp4::kKvLaunch * 256 / threads;
    for (int64_t at = 0; at < count; at += most) {
        launch(static_cast<int>(at), static_cast<unsigned>(count - at < most ? count - at : most));
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}

inline KvView kv_view(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s) {
    return KvView{c->data,   c->pages,    c->kv_heads,    s->table, s->kv_lens,
                  s->q_starts, s->table_pitch, static_cast<int>(s->seqs), static_cast<int>(s->total)};
}

__device__ __forceinline__ float e4m3_f32(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8(byte, 0); }

__device__ __forceinline__ f16x2 as_f16x2(uint32_t u) {
    f16x2 r;
    __builtin_memcpy(&r, &u, sizeof r);
    return r;
}

// An e4m3 byte b (0x00..0x7E) shifted into an f16's exponent and fraction is
// the value times 2^-8 (exponent biases 7 and 15), subnormals included, so a
// scale costs a byte shuffle and a shift; the 2^8 goes into the e2m1 decode,
// whose conversion takes a power of two for free.  e2m1 x e4m3 has 6
// significant bits and lies in [2^-10, 2688]: exact in f16.
constexpr float kScaleShift = 256.0f;

// Byte `sel` of v, in both halves, as such a scale pair.
template <int sel>
__device__ __forceinline__ f16x2 scale_both(uint32_t v) {
    constexpr uint32_t pick = 0x0c000c00u | uint32_t(sel) | (uint32_t(sel) << 16);
    return as_f16x2(__builtin_amdgcn_perm(0u, v, pick) << 7);
}

// Bytes 2 * half and 2 * half + 1 of v as a scale pair.
template <int half>
__device__ __forceinline__ f16x2 scale_pair(uint32_t v) {
    constexpr uint32_t pick = 0x0c000c00u | uint32_t(2 * half) | (uint32_t(2 * half + 1) << 16);
    return as_f16x2(__builtin_amdgcn_perm(0u, v, pick) << 7);
}

template <int sel>
__device__ __forceinline__ f16x2 codes_f16(uint32_t w) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, kScaleShift, sel);
}

__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight codes along a row (one scale) as a matrix operand.
__device__ __forceinline__ f16x8 decode_row(uint32_t w, f16x2 s) {
    return join(codes_f16<0>(w) * s, codes_f16<1>(w) * s, codes_f16<2>(w) * s, codes_f16<3>(w) * s);
}

// Eight codes of consecutive slots at one dim (a scale each).
__device__ __forceinline__ f16x8 decode_slots(uint32_t w, const f16x2 (&s)[4]) {
    return join(codes_f16<0>(w) * s[0], codes_f16<1>(w) * s[1], codes_f16<2>(w) * s[2], codes_f16<3>(w) * s[3]);
}

// The number of sequences, less one, for which below(s) holds, where it holds
// for none after one for which it does not.  All 64 lanes take part.
template <class Fn>
__device__ __forceinline__ int last_sequence(const KvView& v, Fn below) {
    const int lane = threadIdx.x & 63;
    int found = 0;
    for (int base = 0; base < v.seqs; base += 64) {
        const int s = base + lane;
        const int n = __popcll(__ballot(s < v.seqs && below(s)));
        found += n;
        if (n < 64) break;
    }
    return found - 1;
}

// The sequence that unit `u` belongs to, where sequence s's units begin at
// start(s) / 8 + 2 s: enough for every 8-slot block its rows touch, wherever
// they begin.
__device__ __forceinline__ int unit_sequence(const KvView& v, int u) {
    return last_sequence(v, [&](int s) { return v.start(s) / 8 + 2 * s <= u; });
}

inline int64_t unit_count(const nvfp4_kv_seqs_t* s) { return s->total / 8 + 2 * s->seqs; }

}  // namespace
