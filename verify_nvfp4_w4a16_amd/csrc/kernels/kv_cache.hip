// Filling and reading the paged NVFP4 cache (include/nvfp4_kv.h).
//
// A unit of work is one block of 8 slots of one sequence and head: V's codes
// of 8 slots share a dword at each dim, so one workgroup owns the block and
// merges the new rows' nibbles into it, with no atomics.  A workgroup has D
// threads: first one thread for each 16-dim group of the block's K and V rows
// (8 slots x D/16 groups x 2), then one thread for each dim's V dword.
// Bound by latency at one token a sequence and by the bf16 rows' bytes for
// prompts; see the measurements at the launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../host/kv_shapes.h"
#include "kv_common.h"
#include "setup.h"

namespace {

// Nearest e4m3 code to u >= 0, ties to even, saturating at 448.  The
// quantum's reciprocal is a power of two, so u / quantum is exact.
__device__ __forceinline__ uint32_t e4m3_code(double u) {
    if (!(u < 448.0)) return 0x7E;
    int e;
    (void)frexp(u, &e);                       // u in [2^(e-1), 2^e); 0 gives e = 0
    if (u == 0.0) return 0;
    const int lo = e - 1 < -6 ? -6 : e - 1;
    const double r = rint(ldexp(u, 3 - lo));  // 0..16 quanta of 2^(lo - 3)
    const uint32_t n = static_cast<uint32_t>(r);
    // codes are consecutive across binades: subnormals 0..7 at lo = -6
    const uint32_t code = lo == -6 ? n : ((uint32_t(lo + 7) << 3) + (n - 8));
    return code > 0x7E ? 0x7E : code;
}

// The e2m1 code of x at the group scale big = e4m3 * t: a magnitude is at
// least a threshold times big, compared in 64 bits, where the product of the
// 28-bit big and a 3-bit threshold is exact (as is the comparison with x, a
// bf16), so ties are real ties and go to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float x, double big) {
    const double a = fabs(double(x));
    const uint32_t m = uint32_t(a > 0.25 * big) + uint32_t(a >= 0.75 * big) + uint32_t(a > 1.25 * big) +
                       uint32_t(a >= 1.75 * big) + uint32_t(a > 2.5 * big) + uint32_t(a >= 3.5 * big) +
                       uint32_t(a > 5.0 * big);
    return m | (x < 0.0f && m ? 8u : 0u);
}

struct Rows {
    const uint16_t* p;
    int64_t pitch, head_pitch;
};

// One group of 16 of a row: its scale byte and its codes (code i in nibble i).
__device__ __forceinline__ uint64_t quantise16(const uint16_t* row, float t, uint32_t* scale) {
    float x[16];
    const u32x4 lo = load16(row), hi = load16(row + 8);
    uint16_t raw[16];
    __builtin_memcpy(raw, &lo, 16);
    __builtin_memcpy(raw + 8, &hi, 16);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = bf16_to_f32(raw[i]);
        x[i] = x[i] != x[i] ? 0.0f : x[i];    // a NaN is stored as 0
        amax = fmaxf(amax, fabsf(x[i]));
    }
    const uint32_t s = e4m3_code((double(amax) / 6.0) / double(t));
    *scale = s;
    const double big = double(e4m3_f32(s)) * double(t);
    uint64_t codes = 0;
    if (s != 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) codes |= uint64_t(e2m1_code(x[i], big)) << (4 * i);
    }
    return codes;
}

template <int D>
__global__ void __launch_bounds__(D)
kv_append_kernel(KvView v, Rows kr, Rows vr, float kt, float vt) {
    constexpr int kGroups = D / 16;
    __shared__ uint8_t vcode[8][D];
    const int u = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int s = unit_sequence(v, u);
    if (s < 0) return;
    const int t0 = v.start(s), nq = v.start(s + 1) - t0;
    if (nq <= 0) return;
    const int n = v.len(s), first = n - nq;            // slot of the first new token, maybe negative
    const int block = (first < 0 ? 0 : first / 8) + (u - (t0 / 8 + 2 * s));
    const int slot0 = block * 8;
    if (slot0 >= n) return;
    uint8_t* rec = v.record<D>(s, slot0 / kPage, h);
    if (!rec) return;
    const int in_page = slot0 % kPage;
    const int lo = first > slot0 ? first - slot0 : 0;  // new slots of the block: [lo, hi)
    const int hi = n - slot0 < 8 ? n - slot0 : 8;

    const bool is_v = tid >= 8 * kGroups;
    const int item = tid % (8 * kGroups);
    const int i = item / kGroups, g = item % kGroups;  // slot in the block, group
    if (i >= lo && i < hi) {
        const int64_t token = t0 + (slot0 + i - first);
        const Rows& r = is_v ? vr : kr;
        uint32_t scale;
        const uint64_t codes = quantise16(r.p + token * r.pitch + h * r.head_pitch + g * 16, is_v ? vt : kt, &scale);
        if (is_v) {
#pragma unroll
            for (int j = 0; j < 16; ++j) vcode[i][g * 16 + j] = uint8_t((codes >> (4 * j)) & 15);
            rec[KvRecord<D>::v_scale(in_page / 8, g) + i] = uint8_t(scale);
        } else {
            *reinterpret_cast<uint64_t*>(rec + KvRecord<D>::k_code(in_page + i) + g * 8) = codes;
            rec[KvRecord<D>::k_scale(in_page + i, g)] = uint8_t(scale);
        }
    }
    __syncthreads();
    uint32_t* word = reinterpret_cast<uint32_t*>(rec + KvRecord<D>::v_code(in_page / 8, tid));
    uint32_t w = lo == 0 && hi == 8 ? 0u : *word;
    for (int j = lo; j < hi; ++j) w = (w & ~(15u << (4 * j))) | (uint32_t(vcode[j][tid]) << (4 * j));
    *word = w;
}

// bf16 of the fp32 product t * (e4m3 * e2m1), two codes of byte `sel`.
template <int sel>
__device__ __forceinline__ uint32_t values2(uint32_t w, float scale, float t) {
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, sel);
    return uint32_t(f32_to_bf16_rne(c[0] * scale * t)) | (uint32_t(f32_to_bf16_rne(c[1] * scale * t)) << 16);
}

// The same units, the other way; rows whose slot is negative or whose page is
// outside the cache become zeros.
template <int D>
__global__ void __launch_bounds__(D)
kv_read_kernel(KvView v, uint16_t* k_out, uint16_t* v_out, float kt, float vt) {
    constexpr int kGroups = D / 16;
    __shared__ uint16_t vval[8][D + 8];
    const int u = blockIdx.x, h = blockIdx.y, tid = threadIdx.x;
    const int s = unit_sequence(v, u);
    if (s < 0) return;
    const int t0 = v.start(s), nq = v.start(s + 1) - t0;
    const int first = v.len(s) - nq;
    // blocks of 8 slots counted from the one that holds slot `first` (also below 0)
    const int slot0 = ((first & ~7)) + 8 * (u - (t0 / 8 + 2 * s));
    if (nq <= 0 || slot0 >= first + nq) return;
    const int lo = first > slot0 ? first - slot0 : 0;
    const int hi = first + nq - slot0 < 8 ? first + nq - slot0 : 8;
    const uint8_t* rec = slot0 >= 0 ? v.record<D>(s, slot0 / kPage, h) : nullptr;
    const int in_page = slot0 & (kPage - 1);

    if (rec) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + KvRecord<D>::v_code(in_page / 8, tid));
        const uint64_t sc = *reinterpret_cast<const uint64_t*>(rec + KvRecord<D>::v_scale(in_page / 8, tid / 16));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x2 c = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0)
                            : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1)
                            : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2)
                                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
            vval[2 * j][tid] = f32_to_bf16_rne(c[0] * e4m3_f32(uint32_t(sc >> (16 * j)) & 0xff) * vt);
            vval[2 * j + 1][tid] = f32_to_bf16_rne(c[1] * e4m3_f32(uint32_t(sc >> (16 * j + 8)) & 0xff) * vt);
        }
    }
    __syncthreads();
    const bool is_v = tid >= 8 * kGroups;
    const int item = tid % (8 * kGroups);
    const int i = item / kGroups, g = item % kGroups;
    if (i < lo || i >= hi) return;
    u32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
    if (rec && is_v) {
        a = load16(&vval[i][g * 16]);
        b = load16(&vval[i][g * 16 + 8]);
    } else if (rec) {
        const u32x2 w = *reinterpret_cast<const u32x2*>(rec + KvRecord<D>::k_code(in_page + i) + g * 8);
        const float sc = e4m3_f32(rec[KvRecord<D>::k_scale(in_page + i, g)]);
        a = u32x4{values2<0>(w[0], sc, kt), values2<1>(w[0], sc, kt), values2<2>(w[0], sc, kt), values2<3>(w[0], sc, kt)};
        b = u32x4{values2<0>(w[1], sc, kt), values2<1>(w[1], sc, kt), values2<2>(w[1], sc, kt), values2<3>(w[1], sc, kt)};
    }
    const int64_t token = t0 + (slot0 + i - first);
    uint16_t* out = (is_v ? v_out : k_out) + (token * v.kv_heads + h) * D + g * 16;
    *reinterpret_cast<u32x4*>(out) = a;
    *reinterpret_cast<u32x4*>(out + 8) = b;
}

template <int D>
int launch_append(const KvView& v, const Rows& k, const Rows& vr, float kt, float vt, unsigned units, hipStream_t st) {
    hipLaunchKernelGGL(kv_append_kernel<D>, dim3(units, v.kv_heads), dim3(D), 0, st, v, k, vr, kt, vt);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

template <int D>
int launch_read(const KvView& v, uint16_t* k, uint16_t* vo, float kt, float vt, unsigned units, hipStream_t st) {
    hipLaunchKernelGGL(kv_read_kernel<D>, dim3(units, v.kv_heads), dim3(D), 0, st, v, k, vo, kt, vt);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace

extern "C" int nvfp4_kv_append(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const void* k, int64_t k_pitch,
                               int64_t k_head_pitch, const void* v, int64_t v_pitch, int64_t v_head_pitch,
                               void* stream) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(k, k_pitch, k_head_pitch, seqs->total)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(v, v_pitch, v_head_pitch, seqs->total)) != NVFP4_OK) return st;
    if (seqs->seqs == 0 || seqs->total == 0) return NVFP4_OK;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const KvView view = kv_view(cache, seqs);
    const Rows kr{static_cast<const uint16_t*>(k), k_pitch, k_head_pitch};
    const Rows vr{static_cast<const uint16_t*>(v), v_pitch, v_head_pitch};
    const unsigned units = static_cast<unsigned>(unit_count(seqs));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch_append<64>(view, kr, vr, cache->k_scale, cache->v_scale, units, s);
        case 128: return launch_append<128>(view, kr, vr, cache->k_scale, cache->v_scale, units, s);
        default: return launch_append<256>(view, kr, vr, cache->k_scale, cache->v_scale, units, s);
    }
}

extern "C" int nvfp4_kv_read(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, void* k_out, void* v_out,
                             void* stream) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(k_out, 0, 0, seqs->total)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(v_out, 0, 0, seqs->total)) != NVFP4_OK) return st;
    if (seqs->seqs == 0 || seqs->total == 0) return NVFP4_OK;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const KvView view = kv_view(cache, seqs);
    uint16_t* ko = static_cast<uint16_t*>(k_out);
    uint16_t* vo = static_cast<uint16_t*>(v_out);
    const unsigned units = static_cast<unsigned>(unit_count(seqs));
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch_read<64>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
        case 128: return launch_read<128>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
        default: return launch_read<256>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
    }
}
