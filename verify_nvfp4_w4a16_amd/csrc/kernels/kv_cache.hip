// Filling and reading the paged NVFP4 cache (include/nvfp4_kv.h).
//
// V's codes of 8 slots share a dword at each dim, so a workgroup owns whole
// 8-slot blocks (a page's eight for append, one for read) of one sequence and head and
// merges the new rows' nibbles into them, with no atomics.  A thread takes one
// 16-dim group of a row, then dwords of V at a dim.  Bound by latency at one
// token a sequence and by the bf16 rows' bytes for prompts.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../host/kv_index.h"
#include "../host/kv_shapes.h"
#include "kv_common.h"
#include "setup.h"

namespace {

// The rounding rules in exact arithmetic: a code is settled by comparing the
// bf16 magnitude with a boundary times a scale, which 64 bits hold exactly (the
// tensor scale has 24 bits, an e4m3 value 4, a boundary at most 5), so a tie is
// a real tie.  No quotient is formed, where 64 bits would cost most.
struct Scale {
    double t, six_t;
    float inverse;   // 2^exponent / (6 t), for a first guess: 1 / (6 t) itself leaves fp32 at the largest and the smallest t
    int exponent;
    bool near_one;   // quotients can be formed in fp32: neither they nor the scales leave its range
    bool short_t;    // t has 8 bits, so ties are possible
};

// On the host, so that the kernel has them as scalars.
Scale scale_of(float t) {
    int e;
    const float m = static_cast<float>(std::frexp(double(t), &e));
    uint32_t bits;
    std::memcpy(&bits, &t, sizeof bits);
    return Scale{double(t), 6.0 * double(t), 1.0f / (6.0f * m), e, t > 0x1p-60f && t < 0x1p60f, (bits & 0xffff) == 0};
}

// The e4m3 code nearest to amax / (6 t), ties to even, saturating at 448.
__device__ __forceinline__ uint32_t e4m3_code(float amax, const Scale& sc) {
    // (the power of two saturates only where the quotient does)
    const float guess = fminf(__builtin_amdgcn_ldexpf(amax, -sc.exponent) * sc.inverse, 448.0f);
    const uint32_t c = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(guess, guess, 0, false)) & 0x7f;
    const double a = double(amax), v = double(e4m3_f32(c));
    if (c < 0x7E) {
        const double up = 0.5 * (v + double(e4m3_f32(c + 1))) * sc.six_t;
        if (a > up || (a == up && (c & 1))) return c + 1;
    }
    if (c > 0) {
        const double down = 0.5 * (v + double(e4m3_f32(c - 1))) * sc.six_t;
        if (a < down || (a == down && (c & 1))) return c - 1;
    }
    return c;
}

// The least bf16 magnitude (as its bits) that is above bound * big, or equal
// to it where STRICT is false.
template <bool STRICT>
__device__ __forceinline__ uint32_t least_above(double bound, double big) {
    const double at = bound * big;
    const float f = float(at);
    const uint32_t u = f32_bits(f);
    const double back = double(f);
    return (u >> 16) + uint32_t((u & 0xffff) != 0 || (STRICT ? at >= back : at > back));
}

struct Rows {
    const uint16_t* p;
    int64_t pitch, head_pitch;
};

typedef int16_t i16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pick(uint32_t mask, uint32_t yes, uint32_t no) { return (mask & yes) | (~mask & no); }

// -1 in each half where the magnitude there is at least the bound (bound less 1 is given).
__device__ __forceinline__ uint32_t reaches(uint32_t mags, uint32_t bound_less_1) {
    i16x2 m, b;
    __builtin_memcpy(&m, &mags, 4);
    __builtin_memcpy(&b, &bound_less_1, 4);
    const i16x2 d = (b - m) >> 15;
    uint32_t r;
    __builtin_memcpy(&r, &d, 4);
    asm("" : "+v"(r));   // a mask to the compiler too: it would go back to a comparison and a select a half
    return r;
}

// The codes of 16 elements (code i in nibble i) by the boundaries alone.
// Two elements at a time in halves of a register: three halving steps among
// the seven boundaries give a code's bits as masks, with no carries and no
// branches (20 operations an element).
__device__ __forceinline__ uint64_t codes_exact(const u32x4 lo, const u32x4 hi, const uint32_t (&mag)[8], double big) {
    // boundaries between the magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: a tie goes to the even code
    uint32_t b[7] = {least_above<true>(0.25, big), least_above<false>(0.75, big), least_above<true>(1.25, big),
                     least_above<false>(1.75, big), least_above<true>(2.5, big), least_above<false>(3.5, big),
                     least_above<true>(5.0, big)};
#pragma unroll
    for (int j = 0; j < 7; ++j) b[j] = (b[j] - 1) * 0x10001u;   // at least 1, at most 0x7f80: signed halves hold all differences
    uint32_t codes[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m2 = reaches(mag[i], b[3]);
        const uint32_t m1 = reaches(mag[i], pick(m2, b[5], b[1]));
        const uint32_t m0 = reaches(mag[i], pick(m2, pick(m1, b[6], b[4]), pick(m1, b[2], b[0])));
        uint32_t c = pick(0x00040004u, m2, pick(0x00020002u, m1, m0 & 0x00010001u));
        // the sign, but for a zero
        const uint32_t some = (m2 | m1 | m0) & 0x00080008u;
        c |= ((i < 4 ? lo[i] : hi[i - 4]) >> 12) & some;
        codes[i / 4] |= ((c | c >> 12) & 0xff) << (8 * (i % 4));
    }
    return uint64_t(codes[1]) << 32 | codes[0];
}

// Codes -0 made 0.
__device__ __forceinline__ uint32_t no_minus_zero(uint32_t w) {
    const uint32_t some = (w | w >> 1 | w >> 2) & 0x11111111u;
    return w & (some << 3 | 0x77777777u);
}

// The same codes by quotients in fp32, whose error is below 2^-22, and the
// conversion to e2m1.
//  * A tensor scale of 8 bits (a bf16 number, as powers of two are): a boundary
//    times the scales has at most 15 bits, so an element either is at it or
//    2^-15 of it away; quotients rounded to 18 bits are then on a boundary or
//    on its side exactly where the true ones are, and ties are the conversion's.
//  * Any other: no bf16 number is a tie.  Quotients 2^-20 lower and higher
//    enclose the true one; where their codes differ the boundaries decide.
template <bool SHORT>
__device__ __forceinline__ uint64_t codes_fast(const u32x4 lo, const u32x4 hi, const uint32_t (&mag)[8], double big) {
    const float inverse = __builtin_amdgcn_rcpf(float(big));
    const float low = inverse * (1.0f - 0x1p-20f), high = inverse * (1.0f + 0x1p-20f);
    auto element = [&](int i) { return bits_f32(i % 2 ? (i < 8 ? lo : hi)[i / 2 % 4] & 0xffff0000u : (i < 8 ? lo : hi)[i / 2 % 4] << 16); };
    auto rounded = [](float x) { return bits_f32((f32_bits(x) + 0x10) & ~0x1fu); };
    uint32_t w[2] = {0, 0}, v[2] = {0, 0};
    auto put = [&](auto byte) {
        constexpr int j = decltype(byte)::value;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const float a = element(8 * x + 2 * j), b = element(8 * x + 2 * j + 1);
            if constexpr (SHORT) {
                w[x] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[x], rounded(a * inverse), rounded(b * inverse), 1.0f, j);
            } else {
                w[x] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[x], a * low, b * low, 1.0f, j);
                v[x] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(v[x], a * high, b * high, 1.0f, j);
            }
        }
    };
    put(std::integral_constant<int, 0>{});
    put(std::integral_constant<int, 1>{});
    put(std::integral_constant<int, 2>{});
    put(std::integral_constant<int, 3>{});
    if (!SHORT && (w[0] != v[0] || w[1] != v[1])) return codes_exact(lo, hi, mag, big);
    return uint64_t(no_minus_zero(w[1])) << 32 | no_minus_zero(w[0]);
}

// One group of 16 of a row: its scale byte and its codes (code i in nibble i).
__device__ __forceinline__ uint64_t quantise16(u32x4 lo, u32x4 hi, const Scale& sc, uint32_t* scale) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    uint32_t mag[8];
    u16x2 most = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        mag[i] = (i < 4 ? lo[i] : hi[i - 4]) & 0x7fff7fffu;
        u16x2 m;
        __builtin_memcpy(&m, &mag[i], 4);
        most = __builtin_elementwise_max(most, m);
    }
    uint32_t top = max(uint32_t(most[0]), uint32_t(most[1]));
    if (top > 0x7f80) {   // a NaN is stored as 0
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t here = ~0u;
            if ((mag[i] & 0xffff) > 0x7f80) here &= 0xffff0000u;
            if (mag[i] > 0x7f80ffffu) here &= 0xffffu;
            mag[i] &= here;
            if (i < 4)
                lo[i] &= here;
            else
                hi[i - 4] &= here;
            top = max(top, max(mag[i] & 0xffff, mag[i] >> 16));
        }
    }
    const uint32_t s = e4m3_code(bits_f32(top << 16), sc);
    *scale = s;
    if (s == 0) return 0;
    const double big = double(e4m3_f32(s)) * sc.t;
    if (!sc.near_one) return codes_exact(lo, hi, mag, big);
    return sc.short_t ? codes_fast<true>(lo, hi, mag, big) : codes_fast<false>(lo, hi, mag, big);
}

// A workgroup takes one page's new slots for one head, so that a whole page of
// new rows is written in whole lines; the heads of a page lie next to each
// other in the grid, as their rows do in memory.  Prompts are bound by the rows'
// bytes (32,800 tokens of 8 heads of 128: 46 us for 172 MB, 3.7 TB/s; 50 us with
// the codes by the boundaries alone; at a tensor scale of 24 bits 58 us), single tokens by latency (48: 6 us).
template <int D>
__global__ void __launch_bounds__(256)
kv_append_kernel(KvView v, Rows kr, Rows vr, Scale ksc, Scale vsc, int group0) {
    constexpr int kGroups = D / 16, kItems = kPage * kGroups / 256;
    __shared__ uint64_t vcode[kPage][kGroups];              // 16 codes each
    __shared__ __attribute__((aligned(16))) uint8_t scales[8 * D];   // K's and V's, in the record's order
    const int group = group0 + static_cast<int>(blockIdx.x), u = group / v.kv_heads, h = group % v.kv_heads, tid = threadIdx.x;
    const int s = last_sequence(v, [&](int i) { return nvfp4::kv_append_unit(v.start(i), i) <= u; });
    if (s < 0) return;
    const int t0 = v.start(s), nq = v.start(s + 1) - t0;
    if (nq <= 0) return;
    const int n = v.len(s), first = n - nq;            // slot of the first new token, maybe negative
    const int page = nvfp4::kv_append_page(u, t0, s, first), slot0 = page * kPage;
    if (page < 0 || slot0 >= n) return;
    const int id = v.page_id(s, page);
    const int lo = first > slot0 ? first - slot0 : 0;  // new slots of the page: [lo, hi)
    const int hi = n - slot0 < kPage ? n - slot0 : kPage;
    const bool whole = lo == 0 && hi == kPage;

    u32x4 rows[kItems][4];
#pragma unroll
    for (int x = 0; x < kItems; ++x) {
        const int i = (x * 256 + tid) / kGroups, g = (x * 256 + tid) % kGroups;   // slot, group
        if (i < lo || i >= hi) continue;
        const int64_t token = t0 + (slot0 + i - first);
        const uint16_t* kp = kr.p + token * kr.pitch + h * kr.head_pitch + g * 16;
        const uint16_t* vp = vr.p + token * vr.pitch + h * vr.head_pitch + g * 16;
        rows[x][0] = load16_stream(kp), rows[x][1] = load16_stream(kp + 8);
        rows[x][2] = load16_stream(vp), rows[x][3] = load16_stream(vp + 8);
    }
    uint8_t* rec = v.record_of<D>(id, h);   // the page's number came while the rows were on their way
    if (!rec) return;
#pragma unroll
    for (int x = 0; x < kItems; ++x) {
        const int i = (x * 256 + tid) / kGroups, g = (x * 256 + tid) % kGroups;
        if (i < lo || i >= hi) continue;
        uint32_t ks, vs;
        *reinterpret_cast<uint64_t*>(rec + KvRecord<D>::k_code(i) + g * 8) = quantise16(rows[x][0], rows[x][1], ksc, &ks);
        vcode[i][g] = quantise16(rows[x][2], rows[x][3], vsc, &vs);
        const int k_at = KvRecord<D>::k_scale(i, g), v_at = KvRecord<D>::v_scale(i / 8, g) + i % 8;
        if (whole) {
            scales[k_at - KvRecord<D>::kKScales] = uint8_t(ks);
            scales[v_at - KvRecord<D>::kKScales] = uint8_t(vs);
        } else {
            rec[k_at] = uint8_t(ks);
            rec[v_at] = uint8_t(vs);
        }
    }
    __syncthreads();
    if (whole && tid < D / 2)
        *reinterpret_cast<u32x4*>(rec + KvRecord<D>::kKScales + 16 * tid) = *reinterpret_cast<const u32x4*>(scales + 16 * tid);
    // V's dwords: 8 slots at a dim, the ones that are not new kept
    for (int x = tid; x < 8 * D; x += 256) {
        const int block = x / D, dim = x % D;
        const int from = max(lo - 8 * block, 0), to = min(hi - 8 * block, 8);
        if (from >= to) continue;
        uint32_t* word = reinterpret_cast<uint32_t*>(rec + KvRecord<D>::v_code(block, dim));
        uint32_t w = from == 0 && to == 8 ? 0u : *word;
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(&vcode[8 * block][dim / 16]) + (dim / 8 & 1);
        const int shift = 4 * (dim % 8);
        if (from == 0 && to == 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) w |= (codes[2 * kGroups * j] >> shift & 15u) << (4 * j);
        } else {
            for (int j = from; j < to; ++j) w = (w & ~(15u << (4 * j))) | ((codes[2 * kGroups * j] >> shift & 15u) << (4 * j));
        }
        *word = w;
    }
}

// bf16 of the fp32 product t * (e4m3 * e2m1), two codes of byte `sel`.
template <int sel>
__device__ __forceinline__ uint32_t values2(uint32_t w, float scale, float t) {
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, sel);
    return uint32_t(f32_to_bf16_rne(c[0] * scale * t)) | (uint32_t(f32_to_bf16_rne(c[1] * scale * t)) << 16);
}

// Blocks of 8 slots, the other way; rows whose slot is negative or whose page is
// outside the cache become zeros.  Bound by the rows' bytes (32,800 tokens of 8
// heads of 128: 31 us for 172 MB, 5.5 TB/s).
template <int D>
__global__ void __launch_bounds__(D)
kv_read_kernel(KvView v, uint16_t* k_out, uint16_t* v_out, float kt, float vt, int group0) {
    constexpr int kGroups = D / 16;
    __shared__ uint16_t vval[8][D + 8];
    const int group = group0 + static_cast<int>(blockIdx.x), u = group / v.kv_heads, h = group % v.kv_heads, tid = threadIdx.x;
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
int launch_append(const KvView& v, const Rows& k, const Rows& vr, float kt, float vt, int64_t units, hipStream_t st) {
    if (units * v.kv_heads > 0x7fffffff) return NVFP4_ERR_SHAPE;
    const Scale ks = scale_of(kt), vs = scale_of(vt);
    return launch_sliced(units * v.kv_heads, 256, [&](int first, unsigned n) {
        hipLaunchKernelGGL(kv_append_kernel<D>, dim3(n), dim3(256), 0, st, v, k, vr, ks, vs, first);
    });
}

template <int D>
int launch_read(const KvView& v, uint16_t* k, uint16_t* vo, float kt, float vt, int64_t units, hipStream_t st) {
    if (units * v.kv_heads > 0x7fffffff) return NVFP4_ERR_SHAPE;
    return launch_sliced(units * v.kv_heads, D, [&](int first, unsigned n) {
        hipLaunchKernelGGL(kv_read_kernel<D>, dim3(n), dim3(D), 0, st, v, k, vo, kt, vt, first);
    });
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
    const int64_t units = seqs->total / kPage + 2 * seqs->seqs;
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
    const int64_t units = unit_count(seqs);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch_read<64>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
        case 128: return launch_read<128>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
        default: return launch_read<256>(view, ko, vo, cache->k_scale, cache->v_scale, units, s);
    }
}
