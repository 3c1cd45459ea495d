// Attention over the paged NVFP4 cache (include/nvfp4_kv.h).
//
// The query rows that read one kv head of one sequence (new tokens x query
// heads of the group) form the columns of two transposed products:
//   S^T[slots x rows] = K Q^T,   O^T[dims x rows] += V^T P^T
// so every softmax statistic belongs to one column, that is, to one lane (and
// the lanes that share its column): no value is broadcast, and S^T leaves the
// matrix unit in the layout in which P^T enters it.  K's rows are taken in an
// order that makes a lane's scores those of 8 consecutive slots, V's dwords
// hold 8 consecutive slots of one dim: neither goes through LDS.
// The softmax runs over pages with the running maximum and sum (one pass over
// the cache); the pages of a sequence are split over the wavefronts of a
// workgroup and over workgroups, joined in a fixed order.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../host/kv_shapes.h"
#include "kv_common.h"
#include "kv_scores.h"
#include "setup.h"

namespace {

constexpr int kWaves = 4;

struct AttendArgs {
    KvView v;
    KvScores sc;
    uint16_t* out;
    float* lse;
    float* part_o;    // [splits][total * heads][D]: sums of exp2(z - m) v, without the V scale
    float* part_ml;   // [splits][total * heads][2]: m and the sum of exp2(z - m)
    int splits;
    float v_scale;
};

// What one wavefront holds of a page: codes and scales as the operands need them.
template <int D>
struct PageRegs {
    uint32_t k[4][D / 32];   // slot tile (h, t); D / 8 bytes of one row
    uint32_t ks[D / 64];     // 4 tiles x D/64 groups
    uint32_t v[2][D / 16];   // half page h; one dword a dim
    uint32_t vs[2][2];

    template <int N>
    static __device__ __forceinline__ void load(uint32_t* to, const uint8_t* p) {
        if constexpr (N % 4 == 0) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const u32x4 x = load16_stream(p + 16 * i);
                to[4 * i] = x[0], to[4 * i + 1] = x[1], to[4 * i + 2] = x[2], to[4 * i + 3] = x[3];
            }
        } else if constexpr (N == 2) {
            const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
            to[0] = x[0], to[1] = x[1];
        } else {
            to[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
        }
    }

    __device__ __forceinline__ void load_page(const uint8_t* rec, int n, int b) {
        using R = KvRecord<D>;
#pragma unroll
        for (int ht = 0; ht < 4; ++ht) {
            const int slot = 32 * (ht >> 1) + (n >> 2) * 8 + (ht & 1) * 4 + (n & 3);
            load<D / 32>(k[ht], rec + R::k_code(slot) + b * (D / 8));
        }
        load<D / 64>(ks, rec + R::kKScales + (n * 4 + b) * (D / 16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            load<D / 16>(v[h], rec + R::v_code(4 * h + b, n * (D / 16)));
            load<2>(vs[h], rec + R::v_scale(4 * h + b, n * (D / 16) / 16));
        }
    }

    // The scale pair of slot tile ht and the lane's 16-dim group j.
    template <int I>
    __device__ __forceinline__ f16x2 k_scale() const {
        return scale_both<I % 4>(ks[I / 4]);
    }
};

template <int D, int HT, int J>
__device__ __forceinline__ f32x4 score_groups(const PageRegs<D>& p, const f16x8 (&q)[D / 32], f32x4 acc) {
    if constexpr (J < D / 64) {
        const f16x2 s = p.template k_scale<HT * (D / 64) + J>();
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_row(p.k[HT][2 * J], s), q[2 * J], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_row(p.k[HT][2 * J + 1], s), q[2 * J + 1], acc, 0, 0, 0);
        return score_groups<D, HT, J + 1>(p, q, acc);
    }
    return acc;
}

__device__ __forceinline__ f16x8 to_f16x8(const float* p) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = static_cast<_Float16>(p[i]);
    return r;
}

// Few query rows: a wavefront takes 16 of them and whole pages, decoded from
// registers.  See the launch for the split and what it measured.
template <int D>
__global__ void __launch_bounds__(64 * kWaves)
kv_attend_rows_kernel(AttendArgs a) {
    extern __shared__ float lds[];   // [kWaves][16][D] sums, then [kWaves][16][2] statistics
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, b = lane >> 4;
    const int s = blockIdx.y, split = blockIdx.x % a.splits;
    const int hk = blockIdx.x / a.splits % a.v.kv_heads, tile = blockIdx.x / a.splits / a.v.kv_heads;
    const QueryRows rows(a.v, a.sc, s);
    const int row0 = tile * 16;
    if (row0 >= rows.count) return;

    const Span span = rows.span(a.sc, row0, min(row0 + 16, rows.count) - 1);
    const int page_lo = span.lo / kPage, page_hi = (span.hi + kPage - 1) / kPage;
    const int per = (max(page_hi - page_lo, 0) + a.splits - 1) / a.splits;
    const int begin = page_lo + split * per, end = min(begin + per, page_hi);

    const QueryRow me = rows.row(a.sc, row0 + n);
    f16x8 q[D / 32];
    const float to_log2 = load_query<D>(a.v, a.sc, me, hk, b, q);

    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    PageRegs<D> cur;
    int page = begin + wave;
    const uint8_t* rec = page < end ? a.v.record<D>(s, page, hk) : nullptr;
    if (rec) cur.load_page(rec, n, b);
    while (page < end) {
        const int next = page + kWaves;
        const uint8_t* next_rec = next < end ? a.v.record<D>(s, next, hk) : nullptr;
        PageRegs<D> ahead;
        if (next_rec) ahead.load_page(next_rec, n, b);
        if (rec) {
            const int base = page * kPage;
            f32x4 z[4];
            z[0] = score_groups<D, 0, 0>(cur, q, f32x4{0, 0, 0, 0});
            z[1] = score_groups<D, 1, 0>(cur, q, f32x4{0, 0, 0, 0});
            z[2] = score_groups<D, 2, 0>(cur, q, f32x4{0, 0, 0, 0});
            z[3] = score_groups<D, 3, 0>(cur, q, f32x4{0, 0, 0, 0});
            float p[16];   // [h][8 consecutive slots]
#pragma unroll
            for (int i = 0; i < 16; ++i) p[i] = a.sc.shape(z[i >> 2][i & 3], to_log2);
            if (base < span.lo_all || base + kPage > span.hi_all) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int slot = base + 32 * (i >> 3) + 8 * b + (i & 7);
                    p[i] = slot >= me.lo && slot < me.hi ? p[i] : -INFINITY;
                }
            }
            float top = p[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = fmaxf(top, p[i]);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            if (__any(top > m)) {
                const float grown = fmaxf(m, top);
                const float keep = grown == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
                m = grown;
                l *= keep;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) o[i] *= keep;
            }
            const float base_m = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = __builtin_amdgcn_exp2f(p[i] - base_m);
                l += p[i];
            }
            // slots from the length on hold anything: their scales become 0
            const int left = rows.len - base;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (left < kPage) {
                    const int live = left - 32 * h - 8 * b;
                    const uint64_t mask = live <= 0 ? 0 : live >= 8 ? ~0ull : (1ull << (8 * live)) - 1;
                    cur.vs[h][0] &= uint32_t(mask);
                    cur.vs[h][1] &= uint32_t(mask >> 32);
                }
                const f16x8 pt = to_f16x8(p + 8 * h);
                const f16x2 sc[4] = {scale_pair<0>(cur.vs[h][0]), scale_pair<1>(cur.vs[h][0]),
                                     scale_pair<0>(cur.vs[h][1]), scale_pair<1>(cur.vs[h][1])};
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_slots(cur.v[h][i], sc), pt, o[i], 0, 0, 0);
            }
        }
        cur = ahead;
        rec = next_rec;
        page = next;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (l != l && m == -INFINITY) m = 0.0f;   // all scores NaN: the row stays NaN

    // The wavefronts' results meet in LDS and are joined in wavefront order.
    float* sums = lds + wave * 16 * D;
    float* stats = lds + kWaves * 16 * D;
    if (b == 0) {
        stats[(wave * 16 + n) * 2] = m;
        stats[(wave * 16 + n) * 2 + 1] = l;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
            *reinterpret_cast<f32x4*>(sums + n * D + (4 * b + c) * (D / 16) + i) =
                f32x4{o[i][c], o[i + 1][c], o[i + 2][c], o[i + 3][c]};
    __syncthreads();
    constexpr int kPer = D / 16;   // dims of a thread: 256 threads, 16 rows
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * kPer;
    if (row0 + r >= rows.count) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[(w * 16 + r) * 2]);
    float acc[kPer] = {}, sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stats[(w * 16 + r) * 2] - top);
            sum += f * stats[(w * 16 + r) * 2 + 1];
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += f * lds[(w * 16 + r) * D + d0 + i];
        }
    }
    const int64_t at = rows.place(a.sc, row0 + r, hk);
    if (a.splits > 1) {
        const int64_t slice = int64_t(a.v.total) * a.sc.heads;
        float* po = a.part_o + (split * slice + at) * D + d0;
        if (top > -INFINITY)
#pragma unroll
            for (int i = 0; i < kPer; i += 4)
                *reinterpret_cast<f32x4*>(po + i) = f32x4{acc[i], acc[i + 1], acc[i + 2], acc[i + 3]};
        if (d0 == 0) {
            a.part_ml[(split * slice + at) * 2] = top;
            a.part_ml[(split * slice + at) * 2 + 1] = sum;
        }
        return;
    }
    const float f = sum > 0.0f || sum != sum ? a.v_scale / sum : 0.0f;
    uint16_t* out = a.out + at * D + d0;
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
        uint16_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f32_to_bf16_rne(acc[i + j] * f);
        u32x2 x;
        __builtin_memcpy(&x, w, 8);
        *reinterpret_cast<u32x2*>(out + i) = x;
    }
    if (a.lse && d0 == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
}

// Joins the splits of one row in split order: one wavefront a row.
template <int D>
__global__ void __launch_bounds__(256)
kv_join_kernel(AttendArgs a) {
    const int64_t slice = int64_t(a.v.total) * a.sc.heads;
    const int64_t at = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (at >= slice) return;
    const int token = static_cast<int>(at / a.sc.heads);
    if (token < a.v.start(0) || token >= a.v.start(a.v.seqs)) return;   // no sequence's row
    float top = -INFINITY;
    for (int p = 0; p < a.splits; ++p) top = fmaxf(top, a.part_ml[(p * slice + at) * 2]);
    constexpr int kPer = D / 64;
    float acc[kPer] = {}, sum = 0.0f;
    if (top > -INFINITY) {
        for (int p = 0; p < a.splits; ++p) {
            const float m = a.part_ml[(p * slice + at) * 2];
            if (m == -INFINITY) continue;
            const float f = __builtin_amdgcn_exp2f(m - top);
            sum += f * a.part_ml[(p * slice + at) * 2 + 1];
            const float* po = a.part_o + (p * slice + at) * D + lane * kPer;
#pragma unroll
            for (int i = 0; i < kPer; ++i) acc[i] += f * po[i];
        }
    }
    const float f = sum > 0.0f || sum != sum ? a.v_scale / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) a.out[at * D + lane * kPer + i] = f32_to_bf16_rne(acc[i] * f);
    if (a.lse && lane == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
}

// Workgroups that each get `splits` parts of their sequences' pages.
int split_count(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q) {
    const int64_t rows = q->max_q * (q->heads / c->kv_heads);
    const int64_t base = s->seqs * c->kv_heads * ((rows + 15) / 16);
    int64_t slots = q->max_kv;
    if (q->window > 0) slots = std::min(slots, q->window + q->max_q);
    const int64_t pages = (slots + kPage - 1) / kPage;
    if (base == 0 || pages == 0) return 1;
    int64_t splits = std::max<int64_t>((1024 + base - 1) / base, (slots + 4095) / 4096);
    splits = std::min(splits, (pages + kWaves - 1) / kWaves);
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(splits, 256)));
}

int64_t workspace_bytes_of(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q) {
    const int splits = split_count(c, s, q);
    return splits == 1 ? 0 : int64_t(splits) * s->total * q->heads * (c->head_dim + 2) * int64_t(sizeof(float));
}

template <int D>
constexpr size_t rows_lds() {
    return (kWaves * 16 * D + kWaves * 16 * 2) * sizeof(float);
}

template <int D>
bool allow_lds() {
    return hipFuncSetAttribute(reinterpret_cast<const void*>(kv_attend_rows_kernel<D>),
                               hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLdsBytes) == hipSuccess;
}

template <int D>
int launch_attend(const AttendArgs& a, int64_t rows, hipStream_t st) {
    const int64_t blocks = (rows + 15) / 16 * a.v.kv_heads * a.splits;
    if (blocks > 0x7fffffff) return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL(kv_attend_rows_kernel<D>, dim3(static_cast<unsigned>(blocks), a.v.seqs), dim3(64 * kWaves),
                       rows_lds<D>(), st, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    if (a.splits > 1) {
        const int64_t slice = int64_t(a.v.total) * a.sc.heads;
        hipLaunchKernelGGL(kv_join_kernel<D>, dim3(static_cast<unsigned>((slice + 3) / 4)), dim3(256), 0, st, a);
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}

}  // namespace

namespace nvfp4 {

int kv_setup() { return allow_lds<64>() && allow_lds<128>() && allow_lds<256>() ? NVFP4_OK : NVFP4_ERR_HIP; }

}  // namespace nvfp4

extern "C" int nvfp4_kv_attention_workspace(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                            const nvfp4_kv_queries_t* queries, int64_t* bytes) {
    int st;
    if (!bytes) return NVFP4_ERR_NULL;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_queries(cache, seqs, queries)) != NVFP4_OK) return st;
    *bytes = workspace_bytes_of(cache, seqs, queries);
    return NVFP4_OK;
}

extern "C" int nvfp4_kv_attention(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                  const nvfp4_kv_queries_t* queries, void* out, float* lse, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_queries(cache, seqs, queries)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(out, 0, 0, seqs->total)) != NVFP4_OK) return st;
    if ((reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 15)) return NVFP4_ERR_ALIGN;
    if (seqs->seqs == 0 || seqs->total == 0 || queries->max_q == 0) return NVFP4_OK;
    const int64_t need = workspace_bytes_of(cache, seqs, queries);
    if (need > 0 && !workspace) return NVFP4_ERR_NULL;
    if (need > workspace_bytes) return NVFP4_ERR_SCRATCH;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;

    AttendArgs a;
    a.v = kv_view(cache, seqs);
    a.sc = kv_scores(cache, queries);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.splits = split_count(cache, seqs, queries);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = a.splits > 1 ? a.part_o + int64_t(a.splits) * seqs->total * queries->heads * cache->head_dim : nullptr;
    a.v_scale = cache->v_scale;
    const int64_t rows = queries->max_q * a.sc.group;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch_attend<64>(a, rows, s);
        case 128: return launch_attend<128>(a, rows, s);
        default: return launch_attend<256>(a, rows, s);
    }
}
