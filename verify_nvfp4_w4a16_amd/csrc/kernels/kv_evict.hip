// The attention weight that cache slots got, and the eviction that goes by it
// (include/nvfp4_kv.h).
//
// Weights: S[rows x slots] = Q K^T with K as the right operand, so a lane owns
// one slot (a column) and adds the rows' exp(z - lse) in registers: sums over
// rows run in row order with no atomics, and each page's K is read and decoded
// once however many rows see it.
//
// Eviction: per (sequence, kv head) the weight of the last slot that stays is
// found by a radix selection over order-preserving keys (most significant
// byte first, counts in LDS), then the slots that stay are numbered in slot
// order and their rows are copied, pages at a time.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../host/kv_shapes.h"
#include "kv_common.h"
#include "kv_scores.h"
#include "setup.h"

namespace {

struct WeightArgs {
    KvView v;
    KvScores sc;
    const float* lse;
    const float* prior;
    float* weights;
    int64_t max_kv;
};

// K of one 16-slot tile (h, t) as f16 operands: lane (n, b) holds slot
// 32 h + 8 (n / 4) + 4 t + n % 4, dims b D/4 ..
template <int D, int HT, int J>
__device__ __forceinline__ void decode_tile(const uint32_t (&codes)[D / 32], const uint32_t (&ks)[D / 64], f16x8 (&out)[D / 32]) {
    if constexpr (J < D / 64) {
        constexpr int i = HT * (D / 64) + J;
        const f16x2 s = scale_both<i % 4>(ks[i / 4]);
        out[2 * J] = decode_row(codes[2 * J], s);
        out[2 * J + 1] = decode_row(codes[2 * J + 1], s);
        decode_tile<D, HT, J + 1>(codes, ks, out);
    }
}

template <int D, int HT>
__device__ __forceinline__ void load_tile(const uint8_t* rec, int n, int b, const uint32_t (&ks)[D / 64], f16x8 (&out)[D / 32]) {
    uint32_t codes[D / 32];
    const int slot = 32 * (HT >> 1) + (n >> 2) * 8 + (HT & 1) * 4 + (n & 3);
    __builtin_memcpy(codes, __builtin_assume_aligned(rec + KvRecord<D>::k_code(slot) + b * (D / 8), D / 8), D / 8);
    decode_tile<D, HT, 0>(codes, ks, out);
}

// One wavefront a page; all rows that see it pass by.
template <int D>
__global__ void __launch_bounds__(256)
kv_weights_kernel(WeightArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = lane & 15, b = lane >> 4;
    const int s = blockIdx.y, hk = blockIdx.x % a.v.kv_heads;
    const int page = blockIdx.x / a.v.kv_heads * 4 + wave;
    const int base = page * kPage;
    if (base >= a.max_kv) return;
    const QueryRows rows(a.v, a.sc, s);
    float sum[4] = {0, 0, 0, 0};
    const uint8_t* rec = base < rows.len ? a.v.record<D>(s, page, hk) : nullptr;
    if (rec && rows.count > 0) {
        uint32_t ks[D / 64];
        __builtin_memcpy(ks, __builtin_assume_aligned(rec + KvRecord<D>::kKScales + (n * 4 + b) * (D / 16), D / 16), D / 16);
        f16x8 k[4][D / 32];
        load_tile<D, 0>(rec, n, b, ks, k[0]);
        load_tile<D, 1>(rec, n, b, ks, k[1]);
        load_tile<D, 2>(rec, n, b, ks, k[2]);
        load_tile<D, 3>(rec, n, b, ks, k[3]);
        // rows that see any slot of this page
        int i_lo = 0, i_hi = rows.new_tokens;
        if (a.sc.causal) i_lo = max(0, base - (rows.len - rows.new_tokens));
        if (a.sc.window > 0) i_hi = min(i_hi, max(0, base + kPage - 1 + a.sc.window - (rows.len - rows.new_tokens)));
        const int r_hi = i_hi * rows.group;
        for (int r0 = i_lo * rows.group; r0 < r_hi; r0 += 16) {
            f16x8 q[D / 32];
            const QueryRow me = rows.row(a.sc, r0 + n);
            const float f_n = load_query<D / 32, 8, 16>(a.sc, query_at(a.sc, me, hk) + b * (D / 4), q);
            const float lse_n = a.lse[rows.place(a.sc, min(r0 + n, rows.count - 1), hk)];
            const bool live_n = r0 + n < r_hi && lse_n != -INFINITY;
            const int lo_n = live_n ? me.lo : 0, hi_n = live_n ? me.hi : 0;
            f32x4 z[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                z[t] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < D / 32; ++i) z[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q[i], k[t][i], z[t], 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {   // row r0 + 4 b + c, held by lane 4 b + c
                const float f = __shfl(f_n, 4 * b + c);
                const float lse = __shfl(lse_n, 4 * b + c) * kLog2e;
                const int lo = __shfl(lo_n, 4 * b + c), hi = __shfl(hi_n, 4 * b + c);
                float x[4] = {z[0][c], z[1][c], z[2][c], z[3][c]};
                a.sc.shape(x, f);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int slot = base + 32 * (t >> 1) + (n >> 2) * 8 + (t & 1) * 4 + (n & 3);
                    const float p = __builtin_amdgcn_exp2f(x[t] - lse);
                    sum[t] += slot >= lo && slot < hi ? p : 0.0f;
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        sum[t] += __shfl_xor(sum[t], 16);
        sum[t] += __shfl_xor(sum[t], 32);
    }
    if (b != 0) return;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int slot = base + 32 * (t >> 1) + (n >> 2) * 8 + (t & 1) * 4 + (n & 3);
        if (slot >= a.max_kv) continue;
        const int64_t at = (int64_t(s) * a.v.kv_heads + hk) * a.max_kv + slot;
        a.weights[at] = slot < rows.len ? (a.prior ? a.prior[at] : 0.0f) + sum[t] : 0.0f;
    }
}

template <int D>
int launch_weights(const WeightArgs& a, hipStream_t st) {
    const int64_t blocks = (a.max_kv + 4 * kPage - 1) / (4 * kPage) * a.v.kv_heads;
    if (blocks > 0x7fffffff) return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL(kv_weights_kernel<D>, dim3(static_cast<unsigned>(blocks), a.v.seqs), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

struct EvictArgs {
    KvView v;
    const float* weights;
    int64_t weights_pitch;
    int keep, sink, recent;
    uint8_t* dst;
    int64_t dst_pages;
    const int32_t* dst_table;
    int64_t dst_pitch;
    int32_t* kept;
    float* kept_weights;
    int32_t* new_lens;

    __device__ __forceinline__ int len(int s) const { return static_cast<int>(min(int64_t(v.len(s)), weights_pitch)); }
};

// fp32 to a key that orders as the numbers do; -0 is 0, NaN is -inf.
__device__ __forceinline__ uint32_t order_key(float x) {
    x = x != x ? -INFINITY : x + 0.0f;
    const uint32_t u = f32_bits(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kSelect = 1024;

// Exclusive sums over the workgroup of two counts, in thread order, and their totals.
__device__ __forceinline__ void scan2(int x, int y, int* before_x, int* before_y, int* all_x, int* all_y, int (*tmp)[2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int sx = x, sy = y;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int ux = __shfl_up(sx, d), uy = __shfl_up(sy, d);
        if (lane >= d) sx += ux, sy += uy;
    }
    __syncthreads();
    if (lane == 63) tmp[wave][0] = sx, tmp[wave][1] = sy;
    __syncthreads();
    int bx = 0, by = 0, ax = 0, ay = 0;
    for (int w = 0; w < kSelect / 64; ++w) {
        if (w < wave) bx += tmp[w][0], by += tmp[w][1];
        ax += tmp[w][0], ay += tmp[w][1];
    }
    *before_x = bx + sx - x, *before_y = by + sy - y, *all_x = ax, *all_y = ay;
}

// Which slots stay: one workgroup a (sequence, head).
__global__ void __launch_bounds__(kSelect)
kv_select_kernel(EvictArgs a) {
    __shared__ int bins[256];
    __shared__ int tmp[kSelect / 64][2];
    __shared__ uint32_t found[2];
    const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const int n = a.len(s);
    const int64_t seq_head = int64_t(s) * a.v.kv_heads + h;
    const float* w = a.weights + seq_head * a.weights_pitch;
    int32_t* kept = a.kept + seq_head * a.keep;
    float* kept_w = a.kept_weights + seq_head * a.keep;
    if (h == 0 && tid == 0) a.new_lens[s] = min(n, a.keep);
    const int lo = n > a.keep ? a.sink : n, hi = n > a.keep ? n - a.recent : n;   // the choice is among [lo, hi)
    int need = n > a.keep ? a.keep - a.sink - a.recent : 0;
    uint32_t key = 0, mask = 0;   // the threshold's known leading bits
    if (need > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelect) bins[i] = 0;
            __syncthreads();
            for (int j = lo + tid; j < hi; j += kSelect) {
                const uint32_t k = order_key(w[j]);
                if ((k & mask) == key) atomicAdd(&bins[(k >> shift) & 255], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int left = need, d = 255;
                while (d > 0 && bins[d] < left) left -= bins[d--];
                found[0] = uint32_t(d), found[1] = uint32_t(left);
            }
            __syncthreads();
            key |= found[0] << shift;
            mask |= 255u << shift;
            need = int(found[1]);   // still wanted among the keys with these leading bits
            __syncthreads();
        }
    }
    // `need` of the slots at the threshold stay, the lowest first
    int at = 0, ties = 0;
    for (int j0 = 0; j0 < n; j0 += kSelect) {
        const int j = j0 + tid;
        bool sure = false, tie = false;
        if (j < n) {
            const uint32_t k = order_key(w[j]);
            const bool open = j >= lo && j < hi;
            sure = !open || (a.keep - a.sink - a.recent > 0 && k > key);
            tie = open && a.keep - a.sink - a.recent > 0 && k == key;
        }
        int bs, bt, as, al;
        scan2(sure, tie, &bs, &bt, &as, &al, tmp);
        const int tie_rank = ties + bt;
        if (sure || (tie && tie_rank < need)) {
            const int to = at + bs + (min(tie_rank, need) - min(ties, need));
            kept[to] = j;
            kept_w[to] = w[j];
        }
        at += as + (min(ties + al, need) - min(ties, need));
        ties += al;
    }
    for (int i = min(n, a.keep) + tid; i < a.keep; i += kSelect) {
        kept[i] = -1;
        kept_w[i] = 0.0f;
    }
}

// The rows that stay, one destination page a workgroup.
template <int D>
__global__ void __launch_bounds__(256)
kv_move_kernel(EvictArgs a) {
    using R = KvRecord<D>;
    __shared__ const uint8_t* from[kPage];
    __shared__ int slot_in[kPage];
    const int s = blockIdx.y, tid = threadIdx.x;
    const int h = blockIdx.x % a.v.kv_heads, page = blockIdx.x / a.v.kv_heads;
    const int n = min(a.len(s), a.keep);
    if (page * kPage >= n) return;
    const int64_t to_page = a.dst_table[int64_t(s) * a.dst_pitch + page];
    if (to_page < 0 || to_page >= a.dst_pages) return;
    uint8_t* to = a.dst + (to_page * a.v.kv_heads + h) * R::kBytes;
    if (tid < kPage) {
        const int at = page * kPage + tid;
        const uint8_t* rec = nullptr;
        int slot = 0;
        if (at < n) {
            const int j = a.kept[(int64_t(s) * a.v.kv_heads + h) * a.keep + at];
            rec = a.v.record<D>(s, j / kPage, h);
            slot = j % kPage;
        }
        from[tid] = rec;
        slot_in[tid] = slot;
    }
    __syncthreads();
    for (int i = tid; i < kPage * (D / 32); i += 256) {   // K codes, 16 bytes each
        const int slot = i / (D / 32), part = i % (D / 32);
        u32x4 x = {0, 0, 0, 0};
        if (from[slot]) x = load16(from[slot] + R::k_code(slot_in[slot]) + 16 * part);
        *reinterpret_cast<u32x4*>(to + R::k_code(slot) + 16 * part) = x;
    }
    for (int i = tid; i < kPage * (D / 16); i += 256) {   // scales
        const int slot = i / (D / 16), g = i % (D / 16);
        const uint8_t* rec = from[slot];
        const int j = slot_in[slot];
        to[R::k_scale(slot, g)] = rec ? rec[R::k_scale(j, g)] : 0;
        to[R::v_scale(slot / 8, g) + slot % 8] = rec ? rec[R::v_scale(j / 8, g) + j % 8] : 0;
    }
    for (int i = tid; i < 8 * D; i += 256) {              // V codes: a dword is 8 slots at a dim
        const int block = i / D, dim = i % D;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint8_t* rec = from[8 * block + e];
            const int j = slot_in[8 * block + e];
            if (rec) w |= (*reinterpret_cast<const uint32_t*>(rec + R::v_code(j / 8, dim)) >> (4 * (j % 8)) & 15u) << (4 * e);
        }
        *reinterpret_cast<uint32_t*>(to + R::v_code(block, dim)) = w;
    }
}

template <int D>
int launch_move(const EvictArgs& a, hipStream_t st) {
    const int64_t blocks = int64_t((a.keep + kPage - 1) / kPage) * a.v.kv_heads;
    if (blocks > 0x7fffffff) return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL(kv_move_kernel<D>, dim3(static_cast<unsigned>(blocks), a.v.seqs), dim3(256), 0, st, a);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

}  // namespace

extern "C" int nvfp4_kv_weights(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                const nvfp4_kv_queries_t* queries, const float* lse, const float* prior,
                                float* weights, void* stream) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_queries(cache, seqs, queries)) != NVFP4_OK) return st;
    if (misaligned(lse, 4) || misaligned(prior, 4) || misaligned(weights, 4)) return NVFP4_ERR_ALIGN;
    if (seqs->seqs == 0 || queries->max_kv == 0) return NVFP4_OK;
    if (!weights || (!lse && seqs->total > 0)) return NVFP4_ERR_NULL;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const WeightArgs a{kv_view(cache, seqs), kv_scores(cache, queries), lse, prior, weights, queries->max_kv};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch_weights<64>(a, s);
        case 128: return launch_weights<128>(a, s);
        default: return launch_weights<256>(a, s);
    }
}

extern "C" int nvfp4_kv_evict(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const float* weights,
                              int64_t weights_pitch, int64_t keep, int64_t sink, int64_t recent,
                              const nvfp4_kv_cache_t* dst, const int32_t* dst_table, int64_t dst_pitch, int32_t* kept,
                              float* kept_weights, int32_t* new_lens, void* stream) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_cache(dst)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, false)) != NVFP4_OK) return st;
    if (dst->kv_heads != cache->kv_heads || dst->head_dim != cache->head_dim) return NVFP4_ERR_SHAPE;
    if (keep < 1 || keep > (int64_t(1) << 30) || sink < 0 || recent < 0 || sink > keep || recent > keep || sink + recent > keep)
        return NVFP4_ERR_SHAPE;
    if (weights_pitch < 0 || weights_pitch > (int64_t(1) << 30)) return NVFP4_ERR_SHAPE;
    if (dst_pitch < 1 || dst_pitch > nvfp4::kKvMaxTablePitch || dst_pitch * kPage < keep) return NVFP4_ERR_SHAPE;
    if (misaligned(weights, 4) || misaligned(dst_table, 4) || misaligned(kept, 4) || misaligned(kept_weights, 4) || misaligned(new_lens, 4))
        return NVFP4_ERR_ALIGN;
    if (seqs->seqs == 0) return NVFP4_OK;
    if ((!weights && weights_pitch > 0) || !dst_table || !kept || !kept_weights || !new_lens) return NVFP4_ERR_NULL;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const EvictArgs a{kv_view(cache, seqs), weights, weights_pitch, static_cast<int>(keep), static_cast<int>(sink),
                      static_cast<int>(recent), dst->data, dst->pages, dst_table, dst_pitch, kept, kept_weights, new_lens};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipLaunchKernelGGL(kv_select_kernel, dim3(cache->kv_heads, static_cast<unsigned>(seqs->seqs)), dim3(kSelect), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    switch (cache->head_dim) {
        case 64: return launch_move<64>(a, s);
        case 128: return launch_move<128>(a, s);
        default: return launch_move<256>(a, s);
    }
}
