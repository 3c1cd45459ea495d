// The attention weight that cache slots got, and the eviction that goes by it
// (include/nvfp4_kv.h).
//
// Weights: S[rows x slots] = Q K^T with K as the right operand, so a lane owns
// one slot (a column) and adds the rows' exp(z - lse) in registers: sums over
// rows run in row order with no atomics.  The rows are staged in LDS, 64 or 128
// at a time, and a page's K is read and decoded once for each such block.
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

// One page's K of a lane (n, b): of each 16-slot tile ht = (h, t) the slot
// 32 h + 8 (n / 4) + 4 t + n % 4, dims b D/4 ..
template <int D>
struct KRegs {
    uint32_t codes[4][D / 32], scales[D / 64];

    static __device__ __forceinline__ int slot(int ht, int n) { return 32 * (ht >> 1) + (n >> 2) * 8 + (ht & 1) * 4 + (n & 3); }
    __device__ __forceinline__ void load(const uint8_t* rec, int n, int b) {
#pragma unroll
        for (int ht = 0; ht < 4; ++ht)
            __builtin_memcpy(codes[ht], __builtin_assume_aligned(rec + KvRecord<D>::k_code(slot(ht, n)) + b * (D / 8), D / 8), D / 8);
        __builtin_memcpy(scales, __builtin_assume_aligned(rec + KvRecord<D>::kKScales + (n * 4 + b) * (D / 16), D / 16), D / 16);
    }
    template <int HT, int J>
    __device__ __forceinline__ void decode(f16x8 (&out)[D / 32]) const {
        if constexpr (J < D / 64) {
            constexpr int i = HT * (D / 64) + J;
            const f16x2 s = scale_both<i % 4>(scales[i / 4]);
            out[2 * J] = decode_row(codes[HT][2 * J], s);
            out[2 * J + 1] = decode_row(codes[HT][2 * J + 1], s);
            decode<HT, J + 1>(out);
        }
    }
};

// Query rows of a workgroup in LDS: f16, each row's 16-byte chunks permuted so
// that the 16 rows of a matrix operand's read fall on different banks, and
// what a row's scores need.
template <int D, int ROWS>
struct QueryBlock {
    static constexpr int kRows = ROWS;

    f16x8 q[kRows * D / 8];
    float f[kRows], lse[kRows];   // the factor of its sums; lse * log2(e), +inf for a row that gives nothing
    int lo[kRows], hi[kRows];

    static __device__ __forceinline__ int chunk_at(int row, int chunk) {
        return row * (D / 8) + (chunk ^ (D == 64 ? (row >> 1) & 7 : row & 15));
    }
    // Rows r0 .. of the sequence, by all 256 threads, D / 8 lanes a row: all
    // loads first (rows past the last are loaded as the last).
    __device__ __forceinline__ void fill(const WeightArgs& a, const QueryRows& rows, int hk, int r0) {
        constexpr int kLanes = D / 8, kStep = 256 / kLanes, kTurns = kRows / kStep;
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));   // what follows from it is found anew: kept between blocks it would not fit the registers
        const int chunk = tid % kLanes, row = tid / kLanes;
        const int many = (min(rows.count - r0, kRows) + 15) / 16 * 16;   // whole tiles
        u32x4 raw[kTurns][1];
#pragma unroll
        for (int x = 0; x < kTurns; ++x)
            raw[x][0] = load16(query_at(a.sc, rows.row(a.sc, r0 + x * kStep + row), hk) + 8 * chunk);
        const int own = min(tid, kRows - 1);   // the row whose statistics this thread brings
        const QueryRow mine = rows.row(a.sc, r0 + own);
        const float l = a.lse[rows.place(a.sc, mine, hk)];
#pragma unroll
        for (int x = 0; x < kTurns; ++x) {
            const int i = x * kStep + row;
            if (i >= many) break;
            f16x8 y[1];
            const float factor = convert_query<1, 1, kLanes>(a.sc, raw[x], y);
            q[chunk_at(i, chunk)] = y[0];
            if (chunk == 0) f[i] = factor;
        }
        if (tid < kRows) {
            lse[own] = l == -INFINITY || r0 + own >= rows.count ? INFINITY : l * kLog2e;
            lo[own] = mine.lo, hi[own] = mine.hi;
        }
    }
};

// PAGES pages a wavefront, or SHARE wavefronts' together, which then take the
// tiles of rows in turn; all rows that see them pass by, ROWS at a time (with
// more than one page a wavefront there are no more than ROWS).  One
// token's weights are bound by latency and the slots' bytes (16 sequences of 100
// .. 16383 slots, 8 heads of 128: 13.7 us for 21 MB, most of it weights and
// their priors), those of many by the exponentials and the products beside the
// waits of staging (32 tokens of 32 heads over 4 x 9001 .. 32768 slots: 37 us,
// 590 TFLOP/s; three workgroups a CU, for which a page's sums wait in LDS while
// the wavefront is at another page, took 39 us where two took 53).
template <int D, int PAGES, int ROWS, int SHARE>
__global__ void __launch_bounds__(256, D == 256 ? 2 : 3)
kv_weights_kernel(WeightArgs a) {
    using Block = QueryBlock<D, ROWS>;
    constexpr int kGroup = 4 / SHARE * PAGES;   // pages of the workgroup
    __shared__ Block block;
    __shared__ f32x4 sums[4][PAGES][64];   // of a wavefront's pages, a lane's slots: in registers only while their page is
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, b = lane >> 4;
    const int s = blockIdx.y, hk = blockIdx.x % a.v.kv_heads;
    const int group0 = blockIdx.x / a.v.kv_heads * kGroup;     // the workgroup's first page
    const int page0 = group0 + wave / SHARE * PAGES;
    const int64_t out = (int64_t(s) * a.v.kv_heads + hk) * a.max_kv;
    if (group0 * kPage >= a.v.len(s)) {   // beyond the sequence: most workgroups where lengths differ much
        for (int64_t j = int64_t(group0) * kPage + threadIdx.x; j < min(a.max_kv, int64_t(group0 + kGroup) * kPage); j += 256)
            a.weights[out + j] = 0.0f;
        return;
    }
    const QueryRows rows(a.v, a.sc, s);

    // rows that see any slot of the workgroup's pages
    const int first = group0 * kPage, past = first + kGroup * kPage, shift = rows.len - rows.new_tokens;
    int i_lo = 0, i_hi = first < rows.len && a.v.pages > 0 ? rows.new_tokens : 0;
    if (a.sc.causal) i_lo = max(0, first - shift);
    if (a.sc.window > 0) i_hi = min(i_hi, max(0, past - 1 + a.sc.window - shift));
    const int r_lo = i_lo * rows.group, r_hi = i_hi * rows.group;

    // lane x has the id of page x
    int ids = -1;
    if (r_lo < r_hi && lane < PAGES && (page0 + lane) * kPage < rows.len) ids = a.v.page_id(s, page0 + lane);
    KRegs<D> raw;
    if (r_lo < r_hi) raw.load(a.v.record_or_first<D>(__builtin_amdgcn_readlane(ids, 0), hk), n, b);
    auto my_slot = [&](int x) { return (page0 + x) * kPage + KRegs<D>::slot(b, n); };   // that this lane writes
#pragma unroll
    for (int x = 0; x < PAGES; ++x) sums[wave][x][lane] = f32x4{0, 0, 0, 0};
    auto decode = [&](f16x8 (&k)[4][D / 32]) {
        raw.template decode<0, 0>(k[0]);
        raw.template decode<1, 0>(k[1]);
        raw.template decode<2, 0>(k[2]);
        raw.template decode<3, 0>(k[3]);
    };
    // the rows r0 .. of the block over page x, whose K is k
    auto look = [&](const f16x8 (&k)[4][D / 32], int x, int r0) {
        const int tiles = (min(r_hi - r0, Block::kRows) + 15) / 16;
        if (!a.v.has(__builtin_amdgcn_readlane(ids, x))) return;
        f32x4 sum = sums[wave][x][lane];
        const int base = (page0 + x) * kPage;
        // Tokens in order see ever later slots: those from see_lo on and before see_hi see
        // all of the page, and so do their rows (and those past the last, which give nothing).
        const int see_lo = a.sc.causal ? min(max(base + kPage - 1 - shift, 0), rows.new_tokens) : 0;
        const int see_hi = a.sc.window > 0 ? max(base + a.sc.window - shift, 0) : rows.new_tokens;
        const bool simple = a.sc.cap == 0.0f && base + kPage <= rows.len;
        const int full_lo = simple ? (see_lo * rows.group - r0 + 15) / 16 : tiles;   // in tiles
        const int full_hi = see_hi >= rows.new_tokens ? tiles : (see_hi * rows.group - r0) / 16;
        const int t_lo = min(max(full_lo, 0), tiles), t_hi = max(min(full_hi, tiles), t_lo);

        auto products = [&](int t, f32x4 (&z)[4]) {
#pragma unroll
            for (int ht = 0; ht < 4; ++ht) z[ht] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const f16x8 q = block.q[Block::chunk_at(16 * t + n, b * (D / 32) + i)];
#pragma unroll
                for (int ht = 0; ht < 4; ++ht) z[ht] = __builtin_amdgcn_mfma_f32_16x16x32_f16(q, k[ht][i], z[ht], 0, 0, 0);
            }
        };
        auto add_full = [&](int t, const f32x4 (&z)[4]) {
            const f32x4 f = *reinterpret_cast<const f32x4*>(block.f + 16 * t + 4 * b);
            const f32x4 lse = *reinterpret_cast<const f32x4*>(block.lse + 16 * t + 4 * b);
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int ht = 0; ht < 4; ++ht) sum[ht] += __builtin_amdgcn_exp2f(__builtin_fmaf(z[ht][c], f[c], -lse[c]));
        };
        auto add_seen = [&](int t, const f32x4 (&z)[4]) {
            int n = lane & 15, b = lane >> 4;
            asm volatile("" : "+v"(n), "+v"(b));   // what follows from them is found anew: kept beside the tiles it would not fit the registers
            const f32x4 f = *reinterpret_cast<const f32x4*>(block.f + 16 * t + 4 * b);
            const f32x4 lse = *reinterpret_cast<const f32x4*>(block.lse + 16 * t + 4 * b);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int lo = block.lo[16 * t + 4 * b + c], hi = block.hi[16 * t + 4 * b + c];
                float y[4] = {z[0][c], z[1][c], z[2][c], z[3][c]};
                a.sc.shape(y, f[c]);
#pragma unroll
                for (int ht = 0; ht < 4; ++ht) {
                    const int slot = base + KRegs<D>::slot(ht, n);
                    const float p = __builtin_amdgcn_exp2f(y[ht] - lse[c]);
                    sum[ht] += slot >= lo && slot < hi ? p : 0.0f;
                }
            }
        };
        f32x4 z[4];
        int t = wave % SHARE;
#pragma unroll 1
        for (; t < t_lo; t += SHARE) products(t, z), add_seen(t, z);
#pragma unroll 1
        for (; t < t_hi; t += SHARE) products(t, z), add_full(t, z);
#pragma unroll 1
        for (; t < tiles; t += SHARE) products(t, z), add_seen(t, z);
        sums[wave][x][lane] = sum;
    };
    auto stage = [&](int r0) {
        if (r0 != r_lo) __syncthreads();
        block.fill(a, rows, hk, r0);
        __syncthreads();
    };
    if constexpr (PAGES == 1) {   // decoded once for all rows
        f16x8 k[4][D / 32];
        if (r_lo < r_hi) decode(k);
        for (int r0 = r_lo; r0 < r_hi; r0 += Block::kRows) {
            stage(r0);
            look(k, 0, r0);
        }
    } else if (r_lo < r_hi) {     // one block has all rows
        stage(r_lo);
#pragma unroll 1
        for (int x = 0; x < PAGES; ++x) {
            f16x8 k[4][D / 32];
            decode(k);
            raw.load(a.v.record_or_first<D>(__builtin_amdgcn_readlane(ids, min(x + 1, PAGES - 1)), hk), n, b);
            look(k, x, r_lo);
        }
    }
    if constexpr (SHARE > 1) {
        __syncthreads();
        if (wave % SHARE > 0) return;
    }
    // a lane of group b has tile b's slot n of each page
    float before[PAGES];
#pragma unroll
    for (int x = 0; x < PAGES; ++x) before[x] = a.prior ? a.prior[out + min(int64_t(my_slot(x)), a.max_kv - 1)] : 0.0f;
#pragma unroll
    for (int x = 0; x < PAGES; ++x) {
        f32x4 sum = sums[wave][x][lane];
#pragma unroll
        for (int w = 1; w < SHARE; ++w) sum += sums[wave + w][x][lane];
#pragma unroll
        for (int ht = 0; ht < 4; ++ht) {
            sum[ht] += __shfl_xor(sum[ht], 16);
            sum[ht] += __shfl_xor(sum[ht], 32);
        }
        const float w = b < 2 ? (b == 0 ? sum[0] : sum[1]) : (b == 2 ? sum[2] : sum[3]);
        const int slot = my_slot(x);
        if (slot < a.max_kv) a.weights[out + slot] = slot < rows.len ? before[x] + w : 0.0f;
    }
}

template <int D>
int launch_weights(const WeightArgs& a, int64_t rows, hipStream_t st) {
    // Up to 32 rows a kv head: one page a wavefront where the cache has few, so
    // that all are under way at once, two where it has many (16 sequences of
    // 100 .. 16383 slots, 8 heads: 15.4 us with one, 13.7 with two, 14.3 with
    // four; 4 sequences: 7.1, 8.3, 10.0).
    // More rows: one page a wavefront, decoded once for all blocks of rows
    // (4 sequences of 4096 slots, 2048 rows of 8 heads: 139 us; a page a workgroup
    // 227, four a wavefront 396).  One a workgroup, whose wavefronts take every fourth
    // tile of the rows, where there are fewer workgroups than CUs (1 sequence:
    // 110, 74, 394).  Four a wavefront where one block holds the rows, which is then
    // staged once for all of them, and the card is full with such (16384 slots,
    // 128 rows: 39, 75, 31).
    constexpr int kRows = D == 256 ? 64 : 128;   // LDS holds no more for two workgroups at D = 256
    const int64_t each = (a.max_kv + kPage - 1) / kPage, all = each * a.v.kv_heads * a.v.seqs;
    const int pages = rows <= 32 ? (all > 8192 ? 8 : 4) : all < 4 * 256 ? 1 : rows <= kRows && all >= 16 * 256 ? 16 : 4;   // of a workgroup
    const int64_t blocks = (each + pages - 1) / pages * a.v.kv_heads;
    if (blocks > 0x7fffffff) return NVFP4_ERR_SHAPE;
    const auto kernel = rows <= 32   ? (pages == 4 ? kv_weights_kernel<D, 1, 32, 1> : kv_weights_kernel<D, 2, 32, 1>)
                        : pages == 1 ? kv_weights_kernel<D, 1, kRows, 4>
                        : pages == 4 ? kv_weights_kernel<D, 1, kRows, 1>
                                     : kv_weights_kernel<D, 4, kRows, 1>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks), a.v.seqs), dim3(256), 0, st, a);
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

// fp32 to a key that orders as the numbers do; -0 is 0, NaN is -inf.  None is below 0x7fffff.
__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = f32_bits(fmaxf(x, -INFINITY) + 0.0f);
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}

constexpr uint32_t kZeroKey = 0x80000000u;

constexpr int kSelect = 1024;
constexpr int kSelectWaves = kSelect / 64;
constexpr int kSelectBins = 2048;

// A lane's value plus those of all lanes before it, by moves between lanes.
__device__ __forceinline__ uint32_t scan32(uint32_t x) {
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x111, 0xf, 0xf, false));   // 1, 2, 4, 8 lanes within a row of 16
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x112, 0xf, 0xf, false));
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x114, 0xf, 0xf, false));
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x118, 0xf, 0xf, false));
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x142, 0xa, 0xf, false));   // a row's last into the next
    x += uint32_t(__builtin_amdgcn_update_dpp(0, int(x), 0x143, 0xc, 0xf, false));   // the first half's last into the second
    return x;
}

// The keys of one (sequence, head): wavefront w has the slots
// [w, w + 1) * span, 64 neighbours at a time.  A slot outside the choice
// [lo, hi) has key 0, below every weight's.  HELD > 0: the keys stay in HELD
// registers a lane and SHARED places of LDS; 0: the weights are read again each
// time.
template <int HELD, int SHARED>
struct Keys {
    const float* w;
    uint32_t* shared;
    int lo, hi, begin, end;   // begin, end: of this wavefront
    uint32_t held[HELD > 0 ? HELD : 1];

    __device__ __forceinline__ Keys(const float* weights, uint32_t* lds, int n, int first, int past)
        : w(weights), shared(lds), lo(first), hi(past) {
        const int span = (n + kSelect - 1) / kSelect * 64;   // at most (HELD + SHARED) * 64, by the choice of HELD
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
        begin = min(wave * span, n), end = min(begin + span, n);
        if constexpr (HELD > 0) {
#pragma unroll
            for (int i = 0; i < SHARED; ++i) {
                const int j = begin + (HELD + i) * 64 + lane;
                const float x = w[min(j, n - 1)];
                shared[i * kSelect + threadIdx.x] = j >= lo && j < hi ? order_key(x) : 0;
            }
#pragma unroll
            for (int i = 0; i < HELD; ++i) held[i] = f32_bits(w[min(begin + i * 64 + lane, n - 1)]);
#pragma unroll
            for (int i = 0; i < HELD; ++i) {
                const int j = begin + i * 64 + lane;
                held[i] = order_key(bits_f32(held[i]));
                if (begin + i * 64 < lo || begin + i * 64 + 64 > hi) held[i] = j >= lo && j < hi ? held[i] : 0;
            }
        }
    }
    // fn(slot, key) for every 64 slots of the wavefront, all lanes together
    template <class Fn>
    __device__ __forceinline__ void each(Fn fn) const {
        const int lane = threadIdx.x & 63;
        if constexpr (HELD > 0) {
            int last = end;
            asm volatile("" : "+s"(last));   // compared anew: kept from one walk to the next, the results would fill the registers
#pragma unroll
            for (int i = 0; i < HELD; ++i)
                if (begin + i * 64 < last) fn(begin + i * 64 + lane, held[i]);
            for (int i = 0; i < SHARED && begin + (HELD + i) * 64 < last; ++i)
                fn(begin + (HELD + i) * 64 + lane, shared[i * kSelect + threadIdx.x]);
        } else {
            for (int j0 = begin; j0 < end; j0 += 64) {
                const int j = j0 + lane;
                fn(j, j >= lo && j < hi ? order_key(w[j]) : 0);
            }
        }
    }
};

// Which slots stay: one workgroup a (sequence, head).  Bound by instructions on
// the CUs that have one (65000 slots of a head: 39 us, of which the first digits
// take 8 and the numbering 9).
template <int HELD, int SHARED>
__global__ void __launch_bounds__(kSelect)
kv_select_kernel(EvictArgs a) {
    __shared__ uint32_t more[SHARED > 0 ? SHARED * kSelect : 1];
    __shared__ uint32_t bins[kSelectBins];
    __shared__ uint32_t tmp[kSelectWaves][2];
    __shared__ uint32_t found[2];
    const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int n = a.len(s);
    const int64_t seq_head = int64_t(s) * a.v.kv_heads + h;
    const float* w = a.weights + seq_head * a.weights_pitch;
    int32_t* kept = a.kept + seq_head * a.keep;
    float* kept_w = a.kept_weights + seq_head * a.keep;
    if (h == 0 && tid == 0) a.new_lens[s] = min(n, a.keep);
    // slots that stay whatever they weigh: all, or the first and the last ones
    const bool all = n <= a.keep;
    const int lo = all ? n : a.sink, hi = all ? n : n - a.recent;   // the choice is among [lo, hi)
    const int wanted = all ? 0 : a.keep - a.sink - a.recent;
    for (int i = tid; i < a.keep; i += kSelect) {
        if (i >= lo && i < lo + wanted) continue;
        const int j = i < lo ? i : i - lo - wanted + hi;
        kept[i] = j < n ? j : -1;
        kept_w[i] = j < n ? w[j] : 0.0f;
    }
    if (wanted == 0) return;
    const Keys<HELD, SHARED> keys(w, more, n, lo, hi);
    // the key of the last slot that is chosen, 11, 11 and 10 bits at a time
    uint32_t need = uint32_t(wanted), mask = 0, key = 0;
    auto clear = [&] {
        bins[tid] = bins[tid + kSelect] = 0;
        __syncthreads();
    };
    // the bin in which the last of them lies: the next bits of the key
    auto settle = [&](int shift, uint32_t digits) {
        __syncthreads();
        // thread t has bins 2 (1023 - t) + 1 and 2 (1023 - t): the highest first
        const int at = 2 * (kSelect - 1 - tid);
        const uint32_t high = bins[at + 1], low = bins[at];
        const uint32_t sum = scan32(high + low);
        if (lane == 63) tmp[wave][0] = sum;
        __syncthreads();
        uint32_t before = sum - high - low;
        for (int i = 0; i < wave; ++i) before += tmp[i][0];
        if (before < need && before + high >= need)
            found[0] = uint32_t(at + 1), found[1] = need - before;
        else if (before + high < need && before + high + low >= need)
            found[0] = uint32_t(at), found[1] = need - before - high;
        __syncthreads();
        key |= found[0] << shift;
        mask |= digits << shift;
        need = found[1];   // still wanted among the keys with these leading bits
    };
    // A slot outside the choice has a digit below every other's.  The many zeros of
    // a fresh cache would all meet in one place: a wavefront adds its own at once.
    clear();
    uint32_t zeros = 0;
    keys.each([&](int, uint32_t k) {
        if (k != kZeroKey)
            atomicAdd(&bins[k >> 21], 1u);
        else
            ++zeros;
    });
    zeros = scan32(zeros);
    if (lane == 63 && zeros > 0) atomicAdd(&bins[kZeroKey >> 21], zeros);
    settle(21, 2047);
    // What is left may be the same number: a lane adds a run of equal digits at once.
#pragma unroll 1
    for (int shift = 10; shift >= 0; shift -= 10) {
        const uint32_t digits = shift > 0 ? 2047 : 1023;
        clear();
        uint32_t digit = 0, run = 0;
        keys.each([&](int, uint32_t k) {
            if ((k & mask) != key) return;
            const uint32_t d = (k >> shift) & digits;
            if (d != digit) {
                if (run > 0) atomicAdd(&bins[digit], run);
                digit = d, run = 0;
            }
            ++run;
        });
        if (run > 0) atomicAdd(&bins[digit], run);
        settle(shift, digits);
    }
    // `need` of the slots at the key stay, the lowest first.  Wavefronts count
    // theirs, then number them from where those before them end.
    uint32_t mine = 0, ties = 0;
    keys.each([&](int, uint32_t k) {
        mine += uint32_t(k > key);
        ties += uint32_t(k == key);
    });
    mine = scan32(mine), ties = scan32(ties);
    if (lane == 63) tmp[wave][0] = mine, tmp[wave][1] = ties;
    __syncthreads();
    uint32_t above = 0, seen = 0;   // chosen slots and ties before
    for (int i = 0; i < wave; ++i) above += tmp[i][0], seen += tmp[i][1];
    key = uint32_t(__builtin_amdgcn_readfirstlane(int(key)));
    asm("" : "+s"(key));   // compared anew: kept from the count, the comparisons' results would fill the registers
    auto before = [&](uint64_t lanes) { return __builtin_amdgcn_mbcnt_hi(uint32_t(lanes >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(lanes), 0)); };
    // Of many slots the weights are fetched afterwards, together: fetched and
    // stored one after the other they would be waited for at every step.
    constexpr bool kAtOnce = HELD > 0 && HELD <= 16;
    auto keep = [&](uint32_t to, int j) {
        kept[to] = j;
        if constexpr (kAtOnce) kept_w[to] = w[j];
    };
    keys.each([&](int j, uint32_t k) {
        const uint64_t high = __ballot(k > key), equal = __ballot(k == key);
        if (!(high | equal)) return;
        if (!equal) {
            if (k > key) keep(uint32_t(lo) + above + min(seen, need) + before(high), j);
        } else {
            const uint32_t rank = seen + before(equal);
            if (k > key || (k == key && rank < need)) keep(uint32_t(lo) + above + before(high) + min(rank, need), j);
            seen += uint32_t(__popcll(equal));
        }
        above += uint32_t(__popcll(high));
    });
    if constexpr (!kAtOnce) {
        __syncthreads();
        for (int i = lo + tid; i < lo + wanted; i += kSelect) kept_w[i] = w[kept[i]];
    }
}

// The rows that stay, one destination page a workgroup.  Bound by its loads: a
// row's V lies in dwords of 8 slots at each dim, so 8 times its codes are loaded
// (8 sequences of up to 65000 slots cut to 4000, 8 heads of 128: 40 us for 37
// MB of pages, of whose sources 104 MB come from beyond L2).
// Threads of it: 16 bytes of K and 4 dwords of V each (at D = 256 half as many
// threads took 19.9 us instead of 16.0 for one sequence cut to 256 slots).
template <int D>
constexpr int kMoveThreads = 2 * D;

template <int D>
__global__ void __launch_bounds__(kMoveThreads<D>)
kv_move_kernel(EvictArgs a) {
    using R = KvRecord<D>;
    __shared__ const uint8_t* from[kPage];
    __shared__ int slot_in[kPage];
    __shared__ bool live[kPage];
    const int s = blockIdx.y, tid = threadIdx.x;
    const int h = blockIdx.x % a.v.kv_heads, page = blockIdx.x / a.v.kv_heads;
    // the length, the kept slots and the page they go to are asked for together
    const int at = page * kPage + (tid & 63);
    const int j = max(a.kept[(int64_t(s) * a.v.kv_heads + h) * a.keep + min(at, a.keep - 1)], 0);
    const int64_t to_page = a.dst_table[int64_t(s) * a.dst_pitch + page];
    const int id = a.v.page_id(s, min(j / kPage, static_cast<int>(a.v.table_pitch) - 1));
    const int n = min(a.len(s), a.keep);
    if (page * kPage >= n) return;
    if (to_page < 0 || to_page >= a.dst_pages) return;
    uint8_t* to = a.dst + (to_page * a.v.kv_heads + h) * R::kBytes;
    if (tid < kPage) {
        live[tid] = at < n && a.v.has(id);
        from[tid] = a.v.pages > 0 ? a.v.record_or_first<D>(id, h) : to;   // (a cache without pages has no live slot)
        slot_in[tid] = j % kPage;
    }
    __syncthreads();
    // All loads first, from a place that is there in any case: with a branch
    // around each they would wait for one another.
    constexpr int kThreads = kMoveThreads<D>, kKParts = kPage * (D / 32) / kThreads, kVDwords = 8 * D / kThreads;
    u32x4 kc[kKParts];
#pragma unroll
    for (int i = 0; i < kKParts; ++i) {   // K codes, 16 bytes each
        const int slot = (i * kThreads + tid) / (D / 32), part = (i * kThreads + tid) % (D / 32);
        kc[i] = load16(from[slot] + R::k_code(slot_in[slot]) + 16 * part);
    }
    uint32_t vc[kVDwords][8];
#pragma unroll
    for (int i = 0; i < kVDwords; ++i) {   // V codes: a dword is 8 slots at a dim
        const int block = (i * kThreads + tid) / D, dim = (i * kThreads + tid) % D;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int j = slot_in[8 * block + e];
            vc[i][e] = *reinterpret_cast<const uint32_t*>(from[8 * block + e] + R::v_code(j / 8, dim));
        }
    }
    // scales, as whole words of the page (a byte at a time: 4 us more of the kernel's 40)
    constexpr int kPerDims = D / 64;   // bytes of a slot in a word of K's
    if (tid < 8 * R::kGroups) {        // V: the 8 slots of a block and group
        const int block = tid / R::kGroups, g = tid % R::kGroups;
        uint64_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int slot = 8 * block + e, j = slot_in[slot];
            const uint64_t x = from[slot][R::v_scale(j / 8, g) + j % 8];
            w |= (live[slot] ? x : 0) << (8 * e);
        }
        *reinterpret_cast<uint64_t*>(to + R::v_scale(block, g)) = w;
    } else if (tid >= kThreads - 64) {   // K: the slots 8 a + r + 4 t + 32 h at a quarter of the dims
        const int row = (tid & 63) / 4, quarter = tid & 3, slot0 = 8 * (row / 4) + row % 4;
        uint8_t w[4 * kPerDims];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int slot = slot0 + 32 * (e >> 1) + 4 * (e & 1);
            uint32_t x = 0;
            __builtin_memcpy(&x, __builtin_assume_aligned(from[slot] + R::k_scale(slot_in[slot], quarter * kPerDims), kPerDims), kPerDims);
            x = live[slot] ? x : 0;
            __builtin_memcpy(w + e * kPerDims, &x, kPerDims);
        }
        __builtin_memcpy(__builtin_assume_aligned(to + R::k_scale(slot0, quarter * kPerDims), 4 * kPerDims), w, 4 * kPerDims);
    }
#pragma unroll
    for (int i = 0; i < kKParts; ++i) {
        const int slot = (i * kThreads + tid) / (D / 32), part = (i * kThreads + tid) % (D / 32);
        const u32x4 none = {0, 0, 0, 0};
        *reinterpret_cast<u32x4*>(to + R::k_code(slot) + 16 * part) = live[slot] ? kc[i] : none;
    }
#pragma unroll
    for (int i = 0; i < kVDwords; ++i) {
        const int block = (i * kThreads + tid) / D, dim = (i * kThreads + tid) % D;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int slot = 8 * block + e;
            w |= (live[slot] ? vc[i][e] >> (4 * (slot_in[slot] % 8)) & 15u : 0u) << (4 * e);
        }
        *reinterpret_cast<uint32_t*>(to + R::v_code(block, dim)) = w;
    }
}

template <int D>
int launch_move(const EvictArgs& a, hipStream_t st) {
    const int64_t blocks = int64_t((a.keep + kPage - 1) / kPage) * a.v.kv_heads;
    if (blocks > 0x7fffffff) return NVFP4_ERR_SHAPE;
    hipLaunchKernelGGL(kv_move_kernel<D>, dim3(static_cast<unsigned>(blocks), a.v.seqs), dim3(kMoveThreads<D>), 0, st, a);
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
        case 64: return launch_weights<64>(a, queries->max_q * a.sc.group, s);
        case 128: return launch_weights<128>(a, queries->max_q * a.sc.group, s);
        default: return launch_weights<256>(a, queries->max_q * a.sc.group, s);
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
    if (dst->k_scale != cache->k_scale || dst->v_scale != cache->v_scale) return NVFP4_ERR_SHAPE;   // codes are copied as they are
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
    // Keys held up to 65536 slots a sequence (51 in registers and 13 in LDS a lane, which is what a
    // 1024-thread workgroup's registers take) and read once; of longer sequences they are read five
    // times (8 sequences of up to 65000 slots, 8 heads: 92 us instead of 39).
    const int64_t longest = std::min(weights_pitch, seqs->table_pitch * kPage);
    const auto select = longest <= 4 * kSelect    ? kv_select_kernel<4, 0>
                        : longest <= 16 * kSelect ? kv_select_kernel<16, 0>
                        : longest <= 64 * kSelect ? kv_select_kernel<51, 13>
                                                  : kv_select_kernel<0, 0>;
    hipLaunchKernelGGL(select, dim3(cache->kv_heads, static_cast<unsigned>(seqs->seqs)), dim3(kSelect), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    switch (cache->head_dim) {
        case 64: return launch_move<64>(a, s);
        case 128: return launch_move<128>(a, s);
        default: return launch_move<256>(a, s);
    }
}
