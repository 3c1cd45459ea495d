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

#include <cstdint>

#include "../host/draft_shapes.h"
#include "../host/kv_index.h"
#include "../host/kv_plan.h"
#include "../host/kv_shapes.h"
#include "../host/tree_plan.h"
#include "kv_common.h"
#include "kv_pages.h"
#include "kv_scores.h"
#include "setup.h"

namespace {

constexpr int kWaves = nvfp4::kKvWaves, kRowTile = nvfp4::kKvRowTile, kTileRows = nvfp4::kKvTileRows;
constexpr int kItems = nvfp4::kKvItems;

struct AttendArgs {
    KvView v;
    KvScores sc;
    uint16_t* out;
    float* lse;
    float* part_o;    // [splits][total * heads][D]: sums of exp2(z - m) v, without the V scale
    float* part_ml;   // [splits][total * heads][2]: m and the sum of exp2(z - m)
    int tile;         // rows of a many-row workgroup, 0: few rows
    int splits;       // workgroups over the pages of a row tile, `chunk` pages each
    int chunk;
    int row_tiles;    // of the longest sequence (tile: that there can be)
    int32_t* plan;    // few rows: the planned items (kv_plan_kernel), or NULL where splits and chunk say all
    float v_scale;
    int group0;       // first workgroup of the launch (launch_sliced)
};

// This workgroup's number among all of the grid's first axis.
__device__ __forceinline__ int group_of(const AttendArgs& a) { return a.group0 + static_cast<int>(blockIdx.x); }

__device__ __forceinline__ int pages_lo(const Span& s) { return s.lo / kPage; }
__device__ __forceinline__ int pages_hi(const Span& s) { return (s.hi + kPage - 1) / kPage; }

// Tile: the workgroups that take the pages of a row tile (at least one).
__device__ __forceinline__ int used_splits(const AttendArgs& a, const Span& s) {
    return min(max((pages_hi(s) - pages_lo(s) + a.chunk - 1) / a.chunk, 1), a.splits);
}

// Few rows.  A segment is one row tile and kv head of a sequence: the pages
// its rows see, at least one.  Segments are cut into chunks of the same number
// of pages, and each chunk is a workgroup's item.  Where the host's bound on
// the lengths does not leave many workgroups without work, the grid itself
// numbers the items: parts x sequences x segments.  Else a first kernel counts
// them from the lengths: the whole chunks of all segments, then what is left
// at the segments' ends, so that long and short sequences together keep the
// card evenly busy to the end.  (A workgroup without work still holds its
// registers and LDS while it reads a length: 32 one-token steps over 3 ..
// 131071 slots took 178 us with 14000 such, 124 us planned, of which the plan
// takes 5 us.)
template <class Rows>
__device__ __forceinline__ int segment_pages(const AttendArgs& a, const Rows& rows) {
    const Span span = rows.span(a.sc, 0, rows.count - 1);
    return max(pages_hi(span) - pages_lo(span), 1);
}

template <class Rows>
__device__ __forceinline__ int segment_count(const AttendArgs& a, const Rows& rows) {
    return (rows.count + kRowTile - 1) / kRowTile * a.v.kv_heads;
}

constexpr int kPlanThreads = 1024;

// plan: [0] the chunk, [1] the number of whole chunks, [2 + s] the whole chunks
// before sequence s, [2 + seqs + s] the rests before it.
__global__ void __launch_bounds__(kPlanThreads)
kv_plan_kernel(AttendArgs a) {
    __shared__ int64_t tmp[kPlanThreads / 64][2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // sums of x and y over the threads before this one; the totals are added to all_x and all_y
    auto scan = [&](int64_t x, int64_t y, int64_t* before_x, int64_t* before_y, int64_t* all_x, int64_t* all_y) {
        int64_t sx = x, sy = y;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t ux = __shfl_up(sx, d), uy = __shfl_up(sy, d);
            if (lane >= d) sx += ux, sy += uy;
        }
        __syncthreads();
        if (lane == 63) tmp[wave][0] = sx, tmp[wave][1] = sy;
        __syncthreads();
        int64_t bx = *all_x, by = *all_y, ax = bx, ay = by;
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < wave) bx += tmp[w][0], by += tmp[w][1];
            ax += tmp[w][0], ay += tmp[w][1];
        }
        *before_x = bx + sx - x, *before_y = by + sy - y, *all_x = ax, *all_y = ay;
    };
    int64_t all = 0, none = 0, b0, b1;
    for (int s = tid; s - tid < a.v.seqs; s += kPlanThreads) {
        int64_t size = 0;
        if (s < a.v.seqs) {
            const QueryRows rows(a.v, a.sc, s);
            if (rows.count > 0) size = int64_t(segment_count(a, rows)) * segment_pages(a, rows);
        }
        scan(size, 0, &b0, &b1, &all, &none);
    }
    // about kItems chunks, none shorter than the host's
    const int chunk = static_cast<int>(max((all + kItems - 1) / kItems, int64_t(a.chunk)));
    int64_t whole = 0, rest = 0;
    for (int s = tid; s - tid < a.v.seqs; s += kPlanThreads) {
        int64_t w = 0, r = 0;
        if (s < a.v.seqs) {
            const QueryRows rows(a.v, a.sc, s);
            if (rows.count > 0) {
                const int pages = segment_pages(a, rows), count = segment_count(a, rows);
                w = int64_t(count) * (pages / chunk), r = pages % chunk ? count : 0;
            }
        }
        scan(w, r, &b0, &b1, &whole, &rest);
        if (s < a.v.seqs) a.plan[2 + s] = static_cast<int>(b0), a.plan[2 + a.v.seqs + s] = static_cast<int>(b1);
    }
    if (tid == 0) a.plan[0] = chunk, a.plan[1] = static_cast<int>(whole);
}

struct Item {
    int s, segment, part, chunk;   // s < 0: none
};

// The last of the ascending p[0 .. n) that is at most w, by 64 at a time.
__device__ __forceinline__ int last_at_most(const int32_t* p, int n, int w) {
    const int lane = threadIdx.x & 63;
    int at = 0;
    for (int step = n > 4096 ? 4096 : n > 64 ? 64 : 1;; step /= 64) {
        const int i = at + lane * step;
        at += (__popcll(__ballot(i < n && p[i] <= w)) - 1) * step;
        if (step == 1) return at;
    }
}

__device__ __forceinline__ Item find_item(const AttendArgs& a, int w) {
    const int segments = a.row_tiles * a.v.kv_heads;
    if (!a.plan) return Item{w / segments % a.v.seqs, w % segments, w / segments / a.v.seqs, a.chunk};
    const int chunk = a.plan[0], whole = a.plan[1];
    const bool rest = w >= whole;
    if (rest) w -= whole;
    const int32_t* before = a.plan + 2 + (rest ? a.v.seqs : 0);
    const int s = last_at_most(before, a.v.seqs, w), in = w - before[s];
    // the last of equal entries is the one that has items, unless w lies after all
    const QueryRows rows(a.v, a.sc, s);
    if (rows.count == 0) return Item{-1, 0, 0, 0};
    const int pages = segment_pages(a, rows), each = rest ? (pages % chunk != 0) : pages / chunk;
    if (each == 0 || in >= each * segment_count(a, rows)) return Item{-1, 0, 0, 0};
    return Item{s, in / each, rest ? pages / chunk : in % each, chunk};
}

// A row of sums in LDS: 16 bytes more than its dims, so that the 16 rows that are
// written at once begin on different banks.
template <int D>
constexpr int kSumRow = D + 4;

// 16 query rows and one item's pages: the wavefronts take every fourth page,
// decoded from registers, and join in LDS in wavefront order.  A long cache is
// bound by its reads (32 one-token steps of 32 heads over 3 .. 131071 slots of 8
// heads of 128: 103 us for 575 MB, 5.6 TB/s with what the memory-side cache
// kept), a short one by the chain of dependent reads and one page's work (777
// slots: 10 us; at D = 256 that work and 16 rows of sums in 241 registers leave
// two wavefronts a SIMD: 16 verify rounds of 5 tokens in a window of 1500 take 24 us for 40 MB).
template <int D, bool TREE>
__global__ void __launch_bounds__(64 * kWaves, 2)
kv_attend_rows_kernel(AttendArgs a) {
    extern __shared__ float lds[];   // [kWaves][16][kSumRow<D>] sums, then [kWaves][16][2] statistics
    // the wavefront's number as a scalar: its pages and their addresses are then scalars too
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int n = lane & 15, b = lane >> 4;
    const Item item = find_item(a, group_of(a));
    if (item.s < 0) return;
    const int s = item.s, hk = item.segment % a.v.kv_heads, row0 = item.segment / a.v.kv_heads * kRowTile;
    const QueryRowsOf<TREE> rows(a.v, a.sc, s);
    if (row0 >= rows.count) return;
    const int pages = segment_pages(a, rows);
    if (item.part > 0 && item.part * item.chunk >= pages) return;
    const Span whole = rows.span(a.sc, 0, rows.count - 1), span = rows.span(a.sc, row0, min(row0 + kRowTile, rows.count) - 1);
    const int begin = pages_lo(whole) + item.part * item.chunk, end = min(begin + item.chunk, pages_hi(whole));

    // Page numbers are read 64 at a time, one a lane, so that a page's loads
    // never wait for the table.  The next page's K is on its way once the
    // scores are formed, its V once the sums are: one set of registers, with
    // which three wavefronts a SIMD cover the wait at D = 128, measured better
    // than two sets and two wavefronts.
    int page = begin + wave, ids = -1, at_id = 0, id = -1;
    auto read_ids = [&](int p) {
        const int mine = p + kWaves * lane;
        ids = mine < end ? a.v.page_id(s, mine) : -1;
        at_id = 0;
    };
    PageRegs<D, !TREE> cur;   // a tree's row tiles read the same pages
    const bool any = page < end && a.v.pages > 0;
    if (any) {
        read_ids(page);
        id = __builtin_amdgcn_readlane(ids, at_id++);
        const uint8_t* rec = a.v.record_or_first<D>(id, hk);
        cur.load_k(rec, n, b);
        cur.load_v(rec, n, b);
    }
    const QueryRow me = rows.row(a.sc, row0 + n);
    f16x8 q[D / 32];
    const float to_log2 = load_query<D / 32, 8, 16>(a.sc, query_at(a.sc, me, hk) + b * (D / 4), q);

    f32x4 o[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    if (any) __builtin_amdgcn_s_waitcnt(0x0f70);   // all loads: the loop's waits then count its own alone
    while (page < end && a.v.pages > 0) {
        const int base = page * kPage;
        const bool here = a.v.has(id);
        f32x4 z[4];
        z[0] = score_groups<D, !TREE, 0, 0>(cur, q, f32x4{0, 0, 0, 0});
        z[1] = score_groups<D, !TREE, 1, 0>(cur, q, f32x4{0, 0, 0, 0});
        z[2] = score_groups<D, !TREE, 2, 0>(cur, q, f32x4{0, 0, 0, 0});
        z[3] = score_groups<D, !TREE, 3, 0>(cur, q, f32x4{0, 0, 0, 0});
        if (at_id == 64) read_ids(page + kWaves);
        id = __builtin_amdgcn_readlane(ids, at_id++);
        const uint8_t* next = a.v.record_or_first<D>(id, hk);
        cur.load_k(next, n, b);
        float p[16];   // [h][8 consecutive slots]
#pragma unroll
        for (int i = 0; i < 16; ++i) p[i] = z[i >> 2][i & 3];
        a.sc.shape(p, to_log2);
        if (!here || base < span.lo_all || base + kPage > span.hi_all) {
            if constexpr (TREE) {
                int r = row0 + n;   // worked out anew: kept, what follows from it would cost a wavefront a SIMD
                asm volatile("" : "+v"(r));
                const QueryRow who = rows.row(a.sc, r);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t seen = here ? rows.seen8(a.sc, who, base + 32 * h + 8 * b) : 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[8 * h + i] = seen >> i & 1 ? p[8 * h + i] : -INFINITY;
                }
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int slot = base + 32 * (i >> 3) + 8 * b + (i & 7);
                    p[i] = here && slot >= me.lo && slot < me.hi ? p[i] : -INFINITY;
                }
            }
        }
        float top = p[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, p[i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        if (__any(top > m + kSlack)) {
            const float grown = fmaxf(m, top);
            const float keep = grown == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
            m = grown;
            l *= keep;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) o[i] *= keep;
        }
        const float base_m = m == -INFINITY ? 0.0f : m - kLift;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            p[i] = __builtin_amdgcn_exp2f(p[i] - base_m);
            l += p[i];
        }
        // slots from the length on hold anything, and so does the page that stands in for none: their scales become 0
        const int left = here ? rows.len - base : 0;
        if (left < kPage) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int live = left - 32 * h - 8 * b;
                const uint64_t mask = live <= 0 ? 0 : live >= 8 ? ~0ull : (1ull << (8 * live)) - 1;
                cur.vs[h][0] &= uint32_t(mask);
                cur.vs[h][1] &= uint32_t(mask >> 32);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f16x8 pt = to_f16x8(p + 8 * h);
            const f16x2 sc[4] = {scale_pair<0>(cur.vs[h][0]), scale_pair<1>(cur.vs[h][0]),
                                 scale_pair<0>(cur.vs[h][1]), scale_pair<1>(cur.vs[h][1])};
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                o[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_slots(cur.v[h][i], sc), pt, o[i], 0, 0, 0);
        }
        cur.load_v(next, n, b);
        page += kWaves;
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (l != l && m == -INFINITY) m = 0.0f;   // all scores NaN: the row stays NaN
    m -= kLift;                               // what the sums are held against

    // The wavefronts' results meet in LDS and are joined in wavefront order.
    float* sums = lds + wave * 16 * kSumRow<D>;
    float* stats = lds + kWaves * 16 * kSumRow<D>;
    if (b == 0) {
        stats[(wave * 16 + n) * 2] = m;
        stats[(wave * 16 + n) * 2 + 1] = l;
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < D / 16; i += 4)
            *reinterpret_cast<f32x4*>(sums + n * kSumRow<D> + (4 * b + c) * (D / 16) + i) =
                f32x4{o[i][c], o[i + 1][c], o[i + 2][c], o[i + 3][c]};
    __syncthreads();
    // 16 threads a row, each with 4 dims of every 64
    constexpr int kParts = D / 64;
    const int r = threadIdx.x >> 4, d0 = (threadIdx.x & 15) * 4;
    if (row0 + r >= rows.count) return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[(w * 16 + r) * 2]);
    f32x4 acc[kParts];
#pragma unroll
    for (int i = 0; i < kParts; ++i) acc[i] = f32x4{0, 0, 0, 0};
    float sum = 0.0f;
    if (top > -INFINITY) {
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(stats[(w * 16 + r) * 2] - top);
            sum += f * stats[(w * 16 + r) * 2 + 1];
#pragma unroll
            for (int i = 0; i < kParts; ++i)
                acc[i] += f * *reinterpret_cast<const f32x4*>(lds + (w * 16 + r) * kSumRow<D> + 64 * i + d0);
        }
    }
    const int64_t at = rows.place(a.sc, row0 + r, hk);
    if (pages > item.chunk) {
        const int64_t to = int64_t(group_of(a)) * kRowTile + r;
        float* po = a.part_o + to * D + d0;
        if (top > -INFINITY)
#pragma unroll
            for (int i = 0; i < kParts; ++i) *reinterpret_cast<f32x4*>(po + 64 * i) = acc[i];
        if (d0 == 0) {
            a.part_ml[to * 2] = top;
            a.part_ml[to * 2 + 1] = sum;
        }
        return;
    }
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;   // V's scale apart: their quotient may be too small for fp32
    uint16_t* out = a.out + at * D + d0;
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
        uint16_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = f32_to_bf16_rne(acc[i][j] * f * a.v_scale);
        u32x2 x;
        __builtin_memcpy(&x, w, 8);
        *reinterpret_cast<u32x2*>(out + 64 * i) = x;
    }
    if (a.lse && d0 == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
}

// ---- many query rows

// A workgroup takes 128 rows, 32 a wavefront (or 64 and the page's halves
// apart, joined at the end, where there are no more), and decodes each page once for
// all of them into LDS as f16: K [64 slots][D], V [D][64 slots], in 16-byte
// chunks whose place within a row is permuted so that the lanes of a matrix
// operand's read fall on different banks.  Bound by the matrix unit and the
// vector unit taking turns (a page's 32 products a wavefront take 1024 cycles,
// its decode share and exponentials about 1400) at the 1.9 GHz that the card
// holds under them: ragged prompt chunks of 700 .. 4099 tokens over 4100 ..
// 8192 slots, 32 heads of 128, take 767 us, 891 TFLOP/s.
// HALVES 2: wavefronts 0 and 1 have the first 32 slots of each page, 2 and 3 the last.
template <int D, int HALVES>
__global__ void __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2)
kv_attend_tile_kernel(AttendArgs a) {
    extern __shared__ char tiles[];   // two pages
    constexpr int kStep = D == 256 || HALVES == 2 ? 1 : 2;   // 32-slot tiles between rescalings: registers decide
    constexpr int kRows = kTileRows / HALVES;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row_wave = wave % (kWaves / HALVES), my_half = wave / (kWaves / HALVES);   // my_half: HALVES 2 only
    const int n = lane & 31, b = lane >> 5;
    const int s = blockIdx.y, split = blockIdx.z;
    const int hk = group_of(a) % a.v.kv_heads;
    const QueryRows rows(a.v, a.sc, s);
    // the last rows see most: they begin first
    const int tile = a.row_tiles - 1 - group_of(a) / a.v.kv_heads;
    const int row0 = tile * kRows;
    if (row0 >= rows.count) return;

    const Span all = rows.span(a.sc, row0, min(row0 + kRows, rows.count) - 1);
    const int used = used_splits(a, all);
    if (split >= used) return;
    const int begin = pages_lo(all) + split * a.chunk;
    const int end = split + 1 < used ? begin + a.chunk : pages_hi(all);

    const int my0 = row0 + row_wave * 32;
    const QueryRow me = rows.row(a.sc, my0 + n);
    const Span span = rows.span(a.sc, min(my0, rows.count - 1), min(my0 + 32, rows.count) - 1);
    f16x8 q[D / 16];   // step i: dims 16 i + 8 b ..
    float to_log2 = load_query<D / 16, 16, 32>(a.sc, query_at(a.sc, me, hk) + 8 * b, q);
    if (to_log2 < 0.0f) {   // a negative scale goes into the query, so that the largest sum is the largest score
#pragma unroll
        for (int i = 0; i < D / 16; ++i) q[i] = -q[i];
        to_log2 = -to_log2;
    }
    // Hidden scores are -inf before they meet the factor, so that is never 0 (a scale of 0, a row of zeros over small
    // keys): sums stay below 2^35, and times 2^-126 they weigh alike as they would times 0.
    to_log2 = fmaxf(to_log2, 0x1p-126f);
    // scores are formed with the exponential's argument; capped ones are whole before
    const float factor = a.sc.cap == 0.0f ? to_log2 : 1.0f;

    f32x16 o[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
    // Row r of a 32-slot operand is slot r with bits 2 and 3 exchanged: a
    // lane's scores 8 t .. 8 t + 7 are then those of 8 consecutive slots.
    const int slot_n = (n & ~12) | ((n & 4) << 1) | ((n & 8) >> 1);

    PageShare<D> share;
    const int last = a.v.pages > 0 ? end : begin;
    int id = begin < last ? a.v.page_id(s, begin) : -1;
    int next_id = begin + 1 < last ? a.v.page_id(s, begin + 1) : -1;
    if (begin < last) share.load(a.v.record_or_first<D>(id, hk), tid);
    for (int page = begin; page < last; ++page) {
        char* lds = tiles + ((page - begin) & 1) * PageTiles<D>::kBytes;
        const int base = page * kPage;
        share.put(lds, tid, rows.len - base);
        const bool here = a.v.has(id);
        id = next_id;
        __syncthreads();
        share.load(a.v.record_or_first<D>(id, hk), tid);
        next_id = page + 2 < last ? a.v.page_id(s, page + 2) : -1;
        if (!here || base >= span.hi || base + kPage <= span.lo) continue;

#pragma unroll
        for (int turn = 0; turn < 2 / HALVES; turn += kStep) {   // kStep 32-slot tiles at a time
            const int half = HALVES == 2 ? my_half : turn;
            f32x16 z[kStep];
#pragma unroll
            for (int h = 0; h < kStep; ++h) {
                z[h] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const f16x8 k = *reinterpret_cast<const f16x8*>(lds + PageTiles<D>::k_at(32 * (half + h) + slot_n, 2 * i + b));
                    z[h] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[i], z[h], 0, 0, 0);
                }
            }
            reads_ahead<kStep * D / 16>();
            float p[16 * kStep];   // [t][8 consecutive slots]: slot 32 half + 16 t + 8 b + j
#pragma unroll
            for (int i = 0; i < 16 * kStep; ++i) p[i] = z[i >> 4][i & 15];
            if (a.sc.cap != 0.0f) a.sc.shape(p, to_log2);
            if (base < span.lo_all || base + kPage > span.hi_all) {
#pragma unroll
                for (int i = 0; i < 16 * kStep; ++i) {
                    const int slot = base + 32 * half + 16 * (i >> 3) + 8 * b + (i & 7);
                    p[i] = slot >= me.lo && slot < me.hi ? p[i] : -INFINITY;
                }
            }
            float top = p[0];
#pragma unroll
            for (int i = 1; i < 16 * kStep; ++i) top = fmaxf(top, p[i]);
            top = fmaxf(top, __shfl_xor(top, 32)) * factor;
            if (__any(top > m + kSlack)) {
                const float grown = fmaxf(m, top);
                const float keep = grown == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
                m = grown;
                l *= keep;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) o[i] *= keep;
            }
            const float base_m = m == -INFINITY ? 0.0f : m - kLift;
            f16x8 pt[2 * kStep];
#pragma unroll
            for (int i = 0; i < 16 * kStep; ++i) {
                const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], factor, -base_m));
                l += e;
                pt[i >> 3][i & 7] = static_cast<_Float16>(e);
            }
#pragma unroll
            for (int t = 0; t < 2 * kStep; ++t)
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const f16x8 v = *reinterpret_cast<const f16x8*>(lds + PageTiles<D>::v_at(32 * i + n, 2 * (2 * half + t) + b));
                    o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pt[t], o[i], 0, 0, 0);
                }
            reads_ahead<2 * kStep * (D / 32)>();
        }
    }
    l += __shfl_xor(l, 32);
    if (l != l && m == -INFINITY) m = 0.0f;   // all scores NaN: the row stays NaN
    m -= kLift;                               // what the sums are held against
    if constexpr (HALVES == 2) {
        // the second half's results through LDS to the first's wavefronts, lane by lane
        constexpr int kParts = D / 32 * 16 + 2;
        float* meet = reinterpret_cast<float*>(tiles) + row_wave * 64 * kParts + lane;
        __syncthreads();
        if (my_half == 1) {
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int c = 0; c < 16; ++c) meet[(16 * i + c) * 64] = o[i][c];
            meet[(kParts - 2) * 64] = m;
            meet[(kParts - 1) * 64] = l;
        }
        __syncthreads();
        if (my_half == 0) {
            const float other_m = meet[(kParts - 2) * 64], grown = fmaxf(m, other_m);
            const float f0 = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - grown);
            const float f1 = other_m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(other_m - grown);
            l = l * f0 + meet[(kParts - 1) * 64] * f1;
            m = grown;
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int c = 0; c < 16; ++c) o[i][c] = o[i][c] * f0 + meet[(16 * i + c) * 64] * f1;
        }
    }

    const bool live = my0 + n < rows.count;
    const int64_t at = rows.place(a.sc, min(my0 + n, rows.count - 1), hk);
    if (used > 1) {
        if (!live || (HALVES == 2 && my_half == 1)) return;
        const int64_t slice = int64_t(a.v.total) * a.sc.heads;
        float* po = a.part_o + (split * slice + at) * D;
        if (m > -INFINITY)
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
#pragma unroll
                for (int c = 0; c < 16; c += 4)
                    *reinterpret_cast<f32x4*>(po + 32 * i + 2 * c + 4 * b) = f32x4{o[i][c], o[i][c + 1], o[i][c + 2], o[i][c + 3]};
        if (b == 0) {
            a.part_ml[(split * slice + at) * 2] = m;
            a.part_ml[(split * slice + at) * 2 + 1] = l;
        }
        return;
    }
    // bf16 rows through LDS, then 16-byte stores along them
    const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
    if (a.lse && live && b == 0 && (HALVES == 1 || my_half == 0)) a.lse[at] = (m + log2f(l)) * kLn2;
    __syncthreads();
    constexpr int kRow = D * 2 + 16;   // bytes of a staged row
    char* stage = tiles + wave * 32 * kRow;   // the second half's wavefronts stage for nothing
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int c = 0; c < 16; c += 4) {
            uint16_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = f32_to_bf16_rne(o[i][c + j] * f * a.v_scale);
            u32x2 x;
            __builtin_memcpy(&x, w, 8);
            *reinterpret_cast<u32x2*>(stage + n * kRow + (32 * i + 2 * c + 4 * b) * 2) = x;
        }
    __syncthreads();
    if (HALVES == 2 && my_half == 1) return;
    for (int i = lane; i < 32 * (D / 8); i += 64) {
        const int r = i / (D / 8), part = i % (D / 8);
        if (my0 + r >= rows.count) break;
        *reinterpret_cast<u32x4*>(a.out + rows.place(a.sc, my0 + r, hk) * D + 8 * part) =
            *reinterpret_cast<const u32x4*>(stage + r * kRow + 16 * part);
    }
}

// Joins the parts of one row, one workgroup a row: the wavefronts take every
// fourth part and meet in LDS, both in a fixed order.  Bound by latency (1024
// rows of up to 37 parts: 6.8 us).
template <int D>
__global__ void __launch_bounds__(64 * kWaves)
kv_join_kernel(AttendArgs a) {
    __shared__ float sums[kWaves][D];
    __shared__ float weight[kWaves];
    const int64_t slice = int64_t(a.v.total) * a.sc.heads;
    const int64_t at = group_of(a);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int token = static_cast<int>(at / a.sc.heads), head = static_cast<int>(at % a.sc.heads);
    const int s = last_sequence(a.v, [&](int i) { return a.v.start(i) <= token; });
    if (s < 0) return;
    const QueryRows rows(a.v, a.sc, s);
    const int r = nvfp4::kv_row_of(token, rows.first_token, rows.group, head % rows.group, rows.count);
    if (r < 0) return;   // no sequence's row
    // where part p of the row lies: the parts of a tile a slice apart, an item's by its number
    int used;
    int64_t first, step, last;
    if (a.tile) {
        const int row0 = r / a.tile * a.tile;
        used = used_splits(a, rows.span(a.sc, row0, min(row0 + a.tile, rows.count) - 1));
        first = at, step = slice, last = at + (used - 1) * slice;
    } else {
        const int pages = segment_pages(a, rows), chunk = a.plan ? a.plan[0] : a.chunk;
        const int segment = r / kRowTile * a.v.kv_heads + head / rows.group;
        used = (pages + chunk - 1) / chunk;
        if (a.plan) {
            first = a.plan[2 + s] + segment * (pages / chunk), step = 1;
            last = pages % chunk ? a.plan[1] + a.plan[2 + a.v.seqs + s] + segment : first + used - 1;
        } else {
            step = int64_t(a.row_tiles) * a.v.kv_heads * a.v.seqs;
            first = int64_t(s) * a.row_tiles * a.v.kv_heads + segment;
            last = first + (used - 1) * step;
        }
        first = first * kRowTile + r % kRowTile, last = last * kRowTile + r % kRowTile, step *= kRowTile;
    }
    if (used == 1) return;         // written already
    auto place = [&](int p) { return p == used - 1 ? last : first + p * step; };

    float top = -INFINITY;
    for (int p = lane; p < used; p += 64) top = fmaxf(top, a.part_ml[place(p) * 2]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    constexpr int kPer = D / 64;
    float acc[kPer] = {}, sum = 0.0f;
#pragma unroll 4
    for (int p = wave; p < used; p += kWaves) {
        const float m = a.part_ml[place(p) * 2];
        const float part = a.part_ml[place(p) * 2 + 1];
        const float* po = a.part_o + place(p) * D + lane * kPer;
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        sum += m == -INFINITY ? 0.0f : f * part;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float x = po[i];   // not written where the part saw nothing
            acc[i] += m == -INFINITY ? 0.0f : f * x;
        }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) sums[wave][lane * kPer + i] = acc[i];
    if (lane == 0) weight[wave] = sum;
    __syncthreads();
    if (tid >= D / 2) return;
    sum = weight[0] + weight[1] + weight[2] + weight[3];
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;   // V's scale apart: their quotient may be too small for fp32
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int d = 2 * tid + j;
        const float x = sums[0][d] + sums[1][d] + sums[2][d] + sums[3][d];
        w |= uint32_t(f32_to_bf16_rne(x * f * a.v_scale)) << (16 * j);
    }
    *reinterpret_cast<uint32_t*>(a.out + at * D + 2 * tid) = w;
    if (a.lse && tid == 0) a.lse[at] = (top + log2f(sum)) * kLn2;
}

template <int D>
constexpr size_t rows_lds() {
    return (kWaves * 16 * kSumRow<D> + kWaves * 16 * 2) * sizeof(float);
}

template <int D>
constexpr size_t tile_lds() {
    return 2 * PageTiles<D>::kBytes;   // at least the staged rows of the output
}

template <int D>
bool allow_lds() {
    static_assert(tile_lds<D>() >= 2 * 64 * (D / 2 + 2) * sizeof(float));
    static_assert(tile_lds<D>() >= kTileRows * (D * 2 + 16) && tile_lds<D>() <= kMaxLdsBytes);
    for (const void* fn : {reinterpret_cast<const void*>(kv_attend_rows_kernel<D, false>),
                           reinterpret_cast<const void*>(kv_attend_rows_kernel<D, true>),
                           reinterpret_cast<const void*>(kv_attend_tile_kernel<D, 1>),
                           reinterpret_cast<const void*>(kv_attend_tile_kernel<D, 2>)})
        if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLdsBytes) != hipSuccess) return false;
    return true;
}

template <class Kernel>
int launch_groups(Kernel kernel, AttendArgs a, int64_t count, unsigned y, unsigned z, size_t lds, hipStream_t st) {
    return launch_sliced(count, 64 * kWaves, [&](int first, unsigned n) {
        a.group0 = first;
        hipLaunchKernelGGL(kernel, dim3(n, y, z), dim3(64 * kWaves), lds, st, a);
    });
}

template <int D, bool TREE>
int launch_attend(AttendArgs a, const nvfp4::KvPlan& plan, hipStream_t st) {
    int ok;
    if (plan.tile) {
        a.row_tiles = static_cast<int>(nvfp4::kv_row_tiles(plan, a.v.total, a.sc.group));
        // parts of a tile's pages along the slowest axis: those that short sequences do not need come last
        ok = launch_groups(plan.tile == kTileRows ? kv_attend_tile_kernel<D, 1> : kv_attend_tile_kernel<D, 2>, a,
                           int64_t(a.row_tiles) * a.v.kv_heads, a.v.seqs, plan.splits, tile_lds<D>(), st);
    } else {
        if (plan.planned) {
            hipLaunchKernelGGL(kv_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
            if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
        }
        ok = launch_groups(kv_attend_rows_kernel<D, TREE>, a, plan.items, 1, 1, rows_lds<D>(), st);
    }
    if (ok != NVFP4_OK || plan.part_rows == 0) return ok;
    return launch_groups(kv_join_kernel<D>, a, int64_t(a.v.total) * a.sc.heads, 1, 1, 0, st);
}

}  // namespace

namespace nvfp4 {

int kv_setup() { return allow_lds<64>() && allow_lds<128>() && allow_lds<256>() ? NVFP4_OK : NVFP4_ERR_HIP; }

}  // namespace nvfp4

namespace {

// Argument checks that the calls share.
int check_call(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries) {
    int st;
    if ((st = nvfp4::check_kv_cache(cache)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_seqs(seqs, true)) != NVFP4_OK) return st;
    return nvfp4::check_kv_queries(cache, seqs, queries);
}

// tree: NULL where rows see by their order.
int attend(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries,
           const nvfp4_kv_tree_t* tree, void* out, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    int st;
    if ((st = check_call(cache, seqs, queries)) != NVFP4_OK) return st;
    if (tree && (st = nvfp4::check_kv_tree(seqs, queries, tree)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_kv_rows(out, 0, 0, seqs->total)) != NVFP4_OK) return st;
    if ((reinterpret_cast<uintptr_t>(lse) & 3) || (reinterpret_cast<uintptr_t>(workspace) & 15)) return NVFP4_ERR_ALIGN;
    if (seqs->seqs == 0 || seqs->total == 0 || queries->max_q == 0) return NVFP4_OK;
    const int64_t need = tree ? nvfp4::tree_workspace_bytes(cache, seqs, queries) : nvfp4::kv_workspace_bytes(cache, seqs, queries);
    if (need > 0 && !workspace) return NVFP4_ERR_NULL;
    if (need > workspace_bytes) return NVFP4_ERR_SCRATCH;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    if (tree && nvfp4::tree_plan(cache, seqs, queries).rows)
        return nvfp4::tree_attend(cache, seqs, queries, tree, out, lse, workspace, stream);

    AttendArgs a;
    a.v = kv_view(cache, seqs);
    a.sc = kv_scores(cache, queries);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    const nvfp4::KvPlan plan = nvfp4::kv_plan(cache, seqs, queries, tree != nullptr);
    a.tile = plan.tile;
    a.splits = plan.splits;
    a.chunk = plan.chunk;
    a.row_tiles = static_cast<int>(plan.row_tiles);
    a.plan = plan.planned ? static_cast<int32_t*>(workspace) : nullptr;
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + (plan.planned ? nvfp4::kv_plan_bytes(seqs) : 0));
    a.part_ml = plan.part_rows > 0 ? a.part_o + plan.part_rows * cache->head_dim : nullptr;
    a.v_scale = cache->v_scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (tree) {
        a.sc.causal = 1;   // what a tree's rows see together, and so its pages, are a chain's
        a.sc.tree = kv_tree(tree, queries);
        switch (cache->head_dim) {
            case 64: return launch_attend<64, true>(a, plan, s);
            case 128: return launch_attend<128, true>(a, plan, s);
            default: return launch_attend<256, true>(a, plan, s);
        }
    }
    switch (cache->head_dim) {
        case 64: return launch_attend<64, false>(a, plan, s);
        case 128: return launch_attend<128, false>(a, plan, s);
        default: return launch_attend<256, false>(a, plan, s);
    }
}

}  // namespace

extern "C" int nvfp4_kv_attention_workspace(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                            const nvfp4_kv_queries_t* queries, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    const int st = check_call(cache, seqs, queries);
    if (st != NVFP4_OK) return st;
    *bytes = nvfp4::kv_workspace_bytes(cache, seqs, queries);
    return NVFP4_OK;
}

extern "C" int nvfp4_kv_attention(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries,
                                  void* out, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
    return attend(cache, seqs, queries, nullptr, out, lse, workspace, workspace_bytes, stream);
}

extern "C" int nvfp4_kv_tree_attention_workspace(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                                 const nvfp4_kv_queries_t* queries, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    const int st = check_call(cache, seqs, queries);
    if (st != NVFP4_OK) return st;
    if (queries->max_q > NVFP4_TREE_MAX) return NVFP4_ERR_SHAPE;
    *bytes = nvfp4::tree_workspace_bytes(cache, seqs, queries);
    return NVFP4_OK;
}

extern "C" int nvfp4_kv_tree_attention(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs,
                                       const nvfp4_kv_queries_t* queries, const nvfp4_kv_tree_t* tree, void* out, float* lse,
                                       void* workspace, int64_t workspace_bytes, void* stream) {
    if (!tree) return NVFP4_ERR_NULL;
    return attend(cache, seqs, queries, tree, out, lse, workspace, workspace_bytes, stream);
}
