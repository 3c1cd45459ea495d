// Attention of the nodes of drafted trees over the paged NVFP4 cache
// (include/nvfp4_draft.h), the products and the softmax of kv_attention.hip.
//
// The rows of a tree all see the same pages, so the work is a list of segments
// (sequence, kv head, row tile), each with the sequence's number of pages.
// The list is cut into equal ranges of pages, whatever the sequences' lengths,
// and a workgroup takes a range, one segment's piece after the other.  Segments
// that lie within a range are finished by it; the parts of the others are joined
// by a second kernel, in the order of their pages.  (Cut by the longest sequence's
// pages instead, 32 trees of 9 .. 16 nodes x 4 heads over 1000 .. 16000 slots took 175 us
// and now 105, four of 200 .. 255 over 20000 .. 65000 slots 1010 and now 679.)
// Few pages go to the 16-row workgroups of kv_attention.hip (host/tree_plan.cpp).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

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

constexpr int kWaves = nvfp4::kTreeWaves;

struct TreeArgs {
    KvView v;
    KvScores sc;
    uint16_t* out;
    float* lse;
    float* part_o;     // [2 parts][rows of a tile][D]: sums of exp2(z - m) v, without the V scale
    float* part_ml;    // [2 parts][rows of a tile][2]: m and the sum of exp2(z - m)
    int64_t* sums;     // [seqs + 1][2] segments and pages before a sequence's
    int added;         // a kernel before has added them up; 0: each wavefront does, and the first workgroup leaves them for the join
    int rows;          // of a tile
    int whole;         // nothing is cut
    int ranges;        // that the pages are cut into
    int least;         // pages of a range at least
    int group0;        // first workgroup of the launch
    float v_scale;
};

using TreeRows = QueryRowsOf<true>;

__device__ __forceinline__ int tiles_of(const TreeArgs& a, const TreeRows& r) { return (r.count + a.rows - 1) / a.rows; }

// The pages that the rows of a sequence see, at least one, and the first of them.
__device__ __forceinline__ int pages_of(const TreeArgs& a, const TreeRows& r, int* first) {
    const Span s = r.span(a.sc, 0, r.count - 1);
    *first = s.lo / kPage;
    return max((s.hi + kPage - 1) / kPage - *first, 1);
}

// A segment counts for its pages and, ahead of them, for what beginning one takes (its place in the list, its first
// page's latency, its queries): four pages' time (with none counted, 32 small trees took 120 us and not 105).
constexpr int kStart = 4;

struct Size {
    int64_t segments, pages;   // counted
};

__device__ __forceinline__ Size size_of(const TreeArgs& a, int s) {
    if (s >= a.v.seqs) return Size{0, 0};
    const TreeRows r(a.v, a.sc, s);
    if (r.count <= 0) return Size{0, 0};
    int first;
    const int64_t n = int64_t(tiles_of(a, r)) * a.v.kv_heads;
    return Size{n, n * (kStart + pages_of(a, r, &first))};
}

// Pages of a range, of all that are counted.
__device__ __forceinline__ int64_t range_of(const TreeArgs& a, int64_t all) { return max((all + a.ranges - 1) / a.ranges, int64_t(a.least)); }

// What a workgroup does at a time: pages skip .. skip + take - 1 of segment `index` of sequence s.
struct Piece {
    int s, index, skip, take, pages;   // s < 0: none
    int page0;                         // the segment's first page
    int counted;                       // what the piece counts for in its range
};

// The segments and pages before each sequence, and how the pages are cut.  Up to
// 64 sequences are a lane each of every wavefront that asks; more are added up by a kernel before.
struct Cut {
    Size mine;      // before sequence `lane` (up to 64 sequences)
    int64_t all;    // pages
    int64_t each;   // of a range

    __device__ __forceinline__ explicit Cut(const TreeArgs& a) {
        const int lane = threadIdx.x & 63;
        if (a.added) {
            all = a.sums[2 * a.v.seqs + 1];
        } else {
            const Size size = size_of(a, lane);
            mine = size;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t n = __shfl_up(mine.segments, d), p = __shfl_up(mine.pages, d);
                if (lane >= d) mine.segments += n, mine.pages += p;
            }
            all = __shfl(mine.pages, 63);
            mine.segments -= size.segments, mine.pages -= size.pages;
        }
        each = range_of(a, all);
    }
    // For the join.
    __device__ __forceinline__ void leave(const TreeArgs& a) const {
        const int i = threadIdx.x;
        if (a.added || i >= a.v.seqs) return;   // at most as many as lanes
        a.sums[2 * i] = mine.segments, a.sums[2 * i + 1] = mine.pages;
        if (i == 0) a.sums[2 * a.v.seqs + 1] = all;
    }
    __device__ __forceinline__ Size before(const TreeArgs& a, int s) const {
        if (a.added) return Size{a.sums[2 * s], a.sums[2 * s + 1]};
        return Size{__shfl(mine.segments, s), __shfl(mine.pages, s)};
    }
    // The last sequence that has at most `at` segments (where nothing is cut) or pages before it.
    __device__ __forceinline__ int sequence(const TreeArgs& a, int64_t at) const {
        const int lane = threadIdx.x & 63;
        if (!a.added) return __popcll(__ballot(lane < a.v.seqs && (a.whole ? mine.segments : mine.pages) <= at)) - 1;
        return find(a, at, a.whole ? 0 : 1);
    }
    // The same by what a kernel left, of segments (0) or pages (1).
    static __device__ __forceinline__ int find(const TreeArgs& a, int64_t at, int which) {
        const int lane = threadIdx.x & 63;
        int s = 0;
        for (int step = a.v.seqs > 4096 ? 4096 : a.v.seqs > 64 ? 64 : 1;; step /= 64) {
            const int i = s + lane * step;
            s += (__popcll(__ballot(i < a.v.seqs && a.sums[2 * min(i, a.v.seqs) + which] <= at)) - 1) * step;
            if (step == 1) return s;
        }
    }
    // The piece of range w that begins `done` into it.
    __device__ __forceinline__ Piece piece(const TreeArgs& a, int w, int done) const {
        const int64_t at = a.whole ? w : w * each + done, stop = min((w + int64_t(1)) * each, all);
        if (a.whole ? done > 0 : at >= stop) return Piece{-1, 0, 0, 0, 0, 0, 0};
        const int s = __builtin_amdgcn_readfirstlane(sequence(a, at));
        const TreeRows rows(a.v, a.sc, s);
        if (rows.count <= 0) return Piece{-1, 0, 0, 0, 0, 0, 0};   // after the last segment
        int page0;
        const int pages = pages_of(a, rows, &page0);
        const Size b = before(a, s);
        if (a.whole) {
            const int64_t t = at - b.segments;
            return Piece{t < int64_t(tiles_of(a, rows)) * a.v.kv_heads ? s : -1, static_cast<int>(t), 0, pages, pages, page0, 1};
        }
        const int64_t in = at - b.pages, t = in / (kStart + pages);
        const int from = static_cast<int>(in - t * (kStart + pages)), to = static_cast<int>(min(int64_t(kStart + pages), from + stop - at));
        return Piece{s, static_cast<int>(t), max(from - kStart, 0), max(to - kStart, 0) - max(from - kStart, 0), pages, page0, to - from};
    }
};

constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
kv_tree_sums_kernel(TreeArgs a) {
    __shared__ Size tmp[kPlanThreads / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Size all{0, 0};
    for (int base = 0; base < a.v.seqs; base += kPlanThreads) {
        const Size size = size_of(a, base + tid);
        Size sum = size;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t n = __shfl_up(sum.segments, d), p = __shfl_up(sum.pages, d);
            if (lane >= d) sum.segments += n, sum.pages += p;
        }
        __syncthreads();
        if (lane == 63) tmp[wave] = sum;
        __syncthreads();
        Size front = all;
#pragma unroll 1
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            if (w < wave) front.segments += tmp[w].segments, front.pages += tmp[w].pages;
            all.segments += tmp[w].segments, all.pages += tmp[w].pages;
        }
        if (base + tid < a.v.seqs) {
            a.sums[2 * (base + tid)] = front.segments + sum.segments - size.segments;
            a.sums[2 * (base + tid) + 1] = front.pages + sum.pages - size.pages;
        }
    }
    if (tid == 0) a.sums[2 * a.v.seqs] = all.segments, a.sums[2 * a.v.seqs + 1] = all.pages;
}

__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

template <int D>
constexpr int kPageBytes = KTile<D>::kBytes + VTile<D>::kBytes;

// HALVES 1: 128 rows, 32 a wavefront; 2: 64, with the first 32 slots of a page
// on wavefronts 0 and 1 and the last on 2 and 3.  A page is decoded once for all of them
// into LDS, two pages after its loads began (what every wavefront holds of both is 22 registers).  Bound by the
// matrix unit and the vector unit taking turns, as in kv_attention.hip: at 128 rows of 128
// dims a page takes a wavefront 1024 cycles of products and about 1200 of vector work, and
// a workgroup 2.4 us with two of them on a CU (four of 200 .. 255 nodes over 20000 .. 65000 slots:
// 832 TFLOP/s of what they see, 890 of the tiles' rows).  Products of the
// next half beside the exponentials of this one left registers for one operand's read ahead, and were no faster.
//
// Causal rows of many tokens keep kv_attention.hip's kernel, whose tiles see pages of their own and
// are cut one by one, and its layout of a page in LDS.  Chains in that | in this, us: D = 128, 32 of 16 x 4 rows
// over 4000 slots 88 | 75, 4 of 255 x 4 over 32000 606 | 601; D = 256, 16 of 64 x 2 over 8000 244 | 214; D = 64, 64 of
// 64 x 4 over 4000 183 | 211.  Ranges over segments that see different pages are not tried.
template <int D, int HALVES>
__global__ void __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2)
kv_tree_tile_kernel(TreeArgs a) {
    extern __shared__ char tiles[];   // two pages
    constexpr int kRows = 32 * kWaves / HALVES, kPer = D / 32, kAheadPages = 2;
    // a turn leaves nothing to the next but how far the range is done
#pragma clang loop unroll(disable)
    for (int done = 0;;) {
        int s, hk, row0, begin, take, skip, pages;
        {
            const Cut cut(a);
            if (done == 0 && blockIdx.x == 0 && !a.whole) cut.leave(a);
            const Piece piece = cut.piece(a, a.group0 + static_cast<int>(blockIdx.x), done);
            s = scalar(piece.s), take = scalar(piece.take), skip = scalar(piece.skip), pages = scalar(piece.pages);
            if (s < 0) return;
            hk = scalar(piece.index % a.v.kv_heads), row0 = scalar(piece.index / a.v.kv_heads * kRows);
            begin = scalar(piece.page0) + skip;
            done += scalar(piece.counted);
        }
        if (take == 0) continue;   // the range ends where a segment's pages begin
        const int end = begin + take;
        // what follows from a lane's number is formed in each turn: kept from one to the next it would take 40 registers
        int tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        const int row_wave = wave % (kWaves / HALVES), my_half = wave / (kWaves / HALVES);   // my_half: HALVES 2 only
        const int n = lane & 31, b = lane >> 5;
        const TreeRows rows(a.v, a.sc, s);

        const int my0 = row0 + row_wave * 32;
        const bool busy = my0 < rows.count;      // a wavefront without rows only helps to decode
        KShare<D> k_set[kAheadPages];   // pages on their way
        VShare<D> v_set[kAheadPages];
        int id[kAheadPages];
        // Page numbers are read 64 at a time, one a lane, so that a page's loads never wait for the table.
        int ids = -1, at_id = 0;
        auto next_id = [&]() {
            if ((at_id & 63) == 0) {
                const int mine = begin + at_id + lane;
                ids = mine < end ? a.v.page_id(s, mine) : -1;
            }
            return __builtin_amdgcn_readlane(ids, at_id++ & 63);
        };
        const int last = a.v.pages > 0 ? end : begin;
        if (begin < last) {
#pragma unroll
            for (int x = 0; x < kAheadPages; ++x) {
                id[x] = next_id();
                const uint8_t* rec = a.v.record_or_first<D>(id[x], hk);
                k_set[x].load(rec, tid);
                v_set[x].load(rec, tid);
            }
        }
        const QueryRow me = rows.row(a.sc, my0 + n);
        const Span span = rows.span(a.sc, 0, rows.count - 1);
        f16x8 q[D / 16];   // step i: dims 16 i + 8 b ..
        float to_log2 = load_query<D / 16, 16, 32>(a.sc, query_at(a.sc, me, hk) + 8 * b, q);
        if (to_log2 < 0.0f) {   // a negative scale goes into the query, so that the largest sum is the largest score
#pragma unroll
            for (int i = 0; i < D / 16; ++i) q[i] = -q[i];
            to_log2 = -to_log2;
        }
        // Hidden scores are -inf before they meet the factor, so that is never 0.
        to_log2 = fmaxf(to_log2, 0x1p-126f);
        const float factor = a.sc.cap == 0.0f ? to_log2 : 1.0f;

        f32x16 o[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = f32x16{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        float m = -INFINITY, l = 0.0f;

        int page = begin;
        auto step = [&](auto which) {
            constexpr int X = decltype(which)::value;
            char* const k_tile = tiles + ((page - begin) & 1) * kPageBytes<D>;
            char* const v_tile = k_tile + KTile<D>::kBytes;
            const int base = page * kPage, left = rows.len - base;
            k_set[X].put(k_tile, tid);
            // what lies beyond the sequence's end may hold anything, and becomes 0 in V (scores of such slots are masked)
            if (left < kPage) v_set[X].cut(tid, left);
            v_set[X].put(v_tile, tid);
            const bool here = a.v.has(id[X]);
            gemm_lds_barrier();
            id[X] = next_id();
            const uint8_t* rec = a.v.record_or_first<D>(id[X], hk);
            k_set[X].load(rec, tid);
            v_set[X].load(rec, tid);
            ++page;
            if (!here || !busy) return;
            const char* k_lane = k_tile + KTile<D>::at(n, b);
            const char* v_lane = v_tile + VTile<D>::at(n, b);

#pragma unroll
            for (int turn = 0; turn < 2 / HALVES; ++turn) {   // 32 slots at a time
                const int half = HALVES == 2 ? my_half : turn;
                f32x16 z = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const f16x8 k = *reinterpret_cast<const f16x8*>(k_lane + KTile<D>::at(32 * half, 2 * i));
                    z = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[i], z, 0, 0, 0);
                }
                reads_ahead<D / 16>();
                float p[16];   // [t][8 consecutive slots]: slot 32 half + 16 t + 8 b + j
#pragma unroll
                for (int i = 0; i < 16; ++i) p[i] = z[i];
                // What is rare comes apart, and works out anew which row it is: kept, that would take 30 registers.
                if (a.sc.cap != 0.0f) a.sc.shape(p, to_log2);
                if (base < span.lo_all || base + kPage > span.hi_all) {
                    int r = my0 + n;
                    asm volatile("" : "+v"(r));
                    const QueryRow who = rows.row(a.sc, r);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t seen = rows.seen8(a.sc, who, base + 32 * half + 16 * t + 8 * b);
#pragma unroll
                        for (int i = 0; i < 8; ++i) p[8 * t + i] = seen >> i & 1 ? p[8 * t + i] : -INFINITY;
                    }
                }
                float top = p[0];
#pragma unroll
                for (int i = 1; i < 16; ++i) top = __builtin_elementwise_maximum(top, p[i]);   // (three at a time; fmaxf would first quiet each)
                top = fmaxf(top, __shfl_xor(top, 32)) * factor;
                if (__any(top > m + kSlack)) {
                    const float grown = top > m + kSlack ? top : m;   // a row by its own scores alone
                    const float keep = grown == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(m - grown);
                    m = grown;
                    l *= keep;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) o[i] *= keep;
                }
                const float base_m = m == -INFINITY ? 0.0f : m - kLift;
                f16x8 pt[2];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(p[i], factor, -base_m));
                    l += e;
                    pt[i >> 3][i & 7] = static_cast<_Float16>(e);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        const f16x8 v = *reinterpret_cast<const f16x8*>(v_lane + VTile<D>::at(32 * i, 2 * (2 * half + t)));
                        o[i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, pt[t], o[i], 0, 0, 0);
                    }
                reads_ahead<2 * (D / 32)>();
            }
        };
        while (page < last) {
            step(std::integral_constant<int, 0>{});
            if (page >= last) break;
            step(std::integral_constant<int, 1>{});
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

        const bool live = my0 + n < rows.count && (HALVES == 1 || my_half == 0);
        const int64_t place = rows.place(a.sc, min(my0 + n, rows.count - 1), hk);
        if (take < pages) {
            if (live) {
                // a segment that begins in this range, or one from before it
                const int64_t to = (2 * int64_t(blockIdx.x) + (skip == 0)) * kRows + row_wave * 32 + n;
                float* po = a.part_o + to * D;
                if (m > -INFINITY)
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        float x[kPer];   // consecutive dims: V's rows lie so
#pragma unroll
                        for (int i = 0; i < kPer; ++i) x[i] = o[i][c];
                        __builtin_memcpy(__builtin_assume_aligned(po + kPer * ((c & 3) + 8 * (c >> 2) + 4 * b), kPer * 4), x, sizeof x);
                    }
                if (b == 0) {
                    a.part_ml[to * 2] = m;
                    a.part_ml[to * 2 + 1] = l;
                }
            }
        } else {
            // bf16 rows through LDS, then 16-byte stores along them
            const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
            if (a.lse && live && b == 0) a.lse[place] = (m + log2f(l)) * kLn2;
            __syncthreads();
            constexpr int kRow = D * 2 + 16;   // bytes of a staged row
            char* stage = tiles + wave * 32 * kRow;   // the second half's wavefronts stage for nothing
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                uint16_t w[kPer];
#pragma unroll
                for (int i = 0; i < kPer; ++i) w[i] = f32_to_bf16_rne(o[i][c] * f * a.v_scale);
                __builtin_memcpy(__builtin_assume_aligned(stage + n * kRow + kPer * ((c & 3) + 8 * (c >> 2) + 4 * b) * 2, kPer * 2), w, sizeof w);
            }
            __syncthreads();
            if (HALVES == 1 || my_half == 0)
                for (int i = lane; i < 32 * (D / 8); i += 64) {
                    const int r = i / (D / 8), part = i % (D / 8);
                    if (my0 + r >= rows.count) break;
                    *reinterpret_cast<u32x4*>(a.out + rows.place(a.sc, my0 + r, hk) * D + 8 * part) =
                        *reinterpret_cast<const u32x4*>(stage + r * kRow + 16 * part);
                }
        }
        __syncthreads();   // the next piece's pages take the LDS
    }
}

// Joins the parts of the segments that ranges cut: a workgroup takes the segment that the beginning of its range cuts, if
// it is the first to cut it, and 16 of its rows, 16 lanes a row.  So it takes as long as the cuts, not
// the rows, ask for: 8.9 us behind 32 trees of 9 .. 16 nodes x 32 heads, latency (a wavefront for each four rows
// of all 9.1; but behind 600 trees of 16 nodes over 300 slots, 214 us in all and now 179).
constexpr int kJoinRows = 16;

template <int D>
__global__ void __launch_bounds__(256)
kv_tree_join_kernel(TreeArgs a) {
    constexpr int kLanes = 16, kPer = D / kLanes;
    const int me = threadIdx.x % kLanes, range = blockIdx.x + 1;
    const int64_t all = a.sums[2 * a.v.seqs + 1], each = range_of(a, all), at = range * each;
    if (at >= all) return;
    const int s = __builtin_amdgcn_readfirstlane(Cut::find(a, at, 1));
    const TreeRows rows(a.v, a.sc, s);
    if (rows.count <= 0) return;
    int page0;
    const int pages = pages_of(a, rows, &page0);
    const int64_t before = a.sums[2 * s + 1], in = at - before;
    // (a division of 64 bits takes as long as a read)
    const int64_t t = in >> 32 ? in / (kStart + pages) : uint32_t(in) / uint32_t(kStart + pages);
    const int64_t begin = before + t * (kStart + pages) + kStart;   // of its pages
    if (begin >= at || begin < at - each) return;                   // they begin in this range, or before the last one
    const int64_t over = begin + pages - 1 - at;                    // fewer than the pages
    const int first = range - 1, last = range + (over < each ? 0 : static_cast<int>(uint32_t(over) / uint32_t(each)));
    const int in_tile = blockIdx.y * kJoinRows + threadIdx.x / kLanes;
    const int hk = static_cast<int>(t % a.v.kv_heads), r = static_cast<int>(t / a.v.kv_heads) * a.rows + in_tile;
    if (r >= rows.count) return;
    auto part = [&](int w) { return (2 * int64_t(w) + (w == first)) * a.rows + in_tile; };
    float top = -INFINITY;
    for (int w = first + me; w <= last; w += kLanes) top = fmaxf(top, a.part_ml[part(w) * 2]);
#pragma unroll
    for (int d = 1; d < kLanes; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    float acc[kPer] = {}, sum = 0.0f;
#pragma unroll 2
    for (int w = first; w <= last; ++w) {
        const int64_t p = part(w);
        const float m = a.part_ml[p * 2], l = a.part_ml[p * 2 + 1];
        const float f = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        sum += m == -INFINITY ? 0.0f : f * l;
        float x[kPer];   // not written where the part saw nothing
        __builtin_memcpy(x, __builtin_assume_aligned(a.part_o + p * D + me * kPer, 16), sizeof x);
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] += m == -INFINITY ? 0.0f : f * x[i];
    }
    const float f = sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;   // V's scale apart: their quotient may be too small for fp32
    uint16_t w[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) w[i] = f32_to_bf16_rne(acc[i] * f * a.v_scale);
    const int64_t row = rows.place(a.sc, r, hk);
    __builtin_memcpy(__builtin_assume_aligned(a.out + row * D + me * kPer, 2 * kPer > 16 ? 16 : 2 * kPer), w, sizeof w);
    if (a.lse && me == 0) a.lse[row] = (top + log2f(sum)) * kLn2;
}

template <int D>
constexpr size_t tile_lds() {
    return 2 * kPageBytes<D>;   // at least the staged rows of the output
}
template <int D>
bool allow_lds() {
    static_assert(tile_lds<D>() >= 2 * 64 * (D / 2 + 2) * sizeof(float));
    static_assert(tile_lds<D>() >= 32 * kWaves * (D * 2 + 16) && tile_lds<D>() <= kMaxLdsBytes);
    for (const void* fn : {reinterpret_cast<const void*>(kv_tree_tile_kernel<D, 1>), reinterpret_cast<const void*>(kv_tree_tile_kernel<D, 2>)})
        if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLdsBytes) != hipSuccess) return false;
    return true;
}

template <int D>
int launch(TreeArgs a, const nvfp4::TreePlan& plan, hipStream_t st) {
    if (a.added) {
        hipLaunchKernelGGL(kv_tree_sums_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    // ranges are one launch's; whole segments may take several
    const int ok = launch_sliced(plan.workgroups, 64 * kWaves, [&](int first, unsigned n) {
        a.group0 = first;
        hipLaunchKernelGGL((plan.rows == 128 ? kv_tree_tile_kernel<D, 1> : kv_tree_tile_kernel<D, 2>), dim3(n), dim3(64 * kWaves), tile_lds<D>(),
                           st, a);
    });
    if (ok != NVFP4_OK) return ok;
    if (!plan.whole && plan.ranges > 1) {
        hipLaunchKernelGGL(kv_tree_join_kernel<D>, dim3(plan.ranges - 1, a.rows / kJoinRows), dim3(256), 0, st, a);
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}

}  // namespace

namespace nvfp4 {

int tree_setup() { return allow_lds<64>() && allow_lds<128>() && allow_lds<256>() ? NVFP4_OK : NVFP4_ERR_HIP; }

int tree_attend(const nvfp4_kv_cache_t* cache, const nvfp4_kv_seqs_t* seqs, const nvfp4_kv_queries_t* queries,
                const nvfp4_kv_tree_t* tree, void* out, float* lse, void* workspace, void* stream) {
    const TreePlan plan = tree_plan(cache, seqs, queries);
    TreeArgs a;
    a.v = kv_view(cache, seqs);
    a.sc = kv_scores(cache, queries);
    a.sc.causal = 1;
    a.sc.tree = kv_tree(tree, queries);
    a.out = static_cast<uint16_t*>(out);
    a.lse = lse;
    a.rows = plan.rows;
    a.whole = plan.whole;
    a.ranges = plan.ranges;
    a.least = plan.least;
    a.added = plan.added;
    a.sums = static_cast<int64_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + tree_sum_bytes(seqs));
    a.part_ml = a.part_o + int64_t(2) * plan.ranges * plan.rows * cache->head_dim;
    a.v_scale = cache->v_scale;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    switch (cache->head_dim) {
        case 64: return launch<64>(a, plan, s);
        case 128: return launch<128>(a, plan, s);
        default: return launch<256>(a, plan, s);
    }
}

}  // namespace nvfp4
