// The whole numbers of a verify round (include/nvfp4_draft.h): page tables and
// slot maps of a step, what the nodes of a drafted tree see, and the branch
// that the model accepts.  All of it is bound by latency: scans over the
// sequences, chains of parents, and the launches themselves.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../host/draft_shapes.h"
#include "../host/kv_shapes.h"
#include "setup.h"

namespace {

constexpr int kPage = NVFP4_KV_PAGE;
constexpr int kTreeMax = NVFP4_TREE_MAX;
constexpr int kScanThreads = nvfp4::kPagesBlock;
constexpr int kFillThreads = 256, kFillEach = 8;   // tokens of a thread
// Slots and positions of this many tokens at most are filled by the workgroup
// that makes the tables, which spares a launch: 64 sequences of 16 tokens 5.6
// us and 7.8 by a kernel of their own, of 64 tokens 9.5 and 9.0 (and 3 us of
// the host), of 128 tokens 15 and 8.6.
constexpr int kFillInline = 4096;

struct PagesArgs {
    int32_t* pool;
    const int32_t* state;
    int32_t* table;
    const int32_t *held, *keep, *fresh;
    int32_t *state_out, *held_out, *kv_lens, *q_starts, *slots, *positions;
    int64_t table_pitch;
    int capacity, seqs, total;
};

// The last of the ascending p[first .. last] that is at most t, where p[first] is.
__device__ __forceinline__ int last_at_most(const int32_t* p, int first, int last, int t) {
    while (first < last) {
        const int mid = (first + last + 1) / 2;
        if (p[mid] <= t)
            first = mid;
        else
            last = mid - 1;
    }
    return first;
}

// Token t's slot and position, where it belongs to one of the sequences first .. last.
__device__ __forceinline__ void fill_token(const PagesArgs& a, int t, int first, int last, int tokens) {
    int slot = -1, where = -1;
    if (t < tokens) {
        const int s = last_at_most(a.q_starts, first, last, t);
        where = a.kv_lens[s] - a.q_starts[s + 1] + t;
        const int page = a.table[s * a.table_pitch + where / kPage];
        if (page >= 0 && page < (1 << 25)) slot = page * kPage + where % kPage;
    }
    if (a.slots) a.slots[t] = slot;
    if (a.positions) a.positions[t] = where;
}

// v of the lane that a data-parallel move names, 0 where there is none or its
// row (16 lanes) is not among ROWS.
template <int CONTROL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
    return __builtin_amdgcn_update_dpp(0u, v, CONTROL, ROWS, 0xf, false);
}

// op over the lanes up to this one, of its row and of the wavefront, for which 0 changes nothing.
template <class Op>
__device__ __forceinline__ uint32_t row_scan(uint32_t v, Op op) {
    v = op(v, moved<0x111>(v));   // from 1, 2, 4 and 8 lanes before
    v = op(v, moved<0x112>(v));
    v = op(v, moved<0x114>(v));
    return op(v, moved<0x118>(v));
}
template <class Op>
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, Op op) {
    v = row_scan(v, op);
    v = op(v, moved<0x142, 0xa>(v));      // the last lane of rows 0 and 2, to the rows after
    return op(v, moved<0x143, 0xc>(v));   // lane 31, to the second half
}

// The same over the threads of the workgroup, N values at a time, with the
// whole and what lies in the wavefronts before.  Through lanes' moves and one
// barrier: with shuffles, which go through LDS, three such scans were half of
// the 7 us of a step of 48 sequences.
constexpr int kScanWaves = kScanThreads / 64;

template <int N, class Op>
__device__ __forceinline__ void group_scan(uint32_t (&v)[N], uint32_t (&all)[N], uint32_t (&front)[N],
                                           uint32_t (&tmp)[kScanWaves][N], Op op) {
    static_assert(kScanWaves == 16);   // a row
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = wave_scan(v[k], op);
        if (lane == 63) tmp[wave][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t waves = row_scan(tmp[lane & 15][k], op);
        all[k] = __builtin_amdgcn_readlane(waves, 15);
        front[k] = wave > 0 ? __builtin_amdgcn_readlane(waves, wave - 1) : 0;
        v[k] = op(v[k], front[k]);
    }
}

// Pages that are given out or come back are found a chunk at a time: each
// sequence marks the first of its own in the chunk, and the largest mark up to a
// page is its sequence (a search for each of 6500 pages kept LDS busy for 8 us).
constexpr int kEach = 4, kChunk = kEach * kScanThreads;   // pages of a thread, one after the other

struct Marks {
    alignas(16) uint32_t at[kChunk];   // cleared 16 bytes at a time
    uint32_t tmp[kScanWaves][1];
};
static_assert(alignof(Marks) >= alignof(uint4));

// The sequences (threads of the block) of pages at + 4 tid .., of which a
// thread has `own` pages from `from` on.
__device__ __forceinline__ void owners(Marks& m, int at, int from, int own, int (&whose)[kEach]) {
    const int tid = threadIdx.x;
    *reinterpret_cast<uint4*>(m.at + kEach * tid) = uint4{0, 0, 0, 0};
    __syncthreads();
    if (own > 0 && from < at + kChunk && from + own > at) m.at[max(from - at, 0)] = tid + 1;
    __syncthreads();
    uint32_t mine[kEach], last[1], all[1], front[1];
#pragma unroll
    for (int x = 0; x < kEach; ++x) mine[x] = x ? max(m.at[kEach * tid + x], mine[x - 1]) : m.at[kEach * tid];
    last[0] = mine[kEach - 1];
    group_scan(last, all, front, m.tmp, [](uint32_t x, uint32_t y) { return max(x, y); });
    const uint32_t before = max(moved<0x138>(last[0]), front[0]);   // up to the lane before
#pragma unroll
    for (int x = 0; x < kEach; ++x) whose[x] = static_cast<int>(max(mine[x], before)) - 1;
}

// One workgroup takes the sequences 1024 at a time.  Whether a sequence is
// granted depends on what those before it ask for, not on what they get, so
// two scans over the sequences settle a block of them: of what is asked, then
// of what is given.  Pages are given out from entries of the ring before
// `count` and come back to entries from there on, so neither waits for the
// other and their order is fixed.
__global__ void __launch_bounds__(kScanThreads)
kv_pages_kernel(PagesArgs a, int fill) {
    __shared__ uint32_t tmp_ask[kScanWaves][2], tmp_got[kScanWaves][3];
    __shared__ Marks marks;
    __shared__ int take_from[kScanThreads], give_from[kScanThreads];     // pages that are taken and given before each sequence's
    __shared__ int first_page[kScanThreads], need_page[kScanThreads];    // a sequence's pages held and needed
    const int tid = threadIdx.x;
    const int h0 = a.state[0] % a.capacity, head = h0 < 0 ? h0 + a.capacity : h0;
    const int count = min(max(a.state[1], 0), a.capacity), room = a.capacity - count;
    // Sums of what is asked are held at one more than there is: what is beyond
    // it is not granted, however far.
    const uint32_t over = uint32_t(max(a.total, count)) + 1;
    const auto plus = [](uint32_t x, uint32_t y) { return x + y; };
    const auto plus_held = [=](uint32_t x, uint32_t y) { return min(x + y, over); };
    __syncthreads();                // state_out may be state
    uint32_t asked = 0, paged = 0;   // tokens and pages that the sequences before this block ask for
    int given = 0, taken = 0, freed = 0;
    for (int base = 0; base < a.seqs; base += kScanThreads) {
        const int s = base + tid;
        const bool here = s < a.seqs;
        int held = 0, keep = 0;
        int64_t fresh = 0, need = 0, extra = 0;
        bool fits = false;
        if (here) {
            held = static_cast<int>(min(int64_t(max(a.held[s], 0)), a.table_pitch));
            keep = min(max(a.keep[s], 0), held * kPage);
            fresh = max(a.fresh[s], 0);
            need = (keep + fresh + kPage - 1) / kPage;
            fits = need <= a.table_pitch;
            extra = fits && need > held ? need - held : 0;
        }
        uint32_t ask[2] = {fits ? static_cast<uint32_t>(min(fresh, int64_t(over))) : 0, static_cast<uint32_t>(min(extra, int64_t(over)))};
        uint32_t all_ask[2], front_ask[2];
        group_scan(ask, all_ask, front_ask, tmp_ask, plus_held);
        const bool granted = fits && (extra == 0 || plus_held(paged, ask[1]) <= uint32_t(count)) &&
                             (fresh == 0 || plus_held(asked, ask[0]) <= uint32_t(a.total));
        const int got = granted ? static_cast<int>(fresh) : 0;
        const int after = granted ? static_cast<int>(need) : held;
        const int take = max(after - held, 0), give = max(held - after, 0);
        uint32_t sum[3] = {uint32_t(got), uint32_t(take), uint32_t(give)}, all[3], front[3];
        group_scan(sum, all, front, tmp_got, plus);
        const int my_take = static_cast<int>(sum[1]) - take, my_give = static_cast<int>(sum[2]) - give;
        if (here) {
            a.held_out[s] = after;
            a.kv_lens[s] = keep + got;
            a.q_starts[s] = given + static_cast<int>(sum[0]) - got;
        }
        take_from[tid] = my_take;
        give_from[tid] = my_give;
        first_page[tid] = held;
        need_page[tid] = after;
        const int takes = static_cast<int>(all[1]), gives = min(static_cast<int>(all[2]), room - freed);
        for (int at = 0; at < takes; at += kChunk) {
            int q[kEach], page[kEach];
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int64_t from = int64_t(head) + taken + min(at + kEach * tid + x, takes - 1);
                page[x] = a.pool[from >= a.capacity ? from - a.capacity : from];
            }
            owners(marks, at, my_take, take, q);
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int i = at + kEach * tid + x;
                if (i < takes) a.table[(base + q[x]) * a.table_pitch + first_page[q[x]] + (i - take_from[q[x]])] = page[x];
            }
        }
        for (int at = 0; at < gives; at += kChunk) {
            int q[kEach], page[kEach];
            owners(marks, at, my_give, give, q);
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int i = at + kEach * tid + x;
                if (i < gives) page[x] = a.table[(base + q[x]) * a.table_pitch + need_page[q[x]] + (i - give_from[q[x]])];
            }
#pragma unroll
            for (int x = 0; x < kEach; ++x) {
                const int64_t to = int64_t(head) + count + freed + at + kEach * tid + x;
                if (at + kEach * tid + x < gives) a.pool[to >= a.capacity ? to - a.capacity : to] = page[x];
            }
        }
        asked = plus_held(asked, all_ask[0]), paged = plus_held(paged, all_ask[1]);
        given += static_cast<int>(all[0]), taken += takes, freed += gives;
        __syncthreads();
    }
    if (tid == 0) {
        const int64_t h = int64_t(head) + taken;
        a.state_out[0] = static_cast<int>(h >= a.capacity ? h - a.capacity : h);
        a.state_out[1] = count - taken + freed;
        a.q_starts[a.seqs] = given;
    }
    if (!fill) return;
    __syncthreads();
    for (int t = tid; t < a.total; t += kScanThreads) fill_token(a, t, 0, max(a.seqs - 1, 0), given);
}

// The last sequence that begins at token t or before it, by a wavefront: two
// steps for 4096 sequences, where halves take twelve loads one after the other.
__device__ __forceinline__ int last_start(const PagesArgs& a, int t) {
    const int lane = threadIdx.x & 63;
    int s = 0;
    for (int step = a.seqs > 4096 ? 4096 : 64;; step /= 64) {
        const int i = s + lane * step;
        s += (__popcll(__ballot(i < a.seqs && a.q_starts[min(i, a.seqs)] <= t)) - 1) * step;
        if (step == 1) return s;
    }
}

// Slots and positions of many tokens, once the tables are made.  Latency again:
// 410000 tokens of 500 prompts took 9.8 us with a search and a page number for
// each, 7.6 with those of a thread one after the other.
__global__ void __launch_bounds__(kFillThreads)
kv_slots_kernel(PagesArgs a) {
    const int t0 = blockIdx.x * (kFillThreads * kFillEach), end = min(t0 + kFillThreads * kFillEach, a.total);
    const int tokens = a.q_starts[a.seqs];
    int first = 0, last = 0;
    if (t0 < tokens && a.seqs > 0) {   // the sequences that the workgroup's tokens are of
        first = last_start(a, t0);
        last = last_start(a, end - 1);
    }
    // a thread's tokens follow one another, so most are of the sequence and page of the one before
    const int mine = t0 + threadIdx.x * kFillEach;
    if (mine >= a.total) return;
    int slots[kFillEach], positions[kFillEach];
    int s = first, until = -1, to_slot = 0, held = -1, page = -1;
#pragma unroll
    for (int i = 0; i < kFillEach; ++i) {
        const int t = mine + i;
        slots[i] = positions[i] = -1;
        if (t >= tokens) continue;
        if (t >= until) {
            if (i > 0) {   // mostly the next one's first
                s = min(s + 1, last);
                until = a.q_starts[s + 1];
            }
            if (t >= until) {
                s = last_at_most(a.q_starts, s, last, t);
                until = a.q_starts[s + 1];
            }
            to_slot = a.kv_lens[s] - until;
            held = -1;
        }
        positions[i] = to_slot + t;
        if (positions[i] / kPage != held) {
            held = positions[i] / kPage;
            page = a.table[s * a.table_pitch + held];
        }
        if (page >= 0 && page < (1 << 25)) slots[i] = page * kPage + positions[i] % kPage;
    }
    auto store = [&](int32_t* to, const int (&x)[kFillEach]) {
        if (mine + kFillEach <= a.total) {
            __builtin_memcpy(to + mine, x, sizeof x);
        } else {
#pragma unroll
            for (int i = 0; i < kFillEach; ++i)
                if (mine + i < a.total) to[mine + i] = x[i];
        }
    };
    if (a.slots) store(a.slots, slots);
    if (a.positions) store(a.positions, positions);
}

// ---- trees

struct TreeArgs {
    const int32_t *kv_lens, *q_starts;
    int total, max_q;
};

// A sequence's first row, its nodes and the slots before them.
struct Tree {
    int row0, nodes, len;

    __device__ __forceinline__ Tree(const TreeArgs& a, int s) {
        row0 = min(max(a.q_starts[s], 0), a.total);
        nodes = min(max(min(max(a.q_starts[s + 1], 0), a.total) - row0, 0), a.max_q);
        len = max(a.kv_lens[s], 0);
    }
};

// A node's mask is its parent's with its own bit, so a node's way to the root
// doubles with every step: eight steps for 256 nodes.  A workgroup is a tree.
__global__ void __launch_bounds__(kTreeMax)
kv_tree_kernel(TreeArgs a, const int32_t* parents, uint64_t* masks, int32_t* positions, int words) {
    __shared__ uint64_t seen[kTreeMax][NVFP4_TREE_WORDS];
    __shared__ int up[kTreeMax];
    const Tree t(a, blockIdx.x);
    const int i = threadIdx.x;
    uint64_t m[NVFP4_TREE_WORDS] = {};
    int next = i;
    if (i < t.nodes) {
        const int p = parents[t.row0 + i];
        if (p >= 0 && p < i) next = p;
#pragma unroll
        for (int w = 0; w < NVFP4_TREE_WORDS; ++w) {
            m[w] = i >> 6 == w ? 1ull << (i & 63) : 0;
            seen[i][w] = m[w];
        }
        up[i] = next;
    }
    for (int reach = 1; reach < a.max_q; reach *= 2) {
        __syncthreads();
        uint64_t more[NVFP4_TREE_WORDS] = {};
        int far = next;
        if (i < t.nodes) {
#pragma unroll
            for (int w = 0; w < NVFP4_TREE_WORDS; ++w) more[w] = seen[next][w];
            far = up[next];
        }
        __syncthreads();
        if (i < t.nodes) {
            next = far;
            up[i] = far;
#pragma unroll
            for (int w = 0; w < NVFP4_TREE_WORDS; ++w) seen[i][w] = m[w] |= more[w];
        }
    }
    if (i >= t.nodes) return;
    int depth = -1;
#pragma unroll
    for (int w = 0; w < NVFP4_TREE_WORDS; ++w) {
        depth += __popcll(m[w]);
        if (w < words) masks[int64_t(t.row0 + i) * words + w] = m[w];
    }
    positions[t.row0 + i] = t.len - t.nodes + depth;
}

// Each node's continuation that the model agrees with, the lowest first (a
// minimum: no order matters), then one thread walks from the root.
__global__ void __launch_bounds__(kTreeMax)
tree_accept_kernel(TreeArgs a, const int32_t* drafted, const int32_t* parents, const int32_t* chosen, int32_t* path,
                   int32_t* counts, int32_t* token, int32_t* new_lens) {
    __shared__ int next[kTreeMax], way[kTreeMax];
    __shared__ int steps;
    const int s = blockIdx.x, i = threadIdx.x;
    const Tree t(a, s);
    if (i < kTreeMax) next[i] = kTreeMax;
    __syncthreads();
    if (i < t.nodes) {
        const int p = parents[t.row0 + i], mine = drafted[t.row0 + i];
        if (p >= 0 && p < i && mine >= 0 && chosen[t.row0 + p] == mine) atomicMin(&next[p], i);
    }
    __syncthreads();
    if (i == 0) {
        int n = 0;
        for (int at = 0; at < t.nodes; at = next[at]) way[n++] = at;
        steps = n;
        counts[s] = n;
        token[s] = n ? chosen[t.row0 + way[n - 1]] : -1;
        new_lens[s] = max(t.len - t.nodes + n, 0);
    }
    __syncthreads();
    if (i < a.max_q) path[int64_t(s) * a.max_q + i] = i < steps ? way[i] : -1;
}

int status() { return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

unsigned tree_threads(int64_t max_q) { return static_cast<unsigned>((max_q + 63) / 64 * 64); }

}  // namespace

extern "C" int nvfp4_kv_pages(const nvfp4_kv_pages_t* p, int32_t* state_out, int32_t* held_out, int32_t* kv_lens,
                              int32_t* q_starts, int32_t* slots, int32_t* positions, void* stream) {
    int st;
    if ((st = nvfp4::check_kv_pages(p, state_out, held_out, kv_lens, q_starts, slots, positions)) != NVFP4_OK) return st;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const PagesArgs a{p->pool, p->state, p->table, p->held, p->keep, p->fresh, state_out, held_out, kv_lens, q_starts,
                      slots, positions, p->table_pitch, static_cast<int>(p->capacity), static_cast<int>(p->seqs), static_cast<int>(p->total)};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool wanted = p->total > 0 && (slots || positions), inside = p->total <= kFillInline;
    hipLaunchKernelGGL(kv_pages_kernel, dim3(1), dim3(kScanThreads), 0, s, a, wanted && inside ? 1 : 0);
    if ((st = status()) != NVFP4_OK || !wanted || inside) return st;
    const int64_t each = kFillThreads * kFillEach;
    hipLaunchKernelGGL(kv_slots_kernel, dim3(static_cast<unsigned>((p->total + each - 1) / each)), dim3(kFillThreads), 0, s, a);
    return status();
}

extern "C" int nvfp4_kv_tree(const int32_t* parents, const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs,
                             int64_t total, int64_t max_q, uint64_t* masks, int32_t* positions, void* stream) {
    int st;
    if ((st = nvfp4::check_trees(kv_lens, q_starts, seqs, total, max_q)) != NVFP4_OK) return st;
    if (seqs == 0 || total == 0) return NVFP4_OK;
    if ((st = nvfp4::check_words(parents)) != NVFP4_OK || (st = nvfp4::check_words(positions)) != NVFP4_OK) return st;
    if ((st = nvfp4::check_words(masks)) != NVFP4_OK) return st;
    if (reinterpret_cast<uintptr_t>(masks) & 7) return NVFP4_ERR_ALIGN;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const TreeArgs a{kv_lens, q_starts, static_cast<int>(total), static_cast<int>(max_q)};
    hipLaunchKernelGGL(kv_tree_kernel, dim3(static_cast<unsigned>(seqs)), dim3(tree_threads(max_q)), 0,
                       static_cast<hipStream_t>(stream), a, parents, masks, positions, static_cast<int>((max_q + 63) / 64));
    return status();
}

extern "C" int nvfp4_tree_accept(const int32_t* drafted, const int32_t* parents, const int32_t* chosen,
                                 const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs, int64_t total,
                                 int64_t max_q, int32_t* path, int32_t* counts, int32_t* token, int32_t* new_lens,
                                 void* stream) {
    int st;
    if ((st = nvfp4::check_trees(kv_lens, q_starts, seqs, total, max_q)) != NVFP4_OK) return st;
    if (seqs == 0) return NVFP4_OK;
    for (const void* p : {static_cast<const void*>(path), static_cast<const void*>(counts), static_cast<const void*>(token),
                          static_cast<const void*>(new_lens)})
        if ((st = nvfp4::check_words(p)) != NVFP4_OK) return st;
    if (total > 0)
        for (const int32_t* p : {drafted, parents, chosen})
            if ((st = nvfp4::check_words(p)) != NVFP4_OK) return st;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const TreeArgs a{kv_lens, q_starts, static_cast<int>(total), static_cast<int>(max_q)};
    hipLaunchKernelGGL(tree_accept_kernel, dim3(static_cast<unsigned>(seqs)), dim3(tree_threads(max_q)), 0,
                       static_cast<hipStream_t>(stream), a, drafted, parents, chosen, path, counts, token, new_lens);
    return status();
}
