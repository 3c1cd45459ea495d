// The next token from a row of logits (include/nvfp4_kv.h, nvfp4_sample).
//
// A token's weight w = floor(2^30 exp((l - max l) / T)) is an integer that
// fp32 holds exactly (the exponential has 24 bits), so its bits order as the
// weights do, and sums of weights are exact in 64 bits: thresholds and the
// running mass come out the same in whatever order threads add.  Nothing is
// sorted.  Three launches over chunks of 16384 logits: the largest logit; the
// number and the mass of tokens by bins of the weight (6 % wide wherever the
// threshold lies: 5 bits of the exponent and 4 of the fraction); and one
// workgroup a row that finds the bins of the thresholds, gathers those bins'
// tokens into LDS (from the row itself if they are too many), settles the
// thresholds among them, and searches the running mass first by chunks and
// then inside one.  For 192 rows of 151552 fp32 logits the launches take 19, 28
// and 36 us: the first is bound by the read (6 TB/s with what the memory-side
// cache kept), the second by the exponential's 40 operations a token, the third
// by the slowest row's gather (a CU reads its row at 40 GB/s or so) and ranking.
// One row takes 2.5, 5.7 and 15 us, a chain of short steps and barriers.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "nvfp4_kv.h"
#include "nvfp4_common.h"
#include "setup.h"

namespace {

constexpr int kThreads = 1024;
constexpr int kRowWaves = kThreads / 64;
constexpr float kSteps = 1073741824.0f;      // 2^30
constexpr uint32_t kOneBits = 0x3f800000u;   // 1.0f: the smallest weight
constexpr uint32_t kTopKey = 30u << 23;      // 2^30: the largest
constexpr int kPer = 16;                     // tokens of a thread in one chunk
constexpr int kChunk = kThreads * kPer;
constexpr int kMaxChunks = (1 << 22) / kChunk;
constexpr int kBinShift = 19;                // bins by 5 bits of the exponent and 4 of the fraction: 6 % wide
constexpr int kBins = (30 << 4) + 1;
constexpr int kDigit = 10;                   // bits of a selection step within a bin
constexpr int kMassBits = 45;                // a chunk's bin: at most 2^14 tokens of 2^30, the number above the mass
constexpr unsigned long long kOneToken = 1ull << kMassBits;
constexpr int kListMax = 8192;
constexpr int kShort = 256;                  // list length up to which every token is ranked against all
constexpr uint32_t kNoKey = 0xffffffffu;
constexpr int kMaxThreads = 256;             // launch 1: pieces of 4096

struct SampleArgs {
    const void* logits;
    int64_t pitch;
    int vocab;
    const float* u;
    const float* temperature;
    const int32_t* top_k;
    const float* top_p;
    const float* min_p;
    int32_t* token;
    float* logprob;
    int chunks;
    int pieces;
    float* piece_max;            // [rows][pieces]
    unsigned long long* bins;    // [rows][chunks][kBins]
};

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int i) {
    float x;
    if constexpr (F32)
        x = static_cast<const float*>(row)[i];
    else
        x = bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
    return x != x ? -INFINITY : x;
}

// inverse is 1 / T, or +inf for the maximum alone: what is less is then at -inf.  0 or NaN for x NaN.
__device__ __forceinline__ float weight(float x, float top, float inverse) {
    const float w = floorf(expf((x - top) * inverse) * kSteps);
    return x == top ? kSteps : w;
}

__device__ __forceinline__ uint32_t weight_key(float w) { return f32_bits(w) - kOneBits; }   // w >= 1
__device__ __forceinline__ float key_weight(uint32_t k) { return bits_f32(k + kOneBits); }
__device__ __forceinline__ uint64_t key_mass(uint32_t k) { return uint32_t(key_weight(k)); }   // at most 2^30, or the bound of its bin

__device__ __forceinline__ int key_bin(uint32_t k) { return int(k >> kBinShift); }

// ---- launch 1: the largest logit of each piece

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int r, int size) {
    return static_cast<const char*>(a.logits) + int64_t(r) * a.pitch * size;
}

// The thread's kPer logits of the THREADS * kPer from `begin` on, 16 bytes at a
// time where a row has as many (WIDE), at whatever address it begins.  load()
// only loads, from places held to the row so that it never branches; clip()
// then puts what the row's last 16 bytes hold in their places, and -inf beyond
// the vocabulary; raw() gives element e, token token_at(e).  (A value at a time
// where rows are not whole 16 bytes: 51475 bf16 logits took 32 us instead of 24.)
template <bool F32, bool WIDE, int THREADS>
struct Piece {
    static constexpr int kVec = WIDE ? (F32 ? 4 : 8) : 1;
    u32x4 wide[WIDE ? kPer / kVec : 1];
    float one[WIDE ? 1 : kPer];

    static __device__ __forceinline__ int token_at(int begin, int e) {
        return begin + (e / kVec * THREADS + int(threadIdx.x)) * kVec + e % kVec;
    }
    __device__ __forceinline__ void load(const void* row, int begin, int vocab) {
#pragma unroll
        for (int v = 0; v < kPer / kVec; ++v) {
            const int i = min(token_at(begin, v * kVec), vocab - kVec);
            if constexpr (WIDE)
                __builtin_memcpy(&wide[v], static_cast<const char*>(row) + int64_t(i) * (F32 ? 4 : 2), 16);
            else
                one[v] = F32 ? static_cast<const float*>(row)[i] : bf16_to_f32(static_cast<const uint16_t*>(row)[i]);
        }
    }
    __device__ __forceinline__ float raw(int e) const {
        if constexpr (WIDE) {
            const int v = e / kVec, j = e % kVec;
            const uint32_t w = F32 ? wide[v][j % 4] : wide[v][j / 2 % 4];
            return F32 ? bits_f32(w) : bits_f32(j % 2 ? w & 0xffff0000u : w << 16);
        } else {
            return one[e];
        }
    }
    __device__ __forceinline__ void clip(int begin, int vocab) {
        if (token_at(begin, kPer - 1) < vocab) return;   // this thread's last
#pragma unroll
        for (int v = 0; v < kPer / kVec; ++v) {
            const int past = token_at(begin, v * kVec) + kVec - vocab;   // elements beyond the row
            if (past <= 0) continue;
            if constexpr (WIDE) {
                // what was loaded is the row's last kVec: the element wanted first lies `past` later
                constexpr int kBits = F32 ? 32 : 16;
                const uint64_t fill = F32 ? 0xff800000ff800000u : 0xff80ff80ff80ff80u;   // -inf
                uint64_t lo = uint64_t(wide[v][1]) << 32 | wide[v][0], hi = uint64_t(wide[v][3]) << 32 | wide[v][2];
                int shift = min(past, kVec) * kBits;
                if (shift >= 64) lo = hi, hi = fill, shift -= 64;
                if (shift >= 64) lo = fill, shift -= 64;
                if (shift > 0) {
                    lo = lo >> shift | hi << (64 - shift);
                    hi = hi >> shift | fill << (64 - shift);
                }
                wide[v] = u32x4{uint32_t(lo), uint32_t(lo >> 32), uint32_t(hi), uint32_t(hi >> 32)};
            } else {
                one[v] = -INFINITY;
            }
        }
    }
};

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kMaxThreads)
sample_max_kernel(SampleArgs a) {
    __shared__ float tmp[kMaxThreads / 64];
    const int r = blockIdx.y, c = blockIdx.x;
    Piece<F32, WIDE, kMaxThreads> p;
    const int begin = c * kMaxThreads * kPer;
    p.load(row_of(a, r, F32 ? 4 : 2), begin, a.vocab);   // (the last tokens again where there are none)
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) top = fmaxf(top, p.raw(j));   // passes NaN over
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kMaxThreads / 64; ++w) top = fmaxf(top, tmp[w]);
        a.piece_max[int64_t(r) * a.pieces + c] = top;
    }
}

__device__ __forceinline__ float row_max(const SampleArgs& a, int r) {
    float top = -INFINITY;
    for (int c = threadIdx.x & 63; c < a.pieces; c += 64) top = fmaxf(top, a.piece_max[int64_t(r) * a.pieces + c]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    return top;
}

__device__ __forceinline__ float row_inverse(const SampleArgs& a, int r) {
    const float t = a.temperature ? a.temperature[r] : 1.0f;
    return t > 0.0f ? 1.0f / t : INFINITY;
}

// Bounds of the logits whose weight is at least, or at most, w.  Wide by 1e-4 of
// the weight, which is far more than log and exp are off, and by 4 roundings of
// the bound itself.
__device__ __forceinline__ float logit_below(float w, float top, float inverse) {
    const float x = top + (logf(w / kSteps) - 1e-4f) / inverse;
    return x - fabsf(x) * 0x1p-21f;
}
__device__ __forceinline__ float logit_above(float w, float top, float inverse) {
    const float x = top + (logf(w / kSteps) + 1e-4f) / inverse;
    return x + fabsf(x) * 0x1p-21f;
}

struct Range {
    float lo, hi;
    __device__ __forceinline__ bool has(float x) const { return __builtin_amdgcn_fmed3f(x, lo, hi) == x; }   // not NaN
};

// ---- launch 2: each chunk's tokens and mass by bins of the weight

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads)
sample_bins_kernel(SampleArgs a) {
    __shared__ unsigned long long bins[kBins];
    const int r = blockIdx.y, c = blockIdx.x, tid = threadIdx.x;
    Piece<F32, WIDE, kThreads> p;
    p.load(row_of(a, r, F32 ? 4 : 2), c * kChunk, a.vocab);
    const float top = row_max(a, r), inverse = row_inverse(a, r);
    if (tid < kBins) bins[tid] = 0;
    __syncthreads();
    p.clip(c * kChunk, a.vocab);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float w = weight(p.raw(j), top, inverse);
        if (w >= 1.0f) atomicAdd(&bins[key_bin(weight_key(w))], kOneToken | (unsigned long long)uint32_t(w));
    }
    __syncthreads();
    if (tid < kBins) a.bins[(int64_t(r) * a.chunks + c) * kBins + tid] = bins[tid];
}

// ---- launch 3: the thresholds and the draw, one workgroup a row

// x of the lane that the row operation CTRL names, 0 where there is none or the
// row is not in ROWS: a move between lanes inside the vector unit (a scan by
// shuffles goes through LDS and took 1.3 us a workgroup, this 0.5 us).
template <int CTRL, int ROWS>
__device__ __forceinline__ uint64_t lane_move(uint64_t x) {
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(x)), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(x >> 32)), CTRL, ROWS, 0xf, false);
    return (uint64_t(hi) << 32) | lo;
}

// Sum over this lane and those before it.
__device__ __forceinline__ uint64_t wave_scan(uint64_t x) {
    x += lane_move<0x111, 0xf>(x);   // 1, 2, 4 and 8 lanes within each row of 16
    x += lane_move<0x112, 0xf>(x);
    x += lane_move<0x114, 0xf>(x);
    x += lane_move<0x118, 0xf>(x);
    x += lane_move<0x142, 0xa>(x);   // row 0's last into row 1, row 2's into row 3
    x += lane_move<0x143, 0xc>(x);   // the first half's last into rows 2 and 3
    return x;
}

__device__ __forceinline__ uint64_t last_lane(uint64_t x) {
    return (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(uint32_t(x >> 32)), 63))) << 32) |
           uint32_t(__builtin_amdgcn_readlane(int(uint32_t(x)), 63));
}

__device__ __forceinline__ uint64_t wave_sum(uint64_t x) { return last_lane(wave_scan(x)); }

// Sum over the threads before this one, and over all.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* tmp, uint64_t* all) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t sum = wave_scan(x);
    __syncthreads();
    if (lane == 63) tmp[wave] = sum;
    __syncthreads();
    const uint64_t mine = tmp[lane & (kRowWaves - 1)];
    const uint64_t waves = wave_scan(lane < kRowWaves ? mine : 0);   // lane i: wavefronts 0 .. i
    *all = last_lane(waves);
    const uint64_t before = wave == 0 ? 0 : (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(uint32_t(waves >> 32)), (wave - 1) & 63))) << 32) |
                                                uint32_t(__builtin_amdgcn_readlane(int(uint32_t(waves)), (wave - 1) & 63));
    return before + sum - x;
}

struct Listed {
    uint32_t key, index;   // kNoKey: not one of the bins' after all
};

struct RowShared {
    uint32_t count[kThreads];        // a selection step's bins
    uint64_t mass[kThreads];
    uint32_t above_n[kThreads];      // the row's bins: tokens and mass in higher ones
    uint64_t above_m[kThreads];
    uint64_t tmp[kRowWaves];
    uint64_t found[4];
    uint64_t chunk_mass[kMaxChunks];
    Listed list[kListMax];
    int listed;
    int chunk_has[kMaxChunks];       // tokens of those bins
};

// The lowest of the row's bins at which fewer than `most` tokens, or a mass
// below `limit`, lie above.  Both fall towards higher bins, so every wavefront
// finds it by itself in two looks of 64 lanes.  The caller knows that the rule
// ends among the row's tokens, and then the bin has one.
template <bool BY_MASS>
__device__ __forceinline__ int row_bin(const RowShared& sh, uint64_t most, double limit) {
    const int lane = threadIdx.x & 63;
    auto holds = [&](int bin) { return BY_MASS ? double(sh.above_m[bin]) < limit : sh.above_n[bin] < most; };
    static_assert(kBins <= 8 * 64);
    // bin 8 i + 7 of lane i: the first lane for which it holds has the bin among its eight
    const int eight = 8 * (__ffsll(static_cast<unsigned long long>(__ballot(holds(min(8 * lane + 7, kBins - 1))))) - 1);
    return min(eight + __ffsll(static_cast<unsigned long long>(__ballot(holds(min(eight + (lane & 7), kBins - 1))))) - 1, kBins - 1);
}

// Of `size` (at most kThreads) bins in sh.count and sh.mass the lowest with
// any token at which those above it are fewer than `most` (by count) or weigh
// less than `limit` (by mass), `above` of either being above all the bins.
// found = bin, above it, its tokens; bin ~0 if none.
template <bool BY_MASS>
__device__ void find_bin(RowShared& sh, int size, uint64_t above, uint64_t most, double limit) {
    const int tid = threadIdx.x, bin = size - 1 - tid;   // thread 0 has the highest
    const uint32_t n = bin >= 0 ? sh.count[bin] : 0;
    const uint64_t m = bin >= 0 ? sh.mass[bin] : 0;
    uint64_t all;
    const uint64_t mine = above + block_scan(BY_MASS ? m : n, sh.tmp, &all);
    const bool ok = n > 0 && (BY_MASS ? double(mine) < limit : mine < most);
    // of the threads that qualify the last one has the lowest bin
    const uint64_t ballot = __ballot(ok);
    __syncthreads();
    if (tid == 0) sh.found[0] = ~0ull;
    if ((tid & 63) == 0) sh.tmp[tid >> 6] = ballot ? uint64_t(tid + 63 - __clzll(ballot)) : ~0ull;
    __syncthreads();
    uint64_t last = ~0ull;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) last = sh.tmp[w] != ~0ull ? sh.tmp[w] : last;
    if (uint64_t(tid) == last) sh.found[0] = uint64_t(bin), sh.found[1] = mine, sh.found[2] = n;
    __syncthreads();
}

// The tokens of some bins, from the list in LDS or, where they are too many for it, from the row itself.
template <bool F32>
struct Tokens {
    const void* row;
    int vocab;
    float top, inverse;
    bool in_list;

    template <class Fn>
    __device__ __forceinline__ void each(const RowShared& sh, Fn fn) const {
        if (in_list) {
            for (int i = threadIdx.x; i < sh.listed; i += kThreads) fn(sh.list[i].key, sh.list[i].index);
        } else {
            for (int i = threadIdx.x; i < vocab; i += kThreads) {
                const float w = weight(logit<F32>(row, i), top, inverse);
                if (w >= 1.0f) fn(weight_key(w), uint32_t(i));
            }
        }
    }
};

// The exact key at which find_bin's rule stops within bin `bin`, `above` of
// either above the bin; found[1] and [2] as there, for the tokens of that key.
template <bool BY_MASS, bool F32>
__device__ uint32_t find_key(RowShared& sh, const Tokens<F32>& tokens, int bin, uint64_t above, uint64_t most, double limit) {
    uint32_t key = uint32_t(bin) << kBinShift, mask = ~0u << kBinShift;
    for (int shift = kBinShift - kDigit;; shift -= kDigit) {
        const int down = shift < 0 ? 0 : shift;
        const int size = 1 << (shift < 0 ? kDigit + shift : kDigit);
        sh.count[threadIdx.x] = 0, sh.mass[threadIdx.x] = 0;
        __syncthreads();
        tokens.each(sh, [&](uint32_t k, uint32_t) {
            if ((k & mask) != key) return;
            const int d = (k >> down) & (size - 1);
            // Small weights are few integers, the same for many tokens: a wavefront's
            // first one is counted at once for all lanes that share it.
            const int common = __builtin_amdgcn_readfirstlane(d);
            const uint64_t same = __ballot(d == common);
            if (d != common)
                atomicAdd(&sh.count[d], 1u);
            else if (int(threadIdx.x & 63) == __ffsll(static_cast<unsigned long long>(same)) - 1)
                atomicAdd(&sh.count[d], uint32_t(__popcll(same)));
            if (down > 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[d]), (unsigned long long)key_mass(k));
        });
        __syncthreads();
        // at the last step a bin is one weight; the thread's bin is the one that find_bin has it read
        const int own = size - 1 - int(threadIdx.x);
        if (down == 0 && own >= 0) sh.mass[own] = sh.count[own] * key_mass(key | uint32_t(own));
        find_bin<BY_MASS>(sh, size, above, most, limit);
        // a bin that holds the rule's last token always has one here
        key |= uint32_t(sh.found[0]) << down;
        mask |= uint32_t(size - 1) << down;
        above = sh.found[1];
        if (down == 0) return key;
    }
}

// The index below which `ties` of the tokens with this key lie.
template <bool F32>
__device__ uint32_t find_index(RowShared& sh, const Tokens<F32>& tokens, uint32_t key, uint64_t ties) {
    uint32_t at = 0, mask = 0;   // leading bits of the last index that stays
    uint64_t left = ties;
    for (int shift = kDigit + 2;; shift -= kDigit) {   // an index has 22 bits at most
        const int down = shift < 0 ? 0 : shift;
        const int size = 1 << (shift < 0 ? kDigit + shift : kDigit);
        sh.count[threadIdx.x] = 0;
        __syncthreads();
        tokens.each(sh, [&](uint32_t k, uint32_t i) {
            if (k == key && (i & mask) == at) atomicAdd(&sh.count[(i >> down) & (size - 1)], 1u);
        });
        __syncthreads();
        // the first bin at which the tokens up to it are `left` or more
        const int tid = threadIdx.x;
        const uint64_t n = tid < size ? sh.count[tid] : 0;
        uint64_t all;
        const uint64_t before = block_scan(n, sh.tmp, &all);
        if (before < left && before + n >= left) sh.found[0] = uint64_t(tid), sh.found[1] = before;
        __syncthreads();
        at |= uint32_t(sh.found[0]) << down;
        mask |= uint32_t(size - 1) << down;
        left -= sh.found[1];
        __syncthreads();
        if (down == 0) return at + 1;
    }
}

// The rules that cut a row's tokens, and where each may cut.
struct Cuts {
    bool by_count, by_mass, only_first;
    uint64_t k;
    float p;
    double low;
    int bin_k, bin_p_lo, bin_p_hi, bin_m;   // -1: none

    __device__ __forceinline__ bool wanted(int bin) const {
        return bin == bin_k || bin == bin_m || (bin >= bin_p_lo && bin <= bin_p_hi);
    }
};

// Tokens stay whose key is above `key`, or equal to it with an index below `index`.
struct Cut {
    uint32_t key, index;
};

// A list of few tokens: each is ranked against the others of its bin, which
// settles all rules at once.  WAVE: at most 64, one a lane, by every wavefront
// for itself and without a barrier; else one for four neighbouring lanes, which
// share its comparisons (256 tokens by one lane each took 26 us).
template <bool F32, bool WAVE>
__device__ Cut cut_short(RowShared& sh, const Cuts& c) {
    constexpr int kShare = WAVE ? 1 : kThreads / kShort;
    static_assert(kShare == 1 || kShare == 4);
    const int at_list = (threadIdx.x & (WAVE ? 63 : kThreads - 1)) / kShare, part = threadIdx.x % kShare, n = sh.listed;
    const bool mine = at_list < n && sh.list[at_list].key != kNoKey;
    const uint32_t key = mine ? sh.list[at_list].key : 0, index = mine ? sh.list[at_list].index : 0;
    const int bin = key_bin(key);
    uint32_t rank = 0;
    uint64_t before = 0;   // the mass before it in its bin
    const int others = __any(mine) ? n : 0;
    const uint32_t width = (uint32_t(bin + 1) << kBinShift) - key;   // from its key to its bin's end
#pragma unroll 8
    for (int i = part; i < others; i += kShare) {
        const uint32_t k = sh.list[i].key, higher = k - key;
        const bool first = higher < width && (higher > 0 || sh.list[i].index < index);
        rank += first;
        before += first ? uint32_t(key_weight(k)) : 0;
    }
    if constexpr (kShare == 4) {
        rank += __shfl_xor(rank, 1), before += __shfl_xor(before, 1);
        rank += __shfl_xor(rank, 2), before += __shfl_xor(before, 2);
    }
    uint64_t mass = sh.found[3];   // of the whole row
    if (c.by_count) {
        const bool top_k = mine && bin == c.bin_k && sh.above_n[bin] + rank < c.k;
        uint64_t in_bin = top_k && part == 0 ? key_mass(key) : 0;
        if constexpr (WAVE)
            in_bin = wave_sum(in_bin);
        else
            block_scan(in_bin, sh.tmp, &in_bin);
        mass = sh.above_m[c.bin_k] + in_bin;
    }
    const double limit = double(c.p) * double(mass);
    int at = max(c.bin_k, c.bin_m);   // the bin of the highest cut
    if (c.by_mass && !c.only_first) at = max(at, row_bin<true>(sh, 0, limit));
    bool stays = mine && bin == at;
    if (c.only_first)
        stays = stays && rank == 0 && sh.above_n[bin] == 0;
    else {
        if (c.by_count) stays = stays && sh.above_n[bin] + rank < c.k;
        if (c.by_mass) stays = stays && double(sh.above_m[bin] + before) < limit;
        stays = stays && double(key_weight(key)) >= c.low;
    }
    // the last that stays: the smallest of (key, then the larger index)
    uint64_t last = stays ? (uint64_t(key) << 32) | (0xffffffffu - index) : ~0ull;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) last = min(last, uint64_t(__shfl_xor(last, d)));
    if constexpr (!WAVE) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) sh.tmp[threadIdx.x >> 6] = last;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kRowWaves; ++w) last = min(last, sh.tmp[w]);
    }
    if (last == ~0ull) return Cut{((uint32_t(at) + 1) << kBinShift) - 1, 0};   // none of that bin
    return Cut{uint32_t(last >> 32), 0xffffffffu - uint32_t(last) + 1};
}

// Any number of tokens: radix selections within the bins.
template <bool F32>
__device__ Cut cut_long(RowShared& sh, const Cuts& c, const Tokens<F32>& tokens) {
    uint32_t key = 0;
    uint64_t stay = ~0ull, same = 0;   // of the `same` tokens at the key the first `stay` stay
    uint64_t mass = sh.found[3];
    __syncthreads();
    if (c.only_first) {
        key = kTopKey, stay = 1, same = ~0ull;
    } else {
        if (c.by_count) {
            key = find_key<false>(sh, tokens, c.bin_k, sh.above_n[c.bin_k], c.k, 0.0);
            stay = c.k - sh.found[1];
            same = sh.found[2];
            uint64_t part = 0, in_bin;   // the mass of the top k
            tokens.each(sh, [&](uint32_t t, uint32_t) { part += key_bin(t) == c.bin_k && t > key ? key_mass(t) : 0; });
            block_scan(part, sh.tmp, &in_bin);
            mass = sh.above_m[c.bin_k] + in_bin + stay * key_mass(key);
        }
        if (c.by_mass) {
            const double limit = double(c.p) * double(mass);
            const int bin = row_bin<true>(sh, 0, limit);
            const uint32_t key_p = find_key<true>(sh, tokens, bin, sh.above_m[bin], 0, limit);
            const uint64_t above = sh.found[1], n = sh.found[2], w = key_mass(key_p);
            // of these the e-th stays if above + e w < limit
            uint64_t e = uint64_t(fmin((limit - double(above)) / double(w), double(n)));
            while (e > 0 && !(double(above + (e - 1) * w) < limit)) --e;
            while (e < n && double(above + e * w) < limit) ++e;
            if (!c.by_count || key_p > key)
                key = key_p, stay = e, same = n;
            else if (key_p == key)
                stay = min(stay, e);
        }
        if (c.bin_m >= 0) {
            // low has the 24 bits of min_p, so the least weight that stays is exact in fp32
            const uint32_t key_m = weight_key(float(ceil(c.low)));
            if (key < key_m) key = key_m, stay = same = ~0ull;
        }
    }
    __syncthreads();
    return Cut{key, stay < same ? find_index(sh, tokens, key, stay) : 0xffffffffu};
}

template <bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads)
sample_draw_kernel(SampleArgs a) {
    extern __shared__ char raw[];
    RowShared& sh = *reinterpret_cast<RowShared*>(raw);
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const void* row = row_of(a, r, F32 ? 4 : 2);
    const uint64_t* bins = reinterpret_cast<const uint64_t*>(a.bins) + int64_t(r) * a.chunks * kBins;

    // Every wavefront takes one chunk's bins (and every sixteenth after it),
    // kept in registers: the sums over chunks go through LDS.
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int kLaneBins = (kBins + 63) / 64;
    uint64_t held[kLaneBins];
    auto load_bins = [&](int c, uint64_t (&to)[kLaneBins]) {
#pragma unroll
        for (int i = 0; i < kLaneBins; ++i) to[i] = bins[c * kBins + min(lane + 64 * i, kBins - 1)];
    };
    load_bins(min(wave, a.chunks - 1), held);
    auto each_chunk = [&](auto fn) {   // fn(chunk, its bins of this lane)
        if (wave < a.chunks) fn(wave, held);
        for (int c = wave + kRowWaves; c < a.chunks; c += kRowWaves) {
            uint64_t more[kLaneBins];
            load_bins(c, more);
            fn(c, more);
        }
    };
    if (tid < kBins) sh.count[tid] = 0, sh.mass[tid] = 0;
    if (tid == 0) sh.listed = 0;
    __syncthreads();
    each_chunk([&](int, const uint64_t (&x)[kLaneBins]) {
#pragma unroll
        for (int i = 0; i < kLaneBins; ++i) {
            const int bin = lane + 64 * i;
            if (bin >= kBins || x[i] == 0) continue;
            atomicAdd(&sh.count[bin], uint32_t(x[i] >> kMassBits));
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[bin]), (unsigned long long)(x[i] & (kOneToken - 1)));
        }
    });
    const float top = row_max(a, r), inverse = row_inverse(a, r);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    Cuts cuts;
    const int k = !a.temperature || a.temperature[r] > 0.0f ? (a.top_k ? a.top_k[r] : 0) : 1;
    cuts.k = uint64_t(max(k, 0));
    cuts.p = a.top_p ? a.top_p[r] : 1.0f;
    cuts.low = a.min_p ? double(a.min_p[r]) * double(kSteps) : 0.0;
    // the row's bins, the highest at thread 0, and what lies above each
    __syncthreads();
    const int my_bin = kBins - 1 - tid;
    const uint64_t n = my_bin >= 0 ? sh.count[my_bin] : 0, m = my_bin >= 0 ? sh.mass[my_bin] : 0;
    uint64_t some, mass;
    const uint64_t above_n = block_scan(n, sh.tmp, &some), above_m = block_scan(m, sh.tmp, &mass);
    if (my_bin >= 0) sh.above_n[my_bin] = uint32_t(above_n), sh.above_m[my_bin] = above_m;
    if (tid == 0) sh.found[3] = mass;
    __syncthreads();

    // Which bins hold a cut: that of the top k, those that may hold the top
    // p's (the mass of the top k is known to within its last bin), and min_p's.
    cuts.by_count = k > 0 && uint64_t(k) < some;
    cuts.by_mass = !(cuts.p >= 1.0f);
    cuts.only_first = !(cuts.low <= double(kSteps)) || (cuts.by_mass && !(double(cuts.p) * double(mass) > 0.0));
    cuts.bin_k = cuts.bin_p_lo = cuts.bin_p_hi = cuts.bin_m = -1;
    if (cuts.only_first) {
        cuts.bin_m = kBins - 1;
    } else {
        uint64_t mass_lo = mass, mass_hi = mass;
        if (cuts.by_count) {
            cuts.bin_k = row_bin<false>(sh, cuts.k, 0.0);
            const uint64_t in_bin = cuts.k - sh.above_n[cuts.bin_k];
            mass_lo = sh.above_m[cuts.bin_k] + in_bin * key_mass(uint32_t(cuts.bin_k) << kBinShift);
            mass_hi = sh.above_m[cuts.bin_k] + in_bin * key_mass(uint32_t(cuts.bin_k + 1) << kBinShift);
        }
        if (cuts.by_mass) {
            cuts.bin_p_lo = row_bin<true>(sh, 0, double(cuts.p) * double(mass_hi));
            cuts.bin_p_hi = row_bin<true>(sh, 0, double(cuts.p) * double(mass_lo));
        }
        if (cuts.low > 1.0) cuts.bin_m = key_bin(weight_key(float(fmin(ceil(cuts.low), double(kSteps)))));
    }
    if (cuts.only_first) cuts.by_count = cuts.by_mass = false;
    const bool any = cuts.bin_k >= 0 || cuts.bin_p_hi >= 0 || cuts.bin_m >= 0;

    Cut cut{0, 0xffffffffu};
    Tokens<F32> tokens{row, a.vocab, top, inverse, true};
    if (any) {
        // Their tokens into the list, from the chunks that have any.
        auto tokens_of = [&](int lo, int hi) {   // of a range of bins
            if (hi < 0) return 0u;
            return (lo > 0 ? sh.above_n[lo - 1] : uint32_t(some)) - sh.above_n[hi];
        };
        const uint64_t many = uint64_t(tokens_of(cuts.bin_k, cuts.bin_k)) + tokens_of(cuts.bin_p_lo, cuts.bin_p_hi) +
                              tokens_of(cuts.bin_m, cuts.bin_m);   // or less, where they overlap
        tokens.in_list = many <= uint64_t(kListMax) && top < INFINITY;   // d of an infinite logit is none
        if (tokens.in_list) {
            each_chunk([&](int c, const uint64_t (&x)[kLaneBins]) {
                bool has = false;
#pragma unroll
                for (int i = 0; i < kLaneBins; ++i) has |= lane + 64 * i < kBins && x[i] != 0 && cuts.wanted(lane + 64 * i);
                has = __any(has);
                if (lane == 0) sh.chunk_has[c] = has;
            });
            __syncthreads();
            // First by the logit alone, a little wider than the bins.  What
            // passes is few, and gets its exact weight afterwards.
            Range r0{INFINITY, -INFINITY}, r1 = r0, r2 = r0;
            int ranges = 0;
            auto add_range = [&](int lo, int hi) {
                r2 = r1, r1 = r0;
                r0 = Range{logit_below(key_weight(uint32_t(lo) << kBinShift), top, inverse),
                           logit_above(key_weight(uint32_t(hi + 1) << kBinShift) + 1.0f, top, inverse)};
                ++ranges;
            };
            if (cuts.bin_p_hi >= 0) add_range(cuts.bin_p_lo, cuts.bin_p_hi);
            if (cuts.bin_k >= 0 && (cuts.bin_k < cuts.bin_p_lo || cuts.bin_k > cuts.bin_p_hi)) add_range(cuts.bin_k, cuts.bin_k);
            if (cuts.bin_m >= 0 && (cuts.bin_m < cuts.bin_p_lo || cuts.bin_m > cuts.bin_p_hi) && cuts.bin_m != cuts.bin_k)
                add_range(cuts.bin_m, cuts.bin_m);
            auto next_chunk = [&](int c) {
                while (c < a.chunks && !sh.chunk_has[c]) ++c;
                return c;
            };
            auto gather = [&](auto count) {
                constexpr int kRanges = decltype(count)::value;
                int c = next_chunk(0);
                Piece<F32, WIDE, kThreads> piece, ahead;
                piece.load(row, min(c, a.chunks - 1) * kChunk, a.vocab);
                while (c < a.chunks) {
                    const int next = next_chunk(c + 1);
                    ahead.load(row, min(next, a.chunks - 1) * kChunk, a.vocab);   // also past the end, so that no wait depends on a branch
                    piece.clip(c * kChunk, a.vocab);
                    uint64_t hits[kPer];   // of the wavefront: places in the list are taken for all its tokens at once
                    int many_hits = 0;
#pragma unroll
                    for (int j = 0; j < kPer; ++j) {
                        const float x = piece.raw(j);
                        hits[j] = __ballot(r0.has(x));
                        if constexpr (kRanges > 1) hits[j] |= __ballot(r1.has(x));
                        if constexpr (kRanges > 2) hits[j] |= __ballot(r2.has(x));
                        many_hits += __popcll(hits[j]);
                    }
                    if (many_hits) {
                        int first = 0;
                        if (lane == 0) first = atomicAdd(&sh.listed, many_hits);   // the order of the list matters to nothing below
                        first = __builtin_amdgcn_readfirstlane(first);
                        if (first + many_hits <= kListMax) {   // else the list is not used
#pragma unroll
                            for (int j = 0; j < kPer; ++j) {
                                if (!hits[j]) continue;
                                if (hits[j] >> lane & 1)
                                    sh.list[__builtin_amdgcn_mbcnt_hi(uint32_t(hits[j] >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(hits[j]), first))] =
                                        Listed{f32_bits(piece.raw(j)), uint32_t(piece.token_at(c * kChunk, j))};
                                first += __popcll(hits[j]);
                            }
                        }
                    }
                    piece = ahead;
                    c = next;
                }
            };
            if (ranges == 1)
                gather(std::integral_constant<int, 1>{});
            else if (ranges == 2)
                gather(std::integral_constant<int, 2>{});
            else
                gather(std::integral_constant<int, 3>{});
            __syncthreads();
            tokens.in_list = sh.listed <= kListMax;
            if (tokens.in_list)
                for (int i = tid; i < sh.listed; i += kThreads) {
                    const float w = weight(bits_f32(sh.list[i].key), top, inverse);
                    const uint32_t t = w >= 1.0f && int(sh.list[i].index) < a.vocab ? weight_key(w) : kNoKey;
                    sh.list[i].key = t != kNoKey && cuts.wanted(key_bin(t)) ? t : kNoKey;
                }
            __syncthreads();
        }
        cut = tokens.in_list && sh.listed <= 64       ? cut_short<F32, true>(sh, cuts)
              : tokens.in_list && sh.listed <= kShort ? cut_short<F32, false>(sh, cuts)
                                                      : cut_long<F32>(sh, cuts, tokens);
    }

    // The mass that stays, by chunks: whole bins above the cut's, and that bin's tokens.
    const int bin = any ? key_bin(cut.key) : -1;
    __syncthreads();
    each_chunk([&](int c, const uint64_t (&x)[kLaneBins]) {
        uint64_t sum = 0;
#pragma unroll
        for (int i = 0; i < kLaneBins; ++i) {
            const int b = lane + 64 * i;
            sum += b < kBins && b > bin ? x[i] & (kOneToken - 1) : 0;
        }
        sum = wave_sum(sum);
        if (lane == 0) sh.chunk_mass[c] = sum;
    });
    __syncthreads();
    if (any)
        tokens.each(sh, [&](uint32_t t, uint32_t i) {
            if (key_bin(t) == bin && (t > cut.key || (t == cut.key && i < cut.index)))
                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunk_mass[i / kChunk]), (unsigned long long)key_mass(t));
        });
    __syncthreads();
    uint64_t total;
    const uint64_t chunk_before = block_scan(tid < a.chunks ? sh.chunk_mass[tid] : 0, sh.tmp, &total);
    const double at = double(a.u[r]) * double(total);
    uint64_t target = at >= 0.0 ? uint64_t(fmin(at, 9007199254740992.0)) : 0;
    target = min(target, total - 1);
    if (tid < a.chunks && target >= chunk_before && target < chunk_before + sh.chunk_mass[tid])
        sh.found[0] = uint64_t(tid), sh.found[1] = chunk_before;
    __syncthreads();
    const int begin = int(sh.found[0]) * kChunk + tid * kPer;
    const uint64_t base = sh.found[1];
    Piece<F32, WIDE, 1> last;   // consecutive tokens
    const int lane_begin = begin - tid * Piece<F32, WIDE, 1>::kVec;
    last.load(row, lane_begin, a.vocab);
    last.clip(lane_begin, a.vocab);
    uint32_t w[kPer];
    uint64_t sum = 0;
    // most rows keep few tokens: what lies below the cut needs no exponential
    const float low = any ? logit_below(key_weight(cut.key), top, inverse) : -INFINITY;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        w[j] = 0;
        const float x = last.raw(j);
        if (!__any(!(x < low))) continue;   // (below an infinite maximum low is NaN)
        const float y = weight(x, top, inverse);
        const uint32_t t = y >= 1.0f ? weight_key(y) : 0;
        w[j] = y >= 1.0f && (t > cut.key || (t == cut.key && uint32_t(begin + j) < cut.index)) ? uint32_t(y) : 0;
        sum += w[j];
    }
    uint64_t all;
    uint64_t run = base + block_scan(sum, sh.tmp, &all);
    if (target < run || target >= run + sum) return;
    int token = 0;
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const bool here = target >= run && target < run + w[j];
        token = here ? begin + j : token;
        mine = here ? w[j] : mine;
        run += w[j];
    }
    a.token[r] = token;
    if (a.logprob) a.logprob[r] = float(log(double(mine) / double(total)));
}

bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

int check_sample_shape(int64_t rows, int64_t vocab) {
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= (int64_t(1) << 22) ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

int64_t pieces_of(int64_t vocab) { return (vocab + kMaxThreads * kPer - 1) / (kMaxThreads * kPer); }

// The bins of every row's chunks, then the pieces' maxima.
int64_t bins_bytes(int64_t rows, int64_t chunks) { return (rows * chunks * kBins * 8 + 15) / 16 * 16; }

template <bool F32, bool WIDE>
int launch_sample(const SampleArgs& a, int64_t rows, hipStream_t s) {
    const unsigned n = static_cast<unsigned>(rows);
    hipLaunchKernelGGL((sample_max_kernel<F32, WIDE>), dim3(a.pieces, n), dim3(kMaxThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    hipLaunchKernelGGL((sample_bins_kernel<F32, WIDE>), dim3(a.chunks, n), dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    hipLaunchKernelGGL((sample_draw_kernel<F32, WIDE>), dim3(n), dim3(kThreads), sizeof(RowShared), s, a);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace

namespace nvfp4 {

int sample_setup() {
    for (const void* fn : {reinterpret_cast<const void*>(sample_draw_kernel<true, true>),
                           reinterpret_cast<const void*>(sample_draw_kernel<true, false>),
                           reinterpret_cast<const void*>(sample_draw_kernel<false, true>),
                           reinterpret_cast<const void*>(sample_draw_kernel<false, false>)})
        if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLdsBytes) != hipSuccess) return NVFP4_ERR_HIP;
    return NVFP4_OK;
}

}  // namespace nvfp4

extern "C" int nvfp4_sample_workspace(int64_t rows, int64_t vocab, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    const int st = check_sample_shape(rows, vocab);
    const int64_t chunks = (vocab + kChunk - 1) / kChunk;
    if (st == NVFP4_OK) *bytes = bins_bytes(rows, chunks) + rows * pieces_of(vocab) * int64_t(sizeof(float));
    return st;
}

extern "C" int nvfp4_sample(const void* logits, int logits_type, int64_t rows, int64_t vocab, int64_t pitch,
                            const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, int32_t* token, float* logprob, void* workspace,
                            int64_t workspace_bytes, void* stream) {
    int64_t need;
    int st = nvfp4_sample_workspace(rows, vocab, &need);
    if (st != NVFP4_OK) return st;
    if (pitch < vocab || pitch > (int64_t(1) << 31)) return NVFP4_ERR_SHAPE;
    if (logits_type != NVFP4_LOGITS_BF16 && logits_type != NVFP4_LOGITS_F32) return NVFP4_ERR_DTYPE;
    if (rows == 0) return NVFP4_OK;
    if (!logits || !u || !token || (need > 0 && !workspace)) return NVFP4_ERR_NULL;
    if (misaligned(logits, logits_type == NVFP4_LOGITS_F32 ? 4 : 2) || misaligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    for (const void* p : {(const void*)u, (const void*)temperature, (const void*)top_k, (const void*)top_p,
                          (const void*)min_p, (const void*)token, (const void*)logprob})
        if (misaligned(p, 4)) return NVFP4_ERR_ALIGN;
    if (need > workspace_bytes) return NVFP4_ERR_SCRATCH;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const int64_t chunks = (vocab + kChunk - 1) / kChunk;
    char* ws = static_cast<char*>(workspace);
    const SampleArgs a{logits, pitch, static_cast<int>(vocab), u, temperature, top_k, top_p, min_p, token, logprob,
                       static_cast<int>(chunks), static_cast<int>(pieces_of(vocab)),
                       reinterpret_cast<float*>(ws + bins_bytes(rows, chunks)),
                       reinterpret_cast<unsigned long long*>(ws)};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool f32 = logits_type == NVFP4_LOGITS_F32, wide = vocab >= (f32 ? 4 : 8);
    if (f32) return wide ? launch_sample<true, true>(a, rows, s) : launch_sample<true, false>(a, rows, s);
    return wide ? launch_sample<false, true>(a, rows, s) : launch_sample<false, false>(a, rows, s);
}
