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
// then inside one.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

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
    float* chunk_max;            // [rows][chunks]
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

// inverse is 1 / T, or 0 for the maximum alone.
__device__ __forceinline__ float weight(float x, float top, float inverse) {
    if (x == top) return kSteps;
    if (inverse == 0.0f) return 0.0f;
    return floorf(expf((x - top) * inverse) * kSteps);
}

__device__ __forceinline__ uint32_t weight_key(float w) { return f32_bits(w) - kOneBits; }   // w >= 1
__device__ __forceinline__ float key_weight(uint32_t k) { return bits_f32(k + kOneBits); }

__device__ __forceinline__ int key_bin(uint32_t k) { return int(k >> kBinShift); }

// ---- launch 1: the largest logit of each chunk

template <bool F32>
__device__ __forceinline__ void load_chunk(const void* row, int begin, int vocab, float (&x)[kPer]) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = begin + j * kThreads + int(threadIdx.x);
        x[j] = i < vocab ? logit<F32>(row, i) : -INFINITY;
    }
}

__device__ __forceinline__ const void* row_of(const SampleArgs& a, int r, int size) {
    return static_cast<const char*>(a.logits) + int64_t(r) * a.pitch * size;
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
sample_max_kernel(SampleArgs a) {
    __shared__ float tmp[kRowWaves];
    const int r = blockIdx.y, c = blockIdx.x;
    float x[kPer];
    load_chunk<F32>(row_of(a, r, F32 ? 4 : 2), c * kChunk, a.vocab, x);
    float top = x[0];
#pragma unroll
    for (int j = 1; j < kPer; ++j) top = fmaxf(top, x[j]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kRowWaves; ++w) top = fmaxf(top, tmp[w]);
        a.chunk_max[int64_t(r) * a.chunks + c] = top;
    }
}

__device__ __forceinline__ float row_max(const SampleArgs& a, int r) {
    float top = -INFINITY;
    for (int c = threadIdx.x & 63; c < a.chunks; c += 64) top = fmaxf(top, a.chunk_max[int64_t(r) * a.chunks + c]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    return top;
}

__device__ __forceinline__ float row_inverse(const SampleArgs& a, int r) {
    const float t = a.temperature ? a.temperature[r] : 1.0f;
    return t > 0.0f ? 1.0f / t : 0.0f;
}

// ---- launch 2: each chunk's tokens and mass by bins of the weight

template <bool F32>
__global__ void __launch_bounds__(kThreads)
sample_bins_kernel(SampleArgs a) {
    __shared__ unsigned long long bins[kBins];
    const int r = blockIdx.y, c = blockIdx.x, tid = threadIdx.x;
    float x[kPer];
    load_chunk<F32>(row_of(a, r, F32 ? 4 : 2), c * kChunk, a.vocab, x);
    const float top = row_max(a, r), inverse = row_inverse(a, r);
    if (tid < kBins) bins[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const float w = weight(x[j], top, inverse);
        if (w >= 1.0f) atomicAdd(&bins[key_bin(weight_key(w))], kOneToken | (unsigned long long)w);
    }
    __syncthreads();
    if (tid < kBins) a.bins[(int64_t(r) * a.chunks + c) * kBins + tid] = bins[tid];
}

// ---- launch 3: the thresholds and the draw, one workgroup a row

__device__ __forceinline__ uint64_t wave_sum(uint64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// Sum over the threads before this one, and over all.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* tmp, uint64_t* all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint64_t sum = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t y = __shfl_up(sum, d);
        if (lane >= d) sum += y;
    }
    __syncthreads();
    if (lane == 63) tmp[wave] = sum;
    __syncthreads();
    uint64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) {
        const uint64_t y = tmp[w];
        if (w < wave) before += y;
        total += y;
    }
    *all = total;
    return before + sum - x;
}

struct RowShared {
    uint32_t count[kThreads];
    uint64_t mass[kThreads];
    uint64_t tmp[kRowWaves];
    uint64_t found[4];
    uint64_t chunk_mass[kMaxChunks];
    uint32_t list_key[kListMax];
    uint32_t list_index[kListMax];
    int listed;
};

// Of `size` (at most kThreads) bins in sh.count and sh.mass the lowest with
// any token at which those above it are fewer than `most` (by count) or weigh
// less than `limit` (by mass), `above` of either being above all the bins.
// found = bin, above it, its tokens, its mass; bin -1 if none.
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
    if (uint64_t(tid) == last) sh.found[0] = uint64_t(bin), sh.found[1] = mine, sh.found[2] = n, sh.found[3] = m;
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
            for (int i = threadIdx.x; i < sh.listed; i += kThreads) fn(sh.list_key[i], sh.list_index[i]);
        } else {
            for (int i = threadIdx.x; i < vocab; i += kThreads) {
                const float w = weight(logit<F32>(row, i), top, inverse);
                if (w >= 1.0f) fn(weight_key(w), uint32_t(i));
            }
        }
    }
};

// The exact key at which find_bin's rule stops within bin `bin`, above of
// either above the bin: found as there, for the tokens of that key.
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
            atomicAdd(&sh.count[d], 1u);
            atomicAdd(reinterpret_cast<unsigned long long*>(&sh.mass[d]), (unsigned long long)key_weight(k));
        });
        __syncthreads();
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

template <bool F32>
__global__ void __launch_bounds__(kThreads)
sample_draw_kernel(SampleArgs a) {
    extern __shared__ char raw[];
    RowShared& sh = *reinterpret_cast<RowShared*>(raw);
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const void* row = row_of(a, r, F32 ? 4 : 2);
    const float top = row_max(a, r), inverse = row_inverse(a, r);
    if (top == -INFINITY) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    const int k = inverse > 0.0f ? (a.top_k ? a.top_k[r] : 0) : 1;
    const float p = a.top_p ? a.top_p[r] : 1.0f;
    double low = a.min_p ? double(a.min_p[r]) * double(kSteps) : 0.0;
    const uint64_t* bins = reinterpret_cast<const uint64_t*>(a.bins) + int64_t(r) * a.chunks * kBins;

    // the row's bins
    uint64_t mine_n = 0, mine_m = 0;
    if (tid < kBins)
        for (int c = 0; c < a.chunks; ++c) {
            const uint64_t x = bins[c * kBins + tid];
            mine_n += x >> kMassBits, mine_m += x & (kOneToken - 1);
        }
    uint64_t some, mass;
    block_scan(mine_n, sh.tmp, &some);
    block_scan(mine_m, sh.tmp, &mass);
    auto put_bins = [&] {
        __syncthreads();
        sh.count[tid] = uint32_t(mine_n), sh.mass[tid] = mine_m;
        __syncthreads();
    };
    put_bins();

    // Which bins hold a threshold: that of the top k, those that may hold the
    // top p's (the mass of the top k is known to within its last bin), and
    // that of min_p.
    const bool by_count = k > 0 && uint64_t(k) < some;
    bool only_first = !(low <= double(kSteps));
    int bin_k = -1, bin_p_lo = -1, bin_p_hi = -1, bin_m = -1;
    uint64_t above_k = 0;
    uint64_t mass_lo = mass, mass_hi = mass;
    if (by_count) {
        find_bin<false>(sh, kBins, 0, uint64_t(k), 0.0);
        bin_k = int(sh.found[0]);
        above_k = sh.found[1];
        const uint64_t in_bin = uint64_t(k) - above_k;
        uint64_t all;
        const uint64_t above_mass = (block_scan(tid < kBins && tid > bin_k ? mine_m : 0, sh.tmp, &all), all);
        mass_lo = above_mass + in_bin * uint64_t(key_weight(uint32_t(bin_k) << kBinShift));
        mass_hi = above_mass + in_bin * uint64_t(key_weight(uint32_t(bin_k + 1) << kBinShift));
    }
    const bool by_mass = !(p >= 1.0f);
    if (by_mass) {
        if (!(double(p) * double(mass) > 0.0)) only_first = true;
        if (!only_first) {
            find_bin<true>(sh, kBins, 0, 0, double(p) * double(mass_hi));
            bin_p_lo = int(sh.found[0]);
            find_bin<true>(sh, kBins, 0, 0, double(p) * double(mass_lo));
            bin_p_hi = int(sh.found[0]);
        }
    }
    if (low > 1.0 && !only_first) bin_m = key_bin(weight_key(float(fmin(ceil(low), double(kSteps)))));
    if (only_first) bin_k = bin_p_lo = bin_p_hi = -1, bin_m = kBins - 1;
    const int lowest = min(min(bin_k < 0 ? kBins : bin_k, bin_p_lo < 0 ? kBins : bin_p_lo), bin_m < 0 ? kBins : bin_m);
    auto wanted = [&](int bin) { return bin == bin_k || bin == bin_m || (bin >= bin_p_lo && bin <= bin_p_hi); };

    // Their tokens into the list.
    Tokens<F32> tokens{row, a.vocab, top, inverse, true};
    if (lowest < kBins) {
        uint64_t many;
        block_scan(tid < kBins && wanted(tid) ? mine_n : 0, sh.tmp, &many);
        tokens.in_list = many <= uint64_t(kListMax);
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        if (tokens.in_list) {
            // nothing below this can lie in the lowest of the bins (log and exp are off by far less than 1e-3)
            const float cut = logf(key_weight(uint32_t(lowest) << kBinShift) / kSteps) - 1e-3f;
            for (int begin = 0; begin < a.vocab; begin += kChunk) {
                float x[kPer];
                load_chunk<F32>(row, begin, a.vocab, x);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    if (!(x[j] == top) && !((x[j] - top) * inverse >= cut)) continue;
                    const float w = weight(x[j], top, inverse);
                    if (w < 1.0f || !wanted(key_bin(weight_key(w)))) continue;
                    const int at = atomicAdd(&sh.listed, 1);   // the order of the list matters to nothing below
                    sh.list_key[at] = weight_key(w);
                    sh.list_index[at] = uint32_t(begin + j * kThreads + tid);
                }
            }
            __syncthreads();
        }
    }

    // The threshold: tokens stay above `key`, and at it below index `index`.
    uint32_t key = 0, index = 0xffffffffu;
    uint64_t stay = ~0ull, same = 0;   // of the `same` tokens at the key the first `stay` stay
    if (only_first) {
        key = kTopKey;
        stay = 1;
        uint64_t n;
        block_scan(tid == kBins - 1 ? mine_n : 0, sh.tmp, &n);
        same = n;
    } else {
        if (by_count) {
            key = find_key<false>(sh, tokens, bin_k, above_k, uint64_t(k), 0.0);
            stay = uint64_t(k) - sh.found[1];
            same = sh.found[2];
            uint64_t part = 0;   // the mass of the top k
            tokens.each(sh, [&](uint32_t t, uint32_t) { part += key_bin(t) == bin_k && t > key ? uint64_t(key_weight(t)) : 0; });
            uint64_t in_bin, above;
            block_scan(part, sh.tmp, &in_bin);
            block_scan(tid < kBins && tid > bin_k ? mine_m : 0, sh.tmp, &above);
            mass = above + in_bin + stay * uint64_t(key_weight(key));
        }
        if (by_mass) {
            const double limit = double(p) * double(mass);
            put_bins();
            find_bin<true>(sh, kBins, 0, 0, limit);
            const int bin = int(sh.found[0]);
            const uint64_t above_bin = sh.found[1];
            const uint32_t key_p = find_key<true>(sh, tokens, bin, above_bin, 0, limit);
            const uint64_t above = sh.found[1], n = sh.found[2], w = uint64_t(key_weight(key_p));
            // of these the e-th stays if above + e w < limit
            uint64_t e = uint64_t(fmin((limit - double(above)) / double(w), double(n)));
            while (e > 0 && !(double(above + (e - 1) * w) < limit)) --e;
            while (e < n && double(above + e * w) < limit) ++e;
            if (!by_count || key_p > key)
                key = key_p, stay = e, same = n;
            else if (key_p == key)
                stay = min(stay, e);
        }
        if (bin_m >= 0) {
            // low has the 24 bits of min_p, so the least weight that stays is exact in fp32
            const uint32_t key_m = weight_key(float(ceil(low)));
            if (key < key_m) key = key_m - 1, stay = 0, same = 0;
        }
    }
    if (stay < same) index = stay ? find_index(sh, tokens, key, stay) : 0;
    const bool none_at_key = stay == 0;
    if (none_at_key) index = 0;

    // The mass that stays, by chunks: whole bins above the threshold's, and that bin's tokens.
    const int bin = key_bin(key);
    const bool all_of_bin = key == 0 && !none_at_key && index == 0xffffffffu;   // no threshold at all
    for (int c = tid; c < a.chunks; c += kThreads) sh.chunk_mass[c] = 0;
    __syncthreads();
    for (int c = tid >> 6; c < a.chunks; c += kRowWaves) {
        uint64_t m = 0;
        for (int b = lane; b < kBins; b += 64)
            if (b > bin || (all_of_bin && b == bin)) m += bins[c * kBins + b] & (kOneToken - 1);
        m = wave_sum(m);
        if (lane == 0) sh.chunk_mass[c] = m;
    }
    __syncthreads();
    if (!all_of_bin)
        tokens.each(sh, [&](uint32_t t, uint32_t i) {
            if (key_bin(t) == bin && (t > key || (t == key && i < index)))
                atomicAdd(reinterpret_cast<unsigned long long*>(&sh.chunk_mass[i / kChunk]), (unsigned long long)key_weight(t));
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
    float w[kPer];
    uint64_t sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int i = begin + j;
        w[j] = i < a.vocab ? weight(logit<F32>(row, i), top, inverse) : 0.0f;
        const uint32_t t = w[j] >= 1.0f ? weight_key(w[j]) : 0;
        if (w[j] < 1.0f || t < key || (t == key && uint32_t(i) >= index)) w[j] = 0.0f;
        sum += uint64_t(w[j]);
    }
    uint64_t all;
    uint64_t run = base + block_scan(sum, sh.tmp, &all);
    if (target < run || target >= run + sum) return;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        if (target >= run && target < run + uint64_t(w[j])) {
            a.token[r] = begin + j;
            if (a.logprob) a.logprob[r] = logf(float(double(w[j]) / double(total)));
        }
        run += uint64_t(w[j]);
    }
}

bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

int check_sample_shape(int64_t rows, int64_t vocab) {
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= (int64_t(1) << 22) ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

// The bins of every row's chunks, then their maxima.
int64_t bins_bytes(int64_t rows, int64_t chunks) { return (rows * chunks * kBins * 8 + 15) / 16 * 16; }

template <bool F32>
int launch_sample(const SampleArgs& a, int64_t rows, hipStream_t s) {
    const dim3 grid(a.chunks, static_cast<unsigned>(rows));
    hipLaunchKernelGGL(sample_max_kernel<F32>, grid, dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    hipLaunchKernelGGL(sample_bins_kernel<F32>, grid, dim3(kThreads), 0, s, a);
    if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    hipLaunchKernelGGL(sample_draw_kernel<F32>, dim3(grid.y), dim3(kThreads), sizeof(RowShared), s, a);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}

}  // namespace

namespace nvfp4 {

int sample_setup() {
    for (const void* fn : {reinterpret_cast<const void*>(sample_draw_kernel<true>), reinterpret_cast<const void*>(sample_draw_kernel<false>)})
        if (hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, kMaxLdsBytes) != hipSuccess) return NVFP4_ERR_HIP;
    return NVFP4_OK;
}

}  // namespace nvfp4

extern "C" int nvfp4_sample_workspace(int64_t rows, int64_t vocab, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    const int st = check_sample_shape(rows, vocab);
    const int64_t chunks = (vocab + kChunk - 1) / kChunk;
    if (st == NVFP4_OK) *bytes = bins_bytes(rows, chunks) + rows * chunks * int64_t(sizeof(float));
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
                       static_cast<int>(chunks), reinterpret_cast<float*>(ws + bins_bytes(rows, chunks)),
                       reinterpret_cast<unsigned long long*>(ws)};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return logits_type == NVFP4_LOGITS_F32 ? launch_sample<true>(a, rows, s) : launch_sample<false>(a, rows, s);
}
