// The next token from a row of logits (include/nvfp4_kv.h, nvfp4_sample).
//
// A token's weight w = floor(2^30 exp((l - max l) / T)) is an integer that
// fp32 holds exactly (the exponential has 24 bits), so its bits order as the
// weights do, and sums of weights are exact in 64 bits: thresholds and the
// running mass come out the same in whatever order threads add.  Nothing is
// sorted: the weight of the last token that stays is found by a radix
// selection on those bits (5 of the exponent and 6 of the fraction first, so
// that a bin is 1.6 % wide wherever the threshold lies), by count for top-k
// and by mass for top-p, and the draw is a search in the running mass by index.
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

// Tokens stay whose key is above `key`, or equal to it for the first `ties`
// by index; and whose weight is at least `low`.
struct Threshold {
    uint32_t key;
    int ties;
    double low;
};

__device__ __forceinline__ uint64_t wave_sum(uint64_t x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ uint64_t block_sum(uint64_t x, uint64_t* tmp) {
    x = wave_sum(x);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = x;
    __syncthreads();
    uint64_t all = 0;
    for (int w = 0; w < kRowWaves; ++w) all += tmp[w];
    return all;
}

struct Bins {
    uint32_t count[2048];
    uint64_t mass[2048];
};

// The lowest key at which the tokens above it are fewer than `most` (by count)
// or weigh less than `limit` (by mass), the count or mass above it, and how
// many tokens have it.  The caller knows that one exists.
template <bool F32, bool BY_MASS>
__device__ void descend(const void* row, int vocab, float top, float inverse, uint64_t most, double limit, Bins& bins,
                        uint64_t* tmp, uint32_t* key_out, uint64_t* above_out, uint32_t* same_out) {
    const int tid = threadIdx.x;
    uint32_t key = 0, mask = 0;
    uint64_t above = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 17 : level == 1 ? 8 : 0;
        const int size = level == 0 ? 2048 : level == 1 ? 512 : 256;
        for (int i = tid; i < size; i += kThreads) bins.count[i] = 0, bins.mass[i] = 0;
        __syncthreads();
        for (int i = tid; i < vocab; i += kThreads) {
            const float w = weight(logit<F32>(row, i), top, inverse);
            if (w < 1.0f) continue;
            const uint32_t k = weight_key(w);
            if ((k & mask) != key) continue;
            const int d = (k >> shift) & (size - 1);
            atomicAdd(&bins.count[d], 1u);
            if constexpr (BY_MASS) atomicAdd(reinterpret_cast<unsigned long long*>(&bins.mass[d]), (unsigned long long)w);
        }
        __syncthreads();
        if (tid == 0) {
            int best = -1;
            uint64_t sum = above, best_above = above;
            for (int d = size - 1; d >= 0; --d) {
                if (!bins.count[d]) continue;
                if (BY_MASS ? !(double(sum) < limit) : sum >= most) break;
                best = d, best_above = sum;
                sum += BY_MASS ? bins.mass[d] : bins.count[d];
            }
            tmp[0] = uint64_t(best < 0 ? 0 : best);
            tmp[1] = best_above;
            tmp[2] = best < 0 ? 0 : bins.count[best];
        }
        __syncthreads();
        key |= uint32_t(tmp[0]) << shift;
        mask |= uint32_t(size - 1) << shift;
        above = tmp[1];
        *same_out = uint32_t(tmp[2]);
        __syncthreads();
    }
    *key_out = key;
    *above_out = above;
}

// One workgroup a row.
template <bool F32>
__global__ void __launch_bounds__(kThreads)
sample_row_kernel(SampleArgs a) {
    __shared__ Bins bins;
    __shared__ uint64_t tmp[kRowWaves];
    __shared__ uint64_t wave_mass[kRowWaves];
    __shared__ uint32_t wave_ties[kRowWaves];
    const int r = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const void* row = static_cast<const char*>(a.logits) + int64_t(r) * a.pitch * (F32 ? 4 : 2);

    float top = -INFINITY;
    for (int i = tid; i < a.vocab; i += kThreads) top = fmaxf(top, logit<F32>(row, i));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) tmp[wave] = f32_bits(top);
    __syncthreads();
    for (int w = 0; w < kRowWaves; ++w) top = fmaxf(top, bits_f32(uint32_t(tmp[w])));
    __syncthreads();
    if (top == -INFINITY) {
        if (tid == 0) {
            a.token[r] = -1;
            if (a.logprob) a.logprob[r] = -INFINITY;
        }
        return;
    }
    const float t = a.temperature ? a.temperature[r] : 1.0f;
    const float inverse = t > 0.0f ? 1.0f / t : 0.0f;
    const int k = t > 0.0f ? (a.top_k ? a.top_k[r] : 0) : 1;
    const float p = a.top_p ? a.top_p[r] : 1.0f;

    // mass and number of tokens with any weight
    uint64_t mass = 0, some = 0;
    for (int i = tid; i < a.vocab; i += kThreads) {
        const float w = weight(logit<F32>(row, i), top, inverse);
        mass += uint64_t(w);
        some += w >= 1.0f;
    }
    mass = block_sum(mass, tmp);
    some = block_sum(some, tmp);
    Threshold th{0, 0x7fffffff, a.min_p ? double(a.min_p[r]) * double(kSteps) : 0.0};
    uint32_t same;
    uint64_t above;
    if (k > 0 && uint64_t(k) < some) {
        descend<F32, false>(row, a.vocab, top, inverse, uint64_t(k), 0.0, bins, tmp, &th.key, &above, &same);
        th.ties = k - int(above);
        uint64_t m = 0;   // the mass of the top k
        for (int i = tid; i < a.vocab; i += kThreads) {
            const float w = weight(logit<F32>(row, i), top, inverse);
            if (w >= 1.0f && weight_key(w) > th.key) m += uint64_t(w);
        }
        mass = block_sum(m, tmp) + uint64_t(th.ties) * uint64_t(key_weight(th.key));
    }
    if (!(p >= 1.0f)) {
        const double limit = double(p) * double(mass);
        if (limit > 0.0) {
            uint32_t key;
            descend<F32, true>(row, a.vocab, top, inverse, 0, limit, bins, tmp, &key, &above, &same);
            // of the tokens with this weight the e-th stays if above + e w < limit
            const uint64_t w = uint64_t(key_weight(key));
            int ties = int(fmin((limit - double(above)) / double(w), 2147483000.0));
            while (ties > 0 && !(double(above + uint64_t(ties - 1) * w) < limit)) --ties;
            while (double(above + uint64_t(ties) * w) < limit && ties < 0x7ffffff0) ++ties;
            if (key > th.key)
                th.key = key, th.ties = ties;
            else if (key == th.key)
                th.ties = min(th.ties, ties);
        } else {
            th.key = kTopKey, th.ties = 1;
        }
    }
    if (!(th.low <= double(kSteps))) th.key = kTopKey, th.ties = 1, th.low = 0.0;

    // The mass that stays, by wavefronts of contiguous indices.
    const int per = (a.vocab + kRowWaves - 1) / kRowWaves;
    const int begin = min(wave * per, a.vocab), end = min(begin + per, a.vocab);
    uint64_t sure = 0, ties = 0;
    for (int i = begin + lane; i < end; i += 64) {
        const float w = weight(logit<F32>(row, i), top, inverse);
        if (w < 1.0f || double(w) < th.low) continue;
        const uint32_t key = weight_key(w);
        if (key > th.key) sure += uint64_t(w);
        ties += key == th.key;
    }
    sure = wave_sum(sure);
    ties = wave_sum(ties);
    if (lane == 0) wave_mass[wave] = sure, wave_ties[wave] = uint32_t(ties);
    __syncthreads();
    const uint64_t tie_w = uint64_t(key_weight(th.key));
    uint64_t before = 0, total = 0, mine = 0;
    int seen = 0, my_seen = 0;
    for (int w = 0; w < kRowWaves; ++w) {
        const int stay = min(int(wave_ties[w]), max(0, th.ties - seen));
        const uint64_t m = wave_mass[w] + uint64_t(stay) * tie_w;
        if (w == wave) before = total, mine = m, my_seen = seen;
        total += m;
        seen += int(wave_ties[w]);
    }
    const double at = double(a.u[r]) * double(total);
    uint64_t target = at >= 0.0 ? uint64_t(fmin(at, 9007199254740992.0)) : 0;
    target = min(target, total - 1);
    if (target < before || target >= before + mine) return;
    uint64_t run = before;
    for (int i0 = begin; i0 < end; i0 += 64) {
        const int i = i0 + lane;
        const float w = i < end ? weight(logit<F32>(row, i), top, inverse) : 0.0f;
        const bool some_w = w >= 1.0f && double(w) >= th.low;
        const bool tie = some_w && weight_key(w) == th.key;
        const uint64_t tie_mask = __ballot(tie);
        const int rank = my_seen + __popcll(tie_mask & ((1ull << lane) - 1));
        my_seen += __popcll(tie_mask);
        const bool stays = some_w && (weight_key(w) > th.key || (tie && rank < th.ties));
        uint64_t sum = stays ? uint64_t(w) : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint64_t x = __shfl_up(sum, d);
            if (lane >= d) sum += x;
        }
        const uint64_t past = __ballot(run + sum > target);
        if (past) {
            if (lane == __ffsll(static_cast<unsigned long long>(past)) - 1) {
                a.token[r] = i;
                if (a.logprob) a.logprob[r] = logf(float(double(w) / double(total)));
            }
            return;
        }
        run += __shfl(sum, 63);
    }
}

bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

int check_sample_shape(int64_t rows, int64_t vocab) {
    return rows >= 0 && rows <= 65535 && vocab >= 1 && vocab <= (int64_t(1) << 22) ? NVFP4_OK : NVFP4_ERR_SHAPE;
}

}  // namespace

extern "C" int nvfp4_sample_workspace(int64_t rows, int64_t vocab, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    const int st = check_sample_shape(rows, vocab);
    if (st == NVFP4_OK) *bytes = 0;
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
    const SampleArgs a{logits, pitch, static_cast<int>(vocab), u, temperature, top_k, top_p, min_p, token, logprob};
    const hipStream_t s = static_cast<hipStream_t>(stream);
    auto fn = logits_type == NVFP4_LOGITS_F32 ? sample_row_kernel<true> : sample_row_kernel<false>;
    hipLaunchKernelGGL(fn, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0, s, a);
    return hipGetLastError() == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP;
}
