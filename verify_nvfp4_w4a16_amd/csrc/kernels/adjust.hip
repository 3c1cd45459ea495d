// Penalties, biases and grammar masks on logits (include/nvfp4_draft.h).
//
// A workgroup takes a piece of the vocabulary and up to kRows rows of one
// sequence.  It counts the sequence's history into LDS, a word a token (counts
// are whole numbers, so the order of the atomic additions changes nothing),
// then streams its rows' logits once: read, adjust by the word, write.  A
// row's own drafted tokens are counted in before the row and out after it.
// A row's logits are loaded while the history is counted or the row before is
// written.
//
// Bounds: 192 rows of 151552 bf16 logits take 20 us without penalties (5.8 TB/s;
// a plain copy 17), 48 us with biases, grammars and histories of 4000 tokens
// each: in copies that leave parts out, 44 without the additions in LDS, 38
// without applying them, 33 without a history.  (A list of the touched tokens, adjusted
// after the row went by, took 62: its additions give back what was there before.)
// 8 trees of 48 rows in fp32 take 109 us (4.3 TB/s).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../host/draft_shapes.h"
#include "nvfp4_common.h"
#include "setup.h"

namespace {

// 32 KiB of words and eight wavefronts: four workgroups fill a CU.  16384 tokens (two workgroups) took 64 us
// instead of 48 for 192 rows of 151552 bf16 logits with 4000 tokens of history each, and 4096 tokens of 256
// threads 51 us, since each piece reads the whole history.
constexpr int kThreads = 512;
constexpr int kPiece = 8192;   // tokens of a workgroup
// Rows that share the counted history.  For trees of 48 rows, fp32, histories of 500..6000 tokens | of 32768:
// 2 rows 108 | 139 us, 3 rows 109 | 136, 4 rows 115 | 129, 8 rows 132 | 138: many rows leave the card idle at the end.
constexpr int kRows = 3;

// A token's word: how often it was said, its place in the bias list plus 1, and whether the prompt has it.
constexpr uint32_t kCount = (1u << 20) - 1;
constexpr int kBiasShift = 20;
constexpr uint32_t kBias = 0x7ffu << kBiasShift;
constexpr uint32_t kPrompt = 1u << 31;
static_assert(nvfp4::kHistoryMax + NVFP4_TREE_MAX < kCount && NVFP4_BIAS_MAX < 0x7ff);

struct AdjustArgs {
    nvfp4_adjust_t a;
    void* out;
    int vocab, pieces, seqs, rows, per;   // per: rows of a unit, kRows or 1
    int unit0;                            // first unit of the launch
};

// Rows may begin at any element, so whole vectors are read from wherever they begin.
template <class V>
__device__ __forceinline__ V load_any(const void* p) {
    V v;
    __builtin_memcpy(&v, p, sizeof v);
    return v;
}

// The first unit of sequence s.  Units of one row are counted as the rows are; others are kRows rows of a
// sequence, and a unit more for each sequence is enough wherever its rows begin.
__device__ __forceinline__ int first_unit(int start, int s, int per) { return per == 1 ? start : start / kRows + s; }

template <class In, class Out>
__global__ void __launch_bounds__(kThreads)
adjust_kernel(AdjustArgs args) {
    constexpr int kEach = 16 / sizeof(In);                      // logits of a load
    constexpr int kLoads = kPiece / (kThreads * kEach);         // loads of a thread for a row
    __shared__ __attribute__((aligned(16))) uint32_t words[kPiece];
    __shared__ float bias[NVFP4_BIAS_MAX];
    const nvfp4_adjust_t& a = args.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int unit = args.unit0 + blockIdx.x / args.pieces, piece = blockIdx.x % args.pieces;
    const int from = piece * kPiece, size = min(kPiece, args.vocab - from);

    // the sequence of this unit and its rows
    int s = unit, row0 = unit, row_end = unit + 1, first = unit;
    if (a.q_starts) {
        auto start = [&](int i) { return min(max(a.q_starts[min(i, args.seqs)], 0), args.rows); };
        // the last sequence whose first unit is this one or before it, 256 of them in one latency
        int end = first = 0, found = 0;
        for (int base = 0; base < args.seqs; base += 256) {
            int begins[4], ends[4], n = 0;
#pragma unroll
            for (int y = 0; y < 4; ++y) begins[y] = start(base + 64 * y + lane), ends[y] = start(base + 64 * y + lane + 1);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = base + 64 * y + lane;
                const int here = __popcll(__ballot(i < args.seqs && first_unit(begins[y], i, args.per) <= unit));
                if (n == 64 * y && here) first = __builtin_amdgcn_readlane(begins[y], here - 1), end = __builtin_amdgcn_readlane(ends[y], here - 1);
                if (n == 64 * y) n += here;
            }
            found += n;
            if (n < 256) break;
        }
        s = found - 1;
        if (s < 0) return;
        row0 = first + (unit - first_unit(first, s, args.per)) * args.per;
        if (row0 < first) return;            // as happens where starts descend
        row_end = min(row0 + args.per, end);
        if (row0 >= row_end) return;
    }

    // a row's logits are on their way while the history is counted, and the next row's while one is written
    u32x4 raw[kLoads];
    auto fetch = [&](int row) {
        const In* in = static_cast<const In*>(a.logits) + row * a.pitch + from;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
            const int i = (x * kThreads + tid) * kEach;
            if (i + kEach <= size) {
                raw[x] = load_any<u32x4>(in + i);
            } else {   // the end of the vocabulary
                In some[kEach];
#pragma unroll
                for (int j = 0; j < kEach; ++j) some[j] = i + j < size ? in[i + j] : In(0);
                __builtin_memcpy(&raw[x], some, sizeof some);
            }
        }
    };
    fetch(row0);

    const float r_in = a.repetition ? a.repetition[s] : 1.0f;
    const float r = r_in > 0.0f ? r_in : 1.0f;
    const float up = r < 0x1p-64f ? 0x1p64f : 1.0f, lifted = r * up, inverse = 1.0f / lifted;   // 1 / r itself may be no number
    const float p = a.presence ? a.presence[s] : 0.0f, f = a.frequency ? a.frequency[s] : 0.0f;
    const bool penalised = r != 1.0f || p != 0.0f || f != 0.0f;
    const bool counted = penalised && a.history, drafts = penalised && a.drafted, biased = a.bias_tokens && a.bias_width > 0;
    const bool worded = counted || drafts || biased;
    const int32_t* said = a.history + s * a.history_pitch;
    u32x4 t[4] = {};   // four loads of the history at a time; the first goes out before its length is known
    if (counted && tid * 4 + 4 <= a.history_pitch) t[0] = load_any<u32x4>(said + tid * 4);
    if (worded) {
        for (int i = tid * 4; i < kPiece; i += kThreads * 4) *reinterpret_cast<u32x4*>(words + i) = u32x4{0, 0, 0, 0};
        __syncthreads();
    }
    if (counted) {
        const int len = static_cast<int>(min(int64_t(max(a.history_lens[s], 0)), a.history_pitch));
        const int prompt = a.prompt_lens ? min(max(a.prompt_lens[s], 0), len) : 0;
        auto put = [&](int at, uint32_t token) {
            const uint32_t v = token - uint32_t(from);
            if (v >= uint32_t(size)) return;
            if (at < prompt)
                atomicOr(&words[v], kPrompt);
            else
                atomicAdd(&words[v], 1u);
        };
        constexpr int kStep = kThreads * 4;
        for (int base = 0; base < len; base += 4 * kStep) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = base + y * kStep + tid * 4;
                if (i + 4 <= len && base + y) t[y] = load_any<u32x4>(said + i);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int i = base + y * kStep + tid * 4;
                if (i + 4 <= len) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) put(i + j, t[y][j]);
                } else {
                    for (int j = i; j < len; ++j) put(j, static_cast<uint32_t>(said[j]));
                }
            }
        }
    }
    if (biased) {
        __syncthreads();
        // the last entry of a token counts: the largest place wins, above a count that both find
        for (int i = tid; i < a.bias_width; i += kThreads) {
            const uint32_t v = uint32_t(a.bias_tokens[s * a.bias_width + i]) - uint32_t(from);
            if (v >= uint32_t(size)) continue;
            bias[i] = a.bias_values[s * a.bias_width + i];
            atomicMax(&words[v], (words[v] & ~kBias) | uint32_t(i + 1) << kBiasShift);
        }
    }
    if (worded) __syncthreads();

    for (int row = row0; row < row_end; ++row) {
        // the row's drafted tokens, one a thread
        int drafted = -1;
        if (drafts) {
            const int node = tid;
            if (node < 64 * a.mask_words && first + node < args.rows && (a.masks[row * a.mask_words + node / 64] >> (node & 63) & 1)) {
                const uint32_t v = uint32_t(a.drafted[first + node]) - uint32_t(from);
                if (v < uint32_t(size)) drafted = static_cast<int>(v);
            }
            if (drafted >= 0) atomicAdd(&words[drafted], 1u);
            __syncthreads();
        }
        const uint32_t* allowed = nullptr;
        if (a.allowed) {
            const int64_t state = a.allowed_rows ? a.allowed_rows[row] : row;
            if (state >= 0 && state < a.states) allowed = a.allowed + state * a.allowed_pitch + from / 32;
        }
        Out* out = static_cast<Out*>(args.out) + row * a.out_pitch + from;
        auto one = [&](float x, int i) {
            const uint32_t w = worded ? words[i] : 0;
            if (w) {
                const uint32_t n = w & kCount;
                if (penalised && (w & (kPrompt | kCount))) {
                    // x / r, correctly rounded: the product is within two steps, corrected by its remainder within one,
                    // and from there a remainder settles it (1 / r is rounded correctly itself)
                    const float y = x * up, q = y * inverse;
                    float best = __builtin_fmaf(__builtin_fmaf(-q, lifted, y), inverse, q);
                    best = __builtin_fmaf(__builtin_fmaf(-best, lifted, y), inverse, best);
                    x = x > 0.0f ? (__builtin_isfinite(best) ? best : q) : x * r;
                    if (n) x = x - p - f * float(n);
                }
                if (w & kBias) x += bias[((w & kBias) >> kBiasShift) - 1];
            }
            return x;
        };
        float x[kLoads][kEach];
#pragma unroll
        for (int y = 0; y < kLoads; ++y)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (std::is_same_v<In, float>) {
                    x[y][j] = bits_f32(raw[y][j]);
                } else {
                    x[y][2 * j] = bits_f32(raw[y][j] << 16);
                    x[y][2 * j + 1] = bits_f32(raw[y][j] & 0xffff0000u);
                }
            }
        if (row + 1 < row_end) fetch(row + 1);
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
            const int i = (y * kThreads + tid) * kEach;
            if (i >= size) break;
            uint32_t bits = ~0u;
            if (allowed) bits = allowed[i / 32] >> (i % 32);
#pragma unroll
            for (int j = 0; j < kEach; ++j) {
                x[y][j] = one(x[y][j], i + j);
                if (!(bits >> j & 1)) x[y][j] = -INFINITY;
            }
            if (i + kEach <= size) {
                if constexpr (std::is_same_v<Out, float>) {
                    __builtin_memcpy(out + i, x[y], sizeof x[y]);
                } else {
                    uint16_t w[kEach];
#pragma unroll
                    for (int j = 0; j < kEach; ++j) w[j] = f32_to_bf16_rne(x[y][j]);
                    __builtin_memcpy(out + i, w, sizeof w);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    if (i + j >= size) continue;
                    if constexpr (std::is_same_v<Out, float>)
                        out[i + j] = x[y][j];
                    else
                        out[i + j] = f32_to_bf16_rne(x[y][j]);
                }
            }
        }
        if (drafts) {
            __syncthreads();
            if (drafted >= 0) atomicSub(&words[drafted], 1u);
        }
    }
}

}  // namespace

extern "C" int nvfp4_adjust_logits(const nvfp4_adjust_t* adjust, void* out, void* stream) {
    int st;
    if ((st = nvfp4::check_adjust(adjust, out)) != NVFP4_OK) return st;
    if (adjust->rows == 0 || adjust->seqs == 0) return NVFP4_OK;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    AdjustArgs a{*adjust, out, static_cast<int>(adjust->vocab), static_cast<int>((adjust->vocab + kPiece - 1) / kPiece),
                 static_cast<int>(adjust->seqs), static_cast<int>(adjust->rows), 1, 0};
    // units of one row where those are fewer
    const bool single = !adjust->q_starts || adjust->rows <= adjust->rows / kRows + adjust->seqs;
    a.per = single ? 1 : kRows;
    const int64_t units = single ? adjust->rows : adjust->rows / kRows + adjust->seqs;
    const dim3 block(kThreads);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const bool in32 = adjust->logits_type == NVFP4_LOGITS_F32, out32 = adjust->out_type == NVFP4_LOGITS_F32;
    const auto kernel = in32 ? (out32 ? adjust_kernel<float, float> : adjust_kernel<float, uint16_t>)
                             : (out32 ? adjust_kernel<uint16_t, float> : adjust_kernel<uint16_t, uint16_t>);
    const int64_t most = (int64_t(1) << 31) / kThreads / a.pieces;   // a launch holds fewer than 2^32 threads
    for (int64_t at = 0; at < units; at += most) {
        a.unit0 = static_cast<int>(at);
        const int64_t n = units - at < most ? units - at : most;
        hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(n * a.pieces)), block, 0, s, a);
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}
