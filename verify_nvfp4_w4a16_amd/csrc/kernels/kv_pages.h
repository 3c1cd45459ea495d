// Pages of the NVFP4 cache as the attention kernels' lanes take them: decoded
// from registers by one wavefront, or once for a workgroup into LDS.
#pragma once

#include "kv_common.h"

namespace {

// Scores may outgrow the running maximum by this much (in powers of two)
// before the sums are rescaled.
constexpr float kSlack = 8.0f;
// Weights are held times this power of two, in f16 and in the sums: they reach
// 2^15, and those below 2^-32 of the largest are lost in f16, not below 2^-25.
constexpr float kLift = 7.0f;

// What one wavefront holds of a page: codes and scales as the operands need them.
// STREAM: read once, and kept out of the way of what is read again.
template <int D, bool STREAM = true>
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
                const u32x4 x = STREAM ? load16_stream(p + 16 * i) : load16(p + 16 * i);
                to[4 * i] = x[0], to[4 * i + 1] = x[1], to[4 * i + 2] = x[2], to[4 * i + 3] = x[3];
            }
        } else if constexpr (N == 2) {
            const u32x2* at = reinterpret_cast<const u32x2*>(p);
            const u32x2 x = STREAM ? __builtin_nontemporal_load(at) : *at;
            to[0] = x[0], to[1] = x[1];
        } else {
            const uint32_t* at = reinterpret_cast<const uint32_t*>(p);
            to[0] = STREAM ? __builtin_nontemporal_load(at) : *at;
        }
    }

    // An offset that the compiler sees anew at every use: a load then takes it beside a scalar address, where one kept
    // from before a loop would be widened to 64 bits and added up for each load.
    static __device__ __forceinline__ uint32_t here(int off) {
        uint32_t o = uint32_t(off);
        asm volatile("" : "+v"(o));
        return o;
    }
    __device__ __forceinline__ void load_k_codes(const uint8_t* rec, int n, int b, int ht) {
        const int slot = 32 * (ht >> 1) + (n >> 2) * 8 + (ht & 1) * 4 + (n & 3);
        load<D / 32>(k[ht], rec + here(KvRecord<D>::k_code(slot) + b * (D / 8)));
    }
    __device__ __forceinline__ void load_k_scales(const uint8_t* rec, int n, int b) {
        load<D / 64>(ks, rec + here(KvRecord<D>::kKScales + (n * 4 + b) * (D / 16)));
    }
    __device__ __forceinline__ void load_k(const uint8_t* rec, int n, int b) {
#pragma unroll
        for (int ht = 0; ht < 4; ++ht) load_k_codes(rec, n, b, ht);
        load_k_scales(rec, n, b);
    }
    __device__ __forceinline__ void load_v_half(const uint8_t* rec, int n, int b, int h) {
        using R = KvRecord<D>;
        load<D / 16>(v[h], rec + here(R::v_code(4 * h + b, n * (D / 16))));
        load<2>(vs[h], rec + here(R::v_scale(4 * h + b, n * (D / 16) / 16)));
    }
    __device__ __forceinline__ void load_v(const uint8_t* rec, int n, int b) {
        load_v_half(rec, n, b, 0);
        load_v_half(rec, n, b, 1);
    }

    // The scale pair of slot tile ht and the lane's 16-dim group j.
    template <int I>
    __device__ __forceinline__ f16x2 k_scale() const {
        return scale_both<I % 4>(ks[I / 4]);
    }
};

template <int D, bool STREAM, int HT, int J>
__device__ __forceinline__ f32x4 score_groups(const PageRegs<D, STREAM>& p, const f16x8 (&q)[D / 32], f32x4 acc) {
    if constexpr (J < D / 64) {
        const f16x2 s = p.template k_scale<HT * (D / 64) + J>();
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_row(p.k[HT][2 * J], s), q[2 * J], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(decode_row(p.k[HT][2 * J + 1], s), q[2 * J + 1], acc, 0, 0, 0);
        return score_groups<D, STREAM, HT, J + 1>(p, q, acc);
    }
    return acc;
}

__device__ __forceinline__ f16x8 to_f16x8(const float* p) {
    f16x8 r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = static_cast<_Float16>(p[i]);
    return r;
}

// A page decoded into LDS as f16: K [64 slots][D], V [D][64 slots], in 16-byte
// chunks whose place within a row is permuted so that the lanes of a matrix
// operand's read fall on different banks.
template <int D>
struct PageTiles {
    static constexpr int kBytes = 2 * kPage * D * 2;

    static __device__ __forceinline__ int k_at(int slot, int chunk) {
        return (slot * (D / 8) + (chunk ^ (D == 64 ? (slot >> 1) & 7 : slot & 15))) * 16;
    }
    static __device__ __forceinline__ int v_at(int dim, int block) {
        // rows of 8 chunks: reads run along the dims, writes along every fourth (D = 128)
        return kPage * D * 2 + (dim * 8 + (block ^ ((dim >> 1) & 7) ^ ((dim >> 4) & 1))) * 16;
    }
};

// A thread's share of a page: D / 4 dims of one slot's K, D / 32 dims of one
// 8-slot block's V.
template <int D>
struct PageShare {
    uint32_t k[D / 32], v[D / 32];
    uint32_t ks, vs[2];

    __device__ __forceinline__ void load(const uint8_t* rec, int tid) {
        using R = KvRecord<D>;
        const int slot = tid >> 2, part = tid & 3;
        PageRegs<D>::template load<D / 32>(k, rec + R::k_code(slot) + part * (D / 8));
        const uint8_t* p = rec + R::k_scale(slot, part * (D / 64));
        if constexpr (D == 64)
            ks = *p;
        else if constexpr (D == 128)
            ks = *reinterpret_cast<const uint16_t*>(p);
        else
            ks = *reinterpret_cast<const uint32_t*>(p);
        const int block = tid >> 5, dim = (tid & 31) * (D / 32);
        PageRegs<D>::template load<D / 32>(v, rec + R::v_code(block, dim));
        PageRegs<D>::template load<2>(vs, rec + R::v_scale(block, dim / 16));
    }

    template <int J>
    __device__ __forceinline__ void put_k(char* lds, int slot, int part) const {
        if constexpr (J < D / 64) {
            const f16x2 s = scale_both<J>(ks);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                *reinterpret_cast<f16x8*>(lds + PageTiles<D>::k_at(slot, part * (D / 32) + 2 * J + e)) =
                    decode_row(k[2 * J + e], s);
            put_k<J + 1>(lds, slot, part);
        }
    }

    // left: slots of the page before the sequence's end; what lies after may
    // hold anything, and becomes 0 in V (scores of such slots are masked).
    __device__ __forceinline__ void put(char* lds, int tid, int left) {
        put_k<0>(lds, tid >> 2, tid & 3);
        const int block = tid >> 5, dim = (tid & 31) * (D / 32);
        if (left < kPage) {
            const int live = left - 8 * block;
            const uint64_t mask = live <= 0 ? 0 : live >= 8 ? ~0ull : (1ull << (8 * live)) - 1;
            vs[0] &= uint32_t(mask);
            vs[1] &= uint32_t(mask >> 32);
        }
        const f16x2 sc[4] = {scale_pair<0>(vs[0]), scale_pair<1>(vs[0]), scale_pair<0>(vs[1]), scale_pair<1>(vs[1])};
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            *reinterpret_cast<f16x8*>(lds + PageTiles<D>::v_at(dim + i, block)) = decode_slots(v[i], sc);
    }
};

// The same two tiles apart and with 16 bytes between rows instead, so that a
// lane's reads differ by constants alone and their addresses take one register,
// not thirty.  K's rows are slots in the order that makes a lane's scores those
// of 8 consecutive ones (bits 2 and 3 of their numbers exchanged); V's are every
// D / 32nd dim, then the ones after those, so that a thread's dims go to rows 32
// apart.  The sixteen lanes of a read or write then fall on different banks (D = 128).
template <int D>
struct KTile {
    static constexpr int kRow = 2 * D + 16, kBytes = kPage * kRow;
    static __device__ __forceinline__ int at(int row, int chunk) { return row * kRow + chunk * 16; }
};

template <int D>
struct VTile {
    static constexpr int kRow = 2 * kPage + 16, kBytes = D * kRow;
    static __device__ __forceinline__ int at(int row, int block) { return row * kRow + block * 16; }
};

// A thread's share of them: D / 4 dims of one slot's K ...
template <int D>
struct KShare {
    uint32_t codes[D / 32], scales;

    __device__ __forceinline__ void load(const uint8_t* rec, int tid) {
        using R = KvRecord<D>;
        const int slot = tid >> 2, part = tid & 3;
        PageRegs<D, false>::template load<D / 32>(codes, rec + R::k_code(slot) + part * (D / 8));
        const uint8_t* p = rec + R::k_scale(slot, part * (D / 64));
        if constexpr (D == 64)
            scales = *p;
        else if constexpr (D == 128)
            scales = *reinterpret_cast<const uint16_t*>(p);
        else
            scales = *reinterpret_cast<const uint32_t*>(p);
    }
    __device__ __forceinline__ void put(char* tile, int tid) const {
        const int slot = tid >> 2, row = (slot & ~12) | ((slot & 4) << 1) | ((slot & 8) >> 1);
        put_groups<0>(tile + KTile<D>::at(row, (tid & 3) * (D / 32)));
    }
    template <int J>
    __device__ __forceinline__ void put_groups(char* to) const {
        if constexpr (J < D / 64) {
            const f16x2 s = scale_both<J>(scales);
            *reinterpret_cast<f16x8*>(to + 32 * J) = decode_row(codes[2 * J], s);
            *reinterpret_cast<f16x8*>(to + 32 * J + 16) = decode_row(codes[2 * J + 1], s);
            put_groups<J + 1>(to);
        }
    }
};

// ... and D / 32 dims of one 8-slot block's V.
template <int D>
struct VShare {
    uint32_t codes[D / 32], scales[2];

    __device__ __forceinline__ void load(const uint8_t* rec, int tid) {
        using R = KvRecord<D>;
        const int block = tid >> 5, dim = (tid & 31) * (D / 32);
        PageRegs<D, false>::template load<D / 32>(codes, rec + R::v_code(block, dim));
        PageRegs<D, false>::template load<2>(scales, rec + R::v_scale(block, dim / 16));
    }
    // Slots from the `left`th on may hold anything and become 0.
    __device__ __forceinline__ void cut(int tid, int left) {
        const int live = left - 8 * (tid >> 5);
        const uint64_t mask = live <= 0 ? 0 : live >= 8 ? ~0ull : (1ull << (8 * live)) - 1;
        scales[0] &= uint32_t(mask);
        scales[1] &= uint32_t(mask >> 32);
    }
    __device__ __forceinline__ void put(char* tile, int tid) const {
        const f16x2 s[4] = {scale_pair<0>(scales[0]), scale_pair<1>(scales[0]), scale_pair<0>(scales[1]), scale_pair<1>(scales[1])};
        char* to = tile + VTile<D>::at(tid & 31, tid >> 5);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) *reinterpret_cast<f16x8*>(to + VTile<D>::at(32 * i, 0)) = decode_slots(codes[i], s);
    }
};

// Order of N matrix instructions and the LDS reads of their operands: kAhead
// reads ahead of the instruction that takes them.  Left alone the compiler reads
// one ahead, and each instruction (32 cycles) waits most of a read's latency.
constexpr int kAhead = 3;

template <int N>
__device__ __forceinline__ void reads_ahead() {
    __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
    for (int i = 0; i < N - kAhead; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kAhead, 0);
}

}  // namespace
