// The accepted branch's move in the paged NVFP4 cache (include/nvfp4_draft.h).
//
// A slot's K row is bytes of its own, but V's codes of 8 slots share a dword at
// each dim, so a workgroup (one sequence, head and layer) makes whole dwords:
// 32 slots at a time, blocks of 8 aligned as they lie, it reads every source,
// waits, and merges them into place.  A path ascends, so a source never lies
// before the place it goes to: what one turn writes, no later one reads.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../host/draft_shapes.h"
#include "../host/kv_shapes.h"
#include "kv_common.h"
#include "setup.h"

namespace {

constexpr int kTurn = 32;           // slots of a turn
constexpr int kTreeMax = NVFP4_TREE_MAX;
constexpr int kLayers = 64;         // caches of a launch

struct Layers {
    uint8_t* data[kLayers];
};

// Bound by latency: the path, the pages' numbers, then one read and one write.
template <int D>
__global__ void __launch_bounds__(256)
kv_shift_kernel(KvView v, Layers layers, const int32_t* path, int max_q) {
    constexpr int kGroups = D / 16;
    constexpr int kItems = kTurn * kGroups / 256 < 1 ? 1 : kTurn * kGroups / 256;   // K rows' pieces of 16 dims, of a thread
    constexpr int kWords = kTurn / 8 * D / 256;                                     // V's dwords of a thread
    __shared__ int from[kTreeMax + 8];      // the node that comes to each place
    __shared__ int ids[kTreeMax / kPage + 2];
    __shared__ int bad[2];                  // the first entry that ends the path, and the first that moves
    const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
    const int row0 = v.start(s), nq = min(max(v.start(s + 1) - row0, 0), max_q);
    const int n = v.len(s), before = n - nq;                       // before may be negative
    const int page0 = max(before, 0) / kPage;
    if (tid < 2) bad[tid] = nq;
    if (tid < kTreeMax / kPage + 2) ids[tid] = (page0 + tid) * kPage < n ? v.page_id(s, page0 + tid) : -1;
    int mine = -1;
    if (tid < nq) {
        mine = path[int64_t(s) * max_q + tid];
        from[tid] = mine;
    }
    __syncthreads();
    if (tid < nq) {
        if (mine < 0 || mine >= nq) atomicMin(&bad[0], tid);
        if (mine != tid) atomicMin(&bad[1], tid);
    }
    __syncthreads();
    const int count = bad[0];
    if (bad[1] >= count) return;            // all where they are
    uint8_t* data = layers.data[blockIdx.z];
    // the record that holds a slot; nullptr for one that is not there
    auto record = [&](int slot) -> uint8_t* {
        if (slot < 0) return nullptr;
        const int id = ids[slot / kPage - page0];
        return v.has(id) ? data + (int64_t(id) * v.kv_heads + h) * KvRecord<D>::kBytes : nullptr;
    };
    // places of the tree's slots, by turns that begin at a block of 8 slots
    const int lo = before + bad[1], hi = before + count;
    for (int at = max(lo, 0) & ~7; at < hi; at += kTurn) {
        u32x2 k[kItems];
        uint8_t ks[kItems], vs[kItems];
        bool moves[kItems];
#pragma unroll
        for (int x = 0; x < kItems; ++x) {
            const int item = x * 256 + tid, slot = at + item / kGroups, g = item % kGroups;
            moves[x] = item < kTurn * kGroups && slot >= lo && slot < hi;
            if (!moves[x]) continue;
            const int src = before + from[slot - before];
            const uint8_t* rec = record(src);
            moves[x] = rec && src != slot;
            if (!moves[x]) continue;
            const int p = src % kPage;
            k[x] = *reinterpret_cast<const u32x2*>(rec + KvRecord<D>::k_code(p) + 8 * g);
            ks[x] = rec[KvRecord<D>::k_scale(p, g)];
            vs[x] = rec[KvRecord<D>::v_scale(p / 8, g) + p % 8];
        }
        uint32_t w[kWords], mask[kWords];
#pragma unroll
        for (int x = 0; x < kWords; ++x) {
            const int item = x * 256 + tid, slot0 = at + item / D * 8, dim = item % D;
            w[x] = mask[x] = 0;
            uint32_t word[8];
            int shift[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int slot = slot0 + j;
                shift[j] = -1;
                if (slot < lo || slot >= hi) continue;
                const int src = before + from[slot - before];
                const uint8_t* rec = record(src);
                if (!rec || src == slot) continue;
                word[j] = *reinterpret_cast<const uint32_t*>(rec + KvRecord<D>::v_code(src % kPage / 8, dim));
                shift[j] = 4 * (src % 8);
            }
            uint8_t* rec = slot0 < hi ? record(slot0) : nullptr;
            const uint32_t old = rec ? *reinterpret_cast<const uint32_t*>(rec + KvRecord<D>::v_code(slot0 % kPage / 8, dim)) : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (shift[j] < 0) continue;
                w[x] |= (word[j] >> shift[j] & 15u) << (4 * j);
                mask[x] |= 15u << (4 * j);
            }
            w[x] |= old & ~mask[x];
        }
        __syncthreads();   // every source of the turn has been read
#pragma unroll
        for (int x = 0; x < kItems; ++x) {
            if (!moves[x]) continue;
            const int item = x * 256 + tid, slot = at + item / kGroups, g = item % kGroups, p = slot % kPage;
            uint8_t* rec = record(slot);
            if (!rec) continue;
            *reinterpret_cast<u32x2*>(rec + KvRecord<D>::k_code(p) + 8 * g) = k[x];
            rec[KvRecord<D>::k_scale(p, g)] = ks[x];
            rec[KvRecord<D>::v_scale(p / 8, g) + p % 8] = vs[x];
        }
#pragma unroll
        for (int x = 0; x < kWords; ++x) {
            const int item = x * 256 + tid, slot0 = at + item / D * 8, dim = item % D;
            uint8_t* rec = mask[x] ? record(slot0) : nullptr;
            if (rec) *reinterpret_cast<uint32_t*>(rec + KvRecord<D>::v_code(slot0 % kPage / 8, dim)) = w[x];
        }
        __syncthreads();   // a turn's writes before the next one's reads of the dwords beside them
    }
}

template <int D>
void launch(const KvView& v, const Layers& layers, int count, const int32_t* path, int max_q, hipStream_t st) {
    hipLaunchKernelGGL(kv_shift_kernel<D>, dim3(v.kv_heads, v.seqs, count), dim3(256), 0, st, v, layers, path, max_q);
}

}  // namespace

extern "C" int nvfp4_kv_move(const nvfp4_kv_cache_t* caches, int64_t count, const nvfp4_kv_seqs_t* seqs,
                             const int32_t* path, int64_t max_q, void* stream) {
    int st;
    if ((st = nvfp4::check_kv_move(caches, count, seqs, path, max_q)) != NVFP4_OK) return st;
    if (seqs->seqs == 0 || seqs->total == 0 || caches[0].pages == 0) return NVFP4_OK;
    if ((st = nvfp4::device_setup()) != NVFP4_OK) return st;
    const KvView v = kv_view(caches, seqs);
    for (int64_t at = 0; at < count; at += kLayers) {
        Layers layers{};
        const int n = static_cast<int>(count - at < kLayers ? count - at : kLayers);
        for (int i = 0; i < n; ++i) layers.data[i] = caches[at + i].data;
        switch (caches[0].head_dim) {
            case 64: launch<64>(v, layers, n, path, static_cast<int>(max_q), static_cast<hipStream_t>(stream)); break;
            case 128: launch<128>(v, layers, n, path, static_cast<int>(max_q), static_cast<hipStream_t>(stream)); break;
            default: launch<256>(v, layers, n, path, static_cast<int>(max_q), static_cast<hipStream_t>(stream));
        }
        if (hipGetLastError() != hipSuccess) return NVFP4_ERR_HIP;
    }
    return NVFP4_OK;
}
