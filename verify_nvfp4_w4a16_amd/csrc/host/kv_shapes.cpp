// Host checks of the paged NVFP4 cache's C ABI (include/nvfp4_kv.h): what the
// calls share of their argument validation, free of HIP so that it builds
// with a plain C++ compiler.
#include "kv_shapes.h"

#include <cmath>
#include <cstdint>

namespace nvfp4 {

namespace {

bool positive_finite(float f) { return std::isfinite(f) && f > 0.0f; }
bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

}  // namespace

int check_kv_cache(const nvfp4_kv_cache_t* c) {
    if (!c) return NVFP4_ERR_NULL;
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_SHAPE;
    if (c->kv_heads < 1 || c->kv_heads > 1024) return NVFP4_ERR_SHAPE;
    if (c->pages < 0 || c->pages > 0x7fffffff) return NVFP4_ERR_SHAPE;
    if (!positive_finite(c->k_scale) || !positive_finite(c->v_scale)) return NVFP4_ERR_SHAPE;
    if (!c->data && c->pages > 0) return NVFP4_ERR_NULL;
    if (misaligned(c->data, 16)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int check_kv_seqs(const nvfp4_kv_seqs_t* s, bool starts) {
    if (!s) return NVFP4_ERR_NULL;
    if (s->seqs < 0 || s->seqs > 65535 || s->total < 0 || s->total > kKvMaxTotal) return NVFP4_ERR_SHAPE;
    if (s->table_pitch < 1 || s->table_pitch > kKvMaxTablePitch) return NVFP4_ERR_SHAPE;
    if (s->seqs == 0) return NVFP4_OK;
    if (!s->table || !s->kv_lens || (starts && !s->q_starts)) return NVFP4_ERR_NULL;
    if (misaligned(s->table, 4) || misaligned(s->kv_lens, 4) || (starts && misaligned(s->q_starts, 4)))
        return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int check_kv_rows(const void* p, int64_t pitch, int64_t head_pitch, int64_t total) {
    if (pitch < 0 || head_pitch < 0) return NVFP4_ERR_SHAPE;
    if (pitch > kKvMaxPitch || head_pitch > kKvMaxPitch) return NVFP4_ERR_SHAPE;
    if (total > 0 && !p) return NVFP4_ERR_NULL;
    if (misaligned(p, 16) || pitch % 8 || head_pitch % 8) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

int check_kv_queries(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q) {
    if (!q) return NVFP4_ERR_NULL;
    if (q->heads < 1 || q->heads % c->kv_heads || q->heads / c->kv_heads > kKvMaxGroup) return NVFP4_ERR_SHAPE;
    if (q->max_q < 0 || q->max_q > kKvMaxTotal || q->max_kv < 0 || q->max_kv > s->table_pitch * NVFP4_KV_PAGE)
        return NVFP4_ERR_SHAPE;
    // row numbers of a sequence, and of all of them, stay below 2^31
    const int64_t most = 0x7fffffff;
    if (q->max_q * (q->heads / c->kv_heads) > most || s->total * q->heads > most) return NVFP4_ERR_SHAPE;
    if (q->window < 0 || !std::isfinite(q->scale) || !(q->softcap >= 0.0f) || !std::isfinite(q->softcap))
        return NVFP4_ERR_SHAPE;
    if (!std::isfinite(q->scale * c->k_scale)) return NVFP4_ERR_SHAPE;   // every score but 0 would leave fp32
    if (q->causal != 0 && q->causal != 1) return NVFP4_ERR_SHAPE;
    return check_kv_rows(q->q, q->q_pitch, q->q_head_pitch, s->total);
}

}  // namespace nvfp4

extern "C" int nvfp4_kv_record_bytes(int64_t head_dim, int64_t* bytes) {
    if (!bytes) return NVFP4_ERR_NULL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return NVFP4_ERR_SHAPE;
    *bytes = 72 * head_dim;
    return NVFP4_OK;
}
