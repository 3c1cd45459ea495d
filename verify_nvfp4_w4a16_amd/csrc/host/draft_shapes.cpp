// Host checks of the verify round's C ABI (include/nvfp4_draft.h), free of HIP.
#include "draft_shapes.h"

#include <cstdint>
#include <initializer_list>

#include "kv_shapes.h"

namespace nvfp4 {

namespace {

bool misaligned(const void* p, uintptr_t al) { return (reinterpret_cast<uintptr_t>(p) & (al - 1)) != 0; }

bool no_logits(int32_t type) { return type != NVFP4_LOGITS_BF16 && type != NVFP4_LOGITS_F32; }

}  // namespace

int check_words(const void* p) { return !p ? NVFP4_ERR_NULL : misaligned(p, 4) ? NVFP4_ERR_ALIGN : NVFP4_OK; }

int check_kv_pages(const nvfp4_kv_pages_t* p, const int32_t* state_out, const int32_t* held_out, const int32_t* kv_lens,
                   const int32_t* q_starts, const int32_t* slots, const int32_t* positions) {
    int st;
    if (!p) return NVFP4_ERR_NULL;
    if (p->seqs < 0 || p->seqs > 65535 || p->total < 0 || p->total > kKvMaxTotal) return NVFP4_ERR_SHAPE;
    if (p->capacity < 1 || p->capacity > kPoolMax) return NVFP4_ERR_SHAPE;
    if (p->table_pitch < 1 || p->table_pitch > kKvMaxTablePitch) return NVFP4_ERR_SHAPE;
    // what a block of sequences may hold, whatever `held` says, is added up in 32 bits
    if ((p->seqs < kPagesBlock ? p->seqs : int64_t(kPagesBlock)) * p->table_pitch > kPoolMax) return NVFP4_ERR_SHAPE;
    for (const void* a : {static_cast<const void*>(p->pool), static_cast<const void*>(p->state),
                          static_cast<const void*>(state_out), static_cast<const void*>(q_starts)})
        if ((st = check_words(a)) != NVFP4_OK) return st;
    if (p->seqs > 0)
        for (const void* a : {static_cast<const void*>(p->table), static_cast<const void*>(p->held),
                              static_cast<const void*>(p->keep), static_cast<const void*>(p->fresh),
                              static_cast<const void*>(held_out), static_cast<const void*>(kv_lens)})
            if ((st = check_words(a)) != NVFP4_OK) return st;
    return misaligned(slots, 4) || misaligned(positions, 4) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

int check_trees(const int32_t* kv_lens, const int32_t* q_starts, int64_t seqs, int64_t total, int64_t max_q) {
    if (seqs < 0 || seqs > 65535 || total < 0 || total > kKvMaxTotal) return NVFP4_ERR_SHAPE;
    if (max_q < 1 || max_q > NVFP4_TREE_MAX) return NVFP4_ERR_SHAPE;
    if (seqs == 0) return NVFP4_OK;
    const int st = check_words(kv_lens);
    return st != NVFP4_OK ? st : check_words(q_starts);
}

int check_kv_tree(const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q, const nvfp4_kv_tree_t* t) {
    if (!t) return NVFP4_ERR_NULL;
    if (t->words < 1 || t->words > NVFP4_TREE_WORDS || q->max_q > 64 * t->words) return NVFP4_ERR_SHAPE;
    if (t->whole_tree != 0 && t->whole_tree != 1) return NVFP4_ERR_SHAPE;
    if (s->seqs > 0 && s->total > 0 && (!t->masks || (q->window > 0 && !t->positions))) return NVFP4_ERR_NULL;
    return misaligned(t->masks, 8) || misaligned(t->positions, 4) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

int check_adjust(const nvfp4_adjust_t* a, const void* out) {
    int st;
    if (!a) return NVFP4_ERR_NULL;
    if (no_logits(a->logits_type) || no_logits(a->out_type)) return NVFP4_ERR_DTYPE;
    if (a->rows < 0 || a->rows > 65535 || a->seqs < 0 || a->seqs > 65535) return NVFP4_ERR_SHAPE;
    if (a->vocab < 1 || a->vocab > (int64_t(1) << 22)) return NVFP4_ERR_SHAPE;
    if (a->pitch < a->vocab || a->out_pitch < a->vocab || a->pitch > kKvMaxPitch || a->out_pitch > kKvMaxPitch) return NVFP4_ERR_SHAPE;
    if (!a->q_starts && a->seqs != a->rows) return NVFP4_ERR_SHAPE;
    if (a->history && (a->history_pitch < 0 || a->history_pitch > kHistoryMax)) return NVFP4_ERR_SHAPE;
    if (a->bias_tokens && (a->bias_width < 0 || a->bias_width > NVFP4_BIAS_MAX)) return NVFP4_ERR_SHAPE;
    if (a->allowed && (a->allowed_pitch < (a->vocab + 31) / 32 || a->allowed_pitch > kKvMaxPitch || a->states < 0 || a->states > 0x7fffffff))
        return NVFP4_ERR_SHAPE;
    if (a->drafted && (a->mask_words < 1 || a->mask_words > NVFP4_TREE_WORDS)) return NVFP4_ERR_SHAPE;
    if (a->rows == 0 || a->seqs == 0) return NVFP4_OK;
    if (!a->logits || !out) return NVFP4_ERR_NULL;
    if (misaligned(a->logits, a->logits_type == NVFP4_LOGITS_F32 ? 4 : 2) || misaligned(out, a->out_type == NVFP4_LOGITS_F32 ? 4 : 2))
        return NVFP4_ERR_ALIGN;
    // in place each element is read by the thread that writes it; shifted it would not be
    if (a->logits == out && (a->logits_type != a->out_type || a->pitch != a->out_pitch)) return NVFP4_ERR_SHAPE;
    if (a->history && (st = check_words(a->history_lens)) != NVFP4_OK) return st;
    if (a->bias_tokens && (st = check_words(a->bias_values)) != NVFP4_OK) return st;
    if (a->drafted && !a->masks) return NVFP4_ERR_NULL;
    for (const void* p : {static_cast<const void*>(a->q_starts), static_cast<const void*>(a->history),
                          static_cast<const void*>(a->prompt_lens), static_cast<const void*>(a->repetition),
                          static_cast<const void*>(a->presence), static_cast<const void*>(a->frequency),
                          static_cast<const void*>(a->bias_tokens), static_cast<const void*>(a->allowed),
                          static_cast<const void*>(a->allowed_rows), static_cast<const void*>(a->drafted)})
        if (misaligned(p, 4)) return NVFP4_ERR_ALIGN;
    return a->drafted && misaligned(a->masks, 8) ? NVFP4_ERR_ALIGN : NVFP4_OK;
}

int check_kv_move(const nvfp4_kv_cache_t* caches, int64_t count, const nvfp4_kv_seqs_t* s, const int32_t* path, int64_t max_q) {
    int st;
    if (!caches) return NVFP4_ERR_NULL;
    if (count < 1 || count > kMoveCaches || max_q < 1 || max_q > NVFP4_TREE_MAX) return NVFP4_ERR_SHAPE;
    for (int64_t i = 0; i < count; ++i) {
        if ((st = check_kv_cache(caches + i)) != NVFP4_OK) return st;
        if (caches[i].pages != caches[0].pages || caches[i].kv_heads != caches[0].kv_heads || caches[i].head_dim != caches[0].head_dim)
            return NVFP4_ERR_SHAPE;
    }
    // a cache that came twice would be moved twice, by workgroups that do not wait for each other
    const uintptr_t bytes = uintptr_t(caches[0].pages) * caches[0].kv_heads * 72 * caches[0].head_dim;
    for (int64_t i = 1; i < count; ++i)
        for (int64_t j = 0; j < i; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(caches[i].data), b = reinterpret_cast<uintptr_t>(caches[j].data);
            if ((a > b ? a - b : b - a) < bytes) return NVFP4_ERR_SHAPE;
        }
    if ((st = check_kv_seqs(s, true)) != NVFP4_OK) return st;
    return s->seqs > 0 ? check_words(path) : NVFP4_OK;
}

}  // namespace nvfp4
