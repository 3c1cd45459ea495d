// The layout of nvfp4_kv_tree_attention's launches (include/nvfp4_draft.h).
#include "tree_plan.h"

#include <algorithm>
#include <cstdint>

#include "kv_plan.h"

namespace nvfp4 {

TreePlan tree_plan(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q) {
    TreePlan p{};
    const int64_t rows = q->max_q * (q->heads / c->kv_heads);
    const int window = kv_window(q);
    const int64_t slots = window > 0 ? std::min(q->max_kv, window + q->max_q) : q->max_kv;
    const int64_t pages = std::max<int64_t>((slots + NVFP4_KV_PAGE - 1) / NVFP4_KV_PAGE + (window > 0), 1);
    // 16-row workgroups decode every page for themselves, but start at once and need no second launch where
    // a sequence has few pages; 64 or 128 rows that share the decoding pay from so many (16 rows, page) on, whatever the
    // dims.  16-row workgroups | tiles, us, 8 heads: D = 64, 16 trees of 64 x 2 rows over 1000 slots (16384 such) 16 | 32, over
    // 3000 (48128) 66 | 43; D = 128, 32 of 9 x 4 over 3000 (36096) 60 | 59, 16 of 64 x 2 over 1000 24 | 44, over 3000 84 | 61;
    // D = 256, 4 of 64 x 2 over 10000 (40192) 95 | 93, 16 over 1000 45 | 65, over 3000 134 | 109.  At D = 256 a CU holds one tile, and
    // three 16-row workgroups are quicker at any length: 32 of 9 x 4 rows over 3000 101 | 115, over 10000 277 | 338.
    // The lengths are the device's, so the host's bounds decide, and one far above them gives short caches tiles.  max_kv the
    // longest cache | 32768, us, D = 128: 16 of 64 x 2 rows over 1000 slots 25 | 45, 32 of 9 x 4 over 500 14 | 29, 1 of 16 x 4 over
    // 900 10 | 12, 32 of 16 x 4 over 4000 86 | 78; a max_q of 64 instead of 9: 14 | 21.
    const int64_t groups = std::min(s->seqs * c->kv_heads, int64_t(1) << 24), work = groups * std::min((rows + 15) / 16 * pages, int64_t(1) << 24);
    if (rows <= (c->head_dim == 256 ? 48 : 32) || work < kTreeWork) return p;
    // 64 rows, a page's halves on different wavefronts, or 128: 32 trees of 16 x 4 rows over 3000 slots 63 | 79 us
    p.rows = rows <= 64 ? 64 : 128;
    const int64_t segments = std::max<int64_t>(s->seqs * c->kv_heads * ((rows + p.rows - 1) / p.rows), 1);
    p.least = 4;
    // Up to 64 sequences' pages are added up by each wavefront: 64 trees of 16 x 4 rows over 3000 slots 89 us, by a kernel before 104.
    p.added = s->seqs > kTreeLanes;
    // So short, no segment is cut, which spares the join: 600 trees of 16 x 4 rows over 200 slots 160 | 174 us, of 64 x 4 386 | 400.
    p.whole = pages <= p.least;
    // as many ranges as workgroups fit the card at once: two on a CU, one at D = 256
    const int64_t most = c->head_dim == 256 ? 256 : 512;
    const int64_t many = std::min(segments, int64_t(1) << 24);   // more give the most ranges too, and the product stays in 64 bits
    p.ranges = static_cast<int>(std::min((many * pages + p.least - 1) / p.least, most));
    // whole segments: no more than the rows that there are can fill
    const int64_t filled = (s->seqs + s->total * (q->heads / c->kv_heads) / p.rows) * c->kv_heads;
    p.workgroups = p.whole ? std::min(segments, std::max<int64_t>(filled, 1)) : p.ranges;
    return p;
}

int64_t tree_sum_bytes(const nvfp4_kv_seqs_t* s) { return (s->seqs + 1) * 16; }

int64_t tree_workspace_bytes(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q) {
    const TreePlan p = tree_plan(c, s, q);
    if (!p.rows) return kv_workspace_bytes(c, s, q, true);
    if (p.whole && !p.added) return 0;
    const int64_t parts = p.whole ? 0 : int64_t(2) * p.ranges * p.rows;
    return parts * (c->head_dim + 2) * int64_t(sizeof(float)) + tree_sum_bytes(s);
}

}  // namespace nvfp4
