// The layout of nvfp4_kv_attention's launches (include/nvfp4_kv.h).
#include "kv_plan.h"

#include <algorithm>
#include <cstdint>

namespace nvfp4 {

int kv_window(const nvfp4_kv_queries_t* q) { return q->window < q->max_kv ? static_cast<int>(q->window) : 0; }

KvPlan kv_plan(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q, bool few) {
    const int64_t rows = q->max_q * (q->heads / c->kv_heads);
    // Rows of a kv head: up to 32 in 16-row workgroups, each decoding the pages
    // for itself, up to 64 in one workgroup with a page's halves on different
    // wavefronts, else 128 to a workgroup.  32 sequences of 4096 slots, 8 heads
    // of 128: 32 rows take 73 us, decoded once for all 78; 36 rows 94 and 77; 64 rows 119 and 91
    // (and 64 rows over 8192 slots 192 us in 128-row workgroups, 144 in these).
    KvPlan p{};
    p.tile = few || rows <= 32 ? 0 : rows <= kKvTileRows / 2 ? kKvTileRows / 2 : kKvTileRows;
    const int64_t per_tile = p.tile ? p.tile : kKvRowTile;
    p.row_tiles = (rows + per_tile - 1) / per_tile;
    const int64_t base = std::max<int64_t>(s->seqs * c->kv_heads * p.row_tiles, 1);
    const int window = kv_window(q);
    const int64_t slots = window > 0 ? std::min(q->max_kv, window + q->max_q) : q->max_kv;
    const int64_t pages = std::max<int64_t>((slots + NVFP4_KV_PAGE - 1) / NVFP4_KV_PAGE + (window > 0), 1);
    // Pages of a workgroup: as many as leave 512, which fills the card twice, and
    // a page a wavefront at least.  Few rows take 32 at most, so that the last to
    // end is not late by much, and all of 16, which spares the second launch that
    // joins parts: one sequence of 777 slots takes 9.4 us either way on the card,
    // and the host one launch less.  (With 8 pages at least, one sequence of 2048
    // slots took 11.5 us instead of 10.5, at D = 256 16.9 instead of 15.1.)
    const int64_t low = !p.tile && pages <= 16 ? pages : kKvWaves, high = p.tile ? pages : std::max<int64_t>(low, 32);
    const int64_t many = std::min(base, int64_t(1) << 24);   // more give the most pages too, and the product stays in 64 bits
    const int64_t chunk = std::min(std::max((pages * many + 511) / 512, low), std::max<int64_t>(high, 1));
    p.splits = static_cast<int>((pages + chunk - 1) / chunk);
    if (p.tile) {
        p.splits = std::min(p.splits, kKvMaxSplits);
        p.chunk = static_cast<int>((pages + p.splits - 1) / p.splits);
        p.part_rows = p.splits > 1 ? p.splits * s->total * q->heads : 0;
    } else {
        p.chunk = static_cast<int>(chunk);
        p.planned = p.splits > 2 && base * p.splits > 2048;
        // planned: at most kKvItems whole chunks, and a rest a segment
        p.items = static_cast<int>(p.planned ? std::min(base * p.splits, base + kKvItems) : base * p.splits);
        p.part_rows = p.splits > 1 ? int64_t(p.items) * kKvRowTile : 0;
    }
    return p;
}

int64_t kv_row_tiles(const KvPlan& p, int64_t total, int64_t group) { return std::min(p.row_tiles, (total * group + p.tile - 1) / p.tile); }

int64_t kv_plan_bytes(const nvfp4_kv_seqs_t* s) { return (2 + 2 * s->seqs + 3) / 4 * 16; }

int64_t kv_workspace_bytes(const nvfp4_kv_cache_t* c, const nvfp4_kv_seqs_t* s, const nvfp4_kv_queries_t* q, bool few) {
    const KvPlan p = kv_plan(c, s, q, few);
    return p.part_rows * (c->head_dim + 2) * int64_t(sizeof(float)) + (p.planned ? kv_plan_bytes(s) : 0);
}

}  // namespace nvfp4
