// Drives the numbers of workgroups that the cache attention's launches take with the
// ends of every field (built with sanitizers by test_kv_launches.py): each has to fit
// the kernels' 32-bit numbers, and the rows that a call has their row tiles.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../verify_nvfp4_w4a16_amd/csrc/host/draft_shapes.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_plan.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_shapes.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/tree_plan.h"

namespace {

alignas(16) char place[64];
int64_t checks = 0;

void expect(bool ok, const char* what, const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q) {
    ++checks;
    if (ok) return;
    std::printf("failed: %s: kv heads %d dim %d seqs %lld total %lld heads %lld max_q %lld max_kv %lld\n", what, c.kv_heads, c.head_dim,
                (long long)s.seqs, (long long)s.total, (long long)q.heads, (long long)q.max_q, (long long)q.max_kv);
    std::exit(1);
}

void check(const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q) {
    if (nvfp4::check_kv_cache(&c) != NVFP4_OK || nvfp4::check_kv_seqs(&s, true) != NVFP4_OK || nvfp4::check_kv_queries(&c, &s, &q) != NVFP4_OK)
        return;
    if (s.seqs == 0 || s.total == 0 || q.max_q == 0) return;   // nothing is launched
    const int64_t most = 0x7fffffff, group = q.heads / c.kv_heads;
    expect(nvfp4::kKvLaunch * 256 < int64_t(1) << 32, "threads of a launch", c, s, q);
    expect(s.total * q.heads <= most, "rows to join", c, s, q);
    for (int tree = 0; tree <= (q.max_q <= NVFP4_TREE_MAX ? 1 : 0); ++tree) {
        if (tree && nvfp4::tree_plan(&c, &s, &q).rows) {   // tiles, whose layout tree_plan_check.cpp drives
            const nvfp4::TreePlan t = nvfp4::tree_plan(&c, &s, &q);
            expect(t.workgroups >= 1 && t.workgroups <= most && (t.whole || t.workgroups <= nvfp4::kKvLaunch), "workgroups of trees", c, s, q);
            continue;
        }
        const nvfp4::KvPlan p = nvfp4::kv_plan(&c, &s, &q, tree);
        if (!p.tile) {
            expect(p.items >= 0 && int64_t(p.items) * nvfp4::kKvRowTile < int64_t(1) << 40, "items", c, s, q);
            const int64_t all = s.seqs * c.kv_heads * p.row_tiles;
            expect(p.items >= all && (p.planned || p.items == all * p.splits), "items for all", c, s, q);
            continue;
        }
        const int64_t tiles = nvfp4::kv_row_tiles(p, s.total, group), rows = std::min(q.max_q, s.total) * group;
        expect(tiles * c.kv_heads <= most, "workgroups of tiles", c, s, q);
        expect(tiles * p.tile >= rows && (tiles == 0 || (tiles - 1) * p.tile < rows), "tiles of all rows", c, s, q);
    }
}

}  // namespace

int main() {
    const int32_t* w = reinterpret_cast<int32_t*>(place);
    for (int d : {64, 128, 256})
        for (int kv_heads : {1, 2, 8, 128, 257, 1024})
            for (int64_t group : {1, 3, 8, 256})
                for (int64_t n : {0, 1, 2, 64, 4096, 16385, 65535})
                    for (int64_t t : {int64_t(0), int64_t(1), int64_t(257), int64_t(65535), int64_t(1) << 20, int64_t(1) << 24})
                        for (int64_t mq : {int64_t(0), int64_t(1), int64_t(9), int64_t(32), int64_t(33), int64_t(256), int64_t(4099), int64_t(1) << 24})
                            for (int64_t mkv : {0, 64, 2049, 70000, 1 << 29}) {
                                const nvfp4_kv_cache_t c{reinterpret_cast<uint8_t*>(place), 4, kv_heads, d, 1.0f, 1.0f};
                                const nvfp4_kv_seqs_t s{w, w, w, int64_t(1) << 23, n, t};
                                const int64_t heads = kv_heads * group;
                                const nvfp4_kv_queries_t q{place, heads * d, d, heads, mq, mkv, 0, 1.0f, 0.0f, 1};
                                check(c, s, q);
                            }
    std::printf("launches ok, %lld checks\n", (long long)checks);
    return 0;
}
