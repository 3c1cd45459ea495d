// Drives the layout of the tree attention's launches with the ends of every field
// and with random calls (built with sanitizers by test_draft_capi_cpu.py).
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "../verify_nvfp4_w4a16_amd/csrc/host/draft_shapes.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_shapes.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/tree_plan.h"

namespace {

alignas(16) char place[64];
int64_t checks = 0;

void expect(bool ok, const char* what, const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q) {
    ++checks;
    if (ok) return;
    std::printf("failed: %s: kv heads %d seqs %lld total %lld heads %lld max_q %lld max_kv %lld window %lld\n", what, c.kv_heads,
                (long long)s.seqs, (long long)s.total, (long long)q.heads, (long long)q.max_q, (long long)q.max_kv, (long long)q.window);
    std::exit(1);
}

bool valid(const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q) {
    return nvfp4::check_kv_cache(&c) == NVFP4_OK && nvfp4::check_kv_seqs(&s, true) == NVFP4_OK &&
           nvfp4::check_kv_queries(&c, &s, &q) == NVFP4_OK && q.max_q <= NVFP4_TREE_MAX;
}

void check(const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q, std::mt19937_64& g) {
    if (!valid(c, s, q)) return;
    const nvfp4::TreePlan p = nvfp4::tree_plan(&c, &s, &q);
    const int64_t bytes = nvfp4::tree_workspace_bytes(&c, &s, &q);
    expect(bytes >= 0 && bytes < int64_t(1) << 50, "workspace", c, s, q);
    if (!p.rows) return;
    const int64_t group = q.heads / c.kv_heads, rows = q.max_q * group;
    expect(p.rows == 64 || p.rows == 128, "rows", c, s, q);
    expect(p.ranges >= 1 && p.ranges <= 512, "ranges", c, s, q);
    expect(p.workgroups >= 1, "workgroups", c, s, q);
    // what a call's memory can hold fits a launch
    if (s.total * q.heads * c.head_dim < int64_t(1) << 37) expect(p.workgroups * 256 < int64_t(1) << 32, "threads", c, s, q);
    if (!p.whole) {
        expect(bytes >= 2 * int64_t(p.ranges) * p.rows * (c.head_dim + 2) * 4 + (s.seqs + 1) * 16, "parts", c, s, q);
        return;
    }
    // workgroups enough for any sequences of these bounds
    for (int turn = 0; turn < 3; ++turn) {
        int64_t left = s.total, segments = 0;
        for (int64_t i = 0; i < std::min<int64_t>(s.seqs, 3000); ++i) {
            int64_t n = turn == 0 ? q.max_q : int64_t(g() % uint64_t(q.max_q + 1));
            if (turn == 2) n = std::min<int64_t>(n, 1);
            n = std::min(n, left);
            left -= n;
            segments += (n * group + p.rows - 1) / p.rows * c.kv_heads;
        }
        expect(segments <= p.workgroups, "segments", c, s, q);
    }
    (void)rows;
}

}  // namespace

int main() {
    std::mt19937_64 g(5);
    const std::vector<int64_t> seqs = {0, 1, 2, 63, 64, 65, 4096, 65535}, totals = {0, 1, 64, 257, 65536, int64_t(1) << 24},
                               queries = {0, 1, 9, 33, 64, 65, 255, 256}, slots = {0, 1, 64, 65, 257, 4096, 70000, (int64_t(1) << 29)},
                               windows = {0, 1, 64, 500, int64_t(1) << 40};
    for (int d : {64, 128, 256})
        for (int kv_heads : {1, 2, 8, 128})
            for (int group : {1, 3, 8, 256})
                for (int64_t n : seqs)
                    for (int64_t t : totals)
                        for (int64_t mq : queries)
                            for (int64_t mkv : slots) {
                                const nvfp4_kv_cache_t c{reinterpret_cast<uint8_t*>(place), 4, kv_heads, d, 1.0f, 1.0f};
                                const int32_t* w = reinterpret_cast<int32_t*>(place);
                                const nvfp4_kv_seqs_t s{w, w, w, int64_t(1) << 23, n, t};
                                const int64_t heads = int64_t(kv_heads) * group;
                                const nvfp4_kv_queries_t q{place, heads * d, d, heads, mq, mkv, windows[checks % windows.size()], 1.0f, 0.0f, 1};
                                check(c, s, q, g);
                            }
    std::printf("plan ok, %lld checks\n", (long long)checks);
    return 0;
}
