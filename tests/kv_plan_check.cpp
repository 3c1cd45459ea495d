// Drives the layout of the cache attention's launches with the ends of every
// field and with random calls, and checks it against what the kernels make of
// it (built with sanitizers by test_kv_plan.py).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>
#include <random>

#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_plan.h"
#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_shapes.h"

namespace {

alignas(16) char place[64];
int64_t checks = 0;

void expect(bool ok, const char* what, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q) {
    ++checks;
    if (ok) return;
    std::printf("failed: %s: seqs %lld total %lld heads %lld max_q %lld max_kv %lld window %lld causal %d\n", what,
                (long long)s.seqs, (long long)s.total, (long long)q.heads, (long long)q.max_q, (long long)q.max_kv,
                (long long)q.window, q.causal);
    std::exit(1);
}

// Pages that the rows [i0, i1] of a sequence see, as the kernels count them.
int64_t pages_seen(int64_t window, bool causal, int64_t len, int64_t fresh, int64_t i0, int64_t i1) {
    const int64_t lo = window > 0 ? std::max<int64_t>(len - fresh + i0 - window + 1, 0) : 0;
    const int64_t hi = causal ? std::max<int64_t>(std::min(len, len - fresh + i1 + 1), 0) : len;
    return std::max<int64_t>((hi + 63) / 64 - lo / 64, 1);
}

void check(const nvfp4_kv_cache_t& c, const nvfp4_kv_seqs_t& s, const nvfp4_kv_queries_t& q, std::mt19937_64& g) {
    if (nvfp4::check_kv_cache(&c) != NVFP4_OK || nvfp4::check_kv_seqs(&s, true) != NVFP4_OK ||
        nvfp4::check_kv_queries(&c, &s, &q) != NVFP4_OK)
        return;
    const nvfp4::KvPlan p = nvfp4::kv_plan(&c, &s, &q);
    const int64_t bytes = nvfp4::kv_workspace_bytes(&c, &s, &q);
    const int64_t window = nvfp4::kv_window(&q);
    expect(window >= 0 && window < (int64_t(1) << 29) && (window == 0 || window == q.window), "window", s, q);
    expect(p.splits >= 1 && p.chunk >= 1 && p.row_tiles >= 0 && p.part_rows >= 0 && bytes >= 0, "signs", s, q);
    expect(bytes >= p.part_rows * (c.head_dim + 2) * 4 + (p.planned ? (2 + 2 * s.seqs) * 4 : 0), "workspace", s, q);
    if (q.max_q == 0) return;
    if (!p.tile) expect(p.items >= 1, "items", s, q);
    for (int turn = 0; turn < 6; ++turn) {
        auto upto = [&](int64_t most) { return most <= 0 ? 0 : turn < 2 ? most : int64_t(g() % uint64_t(most + 1)); };
        const int64_t len = upto(q.max_kv), fresh = turn == 0 ? q.max_q : std::max<int64_t>(upto(q.max_q), 1);
        const int64_t seen = pages_seen(window, q.causal, len, fresh, 0, fresh - 1);
        if (p.tile) {
            // a tile has the last of its parts take what is left, so only one part may see it all
            if (p.splits > 1) expect(p.part_rows >= p.splits * s.total * q.heads, "parts of a tile", s, q);
        } else {
            const int64_t parts = (seen + p.chunk - 1) / p.chunk;
            expect(parts <= p.splits, "parts of a segment", s, q);
            if (seen > p.chunk) expect(p.part_rows >= int64_t(p.items) * nvfp4::kKvRowTile, "room for parts", s, q);
            const int64_t segments = p.row_tiles * c.kv_heads;
            if (!p.planned) expect(p.items >= segments * s.seqs * p.splits, "an item for each part", s, q);
        }
    }
}

}  // namespace

int main() {
    std::mt19937_64 g(5);
    const int64_t big = std::numeric_limits<int64_t>::max();
    const nvfp4_kv_cache_t cache{reinterpret_cast<uint8_t*>(place), 4, 2, 128, 1.0f, 1.0f};
    int32_t* ints = reinterpret_cast<int32_t*>(place);
    const int64_t windows[] = {0, 1, 63, 64, 65, 1500, 65535, 65536, (int64_t(1) << 29) - 1, int64_t(1) << 29, int64_t(1) << 31,
                               int64_t(1) << 32, big - 65536, big - 1, big};
    const int64_t lens[] = {0, 1, 64, 777, 1025, 2048, 65536, 131071, int64_t(1) << 29};
    const int64_t news[] = {0, 1, 5, 8, 9, 16, 33, 4099, int64_t(1) << 24};
    const int64_t seqs[] = {1, 3, 48, 700, 65535};
    for (int64_t w : windows)
        for (int64_t n : lens)
            for (int64_t m : news)
                for (int64_t count : seqs)
                    for (int64_t group : {1, 4, 127, 256})
                        for (int kv_heads : {1, 8, 1024})
                            for (int causal : {0, 1}) {
                                nvfp4_kv_cache_t c = cache;
                                c.kv_heads = kv_heads;
                                const int64_t heads = group * kv_heads;
                                const int64_t total = std::min(std::min(count * m, nvfp4::kKvMaxTotal), int64_t(0x7fffffff) / heads);
                                const nvfp4_kv_seqs_t s{ints, ints, ints, std::max<int64_t>((n + 63) / 64, 1), count, total};
                                nvfp4_kv_queries_t q{};
                                q.q = place, q.q_pitch = 1024, q.q_head_pitch = 128, q.heads = heads, q.max_q = m, q.max_kv = n;
                                q.window = w, q.scale = 1.0f, q.causal = causal;
                                check(c, s, q, g);
                            }
    for (int i = 0; i < 200000; ++i) {
        auto pick = [&](double low, double high) {
            return int64_t(std::exp(std::uniform_real_distribution<double>(std::log(low), std::log(high))(g)));
        };
        nvfp4_kv_cache_t c = cache;
        c.kv_heads = int32_t(pick(1, 65));
        const int64_t n = pick(1, 400000), m = pick(1, 3000), count = pick(1, 3000), heads = pick(1, 33) * c.kv_heads;
        const nvfp4_kv_seqs_t s{ints, ints, ints, (n + 63) / 64, count, std::min(count * m, int64_t(0x7fffffff) / heads)};
        nvfp4_kv_queries_t q{};
        q.q = place, q.q_pitch = 1024, q.q_head_pitch = 128, q.heads = heads, q.max_q = m, q.max_kv = n;
        q.window = g() % 3 == 0 ? 0 : pick(1, 9e18), q.scale = 1.0f, q.causal = int32_t(g() % 2);
        check(c, s, q, g);
    }
    std::printf("plan ok %lld\n", (long long)checks);
    return 0;
}
