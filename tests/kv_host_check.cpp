// Drives the cache calls' argument checks with the ends of every field's type
// (built with sanitizers by test_kv_host_sanitizers.py).
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_shapes.h"

namespace {

alignas(16) char place[64];
int checks = 0;

void expect(bool ok, const char* what) {
    ++checks;
    if (!ok) {
        std::printf("failed: %s\n", what);
        std::exit(1);
    }
}

}  // namespace

int main() {
    const int64_t big = std::numeric_limits<int64_t>::max(), small = std::numeric_limits<int64_t>::min();
    const int64_t wide[] = {small, -1, 0, 1, 7, 8, 64, 65535, 65536, int64_t(1) << 23, int64_t(1) << 24, (int64_t(1) << 24) + 1,
                            int64_t(1) << 31, int64_t(1) << 32, big - 1, big};
    const float scales[] = {0.0f, -1.0f, 1e-45f, 1.0f, 3e38f, INFINITY, -INFINITY, NAN};

    const nvfp4_kv_cache_t cache{reinterpret_cast<uint8_t*>(place), 4, 2, 128, 1.0f, 1.0f};
    const nvfp4_kv_seqs_t seqs{reinterpret_cast<int32_t*>(place), reinterpret_cast<int32_t*>(place),
                               reinterpret_cast<int32_t*>(place), 4, 2, 8};
    nvfp4_kv_queries_t queries{};
    queries.q = place;
    queries.q_pitch = 1024, queries.q_head_pitch = 128, queries.heads = 8, queries.max_q = 4, queries.max_kv = 256;
    queries.scale = 1.0f, queries.causal = 1;
    expect(nvfp4::check_kv_cache(&cache) == NVFP4_OK, "cache");
    expect(nvfp4::check_kv_seqs(&seqs, true) == NVFP4_OK, "sequences");
    expect(nvfp4::check_kv_queries(&cache, &seqs, &queries) == NVFP4_OK, "queries");
    expect(nvfp4::check_kv_cache(nullptr) == NVFP4_ERR_NULL && nvfp4::check_kv_seqs(nullptr, false) == NVFP4_ERR_NULL &&
               nvfp4::check_kv_queries(&cache, &seqs, nullptr) == NVFP4_ERR_NULL, "null structs");

    for (int64_t v : wide) {
        nvfp4_kv_cache_t c = cache;
        c.pages = v;
        expect((nvfp4::check_kv_cache(&c) == NVFP4_OK) == (v >= 0 && v <= 0x7fffffff), "pages");
        nvfp4_kv_seqs_t s = seqs;
        s.seqs = v;
        expect((nvfp4::check_kv_seqs(&s, true) == NVFP4_OK) == (v >= 0 && v <= 65535), "seqs");
        s = seqs, s.total = v;
        const bool total_ok = v >= 0 && v <= nvfp4::kKvMaxTotal;
        expect((nvfp4::check_kv_seqs(&s, true) == NVFP4_OK) == total_ok, "total");
        s = seqs, s.table_pitch = v;
        const bool pitch_ok = v >= 1 && v <= nvfp4::kKvMaxTablePitch;
        expect((nvfp4::check_kv_seqs(&s, true) == NVFP4_OK) == pitch_ok, "table pitch");
        for (int64_t w : wide) {
            expect((nvfp4::check_kv_rows(place, v, w, 1) == NVFP4_OK) ==
                       (v >= 0 && w >= 0 && v <= nvfp4::kKvMaxPitch && w <= nvfp4::kKvMaxPitch && v % 8 == 0 && w % 8 == 0), "rows");
            // checked sequences only, as every call has them
            nvfp4_kv_queries_t q = queries;
            q.heads = v, q.max_q = w;
            nvfp4::check_kv_queries(&cache, &seqs, &q);
            q = queries, q.max_kv = v, q.window = w;
            expect((nvfp4::check_kv_queries(&cache, &seqs, &q) == NVFP4_OK) == (v >= 0 && v <= 256 && w >= 0), "bounds");
            s = seqs;
            if (total_ok) s.total = v;
            q = queries, q.heads = w;
            nvfp4::check_kv_queries(&cache, &s, &q);
        }
    }
    for (float f : scales) {
        nvfp4_kv_cache_t c = cache;
        c.v_scale = f;
        expect((nvfp4::check_kv_cache(&c) == NVFP4_OK) == (std::isfinite(f) && f > 0), "scale");
        nvfp4_kv_queries_t q = queries;
        q.softcap = f;
        expect((nvfp4::check_kv_queries(&cache, &seqs, &q) == NVFP4_OK) == (std::isfinite(f) && f >= 0), "softcap");
    }
    int64_t bytes = 0;
    for (int64_t v : wide) expect((nvfp4_kv_record_bytes(v, &bytes) == NVFP4_OK) == (v == 64), "record");
    expect(nvfp4_kv_record_bytes(64, nullptr) == NVFP4_ERR_NULL, "record to nowhere");
    std::printf("host ok %d\n", checks);
    return 0;
}
