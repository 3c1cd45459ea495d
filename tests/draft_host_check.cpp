// Drives the verify round's argument checks with the ends of every field's type
// (built with sanitizers by test_draft_capi_cpu.py).
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <limits>

#include "../verify_nvfp4_w4a16_amd/csrc/host/draft_shapes.h"
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
    const int64_t wide[] = {small, -1, 0, 1, 2, 64, 255, 256, 257, 1024, 1025, 65535, 65536, int64_t(1) << 19, (int64_t(1) << 19) + 1,
                            int64_t(1) << 22, int64_t(1) << 23, int64_t(1) << 24, (int64_t(1) << 24) + 1, int64_t(1) << 30,
                            int64_t(1) << 31, (int64_t(1) << 31) + 1, big - 1, big};
    int32_t* w = reinterpret_cast<int32_t*>(place);
    const nvfp4_kv_pages_t pages{w, w, 100, w, 4, w, w, w, 2, 8};
    auto pages_ok = [&](const nvfp4_kv_pages_t& p) { return nvfp4::check_kv_pages(&p, w, w, w, w, w, w) == NVFP4_OK; };
    expect(pages_ok(pages), "pages");
    nvfp4_adjust_t adjust{};
    adjust.logits = place, adjust.rows = 2, adjust.vocab = 100, adjust.pitch = 100, adjust.out_pitch = 100;
    adjust.logits_type = adjust.out_type = NVFP4_LOGITS_F32, adjust.seqs = 2;
    auto adjust_ok = [&](const nvfp4_adjust_t& a) { return nvfp4::check_adjust(&a, place) == NVFP4_OK; };
    expect(adjust_ok(adjust), "adjust");
    const nvfp4_kv_cache_t caches[2] = {{reinterpret_cast<uint8_t*>(uintptr_t(1) << 40), 4, 2, 128, 1.0f, 1.0f},
                                        {reinterpret_cast<uint8_t*>(uintptr_t(1) << 41), 4, 2, 128, 1.0f, 1.0f}};
    const nvfp4_kv_seqs_t seqs{w, w, w, 4, 2, 8};
    expect(nvfp4::check_kv_move(caches, 2, &seqs, w, 16) == NVFP4_OK, "move");
    for (int64_t v : wide) {
        nvfp4_kv_pages_t p = pages;
        p.capacity = v;
        expect(pages_ok(p) == (v >= 1 && v <= nvfp4::kPoolMax), "capacity");
        p = pages, p.table_pitch = v;
        expect(pages_ok(p) == (v >= 1 && v <= nvfp4::kKvMaxTablePitch), "pitch");
        p = pages, p.seqs = v;
        expect(pages_ok(p) == (v >= 0 && v <= 65535), "seqs");
        p = pages, p.total = v;
        expect(pages_ok(p) == (v >= 0 && v <= nvfp4::kKvMaxTotal), "total");
        expect((nvfp4::check_trees(w, w, 2, 8, v) == NVFP4_OK) == (v >= 1 && v <= NVFP4_TREE_MAX), "max_q");
        expect((nvfp4::check_trees(w, w, v, 8, 1) == NVFP4_OK) == (v >= 0 && v <= 65535), "trees");
        expect((nvfp4::check_trees(w, w, 2, v, 1) == NVFP4_OK) == (v >= 0 && v <= nvfp4::kKvMaxTotal), "rows");
        for (int64_t u : wide) {
            nvfp4_kv_queries_t q{};
            q.max_q = v;
            const nvfp4_kv_tree_t t{reinterpret_cast<const uint64_t*>(place), w, u};
            if (v >= 0 && v <= nvfp4::kKvMaxTotal)   // of checked queries
                expect((nvfp4::check_kv_tree(&seqs, &q, &t) == NVFP4_OK) == (u >= 1 && u <= 4 && v <= 64 * u), "words");
            nvfp4_adjust_t a = adjust;
            a.vocab = v, a.pitch = a.out_pitch = u;
            expect(adjust_ok(a) == (v >= 1 && v <= int64_t(1) << 22 && u >= v && u <= nvfp4::kKvMaxPitch), "vocab");
            a = adjust, a.allowed = reinterpret_cast<uint32_t*>(place), a.allowed_pitch = v, a.states = u;
            expect(adjust_ok(a) == (v >= 4 && v <= nvfp4::kKvMaxPitch && u >= 0 && u <= 0x7fffffff), "states");
        }
        nvfp4_adjust_t a = adjust;
        a.history = a.history_lens = w, a.history_pitch = v;
        expect(adjust_ok(a) == (v >= 0 && v <= nvfp4::kHistoryMax), "history");
        a = adjust, a.bias_tokens = w, a.bias_values = reinterpret_cast<float*>(place), a.bias_width = v;
        expect(adjust_ok(a) == (v >= 0 && v <= NVFP4_BIAS_MAX), "bias");
        a = adjust, a.drafted = w, a.masks = reinterpret_cast<uint64_t*>(place), a.mask_words = v;
        expect(adjust_ok(a) == (v >= 1 && v <= 4), "mask words");
        a = adjust, a.rows = a.seqs = v;
        expect(adjust_ok(a) == (v >= 0 && v <= 65535), "rows");
        if (v <= 2) expect((nvfp4::check_kv_move(caches, v, &seqs, w, 16) == NVFP4_OK) == (v >= 1), "count");
        if (v > nvfp4::kMoveCaches) expect(nvfp4::check_kv_move(caches, v, &seqs, w, 16) == NVFP4_ERR_SHAPE, "count");
        expect((nvfp4::check_kv_move(caches, 2, &seqs, w, v) == NVFP4_OK) == (v >= 1 && v <= NVFP4_TREE_MAX), "path");
    }
    std::printf("host ok %d\n", checks);
    return 0;
}
