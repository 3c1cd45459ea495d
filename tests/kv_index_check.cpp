// Drives the page and row arithmetic of the cache kernels with starts in any
// order, the sequences found as the kernels find them (built with sanitizers
// by test_kv_plan.py).
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <utility>
#include <vector>

#include "../verify_nvfp4_w4a16_amd/csrc/host/kv_index.h"

namespace {

int64_t checks = 0;

void expect(bool ok, const char* what) {
    ++checks;
    if (!ok) {
        std::printf("failed: %s\n", what);
        std::exit(1);
    }
}

// As the kernels count: 64 sequences at a time, until one of them is not below.
template <class Fn>
int last_sequence(int seqs, Fn below) {
    int found = 0;
    for (int base = 0; base < seqs; base += 64) {
        int n = 0;
        for (int s = base; s < std::min(base + 64, seqs); ++s) n += below(s);
        found += n;
        if (n < 64) break;
    }
    return found - 1;
}

void check(const std::vector<int>& starts, const std::vector<int>& lens, int total, int pitch, bool ascending) {
    const int seqs = int(lens.size());
    std::vector<int> table(size_t(seqs) * pitch, 7);
    std::set<std::pair<int, int>> filled;
    for (int u = 0; u < total / 64 + 2 * seqs; ++u) {
        const int s = last_sequence(seqs, [&](int i) { return nvfp4::kv_append_unit(starts[i], i) <= u; });
        if (s < 0) continue;
        const int nq = starts[s + 1] - starts[s], n = lens[s], first = n - nq;
        if (nq <= 0) continue;
        const int page = nvfp4::kv_append_page(u, starts[s], s, first);
        expect(page >= -1, "a page or none");
        if (page < 0 || page * 64 >= n) continue;
        expect(table.at(size_t(s) * pitch + page) == 7 && page < pitch, "a page of the sequence's row");
        if (page * 64 + 64 > first) expect(filled.insert({s, page}).second, "a page filled once");
    }
    if (ascending)
        for (int s = 0; s < seqs; ++s) {
            const int nq = starts[s + 1] - starts[s];
            for (int slot = std::max(lens[s] - nq, 0); slot < lens[s]; ++slot) expect(filled.count({s, slot / 64}) == 1, "every new slot's page");
        }
    for (int token = 0; token < total; ++token) {
        const int s = last_sequence(seqs, [&](int i) { return starts[i] <= token; });
        if (s < 0) continue;
        const int group = 3, count = std::max(starts[s + 1] - starts[s], 0) * group;
        for (int head = 0; head < group; ++head) {
            const int r = nvfp4::kv_row_of(token, starts[s], group, head, count);
            expect(r >= -1 && r < count, "a row of the sequence");
            if (ascending) expect((r >= 0) == (token < starts[s + 1]) && (r < 0 || r == (token - starts[s]) * group + head), "the token's row");
        }
    }
}

}  // namespace

int main() {
    std::mt19937_64 g(3);
    for (int turn = 0; turn < 60000; ++turn) {
        const int seqs = turn % 50 ? 1 + int(g() % 6) : 60 + int(g() % 80), total = 1 + int(g() % (turn % 7 == 1 ? 3000 : turn % 3 ? 400 : 20)), pitch = 1 + int(g() % 9);
        std::vector<int> starts(seqs + 1), lens(seqs);
        for (int& x : starts) x = int(g() % (total + 1));
        for (int& x : lens) x = int(g() % (64 * pitch + 1));
        const bool ascending = turn % 2 == 0;
        if (ascending) std::sort(starts.begin(), starts.end());
        check(starts, lens, total, pitch, ascending);
    }
    std::printf("index ok %lld\n", (long long)checks);
    return 0;
}
