// The spans in which the log probabilities' alternatives take the tiles
// (csrc/xent_units.h), walked on the host: every tile of every row tile once, a
// span's tiles one behind another between its first and its last, and a list of
// its own for each row and column half of a span.
#include "xent_units.h"

#include <cstdio>
#include <set>
#include <vector>

using namespace carbon;

int main() {
    const int64_t sizes[] = {1, 8, 255, 256, 257, 300, 1000, 2048, 4097, 8192, 20000};
    const int64_t vocabularies[] = {1, 28, 127, 128, 129, 257, 3000, 5003, 32000, 50257, 131072};
    int64_t walked = 0;
    for (int64_t M : sizes)
        for (int64_t V : vocabularies)
            for (int top : {1, 8, 9, 28})
                for (double share : {1.0, 0.4, 0.0}) {
                    Plan p;
                    const int64_t bytes = make_plan(&p, nullptr, M, 64, V, false, false, top);
                    if (bytes != make_plan(nullptr, nullptr, M, 64, V, false, false, top)) return 1;
                    if (p.Mp == kBM) {                     // stored logits instead
                        if (p.lists != 0 || p.pitch < V || p.pitch % 4 != 0) return 2;
                        continue;
                    }
                    const int kept = (int)(share * (double)M);
                    Walk w(p, kept);
                    const int tiles = (int)((V + p.lwidth - 1) / p.lwidth);
                    std::vector<char> seen((size_t)w.tm * tiles, 0);
                    std::set<std::pair<int, int64_t>> lists;
                    for (uint32_t s = 0;; ++s) {
                        Unit o = w.in_span(s, 0);
                        if (o.left == 0) {
                            if (s != (uint32_t)w.tm * (uint32_t)p.spans) return 3;
                            break;
                        }
                        const int m0 = o.m0, place = o.left >> kSpanShift;
                        if (!lists.insert({m0, place}).second || place >= p.spans) return 4;
                        if ((int64_t)(place + 1) * (p.lwidth / kGroup) > p.lists) return 5;
                        for (int j = 0;; ++j) {
                            o = w.in_span(s, j);
                            ++walked;
                            if (((o.left & kFirst) != 0) != (j == 0) || o.m0 != m0 || o.left >> kSpanShift != place) return 6;
                            if (o.n0 / p.lwidth / p.span != place || o.piece != 0 || o.type != UNIT_L) return 7;
                            if (o.n0 >= V || o.width % 128 != 0 || o.width < 128 || o.width > p.lwidth) return 8;
                            if (o.n0 + o.width < V && o.width != p.lwidth) return 9;
                            char &at = seen[(size_t)(m0 / kBM) * tiles + o.n0 / p.lwidth];
                            if (at) return 10;
                            at = 1;
                            if (o.left & kLast) break;
                            if (j > kSpan) return 11;
                        }
                    }
                    for (char c : seen)
                        if (!c) return 12;
                }
    if (walked < 100000) return 13;
    std::puts("ok");
    return 0;
}
