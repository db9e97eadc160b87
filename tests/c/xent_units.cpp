// The list of units of the output layer's loss and gradients (csrc/xent_units.h)
// walked on the host: the order of the units and what each of them waits for.
//
//   order    whatever a unit waits for is done once all units ahead of it in
//            the list are: the kernel makes progress with any number of CTAs.
//
// Over a grid of sizes, random ones, and numbers of positions that count.
#include "xent_units.h"

#include <cmath>
#include <cstdio>
#include <random>
#include <vector>

using namespace carbon;

namespace {

int failures = 0;

struct Case {
    int64_t M, D, V;
    int kept;
};

// Counters on the host in place of the kernel's.
struct Probe {
    mutable bool ok = true;
    bool wait_count(const unsigned *counter, unsigned n) const {
        ok = ok && *counter >= n;
        return true;
    }
    void add(unsigned *counter) const { ++*counter; }
};

// A plan whose counters lie in `words`.
Plan plan_of(const Case &k, std::vector<unsigned> *words) {
    Plan p;
    make_plan(&p, nullptr, k.M, k.D, k.V, true, false);
    words->assign((size_t)counters(p), 0u);
    p.ticket = words->data();
    p.done_l = p.ticket + 2;
    p.done_t = p.done_l + p.pieces;
    p.done_x = p.done_t + p.pieces;
    p.done_v = p.done_x + p.pieces;
    return p;
}

int64_t units_of(const Walk &w) {
    int64_t n = 0;
    for (int ph = 0; ph < w.phases(); ++ph) n += w.size(ph);
    return n;
}

void fail(const char *rule, const Case &k, const Plan &p, int64_t at, const Unit &o) {
    if (++failures <= 10)
        std::fprintf(stderr, "%s: M %lld D %lld V %lld kept %d (pieces %d, lead %d, buffers %d, slots %d): unit %lld, type %d, piece %d\n",
                     rule, (long long)k.M, (long long)k.D, (long long)k.V, k.kept, p.pieces, p.lead, p.buffers, p.slots,
                     (long long)at, o.type, o.piece);
}

// One unit after the other, in list order.  Also counts them: every L, T and X
// unit of every piece appears once.
void order(const Case &k) {
    std::vector<unsigned> words;
    const Plan p = plan_of(k, &words);
    Walk w(p, k.kept);
    const Probe c;
    for (int64_t u = 0;; ++u) {
        const Unit o = w.at((uint32_t)u);
        if (o.left == 0) break;
        Ready nothing_known;
        nothing_known.wait(p, w, o, c);
        wait_sums(p, w, o, c);
        if (!c.ok) return fail("order", k, p, u, o);
        for (unsigned r = 0; r < kDone; ++r) report_done(p, o, c);
    }
    for (int q = 0; q < p.pieces; ++q)
        if (p.done_l[q] != kDone * w.n_l(q) || p.done_t[q] != kDone * w.n_t(q) || p.done_x[q] != kDone * w.n_x())
            return fail("order: units missing", k, p, q, Unit{});
}

std::vector<Case> cases() {
    std::vector<Case> all;
    auto add = [&](int64_t M, int64_t D, int64_t V) {
        for (int64_t kept : {M, M / 2, M / 9, (int64_t)0}) {
            const Case k{M, D, V, (int)kept};
            Plan p;
            make_plan(&p, nullptr, M, D, V, true, false);
            if (units_of(Walk(p, k.kept)) <= 200000) all.push_back(k);
        }
    };
    for (int64_t M : {1, 64, 256, 257, 512, 1100, 2048, 4096, 4100, 9000, 20000})
        for (int64_t D : {8, 136, 768, 1096, 2048, 3584, 4096, 5120, 8192, 12288})
            for (int64_t V : {1, 129, 4096, 4097, 4160, 4224, 8200, 16384, 32000, 50257, 131072}) add(M, D, V);
    std::mt19937 rng(1);
    auto spread = [&](double lo, double hi) {
        return (int64_t)std::exp(std::uniform_real_distribution<double>(std::log(lo), std::log(hi))(rng));
    };
    for (int i = 0; i < 2000; ++i) add(spread(1, 20000), 8 * spread(1, 1537), spread(1, 140000));
    return all;
}

}  // namespace

int main() {
    const std::vector<Case> all = cases();
    size_t in_place = 0, x_first = 0;
    for (const Case &k : all) {
        Plan p;
        make_plan(&p, nullptr, k.M, k.D, k.V, true, false);
        in_place += p.slots == 1 && p.pieces > 1;
        x_first += p.slots == 1 && p.pieces > 1 && p.lead == p.pieces && k.kept < kPiece;
        order(k);
    }
    // the sizes reach the in-place sums, also where all X units come first
    if (in_place < 100 || x_first < 100) {
        std::fprintf(stderr, "%zu cases add in place, %zu with all X units first\n", in_place, x_first);
        return 1;
    }
    if (failures) {
        std::fprintf(stderr, "%d failures\n", failures);
        return 1;
    }
    std::puts("ok");
    return 0;
}
