// The list of units of the output layer's loss and gradients (csrc/xent_units.h)
// walked on the host: the order of the units and what each of them waits for.
//
//   order    whatever a unit waits for is done once all units ahead of it in
//            the list are: the kernel makes progress with any number of CTAs.
//   enough   whichever units of the list a pair of CTAs has had before, the
//            waits it has made by the time it runs a unit imply that all units
//            whose output this one reads, or whose input it overwrites, are done.
//
// Over a grid of sizes, random ones, and numbers of positions that count.  The
// argument names the rule; the default is `order`.
#include "xent_units.h"

#include <cmath>
#include <cstdio>
#include <cstring>
#include <random>
#include <utility>
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

// Notes the waits that were made, and the counters a unit reports to.
struct Notes {
    mutable std::vector<std::pair<const unsigned *, unsigned>> waits;
    mutable std::vector<unsigned *> adds;
    bool wait_count(const unsigned *counter, unsigned n) const {
        waits.push_back({counter, n});
        return true;
    }
    void add(unsigned *counter) const { adds.push_back(counter); }
};

// A pair that runs each unit of the list with probability `share`.
void enough(const Case &k, double share, std::mt19937 &rng) {
    std::vector<unsigned> total;
    const Plan p = plan_of(k, &total);
    Walk w(p, k.kept);
    struct Listed {
        Unit o;
        std::vector<size_t> reports;                      // counters, as indexes into `total`
    };
    std::vector<Listed> list;
    std::vector<std::vector<size_t>> of[3];               // per type and piece: places in the list
    for (auto &t : of) t.resize(p.pieces);
    for (uint32_t u = 0;; ++u) {
        const Unit o = w.at(u);
        if (o.left == 0) break;
        const Notes n;
        report_done(p, o, n);
        Listed l{o, {}};
        for (unsigned *a : n.adds) {
            l.reports.push_back((size_t)(a - total.data()));
            *a += kDone;
        }
        of[o.type][o.piece].push_back(list.size());
        list.push_back(l);
    }
    std::vector<char> complete(total.size(), 0);          // counters that this pair has seen at their last value
    auto note = [&](const Notes &n) {
        for (const auto &q : n.waits)
            if (q.second >= *q.first) complete[(size_t)(q.first - total.data())] = 1;
    };
    auto done = [&](const Listed &l) {
        for (size_t r : l.reports)
            if (complete[r]) return true;
        return false;
    };
    Ready ready;
    std::bernoulli_distribution runs(share);
    for (size_t u = 0; u < list.size(); ++u) {
        if (!runs(rng)) continue;
        const Unit &o = list[u].o;
        Notes n;
        ready.wait(p, w, o, n);
        note(n);
        auto all_done = [&](int type, int piece, int from, int to) {      // units of these output columns
            for (size_t i : of[type][piece]) {
                const Unit &q = list[i].o;
                if ((type != UNIT_L || (q.n0 < to && q.n0 + q.width > from)) && !done(list[i])) return false;
            }
            return true;
        };
        bool ok = true;
        if (o.type == UNIT_L) {                           // writes G over that of an earlier piece
            const int q = o.piece - p.buffers;
            ok = q < 0 || (all_done(UNIT_T, q, 0, 0) && all_done(UNIT_X, q, 0, 0));
        } else if (o.type == UNIT_T) {                    // G of 256 vocabulary entries, all positions
            ok = all_done(UNIT_L, o.piece, o.m0, o.m0 + kBM);
        } else {                                          // G of the piece
            ok = all_done(UNIT_L, o.piece, 0, kPiece);
            if (ok && p.slots == 1 && o.piece > 0) {      // and, before its sums go out, the piece before
                Notes s;
                wait_sums(p, w, o, s);
                std::vector<char> before = complete;
                note(s);
                ok = all_done(UNIT_X, o.piece - 1, 0, 0);
                complete = before;                        // another warp has seen this
            }
        }
        if (!ok) return fail("enough", k, p, (int64_t)u, o);
    }
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

int main(int argc, char **argv) {
    const bool walk_enough = argc > 1 && std::strcmp(argv[1], "enough") == 0;
    const std::vector<Case> all = cases();
    std::mt19937 rng(2);
    size_t in_place = 0, x_first = 0;
    for (const Case &k : all) {
        Plan p;
        make_plan(&p, nullptr, k.M, k.D, k.V, true, false);
        in_place += p.slots == 1 && p.pieces > 1;
        x_first += p.slots == 1 && p.pieces > 1 && p.lead == p.pieces && k.kept < kPiece;
        if (!walk_enough) order(k);
        if (!walk_enough || units_of(Walk(p, k.kept)) > 4000) continue;
        for (double share : {1.0, 0.3, 1.0 / 76})
            for (int i = 0; i < 3; ++i) enough(k, share, rng);
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
