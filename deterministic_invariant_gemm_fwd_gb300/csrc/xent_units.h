// xent_units.h - the output layer's products as a list of units: sizes and
// workspace addresses, the order of the units, what each of them waits for, and the
// classes that bound the alternatives.  Used by linear_xent.cu and
// linear_logprob.cu (through xent_tiles.cuh); plain C++ as well, so that the order,
// the waits and the classes can be checked on the host (tests/c/xent_*.cpp).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define XENT_HD __host__ __device__
#else
#define XENT_HD
#endif

namespace carbon {

constexpr int kBM = 256, kBN = 256, kBK = 64;        // a CTA pair's tile; each CTA has 128 rows
constexpr unsigned kDone = 2;                         // reports of a finished unit: one per CTA

constexpr int kGroup = 128;              // vocabulary entries per (max, sum) pair
// Vocabulary entries per piece.  With 2048 dx adds twice as many sums
// (8192 x 768 x 50257, the loss and its gradients in short bursts: 1.77 ms
// instead of 1.54);
// 8192 took 1.50 with twice the memory for G.
constexpr int kPiece = 4096;
// G has room for pieces up to this size, and at least for those in use: half
// of L2 holds what it can of them.
constexpr int64_t kGBytes = 64ll << 20;
constexpr int64_t kSlotBytes = 64ll << 20;    // dx: the pieces' sums side by side up to this size, else added in place
constexpr int kTopSpare = 4;             // alternatives kept beyond those asked for, see linear_logprob.cu
constexpr int kTopMost = 32 - kTopSpare;
constexpr int kTopFew = 12, kTopClassesFew = 16, kTopClassesMany = 32;
XENT_HD inline int top_classes(int listed) { return listed <= kTopFew ? kTopClassesFew : kTopClassesMany; }
// Entries that a run ahead looks at, a multiple of a tile's, where there are eight
// times as many.  Without it every thread's first list takes about fifty logits
// (8192 x 768 x 50257: 465 us for 454 with top 8, 628 for 541 with top 20; 1024
// entries: 453 and 561; where 40% of the alternatives are among the first 2048
// entries 442 for 437 and 586 for 508).
constexpr int kPilot = 2048;
constexpr int kPilotBlock = 32;          // entries whose largest logit it takes
constexpr int kSpan = 8;                 // tiles that a pair takes one after another for the alternatives, at most
constexpr int64_t kCountAhead = 16384;   // longer lists of positions are counted by a kernel of their own

struct Head {
    int kept;                            // positions that count
    float gscale;                        // the gradients' common factor
    float gmax;                          // largest finite |g|, where xent_count_kernel has run
};

// Sizes and workspace addresses, host and device.
struct Plan {
    int64_t M, Mp, D, V;                 // Mp: M rounded up to a tile's rows, at least one tile
    int vocab_groups;                    // pairs per row
    int dtiles, dwidth;                  // column tiles of dx and dtable
    int xblocks;                         // blocks of x per 128 positions
    int vocab_tiles;                     // rows of T units
    int lwidth;                          // vocabulary entries per L unit
    int pieces, buffers;
    int lead;                            // pieces whose L units run ahead of a piece's T and X units
    int slots;                           // pieces' sums of dx kept side by side; 1: added in place
    bool f16, grad;
    Head *head;
    int *ahead;                          // positions that count before each block of 128, or null
    unsigned int *ticket;                // next unit
    unsigned int *joined;                // CTAs of xent_join_kernel that are done
    unsigned int *done_l, *done_t, *done_x;   // finished L, T and X units per piece
    unsigned int *done_v;                // finished L units per 256 vocabulary entries (what a T unit reads)
    int *rowmap, *inverse, *tgt;
    float *lse2, *rfac;                  // gradient: lse log2(e) - k, g / 2^e
    void *xc, *g;
    float *acc;                          // [slots][Mp][D]
    struct float2 *pairs;                // [vocab_groups][Mp]
    float *zt;                           // [Mp]: the target's logit
    // log probabilities
    bool logp;
    float zscale, inv_t;                 // log2(e) over the temperature, for logits as they are formed; 1 / temperature
    float range;                         // largest entropy + 1: bounds the gradient's entries
    float *weighted;                     // [vocab_groups][Mp]: sum of e^(z - max) (z - max), binary
                                         // once joined: zt is the largest logit times zscale, weighted's first
                                         // group log2 of the sum of powers relative to it
    float *c1, *g1;                      // gradient per position: slope along log P, and that of the token's own entry
    int top, listed;                     // alternatives asked for and kept
    float *logits;                       // [M][pitch]: few positions' logits; else null, and lists:
    int64_t pitch;
    bool pilot;                          // this is the run ahead over few entries, which fills their classes
    int piloted;                         // entries below this one have a run ahead for their classes; 0: there is none
    int span, spans;                     // tiles of a row tile that form a unit of the ticket, and their number
    int lists;                           // lists of candidates per row: one per span and column half
    unsigned int *largest;               // [Mp][top_classes]: largest logits (ordered) so far of classes of entries; 0: none
    unsigned int *floor;                 // [Mp]: a value (ordered) that `listed` logits of the row reach, or 0
    unsigned long long *list;            // [Mp][lists][1 + listed]: the number of keys, and keys (ordered logit, ~entry)
};

// 32-bit words that start at zero: ticket, joined and the counters.
XENT_HD inline int64_t counters(const Plan &p) { return 2 + 3 * (int64_t)p.pieces + p.vocab_tiles; }

inline int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Fills the plan; returns the workspace bytes.  top: alternatives per position
// (log probabilities), or -1 for the loss.
inline int64_t make_plan(Plan *out, void *ws, int64_t M, int64_t D, int64_t V, bool grad, bool f16, int top = -1) {
    Plan p = {};
    p.logp = top >= 0;
    p.top = top > 0 ? top : 0;
    p.M = M; p.D = D; p.V = V; p.grad = grad; p.f16 = f16;
    p.Mp = round_up(M > 0 ? M : 1, kBM);
    p.vocab_groups = (int)((V + kGroup - 1) / kGroup);
    p.pieces = grad ? (int)((V + kPiece - 1) / kPiece) : 1;
    // tiles of at most 256 columns, of nearly equal widths
    const int dtiles = (int)((D + kBN - 1) / kBN);
    p.dwidth = (int)round_up((D + dtiles - 1) / dtiles, 128);
    p.dtiles = (int)((D + p.dwidth - 1) / p.dwidth);
    const int64_t tiles256 = p.Mp / kBM * ((V + kBN - 1) / kBN);
    // narrower tiles where 256-wide ones would leave SMs idle for most of a wave
    p.lwidth = tiles256 < 152 * 4 ? 128 : 256;
    // How many pieces' L units run ahead of a piece's T and X units: two units
    // for each of the 76 pairs of CTAs, so that what a T or X unit reads is
    // complete when its turn comes; all of them where that is at most eight
    // each (1 x 768 x 50257: 119 us for the gradient with the loss against 146,
    // 509 x 512 x 32003: 103 against 126; but 1200 x 768 x 50257: 333 against
    // 319).  G has room for the pieces ahead, the one that is read and one
    // more; small ones are all kept.
    const int64_t l_units = p.Mp / kBM * ((kPiece + p.lwidth - 1) / p.lwidth);
    const int64_t lead = l_units * p.pieces <= 8 * 76 ? p.pieces : (2 * 76 + l_units - 1) / l_units;
    int64_t buffers = kGBytes / (p.Mp * 2 * kPiece);
    if (buffers < lead + 2) buffers = lead + 2;
    p.lead = (int)(lead < p.pieces ? lead : p.pieces);
    p.buffers = (int)(buffers < p.pieces ? buffers : p.pieces);
    p.slots = (int64_t)p.pieces * p.Mp * D * 4 <= kSlotBytes ? p.pieces : 1;

    char *base = static_cast<char *>(ws);
    int64_t used = 0;
    auto take = [&](int64_t bytes) {
        char *q = base + used;
        used += round_up(bytes, 128);
        return q;
    };
    p.head = reinterpret_cast<Head *>(take(sizeof(Head)));
    if (M > kCountAhead) p.ahead = reinterpret_cast<int *>(take(4 * (p.Mp / 128)));
    p.vocab_tiles = grad ? (int)((V + kBM - 1) / kBM) : 0;
    p.ticket = reinterpret_cast<unsigned int *>(take(4 * counters(p)));
    p.joined = p.ticket + 1;
    p.done_l = p.ticket + 2;
    p.done_t = p.done_l + p.pieces;
    p.done_x = p.done_t + p.pieces;
    p.done_v = p.done_x + p.pieces;
    p.rowmap = reinterpret_cast<int *>(take(4 * p.Mp));
    p.inverse = reinterpret_cast<int *>(take(4 * p.Mp));
    p.tgt = reinterpret_cast<int *>(take(4 * p.Mp));
    p.xblocks = (int)((D + 63) / 64);
    p.xc = take(2 * p.Mp * p.xblocks * 64);
    if (grad) {
        p.lse2 = reinterpret_cast<float *>(take(4 * p.Mp));
        p.rfac = reinterpret_cast<float *>(take(4 * p.Mp));
        if (p.logp) {
            p.c1 = reinterpret_cast<float *>(take(4 * p.Mp));
            p.g1 = reinterpret_cast<float *>(take(4 * p.Mp));
        }
        p.g = take(2 * p.Mp * kPiece * p.buffers);
        p.acc = reinterpret_cast<float *>(take(4 * (int64_t)p.slots * p.Mp * D));
    } else {
        p.pairs = reinterpret_cast<struct float2 *>(take(8 * (int64_t)p.vocab_groups * p.Mp));
        p.zt = reinterpret_cast<float *>(take(4 * p.Mp));
        if (p.logp) p.weighted = reinterpret_cast<float *>(take(4 * (int64_t)p.vocab_groups * p.Mp));
        if (p.top > 0) {
            p.listed = p.top + kTopSpare;
        }
        if (p.top > 0 && p.Mp == kBM) {
            // one row tile: its logits are less than what they are made of, and a
            // row of them is read in less time than lists take to fill
            // (8 x 768 x 50257, top 5: 43 us instead of 61)
            p.pitch = round_up(V, kGroup);
            p.logits = reinterpret_cast<float *>(take(4 * M * p.pitch));
        } else if (p.top > 0) {
            // Long spans start few lists: one for each pair of CTAs where that is
            // no more than kSpan tiles, else three or more
            const int64_t tiles = (V + p.lwidth - 1) / p.lwidth, all = p.Mp / kBM * tiles;
            int64_t span = (all + 75) / 76;
            if (span > kSpan) span = all / (3 * 76);
            p.span = (int)(span < 1 ? 1 : span > kSpan ? kSpan : span);
            p.spans = (int)((tiles + p.span - 1) / p.span);
            p.lists = p.spans * (p.lwidth / kGroup);
            p.piloted = V >= 8 * kPilot ? kPilot : 0;
            p.largest = reinterpret_cast<unsigned int *>(take(4 * p.Mp * top_classes(p.listed)));
            p.floor = reinterpret_cast<unsigned int *>(take(4 * p.Mp));
            p.list = reinterpret_cast<unsigned long long *>(take(8 * (int64_t)p.lists * (p.listed + 1) * p.Mp));
        }
    }
    if (out) *out = p;
    return used + 128;                   // room to align the base to 128 bytes
}

// ---- classes of entries ----------------------------------------------------------
//
// The largest logits of k classes bound the k-th largest of all only where no entry
// is in two of them.  The run ahead takes entries below `piloted` in blocks of
// kPilotBlock, the run over all takes the others in groups of kGroup and leaves
// those alone (its own classes for them would count a logit twice: of six large
// ones below 2048, twelve classes).

// The class of the block, or group, that starts at `entry`; -1: none of this run's.
XENT_HD inline int pilot_class(const Plan &p, int entry) { return entry < p.piloted ? entry / kPilotBlock % top_classes(p.listed) : -1; }
XENT_HD inline int group_class(const Plan &p, int entry) { return entry < p.piloted ? -1 : entry / kGroup % top_classes(p.listed); }

// ---- the list of units -------------------------------------------------------------

XENT_HD inline int lesser(int a, int b) { return a < b ? a : b; }
XENT_HD inline int row_tiles(int kept) { return kept > kBM ? (kept + kBM - 1) / kBM : 1; }

enum UnitType { UNIT_L = 0, UNIT_T = 1, UNIT_X = 2 };

struct alignas(16) Unit {
    int type, piece;
    int m0, n0;              // output tile: first row, first column (rows of the output for T are table rows)
    int width;               // columns, a multiple of 128
    int left;                // 0: the list has ended; of a span: kFirst, kLast and its place in its row
    int unused[2];
};

constexpr int kFirst = 2, kLast = 4, kSpanShift = 3;

// Phases in list order: L of the first `lead` pieces, then for each piece p: L
// of p + lead, and T and X of p, the longer of these first (T takes a k-block
// per 64 positions, X one per 64 entries).  Where all L units come first, so
// do all of the longer kind: the short units then even out the end.
struct Walk {
    const Plan &p;
    int tm;                  // row tiles of positions
    int kept;
    int phase = 0;
    uint32_t base = 0, count = 0;        // the host has checked that the list is shorter than 2^31

    XENT_HD Walk(const Plan &plan, int n) : p(plan), tm(row_tiles(n)), kept(n) { count = size(0); }

    XENT_HD int cols(int piece) const { return lesser(kPiece, (int)(p.V - (int64_t)piece * kPiece)); }
    XENT_HD uint32_t n_l(int piece) const {
        const int c = p.grad ? cols(piece) : (int)p.V;
        return (uint32_t)tm * (uint32_t)((c + p.lwidth - 1) / p.lwidth);
    }
    XENT_HD uint32_t n_t(int piece) const { return (uint32_t)((cols(piece) + kBM - 1) / kBM) * (uint32_t)p.dtiles; }
    XENT_HD uint32_t n_x() const { return (uint32_t)(tm * p.dtiles); }
    // A phase: its kind of units, or T and X of a piece, and the piece.
    static constexpr int kBoth = 3;
    XENT_HD int phases() const { return !p.grad ? 1 : p.lead == p.pieces ? 3 * p.pieces : p.lead + 2 * p.pieces; }
    XENT_HD int kind_of(int ph, int *piece) const {
        int q = ph - p.lead;
        if (q < 0) { *piece = ph; return UNIT_L; }
        if (p.lead == p.pieces) {
            const bool second = q >= p.pieces;
            *piece = second ? q - p.pieces : q;
            return second == t_first() ? UNIT_X : UNIT_T;
        }
        *piece = q & 1 ? q / 2 : p.lead + q / 2;
        return q & 1 ? kBoth : UNIT_L;
    }
    XENT_HD bool t_first() const { return kept >= kPiece; }
    XENT_HD uint32_t size(int ph) const {
        int q;
        switch (kind_of(ph, &q)) {
        case UNIT_L: return q < p.pieces ? n_l(q) : 0u;
        case UNIT_T: return n_t(q);
        case UNIT_X: return n_x();
        default: return n_t(q) + n_x();
        }
    }
    // The unit at position u of the list (u never decreases).
    XENT_HD Unit at(uint32_t u) {
        Unit o = {};
        while (u >= base + count) {
            if (phase == phases() - 1) return o;
            base += count;
            count = size(++phase);
        }
        uint32_t i = u - base;
        o.left = 1;
        o.type = kind_of(phase, &o.piece);
        if (o.type == UNIT_L) {
            const int c = p.grad ? cols(o.piece) : (int)p.V;
            o.m0 = (int)(i % (uint32_t)tm) * kBM;
            o.n0 = (int)(i / (uint32_t)tm) * p.lwidth;
            o.width = lesser(p.lwidth, (c - o.n0 + 127) / 128 * 128);
        } else {
            if (o.type == kBoth) {
                const uint32_t head = t_first() ? n_t(o.piece) : n_x();
                o.type = (i < head) == t_first() ? UNIT_T : UNIT_X;
                if (i >= head) i -= head;
            }
            o.m0 = (int)(i / (uint32_t)p.dtiles) * kBM;
            o.n0 = (int)(i % (uint32_t)p.dtiles) * p.dwidth;
            o.width = lesser(p.dwidth, (int)(p.D - o.n0 + 127) / 128 * 128);
        }
        return o;
    }
    // Tile j of span s: `span` neighbouring tiles of a row tile, spans in the
    // order of the tiles above.
    XENT_HD Unit in_span(uint32_t s, int j) const {
        Unit o = {};
        if (s >= (uint32_t)tm * (uint32_t)p.spans) return o;
        const int tiles = (int)((p.V + p.lwidth - 1) / p.lwidth), q = (int)(s / (uint32_t)tm), tile = q * p.span + j;
        o.type = UNIT_L;
        o.m0 = (int)(s % (uint32_t)tm) * kBM;
        o.n0 = tile * p.lwidth;
        o.width = lesser(p.lwidth, ((int)p.V - o.n0 + 127) / 128 * 128);
        o.left = 1 | (j == 0 ? kFirst : 0) | (j == p.span - 1 || tile == tiles - 1 ? kLast : 0) | q << kSpanShift;
        return o;
    }
    XENT_HD int k_blocks(const Unit &o) const {
        if (o.type == UNIT_L) return (int)((p.D + kBK - 1) / kBK);
        if (o.type == UNIT_T) return kept > kBK ? (kept + kBK - 1) / kBK : 1;
        return (cols(o.piece) + kBK - 1) / kBK;
    }
};

// ---- what a unit waits for -------------------------------------------------------
//
// Units are handed out in list order and may finish in any; a unit waits only
// for units ahead of it in the list, so that the first unfinished one can always
// go on, however few pairs of CTAs there are.  c.wait_count(counter, n) waits
// until *counter has reached n, c.add(counter) counts one of a unit's kDone
// reports.

// Before a unit's operands are loaded.  The last piece seen complete is
// remembered (an acquiring load costs about 1000 cycles); it says nothing about
// the pieces before it, whose units may still run.
struct Ready {
    int l = -1, tx = -1;                          // the pieces last seen complete
    template <class C>
    XENT_HD bool wait(const Plan &p, const Walk &w, const Unit &o, const C &c) {
        if (!p.grad) return true;
        if (o.type == UNIT_L) {                   // its piece's buffer is free
            const int q = o.piece - p.buffers;
            if (q < 0 || q == tx) return true;
            tx = q;
            return c.wait_count(p.done_t + q, kDone * w.n_t(q)) && c.wait_count(p.done_x + q, kDone * w.n_x());
        }
        if (o.piece == l) return true;
        if (o.type == UNIT_T) {
            const int cols = w.cols(o.piece) - o.m0, n = (lesser(cols, kBM) + p.lwidth - 1) / p.lwidth;
            return c.wait_count(p.done_v + (o.piece * kPiece + o.m0) / kBM, kDone * (unsigned)(n * w.tm));
        }
        l = o.piece;
        return c.wait_count(p.done_l + o.piece, kDone * w.n_l(o.piece));
    }
};

// Whether an X unit adds its sums to those of the piece before.
XENT_HD inline bool adds(const Plan &p, const Unit &o) { return o.type == UNIT_X && p.slots == 1 && o.piece > 0; }

// Before it does: those sums are in memory.  (Not the piece's T units: where
// all X units come first they are later in the list.)
template <class C>
XENT_HD inline bool wait_sums(const Plan &p, const Walk &w, const Unit &o, const C &c) {
    return !adds(p, o) || c.wait_count(p.done_x + (o.piece - 1), kDone * w.n_x());
}

// One of a unit's reports.
template <class C>
XENT_HD inline void report_done(const Plan &p, const Unit &o, const C &c) {
    if (o.type == UNIT_L) {
        c.add(p.done_l + o.piece);
        c.add(p.done_v + (o.piece * kPiece + o.n0) / kBM);
    } else {
        c.add((o.type == UNIT_T ? p.done_t : p.done_x) + o.piece);
    }
}

}  // namespace carbon
