// xent_tiles.cuh - the output layer's products on the tensor cores: preparation
// of the positions that count, the persistent kernel that works through the
// units of xent_units.h, and the sums of dx.  Included by linear_xent.cu (the
// loss), which describes the units, and by what else forms the logits; each
// has its own copies of the kernels and its own status word.
#pragma once

#include "bounds.cuh"
#include "cta_pair.cuh"
#include "device_sync.cuh"
#include "rowvec.cuh"
#include "tcgen05.cuh"
#include "xent_units.h"

namespace carbon {
namespace {

__device__ unsigned int g_xent_status = 0;
#define CHK(idx, len, n) in_bounds(&g_xent_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

static_assert(kBM == kPairRows, "a pair's tile");
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);        // TMA producer, MMA issuer, scheduler, reporter, epilogue
constexpr uint32_t kABytes = 128 * kBK * 2;           // per CTA: 128 rows of A, half of B's columns
constexpr uint32_t kStageBytes = kABytes + kBN / 2 * kBK * 2;
constexpr int kSlots = 6;                             // units known to a CTA at a time

// Shared memory.  As many stages as fit: the tensor cores wait for operands
// more than for anything else (8192 x 768 x 50257, the loss and its gradients
// with five stages and two staging buffers per warp: 1488 us, with six and
// one: 1451).  The loss stores no tiles and needs no staging.
// The lists of alternatives (LIST of them kept per thread of the epilogue) take
// the place of a stage, or of two.
template <bool GRAD, int LIST>
struct Layout {
    static constexpr int kStages = GRAD || LIST > 0 ? (LIST > 12 ? 5 : 6) : 7;
    static constexpr uint32_t kStagingOffset = kStages * kStageBytes;
    static constexpr uint32_t kListOffset = kStagingOffset;           // [LIST][threads of the epilogue] of 8 bytes
    static constexpr uint32_t kBarOffset = kStagingOffset + (GRAD ? kEpiWarps * 4096 : LIST * kEpiWarps * 32 * 8);
    static constexpr int kBars = (2 * kStages + 4 + 3 * kSlots + 1 + 1) / 2 * 2;   // an even number: units follow
    static constexpr uint32_t kUnitOffset = kBarOffset + kBars * 8;
    static constexpr uint32_t kBytes = kUnitOffset + kSlots * 32 + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory per block");
    static_assert(kUnitOffset % 16 == 0, "units are read as 16-byte vectors");
};
// x and G are kept as blocks of 128 positions x 64 columns that are images of
// the MMA's operands in shared memory, for either orientation, so that a load
// is contiguous bytes.
// x: a row of 128 bytes per position, its 16-byte pieces in the order of the
// 128-byte swizzle.
// G: 8 planes of 8 columns, a plane holds 16 bytes per position (the
// unswizzled layout, core matrices of 8 positions x 16 bytes): a warp of 32
// positions writes 512 contiguous bytes a store, straight from its registers.
constexpr int kPlane = 128 * 8, kPlanes = 8 * kPlane;         // elements of a plane, of a block
// G is formed times 2^k, so that probabilities far below the type's (fp16) or
// fp32's (bf16) smallest normal value keep their bits; the sums are multiplied
// by 2^-k before the gradients' common factor (a product of the two factors
// underflows for small gradients).  |G| <= 2^(k+1): no sum comes near fp32's
// range for operands of ordinary size.
constexpr int kScaleBits16 = 12, kScaleBitsBf = 32;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

void *align128(void *p) {
    return reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(p) + 127) & ~static_cast<uintptr_t>(127));
}

// ---- positions that count --------------------------------------------------------

struct ScanArgs {
    const int64_t *targets;
    int64_t ignore_index;
    int reduction;
    float *losses, *lse_out;             // loss
    int64_t *count;
    const float *grad, *lse_in;          // gradient
    // log probabilities: losses are those; their gradient and the entropy's may be null
    float *entropy_out, *top_logp;
    int64_t *top_ids;
    const float *grad_entropy, *entropy_in;
};

__device__ __forceinline__ bool counts(const Plan &p, const ScanArgs &a, int64_t m, int64_t *tgt) {
    *tgt = a.targets[m];
    return *tgt != a.ignore_index && *tgt >= 0 && *tgt < p.V;
}

// |g|, or 0 where it is no finite number: NaN and infinity stay in their own
// rows of G and do not set the others' scale.
__device__ __forceinline__ float finite_size(float g) {
    const float v = fabsf(g);
    return v < INFINITY ? v : 0.0f;
}

// What G's entries of a position may reach (finite gradients), see above; of log
// probabilities: |g (onehot - P)| <= |g|, |P (log P + H)| <= H + 1/e.
template <bool LOGP>
__device__ __forceinline__ float entry_size(const Plan &p, const ScanArgs &a, int64_t m) {
    if (!LOGP) return finite_size(a.grad[m]);
    const float g = a.grad ? a.grad[m] : 0.0f, e = a.grad_entropy ? a.grad_entropy[m] : 0.0f;
    return finite_size(fabsf(g) + fabsf(e) * p.range);
}

// The exponent of the scale that a gradient per position takes out of G: a
// power of two, so that G's rows are rounded as they would be on their own
// (divided by gmax itself, every row's rounding depended on the largest one).
__device__ __forceinline__ int scale_exponent(float gmax) { return gmax == 0.0f ? 0 : ilogbf(gmax); }

// Long lists: positions that count ahead of each block of 128, and the largest
// finite |g| (a gradient per position).  One CTA, a warp per block.
constexpr int kCountThreads = 1024;

template <bool LOGP>
__global__ void __launch_bounds__(kCountThreads)
xent_count_kernel(const Plan p, const ScanArgs a) {
    __shared__ int counted[32];
    __shared__ float top[32];
    wait_prior_grid();
    allow_next_grid();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t blocks = (p.M + 127) / 128;
    float gmax = 0.0f;
    int base = 0;
    for (int64_t b0 = 0; b0 < blocks; b0 += 32) {
        int n = 0;
        for (int j = 0; j < 4; ++j) {
            const int64_t m = (b0 + warp) * 128 + j * 32 + lane;
            int64_t tgt;
            const bool k = m < p.M && counts(p, a, m, &tgt);
            n += __popc(__ballot_sync(0xffffffffu, k));
            if (k && p.grad && a.reduction == CARBON_REDUCE_NONE) gmax = fmaxf(gmax, entry_size<LOGP>(p, a, m));
        }
        if (lane == 0) counted[warp] = n;
        __syncthreads();
        int before = base;
        for (int w = 0; w < 32; ++w) {
            if (w == warp && lane == 0 && b0 + warp < blocks) p.ahead[b0 + warp] = before;
            before += counted[w];
        }
        base = before;
        __syncthreads();
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, o));
    if (lane == 0) top[warp] = gmax;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < 32; ++w) gmax = fmaxf(gmax, top[w]);
        p.head->gmax = gmax;
    }
}

// A CTA per 128 positions and 64 columns: the positions that count move up, in
// order, into x's blocks, with zeros up to the last tile's end and past D; the
// CTAs of the first columns also write what the tiles need of each position,
// and the zeros of ignored ones.  Without `ahead` a CTA counts the positions
// before its own by itself, up to kCountAhead of them: a launch less, and less
// time (16384 positions of width 768, cold: 24 us, with `ahead` 10 and 23 for
// the counting kernel; every block of columns counts, so at width 8192 it is
// 150 against 82 and 23).
constexpr int kPrepThreads = 256;

template <bool LOGP>
__global__ void __launch_bounds__(kPrepThreads)
xent_prepare_kernel(const Plan p, const ScanArgs a, const uint4 *__restrict__ x) {
    __shared__ int part[kPrepThreads / 32], flag_words[4];
    __shared__ float part_max[kPrepThreads / 32];
    __shared__ int place[128];                            // a position's place, or -1
    wait_prior_grid();
    allow_next_grid();
    const int t = threadIdx.x, lane = t % 32, warp = t / 32;
    const int64_t first = (int64_t)blockIdx.x * 128;
    const bool lead = blockIdx.y == 0, last = blockIdx.x == gridDim.x - 1;
    const bool each = p.grad && a.reduction == CARBON_REDUCE_NONE;

    int n = 0;
    float gmax = 0.0f;
    int64_t tgt;
    if (p.ahead == nullptr) {
        const bool all = each && lead;                    // gmax is taken over the whole list
#pragma unroll 8
        for (int64_t m = t; m < (all ? p.M : first); m += kPrepThreads)
            if (counts(p, a, m, &tgt)) {
                n += m < first ? 1 : 0;
                if (all) gmax = fmaxf(gmax, entry_size<LOGP>(p, a, m));
            }
        n = __reduce_add_sync(0xffffffffu, n);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) gmax = fmaxf(gmax, __shfl_xor_sync(0xffffffffu, gmax, o));
        if (lane == 0) { part[warp] = n; part_max[warp] = gmax; }
    }
    int64_t mine = a.ignore_index;
    bool keep = false;
    if (t < 128) {
        const int64_t m = first + t;
        if (m < p.M && CHK(m, 1, p.M)) {
            keep = counts(p, a, m, &mine);
            if (lead && !keep && mine != a.ignore_index) atomicExch(&g_xent_status, (unsigned)CARBON_ERR_OUT_OF_BOUNDS);
        }
        const unsigned word = __ballot_sync(0xffffffffu, keep);
        if (lane == 0) flag_words[warp] = (int)word;
    }
    __syncthreads();
    int base = 0;
    if (p.ahead == nullptr) {
        gmax = 0.0f;
        for (int w = 0; w < kPrepThreads / 32; ++w) { base += part[w]; gmax = fmaxf(gmax, part_max[w]); }
    } else {
        base = p.ahead[blockIdx.x];
        gmax = p.head->gmax;
    }
    int here = 0;                                         // of this CTA's positions
    for (int w = 0; w < 4; ++w) here += __popc((unsigned)flag_words[w]);
    if (t < 128) {
        int pos = base + __popc((unsigned)flag_words[warp] & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) pos += __popc((unsigned)flag_words[w]);
        place[t] = keep ? pos : -1;
        const int64_t m = first + t;
        if (lead && m < p.M) {
            p.inverse[m] = keep ? pos : -1;
            if (keep && CHK(pos, 1, p.Mp)) {
                p.rowmap[pos] = (int)m;
                p.tgt[pos] = (int)mine;
                if (p.grad) {
                    p.lse2[pos] = fmaf(a.lse_in[m], kLog2e, (float)-(p.f16 ? kScaleBits16 : kScaleBitsBf));
                    if (!LOGP) {
                        p.rfac[pos] = !each ? 1.0f : ldexpf(a.grad[m], -scale_exponent(gmax));
                    } else {
                        // G = g onehot - P (g + e (log P + H)), with log P from t = log2(P) + k
                        const int ex = -scale_exponent(gmax);
                        const float g = a.grad ? ldexpf(a.grad[m], ex) : 0.0f;
                        const float e = a.grad_entropy ? ldexpf(a.grad_entropy[m], ex) : 0.0f;
                        const float k = (float)(p.f16 ? kScaleBits16 : kScaleBitsBf) * kLn2;
                        p.rfac[pos] = a.grad_entropy ? -fmaf(e, a.entropy_in[m] - k, g) : -g;
                        p.c1[pos] = -e * kLn2;
                        p.g1[pos] = g;
                    }
                } else if (LOGP && p.lists > 0) {
                    p.floor[pos] = 0u;
                    for (int i = 0; i < top_classes(p.listed); ++i) p.largest[(int64_t)pos * top_classes(p.listed) + i] = 0u;
                }
            } else if (!keep && !p.grad) {
                a.losses[m] = 0.0f;
                a.lse_out[m] = 0.0f;
                if (LOGP) a.entropy_out[m] = 0.0f;
                for (int i = 0; LOGP && i < p.top; ++i) {
                    a.top_ids[m * p.top + i] = -1;
                    a.top_logp[m * p.top + i] = 0.0f;
                }
            }
        }
    }
    __syncthreads();

    // 8 threads per position and 128-byte row of a block
    const int q = t % 8, blk = blockIdx.y;
    const int64_t nvec = p.D / 8;
    uint4 *blocks = static_cast<uint4 *>(p.xc);
    auto put = [&](int64_t pos, uint4 v) {
        const int64_t row = (pos / 128 * p.xblocks + blk) * 128 + pos % 128;
        if (CHK(row * 8, 8, p.Mp * p.xblocks * 8)) blocks[row * 8 + (q ^ (int)(pos & 7))] = v;
    };
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int64_t m = first + u * 32 + t / 8;
        v[u] = place[u * 32 + t / 8] >= 0 && blk * 8 + q < nvec ? x[m * nvec + blk * 8 + q] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (place[u * 32 + t / 8] >= 0) put(place[u * 32 + t / 8], v[u]);
    if (!last) return;

    const int kept = base + here;
    const int64_t rows = (int64_t)row_tiles(kept) * kBM;
    for (int64_t i = kept + t / 8; i < rows; i += kPrepThreads / 8) put(i, make_uint4(0u, 0u, 0u, 0u));
    if (!lead) return;
    for (int64_t i = kept + t; i < rows; i += kPrepThreads) {
        p.tgt[i] = -1;
        if (p.grad) p.lse2[i] = p.rfac[i] = 0.0f;
        if (LOGP && p.grad) p.c1[i] = p.g1[i] = 0.0f;
    }
    for (int i = t; i < counters(p); i += kPrepThreads) p.ticket[i] = 0u;
    if (t == 0) {
        p.head->kept = kept;
        if (a.count) *a.count = kept;
        if (p.grad) {
            float g = !each ? a.grad[0] : ldexpf(1.0f, scale_exponent(gmax));
            if (LOGP) g *= p.inv_t;
            if (a.reduction == CARBON_REDUCE_MEAN) g = __fdiv_rn(g, (float)(kept > 0 ? kept : 1));
            p.head->gscale = g;
        }
    }
}

// Descriptors of the K = 16 slice k of an operand tile (boxes: box_desc).
// G: planes of 128 positions, K along the planes; or (mn) planes of 64
// positions, K along the positions (the strides change places).
__device__ __forceinline__ uint64_t plane_desc(uint32_t base, bool mn, int k) {
    return mn ? smem_desc_noswizzle(base + (uint32_t)k * 256u, 128u, 1024u)
              : smem_desc_noswizzle(base + (uint32_t)k * 4096u, 2048u, 128u);
}

// ---- the tile kernel -------------------------------------------------------------------

struct Maps {
    CUtensorMap w, w_k;         // boxes of 64 x 64 and (reduced along D) 128 rows x 64, 128-byte swizzle
    CUtensorMap x, x_k;         // half a block, the rows of 64 positions, and (reduced along D) a block
    CUtensorMap g_k;            // a block, reduced along its columns
    CUtensorMap g_mn;           // the halves of a block's planes that hold 64 positions, reduced along those
    CUtensorMap dt_out;         // store boxes of 32 rows x 64
    CUtensorMap acc;            // store boxes of 32 rows x 32 fp32
};

template <bool GRAD, int LIST>
struct Ctx : Layout<GRAD, LIST> {
    using Layout<GRAD, LIST>::kStages;
    uint32_t sbase, bars, tmem, rank;
    const Unit *slots;                   // units handed out
    volatile uint32_t *abort_flag;
    __device__ uint32_t full(int s) const { return bars + 8u * s; }                          // used in CTA 0
    __device__ uint32_t empty(int s) const { return bars + 8u * (kStages + s); }
    __device__ uint32_t tfull(int b) const { return bars + 8u * (2 * kStages + b); }
    __device__ uint32_t tempty(int b) const { return bars + 8u * (2 * kStages + 2 + b); }    // used in CTA 0
    __device__ uint32_t sfull(int s) const { return bars + 8u * (2 * kStages + 4 + s); }
    __device__ uint32_t sempty(int s) const { return bars + 8u * (2 * kStages + 4 + kSlots + s); }   // CTA 0
    __device__ uint32_t stored(int s) const { return bars + 8u * (2 * kStages + 4 + 2 * kSlots + s); }
    __device__ uint32_t wanted() const { return bars + 8u * (2 * kStages + 4 + 3 * kSlots); }       // CTA 0
    __device__ bool wait(uint32_t bar, uint32_t parity) const {
        if (mbar_wait(bar, parity)) return true;
        give_up();
        return false;
    }
    __device__ void give_up() const {
        *abort_flag = 1u;
        atomicExch(&g_xent_status, (unsigned)CARBON_ERR_TIMEOUT);
    }
    __device__ bool aborted() const { return *abort_flag != 0u; }
    __device__ void add(unsigned int *counter) const { add_release(counter, 1u); }
    // Waits until *counter reaches n.
    __device__ bool wait_count(const unsigned int *counter, unsigned int n) const {
        if (load_acquire(counter) >= n) return true;
        const uint64_t t0 = global_ns();
        while (load_acquire(counter) < n) {
            __nanosleep(64);
            if (global_ns() - t0 > kWaitBudgetNs) { give_up(); return false; }
        }
        return true;
    }
};

// Units are handed out in list order, one at a time, to whichever pair asks
// next (a pair only waits for units that a running pair already has: the
// kernel makes progress however few of its pairs the GPU runs at once).  One
// thread of CTA 0 takes them and decodes them for every role of both CTAs.
template <class C>
struct Feed {
    const C &c;
    int slot = 0;
    uint32_t ph = 0;
    // The next unit, for a whole warp.  false: none left, or gave up.  The
    // shuffles make the unit warp-uniform to the compiler, so that what the
    // TMA and MMA instructions take from it lives in uniform registers (with
    // one lane's branch instead, four TMA loads took 570 cycles to issue).
    __device__ bool next(Unit *o) {
        const bool ok = !c.aborted() && c.wait(c.sfull(slot), ph);
        if (!__all_sync(0xffffffffu, ok)) return false;
        int v[8];
        ld_shared_v4(smem_addr(c.slots + slot), v[0], v[1], v[2], v[3]);
        ld_shared_v4(smem_addr(c.slots + slot) + 16u, v[4], v[5], v[6], v[7]);
#pragma unroll
        for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(0xffffffffu, v[i], 0);   // uses v: the slot has been read
        *o = Unit{v[0], v[1], v[2], v[3], v[4], v[5], {}};
        return v[5] != 0;
    }
    // The slot may be used again.
    __device__ void release() {
        if (threadIdx.x % 32 == 0) mbar_arrive_cluster(map_rank(c.sempty(slot), 0));
        if (++slot == kSlots) { slot = 0; ph ^= 1u; }
    }
    __device__ bool take(Unit *o) {
        const bool more = next(o);
        release();
        return more;
    }
};
// readers of a unit: producers of both CTAs, the MMA issuer, both reporters and epilogues
constexpr int kReaders = 2 + 1 + 2 + 2 * kEpiWarps;

template <bool SPANS, class C>
__device__ __forceinline__ void hand_out(const Plan &p, Walk w, const C &c) {
    uint32_t span = 0;
    int tile = 0;
    int slot = 0;
    uint32_t ph = 0;
    uint32_t taken = 0;
    for (bool more = true, first = true; more && !c.aborted(); first = false) {
        // one unit ahead of the producer's, no more: units handed out early
        // wait behind a long one while other pairs run later ones (with up to
        // three ahead, the loss and its gradients took 351 us instead of 325
        // at 1200 x 768 x 50257, 1637 instead of 1588 at 8192)
        if (!first) {
            if (!c.wait(c.wanted(), taken)) return;
            taken ^= 1u;
        }
        Unit o;
        if (SPANS) {
            if (tile == 0) span = atomicAdd(p.ticket, 1u);
            o = w.in_span(span, tile);
            tile = o.left & kLast ? 0 : tile + 1;
        } else {
            o = w.at(atomicAdd(p.ticket, 1u));
        }
        if (!c.wait(c.sempty(slot), ph ^ 1u)) return;
        for (uint32_t r = 0; r < 2; ++r) {
            const uint32_t to = map_rank(smem_addr(c.slots + slot), r), bar = map_rank(c.sfull(slot), r);
            mbar_expect_cluster(bar, 32u);
            st_async_v4(to, bar, o.type, o.piece, o.m0, o.n0);
            st_async_v4(to + 16u, bar, o.width, o.left, 0, 0);
        }
        more = o.left != 0;                       // the first one past the end tells the roles to stop
        if (++slot == kSlots) { slot = 0; ph ^= 1u; }
    }
}

// Loads of one accumulation: this CTA's rows of A and columns of B, k-block by
// k-block.  A whole warp runs the loop, one lane issues.  ca, cb: coordinates
// of the first k-block (rows of the table or of x's blocks; planes of G); rows:
// whether each CTA's rows of A hold positions (else they are not loaded: what
// the MMA then reads gives rows that nothing reads); TWO: two boxes
// of B, else one.
template <int TYPE, bool TWO, class C>
__device__ __forceinline__ bool load_blocks(const Maps &maps, const C &c, int nkb, int ca, int cb, int n0, int gstep,
                                            int xstep, bool second, int &s, uint32_t &ph) {
    const uint32_t bytes = (second ? 2u : 1u) * kABytes + 2u * (TWO ? 2u : 1u) * kBlock;      // both CTAs'
    const bool load_a = c.rank == 0 || second;
    for (int kb = 0; kb < nkb; ++kb) {
        if (!__all_sync(0xffffffffu, c.wait(c.empty(s), ph ^ 1u))) return false;
        const uint32_t sa = c.sbase + s * kStageBytes, sb = sa + kABytes, bar = map_rank(c.full(s), 0);
        if (elect_one()) {
            if (c.rank == 0) mbar_arrive_expect_tx(c.full(s), bytes);
            if (TYPE == UNIT_L) {                 // x and the table, both along D
                if (load_a) tma_load_pair(sa, &maps.x_k, bar, 0, ca);
                tma_load_pair(sb, TWO ? &maps.w_k : &maps.w, bar, kb * kBK, cb);
            } else if (TYPE == UNIT_T) {          // G^T and x, along the positions
                const int h = (kb & 1) * 8;
                tma_load_pair_3d(sa, &maps.g_mn, bar, 0, h, ca);
                tma_load_pair_3d(sa + kBlock, &maps.g_mn, bar, 0, h, ca + 8);
                tma_load_pair(sb, &maps.x, bar, 0, cb);
                if (TWO) tma_load_pair(sb + kBlock, &maps.x, bar, 0, cb + 128);
            } else {                              // G and the table, along the vocabulary
                if (load_a) tma_load_pair_3d(sa, &maps.g_k, bar, 0, 0, ca);
                tma_load_pair(sb, &maps.w, bar, n0, cb);
                if (TWO) tma_load_pair(sb + kBlock, &maps.w, bar, n0 + 64, cb);
            }
        }
        __syncwarp();
        if (TYPE == UNIT_L) {
            ca += 128;
        } else if (TYPE == UNIT_T) {              // the block's other half, then the next 128 positions
            ca += (kb & 1) * gstep;
            cb += (kb & 1) ? xstep - 64 : 64;
        } else {
            ca += 8;
            cb += kBK;
        }
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
    return true;
}

template <bool GRAD, class C>
__device__ __forceinline__ void produce(const Plan &p, const Maps &maps, Walk w, const C &c) {
    int s = 0;
    uint32_t ph = 0;
    Unit o;
    Feed<C> feed{c};
    Ready ready;
    const int gstep = GRAD ? kPiece * p.buffers / 64 * 8 : 0, xstep = p.xblocks * 128;   // planes of G, rows of x, per 128 positions
    bool ok = true;
    while (ok && feed.take(&o)) {
        if (c.rank == 0 && elect_one()) mbar_arrive(c.wanted());
        if (GRAD) {
            if (!__all_sync(0xffffffffu, ready.wait(p, w, o, c))) break;
            fence_proxy_async_all();              // other CTAs' G, before this CTA's TMA reads
        }
        const int v0 = o.piece * kPiece;
        const int m0 = o.m0 + (int)c.rank * 128, n0 = o.n0 + (int)c.rank * (o.width / 2);
        const int g0 = GRAD ? (o.piece % p.buffers) * (kPiece / 64) * 8 : 0;
        const int nkb = w.k_blocks(o);
        const bool second = o.m0 + 128 < w.kept;  // CTA 1's rows hold positions
        if (!GRAD || o.type == UNIT_L) {
            const int ca = m0 / 128 * xstep, cb = v0 + n0;
            ok = o.width > 128 ? load_blocks<UNIT_L, true>(maps, c, nkb, ca, cb, 0, 0, 0, second, s, ph)
                               : load_blocks<UNIT_L, false>(maps, c, nkb, ca, cb, 0, 0, 0, second, s, ph);
        } else if (o.type == UNIT_T) {
            const int ca = g0 + m0 / 64 * 8, cb = n0 / 64 * 128;
            ok = o.width > 128 ? load_blocks<UNIT_T, true>(maps, c, nkb, ca, cb, 0, gstep, xstep, true, s, ph)
                               : load_blocks<UNIT_T, false>(maps, c, nkb, ca, cb, 0, gstep, xstep, true, s, ph);
        } else {
            const int ca = m0 / 128 * gstep + g0;
            ok = o.width > 128 ? load_blocks<UNIT_X, true>(maps, c, nkb, ca, v0, n0, 0, 0, second, s, ph)
                               : load_blocks<UNIT_X, false>(maps, c, nkb, ca, v0, n0, 0, 0, second, s, ph);
        }
    }
    // CTA 0 sees every load of both land before the pair may exit (stages not
    // armed in this pass completed earlier, so their wait returns at once)
    for (int i = 0; c.rank == 0 && i < C::kStages; ++i) {
        if (--s < 0) { s = C::kStages - 1; ph ^= 1u; }
        if (!__all_sync(0xffffffffu, mbar_wait(c.full(s), ph))) break;
    }
}

// k-blocks of one accumulation.
template <int TYPE, class C>
__device__ __forceinline__ bool issue_blocks(const C &c, uint32_t d, int width, bool f16, int from, int to, int &s,
                                             uint32_t &ph) {
    constexpr bool A_MN = TYPE == UNIT_T, B_MN = TYPE != UNIT_L;
    const uint32_t idesc = instr_desc(width, A_MN, B_MN, f16);
    for (int kb = from; kb < to; ++kb) {
        if (!__all_sync(0xffffffffu, c.wait(c.full(s), ph))) return false;
        tc_fence_after();
        const uint32_t sa = c.sbase + s * kStageBytes, sb = sa + kABytes;
        if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k)
                mma_pair(d, TYPE == UNIT_L ? box_desc(sa, false, k) : plane_desc(sa, A_MN, k), box_desc(sb, B_MN, k), idesc,
                         (kb | k) != 0 ? 1u : 0u);
            mma_commit_pair(c.empty(s));
        }
        __syncwarp();
        if (++s == C::kStages) { s = 0; ph ^= 1u; }
    }
    return true;
}

// CTA 0 issues the pair's MMAs.  The next unit is taken before the current
// one's last k-blocks are issued, so that the tensor cores have work meanwhile.
template <bool GRAD, bool F16, class C>
__device__ __forceinline__ void issue(Walk w, const C &c) {
    int s = 0, acc = 0;
    uint32_t ph = 0, aph = 0;
    Unit o, next;
    Feed<C> feed{c};
    bool more = feed.take(&next);
    while (more) {
        o = next;
        if (!__all_sync(0xffffffffu, c.wait(c.tempty(acc), aph ^ 1u))) return;
        tc_fence_after();
        const uint32_t d = c.tmem + (uint32_t)(acc * kBN);
        const int nkb = w.k_blocks(o), first = nkb > 4 ? nkb - 4 : 0;
        auto blocks = [&](int from, int to) {
            if (!GRAD || o.type == UNIT_L) return issue_blocks<UNIT_L>(c, d, o.width, F16, from, to, s, ph);
            if (o.type == UNIT_T) return issue_blocks<UNIT_T>(c, d, o.width, F16, from, to, s, ph);
            return issue_blocks<UNIT_X>(c, d, o.width, F16, from, to, s, ph);
        };
        if (!blocks(0, first)) return;
        more = feed.take(&next);
        if (!blocks(first, nkb)) return;
        if (elect_one()) mma_commit_pair(c.tfull(acc));
        __syncwarp();
        if (++acc == 2) { acc = 0; aph ^= 1u; }
    }
}

// The element of v that lies at index i, by comparison (registers have no
// index); 0 where i is not in [0, 64).
__device__ __forceinline__ float pick(const uint32_t (&v)[64], int i) {
    uint32_t r = 0u;
#pragma unroll
    for (int k = 0; k < 64; ++k)
        if (k == i) r = v[k];
    return __uint_as_float(r);
}

// Loss: this thread's row of 128 entries as a (max, sum) pair, and the
// target's logit where it is among them.
__device__ __forceinline__ void loss_rows(const Plan &p, const Unit &o, uint32_t tmem, int row, int half) {
    const int g = half * kGroup;                          // columns of this warp
    if (g >= o.width || o.n0 + g >= p.V) return;
    const int tgt = p.tgt[row] - o.n0;
    float mx = -INFINITY, sum = 0.0f;                     // of z log2(e)
#pragma unroll 1
    for (int c = g; c < g + kGroup && o.n0 + c < p.V; c += 64) {
        uint32_t r[64];
        tmem_ld64(tmem + (uint32_t)c, r);
        if (__any_sync(0xffffffffu, (unsigned)(tgt - c) < 64u)) {
            const float z = pick(r, tgt - c);
            if ((unsigned)(tgt - c) < 64u && CHK(row, 1, p.Mp)) p.zt[row] = z;
        }
        const int64_t n = p.V - o.n0 - c;
        if (n < 64) {                                     // past the vocabulary
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= n) r[i] = __float_as_uint(-INFINITY);
        }
        float top = __uint_as_float(r[0]);
#pragma unroll
        for (int i = 1; i < 64; ++i) top = fmaxf(top, __uint_as_float(r[i]));
        const float now = fmaxf(mx, top * kLog2e), ref = now == -INFINITY ? 0.0f : now;
        sum *= ex2(mx - ref);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i % 4] += ex2(fmaf(__uint_as_float(r[i]), kLog2e, -ref));
        sum += (s[0] + s[1]) + (s[2] + s[3]);
        mx = now;
    }
    const int64_t group = (o.n0 + g) / kGroup;
    if (CHK(group * p.Mp + row, 1, p.vocab_groups * p.Mp)) p.pairs[group * p.Mp + row] = make_float2(mx, sum);
}

// ---- log probabilities ---------------------------------------------------------------

// fp32 numbers in order as unsigned ones (none of them maps to 0), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t b = __float_as_uint(v);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu));
}

// A thread's largest logits of a span, and the entries they belong to: keys of
// (ordered logit, ~entry) in shared memory in no order, the least of them known
// once there are `k`.  Of equal logits those of lower entries are kept (a span's
// entries come in ascending order).
struct TopList {
    uint32_t at;             // this thread's column; the next key kEpiWarps * 256 bytes on
    int k, n, least;
    float floor, cut;        // only larger ones are taken: floor from other threads, cut from here as well
    __device__ uint32_t addr(int e) const { return at + (uint32_t)e * (kEpiWarps * 32 * 8); }
    __device__ uint64_t get(int e) const {
        uint64_t v;
        asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(addr(e)) : "memory");
        return v;
    }
    __device__ void put(int e, uint64_t key) {
        asm volatile("st.shared.u64 [%0], %1;" ::"r"(addr(e)), "l"(key) : "memory");
    }
    __device__ void reset() {
        n = 0;
        cut = floor;
    }
    __device__ void raise(float f) {
        floor = fmaxf(floor, f);
        cut = fmaxf(cut, f);
    }
    template <int LIST>
    __device__ void add(float z, int entry) {
        put(n < k ? n++ : least, (uint64_t)ordered(z) << 32 | (uint32_t)~entry);
        if (n < k) return;
        // U loads at a time, those beyond k read the largest number: a loop that may
        // end at each of them waits for every load by itself (8192 x 768 x 50257,
        // top 8: 479 us instead of 474)
        uint64_t low = ~0ull;
        constexpr int U = LIST > 12 ? 8 : LIST;
#pragma unroll 1
        for (int i = 0; i < k; i += U) {
            uint64_t v[U];
#pragma unroll
            for (int j = 0; j < U; ++j) v[j] = get(i + j);
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (v[j] < low) { low = v[j]; least = i + j; }
        }
        cut = fmaxf(floor, unordered((uint32_t)(low >> 32)));
    }
};

// The k-th largest of S values, 1 <= k <= S: a bitonic sort.
template <int S>
__device__ __forceinline__ uint32_t kth_largest(uint32_t (&v)[S], int k) {
#pragma unroll
    for (int size = 2; size <= S; size *= 2)
#pragma unroll
        for (int step = size / 2; step > 0; step /= 2)
#pragma unroll
            for (int i = 0; i < S; ++i)
                if ((i & step) == 0) {
                    const uint32_t hi = max(v[i], v[i + step]), lo = min(v[i], v[i + step]);
                    const bool down = (i & size) == 0;
                    v[i] = down ? hi : lo;
                    v[i + step] = down ? lo : hi;
                }
    uint32_t t = 0u;
#pragma unroll
    for (int i = 0; i < S; ++i) t = max(t, i >= k - 1 ? v[i] : 0u);
    return t;
}

// The number just below an ordered one; -infinity for 0, which stands for none.
__device__ __forceinline__ float just_below(uint32_t t) {
    if (t == 0u) return -INFINITY;
    const float below = unordered(t - 1u);
    return below == 0.0f ? -0x1p-149f : below;            // 0 is not above -0
}

// A logit below the k-th largest of the largest logits of S classes of entries is
// none of the row's k largest, the classes having no entry in common (xent_units.h).
// (Of 16 classes the 12th largest is about the 21st
// largest logit of all entries so far.)  Ordered; 0: fewer than k classes so far.
template <int S>
__device__ __forceinline__ uint32_t class_bound(const unsigned int *largest, int k) {
    uint32_t v[S];
#pragma unroll
    for (int i = 0; i < S; i += 4) {
        const uint4 q = __ldcg(reinterpret_cast<const uint4 *>(largest + i));
        v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
    return kth_largest(v, k);
}

// v[i] of 32 values, i per thread: five rounds of halves.
__device__ __forceinline__ float select32(const uint32_t *v, int i) {
    uint32_t a[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) a[j] = i & 16 ? v[j + 16] : v[j];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = i & 8 ? a[j + 8] : a[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] = i & 4 ? a[j + 4] : a[j];
#pragma unroll
    for (int j = 0; j < 2; ++j) a[j] = i & 2 ? a[j + 2] : a[j];
    return __uint_as_float(i & 1 ? a[1] : a[0]);
}

// As loss_rows, with the sum that the entropy needs, of differences to the
// largest logit (nothing cancels), and the candidates for the alternatives.
template <int LIST>
__device__ __forceinline__ void logp_rows(const Plan &p, const Unit &o, uint32_t tmem, int row, int half, TopList &list) {
    const int g = half * kGroup;
    if (g >= o.width || o.n0 + g >= p.V) return;
    const int tgt = p.tgt[row] - o.n0;
    if (LIST == 0 && p.pilot) {                           // only the largest of every 32, for the classes
        const int classes = top_classes(p.listed);
#pragma unroll 1
        for (int c = g; c < g + kGroup; c += 64) {
            uint32_t r[64];
            tmem_ld64(tmem + (uint32_t)c, r);
#pragma unroll
            for (int h = 0; h < 64; h += kPilotBlock) {
                float most = __uint_as_float(r[h]);
#pragma unroll
                for (int i = 1; i < kPilotBlock; ++i) most = fmaxf(most, __uint_as_float(r[h + i]));
                const int64_t at = (int64_t)row * classes + pilot_class(p, o.n0 + c + h);
                if (most > -INFINITY && tgt + o.n0 >= 0 && CHK(at, 1, p.Mp * classes)) atomicMax(p.largest + at, ordered(most));
            }
        }
        return;
    }
    float mx = -INFINITY, sum = 0.0f, weighted = 0.0f;    // of z log2(e) / temperature
    float largest = -INFINITY;                            // logit of the chunks that had a candidate
    // only what exceeds it can raise the floor
    const float floor = LIST > 0 ? list.floor : 0.0f;
#pragma unroll 1
    for (int c = g; c < g + kGroup && o.n0 + c < p.V; c += 64) {
        uint32_t r[64];
        tmem_ld64(tmem + (uint32_t)c, r);
        if (__any_sync(0xffffffffu, (unsigned)(tgt - c) < 64u)) {
            const float z = pick(r, tgt - c);
            if ((unsigned)(tgt - c) < 64u && CHK(row, 1, p.Mp)) p.zt[row] = z;
        }
        const int64_t n = p.V - o.n0 - c;
        if (n < 64) {                                     // past the vocabulary
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (i >= n) r[i] = __float_as_uint(-INFINITY);
        }
        if (LIST == 0 && p.logits != nullptr && tgt + o.n0 >= 0) {
            float *to = p.logits + (int64_t)row * p.pitch + o.n0 + c;
            if (CHK(to - p.logits, 64, p.M * p.pitch))
#pragma unroll
                for (int i = 0; i < 64; i += 4) *reinterpret_cast<uint4 *>(to + i) = make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        }
        float most[2];                                    // of either half
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            most[h] = __uint_as_float(r[32 * h]);
#pragma unroll
            for (int i = 1; i < 32; ++i) most[h] = fmaxf(most[h], __uint_as_float(r[32 * h + i]));
        }
        const float top = fmaxf(most[0], most[1]);
        if constexpr (LIST > 0) {
            if (__any_sync(0xffffffffu, top > list.cut)) {
                if (LIST <= kTopFew && __any_sync(0xffffffffu, list.cut == -INFINITY)) {
                    // nothing is known: these entries' own 16 classes of four say what can be left out
                    uint32_t v[kTopClassesFew];
#pragma unroll
                    for (int i = 0; i < kTopClassesFew; ++i)
                        v[i] = ordered(fmaxf(fmaxf(__uint_as_float(r[i]), __uint_as_float(r[i + 16])),
                                             fmaxf(__uint_as_float(r[i + 32]), __uint_as_float(r[i + 48]))));
                    list.raise(just_below(kth_largest(v, list.k)));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!__any_sync(0xffffffffu, most[h] > list.cut)) continue;
                    // bit i: the sign of cut - z (0 for NaN), two instructions each
                    uint32_t more = 0u;
#pragma unroll
                    for (int i = 31; i >= 0; --i)
                        more = __funnelshift_l(__float_as_uint(list.cut - __uint_as_float(r[32 * h + i])), more, 1);
                    while (__any_sync(0xffffffffu, more != 0u)) {
                        const int i = __ffs((int)more) - 1;       // -1 (any value) where there is none
                        const float z = select32(r + 32 * h, i);
                        if (more != 0u && z > list.cut) list.template add<LIST>(z, o.n0 + c + 32 * h + i);
                        more &= more - 1u;
                    }
                }
                largest = fmaxf(largest, top);
            }
        }
        const float now = fmaxf(mx, top * p.zscale), ref = now == -INFINITY ? 0.0f : now;
        const float down = ex2(mx - ref);
        if (mx > -INFINITY) weighted = down * fmaf(mx - ref, sum, weighted);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const float d = fmaf(__uint_as_float(r[i]), p.zscale, -ref), e = ex2(d);
            s[i % 4] += e;
            w[i % 4] = fmaf(e, fmaxf(d, -1000.0f), w[i % 4]);      // 0, not NaN, for a logit of -infinity
        }
        sum = fmaf(sum, down, (s[0] + s[1]) + (s[2] + s[3]));
        weighted += (w[0] + w[1]) + (w[2] + w[3]);
        mx = now;
    }
    const int64_t at = (int64_t)((o.n0 + g) / kGroup) * p.Mp + row;
    if (CHK(at, 1, p.vocab_groups * p.Mp)) {
        p.pairs[at] = make_float2(mx, sum);
        p.weighted[at] = weighted;
    }
    if constexpr (LIST > 0) {
        const int cls = group_class(p, o.n0 + g);
        const int64_t at = (int64_t)row * top_classes(p.listed) + cls;
        if (cls >= 0 && largest > floor && CHK(at, 1, p.Mp * top_classes(p.listed))) atomicMax(p.largest + at, ordered(largest));
    }
}

__device__ __forceinline__ unsigned long long *list_of(const Plan &p, int64_t row, int64_t l) {
    return p.list + (row * p.lists + l) * (p.listed + 1);
}

// The end of a span: its keys, for the join.
__device__ __forceinline__ void put_list(const Plan &p, const Unit &o, int row, int half, const TopList &list) {
    if (half >= p.lwidth / kGroup) return;                // one list per row
    unsigned long long *to = list_of(p, row, (int64_t)(o.left >> kSpanShift) * (p.lwidth / kGroup) + half);
    if (!CHK(to - p.list, p.listed + 1, p.Mp * p.lists * (p.listed + 1))) return;
    to[0] = (unsigned long long)list.n;
    for (int e = 0; e < list.n; ++e) to[1 + e] = list.get(e);
}

template <bool GRAD, bool F16, bool LOGP, int LIST, class C>
__device__ __forceinline__ void epilogue(const Plan &p, const Maps &maps, const Walk w, const C &c, int warp, int lane) {
    const int quarter = warp % 4, half = (warp - 4) / 4;  // 32 rows; one half of the columns
    const uint32_t stg = c.sbase + C::kStagingOffset + (uint32_t)(warp - 4) * 4096u;
    const float gscale = GRAD ? p.head->gscale : 0.0f;
    constexpr float kOne = (float)(1ull << (F16 ? kScaleBits16 : kScaleBitsBf)), kDown = 1.0f / kOne;
    int acc = 0;
    uint32_t aph = 0;
    Unit o;
    TopList list;
    if (LIST > 0) {
        list.at = c.sbase + C::kListOffset + (uint32_t)((warp - 4) * 32 + lane) * 8u;
        list.k = p.listed;
        list.least = 0;
        for (int e = list.k; e < LIST; ++e) list.put(e, ~0ull);
    }
    Feed<C> feed{c};
    for (;;) {
        const int slot = feed.slot;
        if (!feed.take(&o)) return;
        const int row0 = o.m0 + (int)c.rank * 128 + quarter * 32, row = row0 + lane;
        const int c0 = half * (o.width / 2), c1 = c0 + o.width / 2;
        float lse2 = 0.0f, rfac = 0.0f, slope = 0.0f, hit = 0.0f;
        uint32_t known = 0u;
        if constexpr (LIST > 0) {
            // what other spans have proved, used below
            known = __ldcg(p.floor + row);
            if ((o.left & kFirst) != 0) {
                list.floor = p.tgt[row] < 0 ? INFINITY : -INFINITY;
                list.reset();
            }
        }
        int tgt = -1;
        bool dead = false;                                 // a row without a position
        if (GRAD && o.type == UNIT_L) {
            lse2 = p.lse2[row];
            rfac = p.rfac[row];
            if (LOGP) {
                slope = p.c1[row];
                hit = p.g1[row];
            }
            tgt = p.tgt[row];
            dead = tgt < 0;
            tgt -= o.piece * kPiece + o.n0;                 // column of this tile
        }
        if (!__all_sync(0xffffffffu, c.wait(c.tfull(acc), aph))) return;
        tc_fence_after();
        const uint32_t tmem = c.tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kBN);
        if constexpr (LIST > 0) {
            // Classes are looked at where a span starts, and as long as nothing is
            // known (for every tile: 511 us instead of 471 at 8192 x 768 x 50257);
            // the result is left for the row's other threads, which a tile costs one load.
            constexpr int S = LIST <= kTopFew ? kTopClassesFew : kTopClassesMany;
            list.raise(just_below(known));
            if (__any_sync(0xffffffffu, (o.left & kFirst) != 0 || list.floor == -INFINITY)) {
                const uint32_t t = class_bound<S>(p.largest + (int64_t)row * S, p.listed);
                if (just_below(t) > list.floor) {
                    list.raise(just_below(t));
                    if (CHK(row, 1, p.Mp)) atomicMax(p.floor + row, t);
                }
            }
        }
        if (!GRAD) {
            if (LOGP) logp_rows<LIST>(p, o, tmem, row, half, list);
            else loss_rows(p, o, tmem, row, half);
            if (LIST > 0 && (o.left & kLast) != 0) put_list(p, o, row, half, list);
        } else if (o.type == UNIT_L) {
            const int n = (int)(p.V - (int64_t)o.piece * kPiece) - o.n0;   // valid columns of this tile
            // this row's place in plane 0 of the first block
            uint16_t *g_row = static_cast<uint16_t *>(p.g) +
                ((int64_t)(row0 / 128) * (kPiece * p.buffers / 64) + ((o.piece % p.buffers) * kPiece + o.n0) / 64) * kPlanes +
                (row % 128) * 8;
            // whether P - onehot is G as it is (loss); whether no row is dead (log probabilities)
            const bool plain = __all_sync(0xffffffffu, LOGP ? !dead : rfac == 1.0f);
#pragma unroll 1
            for (int cc = c0; cc < c1; cc += 64) {
                uint32_t r[64], g[32];
                tmem_ld64(tmem + (uint32_t)cc, r);
                if (LOGP) {
                    // 2^k P times its factor; that of a P of 0 is held finite
#pragma unroll
                    for (int i = 0; i < 64; ++i) {
                        const float t = fmaf(__uint_as_float(r[i]), p.zscale, -lse2);
                        r[i] = __float_as_uint(ex2(t) * fmaf(slope, fmaxf(t, -300.0f), rfac));
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i)      // 2^k P
                        r[i] = __float_as_uint(ex2(fmaf(__uint_as_float(r[i]), kLog2e, -lse2)));
                }
                if (__any_sync(0xffffffffu, (unsigned)(tgt - cc) < 64u)) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (cc + i == tgt)
                            r[i] = __float_as_uint(LOGP ? fmaf(kOne, hit, __uint_as_float(r[i])) : __uint_as_float(r[i]) - kOne);
                }
                if (cc + 64 > n) {                    // past the vocabulary: exactly zero
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (cc + i >= n) r[i] = 0u;
                }
                if (!plain) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)      // a dead row is zero whatever z is
                        r[i] = dead ? 0u : LOGP ? r[i] : __float_as_uint(__uint_as_float(r[i]) * rfac);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    g[i] = pack2<F16>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                uint16_t *dst = g_row + (int64_t)(cc / 64) * kPlanes;
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (CHK(dst + q * kPlane - static_cast<uint16_t *>(p.g), 8, p.Mp * kPiece * p.buffers))
                        *reinterpret_cast<uint4 *>(dst + q * kPlane) =
                            make_uint4(g[4 * q], g[4 * q + 1], g[4 * q + 2], g[4 * q + 3]);
            }
        } else if (o.type == UNIT_T) {
#pragma unroll 1
            for (int cc = c0; cc < c1 && o.n0 + cc < p.D; cc += 64) {
                uint32_t r[64], g[32];
                tmem_ld64(tmem + (uint32_t)cc, r);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    g[i] = pack2<F16>(__uint_as_float(r[2 * i]) * kDown * gscale, __uint_as_float(r[2 * i + 1]) * kDown * gscale);
                put_rows(stg, lane, &maps.dt_out, g, o.n0 + cc, o.piece * kPiece + row0, false);
            }
        } else {
            // the pieces' sums of dx: a slot each, or added in place in order
            const bool add = adds(p, o);
            if (add) {
                if (!__all_sync(0xffffffffu, wait_sums(p, w, o, c))) return;
                fence_proxy_async_all();
            }
            const int arow = (p.slots > 1 ? o.piece * (int)p.Mp : 0) + row0;
#pragma unroll 1
            for (int cc = c0; cc < c1 && o.n0 + cc < p.D; cc += 64) {
                uint32_t r[64];
                tmem_ld64(tmem + (uint32_t)cc, r);
                put_rows(stg, lane, &maps.acc, r, o.n0 + cc, arow, add);
                if (o.n0 + cc + 32 < p.D) put_rows(stg, lane, &maps.acc, r + 32, o.n0 + cc + 32, arow, add);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(map_rank(c.tempty(acc), 0));
        if (++acc == 2) { acc = 0; aph ^= 1u; }
        if (GRAD) {
            // what other units wait for: G, in memory once the reporter has
            // fenced; sums of dx that the next piece adds to; of a T unit only
            // that it has read G
            if (o.type == UNIT_X && p.slots == 1 && elect_one()) bulk_wait_all();
            __syncwarp();
            if (lane == 0) mbar_arrive(c.stored(slot));
        }
    }
}

// A warp of its own reports finished units, so that the epilogue does not
// wait for its stores to land (5600 cycles a unit when it did).  It holds the
// unit's slot until it has reported, so at most kSlots units are unreported.
template <class C>
__device__ __forceinline__ void report(const Plan &p, const C &c) {
    Unit o;
    Feed<C> feed{c};
    while (feed.next(&o)) {
        if (!__all_sync(0xffffffffu, c.wait(c.stored(feed.slot), feed.ph))) return;
        if (elect_one()) {
            fence_proxy_async_all();                      // G is read by TMA
            report_done(p, o, c);
        }
        feed.release();
    }
}

// LOGP: log probabilities, else the loss; LIST: room for that many alternatives.
template <bool GRAD, bool F16, bool LOGP, int LIST>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
xent_tile_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Plan p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    using L = Layout<GRAD, LIST>;
    uint32_t *words = reinterpret_cast<uint32_t *>(smem + L::kUnitOffset + kSlots * sizeof(Unit));
    Ctx<GRAD, LIST> c;
    c.sbase = smem_addr(smem);
    c.bars = c.sbase + L::kBarOffset;
    c.rank = cluster_rank();
    c.slots = reinterpret_cast<const Unit *>(smem + L::kUnitOffset);
    c.abort_flag = words;
    uint32_t *tmem_slot = words + 1;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;   // warp-uniform
    if (threadIdx.x == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(c.full(s), 1);
            mbar_init(c.empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(c.tfull(b), 1);
            mbar_init(c.tempty(b), 2 * kEpiWarps);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(c.sfull(s), 1);
            mbar_init(c.sempty(s), GRAD ? kReaders : kReaders - 2);
            mbar_init(c.stored(s), kEpiWarps);
        }
        mbar_init(c.wanted(), 1);
        *c.abort_flag = 0u;
        fence_mbar_init();
        prefetch_map(&maps.x_k);
        prefetch_map(&maps.w_k);
    }
    if (warp == 1) tmem_alloc_pair(smem_addr(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                   // both CTAs' barriers are set up
    tc_fence_after();
    c.tmem = *tmem_slot;
    wait_prior_grid();
    allow_next_grid();
    const Walk w(p, p.head->kept);

    if (warp == 0) {
        produce<GRAD>(p, maps, w, c);
    } else if (warp == 1) {
        if (c.rank == 0) issue<GRAD, F16>(w, c);
    } else if (warp == 2) {
        if (lane == 0 && c.rank == 0) hand_out<(LIST > 0)>(p, w, c);
    } else if (warp == 3) {
        if (GRAD) report(p, c);
    } else {
        epilogue<GRAD, F16, LOGP, LIST>(p, maps, w, c, warp, lane);
        if (elect_one()) bulk_wait_all();                  // also after giving up: no copy reads a CTA that has left
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                   // no arrival at, or MMA into, a CTA that has left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(c.tmem, 512);
    }
    cluster_sync_all();                                   // the pair gives its columns back together
}

// ---- sums of dx ----------------------------------------------------------------

// dx: the pieces' sums in order, scaled and rounded; zeros for ignored
// positions.  A warp per position and 256 columns; up to 8 sums are loaded
// before the first is added (MANY: else there is one, and registers for more
// would leave few warps to wait for it).
template <typename T, bool MANY>
__global__ void __launch_bounds__(256)
xent_dx_kernel(const Plan p, T *__restrict__ dx) {
    wait_prior_grid();
    allow_next_grid();
    const int64_t m = (int64_t)blockIdx.x * 8 + threadIdx.x / 32, j = ((int64_t)blockIdx.y * 32 + threadIdx.x % 32) * 8;
    if (m >= p.M || j >= p.D) return;
    const int64_t i = p.inverse[m];
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = 0.0f;
    if (i >= 0) {
        const float gscale = p.head->gscale, down = 1.0f / (float)(1ull << (p.f16 ? kScaleBits16 : kScaleBitsBf));
        const float *src = p.acc + i * p.D + j;
        constexpr int U = MANY ? 8 : 1;
        for (int s0 = 0; s0 < p.slots; s0 += U) {
            float4 lo[U], hi[U];
#pragma unroll
            for (int s = 0; s < U; ++s)
                if (s0 + s < p.slots) {
                    const float4 *q = reinterpret_cast<const float4 *>(src + (int64_t)(s0 + s) * p.Mp * p.D);
                    lo[s] = q[0];
                    hi[s] = q[1];
                }
#pragma unroll
            for (int s = 0; s < U; ++s)
                if (s0 + s < p.slots) {
                    const float w[8] = {lo[s].x, lo[s].y, lo[s].z, lo[s].w, hi[s].x, hi[s].y, hi[s].z, hi[s].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) f[k] = s0 + s == 0 ? w[k] : f[k] + w[k];
                }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = f[k] * down * gscale;
    }
    if (CHK(m * p.D + j, 8, p.M * p.D)) store_f32<T, 8>(dx + m * p.D + j, f);
}

// ---- host side ----------------------------------------------------------------

// 16-bit elements, 128-byte swizzle.
cudaError_t encode(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, int box_inner, int box_outer) {
    return encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)inner, (uint64_t)outer,
                                (uint64_t)inner * 2, (uint32_t)box_inner, (uint32_t)box_outer,
                                CU_TENSOR_MAP_SWIZZLE_128B);
}

// G's blocks (n elements) as [planes][16 groups of 8 positions][64
// elements]: a box of 8 planes and `groups` groups.
cudaError_t encode_blocks(CUtensorMap *m, const void *base, int64_t n, int groups) {
    const uint64_t extent[3] = {64, 16, (uint64_t)(n / kPlane)}, stride[2] = {128, 2048};
    const uint32_t box[3] = {64, (uint32_t)groups, 8};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, extent, stride, box,
                             CU_TENSOR_MAP_SWIZZLE_NONE);
}

bool sizes_ok(int64_t M, int64_t D, int64_t V) {
    int64_t t;
    // tile coordinates and counters are 32-bit; element counts are 64-bit; a
    // launch has up to 65535 column blocks of 64
    return M >= 0 && D >= 0 && V >= 0 && M < (1ll << 30) && D <= 65535ll * 64 && V < (1ll << 30) &&
           !__builtin_mul_overflow(M, D, &t) && !__builtin_mul_overflow(t, (int64_t)16, &t) &&
           !__builtin_mul_overflow(V, D, &t) && !__builtin_mul_overflow(t, (int64_t)16, &t);
}

carbon_status_t check(const void *x, const void *table, const int64_t *targets, int64_t M, int64_t D, int64_t V,
                      int reduction, int dtype) {
    if (!sizes_ok(M, D, V)) return CARBON_ERR_INVALID_ARG;
    if (dtype != CARBON_F32 && dtype != CARBON_BF16 && dtype != CARBON_F16) return CARBON_ERR_INVALID_ARG;
    if (reduction < CARBON_REDUCE_NONE || reduction > CARBON_REDUCE_MEAN) return CARBON_ERR_INVALID_ARG;
    if (dtype == CARBON_F32) return CARBON_ERR_UNSUPPORTED;
    if (M > 0 && (D == 0 || V == 0)) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!x || !table || !targets)) return CARBON_ERR_INVALID_ARG;
    if (D % 8 != 0 || !aligned16(x) || !aligned16(table)) return CARBON_ERR_MISALIGNED;
    return CARBON_OK;
}

// Units, planes of G and rows of x's blocks are counted in 32 bits.
bool list_fits(const Plan &p) {
    // planes are numbered by TMA coordinates
    if (p.Mp * p.xblocks >= (1ll << 31) || (p.grad && p.Mp * kPiece * p.buffers / kPlane >= (1ll << 31)))
        return false;
    const int64_t tm = p.Mp / kBM, l = (p.V + 127) / 128, t = (p.V + kBM - 1) / kBM + p.pieces;
    return tm * (l + p.pieces) + (t + tm * p.pieces) * p.dtiles < (1ll << 31);
}

template <bool GRAD, bool LOGP, int LIST>
cudaError_t launch_tiles(const Plan &p, const void *table, void *dtable, int sms, cudaStream_t s) {
    Maps maps;
    cudaError_t err = encode(&maps.w, table, p.D, p.V, 64, 64);
    if (err == cudaSuccess) err = encode(&maps.w_k, table, p.D, p.V, 64, 128);
    if (err == cudaSuccess)                              // already in the swizzle's order
        err = encode_tensor_map_2d(&maps.x_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.xc, 64, (uint64_t)(p.Mp * p.xblocks), 128,
                                   64, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (GRAD && err == cudaSuccess)
        err = encode_tensor_map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.xc, 64, (uint64_t)(p.Mp * p.xblocks), 128,
                                   64, 64, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (GRAD) {
        const int64_t n = p.Mp * kPiece * p.buffers;
        if (err == cudaSuccess) err = encode_blocks(&maps.g_k, p.g, n, 16);
        if (err == cudaSuccess) err = encode_blocks(&maps.g_mn, p.g, n, 8);
        if (err == cudaSuccess)
            err = encode_tensor_map_2d(&maps.acc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.acc, (uint64_t)p.D,
                                       (uint64_t)(p.Mp * p.slots), (uint64_t)p.D * 4, 32, 32,
                                       CU_TENSOR_MAP_SWIZZLE_128B);
        if (err == cudaSuccess) err = encode(&maps.dt_out, dtable, p.D, p.V, 64, 32);
    } else {
        maps.x = maps.g_k = maps.g_mn = maps.dt_out = maps.acc = maps.x_k;     // unused
    }
    if (err != cudaSuccess) return err;
    auto kern = p.f16 ? xent_tile_kernel<GRAD, true, LOGP, LIST> : xent_tile_kernel<GRAD, false, LOGP, LIST>;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<GRAD, LIST>::kBytes);
    if (err != cudaSuccess) return err;
    count_launch();
    // the pair is the kernel's compile-time cluster
    return launch_k(kern, dim3((unsigned)(sms / 2 * 2)), dim3(kThreads), (size_t)Layout<GRAD, LIST>::kBytes, s, 1, maps, p);
}

template <bool LOGP>
cudaError_t launch_prepare(const Plan &p, const ScanArgs &a, const void *x, cudaStream_t s) {
    if (p.ahead) {
        count_launch();
        const cudaError_t err = launch_k(xent_count_kernel<LOGP>, dim3(1), dim3(kCountThreads), 0, s, 1, p, a);
        if (err != cudaSuccess) return err;
    }
    count_launch();
    return launch_k(xent_prepare_kernel<LOGP>, dim3((unsigned)((p.M + 127) / 128), (unsigned)p.xblocks), dim3(kPrepThreads), 0, s,
                    1, p, a, static_cast<const uint4 *>(x));
}

template <typename T>
cudaError_t launch_dx(const Plan &p, T *dx, cudaStream_t s) {
    count_launch();
    const dim3 grid((unsigned)((p.M + 7) / 8), (unsigned)((p.D + 255) / 256));
    return launch_k(p.slots > 1 ? xent_dx_kernel<T, true> : xent_dx_kernel<T, false>, grid, dim3(256), 0, s, 1, p, dx);
}

}  // namespace
}  // namespace carbon
