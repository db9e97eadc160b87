// linear_xent.cu - output layer and softmax cross entropy without stored
// logits, on the tensor cores.
//
//   z = x . table^T,  lse = log sum_v exp z,  loss = lse - z[target]
//   G = g (softmax(z) - onehot),  dx = G . table,  dtable = G^T . x
//
// Positions that count are first gathered into a dense x (ignored ones cost
// no product, and what they hold reaches no sum).  Then one persistent kernel
// per direction works through units of one output tile; a pair of CTAs (two
// SMs, tcgen05 cta_group::2) shares a tile of 256 rows, each CTA staging its
// own 128 rows of A and half the columns of B:
//   L  256 positions x 256 vocabulary entries of z, reduced over D.
//      Loss: each row's running maximum and sum of exponentials over 128
//      entries go out as one (max, sum) pair; a second kernel joins the pairs
//      in order.  Gradient: exp(z - lse) - onehot goes out as G.
//   T  256 vocabulary entries x up to 256 columns of dtable, reduced over
//      the positions: G^T . x.
//   X  256 positions x up to 256 columns of dx, reduced over a piece of the
//      vocabulary: G . table.
// The gradient takes the vocabulary in pieces of kPiece entries: L units of
// later pieces run before the T and X units of a piece, so that a unit rarely
// waits for the units it reads (counters in the workspace; units are handed
// out in list order and wait only for earlier ones, so the waits end: xent_units.h).
//
// Fixed order: a unit's k-blocks of 64 run in ascending order into one fp32
// accumulator.  dx adds the pieces' sums in order, and a piece's size is
// fixed, so the number of positions does not show in a row's result.
//
// Bound: the tensor cores, for all but few positions: 2 M D V flops for the
// loss and three times that for the gradients (z is formed again; storing it
// would cost 2 M V fp32 or rounded values).  8192 x 768 x 50257 bf16, alone
// in the trace: loss 297 us, 2.1 PFLOP/s, the tensor pipe active in 87% of the
// cycles; gradients 1.03 ms, 1.85 PFLOP/s, 78%: G passes through HBM about
// once each way, and operands arrive late at times.  Called again and again
// they run into the power limit: 359 us, and 1.63 ms for both directions (the
// times of calls below are those of short bursts, before it is reached).  One
// position: the table's bytes, 77 MB in 26 us.
#include "bounds.cuh"
#include "device_sync.cuh"
#include "rowvec.cuh"
#include "tcgen05.cuh"
#include "xent_units.h"

namespace carbon {
namespace {

__device__ unsigned int g_xent_status = 0;
#define CHK(idx, len, n) in_bounds(&g_xent_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (4 + kEpiWarps);        // TMA producer, MMA issuer, scheduler, reporter, epilogue
constexpr uint32_t kBlock = 64 * kBK * 2;             // one 64 x 64 box: 8 KiB
constexpr uint32_t kABytes = 128 * kBK * 2;           // per CTA: 128 rows of A, half of B's columns
constexpr uint32_t kStageBytes = kABytes + kBN / 2 * kBK * 2;
constexpr int kSlots = 6;                             // units known to a CTA at a time

// Shared memory.  As many stages as fit: the tensor cores wait for operands
// more than for anything else (8192 x 768 x 50257, the loss and its gradients
// with five stages and two staging buffers per warp: 1488 us, with six and
// one: 1451).  The loss stores no tiles and needs no staging.
template <bool GRAD>
struct Layout {
    static constexpr int kStages = GRAD ? 6 : 7;
    static constexpr uint32_t kStagingOffset = kStages * kStageBytes;
    static constexpr uint32_t kBarOffset = kStagingOffset + (GRAD ? kEpiWarps * 4096 : 0);
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

// The exponent of the scale that a gradient per position takes out of G: a
// power of two, so that G's rows are rounded as they would be on their own
// (divided by gmax itself, every row's rounding depended on the largest one).
__device__ __forceinline__ int scale_exponent(float gmax) { return gmax == 0.0f ? 0 : ilogbf(gmax); }

// Long lists: positions that count ahead of each block of 128, and the largest
// finite |g| (a gradient per position).  One CTA, a warp per block.
constexpr int kCountThreads = 1024;

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
            if (k && p.grad && a.reduction == CARBON_REDUCE_NONE) gmax = fmaxf(gmax, finite_size(a.grad[m]));
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
                if (all) gmax = fmaxf(gmax, finite_size(a.grad[m]));
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
                    p.rfac[pos] = !each ? 1.0f : ldexpf(a.grad[m], -scale_exponent(gmax));
                }
            } else if (!keep && !p.grad) {
                a.losses[m] = 0.0f;
                a.lse_out[m] = 0.0f;
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
    }
    for (int i = t; i < counters(p); i += kPrepThreads) p.ticket[i] = 0u;
    if (t == 0) {
        p.head->kept = kept;
        if (a.count) *a.count = kept;
        if (p.grad) {
            float g = !each ? a.grad[0] : ldexpf(1.0f, scale_exponent(gmax));
            if (a.reduction == CARBON_REDUCE_MEAN) g = __fdiv_rn(g, (float)(kept > 0 ? kept : 1));
            p.head->gscale = g;
        }
    }
}

// ---- PTX pieces ----------------------------------------------------------------------

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(map), "r"(src), "r"(c0), "r"(c1) : "memory");
}
// *global += shared, element by element (fp32)
__device__ __forceinline__ void tma_add_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(map), "r"(src), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read_0() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void add_release(unsigned int *p, unsigned int v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned int load_acquire(const unsigned int *p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// ---- a pair of CTAs: two SMs share one tile (tcgen05 cta_group::2) -----------

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of a shared-memory location of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// 16 bytes into a CTA's shared memory, counted on a barrier there.
__device__ __forceinline__ void st_async_v4(uint32_t addr, uint32_t bar, int a, int b, int c, int d) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%2, %3, %4, %5}, [%1];"
                 ::"r"(addr), "r"(bar), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void mbar_expect_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t addr, int &a, int &b, int &c, int &d) {
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(addr) : "memory");
}
// An arrival that hands over no memory write of this thread.  (A release at
// cluster scope waits for all of the thread's global stores.)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// TMA load into this CTA's shared memory, counted on a barrier of either CTA.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void tma_load_pair_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1,
                                                 int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(slot_smem), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs so far are done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// Instruction descriptor, kind::f16: fp32 accumulate, A and B both bf16 or
// both fp16, majorness (1: rows/columns contiguous), N, M = 256 (the pair's).
__device__ __forceinline__ uint32_t instr_desc(int n, bool a_mn, bool b_mn, bool f16) {
    return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kBM >> 4) << 24);
}

// Descriptors of the K = 16 slice k of an operand tile.
// Boxes of 64 x 64 with the 128-byte swizzle: rows of 128 bytes along K, or
// (mn) 64-wide blocks whose rows are k.
__device__ __forceinline__ uint64_t box_desc(uint32_t base, bool mn, int k) {
    return mn ? smem_desc(base + (uint32_t)k * 2048u, kBlock, 1024u) : smem_desc(base + (uint32_t)k * 32u, 16u, 1024u);
}
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

template <bool GRAD>
struct Ctx : Layout<GRAD> {
    using Layout<GRAD>::kStages;
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

template <class C>
__device__ __forceinline__ void hand_out(const Plan &p, Walk w, const C &c) {
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
        const Unit o = w.at(atomicAdd(p.ticket, 1u));
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

// 32 lanes x 64 columns of 32-bit: thread t of the warp receives lane (base
// lane + t).  One statement with its wait: no use of v can move above it.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&v)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
        "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
        "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        :
          "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
          "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]),
          "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
          "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
          "=r"(v[30]), "=r"(v[31]), "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]),
          "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]), "=r"(v[41]),
          "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]),
          "=r"(v[54]), "=r"(v[55]), "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]),
          "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
        : "r"(taddr) : "memory");
}

// Sub-tiles of 32 rows x 128 bytes (64 16-bit columns or 32 of fp32) to
// global memory through the warp's 4 KiB staging buffer.  A lane holds a row;
// its 16-byte pieces lie as the 128-byte swizzle expects them.  The elected
// lane, the same one each time, issues every copy and waits for them.
__device__ __forceinline__ void put_rows(uint32_t stg, int lane, const CUtensorMap *map, const uint32_t *r, int col,
                                         int row, bool add) {
    if (elect_one()) bulk_wait_read_0();                  // the last sub-tile has left
    __syncwarp();
#pragma unroll
    for (int g = 0; g < 8; ++g)
        st_shared_v4(stg + lane * 128 + 16 * (g ^ (lane & 7)),
                     make_uint4(r[4 * g], r[4 * g + 1], r[4 * g + 2], r[4 * g + 3]));
    fence_proxy_async_smem();
    __syncwarp();
    if (elect_one()) {
        if (add) tma_add_2d(map, stg, col, row);
        else tma_store_2d(map, stg, col, row);
        bulk_commit();
    }
    __syncwarp();
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

template <bool GRAD, bool F16, class C>
__device__ __forceinline__ void epilogue(const Plan &p, const Maps &maps, const Walk w, const C &c, int warp, int lane) {
    const int quarter = warp % 4, half = (warp - 4) / 4;  // 32 rows; one half of the columns
    const uint32_t stg = c.sbase + C::kStagingOffset + (uint32_t)(warp - 4) * 4096u;
    const float gscale = GRAD ? p.head->gscale : 0.0f;
    constexpr float kOne = (float)(1ull << (F16 ? kScaleBits16 : kScaleBitsBf)), kDown = 1.0f / kOne;
    int acc = 0;
    uint32_t aph = 0;
    Unit o;
    Feed<C> feed{c};
    for (;;) {
        const int slot = feed.slot;
        if (!feed.take(&o)) return;
        const int row0 = o.m0 + (int)c.rank * 128 + quarter * 32, row = row0 + lane;
        const int c0 = half * (o.width / 2), c1 = c0 + o.width / 2;
        float lse2 = 0.0f, rfac = 0.0f;
        int tgt = -1;
        bool dead = false;                                 // a row without a position
        if (GRAD && o.type == UNIT_L) {
            lse2 = p.lse2[row];
            rfac = p.rfac[row];
            tgt = p.tgt[row];
            dead = tgt < 0;
            tgt -= o.piece * kPiece + o.n0;                 // column of this tile
        }
        if (!__all_sync(0xffffffffu, c.wait(c.tfull(acc), aph))) return;
        tc_fence_after();
        const uint32_t tmem = c.tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kBN);
        if (!GRAD) {
            loss_rows(p, o, tmem, row, half);
        } else if (o.type == UNIT_L) {
            const int n = (int)(p.V - (int64_t)o.piece * kPiece) - o.n0;   // valid columns of this tile
            // this row's place in plane 0 of the first block
            uint16_t *g_row = static_cast<uint16_t *>(p.g) +
                ((int64_t)(row0 / 128) * (kPiece * p.buffers / 64) + ((o.piece % p.buffers) * kPiece + o.n0) / 64) * kPlanes +
                (row % 128) * 8;
            const bool plain = __all_sync(0xffffffffu, rfac == 1.0f);
#pragma unroll 1
            for (int cc = c0; cc < c1; cc += 64) {
                uint32_t r[64], g[32];
                tmem_ld64(tmem + (uint32_t)cc, r);
#pragma unroll
                for (int i = 0; i < 64; ++i)          // 2^k P
                    r[i] = __float_as_uint(ex2(fmaf(__uint_as_float(r[i]), kLog2e, -lse2)));
                if (__any_sync(0xffffffffu, (unsigned)(tgt - cc) < 64u)) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (cc + i == tgt) r[i] = __float_as_uint(__uint_as_float(r[i]) - kOne);
                }
                if (cc + 64 > n) {                    // past the vocabulary: exactly zero
#pragma unroll
                    for (int i = 0; i < 64; ++i)
                        if (cc + i >= n) r[i] = 0u;
                }
                if (!plain) {
#pragma unroll
                    for (int i = 0; i < 64; ++i)      // a dead row is zero whatever z is
                        r[i] = dead ? 0u : __float_as_uint(__uint_as_float(r[i]) * rfac);
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

template <bool GRAD, bool F16>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
xent_tile_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Plan p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    using L = Layout<GRAD>;
    uint32_t *words = reinterpret_cast<uint32_t *>(smem + L::kUnitOffset + kSlots * sizeof(Unit));
    Ctx<GRAD> c;
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
        if (lane == 0 && c.rank == 0) hand_out(p, w, c);
    } else if (warp == 3) {
        if (GRAD) report(p, c);
    } else {
        epilogue<GRAD, F16>(p, maps, w, c, warp, lane);
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

// ---- joining ---------------------------------------------------------------------------

// lse and loss of 32 rows: 32 threads per row take every 32nd pair, in order,
// and their pairs are joined in thread order.  The CTA that finishes last adds
// the losses (total not null): every thread its positions in order, the
// threads' sums in a fixed tree, in float64.
__global__ void __launch_bounds__(1024)
xent_join_kernel(const Plan p, float *__restrict__ losses, float *__restrict__ lse, float *__restrict__ total, int mean) {
    __shared__ union {
        float2 pair[32][33];
        double sum[32];
    } sh;
    __shared__ bool finish;
    wait_prior_grid();
    allow_next_grid();
    const int r = threadIdx.x % 32, t = threadIdx.x / 32;
    const int64_t row = (int64_t)blockIdx.x * 32 + r;
    const int kept = p.head->kept;
    if ((int64_t)blockIdx.x * 32 < kept) {                // CTA-uniform
        float mx = -INFINITY, sum = 0.0f;
        auto join = [&](float2 q) {
            const float now = fmaxf(mx, q.x), ref = now == -INFINITY ? 0.0f : now;
            sum = sum * ex2(mx - ref) + q.y * ex2(q.x - ref);
            mx = now;
        };
#pragma unroll 4
        for (int g = t; g < p.vocab_groups; g += 32)
            if (CHK((int64_t)g * p.Mp + row, 1, p.vocab_groups * p.Mp)) join(p.pairs[(int64_t)g * p.Mp + row]);
        sh.pair[t][r] = make_float2(mx, sum);
        __syncthreads();
        if (t == 0 && row < kept) {
            for (int i = 1; i < 32; ++i) join(sh.pair[i][r]);
            const float l = (mx + log2f(sum)) * kLn2;
            const int64_t m = p.rowmap[row];
            lse[m] = l;
            losses[m] = l - p.zt[row];
        }
    }
    if (total == nullptr) return;
    if (t == 0) __threadfence();                          // this CTA's losses, before its count
    __syncthreads();
    if (threadIdx.x == 0) finish = atomicAdd(p.joined, 1u) == gridDim.x - 1;
    __syncthreads();
    if (!finish) return;
    __threadfence();
    double s = 0.0;
#pragma unroll 8
    for (int64_t m = threadIdx.x; m < p.M; m += 1024) s += (double)__ldcg(losses + m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (r == 0) sh.sum[t] = s;
    __syncthreads();
    if (t != 0) return;
    s = sh.sum[r];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (r == 0) total[0] = (float)(mean ? s / (double)(kept > 0 ? kept : 1) : s);
}

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

template <bool GRAD>
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
    auto kern = p.f16 ? xent_tile_kernel<GRAD, true> : xent_tile_kernel<GRAD, false>;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<GRAD>::kBytes);
    if (err != cudaSuccess) return err;
    count_launch();
    // the pair is the kernel's compile-time cluster
    return launch_k(kern, dim3((unsigned)(sms / 2 * 2)), dim3(kThreads), (size_t)Layout<GRAD>::kBytes, s, 1, maps, p);
}

cudaError_t launch_prepare(const Plan &p, const ScanArgs &a, const void *x, cudaStream_t s) {
    if (p.ahead) {
        count_launch();
        const cudaError_t err = launch_k(xent_count_kernel, dim3(1), dim3(kCountThreads), 0, s, 1, p, a);
        if (err != cudaSuccess) return err;
    }
    count_launch();
    return launch_k(xent_prepare_kernel, dim3((unsigned)((p.M + 127) / 128), (unsigned)p.xblocks), dim3(kPrepThreads), 0, s,
                    1, p, a, static_cast<const uint4 *>(x));
}

}  // namespace

carbon_status_t xent_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_xent_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_xent_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

}  // namespace carbon

using namespace carbon;

extern "C" {

int64_t carbon_linear_xent_fwd_workspace(int64_t M, int64_t D, int64_t V) {
    return sizes_ok(M, D, V) ? make_plan(nullptr, nullptr, M, D > 0 ? D : 1, V, false, false) : -1;
}

int64_t carbon_linear_xent_bwd_workspace(int64_t M, int64_t D, int64_t V) {
    return sizes_ok(M, D, V) ? make_plan(nullptr, nullptr, M, D > 0 ? D : 1, V > 0 ? V : 1, true, false) : -1;
}

carbon_status_t carbon_linear_xent_fwd(float *losses, float *total, float *lse, int64_t *count, const void *x,
                                       const void *table, const int64_t *targets, int64_t M, int64_t D, int64_t V,
                                       int64_t ignore_index, carbon_reduce_t reduction, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype, carbon_stream_t stream) {
    carbon_status_t st = check(x, table, targets, M, D, V, reduction, dtype);
    if (st != CARBON_OK) return st;
    if (reduction != CARBON_REDUCE_NONE && !total) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!losses || !lse || !workspace || !aligned16(workspace) ||
                  workspace_bytes < carbon_linear_xent_fwd_workspace(M, D, V)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, losses, total, lse) || !aligned_to(8, count, targets)) return CARBON_ERR_MISALIGNED;
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        cudaError_t err = cudaSuccess;
        if (total) err = cudaMemsetAsync(total, 0, sizeof(float), s);
        if (err == cudaSuccess && count) err = cudaMemsetAsync(count, 0, sizeof(int64_t), s);
        return note_cuda(err);
    }
    Plan p;
    make_plan(&p, align128(workspace), M, D, V, false, dtype == CARBON_F16);
    if (!list_fits(p)) return CARBON_ERR_INVALID_ARG;
    ScanArgs a = {};
    a.targets = targets; a.ignore_index = ignore_index; a.reduction = reduction;
    a.losses = losses; a.lse_out = lse; a.count = count;
    cudaError_t err = launch_prepare(p, a, x, s);
    if (err == cudaSuccess) err = launch_tiles<false>(p, table, nullptr, sms, s);
    if (err == cudaSuccess) {
        count_launch();
        err = launch_k(xent_join_kernel, dim3((unsigned)((M + 31) / 32)), dim3(1024), 0, s, 1, p, losses, lse,
                       reduction == CARBON_REDUCE_NONE ? nullptr : total, reduction == CARBON_REDUCE_MEAN ? 1 : 0);
    }
    return note_cuda(err);
}

carbon_status_t carbon_linear_xent_bwd(void *dx, void *dtable, const float *grad, const void *x, const void *table,
                                       const int64_t *targets, const float *lse, int64_t M, int64_t D, int64_t V,
                                       int64_t ignore_index, carbon_reduce_t reduction, void *workspace,
                                       int64_t workspace_bytes, carbon_dtype_t dtype, carbon_stream_t stream) {
    carbon_status_t st = check(x, table, targets, M, D, V, reduction, dtype);
    if (st != CARBON_OK) return st;
    if (!aligned16(dx) || !aligned16(dtable)) return CARBON_ERR_MISALIGNED;
    if (V * D > 0 && !dtable) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!dx || !grad || !lse || !workspace || !aligned16(workspace) ||
                  workspace_bytes < carbon_linear_xent_bwd_workspace(M, D, V)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, grad, lse) || !aligned_to(8, targets)) return CARBON_ERR_MISALIGNED;
    if (V * D == 0) return CARBON_OK;                     // then M == 0
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) return note_cuda(cudaMemsetAsync(dtable, 0, (size_t)(V * D) * 2, s));
    Plan p;
    make_plan(&p, align128(workspace), M, D, V, true, dtype == CARBON_F16);
    if (!list_fits(p)) return CARBON_ERR_INVALID_ARG;
    ScanArgs a = {};
    a.targets = targets; a.ignore_index = ignore_index; a.reduction = reduction;
    a.grad = grad; a.lse_in = lse;
    cudaError_t err = launch_prepare(p, a, x, s);
    if (err == cudaSuccess) err = launch_tiles<true>(p, table, dtable, sms, s);
    if (err == cudaSuccess) {
        count_launch();
        const dim3 grid((unsigned)((M + 7) / 8), (unsigned)((D + 255) / 256));
        auto join = [&](auto kern, auto *to) { return launch_k(kern, grid, dim3(256), 0, s, 1, p, to); };
        if (p.f16)
            err = p.slots > 1 ? join(xent_dx_kernel<__half, true>, static_cast<__half *>(dx))
                              : join(xent_dx_kernel<__half, false>, static_cast<__half *>(dx));
        else
            err = p.slots > 1 ? join(xent_dx_kernel<__nv_bfloat16, true>, static_cast<__nv_bfloat16 *>(dx))
                              : join(xent_dx_kernel<__nv_bfloat16, false>, static_cast<__nv_bfloat16 *>(dx));
    }
    return note_cuda(err);
}

}  // extern "C"
