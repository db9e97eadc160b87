// lora.cu - a linear layer with low-rank adapters of many requests, and its
// gradients, on the tensor cores.
//
//   y = x . W + bias + u . B_i,   u = s_i (x . A_i),   i the adapter of the row (or none)
//   dx = dy . W^T + du . A_i^T,   du = s_i (dy . B_i^T)
//   dA_i = sum over the rows of i of x^T . du,   dB_i = sum of u^T . dy
//
// Rows stay where they are.  Where the rows of a tile name several adapters, each
// adapter's products run for the whole tile with the lanes of all other rows
// disabled (tcgen05.mma leaves a disabled lane of the accumulator alone), so a
// row gets its own adapter's products and nothing of the others, whatever these
// hold, and its bits do not depend on its neighbours.
//
//   lora_shrink_kernel   u or du: 128 rows and a piece of the reduction per CTA, up
//                        to eight pieces as a cluster that adds them in order; other
//                        CTAs list the adapters of 256 rows and sort the rows by adapter.
//   lora_layer_kernel    y or dx: a pair of CTAs per tile of 256 rows, persistent;
//                        behind the layer's own k-blocks the adapters' are added to
//                        the same accumulator: one rounding, no second pass over y.
//   lora_grads_kernel    dA and dB: 128 columns and up to 1024 rows of one adapter per
//                        CTA, by bulk copies where 64 of them follow each other, else
//                        gathered one by one (no other row enters a sum).
//   lora_join_kernel     adds the pieces of adapters with more rows, in order.
//
// u and du are kept as a pair of 16-bit terms, hi + lo: 16 bits of bf16, 22 of
// fp16, for two small products in place of one.  (One 16-bit term would add half a
// unit of the output's own precision to the adapter's part.)  A third term, lo
// 2^11, serves the adapters' gradients, whose small values fp16's range would cut
// off; there it has an accumulator of its own.
//
// Bound: the layer's own product, 2 M K N flops a direction, for many rows; the
// bytes of W and of the adapters in use for few.
#include "bounds.cuh"
#include "cta_pair.cuh"
#include "rowvec.cuh"

namespace carbon {
namespace {

__device__ unsigned int g_lora_status = 0;
#define CHK(idx, len, n) in_bounds(&g_lora_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

constexpr int kMaxRank = 128;
constexpr int kBK = 64;                               // k-block: one 128-byte swizzle row
constexpr int kPlanes = 3;                            // hi, lo, lo 2^11
constexpr float kLoScale = 2048.0f;
constexpr int kPiece = 1024;                          // rows per piece of an adapter's gradient

__device__ __forceinline__ bool give_up(volatile uint32_t *abort_flag) {
    *abort_flag = 1u;
    atomicExch(&g_lora_status, (unsigned)CARBON_ERR_TIMEOUT);
    return false;
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile uint32_t *abort_flag) {
    return mbar_wait(bar, parity) || give_up(abort_flag);
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        ::"r"(dst), "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2) : "memory");
}

// MMA that leaves the lanes of set bits alone.
__device__ __forceinline__ void mma_masked(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, const uint32_t (&off)[4],
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3])
        : "memory");
}
__device__ __forceinline__ void mma_pair_masked(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, const uint32_t (&off)[8]) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, 1, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%4, %5, %6, %7, %8, %9, %10, %11}, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(off[0]), "r"(off[1]), "r"(off[2]), "r"(off[3]), "r"(off[4]), "r"(off[5]),
          "r"(off[6]), "r"(off[7])
        : "memory");
}

// Instruction descriptor of M = 128 (instr_desc has the pair's 256).
__device__ __forceinline__ uint32_t instr_desc_single(int n, bool a_mn, bool b_mn, bool f16) {
    return (instr_desc(n, a_mn, b_mn, f16) & ~(31u << 24)) | ((128u >> 4) << 24);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t local, uint32_t rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(map_rank(local, rank)) : "memory");
    return v;
}

// ---- which adapters a tile's rows name ----------------------------------------------

template <int ROWS>
struct alignas(16) Groups {
    int id[ROWS];                        // a row's adapter, or -1
    int first[ROWS];                     // the tile's first row with the same one
    int place[ROWS];                     // of a first row: its adapter's place in the list
    int adapter[ROWS];                   // the list, in the order of the first rows
    uint32_t off[ROWS][ROWS / 32];       // lanes to disable: all rows of others
    int count;
};

__device__ __forceinline__ int adapter_of(const int64_t *ids, int64_t m, int64_t M, int64_t n, bool report) {
    if (m >= M) return -1;
    const int64_t v = ids[m];
    if (v >= 0 && v < n) return (int)v;
    if (report && v != -1) atomicExch(&g_lora_status, (unsigned)CARBON_ERR_OUT_OF_BOUNDS);
    return -1;
}

// By all threads of a CTA; ends with a barrier.
template <int ROWS>
__device__ __forceinline__ void find_groups(Groups<ROWS> &g, const int64_t *ids, int64_t m0, int64_t M, int64_t n, bool report) {
    const int t = threadIdx.x, nt = blockDim.x;
    for (int i = t; i < ROWS; i += nt) g.id[i] = adapter_of(ids, m0 + i, M, n, report);
    __syncthreads();
    for (int i = t; i < ROWS; i += nt) {
        const int id = g.id[i];
        int j = g.id[0] == id ? 0 : i;
        if (j != 0 && id >= 0)
            for (int q = 0; q < ROWS; q += 4) {           // independent loads: a search that stops waits for each
                const int4 v = *reinterpret_cast<const int4 *>(g.id + q);
                j = min(min(j, v.x == id ? q : j), min(min(v.y == id ? q + 1 : j, v.z == id ? q + 2 : j), v.w == id ? q + 3 : j));
            }
        g.first[i] = id < 0 ? -1 : j;
    }
    __syncthreads();
    if (t < 32) {
        int count = 0;
        for (int i = t; i < ROWS; i += 32) {
            const unsigned heads = __ballot_sync(0xffffffffu, g.first[i] == i);
            if (g.first[i] == i) {
                const int q = count + __popc(heads & ((1u << t) - 1u));
                g.place[i] = q;
                g.adapter[q] = g.id[i];
                for (int w = 0; w < ROWS / 32; ++w) g.off[q][w] = ~0u;
            }
            count += __popc(heads);
        }
        if (t == 0) g.count = count;
    }
    __syncthreads();
    for (int i = t; i < ROWS; i += nt)
        if (g.first[i] >= 0) atomicAnd(&g.off[g.place[g.first[i]]][i / 32], ~(1u << (i % 32)));
    __syncthreads();
}

// In global memory, per tile of 256 rows: the count, then an entry per adapter.
struct alignas(16) TileEntry {
    int adapter, unused[3];
    uint32_t off[8];
};
struct alignas(16) TileList {
    int count, unused[3];
    TileEntry e[kPairRows];
};

// ---- u and du --------------------------------------------------------------------------

struct ShrinkArgs {
    const int64_t *ids;
    const float *scales;
    void *u;                             // [M][kPlanes][rp]
    TileList *lists;                     // [row tiles of 256]
    int64_t M, n;
    int r, rp;                           // rank, and rounded up to 16
    int k_blocks, per_piece, pieces;     // the reduction in 1, 2, 4 or 8 pieces of per_piece k-blocks
    int cluster, each;                   // CTAs per tile, and their pieces each
    int subsets;                         // clusters per tile: each takes part of the tile's adapters
    int stages_b;                        // stages of adapters
    // clusters ahead of those of the rows: lists of 256 rows, then rows in the order of adapters
    int extra, wide_tiles;
    int64_t sorted;                      // adapters to sort rows by: n, or 0
    int *order, *counts, *starts;
};

constexpr int kShrinkThreads = 192;      // producer, MMA issuer, epilogue
constexpr int kShrinkA = 3, kShrinkB = 12;            // stages of rows, and of adapters at most
constexpr size_t kShrinkSmem = 78 << 10;              // at least: no third CTA on an SM

struct ShrinkLayout {
    uint32_t b_stage, b, groups, bars, total;
};
__host__ __device__ inline ShrinkLayout shrink_layout(bool bwd, int rp, int stages_b) {
    ShrinkLayout l;
    l.b_stage = bwd ? (uint32_t)rp * 128u : (rp > 64 ? 2u : 1u) * kBlock;
    l.b = kShrinkA * 2 * kBlock;
    uint32_t ring = l.b + (uint32_t)stages_b * l.b_stage;
    const uint32_t partial = 128u * (uint32_t)(rp + 4) * 4u;       // over the ring, once it has been used
    if (ring < partial) ring = partial;
    l.groups = ring;
    l.bars = (l.groups + (uint32_t)sizeof(Groups<128>) + 15u) / 16u * 16u;
    l.total = l.bars + (2 * kShrinkA + 2 * kShrinkB + 1) * 8 + 16 + 1024;
    return l;
}
static_assert(sizeof(Groups<256>) <= kShrinkA * 2 * kBlock, "lists of 256 rows are made where the ring lies");

// order[starts[i] ..]: the rows of adapter i, ascending.  By a CTA: each warp
// takes a run of rows, twice.
__device__ __forceinline__ void sort_rows(const ShrinkArgs &a, int64_t mine, int *part) {
    constexpr int W = kShrinkThreads / 32, U = 8;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t per = ((a.M + W - 1) / W + 31) / 32 * 32, from = warp * per, to = min(from + per, a.M);
    int before = 0, here = 0;
    for (int64_t m = from + lane; m - lane < to; m += 32 * U) {
        int64_t id[U];
#pragma unroll
        for (int q = 0; q < U; ++q) id[q] = m + 32 * q < to ? a.ids[m + 32 * q] : -1;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            before += id[q] >= 0 && id[q] < mine ? 1 : 0;
            here += id[q] == mine ? 1 : 0;
        }
    }
    before = __reduce_add_sync(0xffffffffu, before);
    here = __reduce_add_sync(0xffffffffu, here);
    if (lane == 0) { part[warp] = before; part[W + warp] = here; }
    __syncthreads();
    int start = 0, at = 0, count = 0;
    for (int w = 0; w < W; ++w) {
        start += part[w];
        at += w < warp ? part[W + w] : 0;
        count += part[W + w];
    }
    if (threadIdx.x == 0 && CHK(mine, 1, a.n)) { a.counts[mine] = count; a.starts[mine] = start; }
    if (here == 0) return;                                // warp-uniform
    at += start;
    for (int64_t m = from + lane; m - lane < to; m += 32 * U) {
        int64_t id[U];
#pragma unroll
        for (int q = 0; q < U; ++q) id[q] = m + 32 * q < to ? a.ids[m + 32 * q] : -1;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const unsigned hit = __ballot_sync(0xffffffffu, id[q] == mine);
            const int to_at = at + __popc(hit & ((1u << lane) - 1u));
            if (id[q] == mine && CHK(to_at, 1, a.M)) a.order[to_at] = (int)(m + 32 * q);
            at += __popc(hit);
        }
    }
}

// Whole warps run the loops that issue loads and products, one lane issues: what
// these take then lives in uniform registers (one lane's loop took 600 cycles per
// load; 24 adapters in a tile: 20 us).
//
// rows [128 t, ..) of X times P_i, X [M][R]; P_i is A_i [R][r] or the transpose of
// B_i [r][R] (BWD).  The reduction's pieces depend on R alone and are added as a
// balanced tree, so a row's sum is the same however the cluster's CTAs share them.
// The CTAs of the first clusters make what later kernels need of the adapters'
// numbers.
template <bool BWD, bool F16>
__global__ void __launch_bounds__(kShrinkThreads)
lora_shrink_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_p, const ShrinkArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const ShrinkLayout l = shrink_layout(BWD, a.rp, a.stages_b);
    const uint32_t sbase = smem_addr(smem), bars = sbase + l.bars;
    auto a_full = [&](int s) { return bars + 8u * s; };
    auto a_empty = [&](int s) { return bars + 8u * (kShrinkA + s); };
    auto b_full = [&](int s) { return bars + 8u * (2 * kShrinkA + s); };
    auto b_empty = [&](int s) { return bars + 8u * (2 * kShrinkA + kShrinkB + s); };
    const uint32_t done = bars + 8u * (2 * kShrinkA + 2 * kShrinkB);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + l.bars + (2 * kShrinkA + 2 * kShrinkB + 1) * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    Groups<128> &g = *reinterpret_cast<Groups<128> *>(smem + l.groups);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int rank = a.cluster > 1 ? (int)cluster_rank() : 0, cluster = (int)blockIdx.x / a.cluster;
    if (cluster < a.extra) {                              // the whole cluster: nothing here waits for its other CTAs
        wait_prior_grid();
        allow_next_grid();
        const int64_t i = (int64_t)cluster * a.cluster + rank, sort = i - a.wide_tiles;
        if (i < a.wide_tiles) {
            Groups<256> &w = *reinterpret_cast<Groups<256> *>(smem);
            find_groups(w, a.ids, i * kPairRows, a.M, a.n, true);
            TileList &out = a.lists[i];
            if (threadIdx.x == 0) out.count = w.count;
            for (int e = threadIdx.x; e < w.count; e += kShrinkThreads) {
                out.e[e].adapter = w.adapter[e];
                for (int q = 0; q < 8; ++q) out.e[e].off[q] = w.off[e][q];
            }
        } else if (sort < a.sorted) {
            sort_rows(a, sort, reinterpret_cast<int *>(smem));
        }
        return;
    }
    const int wide = a.rp * a.each;                       // accumulators of this CTA's pieces
    const uint32_t cols = wide <= 32 ? 32u : wide <= 64 ? 64u : wide <= 128 ? 128u : 256u;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kShrinkA; ++s) { mbar_init(a_full(s), 1); mbar_init(a_empty(s), 1); }
        for (int s = 0; s < kShrinkB; ++s) { mbar_init(b_full(s), 1); mbar_init(b_empty(s), 1); }
        mbar_init(done, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_map(&map_x);
        prefetch_map(&map_p);
    }
    if (warp == 1) tmem_alloc(smem_addr(tmem_slot), cols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_prior_grid();
    allow_next_grid();

    const int subset = (cluster - a.extra) % a.subsets;
    const int64_t m0 = (int64_t)((cluster - a.extra) / a.subsets) * 128;
    const int share = a.each * a.per_piece, kb0 = min(rank * share, a.k_blocks), kb1 = min(kb0 + share, a.k_blocks);
    // the first rows are on their way while the adapters are looked up
    const int ahead = min(kb1 - kb0, kShrinkA);
    if (threadIdx.x == 0)
        for (int s = 0; s < ahead; ++s) {
            mbar_arrive_expect_tx(a_full(s), 2 * kBlock);
            tma_load_2d(sbase + s * 2 * kBlock, &map_x, a_full(s), (kb0 + s) * kBK, (int)m0);
        }
    __syncwarp();
    find_groups(g, a.ids, m0, a.M, a.n, false);
    const int part_of = (g.count + a.subsets - 1) / a.subsets;
    const int first = __shfl_sync(0xffffffffu, min(subset * part_of, g.count), 0);
    const int last = __shfl_sync(0xffffffffu, min(first + part_of, g.count), 0);
    const bool any = last > first && kb1 > kb0;
    // the rows this cluster makes: those of its adapters, and the first subset's also those without one
    auto has = [&](int row) {
        if (g.id[row] < 0) return subset == 0;
        const int place = g.place[g.first[row]];
        return place >= first && place < last;
    };

    if (warp == 0) {
        int sa = 0, sb = 0;
        uint32_t pa = 0, pb = 0;
        bool ok = any;
        for (int kb = kb0; ok && kb < kb1; ++kb) {
            if (kb - kb0 >= kShrinkA) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(a_empty(sa), pa ^ 1u, abort_flag)))) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(a_full(sa), 2 * kBlock);
                    tma_load_2d(sbase + sa * 2 * kBlock, &map_x, a_full(sa), kb * kBK, (int)m0);
                }
                __syncwarp();
            }
            if (++sa == kShrinkA) { sa = 0; pa ^= 1u; }
            for (int i = first; i < last; ++i) {
                const int adapter = __shfl_sync(0xffffffffu, g.adapter[i], 0);
                if (!(ok = __all_sync(0xffffffffu, wait_bar(b_empty(sb), pb ^ 1u, abort_flag)))) break;
                const uint32_t dst = sbase + l.b + sb * l.b_stage;
                if (elect_one()) {
                    mbar_arrive_expect_tx(b_full(sb), l.b_stage);
                    if (BWD) {
                        tma_load_3d(dst, &map_p, b_full(sb), kb * kBK, 0, adapter);
                    } else {
                        tma_load_3d(dst, &map_p, b_full(sb), 0, kb * kBK, adapter);
                        if (a.rp > 64) tma_load_3d(dst + kBlock, &map_p, b_full(sb), 64, kb * kBK, adapter);
                    }
                }
                __syncwarp();
                if (++sb == a.stages_b) { sb = 0; pb ^= 1u; }
            }
        }
        // Every load has landed before the ring is used again, and before the CTA
        // may exit: the first rows also where nothing is multiplied.
        if (!any) {
            for (int s = 0; s < ahead; ++s) mbar_wait(a_full(s), 0);
        } else {
            for (int i = 0; i < kShrinkA; ++i) {
                if (--sa < 0) { sa = kShrinkA - 1; pa ^= 1u; }
                if (!mbar_wait(a_full(sa), pa)) break;
            }
            for (int i = 0; i < a.stages_b; ++i) {
                if (--sb < 0) { sb = a.stages_b - 1; pb ^= 1u; }
                if (!mbar_wait(b_full(sb), pb)) break;
            }
        }
    } else if (warp == 1 && any) {
        const uint32_t idesc = instr_desc_single(a.rp, false, !BWD, F16);
        int sa = 0, sb = 0, in_piece = 0;
        uint32_t pa = 0, pb = 0, d = tmem;
        bool ok = true;
        for (int kb = kb0; ok && kb < kb1; ++kb) {
            if (!(ok = __all_sync(0xffffffffu, wait_bar(a_full(sa), pa, abort_flag)))) break;
            const uint32_t rows = sbase + sa * 2 * kBlock;
            for (int i = first; i < last; ++i) {
                uint32_t off[4];
#pragma unroll
                for (int w = 0; w < 4; ++w) off[w] = __shfl_sync(0xffffffffu, g.off[i][w], 0);
                if (!(ok = __all_sync(0xffffffffu, wait_bar(b_full(sb), pb, abort_flag)))) break;
                tc_fence_after();
                const uint32_t p = sbase + l.b + sb * l.b_stage;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        mma_masked(d, box_desc(rows, false, k), box_desc(p, !BWD, k), idesc, off,
                                   in_piece > 0 || k > 0 ? 1u : 0u);
                    mma_commit(b_empty(sb));
                }
                __syncwarp();
                if (++sb == a.stages_b) { sb = 0; pb ^= 1u; }
            }
            if (!ok) break;
            if (elect_one()) mma_commit(a_empty(sa));
            __syncwarp();
            if (++sa == kShrinkA) { sa = 0; pa ^= 1u; }
            if (++in_piece == a.per_piece) { in_piece = 0; d += (uint32_t)a.rp; }
        }
        if (ok && elect_one()) mma_commit(done);
        __syncwarp();
    }
    // the products are complete and the producer has seen its last load
    bool have = any;
    if (warp >= 2 && any) {
        have = wait_bar(done, 0, abort_flag);
        tc_fence_after();
    }
    __syncthreads();
    float *part = reinterpret_cast<float *>(smem);
    const int pitch = a.rp + 4;
    if (warp >= 2) {
        const int quarter = warp % 4, row = quarter * 32 + lane;
        const bool mine = have && g.id[row] >= 0 && has(row);
        const int filled = (kb1 - kb0 + a.per_piece - 1) / a.per_piece;       // pieces that hold something
        const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16);
        for (int c = 0; c < a.rp; c += 16) {
            // pieces 2 j and 2 j + 1, and so on: the tree's levels within this CTA
            float sum[3][16];
            for (int q = 0; q < a.each; ++q) {
                uint32_t v[16];
                if (have && q < filled) tmem_ld16(from + (uint32_t)(q * a.rp + c), v);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float f = mine && q < filled ? __uint_as_float(v[i]) : 0.0f;
                    if ((q & 1) == 0) {
                        sum[0][i] = f;
                    } else {
                        f = sum[0][i] + f;
                        if ((q & 2) == 0) {
                            sum[1][i] = f;
                        } else {
                            f = sum[1][i] + f;
                            if ((q & 4) == 0) sum[2][i] = f;
                            else sum[0][i] = sum[2][i] + f;
                        }
                    }
                }
            }
            const int level = a.each == 2 ? 1 : a.each == 4 ? 2 : 0;          // 8: back in 0
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                float f[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] = level == 0 ? sum[0][i + k] : level == 1 ? sum[1][i + k] : sum[2][i + k];
                *reinterpret_cast<float4 *>(part + row * pitch + c + i) = make_float4(f[0], f[1], f[2], f[3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                   // every piece is in its CTA's shared memory

    // this CTA's share of the rows: the rest of the tree, the scale, the terms
    const int rows = 128 / a.cluster, vecs = a.rp / 4;
    uint16_t *u = static_cast<uint16_t *>(a.u);
    for (int i = threadIdx.x; i < rows * vecs; i += kShrinkThreads) {
        const int row = rank * rows + i / vecs, c = i % vecs * 4;
        if (m0 + row >= a.M || !has(row)) continue;
        const uint32_t mine = smem_addr(part + row * pitch + c);
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
            v[q] = q >= a.cluster ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                 : a.cluster > 1 ? ld_cluster_f4(mine, (uint32_t)q) : *reinterpret_cast<const float4 *>(part + row * pitch + c);
#pragma unroll
        for (int step = 1; step < 8; step *= 2)
#pragma unroll
            for (int q = 0; q < 8; q += 2 * step)         // beyond the cluster's CTAs nothing changes
                if (q + step < a.cluster)
                    v[q] = make_float4(v[q].x + v[q + step].x, v[q].y + v[q + step].y, v[q].z + v[q + step].z, v[q].w + v[q + step].w);
        const float4 s = v[0];
        const int id = g.id[row];
        const bool live = id >= 0 && c < a.r;             // what pads the rank is zero, not infinity times zero
        const float scale = live ? a.scales[id] : 0.0f;
        const float w[4] = {s.x * scale, s.y * scale, s.z * scale, s.w * scale};
        float hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float v = live ? w[k] : 0.0f;
            hi[k] = F16 ? __half2float(__float2half_rn(v)) : __bfloat162float(__float2bfloat16_rn(v));
            lo[k] = fabsf(hi[k]) < INFINITY ? v - hi[k] : 0.0f;
        }
        const int64_t at = ((m0 + row) * kPlanes) * a.rp + c;
        if (!CHK(at, 2 * a.rp + 4, a.M * kPlanes * a.rp)) continue;
        *reinterpret_cast<uint2 *>(u + at) = make_uint2(pack2<F16>(hi[0], hi[1]), pack2<F16>(hi[2], hi[3]));
        *reinterpret_cast<uint2 *>(u + at + a.rp) = make_uint2(pack2<F16>(lo[0], lo[1]), pack2<F16>(lo[2], lo[3]));
        *reinterpret_cast<uint2 *>(u + at + 2 * a.rp) =
            make_uint2(pack2<F16>(lo[0] * kLoScale, lo[1] * kLoScale), pack2<F16>(lo[2] * kLoScale, lo[3] * kLoScale));
    }
    cluster_sync_all();                                   // the others have read this CTA's piece
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, cols);
    }
}

// ---- y and dx ---------------------------------------------------------------------------

struct LayerArgs {
    const TileList *lists;
    const void *bias;                    // [cols] or null
    int64_t M, cols;
    int rp, k_blocks;
    int bn, tiles_n, tiles;
    int batch;                           // adapters per stage
};

constexpr int kEpiWarps = 8;
constexpr int kLayerThreads = 32 * (4 + kEpiWarps);
constexpr uint32_t kStageBytes = 4 * kBlock;          // 128 rows of A, and 128 columns of B

// UB: blocks of 128 rows x 64 that hold a CTA's rows of hi and lo.
template <int UB>
struct LayerSmem {
    static constexpr int kStages = UB <= 1 ? 5 : UB == 2 ? 4 : 3;
    static constexpr uint32_t kU = kStages * kStageBytes;
    static constexpr uint32_t kStaging = kU + UB * 2 * kBlock;
    static constexpr uint32_t kBias = kStaging + kEpiWarps * 4096;
    static constexpr uint32_t kBars = kBias + kEpiWarps * 256;
    static constexpr uint32_t kBytes = kBars + (2 * kStages + 6) * 8 + 16 + 1024;
    static_assert(kBytes <= 232448, "shared memory per block");
};

// A tile's adapters in a warp: lane e holds entry e0 + e of the list (off only
// where OFF).
template <bool OFF>
struct Entries {
    int count, adapter;
    uint32_t off[8];
    __device__ void load(const TileList &list, int e0) {
        const TileEntry &e = list.e[e0 + threadIdx.x % 32];       // of 256 places, whatever the count
        count = __ldcg(&list.count);
        adapter = __ldcg(&e.adapter);
        if (OFF) {
            const uint4 lo = __ldcg(reinterpret_cast<const uint4 *>(e.off)), hi = __ldcg(reinterpret_cast<const uint4 *>(e.off) + 1);
            off[0] = lo.x; off[1] = lo.y; off[2] = lo.z; off[3] = lo.w;
            off[4] = hi.x; off[5] = hi.y; off[6] = hi.z; off[7] = hi.w;
        }
    }
};

// The adapters in batches of G (a power of two up to 32), for a whole warp:
// f(n, at) for n adapters that lanes at .. at + n - 1 hold.  false: f gave up.
template <bool OFF, typename F>
__device__ __forceinline__ bool each_batch(const TileList &list, Entries<OFF> &e, int G, F f) {
    for (int e0 = 0; e0 < e.count; e0 += 32) {
        if (e0 > 0) e.load(list, e0);
        for (int at = 0; at < 32 && e0 + at < e.count; at += G)
            if (!f(min(G, e.count - e0 - at), at)) return false;
    }
    return true;
}

// X [M][R] times W [R][cols] (or the transpose of W [cols][R], BWD), plus the
// adapters' terms; the pair's tile is 256 rows x bn columns, each CTA loads its
// own rows of A and half the columns of B.
template <bool BWD, bool F16, int UB>
__global__ void __launch_bounds__(kLayerThreads, 1) __cluster_dims__(2, 1, 1)
lora_layer_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ CUtensorMap map_u, const __grid_constant__ CUtensorMap map_p,
                  const __grid_constant__ CUtensorMap map_out, const LayerArgs a) {
    using L = LayerSmem<UB>;
    constexpr int kStages = L::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_addr(smem), bars = sbase + L::kBars;
    auto full = [&](int s) { return bars + 8u * s; };                           // used in CTA 0
    auto empty = [&](int s) { return bars + 8u * (kStages + s); };
    auto tfull = [&](int b) { return bars + 8u * (2 * kStages + b); };
    auto tempty = [&](int b) { return bars + 8u * (2 * kStages + 2 + b); };      // used in CTA 0
    const uint32_t ufull = bars + 8u * (2 * kStages + 4), uempty = ufull + 8u;    // ufull: used in CTA 0
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + L::kBars + (2 * kStages + 6) * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    const uint32_t rank = cluster_rank();
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) { mbar_init(full(s), 1); mbar_init(empty(s), 1); }
        for (int b = 0; b < 2; ++b) { mbar_init(tfull(b), 1); mbar_init(tempty(b), 2 * kEpiWarps); }
        mbar_init(ufull, 1);
        mbar_init(uempty, 1);
        *abort_flag = 0u;
        fence_mbar_init();
        prefetch_map(&map_x);
        prefetch_map(&map_w);
    }
    if (warp == 1) tmem_alloc_pair(smem_addr(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                   // both CTAs' barriers are set up
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The layer's own operands are older than the kernel before this one, which
    // let this one start only after its own wait: they may be read now.  What it
    // makes, u and the lists, is waited for where it is first read.
    allow_next_grid();
    const int pair = (int)blockIdx.x / 2, pairs = (int)gridDim.x / 2;
    const int half = a.bn / 2;
    // an adapter's part of a stage: 64 of the columns, or (BWD) of the rank, each
    const uint32_t low_blocks = BWD ? (a.rp > 64 ? 2u : 1u) : (uint32_t)(half + 63) / 64u;
    const uint32_t low_block = BWD ? (uint32_t)half * 128u : (uint32_t)a.rp * 128u;

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 0, uph = 0;
        bool ok = true, waited = false;
        Entries<false> entries;
        auto next = [&] { if (++s == kStages) { s = 0; ph ^= 1u; } };
        for (int t = pair; ok && t < a.tiles && *abort_flag == 0u; t += pairs) {
            const int64_t m0 = (int64_t)(t / a.tiles_n) * kPairRows;
            const int rows = (int)(m0 + rank * 128), n0 = t % a.tiles_n * a.bn + (int)rank * half;
            const bool second = m0 + 128 < a.M;           // CTA 1 has rows (else none are loaded: nothing reads what the MMA makes of them)
            const bool load_a = rank == 0 || second;
            const uint32_t b_bytes = BWD ? (uint32_t)half * 128u : (uint32_t)(half + 63) / 64u * kBlock;
            const uint32_t bytes = (second ? 2u : 1u) * 2u * kBlock + 2u * b_bytes;
            const TileList &list = a.lists[t / a.tiles_n];
            bool have_u = false;
            auto load_u = [&] {                           // this CTA's rows of u
                have_u = true;
                if (entries.count == 0) return true;
                if (!__all_sync(0xffffffffu, wait_bar(uempty, uph ^ 1u, abort_flag))) return false;
                uph ^= 1u;
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(ufull, (second ? 2u : 1u) * UB * 2u * kBlock);
                    for (int q = 0; q < UB && load_a; ++q)
                        tma_load_pair(sbase + L::kU + q * 2 * kBlock, &map_u, map_rank(ufull, 0), q * 64, rows);
                }
                __syncwarp();
                return true;
            };
            // the list is on its way during the k-blocks; u follows when the last
            // tile's products are done with its place
            if (waited) entries.load(list, 0);
            for (int kb = 0; kb < a.k_blocks; ++kb) {
                if (waited && kb == kStages && !(ok = load_u())) break;
                if (!(ok = __all_sync(0xffffffffu, wait_bar(empty(s), ph ^ 1u, abort_flag)))) break;
                const uint32_t sa = sbase + s * kStageBytes, sb = sa + 2 * kBlock, bar = map_rank(full(s), 0);
                if (elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
                    if (load_a) tma_load_pair(sa, &map_x, bar, kb * kBK, rows);
                    if (BWD) {
                        tma_load_pair(sb, &map_w, bar, kb * kBK, n0);
                    } else {
                        tma_load_pair(sb, &map_w, bar, n0, kb * kBK);
                        if (half > 64) tma_load_pair(sb + kBlock, &map_w, bar, n0 + 64, kb * kBK);
                    }
                }
                __syncwarp();
                next();
            }
            if (!ok) break;
            if (!waited) {
                wait_prior_grid();
                waited = true;
                entries.load(list, 0);
            }
            if (!have_u && !(ok = load_u())) break;
            ok = each_batch<false>(list, entries, a.batch, [&](int n, int at) {
                if (!__all_sync(0xffffffffu, wait_bar(empty(s), ph ^ 1u, abort_flag))) return false;
                const uint32_t bar = map_rank(full(s), 0);
                if (rank == 0 && elect_one()) mbar_arrive_expect_tx(full(s), 2u * (uint32_t)n * low_blocks * low_block);
                for (int i = 0; i < n; ++i) {
                    const int adapter = __shfl_sync(0xffffffffu, entries.adapter, at + i);
                    const uint32_t sb = sbase + s * kStageBytes + (uint32_t)i * low_blocks * low_block;
                    if (elect_one())
                        for (uint32_t q = 0; q < low_blocks; ++q) {
                            if (BWD) tma_load_pair_3d(sb + q * low_block, &map_p, bar, (int)q * 64, n0, adapter);
                            else tma_load_pair_3d(sb + q * low_block, &map_p, bar, n0 + (int)q * 64, 0, adapter);
                        }
                }
                __syncwarp();
                next();
                return true;
            });
        }
        if (!waited) wait_prior_grid();
        // CTA 0 sees every load of both land before the pair may exit
        for (int i = 0; rank == 0 && i < kStages; ++i) {
            if (--s < 0) { s = kStages - 1; ph ^= 1u; }
            if (!__all_sync(0xffffffffu, mbar_wait(full(s), ph))) break;
        }
        if (rank == 0) mbar_wait(ufull, uph ^ 1u);
    } else if (warp == 1 && rank == 0) {
        int s = 0, acc = 0;
        uint32_t ph = 0, aph = 0, uph = 0;
        bool ok = true, waited = false;
        Entries<true> entries;
        const uint32_t idesc = instr_desc(a.bn, false, !BWD, F16);
        for (int t = pair; ok && t < a.tiles && *abort_flag == 0u; t += pairs) {
            if (!(ok = __all_sync(0xffffffffu, wait_bar(tempty(acc), aph ^ 1u, abort_flag)))) break;
            tc_fence_after();
            const uint32_t d = tmem + (uint32_t)(acc * 256);
            const TileList &list = a.lists[t / a.tiles_n];
            if (waited) entries.load(list, 0);
            for (int kb = 0; kb < a.k_blocks; ++kb) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(full(s), ph, abort_flag)))) break;
                tc_fence_after();
                const uint32_t sa = sbase + s * kStageBytes, sb = sa + 2 * kBlock;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        mma_pair(d, box_desc(sa, false, k), box_desc(sb, !BWD, k), idesc, (kb | k) != 0 ? 1u : 0u);
                    mma_commit_pair(empty(s));
                }
                __syncwarp();
                if (++s == kStages) { s = 0; ph ^= 1u; }
            }
            if (!ok) break;
            if (!waited) {
                wait_prior_grid();
                waited = true;
                entries.load(list, 0);
            }
            if (entries.count > 0) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(ufull, uph, abort_flag)))) break;
                uph ^= 1u;
                ok = each_batch<true>(list, entries, a.batch, [&](int n, int at) {
                    if (!__all_sync(0xffffffffu, wait_bar(full(s), ph, abort_flag))) return false;
                    tc_fence_after();
                    for (int i = 0; i < n; ++i) {
                        uint32_t skip[8];
#pragma unroll
                        for (int w = 0; w < 8; ++w) skip[w] = __shfl_sync(0xffffffffu, entries.off[w], at + i);
                        const uint32_t sb = sbase + s * kStageBytes + (uint32_t)i * low_blocks * low_block;
                        if (elect_one())
                            for (int j = 0; j < a.rp / 16; ++j) {
                                const uint64_t b = BWD ? smem_desc(sb + (uint32_t)(j / 4) * low_block + (uint32_t)(j % 4) * 32u, 16u, 1024u)
                                                       : smem_desc(sb + (uint32_t)j * 2048u, low_block, 1024u);
#pragma unroll
                                for (int plane = 0; plane < 2; ++plane) {       // hi, lo
                                    const uint32_t c = (uint32_t)(plane * a.rp + j * 16);
                                    mma_pair_masked(d, smem_desc(sbase + L::kU + c / 64u * 2u * kBlock + c % 64u * 2u, 16u, 1024u), b, idesc, skip);
                                }
                            }
                        __syncwarp();
                    }
                    if (elect_one()) mma_commit_pair(empty(s));
                    __syncwarp();
                    if (++s == kStages) { s = 0; ph ^= 1u; }
                    return true;
                });
                if (!ok) break;
                if (elect_one()) mma_commit_pair(uempty);
                __syncwarp();
            }
            if (elect_one()) mma_commit_pair(tfull(acc));
            __syncwarp();
            if (++acc == 2) { acc = 0; aph ^= 1u; }
        }
        if (!waited) wait_prior_grid();
    } else if (warp >= 4) {
        const int quarter = warp % 4, part = (warp - 4) / 4;
        const uint32_t stg = sbase + L::kStaging + (uint32_t)(warp - 4) * 4096u;
        float *bias = reinterpret_cast<float *>(smem + L::kBias) + (warp - 4) * 64;
        int acc = 0;
        uint32_t aph = 0;
        for (int t = pair; t < a.tiles && *abort_flag == 0u; t += pairs) {
            const int64_t row0 = (int64_t)(t / a.tiles_n) * kPairRows + rank * 128 + quarter * 32;
            const int n0 = t % a.tiles_n * a.bn;
            if (!__all_sync(0xffffffffu, wait_bar(tfull(acc), aph, abort_flag))) break;
            tc_fence_after();
            const uint32_t from = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * 256);
#pragma unroll 1
            for (int c = part * 64; c < a.bn && n0 + c < a.cols && row0 < a.M; c += 128) {
                uint32_t r[64], o[32];
                tmem_ld64(from + (uint32_t)c, r);
                if (a.bias) {
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 64; q += 32) {
                        const int64_t col = n0 + c + q + lane;
                        const uint16_t v = col < a.cols && CHK(col, 1, a.cols) ? static_cast<const uint16_t *>(a.bias)[col] : 0;
                        bias[q + lane] = F16 ? __half2float(__ushort_as_half(v)) : __uint_as_float((uint32_t)v << 16);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        const float4 b = *reinterpret_cast<const float4 *>(bias + i);
                        r[i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), b.x));
                        r[i + 1] = __float_as_uint(__fadd_rn(__uint_as_float(r[i + 1]), b.y));
                        r[i + 2] = __float_as_uint(__fadd_rn(__uint_as_float(r[i + 2]), b.z));
                        r[i + 3] = __float_as_uint(__fadd_rn(__uint_as_float(r[i + 3]), b.w));
                    }
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = pack2<F16>(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                put_rows(stg, lane, &map_out, o, n0 + c, (int)row0, false);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(tempty(acc), 0));
            if (++acc == 2) { acc = 0; aph ^= 1u; }
        }
        if (elect_one()) bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                                   // no arrival at, or MMA into, a CTA that has left
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
    cluster_sync_all();
}

// ---- dA and dB ---------------------------------------------------------------------------

struct GradArgs {
    const uint16_t *x, *dy;              // [M][K], [M][N]
    const uint16_t *u, *du;              // [M][kPlanes][rp]
    const int *order, *counts, *starts;
    uint16_t *da, *db;                   // [n][K][r], [n][r][N]
    float *parts;                        // [slots][column tiles][rp][128]
    int64_t M, K, N, n;
    int64_t slots;
    int r, rp;
    int tiles_k, tiles;                  // column tiles of dA, of both
};

// A warp finds piece q: its adapter, its place among the adapter's pieces, how
// many these are, and its slot among the pieces of adapters with several.
struct Piece {
    int adapter, j, of, slot;            // adapter -1: there are fewer pieces
};
__device__ __forceinline__ Piece find_piece(const int *counts, int64_t n, int64_t q) {
    const int lane = threadIdx.x % 32;
    int64_t before = 0, slots = 0;
    for (int64_t i0 = 0; i0 < n; i0 += 32) {
        const int c = i0 + lane < n ? (counts[i0 + lane] + kPiece - 1) / kPiece : 0;
        int all = c, several = c > 1 ? c : 0;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, all, o), w = __shfl_up_sync(0xffffffffu, several, o);
            if (lane >= o) { all += v; several += w; }
        }
        const unsigned hit = __ballot_sync(0xffffffffu, q < before + all);
        if (hit != 0u) {
            const int at = __ffs((int)hit) - 1;
            const int of = __shfl_sync(0xffffffffu, c, at);
            const int j = (int)(q - before) - (__shfl_sync(0xffffffffu, all, at) - of);
            const int s = __shfl_sync(0xffffffffu, several, at);
            return Piece{(int)i0 + at, j, of, (int)(slots + s - (of > 1 ? of : 0)) + j};
        }
        before += __shfl_sync(0xffffffffu, all, 31);
        slots += __shfl_sync(0xffffffffu, several, 31);
    }
    return Piece{-1, 0, 0, 0};
}

constexpr int kGradThreads = 160;        // four warps that load and store, the MMA issuer

struct GradLayout {
    uint32_t plane, stage, bars, total;
};
__host__ __device__ inline GradLayout grad_layout(int rp, int stages) {
    GradLayout l;
    l.plane = (rp > 64 ? 2u : 1u) * kBlock;
    l.stage = 2 * kBlock + 2 * l.plane;
    l.bars = (uint32_t)stages * l.stage;
    l.total = l.bars + (2 * stages + 1) * 8 + 16 + sizeof(Piece) + 1024;
    return l;
}

// Bytes that a barrier's phase waits for, without an arrival.
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// 16 bytes, or zeros where there is nothing to read.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// STAGES: as many as leave room for two CTAs on an SM.
template <bool F16, int STAGES>
__global__ void __launch_bounds__(kGradThreads)
lora_grads_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy,
                  const __grid_constant__ CUtensorMap map_u, const __grid_constant__ CUtensorMap map_du, const GradArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const GradLayout l = grad_layout(a.rp, STAGES);
    const uint32_t sbase = smem_addr(smem), bars = sbase + l.bars;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (STAGES + s); };
    const uint32_t done = bars + 8u * (2 * STAGES);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + l.bars + (2 * STAGES + 1) * 8);
    volatile uint32_t *abort_flag = tmem_slot + 1;
    Piece *shared_piece = reinterpret_cast<Piece *>(tmem_slot + 2);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t cols = a.rp <= 16 ? 32u : a.rp <= 32 ? 64u : a.rp <= 64 ? 128u : 256u;      // both terms' accumulators
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(full(s), 128); mbar_init(empty(s), 1); }
        mbar_init(done, 1);
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 4) tmem_alloc(smem_addr(tmem_slot), cols);
    tc_fence_before();
    wait_prior_grid();
    allow_next_grid();
    if (warp == 0) {
        const Piece p = find_piece(a.counts, a.n, blockIdx.x);
        if (lane == 0) *shared_piece = p;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const Piece piece = *shared_piece;
    const bool is_a = (int)blockIdx.y < a.tiles_k;
    const int64_t width = is_a ? a.K : a.N, c0 = (int64_t)((int)blockIdx.y - (is_a ? 0 : a.tiles_k)) * 128;

    if (piece.adapter >= 0) {                             // CTA-uniform
        const int count = min(kPiece, a.counts[piece.adapter] - piece.j * kPiece), blocks = (count + 63) / 64;
        const int *rows = a.order + a.starts[piece.adapter] + piece.j * kPiece;
        if (warp < 4) {
            const uint16_t *src = is_a ? a.x : a.dy, *planes = is_a ? a.du : a.u;
            const int q = threadIdx.x / 2, h = threadIdx.x % 2;       // a row of the block; half of its columns, one of its terms
            const uint32_t line = (uint32_t)q * 128u;
            int s = 0, sent = 0, sent_s = 0;
            uint32_t ph = 0;
            bool ok = true;
            // a block's row of this thread, and whether its 64 rows follow each other
            auto row_of = [&](int b, bool *run) {
                const int at = b * 64;
                *run = at + 64 <= count && rows[at + 63] == rows[at] + 63;
                return at + q < count ? rows[at + q] : -1;
            };
            bool run;
            int m = row_of(0, &run);
            int issued = 0;
            for (int b = 0; ok && b < blocks; ++b) {
                bool next_run = false;
                const int next = b + 1 < blocks ? row_of(b + 1, &next_run) : -1;
                if (!(ok = wait_bar(empty(s), ph ^ 1u, abort_flag))) break;
                const uint32_t to = sbase + s * l.stage;
                if (run) {                                // by bulk copies
                    if (threadIdx.x == 0) {
                        const CUtensorMap *rows_map = is_a ? &map_x : &map_dy, *low_map = is_a ? &map_du : &map_u;
                        const uint32_t lows = a.rp > 64 ? 2u : 1u;
                        mbar_expect_tx(full(s), 2 * kBlock + 2 * l.plane);
                        tma_load_2d(to, rows_map, full(s), (int)c0, m);
                        tma_load_2d(to + kBlock, rows_map, full(s), (int)c0 + 64, m);
                        for (uint32_t p = 0; p < lows; ++p) {
                            tma_load_2d(to + 2 * kBlock + p * kBlock, low_map, full(s), (int)p * 64, m);
                            tma_load_2d(to + 2 * kBlock + l.plane + p * kBlock, low_map, full(s), 2 * a.rp + (int)p * 64, m);
                        }
                    }
                } else {
                    const bool live = m >= 0 && CHK(m, 1, a.M);
                    const uint16_t *x = src + (live ? (int64_t)m * width : 0);
#pragma unroll
                    for (int p = 0; p < 8; ++p) {
                        const int64_t c = c0 + h * 64 + p * 8;
                        const bool there = live && c < width;
                        copy16(to + h * kBlock + line + (uint32_t)((p ^ (q & 7)) * 16), there ? x + c : src, there);
                    }
                    const uint16_t *u = planes + ((live ? (int64_t)m * kPlanes : 0) + h * 2) * a.rp;      // hi, lo 2^11
                    for (int p = 0; p < a.rp / 8; ++p)
                        copy16(to + 2 * kBlock + h * l.plane + (uint32_t)(p / 8) * kBlock + line + (uint32_t)((p % 8 ^ (q & 7)) * 16),
                               u + p * 8, live);
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                ++issued;
                m = next;
                run = next_run;
                if (++s == STAGES) { s = 0; ph ^= 1u; }
                if (b - sent == STAGES - 1) {
                    copies_wait<STAGES - 1>();
                    fence_proxy_async_smem();             // the tensor cores read what this thread's copies wrote
                    mbar_arrive(full(sent_s));
                    ++sent;
                    if (++sent_s == STAGES) sent_s = 0;
                }
            }
            copies_wait<0>();
            fence_proxy_async_smem();
            for (; sent < issued; ++sent) {
                mbar_arrive(full(sent_s));
                if (++sent_s == STAGES) sent_s = 0;
            }
            // after giving up: no bulk copy into a CTA that has left
            for (int i = 0; !ok && i < STAGES && i < issued; ++i) {
                if (--s < 0) { s = STAGES - 1; ph ^= 1u; }
                if (!mbar_wait(full(s), ph)) break;
            }
        } else {
            const uint32_t idesc = instr_desc_single(a.rp, true, true, F16);
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int b = 0; b < blocks; ++b) {
                if (!(ok = __all_sync(0xffffffffu, wait_bar(full(s), ph, abort_flag)))) break;
                tc_fence_after();
                const uint32_t x = sbase + s * l.stage, u = x + 2 * kBlock;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            mma_bf16(tmem + (uint32_t)(term * a.rp), box_desc(x, true, k), box_desc(u + term * l.plane, true, k),
                                     idesc, (b | k) != 0 ? 1u : 0u);
                    mma_commit(empty(s));
                }
                __syncwarp();
                if (++s == STAGES) { s = 0; ph ^= 1u; }
            }
            if (ok && elect_one()) mma_commit(done);
        }
        __syncwarp();
        if (warp < 4 && wait_bar(done, 0, abort_flag)) {
            tc_fence_after();
            const int64_t c = c0 + warp * 32 + lane;
            const uint32_t from = tmem + ((uint32_t)(warp * 32) << 16);
            for (int j = 0; j < a.rp; j += 16) {
                uint32_t v[16], w[16];
                tmem_ld16(from + (uint32_t)j, v);
                tmem_ld16(from + (uint32_t)(a.rp + j), w);
                float f[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] = fmaf(__uint_as_float(w[i]), 1.0f / kLoScale, __uint_as_float(v[i]));
                if (piece.of > 1) {
                    const int64_t at = (((int64_t)piece.slot * a.tiles + blockIdx.y) * a.rp + j) * 128 + warp * 32 + lane;
                    if (CHK(at, 15 * 128 + 1, a.slots * a.tiles * a.rp * 128))
#pragma unroll
                        for (int i = 0; i < 16; ++i) a.parts[at + i * 128] = f[i];
                } else if (is_a && c < width) {
#pragma unroll
                    for (int i = 0; i < 16; i += 8)
                        if (j + i < a.r && CHK((piece.adapter * a.K + c) * a.r + j + i, 8, a.n * a.K * a.r))
                            *reinterpret_cast<uint4 *>(a.da + (piece.adapter * a.K + c) * a.r + j + i) =
                                make_uint4(pack2<F16>(f[i], f[i + 1]), pack2<F16>(f[i + 2], f[i + 3]),
                                           pack2<F16>(f[i + 4], f[i + 5]), pack2<F16>(f[i + 6], f[i + 7]));
                } else if (c < width) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (j + i < a.r && CHK(((int64_t)piece.adapter * a.r + j + i) * a.N + c, 1, a.n * a.N * a.r))
                            a.db[((int64_t)piece.adapter * a.r + j + i) * a.N + c] = (uint16_t)pack2<F16>(f[i], 0.0f);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        tc_fence_after();
        tmem_dealloc(tmem, cols);
    }
}

// Adapters with several pieces: their sums in order, rounded.  Adapters without
// rows: zeros.
template <bool F16>
__global__ void __launch_bounds__(256)
lora_join_kernel(const GradArgs a) {
    __shared__ int first_slot;
    wait_prior_grid();
    allow_next_grid();
    const int64_t adapter = blockIdx.x;
    const int of = (a.counts[adapter] + kPiece - 1) / kPiece;
    if (of == 1) return;
    if (of > 1 && threadIdx.x < 32) {
        int s = 0;
        for (int64_t i = threadIdx.x; i < adapter; i += 32) {
            const int c = (a.counts[i] + kPiece - 1) / kPiece;
            s += c > 1 ? c : 0;
        }
        s = __reduce_add_sync(0xffffffffu, s);
        if (threadIdx.x == 0) first_slot = s;
    }
    __syncthreads();
    const int tile = (int)blockIdx.y;
    const bool is_a = tile < a.tiles_k;
    const int64_t width = is_a ? a.K : a.N, c0 = (int64_t)(tile - (is_a ? 0 : a.tiles_k)) * 128;
    const int64_t stride = (int64_t)a.tiles * a.rp * 128;
    // four columns of the tile at one place of the rank
    const int i = ((int)blockIdx.z * 256 + (int)threadIdx.x) * 4, j = i / 128;
    const int64_t c = c0 + i % 128;
    if (j >= a.r || c >= width) return;                   // widths are multiples of 8
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (of > 1) {
        const int64_t at = ((int64_t)first_slot * a.tiles + tile) * a.rp * 128 + i;
#pragma unroll 8
        for (int q = 0; q < of; ++q) {
            if (!CHK(at + q * stride, 4, a.slots * stride)) continue;
            const float4 v = *reinterpret_cast<const float4 *>(a.parts + at + q * stride);
            f = q == 0 ? v : make_float4(f.x + v.x, f.y + v.y, f.z + v.z, f.w + v.w);
        }
    }
    const uint32_t lo = pack2<F16>(f.x, f.y), hi = pack2<F16>(f.z, f.w);
    if (is_a) {
        uint16_t *to = a.da + (adapter * a.K + c) * a.r + j;
        if (!CHK(to - a.da, 3 * a.r + 1, a.n * a.K * a.r)) return;
        to[0] = (uint16_t)lo;
        to[a.r] = (uint16_t)(lo >> 16);
        to[2 * a.r] = (uint16_t)hi;
        to[3 * a.r] = (uint16_t)(hi >> 16);
    } else if (CHK((adapter * a.r + j) * a.N + c, 4, a.n * a.N * a.r)) {
        *reinterpret_cast<uint2 *>(a.db + (adapter * a.r + j) * a.N + c) = make_uint2(lo, hi);
    }
}

// ---- host side ------------------------------------------------------------------------

struct Sizes {
    int64_t M, K, N, n, r;
    int rp() const { return (int)((r + 15) / 16 * 16); }
};

int64_t up128(int64_t v) { return (v + 127) / 128 * 128; }

bool sizes_ok(const Sizes &z) {
    int64_t t;
    return z.M >= 0 && z.K > 0 && z.N > 0 && z.n > 0 && z.r > 0 && z.M < (1ll << 30) && z.K <= (1ll << 21) && z.N <= (1ll << 21) &&
           z.n < (1ll << 24) && z.r <= kMaxRank &&
           // tiles of a row of tiles, and of all
           !__builtin_mul_overflow(z.M / kPairRows + 1, z.N / 128 + z.K / 128 + 2, &t) && t < (1ll << 31) &&
           !__builtin_mul_overflow(z.n * z.r, z.K + z.N, &t) && t < (1ll << 46);
}

struct Work {
    TileList *lists;
    uint16_t *du;
    int *order, *counts, *starts;
    float *parts;
    int64_t slots, bytes;
};

Work plan_work(void *ws, const Sizes &z, bool bwd, bool grads) {
    Work w = {};
    char *base = static_cast<char *>(ws);
    auto take = [&](int64_t bytes) {
        char *q = base + w.bytes;
        w.bytes += up128(bytes);
        return q;
    };
    w.lists = reinterpret_cast<TileList *>(take((int64_t)sizeof(TileList) * ((z.M + kPairRows - 1) / kPairRows)));
    if (bwd) w.du = reinterpret_cast<uint16_t *>(take(2 * z.M * kPlanes * z.rp()));
    if (grads) {
        w.order = reinterpret_cast<int *>(take(4 * z.M));
        w.counts = reinterpret_cast<int *>(take(4 * z.n));
        w.starts = reinterpret_cast<int *>(take(4 * z.n));
        // an adapter with more than a piece has fewer than twice its rows' worth
        w.slots = 2 * z.M / kPiece;
        w.parts = reinterpret_cast<float *>(take(4 * w.slots * (up128(z.K) + up128(z.N)) * z.rp()));
    }
    return w;
}

cudaError_t encode(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, int box_inner, int box_outer) {
    return encode_tensor_map_2d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, (uint64_t)inner, (uint64_t)outer,
                                (uint64_t)inner * 2, (uint32_t)box_inner, (uint32_t)box_outer, CU_TENSOR_MAP_SWIZZLE_128B);
}
// A stack of matrices; a box lies in one of them, zeros past its edges.
cudaError_t encode_stack(CUtensorMap *m, const void *base, int64_t inner, int64_t outer, int64_t n, int box_outer) {
    const uint64_t extent[3] = {(uint64_t)inner, (uint64_t)outer, (uint64_t)n};
    const uint64_t stride[2] = {(uint64_t)inner * 2, (uint64_t)(inner * outer) * 2};
    const uint32_t box[3] = {64, (uint32_t)box_outer, 1};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, 3, extent, stride, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// u (x and A) or du (dy and B).
template <bool BWD>
cudaError_t launch_shrink(const Sizes &z, bool f16, const void *rows, const void *stack, const int64_t *ids, const float *scales,
                          void *u, const Work &k, bool sort, cudaStream_t s) {
    const int64_t R = BWD ? z.N : z.K;
    CUtensorMap mx, mp;
    cudaError_t err = encode(&mx, rows, R, z.M, 64, 128);
    if (err == cudaSuccess)
        err = BWD ? encode_stack(&mp, stack, z.N, z.r, z.n, z.rp()) : encode_stack(&mp, stack, z.r, z.K, z.n, 64);
    if (err != cudaSuccess) return err;
    ShrinkArgs a = {};
    a.ids = ids; a.scales = scales; a.u = u; a.lists = k.lists;
    a.M = z.M; a.n = z.n; a.r = (int)z.r; a.rp = z.rp();
    a.k_blocks = (int)((R + kBK - 1) / kBK);
    // pieces by the reduction's length alone, so that a row's sum does not depend
    // on the number of rows
    a.pieces = a.k_blocks > 8 ? 8 : a.k_blocks > 4 ? 4 : a.k_blocks > 2 ? 2 : 1;
    a.per_piece = (a.k_blocks + a.pieces - 1) / a.pieces;
    const int64_t tiles = (z.M + 127) / 128;
    // as many CTAs as run at once, two per SM (kShrinkSmem); the accumulators of
    // both fit, so that CTAs of a cluster on one SM never wait for each other's
    a.cluster = a.pieces;
    while (a.cluster > 1 && tiles * a.cluster > 256 && a.pieces / (a.cluster / 2) * a.rp <= 256) a.cluster /= 2;
    a.each = a.pieces / a.cluster;
    // where that leaves CTAs idle, a tile of many adapters goes to several clusters
    const int64_t idle = 152 / (tiles * a.cluster), adapters = z.n < 128 ? z.n : 128;
    a.subsets = (int)(idle < 1 ? 1 : idle < (adapters + 3) / 4 ? idle : (adapters + 3) / 4);
    a.wide_tiles = (int)((z.M + kPairRows - 1) / kPairRows);
    a.sorted = sort ? z.n : 0;
    a.order = k.order; a.counts = k.counts; a.starts = k.starts;
    a.extra = (int)((a.wide_tiles + a.sorted + a.cluster - 1) / a.cluster);
    // few CTAs: a tile's adapters one behind another are what takes the time, and
    // nothing else needs the shared memory
    const int most = a.rp > 64 ? 8 : kShrinkB;
    a.stages_b = tiles * a.cluster <= 152 ? most : a.rp > 64 ? 3 : 4;
    auto kern = f16 ? lora_shrink_kernel<BWD, true> : lora_shrink_kernel<BWD, false>;
    size_t smem = shrink_layout(BWD, a.rp, a.stages_b).total;
    if (smem < kShrinkSmem) smem = kShrinkSmem;
    err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    count_launch();
    return launch_k(kern, dim3((unsigned)((tiles * a.subsets + a.extra) * a.cluster)), dim3(kShrinkThreads), smem, s,
                    (unsigned)a.cluster, mx, mp, a);
}

template <bool BWD, int UB>
cudaError_t launch_layer_u(const CUtensorMap (&m)[5], const LayerArgs &a, bool f16, int sms, cudaStream_t s) {
    auto kern = f16 ? lora_layer_kernel<BWD, true, UB> : lora_layer_kernel<BWD, false, UB>;
    const cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)LayerSmem<UB>::kBytes);
    if (err != cudaSuccess) return err;
    const int pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
    count_launch();
    return launch_k(kern, dim3((unsigned)(2 * pairs)), dim3(kLayerThreads), (size_t)LayerSmem<UB>::kBytes, s, 1, m[0], m[1],
                    m[2], m[3], m[4], a);
}

// y (x, W, B) or dx (dy, W, A).
template <bool BWD>
cudaError_t launch_layer(const Sizes &z, bool f16, const void *rows, const void *w, const void *bias, const void *u,
                         const void *stack, void *out, const TileList *lists, int sms, cudaStream_t s) {
    LayerArgs a = {};
    a.lists = lists; a.bias = bias;
    a.M = z.M; a.cols = BWD ? z.K : z.N;
    a.rp = z.rp();
    a.k_blocks = (int)(((BWD ? z.N : z.K) + kBK - 1) / kBK);
    // The width that leaves the least idle in the last wave; narrower tiles take
    // more operand bytes for their products: 0.29, 0.24 and 0.26 us per k-block of
    // 256, 192 and 128 columns.  (The width does not show in a result.)
    const int64_t tm = (z.M + kPairRows - 1) / kPairRows, pairs = sms / 2;
    auto work = [&](int64_t bn, int64_t each) { return (tm * ((a.cols + bn - 1) / bn) + pairs - 1) / pairs * each; };
    a.bn = 256;
    if (work(192, 205) < work(256, 256)) a.bn = 192;
    if (work(128, 225) < (a.bn == 192 ? work(192, 205) : work(256, 256))) a.bn = 128;
    a.tiles_n = (int)((a.cols + a.bn - 1) / a.bn);
    a.tiles = (int)(tm * a.tiles_n);
    const int low = BWD ? (a.rp > 64 ? 2 : 1) * a.bn / 2 * 128 : (a.bn / 2 + 63) / 64 * a.rp * 128;
    a.batch = 1;
    while (a.batch < 32 && 2 * a.batch * low <= (int)kStageBytes) a.batch *= 2;
    CUtensorMap m[5];
    cudaError_t err = encode(&m[0], rows, BWD ? z.N : z.K, z.M, 64, 128);
    if (err == cudaSuccess) err = encode(&m[1], w, z.N, z.K, 64, BWD ? a.bn / 2 : 64);
    if (err == cudaSuccess) err = encode(&m[2], u, kPlanes * a.rp, z.M, 64, 128);
    if (err == cudaSuccess)
        err = BWD ? encode_stack(&m[3], stack, z.r, z.K, z.n, a.bn / 2) : encode_stack(&m[3], stack, z.N, z.r, z.n, a.rp);
    if (err == cudaSuccess) err = encode(&m[4], out, a.cols, z.M, 64, 32);
    if (err != cudaSuccess) return err;
    const int ub = (2 * a.rp + 63) / 64;
    return ub <= 1 ? launch_layer_u<BWD, 1>(m, a, f16, sms, s)
         : ub == 2 ? launch_layer_u<BWD, 2>(m, a, f16, sms, s)
                   : launch_layer_u<BWD, 4>(m, a, f16, sms, s);
}

carbon_status_t check(const Sizes &z, int dtype) {
    if (!sizes_ok(z)) return CARBON_ERR_INVALID_ARG;
    if (dtype != CARBON_F32 && dtype != CARBON_BF16 && dtype != CARBON_F16) return CARBON_ERR_INVALID_ARG;
    if (dtype == CARBON_F32) return CARBON_ERR_UNSUPPORTED;
    if (z.K % 8 != 0 || z.N % 8 != 0 || z.r % 8 != 0) return CARBON_ERR_MISALIGNED;
    return CARBON_OK;
}

}  // namespace

carbon_status_t lora_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_lora_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_lora_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

}  // namespace carbon

using namespace carbon;

extern "C" {

int64_t carbon_lora_linear_u_elements(int64_t M, int64_t r) {
    const Sizes z = {M, 1, 1, 1, r};
    return sizes_ok(z) ? M * kPlanes * z.rp() : -1;
}

int64_t carbon_lora_linear_fwd_workspace(int64_t M, int64_t K, int64_t N, int64_t n, int64_t r) {
    const Sizes z = {M, K, N, n, r};
    return sizes_ok(z) ? plan_work(nullptr, z, false, false).bytes : -1;
}

int64_t carbon_lora_linear_bwd_workspace(int64_t M, int64_t K, int64_t N, int64_t n, int64_t r) {
    const Sizes z = {M, K, N, n, r};
    return sizes_ok(z) ? plan_work(nullptr, z, true, true).bytes : -1;
}

carbon_status_t carbon_lora_linear_fwd(void *y, void *u, const void *x, const void *w, const void *bias, const void *a,
                                       const void *b, const int64_t *adapters, const float *scales, int64_t M, int64_t K,
                                       int64_t N, int64_t n, int64_t r, void *workspace, int64_t workspace_bytes,
                                       carbon_dtype_t dtype, carbon_stream_t stream) {
    const Sizes z = {M, K, N, n, r};
    carbon_status_t st = check(z, dtype);
    if (st != CARBON_OK) return st;
    if (M > 0 && (!y || !u || !x || !w || !a || !b || !adapters || !scales || !workspace || !aligned16(workspace) ||
                  workspace_bytes < carbon_lora_linear_fwd_workspace(M, K, N, n, r)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(16, y, u, x, w, a, b) || !aligned_to(2, bias) || !aligned_to(8, adapters) || !aligned_to(4, scales))
        return CARBON_ERR_MISALIGNED;
    if (M == 0) return CARBON_OK;
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool f16 = dtype == CARBON_F16;
    const Work k = plan_work(workspace, z, false, false);
    cudaError_t err = launch_shrink<false>(z, f16, x, a, adapters, scales, u, k, false, s);
    if (err == cudaSuccess) err = launch_layer<false>(z, f16, x, w, bias, u, b, y, k.lists, sms, s);
    return note_cuda(err);
}

carbon_status_t carbon_lora_linear_bwd(void *dx, void *da, void *db, const void *dy, const void *x, const void *w,
                                       const void *a, const void *b, const int64_t *adapters, const float *scales,
                                       const void *u, int64_t M, int64_t K, int64_t N, int64_t n, int64_t r,
                                       void *workspace, int64_t workspace_bytes, carbon_dtype_t dtype,
                                       carbon_stream_t stream) {
    const Sizes z = {M, K, N, n, r};
    carbon_status_t st = check(z, dtype);
    if (st != CARBON_OK) return st;
    if (!da != !db || (!dx && !da)) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!dy || !b || !adapters || !scales || !workspace || !aligned16(workspace) ||
                  (dx && (!w || !a)) || (da && (!x || !u)) ||
                  workspace_bytes < carbon_lora_linear_bwd_workspace(M, K, N, n, r)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(16, dx, da, db, dy, x, w, a, b, u) || !aligned_to(8, adapters) || !aligned_to(4, scales))
        return CARBON_ERR_MISALIGNED;
    if (M == 0 && !da) return CARBON_OK;
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool f16 = dtype == CARBON_F16;
    if (M == 0) {
        cudaError_t err = cudaMemsetAsync(da, 0, (size_t)(n * K * r) * 2, s);
        if (err == cudaSuccess) err = cudaMemsetAsync(db, 0, (size_t)(n * r * N) * 2, s);
        return note_cuda(err);
    }
    const Work k = plan_work(workspace, z, true, da != nullptr);
    cudaError_t err = launch_shrink<true>(z, f16, dy, b, adapters, scales, k.du, k, da != nullptr, s);
    if (err == cudaSuccess && dx) err = launch_layer<true>(z, f16, dy, w, nullptr, k.du, a, dx, k.lists, sms, s);
    if (err == cudaSuccess && da) {
        GradArgs g = {};
        g.x = static_cast<const uint16_t *>(x); g.dy = static_cast<const uint16_t *>(dy);
        g.u = static_cast<const uint16_t *>(u); g.du = k.du;
        g.order = k.order; g.counts = k.counts; g.starts = k.starts;
        g.da = static_cast<uint16_t *>(da); g.db = static_cast<uint16_t *>(db);
        g.parts = k.parts; g.slots = k.slots;
        g.M = M; g.K = K; g.N = N; g.n = n;
        g.r = (int)r; g.rp = z.rp();
        g.tiles_k = (int)(up128(K) / 128);
        g.tiles = g.tiles_k + (int)(up128(N) / 128);
        const int stages = g.rp > 64 ? 2 : 3;
        auto kern = g.rp > 64 ? (f16 ? lora_grads_kernel<true, 2> : lora_grads_kernel<false, 2>)
                              : (f16 ? lora_grads_kernel<true, 3> : lora_grads_kernel<false, 3>);
        const size_t smem = grad_layout(g.rp, stages).total;
        CUtensorMap m[4];
        err = encode(&m[0], x, K, M, 64, 64);
        if (err == cudaSuccess) err = encode(&m[1], dy, N, M, 64, 64);
        if (err == cudaSuccess) err = encode(&m[2], u, kPlanes * g.rp, M, 64, 64);
        if (err == cudaSuccess) err = encode(&m[3], k.du, kPlanes * g.rp, M, 64, 64);
        if (err == cudaSuccess) err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        // at most this many pieces: one per adapter with rows, and one for every whole piece of rows
        const int64_t pieces = (n < M ? n : M) + M / kPiece;
        if (err == cudaSuccess) {
            count_launch();
            err = launch_k(kern, dim3((unsigned)pieces, (unsigned)g.tiles), dim3(kGradThreads), smem, s, 1, m[0], m[1], m[2],
                           m[3], g);
        }
        if (err == cudaSuccess) {
            count_launch();
            err = launch_k(f16 ? lora_join_kernel<true> : lora_join_kernel<false>, 
                           dim3((unsigned)n, (unsigned)g.tiles, (unsigned)((r + 7) / 8)), dim3(256), 0, s, 1, g);
        }
    }
    return note_cuda(err);
}

}  // extern "C"
