// embedding.cu - token embedding: out[m] = scale * table[ids[m]], and its
// gradient dtable[v] = scale * sum over m with ids[m] == v of dy[m].
//
// The lookup moves bytes: a warp per token, 16-byte vectors.
//
// The gradient sorts the tokens by (id, position) and adds each row's tokens
// in that order, in fp32, so that the result does not depend on scheduling
// (the Carbon README replaces atomics in scatters with sorted indices, "How
// It Works"):
//   sort    least-significant-digit radix sort of (id, position) pairs with
//           digits of at most 9 bits: one histogram kernel, then one stable
//           scatter kernel per digit that also counts the next digit;
//   runs    each row's range of sorted positions; every aligned chunk of
//           kChunk positions that lies within one row's range is summed by a
//           CTA of its own (a row that very many tokens name is then not one
//           CTA's work);
//   sum     a warp per table row: its positions in ascending order, whole
//           chunks by their sums, one rounding; zeros where there are none.
#include "bounds.cuh"
#include "device_sync.cuh"
#include "rowvec.cuh"

namespace carbon {
namespace {

__device__ unsigned int g_embedding_status = 0;
#define CHK(idx, len, n) in_bounds(&g_embedding_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

constexpr int kRowsPerCta = 4;           // lookup: warps (= tokens) per CTA
constexpr int kSortThreads = 256;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigit = 9;             // bits
constexpr int kBins = 1 << kMaxDigit;
constexpr int kChunk = 64;               // sorted positions per chunk sum
constexpr int kSumWarps = 8;             // table rows per CTA of the sum kernel

// ---- lookup -------------------------------------------------------------------

template <typename T, int N>
__global__ void __launch_bounds__(kRowsPerCta * 32)
embedding_fwd_kernel(T *__restrict__ out, const T *__restrict__ table, const int64_t *__restrict__ ids,
                     int64_t M, int64_t V, int64_t D, float scale) {
    wait_prior_grid();
    allow_next_grid();
    const int64_t m = (int64_t)blockIdx.x * kRowsPerCta + threadIdx.x / 32;
    if (m >= M) return;
    const int lane = threadIdx.x % 32;
    const int64_t id = ids[m], nvec = D / N;
    const bool named = id >= 0 && id < V;
    if (!named && lane == 0) atomicExch(&g_embedding_status, (unsigned)CARBON_ERR_OUT_OF_BOUNDS);
    const T *src = table + (named ? id : 0) * D;
    T *dst = out + m * D;
    constexpr int U = 4;
    for (int64_t i0 = lane; i0 < nvec; i0 += 32 * U) {
        float f[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + 32 * u;
            if (i < nvec && named) {
                load_f32<T, N>(src + i * N, f[u]);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) f[u][k] = 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = i0 + 32 * u;
            if (i < nvec && CHK(m * D + i * N, N, M * D)) {
#pragma unroll
                for (int k = 0; k < N; ++k) f[u][k] *= scale;
                store_f32<T, N>(dst + i * N, f[u]);
            }
        }
    }
}

// ---- sort -----------------------------------------------------------------------

struct SortPlan {
    int passes, digit_bits;
    int tile;                    // keys per CTA
    int64_t blocks;              // CTAs
};

SortPlan make_plan(int64_t M, int64_t V) {
    SortPlan s;
    int bits = 1;
    while (((int64_t)1 << bits) <= V) ++bits;            // keys 0 .. V (V: no row)
    s.passes = (bits + kMaxDigit - 1) / kMaxDigit;
    s.digit_bits = (bits + s.passes - 1) / s.passes;
    // each CTA reads every CTA's histogram: fewer, larger tiles for long lists
    s.tile = M <= 65536 ? 1024 : 8192;
    s.blocks = (M + s.tile - 1) / s.tile;
    return s;
}

// Workspace: two (key, position) arrays, a histogram per pass and CTA, the
// rows' ranges, the chunk sums.
struct Workspace {
    uint32_t *key[2], *pos[2];
    uint32_t *hist;              // [passes][blocks][kBins]
    uint2 *range;                // [V]
    float *chunk_sum;            // [M / kChunk][D]
};

int64_t round16(int64_t b) { return (b + 15) & ~(int64_t)15; }

int64_t lay_out(Workspace *w, void *base, int64_t M, int64_t V, int64_t D, const SortPlan &s) {
    char *p = static_cast<char *>(base);
    int64_t used = 0;
    auto take = [&](int64_t bytes) {
        char *q = p + used;
        used += round16(bytes);
        return q;
    };
    Workspace t;
    for (int i = 0; i < 2; ++i) {
        t.key[i] = reinterpret_cast<uint32_t *>(take(4 * M));
        t.pos[i] = reinterpret_cast<uint32_t *>(take(4 * M));
    }
    t.hist = reinterpret_cast<uint32_t *>(take(4 * s.passes * s.blocks * kBins));
    t.range = reinterpret_cast<uint2 *>(take(8 * V));
    t.chunk_sum = reinterpret_cast<float *>(take(4 * (M / kChunk) * D));
    if (w) *w = t;
    return used;
}

// The sort key of a token: its id, or V for one that adds to no row.
__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V, int64_t padding_idx) {
    return (id >= 0 && id < V && id != padding_idx) ? (uint32_t)id : (uint32_t)V;
}

// Histogram of the first digit of each CTA's tile; clears the later passes'
// histograms and the rows' ranges.
__global__ void __launch_bounds__(kSortThreads)
sort_start_kernel(const int64_t *__restrict__ ids, int64_t M, int64_t V, int64_t padding_idx, int tile,
                  int64_t blocks, int digit_bits, int passes, uint32_t *__restrict__ hist,
                  uint2 *__restrict__ range) {
    __shared__ uint32_t count[kBins];
    wait_prior_grid();
    allow_next_grid();
    const int64_t nthreads = (int64_t)gridDim.x * kSortThreads;
    const int64_t me = (int64_t)blockIdx.x * kSortThreads + threadIdx.x;
    for (int64_t i = me; i < V; i += nthreads) range[i] = make_uint2(0u, 0u);
    for (int64_t i = blocks * kBins + me; i < passes * blocks * kBins; i += nthreads) hist[i] = 0u;
    if ((int64_t)blockIdx.x >= blocks) return;            // CTA-uniform
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) count[d] = 0u;
    __syncthreads();
    const uint32_t mask = (1u << digit_bits) - 1u;
    const int64_t first = (int64_t)blockIdx.x * tile;
    for (int64_t i = first + threadIdx.x; i < first + tile && i < M; i += kSortThreads) {
        const int64_t id = ids[i];
        if (id < 0 || id >= V) atomicExch(&g_embedding_status, (unsigned)CARBON_ERR_OUT_OF_BOUNDS);
        atomicAdd(&count[key_of(id, V, padding_idx) & mask], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) hist[(int64_t)blockIdx.x * kBins + d] = count[d];
}

// One stable pass: each CTA places its tile's pairs by the digit at `shift`.
// A key's place is (keys of smaller digits) + (equal digits in earlier CTAs)
// + (equal digits in earlier warps) + (its rank in its warp's keys): every
// term a count, so the order is that of a sequential stable sort.  With
// hist_next, the next digit is counted for the CTA that will read the place.
template <bool FIRST>
__global__ void __launch_bounds__(kSortThreads)
sort_scatter_kernel(const int64_t *__restrict__ ids, const uint32_t *__restrict__ key_in,
                    const uint32_t *__restrict__ pos_in, uint32_t *__restrict__ key_out,
                    uint32_t *__restrict__ pos_out, const uint32_t *__restrict__ hist,
                    uint32_t *__restrict__ hist_next, int64_t M, int64_t V, int64_t padding_idx, int tile,
                    int64_t blocks, int digit_bits, int shift) {
    __shared__ uint32_t count[kSortWarps][kBins];         // per-warp digit counts, then next places
    __shared__ uint32_t warp_total[kSortWarps];
    wait_prior_grid();
    allow_next_grid();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t mask = (1u << digit_bits) - 1u;
    const int per_warp = tile / kSortWarps;               // a multiple of 32
    const int64_t first = (int64_t)blockIdx.x * tile + (int64_t)warp * per_warp;
    for (int i = threadIdx.x; i < kSortWarps * kBins; i += kSortThreads) (&count[0][0])[i] = 0u;
    __syncthreads();

    auto key_at = [&](int64_t i) -> uint32_t {
        return FIRST ? key_of(ids[i], V, padding_idx) : key_in[i];
    };
    for (int r = 0; r < per_warp; r += 32) {
        const int64_t i = first + r + lane;
        if (i < M) atomicAdd(&count[warp][(key_at(i) >> shift) & mask], 1u);
    }
    __syncthreads();
    // two digits per thread: totals over all CTAs, and over earlier ones
    constexpr int kPer = kBins / kSortThreads;
    uint32_t before[kPer], total[kPer], sum = 0u;
#pragma unroll
    for (int j = 0; j < kPer; ++j) before[j] = total[j] = 0u;
    for (int64_t b = 0; b < blocks; ++b) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t c = hist[b * kBins + threadIdx.x * kPer + j];
            if (b < blockIdx.x) before[j] += c;
            total[j] += c;
        }
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) sum += total[j];
    uint32_t incl = sum;                                  // inclusive scan over the CTA's threads
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) warp_total[warp] = incl;
    __syncthreads();
    uint32_t place = incl - sum;
    for (int w = 0; w < warp; ++w) place += warp_total[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        uint32_t at = place + before[j];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t c = count[w][threadIdx.x * kPer + j];
            count[w][threadIdx.x * kPer + j] = at;
            at += c;
        }
        place += total[j];
    }
    __syncthreads();
    for (int r = 0; r < per_warp; r += 32) {
        const int64_t i = first + r + lane;
        const bool have = i < M;
        const uint32_t key = have ? key_at(i) : 0u;
        // lanes past the end join no group (their digit is out of range)
        const uint32_t digit = have ? (key >> shift) & mask : 0xffffffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        const int rank = __popc(peers & ((1u << lane) - 1u));
        uint32_t at = have ? count[warp][digit] + rank : 0u;
        __syncwarp();
        if (have && rank == 0) count[warp][digit] += __popc(peers);
        __syncwarp();
        if (have && CHK(at, 1, M)) {
            key_out[at] = key;
            pos_out[at] = FIRST ? (uint32_t)i : pos_in[i];
            if (hist_next)
                atomicAdd(&hist_next[(int64_t)(at / (uint32_t)tile) * kBins +
                                     ((key >> (shift + digit_bits)) & mask)], 1u);
        }
    }
}

// ---- sums -----------------------------------------------------------------------

// Rows' ranges of sorted positions, and the sums of whole chunks.  One CTA
// per chunk.
template <typename T, int N>
__global__ void __launch_bounds__(256)
chunk_sum_kernel(const T *__restrict__ dy, const uint32_t *__restrict__ key, const uint32_t *__restrict__ pos,
                 uint2 *__restrict__ range, float *__restrict__ chunk_sum, int64_t M, int64_t V, int64_t D) {
    wait_prior_grid();
    allow_next_grid();
    const int64_t first = (int64_t)blockIdx.x * kChunk;
    const int64_t i = first + threadIdx.x;
    if (threadIdx.x < kChunk && i < M) {
        const uint32_t k = key[i];
        if (k < V && CHK(k, 1, V)) {
            if (i == 0 || key[i - 1] != k) range[k].x = (uint32_t)i;
            if (i == M - 1 || key[i + 1] != k) range[k].y = (uint32_t)i + 1u;
        }
    }
    if (first + kChunk > M) return;
    const uint32_t k = key[first];
    if (k != key[first + kChunk - 1] || k >= V) return;
    for (int64_t v = threadIdx.x; v < D / N; v += blockDim.x) {
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
#pragma unroll 8
        for (int q = 0; q < kChunk; ++q) {
            const int64_t m = pos[first + q];
            float f[N];
            if (!CHK(m * D + v * N, N, M * D)) continue;
            load_f32<T, N>(dy + m * D + v * N, f);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) chunk_sum[(first / kChunk) * D + v * N + j] = acc[j];
    }
}

// A warp per table row.
template <typename T, int N>
__global__ void __launch_bounds__(kSumWarps * 32)
row_sum_kernel(T *__restrict__ dtable, const T *__restrict__ dy, const uint32_t *__restrict__ pos,
               const uint2 *__restrict__ range, const float *__restrict__ chunk_sum, int64_t M, int64_t V,
               int64_t D, float scale, int accumulate) {
    wait_prior_grid();
    allow_next_grid();
    const int64_t v = (int64_t)blockIdx.x * kSumWarps + threadIdx.x / 32;
    if (v >= V) return;
    const int lane = threadIdx.x % 32;
    const uint2 r = range[v];
    T *dst = dtable + v * D;
    const int64_t nvec = D / N;
    if (r.x == r.y) {
        if (accumulate) return;
        float z[N];
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = 0.0f;
        for (int64_t i = lane; i < nvec; i += 32) store_f32<T, N>(dst + i * N, z);
        return;
    }
    for (int64_t i = lane; i < nvec; i += 32) {
        float acc[N];
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        for (uint32_t p = r.x; p < r.y;) {
            float f[N];
            if (p % kChunk == 0 && p + kChunk <= r.y) {
                const float *src = chunk_sum + (int64_t)(p / kChunk) * D + i * N;
#pragma unroll
                for (int j = 0; j < N; ++j) f[j] = src[j];
                p += kChunk;
            } else {
                load_f32<T, N>(dy + (int64_t)pos[p] * D + i * N, f);
                ++p;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] *= scale;
        if (accumulate) {
            float old[N];
            load_f32<T, N>(dst + i * N, old);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += old[j];
        }
        store_f32<T, N>(dst + i * N, acc);
    }
}

// ---- host side ----------------------------------------------------------------

bool sizes_ok(int64_t M, int64_t V, int64_t D) {
    int64_t t;
    return M >= 0 && V >= 0 && D >= 0 && M < 0x7fffffff && V < 0x7fffffff &&
           !__builtin_mul_overflow(M, D, &t) && !__builtin_mul_overflow(t, (int64_t)8, &t) &&
           !__builtin_mul_overflow(V, D, &t) && !__builtin_mul_overflow(t, (int64_t)8, &t);
}

template <typename T, int N>
cudaError_t launch_fwd(void *out, const void *table, const int64_t *ids, int64_t M, int64_t V, int64_t D,
                       float scale, cudaStream_t s) {
    count_launch();
    return launch_k(embedding_fwd_kernel<T, N>, dim3((unsigned)((M + kRowsPerCta - 1) / kRowsPerCta)),
                    dim3(kRowsPerCta * 32), 0, s, 1, static_cast<T *>(out), static_cast<const T *>(table), ids,
                    M, V, D, scale);
}

template <typename T, int N>
cudaError_t launch_sums(void *dtable, const void *dy, const Workspace &w, int sorted, int64_t M, int64_t V,
                        int64_t D, float scale, int accumulate, cudaStream_t s) {
    count_launch(2);
    cudaError_t err = launch_k(chunk_sum_kernel<T, N>, dim3((unsigned)((M + kChunk - 1) / kChunk)), dim3(256), 0,
                               s, 1, static_cast<const T *>(dy), (const uint32_t *)w.key[sorted],
                               (const uint32_t *)w.pos[sorted], w.range, w.chunk_sum, M, V, D);
    if (err != cudaSuccess) return err;
    return launch_k(row_sum_kernel<T, N>, dim3((unsigned)((V + kSumWarps - 1) / kSumWarps)),
                    dim3(kSumWarps * 32), 0, s, 1, static_cast<T *>(dtable), static_cast<const T *>(dy),
                    (const uint32_t *)w.pos[sorted], (const uint2 *)w.range, (const float *)w.chunk_sum, M, V, D,
                    scale, accumulate);
}

}  // namespace

carbon_status_t embedding_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_embedding_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_embedding_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

}  // namespace carbon

using namespace carbon;

extern "C" {

carbon_status_t carbon_embedding_fwd(void *out, const void *table, const int64_t *ids, int64_t M, int64_t V,
                                     int64_t D, float scale, carbon_dtype_t dtype, carbon_stream_t stream) {
    if (!sizes_ok(M, V, D)) return CARBON_ERR_INVALID_ARG;
    if (dtype != CARBON_F32 && dtype != CARBON_BF16 && dtype != CARBON_F16) return CARBON_ERR_INVALID_ARG;
    if (M == 0 || D == 0) return CARBON_OK;
    if (!out || !ids || (V > 0 && !table)) return CARBON_ERR_INVALID_ARG;
    carbon_status_t st = injected_launch_failure();
    if (st != CARBON_OK) return st;
    if ((st = current_device(nullptr, nullptr)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool vec = (D * dtype_size(dtype)) % 16 == 0 && aligned16(out) && aligned16(table);
    cudaError_t err;
    switch (dtype) {
    case CARBON_F32: err = vec ? launch_fwd<float, 4>(out, table, ids, M, V, D, scale, s)
                               : launch_fwd<float, 1>(out, table, ids, M, V, D, scale, s); break;
    case CARBON_BF16: err = vec ? launch_fwd<__nv_bfloat16, 8>(out, table, ids, M, V, D, scale, s)
                                : launch_fwd<__nv_bfloat16, 1>(out, table, ids, M, V, D, scale, s); break;
    default: err = vec ? launch_fwd<__half, 8>(out, table, ids, M, V, D, scale, s)
                       : launch_fwd<__half, 1>(out, table, ids, M, V, D, scale, s); break;
    }
    return note_cuda(err);
}

int64_t carbon_embedding_bwd_workspace(int64_t M, int64_t V, int64_t D) {
    if (!sizes_ok(M, V, D)) return -1;
    return lay_out(nullptr, nullptr, M, V, D, make_plan(M, V));
}

carbon_status_t carbon_embedding_bwd(void *dtable, const void *dy, const int64_t *ids, int64_t M, int64_t V,
                                     int64_t D, float scale, int64_t padding_idx, int accumulate,
                                     void *workspace, int64_t workspace_bytes, carbon_dtype_t dtype,
                                     carbon_stream_t stream) {
    if (!sizes_ok(M, V, D)) return CARBON_ERR_INVALID_ARG;
    if (dtype != CARBON_F32 && dtype != CARBON_BF16 && dtype != CARBON_F16) return CARBON_ERR_INVALID_ARG;
    if (padding_idx < -1 || padding_idx >= V) return CARBON_ERR_INVALID_ARG;
    if (V == 0 || D == 0) return CARBON_OK;
    if (!dtable || (M > 0 && (!dy || !ids || !workspace || !aligned16(workspace)))) return CARBON_ERR_INVALID_ARG;
    const SortPlan plan = make_plan(M, V);
    Workspace w;
    if (M > 0 && workspace_bytes < lay_out(&w, workspace, M, V, D, plan)) return CARBON_ERR_INVALID_ARG;
    carbon_status_t st = injected_launch_failure();
    if (st != CARBON_OK) return st;
    if ((st = current_device(nullptr, nullptr)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (accumulate) return CARBON_OK;
        return note_cuda(cudaMemsetAsync(dtable, 0, (size_t)(V * D) * dtype_size(dtype), s));
    }

    // enough CTAs to clear the ranges quickly as well
    const int64_t clear = (V + 4 * kSortThreads - 1) / (4 * kSortThreads);
    const int64_t grid0 = plan.blocks > clear ? plan.blocks : (clear < 1024 ? clear : (plan.blocks > 1024 ? plan.blocks : 1024));
    count_launch();
    cudaError_t err = launch_k(sort_start_kernel, dim3((unsigned)grid0), dim3(kSortThreads), 0, s, 1, ids, M, V,
                               padding_idx, plan.tile, plan.blocks, plan.digit_bits, plan.passes, w.hist, w.range);
    for (int p = 0; p < plan.passes && err == cudaSuccess; ++p) {
        const uint32_t *h = w.hist + (int64_t)p * plan.blocks * kBins;
        uint32_t *next = p + 1 < plan.passes ? w.hist + (int64_t)(p + 1) * plan.blocks * kBins : nullptr;
        auto kern = p == 0 ? sort_scatter_kernel<true> : sort_scatter_kernel<false>;
        count_launch();
        err = launch_k(kern, dim3((unsigned)plan.blocks), dim3(kSortThreads), 0, s, 1, ids,
                       (const uint32_t *)w.key[(p + 1) & 1], (const uint32_t *)w.pos[(p + 1) & 1], w.key[p & 1],
                       w.pos[p & 1], h, next, M, V, padding_idx, plan.tile, plan.blocks, plan.digit_bits,
                       p * plan.digit_bits);
    }
    if (err != cudaSuccess) return note_cuda(err);
    const int sorted = (plan.passes - 1) & 1;
    const bool vec = (D * dtype_size(dtype)) % 16 == 0 && aligned16(dtable) && aligned16(dy);
    switch (dtype) {
    case CARBON_F32: err = vec ? launch_sums<float, 4>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s)
                               : launch_sums<float, 1>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s); break;
    case CARBON_BF16: err = vec ? launch_sums<__nv_bfloat16, 8>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s)
                                : launch_sums<__nv_bfloat16, 1>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s); break;
    default: err = vec ? launch_sums<__half, 8>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s)
                       : launch_sums<__half, 1>(dtable, dy, w, sorted, M, V, D, scale, accumulate, s); break;
    }
    return note_cuda(err);
}

}  // extern "C"
