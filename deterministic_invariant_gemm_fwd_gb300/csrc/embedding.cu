// embedding.cu - token embedding: out[m] = scale * table[ids[m]], and its
// gradient dtable[v] = scale * sum over m with ids[m] == v of dy[m].
//
// The lookup moves bytes: a warp per token, 16-byte vectors.
//
// Bound of the gradient: the table's bytes (written once whole, 77 MB for
// 50257 x 768 bf16, 11.6 us), then latency: two short kernels that wait for the
// sort.  8192 tokens of 768, cold: sort with clearing 14.8 us, chunks 11, joins
// 8; one after the other 37 us with the host's call.
//
// The gradient sorts the tokens by (id, position) and adds each row's tokens
// in that order, in fp32, so that the result does not depend on scheduling
// (the Carbon README replaces atomics in scatters with sorted indices, "How
// It Works"):
//   sort     least-significant-digit radix sort of (id, position) pairs with
//            digits of at most 9 bits: lists of up to kOneCta tokens in one
//            CTA's shared memory, longer ones with a histogram kernel and a
//            stable scatter kernel per digit that also counts the next one.
//            The other CTAs of these kernels clear the table's gradient,
//            which takes longer than the sort and does not wait for it
//            (leaving part of it to the next kernels, which skip the rows that
//            tokens name, was slower: 44 to 60 us against 37).
//   chunks   a CTA per kChunk sorted positions adds the runs of equal ids in
//            it: a run that lies within the chunk is a finished row, the
//            parts of one that goes on in a neighbouring chunk are kept.
//   joins    the CTA of the chunk in which such a run begins adds its parts in
//            order.  However often a token occurs, no CTA adds more than
//            kChunk rows and the parts of one run.
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
constexpr int kOneCta = 8192;            // tokens that one CTA sorts
constexpr int kOneThreads = 1024;
constexpr int kChunk = 16;               // sorted positions per chunk
constexpr int kFillCtas = 152 * 4;       // CTAs that clear the gradient beside a sort kernel

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

// Workspace: two (key, position) arrays, a histogram per pass and CTA, and
// two partial rows per chunk: of a run that began before it, and of one that
// goes on after it.
struct Workspace {
    uint32_t *key[2], *pos[2];
    uint32_t *hist;              // [passes][blocks][kBins]
    uint32_t *jobs;              // their count, then the chunks in which a run begins that goes on
    float *part;                 // [chunks][2][D]
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
    t.hist = reinterpret_cast<uint32_t *>(take(M <= kOneCta ? 0 : 4 * s.passes * s.blocks * kBins));
    t.jobs = reinterpret_cast<uint32_t *>(take(4 * (1 + (M + kChunk - 1) / kChunk)));
    t.part = reinterpret_cast<float *>(take(4 * 2 * ((M + kChunk - 1) / kChunk) * D));
    if (w) *w = t;
    return used;
}

// Bytes of the gradient that a kernel clears: CTA `cta` of `ctas` takes every
// ctas-th piece.
struct Fill {
    char *base;                  // null: nothing to clear
    int64_t bytes;
};

__device__ __forceinline__ void fill(const Fill &f, int64_t cta, int64_t ctas) {
    if (f.base == nullptr) return;
    const int64_t head = min((int64_t)((16 - (reinterpret_cast<uintptr_t>(f.base) & 15)) & 15), f.bytes);
    const int64_t nvec = (f.bytes - head) / 16, tail = head + nvec * 16;
    uint4 *v = reinterpret_cast<uint4 *>(f.base + head);
    const int64_t n = ctas * blockDim.x, me = cta * blockDim.x + threadIdx.x;
#pragma unroll 4
    for (int64_t i = me; i < nvec; i += n) v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (me < head) f.base[me] = 0;
    if (me < f.bytes - tail) f.base[tail + me] = 0;
}

// The sort key of a token: its id, or V for one that adds to no row.
__device__ __forceinline__ uint32_t key_of(int64_t id, int64_t V, int64_t padding_idx) {
    return (id >= 0 && id < V && id != padding_idx) ? (uint32_t)id : (uint32_t)V;
}

// Places of one digit's keys, for the threads of a CTA with W warps: count
// holds each warp's keys per digit and receives each warp's first place.
// before[j], total[j]: keys of digit (thread * PER + j) placed ahead of this
// CTA's, and of all CTAs.
template <int W, int PER>
__device__ __forceinline__ void digit_places(uint32_t (*count)[kBins], uint32_t *warp_total,
                                             const uint32_t (&before)[PER], const uint32_t (&total)[PER]) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    uint32_t sum = 0u;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum += total[j];
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
    if (threadIdx.x * PER < kBins) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            uint32_t at = place + before[j];
#pragma unroll 8
            for (int w = 0; w < W; ++w) {
                const uint32_t c = count[w][threadIdx.x * PER + j];
                count[w][threadIdx.x * PER + j] = at;
                at += c;
            }
            place += total[j];
        }
    }
    __syncthreads();
}

// Place of this lane's key among the warp's (stable), given the warp's next
// places per digit, which move on.  digit: out of range where there is none.
__device__ __forceinline__ uint32_t next_place(uint32_t *place, uint32_t digit, bool have, int lane) {
    const uint32_t peers = __match_any_sync(0xffffffffu, digit);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    const uint32_t at = have ? place[digit] + rank : 0u;
    __syncwarp();
    if (have && rank == 0) place[digit] += __popc(peers);
    __syncwarp();
    return at;
}

// The whole sort of a list of at most kOneCta tokens, by CTA 0.
struct OneSmem {
    uint32_t count[kOneThreads / 32][kBins];
    uint32_t key[2][kOneCta];
    uint16_t pos[2][kOneCta];
    uint32_t warp_total[kOneThreads / 32];
};

__global__ void __launch_bounds__(kOneThreads)
sort_one_kernel(const int64_t *__restrict__ ids, int M, int64_t V, int64_t padding_idx, int digit_bits, int passes,
                uint32_t *__restrict__ key_out, uint32_t *__restrict__ pos_out, uint32_t *__restrict__ jobs, const Fill f) {
    extern __shared__ __align__(16) uint8_t one_raw[];
    OneSmem &s = *reinterpret_cast<OneSmem *>(one_raw);
    wait_prior_grid();
    allow_next_grid();
    if (blockIdx.x > 0) {
        fill(f, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    constexpr int W = kOneThreads / 32;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) jobs[0] = 0u;
    const uint32_t mask = (1u << digit_bits) - 1u;
    const int per_warp = ((M + W - 1) / W + 31) / 32 * 32, first = warp * per_warp;
    for (int i = threadIdx.x; i < M; i += kOneThreads) {
        const int64_t id = ids[i];
        if (id < 0 || id >= V) atomicExch(&g_embedding_status, (unsigned)CARBON_ERR_OUT_OF_BOUNDS);
        s.key[0][i] = key_of(id, V, padding_idx);
        s.pos[0][i] = (uint16_t)i;
    }
    for (int p = 0; p < passes; ++p) {
        const int in = p & 1, shift = p * digit_bits;
        for (int i = threadIdx.x; i < W * kBins; i += kOneThreads) (&s.count[0][0])[i] = 0u;
        __syncthreads();
        for (int r = 0; r < per_warp; r += 32) {
            const int i = first + r + lane;
            if (i < M) atomicAdd(&s.count[warp][(s.key[in][i] >> shift) & mask], 1u);
        }
        __syncthreads();
        uint32_t before[1] = {0u}, total[1] = {0u};
        if (threadIdx.x < kBins) {
#pragma unroll 8
            for (int w = 0; w < W; ++w) total[0] += s.count[w][threadIdx.x];
        }
        digit_places<W, 1>(s.count, s.warp_total, before, total);
        for (int r = 0; r < per_warp; r += 32) {
            const int i = first + r + lane;
            const bool have = i < M;
            const uint32_t key = have ? s.key[in][i] : 0u;
            const uint32_t at = next_place(s.count[warp], have ? (key >> shift) & mask : 0xffffffffu, have, lane);
            if (have) {
                if (p + 1 < passes) {
                    s.key[in ^ 1][at] = key;
                    s.pos[in ^ 1][at] = s.pos[in][i];
                } else if (CHK(at, 1, M)) {
                    key_out[at] = key;
                    pos_out[at] = s.pos[in][i];
                }
            }
        }
        __syncthreads();
    }
}

// Histogram of the first digit of each CTA's tile; clears the later passes'
// histograms.
__global__ void __launch_bounds__(kSortThreads)
sort_start_kernel(const int64_t *__restrict__ ids, int64_t M, int64_t V, int64_t padding_idx, int tile,
                  int64_t blocks, int digit_bits, int passes, uint32_t *__restrict__ hist,
                  uint32_t *__restrict__ jobs, const Fill f) {
    __shared__ uint32_t count[kBins];
    wait_prior_grid();
    allow_next_grid();
    if ((int64_t)blockIdx.x >= blocks) {                  // CTA-uniform
        fill(f, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) jobs[0] = 0u;
    for (int d = threadIdx.x; d < kBins; d += kSortThreads) {
        count[d] = 0u;
        for (int p = 1; p < passes; ++p) hist[((int64_t)p * blocks + blockIdx.x) * kBins + d] = 0u;
    }
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
                    int64_t blocks, int digit_bits, int shift, const Fill f) {
    __shared__ uint32_t count[kSortWarps][kBins];         // per-warp digit counts, then next places
    __shared__ uint32_t warp_total[kSortWarps];
    wait_prior_grid();
    allow_next_grid();
    if ((int64_t)blockIdx.x >= blocks) {
        fill(f, blockIdx.x - blocks, gridDim.x - blocks);
        return;
    }
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
    uint32_t before[kPer], total[kPer];
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
    digit_places<kSortWarps, kPer>(count, warp_total, before, total);
    for (int r = 0; r < per_warp; r += 32) {
        const int64_t i = first + r + lane;
        const bool have = i < M;
        const uint32_t key = have ? key_at(i) : 0u;
        const uint32_t at = next_place(count[warp], have ? (key >> shift) & mask : 0xffffffffu, have, lane);
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

// A finished row: scaled, added to what is there (accumulate), rounded once.
template <typename T, int N>
__device__ __forceinline__ void write_row(T *dst, float (&acc)[N], float scale, int accumulate) {
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] *= scale;
    if (accumulate) {
        float old[N];
        load_f32<T, N>(dst, old);
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] += old[j];
    }
    store_f32<T, N>(dst, acc);
}

// A CTA per chunk; a thread per column vector.  All rows of the chunk are
// loaded before the first addition (a bound of 128 registers, for more CTAs,
// took some of them out of flight: 37 -> 43 us for the whole gradient of 8192 x
// 768 bf16; so did chunks of 8 or 32 rows, 40 and 42 us).
template <typename T, int N>
__global__ void __launch_bounds__(256)
chunk_kernel(T *__restrict__ dtable, const T *__restrict__ dy, const uint32_t *__restrict__ key,
             const uint32_t *__restrict__ pos, uint32_t *__restrict__ jobs, float *__restrict__ part, int64_t M,
             int64_t V, int64_t D, float scale, int accumulate) {
    __shared__ uint32_t k[kChunk + 2], m[kChunk];         // k[1 + q]: key of position q; V: none
    wait_prior_grid();
    allow_next_grid();
    const int64_t first = (int64_t)blockIdx.x * kChunk;
    if (threadIdx.x < kChunk + 2) {
        const int64_t i = first + (int)threadIdx.x - 1;
        k[threadIdx.x] = i >= 0 && i < M ? key[i] : (uint32_t)V;
        if (threadIdx.x >= 1 && threadIdx.x <= kChunk) m[threadIdx.x - 1] = i < M ? pos[i] : 0u;
    }
    __syncthreads();
    // does a run begin here and go on? (the list's order does not matter: its runs are separate rows)
    if (threadIdx.x == 0 && k[kChunk] < V && k[kChunk + 1] == k[kChunk] && (k[1] != k[kChunk] || k[0] != k[1]))
        jobs[1 + atomicAdd(jobs, 1u)] = blockIdx.x;
    for (int64_t v = threadIdx.x; v < D / N; v += blockDim.x) {
        Pack<T, N> rows[kChunk];
#pragma unroll
        for (int q = 0; q < kChunk; ++q)
            if (k[1 + q] < V && CHK((int64_t)m[q] * D + v * N, N, M * D))
                rows[q] = *reinterpret_cast<const Pack<T, N> *>(dy + (int64_t)m[q] * D + v * N);
        float acc[N];
        bool before = k[0] == k[1];                       // the run began in an earlier chunk
#pragma unroll
        for (int j = 0; j < N; ++j) acc[j] = 0.0f;
#pragma unroll
        for (int q = 0; q < kChunk; ++q) {
            const uint32_t id = k[1 + q];
            if (id >= V) continue;                        // sorted last: nothing follows
            float f[N];
            widen(rows[q], f);
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] += f[j];
            const bool ends = k[2 + q] != id;
            if (!ends && q + 1 < kChunk) continue;
            if (ends && !before) {
                if (CHK(id, 1, V)) write_row<T, N>(dtable + (int64_t)id * D + v * N, acc, scale, accumulate);
            } else {                                      // part 0: of a run from before; part 1: of one that goes on
                float *dst = part + ((int64_t)blockIdx.x * 2 + (before ? 0 : 1)) * D + v * N;
#pragma unroll
                for (int j = 0; j < N; ++j) dst[j] = acc[j];
            }
            before = false;
#pragma unroll
            for (int j = 0; j < N; ++j) acc[j] = 0.0f;
        }
    }
}

// A run that goes on after its first chunk: its parts in order.  A CTA takes 64
// columns of a run at a time; 16 threads per vector of columns take a
// sixteenth of the parts each, and their sums are added in order.
constexpr int kJoinVec = 4, kJoinThreads = 256, kJoinColumns = 16, kJoinGroups = kJoinThreads / kJoinColumns;

template <typename T, int N>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(T *__restrict__ dtable, const uint32_t *__restrict__ key, const uint32_t *__restrict__ jobs,
            const float *__restrict__ part, int64_t M, int64_t V, int64_t D, float scale, int accumulate) {
    static_assert(N == 1 || N == kJoinVec, "columns per thread");
    __shared__ float sums[kJoinGroups][kJoinColumns][N];
    wait_prior_grid();
    allow_next_grid();
    const int64_t chunks = (M + kChunk - 1) / kChunk;
    const int64_t blocks = (D / N + kJoinColumns - 1) / kJoinColumns, work = (int64_t)jobs[0] * blocks;
    for (int64_t j = blockIdx.x; j < work; j += gridDim.x) {
        const int64_t c = jobs[1 + j / blocks];
        const uint32_t id = key[(c + 1) * kChunk];
        int64_t n = 0;                                    // chunks after c that hold a part
        for (;;) {
            const int64_t e = c + 1 + n + threadIdx.x;
            const int found = __syncthreads_count(e < chunks && key[e * kChunk] == id);
            n += found;
            if (found < kJoinThreads) break;
        }
        const int col = threadIdx.x % kJoinColumns, group = threadIdx.x / kJoinColumns;
        const int64_t v = j % blocks * kJoinColumns + col, per = (n + 1 + kJoinGroups - 1) / kJoinGroups;
        float acc[N];
#pragma unroll
        for (int q = 0; q < N; ++q) acc[q] = 0.0f;
        if (v < D / N) {
            const int64_t to = min(n + 1, (group + 1) * per);
#pragma unroll 4
            for (int64_t q = group * per; q < to; ++q) {
                // part 1 of the first chunk, part 0 of the others
                const Pack<float, N> src =
                    *reinterpret_cast<const Pack<float, N> *>(part + ((c + q) * 2 + (q == 0 ? 1 : 0)) * D + v * N);
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += src.e[i];
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) sums[group][col][i] = acc[i];
        __syncthreads();
        if (group == 0 && v < D / N) {
#pragma unroll
            for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] += sums[g][col][i];
            if (CHK(id, 1, V)) write_row<T, N>(dtable + (int64_t)id * D + v * N, acc, scale, accumulate);
        }
        __syncthreads();
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
    const dim3 chunks((unsigned)((M + kChunk - 1) / kChunk));
    const int64_t threads = (D / N + 31) / 32 * 32;
    count_launch();
    cudaError_t err = launch_k(chunk_kernel<T, N>, chunks, dim3((unsigned)(threads < 64 ? 64 : threads < 256 ? threads : 256)),
                               0, s, 1, static_cast<T *>(dtable), static_cast<const T *>(dy),
                               (const uint32_t *)w.key[sorted], (const uint32_t *)w.pos[sorted], w.jobs, w.part, M, V, D,
                               scale, accumulate);
    if (err != cudaSuccess || M <= kChunk) return err;    // one chunk: no run goes on
    count_launch();
    // vectors of 4 columns where a row of the parts and of the table starts on their boundary
    constexpr int J = N == 1 ? 1 : kJoinVec;
    const int64_t most = (int64_t)chunks.x * ((D / J + kJoinColumns - 1) / kJoinColumns);
    return launch_k(join_kernel<T, J>, dim3((unsigned)(most < 152 * 4 ? most : 152 * 4)), dim3(kJoinThreads), 0, s, 1,
                    static_cast<T *>(dtable), (const uint32_t *)w.key[sorted], (const uint32_t *)w.jobs,
                    (const float *)w.part, M, V, D, scale, accumulate);
}

// The kernels of the sort, each clearing its share of the gradient.
cudaError_t launch_sort(const Workspace &w, const SortPlan &plan, const int64_t *ids, int64_t M, int64_t V,
                        int64_t padding_idx, char *clear, int64_t clear_bytes, int *sorted, cudaStream_t s) {
    cudaError_t err;
    auto fill_ctas = [&](int64_t bytes) {                 // at least 16 KiB per CTA
        const int64_t n = (bytes + 16383) / 16384;
        return clear == nullptr ? 0 : n < kFillCtas ? n : (int64_t)kFillCtas;
    };
    if (M <= kOneCta) {
        *sorted = 0;
        if ((err = cudaFuncSetAttribute(sort_one_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)sizeof(OneSmem))) != cudaSuccess)
            return err;
        count_launch();
        // its shared memory leaves room for one CTA per SM
        const int64_t clearing = fill_ctas(clear_bytes);
        return launch_k(sort_one_kernel, dim3((unsigned)(1 + (clearing < 151 ? clearing : 151))), dim3(kOneThreads), sizeof(OneSmem),
                        s, 1, ids, (int)M, V, padding_idx, plan.digit_bits, plan.passes, w.key[0], w.pos[0],
                        w.jobs, Fill{clear, clear_bytes});
    }
    *sorted = (plan.passes - 1) & 1;
    const int64_t share = (clear_bytes / (plan.passes + 1) + 15) & ~(int64_t)15;
    auto part = [&](int i) {                              // of kernel i
        const int64_t from = share * i < clear_bytes ? share * i : clear_bytes;
        const int64_t to = i == plan.passes || from + share > clear_bytes ? clear_bytes : from + share;
        return Fill{clear == nullptr ? nullptr : clear + from, to - from};
    };
    count_launch(1 + plan.passes);
    err = launch_k(sort_start_kernel, dim3((unsigned)(plan.blocks + fill_ctas(share))), dim3(kSortThreads), 0, s, 1, ids, M,
                   V, padding_idx, plan.tile, plan.blocks, plan.digit_bits, plan.passes, w.hist, w.jobs, part(0));
    for (int p = 0; p < plan.passes && err == cudaSuccess; ++p) {
        const uint32_t *h = w.hist + (int64_t)p * plan.blocks * kBins;
        uint32_t *next = p + 1 < plan.passes ? w.hist + (int64_t)(p + 1) * plan.blocks * kBins : nullptr;
        auto kern = p == 0 ? sort_scatter_kernel<true> : sort_scatter_kernel<false>;
        err = launch_k(kern, dim3((unsigned)(plan.blocks + fill_ctas(share))), dim3(kSortThreads), 0, s, 1, ids,
                       (const uint32_t *)w.key[(p + 1) & 1], (const uint32_t *)w.pos[(p + 1) & 1], w.key[p & 1],
                       w.pos[p & 1], h, next, M, V, padding_idx, plan.tile, plan.blocks, plan.digit_bits,
                       p * plan.digit_bits, part(p + 1));
    }
    return err;
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
    if (!aligned_to(dtype_size(dtype), out, table) || !aligned_to(8, ids)) return CARBON_ERR_MISALIGNED;
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
    if (!aligned_to(dtype_size(dtype), dtable, dy) || !aligned_to(8, ids)) return CARBON_ERR_MISALIGNED;
    carbon_status_t st = injected_launch_failure();
    if (st != CARBON_OK) return st;
    if ((st = current_device(nullptr, nullptr)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) {
        if (accumulate) return CARBON_OK;
        return note_cuda(cudaMemsetAsync(dtable, 0, (size_t)(V * D) * dtype_size(dtype), s));
    }

    int sorted = 0;
    cudaError_t err = launch_sort(w, plan, ids, M, V, padding_idx, accumulate ? nullptr : static_cast<char *>(dtable),
                                  accumulate ? 0 : V * D * (int64_t)dtype_size(dtype), &sorted, s);
    if (err != cudaSuccess) return note_cuda(err);
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
