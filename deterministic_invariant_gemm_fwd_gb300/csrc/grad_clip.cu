// grad_clip.cu - the norm of all gradients of a model and their clipping.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + eps))
//
// Two kernels over chunks of the tensors, whose addresses travel as kernel
// parameters (no copy to the device; up to 256 a launch).  A warp takes a run of
// chunks, one each of few.  The first kernel sums squares, a
// number per CTA; the second adds these, each CTA for itself (a launch and a wait
// less than a kernel in between), and scales.  Its warps take their run from the
// end, so that they find in L2 what the first kernel read last.
//
// Order: an element's lane and place in its sum depend on its index in its tensor
// and on the tensors' sizes, not on addresses.  fp32 within 32 elements, float64
// from there on.
//
// Bound: memory.  Each gradient is read twice, the second time partly from L2,
// and written once.
#include "bounds.cuh"
#include "device_sync.cuh"
#include "rowvec.cuh"

#include <math.h>

#include <algorithm>
#include <vector>

namespace carbon {
namespace {

__device__ unsigned int g_clip_status = 0;
#define CHK(idx, len, n) in_bounds(&g_clip_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

constexpr int kThreads = 256, kCtas = 152 * 4;        // of each kernel, at most: four per SM
constexpr int kWarps = kCtas * kThreads / 32;
constexpr int kRounds = 4, kGranule = 8;               // a lane's elements of a block: kRounds granules
constexpr int64_t kBlock = 32 * kRounds * kGranule;    // 1024 elements
constexpr int64_t kChunk = 2 * kBlock;
// Tensors per launch: parameters are copied at each launch, so short lists have a
// table of their own.
constexpr int kFew = 32, kMany = 256;

struct Entry {
    const void *src;
    void *dst;
    int64_t size;
    int first;               // its first chunk
    int dtype;
};
template <int N>
struct Table {
    int n;
    int chunks, per;         // chunks of this table, and per warp
    Entry e[N];
};

// The place in the table of the tensor that a chunk belongs to.
template <int N>
__device__ __forceinline__ int entry_of(const Table<N> &t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= chunk) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// This warp's run of chunks.
template <int N>
__device__ __forceinline__ void run_of(const Table<N> &t, int *from, int *to) {
    const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
    *from = (int)min(w * t.per, (int64_t)t.chunks);
    *to = (int)min((w + 1) * t.per, (int64_t)t.chunks);
}

template <typename T>
__device__ __forceinline__ bool whole_vectors(const T *p, const T *q) {
    return ((reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) & 15u) == 0;
}

// Granules j = 0 .. kRounds - 1 of this thread from element `at` of a tensor of
// n elements: all loads before the first use.  Zeros past the end.
template <typename T>
__device__ __forceinline__ void load_block(const T *src, int64_t at, int64_t n, bool vec, float (&v)[kRounds][kGranule]) {
    if (vec && at + kBlock <= n) {
        constexpr int N = kVec<T>, W = kGranule / N;
        Pack<T, N> raw[kRounds][W];
#pragma unroll
        for (int j = 0; j < kRounds; ++j)
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int64_t i = at + (j * 32 + (int)(threadIdx.x % 32)) * kGranule + w * N;
                if (CHK(i, N, n)) raw[j][w] = *reinterpret_cast<const Pack<T, N> *>(src + i);
            }
#pragma unroll
        for (int j = 0; j < kRounds; ++j)
#pragma unroll
            for (int k = 0; k < kGranule; ++k) v[j][k] = to_f32(raw[j][k / N].e[k % N]);
    } else {
#pragma unroll
        for (int j = 0; j < kRounds; ++j)
#pragma unroll
            for (int k = 0; k < kGranule; ++k) {
                const int64_t i = at + (j * 32 + (int)(threadIdx.x % 32)) * kGranule + k;
                v[j][k] = i < n && CHK(i, 1, n) ? to_f32(src[i]) : 0.0f;
            }
    }
}

// The sum of squares of a thread's elements.  Squares that leave fp32's range
// (all of them small, or one large) are taken of scaled values: below 2^-60 every
// |v| is below 2^-30, and 2^90 brings the smallest subnormal's square to 2^-118;
// from 2^120 on, 2^-70 keeps the largest finite value's below 2^117.
__device__ __forceinline__ double square_sum(const float (&v)[kRounds][kGranule]) {
    auto scaled = [&](float f) {
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kRounds; ++j)
#pragma unroll
            for (int k = 0; k < kGranule; ++k) {
                const float x = v[j][k] * f;
                s[k % 4] = fmaf(x, x, s[k % 4]);
            }
        return (s[0] + s[1]) + (s[2] + s[3]);
    };
    const float s = scaled(1.0f);
    if (s >= 0x1p-60f && s < 0x1p120f) return (double)s;
    if (s < 0x1p-60f) return (double)scaled(0x1p90f) * 0x1p-180;
    return (double)scaled(0x1p-70f) * 0x1p140;               // infinities and NaN stay what they are
}

__device__ __forceinline__ double block_sum(double s) {
    __shared__ double part[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = s;
    __syncthreads();
    s = part[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) s += part[w];
    return s;
}

// The lane's part of a chunk's sum.
template <typename T>
__device__ __forceinline__ double chunk_sum(const Entry &e, int chunk) {
    const T *src = static_cast<const T *>(e.src);
    const bool vec = whole_vectors(src, src);
    double s = 0.0;
#pragma unroll
    for (int b = 0; b < kChunk / kBlock; ++b) {
        const int64_t at = (int64_t)(chunk - e.first) * kChunk + b * kBlock;
        if (at >= e.size) break;
        float v[kRounds][kGranule];
        load_block(src, at, e.size, vec, v);
        s += square_sum(v);
    }
    return s;
}

// sums[blockIdx.x]: of this CTA's warps.
template <int N>
__global__ void __launch_bounds__(kThreads, 4)
clip_sum_kernel(const __grid_constant__ Table<N> t, double *__restrict__ sums) {
    wait_prior_grid();
    allow_next_grid();
    int from, to;
    run_of(t, &from, &to);
    double s = 0.0;
    if (from < to) {
        int at = entry_of(t, from);
        for (int chunk = from; chunk < to; ++chunk) {
            while (at + 1 < t.n && t.e[at + 1].first <= chunk) ++at;
            const Entry &e = t.e[at];
            if (e.dtype == CARBON_F32) s += chunk_sum<float>(e, chunk);
            else if (e.dtype == CARBON_BF16) s += chunk_sum<__nv_bfloat16>(e, chunk);
            else s += chunk_sum<__half>(e, chunk);
        }
    }
    s = block_sum(s);
    if (threadIdx.x == 0) sums[blockIdx.x] = s;
}

// Elements from..to of a tensor of n.  No order to keep here: vectors from the
// first 16-byte boundary on, where source and target have theirs at the same
// elements.
template <typename T>
__device__ __forceinline__ void scale_range(const Entry &e, int64_t from, int64_t to, float factor) {
    const T *src = static_cast<const T *>(e.src);
    T *dst = static_cast<T *>(e.dst);
    constexpr int N = kVec<T>;
    const int off = (int)(reinterpret_cast<uintptr_t>(src) / sizeof(T) % N);
    int64_t head = to;                                    // elements up to here one by one
    if (off == (int)(reinterpret_cast<uintptr_t>(dst) / sizeof(T) % N)) {
        head = from + ((int)(N - (from + off) % N)) % N;
        if (head > to) head = to;
    }
    const int lane = threadIdx.x % 32;
    const int vecs = (int)((to - head) / N);
    const int64_t tail = head + (int64_t)vecs * N;
    constexpr int U = 4;
    const T *in = src + head;
    T *out = dst + head;
    int i = lane;
    for (; i + 32 * (U - 1) < vecs; i += 32 * U) {
        Pack<T, N> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (CHK(head + (i + j * 32) * N, N, e.size)) v[j] = *reinterpret_cast<const Pack<T, N> *>(in + (i + j * 32) * N);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            float f[N];
            widen(v[j], f);
#pragma unroll
            for (int k = 0; k < N; ++k) f[k] *= factor;
            if (CHK(head + (i + j * 32) * N, N, e.size)) store_f32<T, N>(out + (i + j * 32) * N, f);
        }
    }
    for (; i < vecs; i += 32) {
        float f[N];
        if (!CHK(head + i * N, N, e.size)) continue;
        load_f32<T, N>(in + i * N, f);
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] *= factor;
        store_f32<T, N>(out + i * N, f);
    }
    for (int64_t i = from + lane; i < head; i += 32)
        if (CHK(i, 1, e.size)) dst[i] = from_f32<T>(to_f32(src[i]) * factor);
    for (int64_t i = tail + lane; i < to; i += 32)
        if (CHK(i, 1, e.size)) dst[i] = from_f32<T>(to_f32(src[i]) * factor);
}

// sums[0 .. total): every CTA adds them in the same order.  scale: whether the
// tensors are to be scaled; CTA 0 writes the norm where it is not null.
template <int N>
__global__ void __launch_bounds__(kThreads, 4)
clip_scale_kernel(const __grid_constant__ Table<N> t, const double *__restrict__ sums, int total, float *__restrict__ norm,
                  float max_norm, float eps, int scale) {
    wait_prior_grid();
    allow_next_grid();
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < total; i += kThreads) s += sums[i];
    const float n = (float)sqrt(block_sum(s));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    if (!scale) return;
    // 0 / 0 (only zeros) and an infinite bound scale nothing; a NaN norm stays
    const float ratio = n + eps == 0.0f || (max_norm == INFINITY && n == n) ? 1.0f : __fdiv_rn(max_norm, n + eps);
    const float factor = ratio > 1.0f ? 1.0f : ratio;
    int from, to;
    run_of(t, &from, &to);
    if (from >= to) return;
    int at = entry_of(t, to - 1);
    for (int chunk = to - 1; chunk >= from; --chunk) {
        while (t.e[at].first > chunk) --at;
        const Entry &e = t.e[at];
        if (e.src == e.dst && factor == 1.0f) continue;
        const int64_t first = (int64_t)(chunk - e.first) * kChunk, last = min(first + kChunk, e.size);
        if (e.dtype == CARBON_F32) scale_range<float>(e, first, last, factor);
        else if (e.dtype == CARBON_BF16) scale_range<__nv_bfloat16>(e, first, last, factor);
        else scale_range<__half>(e, first, last, factor);
    }
}

// ---- host side ----------------------------------------------------------------

// Chunks are counted in 32 bits.
bool sizes_ok(const int64_t *sizes, int64_t count) {
    if (count < 0 || count > (1ll << 24) || (count > 0 && !sizes)) return false;
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > (1ll << 41)) return false;
        all += (sizes[i] + kChunk - 1) / kChunk;
        if (all >= (1ll << 30)) return false;
    }
    return true;
}

// A table holds at most kFew or kMany tensors that have elements; the sums of as
// many tables as there may be.
int64_t sum_bytes(int64_t count) { return 8 * kCtas * (count <= kFew ? 1 : (count + kMany - 1) / kMany); }

struct Span {
    uintptr_t from, to;
    bool written;
};

// Whether something that is written overlaps anything but itself.
bool overlaps(const void *const *grads, void *const *out, const int64_t *sizes, const int *dtypes, int64_t count) {
    std::vector<Span> v;
    v.reserve((size_t)count * 2);
    for (int64_t i = 0; i < count; ++i) {
        const uintptr_t bytes = (uintptr_t)sizes[i] * dtype_size(dtypes[i]);
        if (bytes == 0) continue;
        const uintptr_t d = reinterpret_cast<uintptr_t>(out[i]), g = reinterpret_cast<uintptr_t>(grads[i]);
        v.push_back({d, d + bytes, true});
        if (g != d) v.push_back({g, g + bytes, false});
    }
    std::sort(v.begin(), v.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
    uintptr_t any = 0, written = 0;
    for (const Span &s : v) {
        if (s.from < (s.written ? any : written)) return true;
        any = std::max(any, s.to);
        if (s.written) written = std::max(written, s.to);
    }
    return false;
}

struct Call {
    float *norm;
    void *const *out;
    const void *const *grads;
    const int64_t *sizes;
    const int *dtypes;
    int64_t count;
    float max_norm, eps;
};

// The tables, in order: all sums before the first scaling.
template <int N>
cudaError_t run_tables(const Call &c, double *sums, cudaStream_t s) {
    Table<N> t;
    int ctas = 0, total = 0, before = 0;                  // of the table at hand, of all tables, of those before it
    auto each_table = [&](auto launch) {
        cudaError_t err = cudaSuccess;
        before = 0;
        for (int64_t i = 0; i < c.count && err == cudaSuccess;) {
            int64_t chunks = 0;
            for (t.n = 0; i < c.count && t.n < N; ++i) {
                if (c.sizes[i] == 0) continue;
                t.e[t.n++] = Entry{c.grads[i], c.out ? c.out[i] : nullptr, c.sizes[i], (int)chunks, c.dtypes[i]};
                chunks += (c.sizes[i] + kChunk - 1) / kChunk;
            }
            if (t.n == 0) break;
            t.chunks = (int)chunks;
            t.per = (int)((chunks + kWarps - 1) / kWarps);
            ctas = (int)((chunks + (int64_t)t.per * (kThreads / 32) - 1) / ((int64_t)t.per * (kThreads / 32)));
            count_launch();
            err = launch();
            before += ctas;
        }
        return err;
    };
    cudaError_t err = each_table([&] {
        return launch_k(clip_sum_kernel<N>, dim3((unsigned)ctas), dim3(kThreads), 0, s, 1, t, sums + before);
    });
    total = before;
    if (err != cudaSuccess) return err;
    if (c.out && total > 0)
        return each_table([&] {
            return launch_k(clip_scale_kernel<N>, dim3((unsigned)ctas), dim3(kThreads), 0, s, 1, t, sums, total,
                            before == 0 ? c.norm : nullptr, c.max_norm, c.eps, 1);
        });
    count_launch();                                       // the norm alone
    return launch_k(clip_scale_kernel<N>, dim3(1), dim3(kThreads), 0, s, 1, t, sums, total, c.norm, c.max_norm, c.eps, 0);
}

}  // namespace

carbon_status_t clip_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_clip_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_clip_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

}  // namespace carbon

using namespace carbon;

extern "C" {

int64_t carbon_clip_grads_workspace(const int64_t *sizes, int64_t count) {
    return sizes_ok(sizes, count) ? sum_bytes(count) : -1;
}

carbon_status_t carbon_clip_grads(float *norm, void *const *out, const void *const *grads, const int64_t *sizes,
                                  const int *dtypes, int64_t count, float max_norm, float eps, void *workspace,
                                  int64_t workspace_bytes, carbon_stream_t stream) try {
    if (!sizes_ok(sizes, count)) return CARBON_ERR_INVALID_ARG;
    if (count > 0 && (!grads || !dtypes)) return CARBON_ERR_INVALID_ARG;
    if (!norm && !out) return CARBON_ERR_INVALID_ARG;
    if (out && (!(max_norm >= 0.0f) || !(eps >= 0.0f))) return CARBON_ERR_INVALID_ARG;
    bool any = false;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != CARBON_F32 && dtypes[i] != CARBON_BF16 && dtypes[i] != CARBON_F16) return CARBON_ERR_INVALID_ARG;
        if (sizes[i] == 0) continue;
        any = true;
        if (!grads[i] || (out && !out[i])) return CARBON_ERR_INVALID_ARG;
    }
    if (any && (!workspace || !aligned16(workspace) || workspace_bytes < sum_bytes(count))) return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, norm)) return CARBON_ERR_MISALIGNED;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] > 0 && !aligned_to(dtype_size(dtypes[i]), grads[i], out ? out[i] : nullptr)) return CARBON_ERR_MISALIGNED;
    if (out && overlaps(grads, out, sizes, dtypes, count)) return CARBON_ERR_INVALID_ARG;
    if (!any && !norm) return CARBON_OK;
    carbon_status_t st = injected_launch_failure();
    if (st != CARBON_OK) return st;
    if ((st = current_device(nullptr, nullptr)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *sums = static_cast<double *>(workspace);

    const Call c = {norm, out, grads, sizes, dtypes, count, max_norm, eps};
    const cudaError_t err = count <= kFew ? run_tables<kFew>(c, sums, s) : run_tables<kMany>(c, sums, s);
    return note_cuda(err);
} catch (...) {
    return CARBON_ERR_INVALID_ARG;        // no memory on the host for the tables
}

}  // extern "C"
