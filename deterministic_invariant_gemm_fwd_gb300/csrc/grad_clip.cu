// grad_clip.cu - the norm of all gradients of a model and their clipping.
//
//   norm = sqrt(sum over tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + eps))
//
// Two kernels over chunks of the tensors, whose addresses travel as kernel
// parameters (no copy to the device; kTensors a launch).  The first sums the
// squares of a chunk per CTA; the second adds the chunks' sums, each CTA for
// itself (a launch and a wait less than a kernel in between), and scales.  It
// takes the chunks from the last to the first, so that it finds in L2 what the
// first kernel read last.
//
// Order: an element's thread and place in its sum depend on its index in its
// tensor alone, not on addresses; a chunk's sum is a tree, the chunks' sums are
// added by index.  fp32 within a thread (64 squares), float64 from there on.
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

constexpr int kThreads = 256, kRounds = 8, kGranule = 8;      // a thread's elements: kRounds granules per block
constexpr int64_t kBlock = (int64_t)kThreads * kRounds * kGranule;     // 16384 elements
constexpr int64_t kMaxChunks = 8192;     // chunks grow beyond this many: the second kernel's CTAs each read every sum
constexpr int kTensors = 256;            // per launch

struct Entry {
    const void *src;
    void *dst;
    int64_t size;
    int first;               // its first chunk
    int dtype;
};
struct Table {
    int n;
    int first, chunks;       // chunks of this table
    int blocks;              // blocks of kBlock elements per chunk
    Entry e[kTensors];
};

__device__ __forceinline__ const Entry &entry_of(const Table &t, int chunk) {
    int lo = 0, hi = t.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (t.e[mid].first <= chunk) lo = mid; else hi = mid - 1;
    }
    return t.e[lo];
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
                const int64_t i = at + ((int64_t)j * kThreads + threadIdx.x) * kGranule + w * N;
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
                const int64_t i = at + ((int64_t)j * kThreads + threadIdx.x) * kGranule + k;
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

template <typename T>
__device__ __forceinline__ double chunk_sum(const Table &t, const Entry &e, int chunk) {
    const T *src = static_cast<const T *>(e.src);
    const bool vec = whole_vectors(src, src);
    double s = 0.0;
    for (int b = 0; b < t.blocks; ++b) {
        const int64_t at = ((int64_t)(chunk - e.first) * t.blocks + b) * kBlock;
        if (at >= e.size) break;
        float v[kRounds][kGranule];
        load_block(src, at, e.size, vec, v);
        s += square_sum(v);
    }
    return s;
}

__global__ void __launch_bounds__(kThreads)
clip_sum_kernel(const __grid_constant__ Table t, double *__restrict__ sums) {
    wait_prior_grid();
    allow_next_grid();
    const int chunk = t.first + (int)blockIdx.x;
    const Entry &e = entry_of(t, chunk);
    double s;
    if (e.dtype == CARBON_F32) s = chunk_sum<float>(t, e, chunk);
    else if (e.dtype == CARBON_BF16) s = chunk_sum<__nv_bfloat16>(t, e, chunk);
    else s = chunk_sum<__half>(t, e, chunk);
    s = block_sum(s);
    if (threadIdx.x == 0) sums[chunk] = s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const Table &t, const Entry &e, int chunk, float factor) {
    const T *src = static_cast<const T *>(e.src);
    T *dst = static_cast<T *>(e.dst);
    if (src == dst && factor == 1.0f) return;
    const bool vec = whole_vectors(src, dst);
    for (int b = 0; b < t.blocks; ++b) {
        const int64_t at = ((int64_t)(chunk - e.first) * t.blocks + b) * kBlock;
        if (at >= e.size) break;
        float v[kRounds][kGranule];
        load_block(src, at, e.size, vec, v);
#pragma unroll
        for (int j = 0; j < kRounds; ++j) {
            const int64_t i = at + ((int64_t)j * kThreads + threadIdx.x) * kGranule;
#pragma unroll
            for (int k = 0; k < kGranule; ++k) v[j][k] *= factor;
            if (vec && at + kBlock <= e.size) {
                constexpr int N = kVec<T>;
#pragma unroll
                for (int w = 0; w < kGranule; w += N) {
                    float f[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) f[k] = v[j][w + k];
                    if (CHK(i + w, N, e.size)) store_f32<T, N>(dst + i + w, f);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kGranule; ++k)
                    if (i + k < e.size && CHK(i + k, 1, e.size)) dst[i + k] = from_f32<T>(v[j][k]);
            }
        }
    }
}

// sums[0 .. total): every CTA adds them in the same order.  scale: whether the
// tensors are to be scaled; CTA 0 writes the norm where it is not null.
__global__ void __launch_bounds__(kThreads)
clip_scale_kernel(const __grid_constant__ Table t, const double *__restrict__ sums, int total, float *__restrict__ norm,
                  float max_norm, float eps, int scale) {
    wait_prior_grid();
    allow_next_grid();
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < total; i += kThreads) s += sums[i];
    const float n = (float)sqrt(block_sum(s));
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    if (!scale) return;
    const float ratio = __fdiv_rn(max_norm, n + eps), factor = ratio > 1.0f ? 1.0f : ratio;     // NaN stays
    for (int i = (int)blockIdx.x; i < t.chunks; i += (int)gridDim.x) {
        const int chunk = t.first + t.chunks - 1 - i;
        const Entry &e = entry_of(t, chunk);
        if (e.dtype == CARBON_F32) chunk_scale<float>(t, e, chunk, factor);
        else if (e.dtype == CARBON_BF16) chunk_scale<__nv_bfloat16>(t, e, chunk, factor);
        else chunk_scale<__half>(t, e, chunk, factor);
    }
}

// ---- host side ----------------------------------------------------------------

// Blocks per chunk, and the number of chunks; false where sizes are invalid.
bool plan_chunks(const int64_t *sizes, int64_t count, int64_t *blocks, int64_t *chunks) {
    if (count < 0 || count > (1ll << 24) || (count > 0 && !sizes)) return false;
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (sizes[i] < 0 || sizes[i] > (1ll << 48)) return false;
        all += (sizes[i] + kBlock - 1) / kBlock;
        if (all > (1ll << 46)) return false;
    }
    *blocks = (all + kMaxChunks - 1) / kMaxChunks;
    if (*blocks < 1) *blocks = 1;
    *chunks = 0;
    for (int64_t i = 0; i < count; ++i) *chunks += (sizes[i] + *blocks * kBlock - 1) / (*blocks * kBlock);
    return *chunks < (1ll << 30) && *blocks < (1ll << 30);
}

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
    int64_t blocks, chunks;
    return plan_chunks(sizes, count, &blocks, &chunks) ? 8 * chunks + 16 : -1;
}

carbon_status_t carbon_clip_grads(float *norm, void *const *out, const void *const *grads, const int64_t *sizes,
                                  const int *dtypes, int64_t count, float max_norm, float eps, void *workspace,
                                  int64_t workspace_bytes, carbon_stream_t stream) try {
    int64_t blocks, chunks;
    if (!plan_chunks(sizes, count, &blocks, &chunks)) return CARBON_ERR_INVALID_ARG;
    if (count > 0 && (!grads || !dtypes)) return CARBON_ERR_INVALID_ARG;
    if (!norm && !out) return CARBON_ERR_INVALID_ARG;
    if (out && (!(max_norm >= 0.0f) || !(eps >= 0.0f))) return CARBON_ERR_INVALID_ARG;
    for (int64_t i = 0; i < count; ++i) {
        if (dtypes[i] != CARBON_F32 && dtypes[i] != CARBON_BF16 && dtypes[i] != CARBON_F16) return CARBON_ERR_INVALID_ARG;
        if (sizes[i] == 0) continue;
        if (!grads[i] || (out && !out[i])) return CARBON_ERR_INVALID_ARG;
    }
    if (chunks > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < 8 * chunks)) return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, norm)) return CARBON_ERR_MISALIGNED;
    for (int64_t i = 0; i < count; ++i)
        if (sizes[i] > 0 && !aligned_to(dtype_size(dtypes[i]), grads[i], out ? out[i] : nullptr)) return CARBON_ERR_MISALIGNED;
    if (out && overlaps(grads, out, sizes, dtypes, count)) return CARBON_ERR_INVALID_ARG;
    if (chunks == 0 && !norm) return CARBON_OK;
    carbon_status_t st = injected_launch_failure();
    if (st != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    double *sums = static_cast<double *>(workspace);

    // the tables, in order: all sums before the first scaling
    Table t;
    auto each_table = [&](auto launch) {
        int64_t i = 0;
        int first = 0;
        cudaError_t err = cudaSuccess;
        do {
            t.n = 0;
            t.first = first;
            t.blocks = (int)blocks;
            for (; i < count && t.n < kTensors; ++i) {
                if (sizes[i] == 0) continue;
                t.e[t.n++] = Entry{grads[i], out ? out[i] : nullptr, sizes[i], first, dtypes[i]};
                first += (int)((sizes[i] + blocks * kBlock - 1) / (blocks * kBlock));
            }
            t.chunks = first - t.first;
            err = launch();
        } while (err == cudaSuccess && i < count);
        return err;
    };
    cudaError_t err = each_table([&] {
        if (t.chunks == 0) return cudaSuccess;
        count_launch();
        return launch_k(clip_sum_kernel, dim3((unsigned)t.chunks), dim3(kThreads), 0, s, 1, t, sums);
    });
    auto scale = [&] {
        const int grid = !out || t.chunks == 0 ? 1 : std::min(t.chunks, sms * 4);
        count_launch();
        return launch_k(clip_scale_kernel, dim3((unsigned)grid), dim3(kThreads), 0, s, 1, t, sums, (int)chunks,
                        t.first == 0 ? norm : nullptr, max_norm, eps, out ? 1 : 0);
    };
    if (err == cudaSuccess) err = out ? each_table(scale) : (t.first = 0, scale());
    return note_cuda(err);
} catch (...) {
    return CARBON_ERR_INVALID_ARG;        // no memory on the host for the tables
}

}  // extern "C"
