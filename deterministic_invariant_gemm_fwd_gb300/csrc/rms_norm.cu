// rms_norm.cu - root-mean-square norm of a residual stream, its 8-bit
// checkpoint, and the gradients.
//
//   h = x + residual,  rstd = 1 / sqrt(mean(h^2) + eps),  n = h * rstd,  y = n * gamma
//   codes = round(n * (127 / max|n|)),  scales = max|n| / 127
//   dx = rstd * (gamma*dy - n * mean(gamma*dy*n)) + dh,  dgamma = sum_m dy * n
//
// Bound: memory.  A group of threads (1, 4, 8 or 16 warps, by the
// row's length) takes a row at a time: each of its threads has up to kMaxHold
// elements, the group reduces and writes.  The forward pass reads a row once,
// into registers.  The gradient, and the forward pass where 16-byte vectors do
// not fit the rows, read them through a ring in shared memory that bulk copies
// fill some rows ahead (held in registers, the gradient's rows arrived one at a
// time: 97 us for 8192 x 4096 bf16).  A copy takes the 16-byte aligned bytes
// around a row, so that odd rows are fetched as fast as aligned ones.  Rows
// too long for a group are read again for each pass.  The order of a row's
// sums depends on D, the dtype, the alignment of the tensors and (fp32 rows
// whose ring holds two tensors but not three) the presence of dh alone.
//
// Measured cold, bf16: forward with residual and 8-bit rows, 8192 x 768: 11 us;
// 8192 x 4096: 45 us, the bytes at the rate of a copy (6.7 TB/s).  Gradient
// 15 us and 55 us (a copy's rate: 40).
// Rows of 1001 elements, 8192 of them: 24.5 and 25 us.  dgamma's second kernel:
// 7 us, a launch and one dependent read of the partial rows.
//
// dgamma: a group takes the rows g, g + groups, ... and adds its columns'
// terms in registers; the groups' sums are added per CTA in group order, then
// over the CTAs in order by a second kernel.
#include "bounds.cuh"
#include "device_sync.cuh"
#include "rowvec.cuh"
#include "tcgen05.cuh"

#include <type_traits>

namespace carbon {
namespace {

__device__ unsigned int g_norm_status = 0;
#define CHK(idx, len, n) in_bounds(&g_norm_status, (int64_t)(idx), (int64_t)(len), (int64_t)(n))

constexpr int kMaxHold = 32;             // fp32 elements of a row that a thread holds
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

// Sum over the G threads of a group; every thread receives it.  buf: one
// float per warp of the group.  The value is the warps' butterfly sums added
// in warp order.
template <int G>
__device__ __forceinline__ float group_sum(float v, float *buf) {
    v = warp_sum(v);
    if constexpr (G == 32) {
        return v;
    } else {
        __syncthreads();
        if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
        __syncthreads();
        const int w0 = threadIdx.x / G * (G / 32);
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) s += buf[w0 + w];
        return s;
    }
}

template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t *buf) {
    v = warp_max_u32(v);
    if constexpr (G == 32) {
        return v;
    } else {
        __syncthreads();
        if (threadIdx.x % 32 == 0) buf[threadIdx.x / 32] = v;
        __syncthreads();
        const int w0 = threadIdx.x / G * (G / 32);
        uint32_t s = 0u;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) s = max(s, buf[w0 + w]);
        return s;
    }
}

// Bits of |v|: ordered like the magnitudes, with NaN above infinity.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale of a row's codes and the factor that makes them, from the bits
// of the row's largest magnitude.
__device__ __forceinline__ void code_scale(uint32_t top_bits, float *scale, float *factor) {
    const float top = __uint_as_float(top_bits);
    if (top_bits >= 0x7f800000u) {                        // infinity or NaN
        *scale = __uint_as_float(0x7fc00000u);
        *factor = 0.0f;
    } else if (top < kTiny) {
        *scale = 0.0f;
        *factor = 0.0f;
    } else {
        *scale = __fdiv_rn(top, 127.0f);
        *factor = __fdiv_rn(127.0f, top);
    }
}

__device__ __forceinline__ int8_t code_of(float n, float factor) {
    // a zero factor gives code 0 also for infinities and NaN
    return factor == 0.0f ? (int8_t)0 : (int8_t)max(-127, min(127, __float2int_rn(n * factor)));
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t *p, const int8_t (&c)[N]) {
    Pack<int8_t, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i) v.e[i] = c[i];
    *reinterpret_cast<Pack<int8_t, N> *>(p) = v;
}

// ---- rows through shared memory ------------------------------------------------

// A tensor of rows of row_bytes bytes.
struct Rows {
    const uint8_t *base;
    int64_t row_bytes, bytes;
};

__host__ __device__ inline uint32_t row_slot(int64_t row_bytes) {       // bytes of a row's place, any alignment
    return (uint32_t)((row_bytes + 15) / 16 * 16 + 16);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

// Starts the copies of row m of every tensor into a stage, by one warp; the
// row lies at its address modulo 16 in its place.  The bulk copies take whole
// 16-byte pieces inside the tensor; bytes of a piece that reaches past either
// end of the tensor are copied here.
template <int K>
__device__ __forceinline__ void start_row(const Rows (&t)[K], int count, int64_t m, uint8_t *stage, uint32_t slot,
                                          uint32_t bar) {
    const int lane = threadIdx.x % 32;
    uint32_t bytes = 0u;
    auto range = [&](const Rows &r, const uint8_t **b0, const uint8_t **b1, const uint8_t **lo, const uint8_t **hi) {
        *b0 = r.base + m * r.row_bytes;
        *b1 = *b0 + r.row_bytes;
        *lo = reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(*b0) & ~(uintptr_t)15);
        *hi = reinterpret_cast<const uint8_t *>((reinterpret_cast<uintptr_t>(*b1) + 15) & ~(uintptr_t)15);
        if (*lo < r.base) *lo += 16;
        if (*hi > r.base + r.bytes) *hi -= 16;
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (k >= count) break;
        const uint8_t *b0, *b1, *lo, *hi;
        range(t[k], &b0, &b1, &lo, &hi);
        if (lo > b0 || hi < b1) {                         // only in the tensor's first and last rows
            uint8_t *place = stage + k * slot + (reinterpret_cast<uintptr_t>(b0) & 15u);
            for (const uint8_t *b = b0 + lane; b < (lo < b1 ? lo : b1); b += 32) place[b - b0] = *b;
            for (const uint8_t *b = (hi > b0 ? hi : b0) + lane; b < b1; b += 32)
                if (b >= lo) place[b - b0] = *b;
            // the stage's next row may come here by a bulk copy: ordered after
            // these writes
            fence_proxy_async_smem();
        }
        if (hi > lo) bytes += (uint32_t)(hi - lo);
    }
    __syncwarp();
    if (lane == 0) {
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (k >= count) break;
            const uint8_t *b0, *b1, *lo, *hi;
            range(t[k], &b0, &b1, &lo, &hi);
            if (hi > lo)                                  // the row's own address modulo 16 is kept
                bulk_load(smem_addr(stage + k * slot) + (lo > b0 ? 16u : 0u), lo, (uint32_t)(hi - lo), bar);
        }
    }
}

// Where row m of tensor k lies in a stage.
template <typename E>
__device__ __forceinline__ const E *staged(const uint8_t *stage, uint32_t slot, int k, const Rows &t, int64_t m) {
    return reinterpret_cast<const E *>(stage + k * slot + (reinterpret_cast<uintptr_t>(t.base + m * t.row_bytes) & 15u));
}

template <int G>
__device__ __forceinline__ void group_sync() {
    if constexpr (G == 32) __syncwarp();
    else __syncthreads();
}

// gamma behind the ring, for the CTA's life (from global memory, its loads were
// what the warps waited for most).
template <typename T>
__device__ __forceinline__ const T *stage_gamma(uint8_t *at, const T *gamma, int D) {
    T *g = reinterpret_cast<T *>(at);
    for (int j = threadIdx.x; j < D; j += blockDim.x) g[j] = gamma[j];
    __syncthreads();
    return g;
}

// Waits for a stage; a wait that gives up is recorded, and the later ones are
// skipped (the rows' results are then meaningless, but the kernel ends).
__device__ __forceinline__ bool wait_stage(uint64_t *bar, uint32_t parity, bool ok) {
    if (!ok) return false;
    if (__all_sync(0xffffffffu, mbar_wait(smem_addr(bar), parity))) return true;
    atomicExch(&g_norm_status, (unsigned)CARBON_ERR_TIMEOUT);
    return false;
}

// CTAs of G threads for G > 32 (one group), of 8 warps (8 groups) for G = 32.
template <int G>
constexpr int kRingThreads = G == 32 ? 256 : G;
constexpr int kMaxStages = 4;

template <typename T>
struct FwdArgs {
    T *y, *h_out;
    float *rstd;
    int8_t *codes;
    float *scales;
    const T *x, *residual, *gamma;
    int64_t M, D;
    float eps;
};

// G threads per row, N elements per vector, H vectors per thread.
template <typename T, int G, int N, int H>
__global__ void __launch_bounds__(G > 128 ? G : 128)
norm_fwd_kernel(const FwdArgs<T> a) {
    constexpr int kThreads = G > 128 ? G : 128, kRows = kThreads / G;
    __shared__ float buf[kThreads / 32];
    wait_prior_grid();
    allow_next_grid();
    const int64_t m0 = (int64_t)blockIdx.x * kRows + threadIdx.x / G;
    const bool live = m0 < a.M;
    const int64_t m = live ? m0 : a.M - 1;                // idle groups repeat the last row, unstored
    const int t = threadIdx.x % G;
    const int nvec = (int)(a.D / N);
    const int64_t row = m * a.D;

    float h[H][N];
    float ss = 0.0f;
#pragma unroll
    for (int u = 0; u < H; ++u) {
        const int i = t + G * u;
        if (i < nvec && CHK(row + i * N, N, a.M * a.D)) {
            load_f32<T, N>(a.x + row + i * N, h[u]);
        } else {
#pragma unroll
            for (int k = 0; k < N; ++k) h[u][k] = 0.0f;
        }
    }
    if (a.residual) {
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec) {
                float r[N];
                load_f32<T, N>(a.residual + row + i * N, r);
#pragma unroll
                for (int k = 0; k < N; ++k) h[u][k] += r[k];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < H; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k) ss = fmaf(h[u][k], h[u][k], ss);
    ss = group_sum<G>(ss, buf);
    const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.D) + a.eps);

    if (live) {
        if (a.rstd && t == 0) a.rstd[m] = rstd;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec) {
                if (a.h_out) store_f32<T, N>(a.h_out + row + i * N, h[u]);
                float g[N], y[N];
                load_f32<T, N>(a.gamma + i * N, g);
#pragma unroll
                for (int k = 0; k < N; ++k) y[k] = h[u][k] * rstd * g[k];
                store_f32<T, N>(a.y + row + i * N, y);
            }
        }
    }
    if (a.codes) {                                        // the same for the whole grid
        uint32_t top = 0u;
#pragma unroll
        for (int u = 0; u < H; ++u)
#pragma unroll
            for (int k = 0; k < N; ++k) top = max(top, magnitude(h[u][k] * rstd));
        top = group_max<G>(top, reinterpret_cast<uint32_t *>(buf));
        float scale, factor;
        code_scale(top, &scale, &factor);
        if (live) {
            if (t == 0) a.scales[m] = scale;
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int i = t + G * u;
                if (i < nvec) {
                    int8_t c[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) c[k] = code_of(h[u][k] * rstd, factor);
                    store_codes<N>(a.codes + row + i * N, c);
                }
            }
        }
    }
}

// Rows that 16-byte vectors do not fit: through the ring, element by element.
template <typename T, int G, int H>
__global__ void __launch_bounds__(kRingThreads<G>)
norm_fwd_ring_kernel(const FwdArgs<T> a, const int stages) {
    constexpr int kThreads = kRingThreads<G>, kRows = kThreads / G;
    __shared__ float buf[kThreads / 32];
    __shared__ __align__(8) uint64_t bars[kRows][kMaxStages];
    extern __shared__ __align__(16) uint8_t ring[];
    const int t = threadIdx.x % G, group = threadIdx.x / G;
    const uint32_t slot = row_slot(a.D * sizeof(T));
    const int count = a.residual ? 2 : 1;
    uint8_t *mine = ring + (size_t)group * stages * count * slot;
    const Rows rows[2] = {
        {reinterpret_cast<const uint8_t *>(a.x), a.D * (int64_t)sizeof(T), a.M * a.D * (int64_t)sizeof(T)},
        {reinterpret_cast<const uint8_t *>(a.residual), a.D * (int64_t)sizeof(T), a.M * a.D * (int64_t)sizeof(T)}};
    if (t == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(smem_addr(&bars[group][s]), 1);
        fence_mbar_init();
    }
    group_sync<G>();
    wait_prior_grid();
    allow_next_grid();
    const int64_t first = (int64_t)blockIdx.x * kRows + group, step = (int64_t)gridDim.x * kRows;
    if (t < 32)
        for (int s = 0; s < stages && first + s * step < a.M; ++s)
            start_row(rows, count, first + s * step, mine + s * count * slot, slot, smem_addr(&bars[group][s]));
    const T *gamma = stage_gamma(ring + (size_t)kRows * stages * count * slot, a.gamma, (int)a.D);
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    const int D = (int)a.D;
    for (int64_t m = first; m < a.M; m += step) {
        ok = wait_stage(&bars[group][s], ph, ok);
        const uint8_t *stage = mine + s * count * slot;
        const T *x = staged<T>(stage, slot, 0, rows[0], m), *res = staged<T>(stage, slot, 1, rows[1], m);   // res: if there is one
        float h[H], ss = 0.0f;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int j = t + G * u;
            h[u] = j < D ? to_f32(x[j]) : 0.0f;
            if (j < D && a.residual) h[u] += to_f32(res[j]);
            ss = fmaf(h[u], h[u], ss);
        }
        ss = group_sum<G>(ss, buf);
        group_sync<G>();                                  // the row has been read
        if (ok && t < 32 && m + stages * step < a.M)
            start_row(rows, count, m + stages * step, mine + s * count * slot, slot, smem_addr(&bars[group][s]));
        if (++s == stages) { s = 0; ph ^= 1u; }

        const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.D) + a.eps);
        const int64_t row = m * a.D;
        if (a.rstd && t == 0) a.rstd[m] = rstd;
        uint32_t top = 0u;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int j = t + G * u;
            if (j < D && CHK(row + j, 1, a.M * a.D)) {
                if (a.h_out) a.h_out[row + j] = from_f32<T>(h[u]);
                a.y[row + j] = from_f32<T>(h[u] * rstd * to_f32(gamma[j]));
            }
            top = max(top, magnitude(h[u] * rstd));
        }
        if (a.codes) {
            top = group_max<G>(top, reinterpret_cast<uint32_t *>(buf));
            float scale, factor;
            code_scale(top, &scale, &factor);
            if (t == 0) a.scales[m] = scale;
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int j = t + G * u;
                if (j < D) a.codes[row + j] = code_of(h[u] * rstd, factor);
            }
            group_sync<G>();
        }
    }
}

// Rows that do not fit a group's registers: a CTA per row, the row read again
// for each pass.  The last pass alone writes, each thread the elements that it
// reads, so that y or h_out may lie over x or residual.
template <typename T>
__global__ void __launch_bounds__(512)
norm_fwd_long_kernel(const FwdArgs<T> a) {
    __shared__ float buf[16];
    wait_prior_grid();
    allow_next_grid();
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t row = m * a.D;
        auto h_at = [&](int64_t j) {
            return to_f32(a.x[row + j]) + (a.residual ? to_f32(a.residual[row + j]) : 0.0f);
        };
        float ss = 0.0f;
        for (int64_t j = threadIdx.x; j < a.D; j += 512) {
            const float h = h_at(j);
            ss = fmaf(h, h, ss);
        }
        ss = group_sum<512>(ss, buf);
        const float rstd = rsqrtf(__fdiv_rn(ss, (float)a.D) + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[m] = rstd;
        float factor = 0.0f;
        if (a.codes) {
            uint32_t top = 0u;
            for (int64_t j = threadIdx.x; j < a.D; j += 512) top = max(top, magnitude(h_at(j) * rstd));
            top = group_max<512>(top, reinterpret_cast<uint32_t *>(buf));
            float scale;
            code_scale(top, &scale, &factor);
            if (threadIdx.x == 0) a.scales[m] = scale;
        }
        for (int64_t j = threadIdx.x; j < a.D; j += 512) {
            const float h = h_at(j);
            if (a.h_out) a.h_out[row + j] = from_f32<T>(h);
            a.y[row + j] = from_f32<T>(h * rstd * to_f32(a.gamma[j]));
            if (a.codes) a.codes[row + j] = code_of(h * rstd, factor);
        }
    }
}

template <typename T>
struct BwdArgs {
    T *dx, *y_out;
    float *partial;                       // [CTAs][D], or null (no dgamma)
    const T *dy, *h;
    const int8_t *codes;
    const float *scales, *rstd;
    const T *gamma, *dh;
    int64_t M, D;
};

// A group's rows come through its ring: n's source, dy and dh.  n and gamma*dy
// stay in registers between the sum over the row and dx.
template <typename T, int G, int N, int H, bool CODES>
__global__ void __launch_bounds__(kRingThreads<G>, G == 128 ? 4 : G == 512 ? 1 : 2)
norm_bwd_kernel(const BwdArgs<T> a, const int stages) {
    constexpr int kThreads = kRingThreads<G>, kRows = kThreads / G;
    using Source = typename std::conditional<CODES, int8_t, T>::type;
    __shared__ float buf[kThreads / 32];
    __shared__ __align__(8) uint64_t bars[kRows][kMaxStages];
    extern __shared__ __align__(16) uint8_t ring[];       // afterwards [kRows][D] of dgamma, kRows > 1
    const int t = threadIdx.x % G, group = threadIdx.x / G;
    const int D = (int)a.D, nvec = D / N;
    const uint32_t slot = row_slot(a.D * sizeof(T));
    const int count = a.dh ? 3 : 2;
    uint8_t *mine = ring + (size_t)group * stages * count * slot;
    const int64_t wide = a.D * (int64_t)sizeof(T);
    const Rows rows[3] = {{CODES ? reinterpret_cast<const uint8_t *>(a.codes) : reinterpret_cast<const uint8_t *>(a.h),
                           a.D * (int64_t)sizeof(Source), a.M * a.D * (int64_t)sizeof(Source)},
                          {reinterpret_cast<const uint8_t *>(a.dy), wide, a.M * wide},
                          {reinterpret_cast<const uint8_t *>(a.dh), wide, a.M * wide}};
    if (t == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(smem_addr(&bars[group][s]), 1);
        fence_mbar_init();
    }
    group_sync<G>();
    wait_prior_grid();
    allow_next_grid();
    const int64_t first = (int64_t)blockIdx.x * kRows + group, step = (int64_t)gridDim.x * kRows;
    if (t < 32)
        for (int s = 0; s < stages && first + s * step < a.M; ++s)
            start_row(rows, count, first + s * step, mine + s * count * slot, slot, smem_addr(&bars[group][s]));
    const T *gamma = stage_gamma(ring + (size_t)kRows * stages * count * slot, a.gamma, D);
    float dg[H][N];
#pragma unroll
    for (int u = 0; u < H; ++u)
#pragma unroll
        for (int k = 0; k < N; ++k) dg[u][k] = 0.0f;
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    // the next row's statistics are loaded a row ahead
    float next_rstd = first < a.M ? a.rstd[first] : 0.0f, next_scale = CODES && first < a.M ? a.scales[first] : 0.0f;
    for (int64_t m = first; m < a.M; m += step) {
        const float rstd = next_rstd, factor = CODES ? next_scale : rstd;
        if (m + step < a.M) {
            next_rstd = a.rstd[m + step];
            if (CODES) next_scale = a.scales[m + step];
        }
        ok = wait_stage(&bars[group][s], ph, ok);
        const uint8_t *stage = mine + s * count * slot;
        const Source *src = staged<Source>(stage, slot, 0, rows[0], m);
        const T *dys = staged<T>(stage, slot, 1, rows[1], m), *dhs = staged<T>(stage, slot, 2, rows[2], m);   // dhs: if there is one
        const int64_t row = m * a.D;
        float n[H][N], gdy[H][N], dot = 0.0f;
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec && CHK(row + i * N, N, a.M * a.D)) {
                float g[N], dy[N];
                load_f32<T, N>(gamma + i * N, g);
                load_f32<Source, N>(src + i * N, n[u]);
                load_f32<T, N>(dys + i * N, dy);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    n[u][k] *= factor;
                    gdy[u][k] = dy[k] * g[k];
                    dg[u][k] = fmaf(dy[k], n[u][k], dg[u][k]);
                    dot = fmaf(gdy[u][k], n[u][k], dot);
                }
                if (a.y_out) {
                    float y[N];
#pragma unroll
                    for (int k = 0; k < N; ++k) y[k] = n[u][k] * g[k];
                    store_f32<T, N>(a.y_out + row + i * N, y);
                }
            }
        }
        dot = group_sum<G>(dot, buf);
        const float mean = __fdiv_rn(dot, (float)a.D);
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec && CHK(row + i * N, N, a.M * a.D)) {
                float d[N];
                if (a.dh) {
                    load_f32<T, N>(dhs + i * N, d);
                } else {
#pragma unroll
                    for (int k = 0; k < N; ++k) d[k] = 0.0f;
                }
#pragma unroll
                for (int k = 0; k < N; ++k) d[k] = fmaf(rstd, fmaf(-n[u][k], mean, gdy[u][k]), d[k]);
                store_f32<T, N>(a.dx + row + i * N, d);
            }
        }
        group_sync<G>();                                  // the stage has been read
        if (ok && t < 32 && m + stages * step < a.M)
            start_row(rows, count, m + stages * step, mine + s * count * slot, slot, smem_addr(&bars[group][s]));
        if (++s == stages) { s = 0; ph ^= 1u; }
    }
    if (!a.partial) return;
    float *out = a.partial + (int64_t)blockIdx.x * a.D;
    if constexpr (kRows == 1) {
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec)
#pragma unroll
                for (int k = 0; k < N; ++k) out[i * N + k] = dg[u][k];
        }
    } else {
        float *group_part = reinterpret_cast<float *>(ring);
        __syncthreads();                                  // every group is done with its ring
#pragma unroll
        for (int u = 0; u < H; ++u) {
            const int i = t + G * u;
            if (i < nvec)
#pragma unroll
                for (int k = 0; k < N; ++k) group_part[group * D + i * N + k] = dg[u][k];
        }
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += kThreads) {
            float sum = 0.0f;
#pragma unroll
            for (int g = 0; g < kRows; ++g) sum += group_part[g * D + j];
            out[j] = sum;
        }
    }
}

// Long rows: a CTA per row; dgamma's terms are added into the CTA's own
// partial row, which only its threads touch.
template <typename T>
__global__ void __launch_bounds__(512)
norm_bwd_long_kernel(const BwdArgs<T> a) {
    __shared__ float buf[16];
    wait_prior_grid();
    allow_next_grid();
    float *out = a.partial ? a.partial + (int64_t)blockIdx.x * a.D : nullptr;
    bool first = true;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const int64_t row = m * a.D;
        const float rstd = a.rstd[m], factor = a.h ? rstd : a.scales[m];
        auto n_at = [&](int64_t j) {
            return (a.h ? to_f32(a.h[row + j]) : (float)a.codes[row + j]) * factor;
        };
        float dot = 0.0f;
        for (int64_t j = threadIdx.x; j < a.D; j += 512) {
            const float n = n_at(j), dy = to_f32(a.dy[row + j]), g = to_f32(a.gamma[j]);
            if (a.y_out) a.y_out[row + j] = from_f32<T>(n * g);
            if (out) out[j] = first ? dy * n : fmaf(dy, n, out[j]);
            dot = fmaf(dy * g, n, dot);
        }
        first = false;
        dot = group_sum<512>(dot, buf);
        const float mean = __fdiv_rn(dot, (float)a.D);
        for (int64_t j = threadIdx.x; j < a.D; j += 512) {
            const float gdy = to_f32(a.dy[row + j]) * to_f32(a.gamma[j]);
            const float d = a.dh ? to_f32(a.dh[row + j]) : 0.0f;
            a.dx[row + j] = from_f32<T>(fmaf(rstd, fmaf(-n_at(j), mean, gdy), d));
        }
    }
}

// dgamma[j] = sum over the CTAs' partial rows: 32 threads per column take
// every 32nd row, in order, and their sums are added in thread order.
constexpr int kGammaRows = 32;

template <typename T>
__global__ void __launch_bounds__(32 * kGammaRows)
dgamma_kernel(T *__restrict__ dgamma, const float *__restrict__ partial, int rows, int64_t D) {
    __shared__ float part[kGammaRows][33];
    wait_prior_grid();
    allow_next_grid();
    const int c = threadIdx.x % 32, r = threadIdx.x / 32;
    const int64_t j = (int64_t)blockIdx.x * 32 + c;
    float s = 0.0f;
    if (j < D) {
#pragma unroll 10
        for (int i = r; i < rows; i += kGammaRows)
            if (CHK((int64_t)i * D + j, 1, rows * D)) s += partial[(int64_t)i * D + j];
    }
    part[r][c] = s;
    __syncthreads();
    if (r == 0 && j < D) {
#pragma unroll
        for (int i = 1; i < kGammaRows; ++i) s += part[i][c];
        dgamma[j] = from_f32<T>(s);
    }
}

// The rows as one line of M * D elements, N at a time; a vector may reach into
// the next row.
template <typename T, int N>
__global__ void __launch_bounds__(256)
norm_expand_kernel(T *__restrict__ out, const int8_t *__restrict__ codes, const float *__restrict__ scales,
                   const T *__restrict__ gamma, int64_t M, int64_t D) {
    wait_prior_grid();
    allow_next_grid();
    const int64_t total = M * D, nvec = (total + N - 1) / N;
    for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < nvec; v += (int64_t)gridDim.x * 256) {
        const int64_t i = v * N;
        // 32-bit division where it will do
        int64_t m = total <= 0xffffffffll ? (int64_t)((uint32_t)i / (uint32_t)D) : i / D;
        int64_t col = i - m * D;
        if (i + N <= total && CHK(i, N, total)) {
            float f[N];
            load_f32<int8_t, N>(codes + i, f);
            float s = scales[m];
            if (col + N <= D) {                           // within a row
#pragma unroll
                for (int k = 0; k < N; ++k) f[k] *= s;
                if (gamma)
#pragma unroll
                    for (int k = 0; k < N; ++k) f[k] *= to_f32(gamma[col + k]);
            } else {
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    f[k] *= s;
                    if (gamma) f[k] *= to_f32(gamma[col]);
                    if (++col == D && k + 1 < N) {
                        col = 0;
                        s = scales[++m];
                    }
                }
            }
            store_f32<T, N>(out + i, f);
        } else {
            for (int64_t j = i; j < total; ++j) {
                const float f = (float)codes[j] * scales[j / D];
                out[j] = from_f32<T>(gamma ? f * to_f32(gamma[j % D]) : f);
            }
        }
    }
}

// ---- host side ----------------------------------------------------------------

bool sizes_ok(int64_t M, int64_t D) {
    int64_t t;
    return M >= 0 && D >= 0 && D < 0x7fffffff && M < 0x7fffffff && !__builtin_mul_overflow(M, D, &t) &&
           !__builtin_mul_overflow(t, (int64_t)8, &t);
}

bool dtype_ok(int dtype) { return dtype == CARBON_F32 || dtype == CARBON_BF16 || dtype == CARBON_F16; }

// Calls f(G, H) for the group that holds a row of D elements: G threads with H
// vectors of N each, at most kMaxHold elements per thread.  Returns false
// where none does.  The gradient, which holds three values per element, takes
// rows of vectors at half as many elements per thread where more than a warp
// shares a row and a larger group is left (bf16, the gradient with dh: 8192 x
// 4096 58 us with 256 threads, 72 with 128; 8192 x 2048 37 us with 128, 44 with
// 256; 4096 x 8192 61 us with 512, 114 with 256).
template <int N, bool GRAD, typename F>
bool with_group(int64_t D, F &&f) {
    using std::integral_constant;
    const int64_t nvec = D / N;
    constexpr int H = kMaxHold / N, kMiddle = GRAD && N > 1 ? H / 2 : H;
    auto held = [&](auto g, auto most) {                  // fewest vectors per thread that hold the row
        constexpr int G = g(), kMost = most();
        if (nvec > G * kMost) return false;
        auto with = [&](auto h) {
            if constexpr (h() <= kMost) f(g, h);
        };
        if constexpr (H == 8) {                           // fp32 vectors
            if (nvec <= G * 2) with(integral_constant<int, 2>());
            else if (nvec <= G * 4) with(integral_constant<int, 4>());
            else if (nvec <= G * 6) with(integral_constant<int, 6>());
            else with(integral_constant<int, 8>());
        } else if constexpr (H == 4) {
            if (nvec <= G) with(integral_constant<int, 1>());
            else if (nvec <= G * 2) with(integral_constant<int, 2>());
            else if (nvec <= G * 3) with(integral_constant<int, 3>());
            else with(integral_constant<int, 4>());
        } else {
            if (nvec <= G * (H / 4)) with(integral_constant<int, H / 4>());
            else with(integral_constant<int, H>());
        }
        return true;
    };
    constexpr integral_constant<int, H> all;
    constexpr integral_constant<int, kMiddle> middle;
    if (held(integral_constant<int, 32>(), all) || held(integral_constant<int, 128>(), middle)) return true;
    if constexpr (kMiddle < H)
        if (held(integral_constant<int, 256>(), middle)) return true;
    return held(integral_constant<int, 512>(), all);
}

// The ring of a kernel with groups of G threads: as many stages as leave room
// for two CTAs per SM of 8 warps, four of 4 warps or one of 16 (more CTAs
// rather than more stages: one CTA's warps work while another's wait; but three
// CTAs of 8 warps with two stages took 70 us where two with four take 58), but
// at least two.  bytes: one stage of all the CTA's groups; gamma: its bytes, behind
// them.  0 where two stages do not fit.
constexpr int64_t kSharedMost = 225 * 1024;

template <int G>
int ring_stages(int64_t bytes, int64_t gamma) {
    int s = (int)(((G == 32 || G == 256 ? 110 * 1024 : G == 128 ? 54 * 1024 : kSharedMost) - gamma) / bytes);
    if (s < 2) s = 2;
    if (s > kMaxStages) s = kMaxStages;
    return s * bytes + gamma <= kSharedMost ? s : 0;
}

// CTAs of the kernels with a ring: as many as run at once, and no more partial
// rows of dgamma than that.
constexpr int kRingCtas = 152 * 4;
int ring_ctas(int64_t M, int rows_per_cta, int64_t smem) {
    const int64_t per_sm = kSharedMost / (smem + 2048) < 4 ? kSharedMost / (smem + 2048) : 4;
    const int64_t want = (M + rows_per_cta - 1) / rows_per_cta, most = 152 * (per_sm > 1 ? per_sm : 1);
    return (int)(want < most ? want : most);
}

template <typename Kern>
cudaError_t allow_shared(Kern kern, int64_t smem) {
    return smem > 48 * 1024 - 2048 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)
                                   : cudaSuccess;
}

template <typename T, int N>
cudaError_t launch_fwd(const FwdArgs<T> &a, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    bool fits = true;
    count_launch();
    const bool held = with_group<N, false>(a.D, [&](auto g, auto h) {
        constexpr int G = g(), H = h();
        if constexpr (N > 1) {
            constexpr int kRows = G > 128 ? 1 : 128 / G;
            err = launch_k(norm_fwd_kernel<T, G, N, H>, dim3((unsigned)((a.M + kRows - 1) / kRows)),
                           dim3(G > 128 ? G : 128), 0, s, 1, a);
        } else {
            constexpr int kRows = kRingThreads<G> / G;
            const int64_t stage = (int64_t)kRows * (a.residual ? 2 : 1) * row_slot(a.D * sizeof(T));
            const int stages = ring_stages<G>(stage, a.D * (int64_t)sizeof(T));
            fits = stages > 0;                            // else fp32 rows too long for two stages
            if (!fits) return;
            auto kern = norm_fwd_ring_kernel<T, G, H>;
            const int64_t smem = stages * stage + a.D * (int64_t)sizeof(T);
            err = allow_shared(kern, smem);
            if (err == cudaSuccess)
                err = launch_k(kern, dim3((unsigned)ring_ctas(a.M, kRows, smem)), dim3(kRingThreads<G>), (size_t)smem, s,
                               1, a, stages);
        }
    });
    if (!held || !fits)
        err = launch_k(norm_fwd_long_kernel<T>, dim3((unsigned)(a.M < 65535 ? a.M : 65535)), dim3(512), 0, s, 1, a);
    return err;
}

template <typename T>
cudaError_t run_fwd(const FwdArgs<T> &a, cudaStream_t s) {
    constexpr int N = kVec<T>;
    const bool vec = a.D % N == 0 && aligned16(a.x) && aligned16(a.y) && aligned16(a.gamma) &&
                     aligned16(a.residual) && aligned16(a.h_out) &&
                     reinterpret_cast<uintptr_t>(a.codes) % N == 0;
    return vec ? launch_fwd<T, N>(a, s) : launch_fwd<T, 1>(a, s);
}

template <typename T, int N, bool CODES>
cudaError_t launch_bwd(const BwdArgs<T> &a, T *dgamma, cudaStream_t s) {
    cudaError_t err = cudaSuccess;
    int ctas = 0;
    bool held = with_group<N, true>(a.D, [&](auto g, auto h) {
        constexpr int G = g(), H = h(), kRows = kRingThreads<G> / G;
        const int64_t stage = (int64_t)kRows * (a.dh ? 3 : 2) * row_slot(a.D * sizeof(T));
        const int stages = ring_stages<G>(stage, a.D * (int64_t)sizeof(T));
        if (stages == 0) return;                          // fp32 rows too long for two stages: the long kernel
        int64_t smem = stages * stage + a.D * (int64_t)sizeof(T);
        const int64_t parts = kRows > 1 ? (int64_t)kRows * a.D * (int64_t)sizeof(float) : 0;
        if (smem < parts) smem = parts;
        ctas = ring_ctas(a.M, kRows, smem);
        auto kern = norm_bwd_kernel<T, G, N, H, CODES>;
        err = allow_shared(kern, smem);
        if (err == cudaSuccess)
            err = launch_k(kern, dim3((unsigned)ctas), dim3(kRingThreads<G>), (size_t)smem, s, 1, a, stages);
    }) && ctas > 0;
    count_launch();
    if (!held) {
        ctas = (int)(a.M < kRingCtas ? a.M : kRingCtas);
        err = launch_k(norm_bwd_long_kernel<T>, dim3((unsigned)ctas), dim3(512), 0, s, 1, a);
    }
    if (err != cudaSuccess || !a.partial) return err;
    count_launch();
    return launch_k(dgamma_kernel<T>, dim3((unsigned)((a.D + 31) / 32)), dim3(32 * kGammaRows), 0, s, 1, dgamma,
                    (const float *)a.partial, ctas, a.D);
}

template <typename T>
cudaError_t run_bwd(const BwdArgs<T> &a, void *dgamma, cudaStream_t s) {
    constexpr int N = kVec<T>;
    const bool vec = a.D % N == 0 && aligned16(a.dx) && aligned16(a.dy) && aligned16(a.gamma) && aligned16(a.h) &&
                     aligned16(a.dh) && aligned16(a.y_out) && reinterpret_cast<uintptr_t>(a.codes) % N == 0;
    T *dg = static_cast<T *>(dgamma);
    if (a.h) return vec ? launch_bwd<T, N, false>(a, dg, s) : launch_bwd<T, 1, false>(a, dg, s);
    return vec ? launch_bwd<T, N, true>(a, dg, s) : launch_bwd<T, 1, true>(a, dg, s);
}

template <typename T>
cudaError_t run_expand(void *out, const int8_t *codes, const float *scales, const void *gamma, int64_t M,
                       int64_t D, cudaStream_t s) {
    constexpr int N = kVec<T>;
    const bool vec = aligned16(out) && reinterpret_cast<uintptr_t>(codes) % N == 0;
    const int64_t total = vec ? (M * D + N - 1) / N : M * D, want = (total + 255) / 256;
    const dim3 grid((unsigned)(want < 152 * 16 ? want : 152 * 16));
    count_launch();
    if (vec)
        return launch_k(norm_expand_kernel<T, N>, grid, dim3(256), 0, s, 1, static_cast<T *>(out), codes, scales,
                        static_cast<const T *>(gamma), M, D);
    return launch_k(norm_expand_kernel<T, 1>, grid, dim3(256), 0, s, 1, static_cast<T *>(out), codes, scales,
                    static_cast<const T *>(gamma), M, D);
}

}  // namespace

carbon_status_t norm_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_norm_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_norm_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

namespace {

carbon_status_t ready() {
    const carbon_status_t st = injected_launch_failure();
    return st != CARBON_OK ? st : current_device(nullptr, nullptr);
}

template <typename T>
cudaError_t fwd_as(void *y, void *h_out, float *rstd, int8_t *codes, float *scales, const void *x,
                   const void *residual, const void *gamma, int64_t M, int64_t D, float eps, cudaStream_t s) {
    const FwdArgs<T> a{static_cast<T *>(y), static_cast<T *>(h_out), rstd, codes, scales,
                       static_cast<const T *>(x), static_cast<const T *>(residual),
                       static_cast<const T *>(gamma), M, D, eps};
    return run_fwd(a, s);
}

template <typename T>
cudaError_t bwd_as(void *dx, void *dgamma, void *y_out, const void *dy, const void *h, const int8_t *codes,
                   const float *scales, const float *rstd, const void *gamma, const void *dh, int64_t M, int64_t D,
                   float *partial, cudaStream_t s) {
    const BwdArgs<T> a{static_cast<T *>(dx), static_cast<T *>(y_out), partial, static_cast<const T *>(dy),
                       static_cast<const T *>(h), codes, scales, rstd, static_cast<const T *>(gamma),
                       static_cast<const T *>(dh), M, D};
    return run_bwd(a, dgamma, s);
}

}  // namespace
}  // namespace carbon

using namespace carbon;

extern "C" {

carbon_status_t carbon_rms_norm_fwd(void *y, void *h_out, float *rstd, int8_t *codes, float *scales,
                                    const void *x, const void *residual, const void *gamma, int64_t M, int64_t D,
                                    float eps, carbon_dtype_t dtype, carbon_stream_t stream) {
    if (!sizes_ok(M, D) || !dtype_ok(dtype) || !(eps >= 0.0f)) return CARBON_ERR_INVALID_ARG;
    if (M == 0 || D == 0) return CARBON_OK;
    if (!y || !x || !gamma || (codes == nullptr) != (scales == nullptr)) return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(dtype_size(dtype), y, h_out, x, residual, gamma) || !aligned_to(4, rstd, scales))
        return CARBON_ERR_MISALIGNED;
    const carbon_status_t st = ready();
    if (st != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
    case CARBON_F32: return note_cuda(fwd_as<float>(y, h_out, rstd, codes, scales, x, residual, gamma, M, D, eps, s));
    case CARBON_BF16: return note_cuda(fwd_as<__nv_bfloat16>(y, h_out, rstd, codes, scales, x, residual, gamma, M, D, eps, s));
    default: return note_cuda(fwd_as<__half>(y, h_out, rstd, codes, scales, x, residual, gamma, M, D, eps, s));
    }
}

int64_t carbon_rms_norm_bwd_workspace(int64_t M, int64_t D) {
    if (!sizes_ok(M, D)) return -1;
    return (M < kRingCtas ? M : kRingCtas) * D * (int64_t)sizeof(float);
}

carbon_status_t carbon_rms_norm_bwd(void *dx, void *dgamma, void *y_out, const void *dy, const void *h,
                                    const int8_t *codes, const float *scales, const float *rstd,
                                    const void *gamma, const void *dh, int64_t M, int64_t D, void *workspace,
                                    int64_t workspace_bytes, carbon_dtype_t dtype, carbon_stream_t stream) {
    if (!sizes_ok(M, D) || !dtype_ok(dtype)) return CARBON_ERR_INVALID_ARG;
    if (D == 0 || (M == 0 && !dgamma)) return CARBON_OK;
    if (M > 0) {
        if (!dx || !dy || !rstd || !gamma) return CARBON_ERR_INVALID_ARG;
        // exactly one source of n
        if (h ? (codes || scales) : (!codes || !scales)) return CARBON_ERR_INVALID_ARG;
        if (dgamma && (!workspace || !aligned16(workspace) || workspace_bytes < carbon_rms_norm_bwd_workspace(M, D)))
            return CARBON_ERR_INVALID_ARG;
    }
    if (!aligned_to(dtype_size(dtype), dx, dgamma, y_out, dy, h, gamma, dh) || !aligned_to(4, scales, rstd))
        return CARBON_ERR_MISALIGNED;
    const carbon_status_t st = ready();
    if (st != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) return note_cuda(cudaMemsetAsync(dgamma, 0, (size_t)D * dtype_size(dtype), s));
    float *partial = dgamma ? static_cast<float *>(workspace) : nullptr;
    switch (dtype) {
    case CARBON_F32: return note_cuda(bwd_as<float>(dx, dgamma, y_out, dy, h, codes, scales, rstd, gamma, dh, M, D, partial, s));
    case CARBON_BF16: return note_cuda(bwd_as<__nv_bfloat16>(dx, dgamma, y_out, dy, h, codes, scales, rstd, gamma, dh, M, D, partial, s));
    default: return note_cuda(bwd_as<__half>(dx, dgamma, y_out, dy, h, codes, scales, rstd, gamma, dh, M, D, partial, s));
    }
}

carbon_status_t carbon_rms_norm_expand(void *out, const int8_t *codes, const float *scales, const void *gamma,
                                       int64_t M, int64_t D, carbon_dtype_t dtype, carbon_stream_t stream) {
    if (!sizes_ok(M, D) || !dtype_ok(dtype)) return CARBON_ERR_INVALID_ARG;
    if (M == 0 || D == 0) return CARBON_OK;
    if (!out || !codes || !scales) return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(dtype_size(dtype), out, gamma) || !aligned_to(4, scales)) return CARBON_ERR_MISALIGNED;
    const carbon_status_t st = ready();
    if (st != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
    case CARBON_F32: return note_cuda(run_expand<float>(out, codes, scales, gamma, M, D, s));
    case CARBON_BF16: return note_cuda(run_expand<__nv_bfloat16>(out, codes, scales, gamma, M, D, s));
    default: return note_cuda(run_expand<__half>(out, codes, scales, gamma, M, D, s));
    }
}

}  // extern "C"
