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
#include "xent_tiles.cuh"

namespace carbon {
namespace {

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
    cudaError_t err = launch_prepare<false>(p, a, x, s);
    if (err == cudaSuccess) err = launch_tiles<false, false, 0>(p, table, nullptr, sms, s);
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
    cudaError_t err = launch_prepare<false>(p, a, x, s);
    if (err == cudaSuccess) err = launch_tiles<true, false, 0>(p, table, dtable, sms, s);
    if (err == cudaSuccess) err = p.f16 ? launch_dx(p, static_cast<__half *>(dx), s) : launch_dx(p, static_cast<__nv_bfloat16 *>(dx), s);
    return note_cuda(err);
}

}  // extern "C"
