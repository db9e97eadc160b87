// linear_logprob.cu - log probabilities of given tokens under the output layer,
// with the distribution's entropy and its largest alternatives, without stored
// logits; and their gradient.
//
//   z = x . table^T,  z' = z / temperature,  lse = log sum_v exp z',  P = exp(z' - lse)
//   log_prob = z'[token] - lse,   entropy = -sum_v P log P
//   G = g (onehot - P) - e P (log P + entropy),   dx = G . table / temperature,  dtable = G^T . x / temperature
//
// The products run as those of the loss do (linear_xent.cu, xent_tiles.cuh), and
// lse has the same bits at temperature 1.  What differs:
//
// Entropy: with m the row's largest z' and S = sum exp(z' - m),
//   entropy = log S - (sum exp(z' - m) (z' - m)) / S,
// two terms that are not negative, so nothing cancels; each 128 entries give a
// (max, sum, weighted sum) triple.
//
// Alternatives: a thread keeps the largest logits that it sees of its row, top + 4
// of them, and a threshold that only a larger logit passes: after a thousand
// entries hardly one in a hundred does.  So that it sees many, the tiles of a row
// tile go to a pair of CTAs in spans of up to eight, and a span starts from what
// the row's finished spans have proved (a value that top + 4 logits reach).  The
// join takes the top + 4 largest of all spans' lists, forms their logits again,
// from exact products with a compensated sum (about 2^-44 relative to the sum of
// the products' magnitudes), and orders them by these: logits that fp32
// accumulators cannot tell apart come in the order of float64, equal ones by
// entry.  (The tensor cores' values differ from these by a few units of 2^-24;
// four spare candidates make room for as many that such an error could move
// across the last place.)
//
// Bound: the tensor cores, as for the loss.
#include "xent_tiles.cuh"

namespace carbon {
namespace {

constexpr int kJoinRows = 32;            // per CTA, a warp each; a multiple of a warp for the first part
constexpr int kFound = 64;               // candidates of a row that the join holds in shared memory

struct JoinArgs {
    float *log_probs, *lse, *entropy, *top_logp;
    int64_t *top_ids;
    const void *x, *table;
    double inv_t;
};

// a + b = s + r exactly
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &r) {
    s = __fadd_rn(a, b);
    const float d = __fsub_rn(s, a);
    r = __fadd_rn(__fsub_rn(a, __fsub_rn(s, d)), __fsub_rn(b, d));
}

// Two 16-bit elements as fp32.
template <bool F16>
__device__ __forceinline__ float2 widen2(uint32_t v) {
    if (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// The logits of `n` <= N entries against x[m], each as an unevaluated sum hi + lo,
// the same in all lanes.
template <bool F16, int N>
__device__ __forceinline__ void exact_logits(const uint4 *x, const uint4 *table, const int64_t (&row)[N], int nvec,
                                             float (&hi)[N], float (&lo)[N]) {
    float s[N], c[N];
#pragma unroll
    for (int q = 0; q < N; ++q) s[q] = c[q] = 0.0f;
    for (int i = threadIdx.x % 32; i < nvec; i += 32) {
        const uint4 xv = __ldg(x + i);
        uint4 w[N];
#pragma unroll
        for (int q = 0; q < N; ++q) w[q] = __ldg(table + row[q] * nvec + i);
        const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const uint32_t ws[4] = {w[q].x, w[q].y, w[q].z, w[q].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 a = widen2<F16>(xs[k]), b = widen2<F16>(ws[k]);
                float r;
                two_sum(s[q], __fmul_rn(a.x, b.x), s[q], r);       // 16-bit factors: exact products
                c[q] += r;
                two_sum(s[q], __fmul_rn(a.y, b.y), s[q], r);
                c[q] += r;
            }
        }
    }
#pragma unroll
    for (int q = 0; q < N; ++q) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float so = __shfl_xor_sync(0xffffffffu, s[q], o), co = __shfl_xor_sync(0xffffffffu, c[q], o);
            float r;
            two_sum(s[q], so, s[q], r);
            c[q] = (c[q] + co) + r;
        }
        two_sum(s[q], c[q], hi[q], lo[q]);
    }
}

// The alternatives of one position, by a warp.  found: room for kFound keys.
template <bool F16>
__device__ __forceinline__ void join_top(const Plan &p, const JoinArgs &a, int64_t row, float lse, uint64_t *found) {
    const int lane = threadIdx.x % 32;
    const unsigned below = (1u << lane) - 1u;
    const uint32_t bound = p.bound[row];
    const int64_t m = p.rowmap[row];
    // every key that reaches the bound: at least `listed` of them where it is set
    int n = 0;
    for (int l0 = 0; l0 < p.lists; l0 += 32) {
        const int l = l0 + lane;
        const int count = l < p.lists && CHK((int64_t)l * p.Mp + row, 1, (int64_t)p.lists * p.Mp)
            ? p.list_count[(int64_t)l * p.Mp + row] : 0;
        const int most = __reduce_max_sync(0xffffffffu, count);
        for (int e = 0; e < most; ++e) {
            const uint64_t key = e < count ? p.list[((int64_t)l * p.listed + e) * p.Mp + row] : 0ull;
            const bool take = e < count && (uint32_t)(key >> 32) >= bound;
            const unsigned mask = __ballot_sync(0xffffffffu, take);
            const int at = n + __popc(mask & below);
            if (take && at < kFound) found[at] = key;
            n += __popc(mask);
        }
    }
    __syncwarp();
    // lane e: the key of place e
    uint64_t mine = 0ull;
    int places = n < p.listed ? n : p.listed;
    if (n <= kFound) {
        const uint64_t u = lane < n ? found[lane] : 0ull, v = lane + 32 < n ? found[lane + 32] : 0ull;
        int ru = 0, rv = 0;
        for (int i = 0; i < n; ++i) {
            const uint64_t w = found[i];
            ru += w > u ? 1 : 0;
            rv += w > v ? 1 : 0;
        }
        __syncwarp();
        if (u != 0ull && ru < places) found[ru] = u;
        if (v != 0ull && rv < places) found[rv] = v;
        __syncwarp();
        if (lane < places) mine = found[lane];
    } else {
        // many equal logits: the largest key below the last one, over and over
        uint64_t last = ~0ull;
        for (int e = 0; e < places; ++e) {
            uint64_t best = 0ull;
            for (int l = lane; l < p.lists; l += 32) {
                const int count = p.list_count[(int64_t)l * p.Mp + row];
                for (int i = 0; i < count; ++i) {
                    const uint64_t key = p.list[((int64_t)l * p.listed + i) * p.Mp + row];
                    if (key < last && key > best) best = key;
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
                best = other > best ? other : best;
            }
            if (lane == e) mine = best;
            last = best;
        }
    }
    // their logits, four at a time; lane e keeps that of place e
    const uint32_t entry = ~(uint32_t)mine;
    const int nvec = (int)(p.D / 8);
    const uint4 *x = static_cast<const uint4 *>(a.x) + m * nvec, *table = static_cast<const uint4 *>(a.table);
    float hi = 0.0f, lo = 0.0f;
    for (int e = 0; e < places; e += 4) {
        int64_t rows[4];
        float h[4], l[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t r = __shfl_sync(0xffffffffu, entry, e + q < places ? e + q : e);
            rows[q] = CHK(r, 1, p.V) ? r : 0;
        }
        exact_logits<F16, 4>(x, table, rows, nvec, h, l);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (lane == e + q) { hi = h[q]; lo = l[q]; }
    }
    if (!(fabsf(hi) < INFINITY) || lo != lo) lo = 0.0f;
    if (hi != hi) hi = -INFINITY;
    int rank = 0;
    for (int i = 0; i < places; ++i) {
        const float ho = __shfl_sync(0xffffffffu, hi, i), lo_o = __shfl_sync(0xffffffffu, lo, i);
        const uint32_t eo = __shfl_sync(0xffffffffu, entry, i);
        const bool same = ho == hi && lo_o == lo;
        rank += ho > hi || (ho == hi && lo_o > lo) || (same && eo < entry) ? 1 : 0;
    }
    if (lane < places && rank < p.top && CHK(m * p.top + rank, 1, p.M * p.top)) {
        a.top_ids[m * p.top + rank] = (int64_t)entry;
        a.top_logp[m * p.top + rank] = (float)(((double)hi + (double)lo) * a.inv_t - (double)lse);
    }
    // fewer logits than places: the rest of them are -infinity
    if (lane >= places && lane < p.top) {
        a.top_ids[m * p.top + lane] = -1;
        a.top_logp[m * p.top + lane] = lse != lse ? lse : -INFINITY;
    }
}

// 32 positions per CTA.  32 threads per position take every 32nd triple, in
// order, and theirs are joined in thread order; then a warp per position joins
// its alternatives.
template <bool F16>
__global__ void __launch_bounds__(32 * kJoinRows)
logp_join_kernel(const Plan p, const JoinArgs a) {
    __shared__ union {
        struct { float max, sum, weighted; } part[32][33];
        uint64_t found[kJoinRows][kFound];
    } sh;
    __shared__ float lse_of[kJoinRows];
    wait_prior_grid();
    allow_next_grid();
    const int r = threadIdx.x % 32, t = threadIdx.x / 32;
    const int64_t first = (int64_t)blockIdx.x * kJoinRows, row = first + r;
    const int kept = p.head->kept;
    if (first >= kept) return;                            // CTA-uniform
    float mx = -INFINITY, sum = 0.0f, weighted = 0.0f;
    auto join = [&](float qm, float qs, float qw) {
        const float now = fmaxf(mx, qm), ref = now == -INFINITY ? 0.0f : now;
        const float a0 = ex2(mx - ref), b0 = ex2(qm - ref);
        // a part without a finite logit has nothing to move
        const float wa = mx > -INFINITY ? a0 * fmaf(mx - ref, sum, weighted) : 0.0f;
        const float wb = qm > -INFINITY ? b0 * fmaf(qm - ref, qs, qw) : 0.0f;
        sum = sum * a0 + qs * b0;
        weighted = wa + wb;
        mx = now;
    };
#pragma unroll 4
    for (int g = t; g < p.vocab_groups; g += 32) {
        const int64_t at = (int64_t)g * p.Mp + row;
        if (!CHK(at, 1, p.vocab_groups * p.Mp)) continue;
        const float2 q = p.pairs[at];
        join(q.x, q.y, p.weighted[at]);
    }
    sh.part[t][r] = {mx, sum, weighted};
    __syncthreads();
    if (t == 0) {
        for (int i = 1; i < 32; ++i) join(sh.part[i][r].max, sh.part[i][r].sum, sh.part[i][r].weighted);
        const float l = (mx + log2f(sum)) * kLn2;
        lse_of[r] = l;
        if (row < kept) {
            const int64_t m = p.rowmap[row];
            a.lse[m] = l;
            a.log_probs[m] = p.zt[row] * p.inv_t - l;
            a.entropy[m] = (log2f(sum) - __fdiv_rn(weighted, sum)) * kLn2;
        }
    }
    if (p.top == 0) return;
    __syncthreads();
    if (first + t < kept) join_top<F16>(p, a, first + t, lse_of[t], sh.found[t]);
}

carbon_status_t check_logp(const void *x, const void *table, const int64_t *tokens, int64_t M, int64_t D, int64_t V,
                           float temperature, int dtype) {
    const carbon_status_t st = check(x, table, tokens, M, D, V, CARBON_REDUCE_NONE, dtype);
    if (st != CARBON_OK) return st;
    if (!(temperature > 0.0f) || !(temperature < INFINITY) || !(1.0f / temperature < INFINITY)) return CARBON_ERR_INVALID_ARG;
    return CARBON_OK;
}

void set_temperature(Plan *p, float temperature) {
    p->zscale = (float)(1.4426950408889634 / (double)temperature);
    p->inv_t = (float)(1.0 / (double)temperature);
    p->range = logf((float)p->V) + 1.0f;
}

}  // namespace

carbon_status_t logp_take_device_status() {
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_xent_status, sizeof v) != cudaSuccess) return CARBON_OK;
    if (v != 0) cudaMemcpyToSymbol(g_xent_status, &zero, sizeof zero);
    return (carbon_status_t)v;
}

}  // namespace carbon

using namespace carbon;

extern "C" {

int64_t carbon_linear_logp_fwd_workspace(int64_t M, int64_t D, int64_t V, int64_t top) {
    return sizes_ok(M, D, V) && top >= 0 && top <= kTopMost
        ? make_plan(nullptr, nullptr, M, D > 0 ? D : 1, V, false, false, (int)top) : -1;
}

int64_t carbon_linear_logp_bwd_workspace(int64_t M, int64_t D, int64_t V) {
    return sizes_ok(M, D, V) ? make_plan(nullptr, nullptr, M, D > 0 ? D : 1, V > 0 ? V : 1, true, false, 0) : -1;
}

carbon_status_t carbon_linear_logp_fwd(float *log_probs, float *entropy, float *lse, int64_t *top_ids,
                                       float *top_log_probs, const void *x, const void *table, const int64_t *tokens,
                                       int64_t M, int64_t D, int64_t V, int64_t top, float temperature,
                                       int64_t ignore_index, void *workspace, int64_t workspace_bytes,
                                       carbon_dtype_t dtype, carbon_stream_t stream) {
    carbon_status_t st = check_logp(x, table, tokens, M, D, V, temperature, dtype);
    if (st != CARBON_OK) return st;
    if (top < 0 || top > kTopMost || (M > 0 && top > V)) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!log_probs || !entropy || !lse || (top > 0 && (!top_ids || !top_log_probs)) || !workspace ||
                  !aligned16(workspace) || workspace_bytes < carbon_linear_logp_fwd_workspace(M, D, V, top)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, log_probs, entropy, lse, top_log_probs) || !aligned_to(8, top_ids, tokens)) return CARBON_ERR_MISALIGNED;
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    if (M == 0) return CARBON_OK;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    Plan p;
    make_plan(&p, align128(workspace), M, D, V, false, dtype == CARBON_F16, (int)top);
    if (!list_fits(p)) return CARBON_ERR_INVALID_ARG;
    set_temperature(&p, temperature);
    ScanArgs a = {};
    a.targets = tokens; a.ignore_index = ignore_index; a.reduction = CARBON_REDUCE_NONE;
    a.losses = log_probs; a.lse_out = lse; a.entropy_out = entropy; a.top_ids = top_ids; a.top_logp = top_log_probs;
    cudaError_t err = launch_prepare<true>(p, a, x, s);
    if (err == cudaSuccess)
        err = top == 0 ? launch_tiles<false, true, 0>(p, table, nullptr, sms, s)
            : p.listed <= 12 ? launch_tiles<false, true, 12>(p, table, nullptr, sms, s)
                             : launch_tiles<false, true, 32>(p, table, nullptr, sms, s);
    if (err == cudaSuccess) {
        const JoinArgs j = {log_probs, lse, entropy, top_log_probs, top_ids, x, table, 1.0 / (double)temperature};
        count_launch();
        err = launch_k(p.f16 ? logp_join_kernel<true> : logp_join_kernel<false>, dim3((unsigned)((M + kJoinRows - 1) / kJoinRows)),
                       dim3(32 * kJoinRows), 0, s, 1, p, j);
    }
    return note_cuda(err);
}

carbon_status_t carbon_linear_logp_bwd(void *dx, void *dtable, const float *grad_log_probs, const float *grad_entropy,
                                       const void *x, const void *table, const int64_t *tokens, const float *lse,
                                       const float *entropy, int64_t M, int64_t D, int64_t V, float temperature,
                                       int64_t ignore_index, void *workspace, int64_t workspace_bytes,
                                       carbon_dtype_t dtype, carbon_stream_t stream) {
    carbon_status_t st = check_logp(x, table, tokens, M, D, V, temperature, dtype);
    if (st != CARBON_OK) return st;
    if (!aligned16(dx) || !aligned16(dtable)) return CARBON_ERR_MISALIGNED;
    if (V * D > 0 && !dtable) return CARBON_ERR_INVALID_ARG;
    if (M > 0 && (!dx || !lse || (grad_entropy && !entropy) || !workspace || !aligned16(workspace) ||
                  workspace_bytes < carbon_linear_logp_bwd_workspace(M, D, V)))
        return CARBON_ERR_INVALID_ARG;
    if (!aligned_to(4, grad_log_probs, grad_entropy, lse, entropy) || !aligned_to(8, tokens)) return CARBON_ERR_MISALIGNED;
    if (V * D == 0) return CARBON_OK;                     // then M == 0
    if ((st = injected_launch_failure()) != CARBON_OK) return st;
    int sms = 0;
    if ((st = current_device(nullptr, &sms)) != CARBON_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (M == 0) return note_cuda(cudaMemsetAsync(dtable, 0, (size_t)(V * D) * 2, s));
    Plan p;
    make_plan(&p, align128(workspace), M, D, V, true, dtype == CARBON_F16, 0);
    if (!list_fits(p)) return CARBON_ERR_INVALID_ARG;
    set_temperature(&p, temperature);
    ScanArgs a = {};
    a.targets = tokens; a.ignore_index = ignore_index; a.reduction = CARBON_REDUCE_NONE;
    a.grad = grad_log_probs; a.grad_entropy = grad_entropy; a.lse_in = lse; a.entropy_in = entropy;
    cudaError_t err = launch_prepare<true>(p, a, x, s);
    if (err == cudaSuccess) err = launch_tiles<true, true, 0>(p, table, dtable, sms, s);
    if (err == cudaSuccess) err = p.f16 ? launch_dx(p, static_cast<__half *>(dx), s) : launch_dx(p, static_cast<__nv_bfloat16 *>(dx), s);
    return note_cuda(err);
}

}  // extern "C"
