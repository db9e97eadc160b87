// linear_logprob.cu - log probabilities of given tokens under the output layer,
// with the distribution's entropy and its largest alternatives, without stored
// logits; and their gradient.
//
//   z = x . table^T,  z' = z / temperature,  lse = log sum_v exp z',  P = exp(z' - lse)
//   log_prob = z'[token] - lse,   entropy = -sum_v P log P
//   G = g (onehot - P) - e P (log P + entropy),   dx = G . table / temperature,  dtable = G^T . x / temperature
//
// The products run as those of the loss do (linear_xent.cu, xent_tiles.cuh).  What
// differs:
//
// Entropy: with m the row's largest z' and S = sum exp(z' - m),
//   entropy = log S - (sum exp(z' - m) (z' - m)) / S,
// two terms that are not negative, so nothing cancels; each 128 entries give a
// (max, sum, weighted sum) triple.  log_prob = (z'[token] - m) - log S likewise.
//
// Alternatives: a thread keeps the largest logits that it sees of its row, top + 4
// of them, and a threshold that only a larger logit passes: after a thousand
// entries hardly one in a hundred does.  So that it sees many, the tiles of a row
// tile go to a pair of CTAs in spans of up to eight; and the largest logits of 16 (or
// 32) classes of entries, which all CTAs keep up to date in global memory, prove
// others too small: the 12th largest of 16 is about the 21st largest of all
// logits so far.  A run over the first 2048 entries, ahead of the others, fills
// these classes for them, in blocks of 32; the others' are groups of 128.  No entry
// is in two classes, else a logit would count twice.  A warp per position takes the
// top + 4 largest of all lists, forms their logits again, from exact products with a
// compensated sum (about 2^-44 relative to the sum of the products' magnitudes), and
// orders them by these: logits that fp32 accumulators cannot tell apart come in the
// order of float64, equal ones by entry.  Up to 256 positions have their logits stored
// instead: filling lists is what would take most of the time there.  (The tensor cores'
// values differ from these by a few units of 2^-24; four spare candidates make room for
// as many that such an error could move across the last place.)
//
// Bound: the tensor cores, as for the loss.  8192 x 768 x 50257 bf16, a call as a
// graph: 332 us, with eight alternatives 454 (the lists in the tile kernel's epilogue,
// whose two warps per scheduler have no time left for them, and 52 for the exact
// logits of twelve candidates each); with the gradient 1.44 ms alone, 1.67 under the
// power limit.  8 positions, five alternatives: 43 us, 24 of them the table.
#include <cfloat>

#include "xent_tiles.cuh"

namespace carbon {
namespace {


struct JoinArgs {
    float *log_probs, *lse, *entropy, *top_logp;
    int64_t *top_ids;
    const void *x, *table;
};

// a + b = s + r exactly
__device__ __forceinline__ void two_sum(float a, float b, float &s, float &r) {
    s = __fadd_rn(a, b);
    const float d = __fsub_rn(s, a);
    r = __fadd_rn(__fsub_rn(a, __fsub_rn(s, d)), __fsub_rn(b, d));
}

// The log probability of a logit z, from the row's largest times log2(e) /
// temperature and log2 of the sum of the others' powers relative to it: a difference of
// logits, rounded once, in place of one of two large numbers (z' - lse was up to 1.5e-4
// above 0 for logits of 8 at temperature 1e-3).  What the sum's own rounding leaves
// above 0 is cut; NaN stays.
__device__ __forceinline__ float log_prob(const Plan &p, float z, float mx, float l2) {
    const float v = (fmaf(z, p.zscale, -mx) - l2) * kLn2;
    return v > 0.0f ? 0.0f : v;
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

// The keys of a position's places, lane e that of place e in each of W warps, put
// in their order and written.  hi_of, lo_of: shared memory for 32 places.
template <bool F16, int W, typename Sync>
__device__ __forceinline__ void put_top(const Plan &p, const JoinArgs &a, int64_t row, uint64_t mine, int places, int part,
                                        float *hi_of, float *lo_of, Sync sync) {
    const int lane = threadIdx.x % 32;
    const float mx = p.zt[row], l2 = p.weighted[row];     // as logp_join_kernel leaves them
    // their logits again, G at a time; lane e then has that of place e
    const uint32_t entry = ~(uint32_t)mine;
    const int64_t m = p.rowmap[row];
    const int nvec = (int)(p.D / 8);
    const uint4 *x = static_cast<const uint4 *>(a.x) + m * nvec, *table = static_cast<const uint4 *>(a.table);
    constexpr int G = W == 1 ? 4 : 1;
    for (int e = part * G; e < places; e += W * G) {
        int64_t rows[G];
        float h[G], l[G];
#pragma unroll
        for (int q = 0; q < G; ++q) {
            const uint32_t r = __shfl_sync(0xffffffffu, entry, e + q < places ? e + q : e);
            rows[q] = CHK(r, 1, p.V) ? r : 0;
        }
        exact_logits<F16, G>(x, table, rows, nvec, h, l);
#pragma unroll
        for (int q = 0; q < G; ++q)
            if (lane == q && e + q < places) {
                hi_of[e + q] = h[q];
                lo_of[e + q] = l[q];
            }
    }
    sync();
    if (part != 0) return;
    float hi = lane < places ? hi_of[lane] : 0.0f, lo = lane < places ? lo_of[lane] : 0.0f;
    if (!(fabsf(hi) < INFINITY) || lo != lo) lo = 0.0f;
    if (hi != hi) hi = -INFINITY;
    int rank = 0;
    for (int i = 0; i < places; ++i) {
        const float ho = __shfl_sync(0xffffffffu, hi, i), lo_o = __shfl_sync(0xffffffffu, lo, i);
        const uint32_t eo = __shfl_sync(0xffffffffu, entry, i);
        const bool same = ho == hi && lo_o == lo;
        rank += ho > hi || (ho == hi && lo_o > lo) || (same && eo < entry) ? 1 : 0;
    }
    // The logarithms from the same logits as log_probs and the sums, whose errors have
    // the same sign: those of the difference mostly cancel.  Not increasing: where
    // the order was decided by less than these errors, the one before counts.
    float z = log_prob(p, unordered((uint32_t)(mine >> 32)), mx, l2);
    int from = lane;                                      // the lane whose rank is this lane's number
    for (int i = 0; i < places; ++i)
        if (__shfl_sync(0xffffffffu, rank, i) == lane) from = i;
    z = __shfl_sync(0xffffffffu, z, from);
    const uint32_t id = __shfl_sync(0xffffffffu, entry, from);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const float before = __shfl_up_sync(0xffffffffu, z, o);
        if (lane >= o) z = fminf(z, before);
    }
    if (lane < p.top && CHK(m * p.top + lane, 1, p.M * p.top)) {
        // fewer logits than places: the rest of them are -infinity
        a.top_ids[m * p.top + lane] = lane < places ? (int64_t)id : -1;
        a.top_logp[m * p.top + lane] = l2 != l2 ? l2 : lane < places ? z : -INFINITY;
    }
}

// The keys found (n of them, more than `places`), in their order: lane e gets that
// of place e.  A key's place is the number of keys above it.
template <int Q, typename Sync>
__device__ __forceinline__ uint64_t in_order(uint64_t *found, int n, int places, int part, Sync sync) {
    const int lane = threadIdx.x % 32;
    uint64_t u[Q];
    int above[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        u[q] = q * 32 + lane < n ? found[q * 32 + lane] : 0ull;
        above[q] = 0;
    }
    for (int i = 0; i < n; ++i) {
        const uint64_t w = found[i];
#pragma unroll
        for (int q = 0; q < Q; ++q) above[q] += w > u[q] ? 1 : 0;
    }
    sync();
    if (part == 0) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (u[q] != 0ull && above[q] < places) found[above[q]] = u[q];
    }
    sync();
    return lane < places ? found[lane] : 0ull;
}

// The alternatives of a position, by W warps: eight where few positions would leave
// most of the GPU idle, else one.
constexpr int kTopThreads = 256;

template <bool F16, bool FEW, int W>
__global__ void __launch_bounds__(kTopThreads)
logp_top_kernel(const Plan p, const JoinArgs a) {
    // candidates: about twice the places asked for, up to four times where these are many
    constexpr int kFound = FEW ? 64 : 256, Q = kFound / 32, kRows = kTopThreads / 32 / W;
    constexpr int S = FEW ? kTopClassesFew : kTopClassesMany;
    __shared__ uint64_t found_all[kRows][kFound];
    __shared__ int count_all[kRows];
    __shared__ float hi_all[kRows][32], lo_all[kRows][32];
    const int lane = threadIdx.x % 32, part = threadIdx.x / 32 % W, mine_at = threadIdx.x / 32 / W;
    auto sync = [] {
        if (W == 1) __syncwarp();
        else __syncthreads();                             // then a CTA has one position
    };
    uint64_t *found = found_all[mine_at];
    int &found_count = count_all[mine_at];
    if (lane == 0 && part == 0) found_count = 0;
    wait_prior_grid();
    allow_next_grid();
    const int64_t row = (int64_t)blockIdx.x * kRows + mine_at;
    if (row >= p.head->kept) return;                      // the same for all threads that sync
    sync();
    // every key that reaches what the tile kernel knew in the end
    const uint32_t bound = class_bound<S>(p.largest + row * S, p.listed);
    constexpr int U = 4;
    for (int l0 = part * 32; l0 < p.lists; l0 += 32 * W) {
        const int l = l0 + lane;
        const unsigned long long *from = list_of(p, row, l < p.lists ? l : 0);
        const int count = l < p.lists ? (int)from[0] : 0;
        for (int e = 0; e < count; e += U) {
            uint64_t key[U];
#pragma unroll
            for (int q = 0; q < U; ++q) key[q] = e + q < count ? from[1 + e + q] : 0ull;
#pragma unroll
            for (int q = 0; q < U; ++q)
                if (key[q] != 0ull && (uint32_t)(key[q] >> 32) >= bound) {
                    const int at = atomicAdd(&found_count, 1);    // in any order: places come from comparisons
                    if (at < kFound) found[at] = key[q];
                }
        }
    }
    sync();
    // lane e: the key of place e
    const int n = found_count, places = n < p.listed ? n : p.listed;
    uint64_t mine = 0ull;
    if (n <= kFound) {
        mine = in_order<Q>(found, n, places, part, sync);
    } else {
        // too many for that (equal logits): the largest key below the last one, over and over
        uint64_t last = ~0ull;
        for (int e = 0; e < places; ++e) {
            uint64_t best = 0ull;
            for (int l = lane; l < p.lists; l += 32) {
                const unsigned long long *from = list_of(p, row, l);
                const int count = (int)from[0];
                for (int i = 0; i < count; ++i) {
                    const uint64_t key = from[1 + i];
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
    put_top<F16, W>(p, a, row, mine, places, part, hi_all[mine_at], lo_all[mine_at], sync);
}

// The alternatives of a position whose logits were stored: a CTA per position.  The
// largest logits of the groups of 128 entries, which the loss's sums come with, say
// where to look: the listed-th largest of them is a bound that only about as many
// groups reach.  (Threads with several groups, beyond 131072 entries, count once.)
constexpr int kScanThreads = 1024;

template <bool F16>
__global__ void __launch_bounds__(kScanThreads)
logp_scan_kernel(const Plan p, const JoinArgs a) {
    constexpr int kFound = 256, W = kScanThreads / 32;
    __shared__ uint64_t found[kFound];
    __shared__ int found_count;
    __shared__ float hi_of[32], lo_of[32];
    __shared__ uint64_t part_best[W];
    wait_prior_grid();
    allow_next_grid();
    const int t = threadIdx.x, lane = t % 32, part = t / 32;
    const int64_t row = blockIdx.x;
    if (row >= p.head->kept) return;                      // CTA-uniform
    // 0: no candidate (NaN, -infinity)
    auto key_of = [](float v) { return v > -INFINITY ? ordered(v) : 0u; };
    auto group_max = [&](int g) { return key_of(__ldcg(&p.pairs[(int64_t)g * p.Mp + row].x)); };
    if (t == 0) found_count = 0;
    uint32_t largest = 0u;
    for (int g = t; g < p.vocab_groups; g += kScanThreads) largest = max(largest, group_max(g));
    uint32_t bound = 0u;                                  // of logits times zscale
    for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = bound | 1u << bit;
        if (__syncthreads_count(largest >= c) >= p.listed) bound = c;
    }
    if (bound == 0u) bound = 1u;                          // fewer groups than that: all of their logits
    // f(ordered logit, entry) for every logit that reaches the bound, a warp per group
    auto each = [&](auto f) {
        for (int g0 = part * 32; g0 < p.vocab_groups; g0 += W * 32) {
            unsigned hit = __ballot_sync(0xffffffffu, g0 + lane < p.vocab_groups && group_max(g0 + lane) >= bound);
            for (; hit != 0u; hit &= hit - 1u) {
                const int at = (g0 + __ffs((int)hit) - 1) * kGroup + 4 * lane;
                if (at >= p.V) continue;
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(p.logits + row * p.pitch + at));    // past V: -infinity
                const float z[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (key_of(z[q] * p.zscale) >= bound) f(ordered(z[q]), at + q);
            }
        }
    };
    each([&](uint32_t k, int entry) {
        const int at = atomicAdd(&found_count, 1);        // in any order: places come from comparisons
        if (at < kFound) found[at] = (uint64_t)k << 32 | (uint32_t)~entry;
    });
    auto sync = [] { __syncthreads(); };
    sync();
    const int n = found_count, places = n < p.listed ? n : p.listed;
    uint64_t mine = 0ull;
    if (n <= kFound) {
        mine = in_order<kFound / 32>(found, n, places, part, sync);
    } else {
        // many equal logits: the largest key below the last one, over and over
        uint64_t last = ~0ull;
        for (int e = 0; e < places; ++e) {
            uint64_t best = 0ull;
            each([&](uint32_t k, int entry) {
                const uint64_t key = (uint64_t)k << 32 | (uint32_t)~entry;
                if (key < last && key > best) best = key;
            });
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t other = __shfl_xor_sync(0xffffffffu, best, o);
                best = other > best ? other : best;
            }
            sync();
            if (lane == 0) part_best[part] = best;
            sync();
            for (int w = 0; w < W; ++w) best = part_best[w] > best ? part_best[w] : best;
            if (lane == e) mine = best;
            last = best;
        }
    }
    put_top<F16, W>(p, a, row, mine, places, part, hi_of, lo_of, sync);
}

// 32 positions per CTA.  32 threads per position take every 32nd triple, in
// order, and theirs are joined in thread order.
__global__ void __launch_bounds__(1024)
logp_join_kernel(const Plan p, const JoinArgs a) {
    __shared__ struct { float max, sum, weighted; } part[32][33];
    wait_prior_grid();
    allow_next_grid();
    const int r = threadIdx.x % 32, t = threadIdx.x / 32;
    const int64_t first = (int64_t)blockIdx.x * 32, row = first + r;
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
    part[t][r] = {mx, sum, weighted};
    __syncthreads();
    if (t == 0 && row < kept) {
        for (int i = 1; i < 32; ++i) join(part[i][r].max, part[i][r].sum, part[i][r].weighted);
        const float l2 = log2f(sum), h = (l2 - __fdiv_rn(weighted, sum)) * kLn2;
        const int64_t m = p.rowmap[row];
        a.lse[m] = (mx + l2) * kLn2;
        a.log_probs[m] = log_prob(p, p.zt[row], mx, l2);
        a.entropy[m] = h < 0.0f ? 0.0f : h;               // NaN stays
        p.zt[row] = mx;                                   // for the alternatives, read above for the last time
        p.weighted[row] = l2;
    }
}

template <bool F16>
cudaError_t launch_top(const Plan &p, const JoinArgs &j, int sms, cudaStream_t s) {
    if (p.logits) return launch_k(logp_scan_kernel<F16>, dim3((unsigned)p.M), dim3(kScanThreads), 0, s, 1, p, j);
    const bool wide = p.M <= sms * (kTopThreads / 32), few = p.listed <= kTopFew;
    const int64_t rows = wide ? 1 : kTopThreads / 32;
    return launch_k(wide ? (few ? logp_top_kernel<F16, true, 8> : logp_top_kernel<F16, false, 8>)
                         : (few ? logp_top_kernel<F16, true, 1> : logp_top_kernel<F16, false, 1>),
                    dim3((unsigned)((p.M + rows - 1) / rows)), dim3(kTopThreads), 0, s, 1, p, j);
}

constexpr double kLog2eDouble = 1.4426950408889634;

// 1 / temperature for logits as they are formed.  The tensor cores' accumulator rounds
// toward zero.  A step of 16 products takes about 2^-25 of the sum so far with it;
// over D / 16 steps that sum is half the final one on average, so a logit comes out
// smaller by D 2^-30 of itself: measured as 1.0 to 1.1 times that in bf16 and 1.1 to
// 1.3 in fp16 for D = 768 to 16384 and zero-mean inputs, 1.1 and 1.6 to 1.8 for
// inputs of mean 1/2 (a sum that fp32 holds exactly loses nothing and gets this
// error instead).  The logits' factors put it back (200 x 2048
// x 50257: mean error of lse 8e-6 without, 3e-7 with; entropy's 9e-7 and 4e-8 of
// itself).  It is a 128th of the bound of one logit's error.
double factor_of(int64_t D, float temperature) { return (1.0 + (double)D * 0x1p-30) / (double)temperature; }

carbon_status_t check_logp(const void *x, const void *table, const int64_t *tokens, int64_t M, int64_t D, int64_t V,
                           float temperature, int dtype) {
    const carbon_status_t st = check(x, table, tokens, M, D, V, CARBON_REDUCE_NONE, dtype);
    if (st != CARBON_OK) return st;
    if (!(temperature > 0.0f) || !(temperature < INFINITY)) return CARBON_ERR_INVALID_ARG;
    if (!(kLog2eDouble * factor_of(D, temperature) < FLT_MAX)) return CARBON_ERR_INVALID_ARG;
    return CARBON_OK;
}

void set_temperature(Plan *p, float temperature) {
    const double factor = factor_of(p->D, temperature);
    p->zscale = (float)(kLog2eDouble * factor);
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
    if (err == cudaSuccess && p.piloted > 0) {
        Plan q = p;                                       // with a ticket of its own
        q.pilot = true;
        q.V = p.piloted;
        q.ticket = p.joined;
        err = launch_tiles<false, true, 0>(q, table, nullptr, sms, s);
    }
    if (err == cudaSuccess)
        err = p.lists == 0 ? launch_tiles<false, true, 0>(p, table, nullptr, sms, s)
            : p.listed <= kTopFew ? launch_tiles<false, true, kTopFew>(p, table, nullptr, sms, s)
                             : launch_tiles<false, true, 32>(p, table, nullptr, sms, s);
    if (err == cudaSuccess) {
        const JoinArgs j = {log_probs, lse, entropy, top_log_probs, top_ids, x, table};
        count_launch();
        err = launch_k(logp_join_kernel, dim3((unsigned)((M + 31) / 32)), dim3(1024), 0, s, 1, p, j);
        if (err == cudaSuccess && top > 0) {
            count_launch();
            err = p.f16 ? launch_top<true>(p, j, sms, s) : launch_top<false>(p, j, sms, s);
        }
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
