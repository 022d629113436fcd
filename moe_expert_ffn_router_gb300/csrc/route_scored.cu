// moe_route_scored: experts chosen by scores plus a balance bias from the best groups,
// weights from the scores alone, the token -> expert grouping; and the gradient of the
// logits.
//
//   p_e = sigmoid(l_e) or softmax(l)_e,  c_e = p_e + b_e
//   a group's value: the sum of its two largest c;  the best groups stay
//   the k largest c of them are chosen (ties to the lower index)
//   w_j = scale p_j, or scale p_j / sum of the chosen p
//
// The bytes are few (a logit row in, 12 bytes per choice out), so what counts is the
// chain of a row: one warp per token, expert lane + 32 q in register q, and a choice is
// two warp-wide reductions of order-preserving integer keys.
//  * The choice is that of 64-bit arithmetic.  A row is worked out in 32 bits, and again
//    in 64 where two values that decide (neighbours among the picks, the last pick and
//    the next, the worst group kept and the best dropped) are within the error of the
//    32-bit ones (under 1 % of rows of 256 experts).  Without a bias c grows with l, and
//    the logits themselves are the keys.
//  * Up to 64 tokens one block chooses and groups.  More: blocks of equal runs of tokens
//    choose and count their experts, and a second launch places every pair from the
//    counts of the runs before its own and a bitmap of tokens per expert in its run.
//    No atomics on order: pairs are sorted by (expert, token).
#include "dense.cuh"
#include "route_scored.cuh"

namespace rvq {
namespace {

constexpr int RS_NT = 256;
constexpr int RS_Q = 8;  // experts per lane

template <class F> struct KeyOf;
template <> struct KeyOf<float> { using type = uint32_t; };
template <> struct KeyOf<double> { using type = uint64_t; };

// Order-preserving keys (after -0 -> +0): larger value, larger key, never 0.
__device__ __forceinline__ uint32_t to_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t to_key(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return (u >> 63) ? ~u : (u | (1ull << 63));
}
__device__ __forceinline__ float from_key(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ double from_key(uint64_t k) {
    return __longlong_as_double((long long)((k >> 63) ? (k & ~(1ull << 63)) : ~k));
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = warp_max((uint32_t)(v >> 32));
    const uint32_t lo = warp_max((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Scores of this lane's experts (0 past the last).
template <class F>
__device__ __forceinline__ void scores(const float (&l)[RS_Q], int E, int lane, int score,
                                       F (&p)[RS_Q]) {
    if (score == MOE_SCORE_SIGMOID) {
#pragma unroll
        for (int q = 0; q < RS_Q; ++q)
            p[q] = lane + 32 * q < E ? F(1) / (F(1) + exp_of(-F(l[q]))) : F(0);
        return;
    }
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q)
        if (lane + 32 * q < E) top = max(top, to_key(l[q]));
    const F m = F(from_key(warp_max(top)));
    F z = F(0);
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        p[q] = lane + 32 * q < E ? exp_of(F(l[q]) - m) : F(0);
        z += p[q];
    }
    z = warp_sum(z);
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) p[q] /= z;
}

// The k experts of a row: lane s < k gets the s-th.  Returns whether two values that
// decide are closer than the arithmetic tells apart (F float).
//
// Error of a 32-bit score: sigmoid 2 units of expf, one of the sum, a half of the
// quotient, at most 4e-7; softmax p (6 + |l - m|) 2^-23 with p |l - m| <= 0.37, and 14
// half steps of the sum, at most 1.7e-6; both of p <= 1.  Two values c are told apart by
// more than twice that and a step of the larger |c|; sums of two by twice as much.
template <class F>
__device__ __forceinline__ bool choose(const float (&l)[RS_Q], const float (&b)[RS_Q], int E, int k,
                                       const RouteRule &rule, int lane, int &my_idx) {
    using Key = typename KeyOf<F>::type;
    const bool biased = rule.bias != nullptr, grouped = rule.top_groups < rule.groups;
    constexpr bool kCheck = sizeof(F) == 4;
    bool near = false;
    Key key[RS_Q];
    float big = 0.f;
    if (biased || grouped) {
        F p[RS_Q];
        scores<F>(l, E, lane, rule.score, p);
#pragma unroll
        for (int q = 0; q < RS_Q; ++q) {
            const F c = biased ? p[q] + F(b[q]) : p[q];
            key[q] = lane + 32 * q < E ? to_key(c) : Key(0);
            if (kCheck) big = fmaxf(big, fabsf((float)c));
        }
    }
    float apart = 0.f;
    if (kCheck && (biased || grouped))
        apart = 3.4e-6f + 2.4e-7f * __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));
    bool in[RS_Q];
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) in[q] = lane + 32 * q < E;
    if (grouped) {
        const int size = E / rule.groups;
        F mine = F(0);
        for (int g = 0; g < rule.groups; ++g) {
            const int lo = g * size - lane, hi = lo + size;  // 32 q of its members
            Key a1 = 0, a2 = 0;
#pragma unroll
            for (int q = 0; q < RS_Q; ++q) {
                if (32 * q < lo || 32 * q >= hi) continue;
                if (key[q] > a1) {
                    a2 = a1;
                    a1 = key[q];
                } else if (key[q] > a2) {
                    a2 = key[q];
                }
            }
            const Key v1 = warp_max(a1);
            const int winner = __ffs(__ballot_sync(0xffffffffu, a1 == v1)) - 1;
            F v = from_key(v1);
            if (size > 1) v += from_key(warp_max(lane == winner ? a2 : a1));
            if (lane == g) mine = v;
        }
        int place = 0;  // of group `lane`
        F worst = F(0), best = F(0);
        for (int g = 0; g < rule.groups; ++g) {
            const F v = __shfl_sync(0xffffffffu, mine, g);
            if (v > mine || (v == mine && g < lane)) ++place;
        }
        const uint32_t kept =
            __ballot_sync(0xffffffffu, lane < rule.groups && place < rule.top_groups);
        if (kCheck) {
            bool any_w = false, any_b = false;
            for (int g = 0; g < rule.groups; ++g) {
                const F v = __shfl_sync(0xffffffffu, mine, g);
                if ((kept >> g) & 1u) {
                    if (!any_w || v < worst) worst = v;
                    any_w = true;
                } else {
                    if (!any_b || v > best) best = v;
                    any_b = true;
                }
            }
            near = !((float)worst - (float)best > 2.f * apart);
        }
#pragma unroll
        for (int q = 0; q < RS_Q; ++q) {
            const int e = lane + 32 * q;
            in[q] = e < E && ((kept >> (e / size)) & 1u);
        }
    }
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        if (!biased) key[q] = to_key(F(l[q]));
        if (!in[q]) key[q] = 0;
    }
    // lane-local best (ties: lower q = lower expert index)
    uint32_t taken = 0u;
    Key lk = 0, last = 0;
    int lq = 0;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q)
        if (key[q] > lk) { lk = key[q]; lq = q; }
    my_idx = 0;
    const int picks = kCheck && biased ? k + 1 : k;  // the next one too, to be told apart
    for (int s = 0; s < picks; ++s) {
        const Key kmax = warp_max(lk);
        if (kCheck && biased && s > 0 && kmax != 0 &&
            !((float)from_key(last) - (float)from_key(kmax) > apart))
            near = true;
        last = kmax;
        const uint32_t cand = lk == kmax ? (uint32_t)(lane + 32 * lq) : 0xffffffffu;
        const uint32_t e = __reduce_min_sync(0xffffffffu, cand);
        if (s < k && lane == s) my_idx = (int)e;
        if ((int)(e & 31) == lane) {
            taken |= 1u << (e >> 5);
            lk = 0;
            lq = 0;
#pragma unroll
            for (int q = 0; q < RS_Q; ++q)
                if (!((taken >> q) & 1u) && key[q] > lk) { lk = key[q]; lq = q; }
        }
    }
    return near;
}

__device__ __noinline__ int choose_64(const float (&l)[RS_Q], const float (&b)[RS_Q], int E, int k,
                                      const RouteRule &rule, int lane) {
    int idx;
    choose<double>(l, b, E, k, rule, lane, idx);
    return idx;
}

// Chosen expert and weight of lane s < k.
__device__ __forceinline__ void route_row(const float *__restrict__ row, int E, int k,
                                          const RouteRule &rule, const float (&b)[RS_Q], int lane,
                                          uint32_t *status, int &my_idx, float &my_w) {
    float l[RS_Q];
    bool bad = false;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const int e = lane + 32 * q;
        l[q] = e < E ? row[e] : 0.f;
        if (!isfinite(l[q])) {  // reported; any finite value keeps the outputs in range
            bad = true;
            l[q] = 0.f;
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_dev_error(status, RVQ_DEV_ERR_NONFINITE);
    if (choose<float>(l, b, E, k, rule, lane, my_idx)) my_idx = choose_64(l, b, E, k, rule, lane);
    // the chosen logit: register my_idx / 32 of lane my_idx % 32
    float mine = 0.f;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const float v = __shfl_sync(0xffffffffu, l[q], my_idx & 31);
        if (q == my_idx >> 5) mine = v;
    }
    const bool on = lane < k;
    const float top = from_key(warp_max(on ? to_key(mine) : 0u));
    float e;
    if (rule.score == MOE_SCORE_SIGMOID) {
        if (rule.renorm) {
            // sigmoids over e^m, m the largest logit up to 0: sums of very negative
            // logits stay away from 0
            const float m = fminf(top, 0.f);
            e = mine <= 0.f ? expf(mine - m) / (1.f + expf(mine)) : 1.f / (1.f + expf(-mine));
        } else {
            e = 1.f / (1.f + expf(-mine));
        }
    } else if (rule.renorm) {
        e = expf(mine - top);
    } else {
        uint32_t all = 0;
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < RS_Q; ++q)
            if (lane + 32 * q < E) all = max(all, to_key(l[q]));
        const float m = from_key(warp_max(all));
#pragma unroll
        for (int q = 0; q < RS_Q; ++q)
            if (lane + 32 * q < E) z += expf(l[q] - m);
        e = expf(mine - m) / warp_sum(z);
    }
    my_w = rule.scale * (rule.renorm ? e / warp_sum(on ? e : 0.f) : e);
}

__device__ __forceinline__ void load_bias(const RouteRule &rule, int E, int lane, uint32_t *status,
                                          float (&b)[RS_Q]) {
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const int e = lane + 32 * q;
        b[q] = rule.bias && e < E ? rule.bias[e] : 0.f;
        if (!isfinite(b[q])) {
            set_dev_error(status, RVQ_DEV_ERR_NONFINITE);
            b[q] = 0.f;
        }
    }
}

// Exclusive prefix of cnt[0 .. E) by warp 0 (E <= 256): cnt becomes it; its end is
// returned to every lane of the warp.
__device__ __forceinline__ int scan_counts(int *cnt, int E, int lane) {
    int v[RS_Q], s = 0;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const int e = lane * RS_Q + q;
        v[q] = e < E ? cnt[e] : 0;
        s += v[q];
    }
    int incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    int run = incl - s;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const int e = lane * RS_Q + q;
        if (e < E) cnt[e] = run;
        run += v[q];
    }
    return __shfl_sync(0xffffffffu, run, 31);
}

// One block, up to 64 tokens: choice and grouping.
template <int NT>
__global__ void __launch_bounds__(NT) route_scored_one_kernel(const RouteScoredJob j) {
    __shared__ uint32_t mask[256][2];
    __shared__ int cnt[256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int i = threadIdx.x; i < 512; i += NT) mask[i >> 1][i & 1] = 0u;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    float b[RS_Q];
    load_bias(j.rule, j.E, lane, j.status, b);
    for (int t = warp; t < j.n; t += NT / 32) {
        int idx;
        float w;
        route_row(j.logits + (int64_t)t * j.E, j.E, j.k, j.rule, b, lane, j.status, idx, w);
        if (lane < j.k) {
            j.idx[t * j.k + lane] = idx;
            j.w[t * j.k + lane] = w;
            atomicOr(&mask[idx][t >> 5], 1u << (t & 31));
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < j.E; e += NT) cnt[e] = __popc(mask[e][0]) + __popc(mask[e][1]);
    __syncthreads();
    if (warp == 0) {
        const int end = scan_counts(cnt, j.E, lane);
        if (lane == 0) j.offsets[j.E] = end;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < j.E; e += NT) j.offsets[e] = cnt[e];
    for (int t = warp; t < j.n && lane < j.k; t += NT / 32) {
        const uint32_t below = (1u << (t & 31)) - 1u;
        const int e = j.idx[t * j.k + lane];  // this thread's own
        const int before = t < 32 ? __popc(mask[e][0] & below)
                                  : __popc(mask[e][0]) + __popc(mask[e][1] & below);
        j.pairs[cnt[e] + before] = t * j.k + lane;
    }
}

// Many tokens, first launch: block b chooses for tokens run * b .. and counts its
// experts into hist[b][E].
__global__ void __launch_bounds__(RS_NT) route_scored_choose_kernel(const RouteScoredJob j) {
    __shared__ int cnt[256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cnt[threadIdx.x] = 0;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    float b[RS_Q];
    load_bias(j.rule, j.E, lane, j.status, b);
    const int t0 = blockIdx.x * j.run, t1 = min(j.n, t0 + j.run);
    for (int t = t0 + warp; t < t1; t += RS_NT / 32) {
        int idx;
        float w;
        route_row(j.logits + (int64_t)t * j.E, j.E, j.k, j.rule, b, lane, j.status, idx, w);
        if (lane < j.k) {
            j.idx[(int64_t)t * j.k + lane] = idx;
            j.w[(int64_t)t * j.k + lane] = w;
            atomicAdd(&cnt[idx], 1);
        }
    }
    __syncthreads();
    if (threadIdx.x < j.E) j.hist[blockIdx.x * j.E + threadIdx.x] = cnt[threadIdx.x];
}

// Second launch: block b places its run's pairs.
__global__ void __launch_bounds__(RS_NT) route_scored_place_kernel(const RouteScoredJob j) {
    extern __shared__ uint32_t mask[];  // [E][words], then [E][words] of 16-bit ranks
    __shared__ int cnt[256], before[256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (j.run + 31) / 32;
    uint16_t *pre = reinterpret_cast<uint16_t *>(mask + j.E * words);
    for (int i = threadIdx.x; i < j.E * words; i += RS_NT) mask[i] = 0u;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    const int t0 = blockIdx.x * j.run, t1 = min(j.n, t0 + j.run);
    const int64_t p0 = (int64_t)t0 * j.k;
    const int np = (t1 - t0) * j.k;
    for (int i = threadIdx.x; i < np; i += RS_NT) {
        const int t = i / j.k;
        atomicOr(&mask[j.idx[p0 + i] * words + (t >> 5)], 1u << (t & 31));
    }
    if (threadIdx.x < j.E) {
        int all = 0, mine = 0;
#pragma unroll 8
        for (int r = 0; r < (int)gridDim.x; ++r) {
            const int c = j.hist[r * j.E + threadIdx.x];
            all += c;
            if (r < (int)blockIdx.x) mine += c;
        }
        cnt[threadIdx.x] = all;
        before[threadIdx.x] = mine;
    }
    __syncthreads();
    if (warp == 0) {
        const int end = scan_counts(cnt, j.E, lane);
        if (blockIdx.x == 0 && lane == 0) j.offsets[j.E] = end;
    }
    for (int e = threadIdx.x; e < j.E; e += RS_NT) {
        int run = 0;
        for (int w = 0; w < words; ++w) {
            pre[e * words + w] = (uint16_t)run;
            run += __popc(mask[e * words + w]);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < j.E) j.offsets[threadIdx.x] = cnt[threadIdx.x];
    for (int i = threadIdx.x; i < np; i += RS_NT) {
        const int t = i / j.k, e = j.idx[p0 + i], at = e * words + (t >> 5);
        j.pairs[cnt[e] + before[e] + pre[at] + __popc(mask[at] & ((1u << (t & 31)) - 1u))] =
            (int32_t)(p0 + i);
    }
}

// Gradient of the logits, one warp per token:
//   renormalised   dp_j = scale (dw_j - sum_i dw_i w_i / scale) / S   (S the chosen sum)
//   else           dp_j = scale dw_j
//   sigmoid        dl_j = dp_j p_j (1 - p_j), 0 elsewhere
//   softmax        dl_e = p_e (dp_e - sum_j dp_j p_j) over all experts; renormalised it
//                  is scale w'_j (dw_j - sum_i dw_i w'_i) of the chosen alone, w' = w / scale
__global__ void __launch_bounds__(RS_NT) route_scored_backward_kernel(const RouteScoredJob j) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (RS_NT / 32) + (int)(threadIdx.x >> 5);
    dependency_wait();
    dependents_may_start();
    if (t >= j.n) return;
    const float *row = j.logits + (int64_t)t * j.E;
    const bool on = lane < j.k;
    const int idx = on ? j.idx[(int64_t)t * j.k + lane] : -1;
    const bool in = idx >= 0 && idx < j.E;  // others take no part
    const float l = in ? row[idx] : 0.f, dw = in ? j.dw[(int64_t)t * j.k + lane] : 0.f;
    const RouteRule &rule = j.rule;
    float g = 0.f, rest = 0.f, m = 0.f, z = 1.f;
    const bool dense = rule.score == MOE_SCORE_SOFTMAX && !rule.renorm;
    float all[RS_Q];
    if (rule.renorm) {
        const float top = from_key(warp_max(in ? to_key(l) : 0u));
        float e = 0.f, slope = 1.f;
        if (in && rule.score == MOE_SCORE_SIGMOID) {
            const float mm = fminf(top, 0.f);
            const float p = 1.f / (1.f + expf(-l));
            e = l <= 0.f ? expf(l - mm) / (1.f + expf(l)) : p;
            slope = 1.f / (1.f + expf(l));  // 1 - p
        } else if (in) {
            e = expf(l - top);
        }
        const float w = e / warp_sum(e);
        const float mean = warp_sum(w * dw);
        g = rule.scale * w * (dw - mean) * slope;
    } else if (rule.score == MOE_SCORE_SIGMOID) {
        g = in ? rule.scale * dw / (1.f + expf(-l)) / (1.f + expf(l)) : 0.f;
    } else {
        uint32_t top = 0;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < RS_Q; ++q) {
            all[q] = lane + 32 * q < j.E ? row[lane + 32 * q] : 0.f;
            if (lane + 32 * q < j.E) top = max(top, to_key(all[q]));
        }
        m = from_key(warp_max(top));
#pragma unroll
        for (int q = 0; q < RS_Q; ++q)
            if (lane + 32 * q < j.E) s += expf(all[q] - m);
        z = warp_sum(s);
        const float p = in ? expf(l - m) / z : 0.f;
        rest = rule.scale * warp_sum(p * dw);
        g = rule.scale * dw;
    }
    float out[RS_Q] = {};
    for (int s = 0; s < j.k; ++s) {
        const int e = __shfl_sync(0xffffffffu, in ? idx : -1, s);
        const float v = __shfl_sync(0xffffffffu, g, s);
#pragma unroll
        for (int q = 0; q < RS_Q; ++q)
            if (e == lane + 32 * q) out[q] += v;
    }
    __syncwarp();  // a gradient in the logits' place: the row is read
    float *o = j.dlogits + (int64_t)t * j.E;
#pragma unroll
    for (int q = 0; q < RS_Q; ++q) {
        const int e = lane + 32 * q;
        if (e < j.E) o[e] = dense ? expf(all[q] - m) / z * (out[q] - rest) : out[q];
    }
}

}  // namespace

int route_scored_run(int n) {
    // runs of whole rounds of a block's warps, one block per SM at most
    const int run = (n + kRouteRuns - 1) / kRouteRuns;
    return (run + RS_NT / 32 - 1) / (RS_NT / 32) * (RS_NT / 32);
}

rvq_status launch_route_scored(const RouteScoredJob &job, cudaStream_t stream) {
    if (job.n <= kRouteOneBlock) {
        if (job.n <= 8)
            RVQ_CUDA(launch_after(route_scored_one_kernel<256>, 1, 256, 0, stream, job));
        else
            RVQ_CUDA(launch_after(route_scored_one_kernel<1024>, 1, 1024, 0, stream, job));
        return RVQ_OK;
    }
    RouteScoredJob j = job;
    j.run = route_scored_run(j.n);
    const unsigned blocks = (unsigned)((j.n + j.run - 1) / j.run);
    const size_t smem = (size_t)j.E * ((j.run + 31) / 32) * 6;
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(route_scored_place_kernel,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10));
        attr_done[dev] = 1;
    }
    RVQ_CUDA(launch_after(route_scored_choose_kernel, blocks, RS_NT, 0, stream, j));
    RVQ_CUDA(launch_after(route_scored_place_kernel, blocks, RS_NT, smem, stream, j));
    return RVQ_OK;
}

rvq_status launch_route_scored_backward(const RouteScoredJob &job, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((job.n + RS_NT / 32 - 1) / (RS_NT / 32));
    RVQ_CUDA(launch_after(route_scored_backward_kernel, blocks, RS_NT, 0, stream, job));
    return RVQ_OK;
}

}  // namespace rvq
