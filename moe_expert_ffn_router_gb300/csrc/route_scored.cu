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
// chain of a row: one warp per token, expert lane + 32 q in register q, a lane's experts
// sorted, and a pick is two warp-wide reductions of order-preserving integer keys.
//  * The choice is that of 64-bit arithmetic.  A row is worked out in 32 bits; where two
//    values that decide are within the error of the 32-bit ones (neighbours among the
//    picks, the last pick and the next: a few rows in ten thousand of 256 experts), those
//    picks alone are compared in 64 bits, and where groups are, the whole row is.  Without
//    a bias c grows with l, and the logits are the keys.
//  * Up to 8 tokens one block chooses and groups (64 would take it 29 us, two launches
//    10).  More: blocks of equal runs of tokens choose and count their experts, and a
//    second launch places every pair from the counts of the runs before its own and a
//    bitmap of tokens per expert in its run.  No atomics decide an order: pairs are sorted
//    by (expert, token).
//
// Measured (GB300; bias, 4 of 8 groups, 16 of 256 experts): one token 6.5 to 6.9 us, 64 10.8,
// 2048 15 to 17 (11.4 without bias and groups), with the softmax, more of whose rows are
// decided in 64 bits, 37; 8 of 64 experts, 4096 tokens 9.0, with the softmax and its gradient
// 13.9.  Latency: some 2400 instructions a token, 1200 of 64 experts; a row that is decided
// in 64 bits adds microseconds to its launch, most of them to fetch that code.
#include "dense.cuh"
#include "route_scored.cuh"

namespace rvq {
namespace {

constexpr int RS_NT = 256;
constexpr int RS_PLACE = 1024;  // threads of a placing block
constexpr int RS_Q = 8;          // experts per lane, at most

// Order-preserving keys (after -0 -> +0): larger value, larger key, never 0.
__device__ __forceinline__ uint32_t to_key(float f) {
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
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

__device__ __forceinline__ float finite_or_0(float v) { return isfinite(v) ? v : 0.f; }

template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// 1 - sigmoid(l) = 1 / (1 + e^l): two units of the exponential, half a step of the sum and
// two units of the quotient, 5.4e-7 of its value
__device__ __forceinline__ float rest32(float l) { return __fdividef(1.f, 1.f + expf(l)); }
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// Groups of a row that stay, as bits: lane g holds the value of group g.
template <class F>
__device__ __forceinline__ uint32_t best_groups(F mine, const RouteRule &rule, int lane) {
    int place = 0;
    for (int g = 0; g < rule.groups; ++g) {
        const F v = __shfl_sync(0xffffffffu, mine, g);
        if (v > mine || (v == mine && g < lane)) ++place;
    }
    return __ballot_sync(0xffffffffu, lane < rule.groups && place < rule.top_groups);
}

// The choice in 64 bits, from the start: for the rows that 32 bits leave open.  Rolled
// loops over keys in shared memory: it runs seldom, and long straight code would cost
// more to fetch than to run.
__device__ __noinline__ int choose_64(const float *row, const float *bias, int E, int k,
                                      const RouteRule &rule, int lane, uint64_t *key) {
    double m = 0.0, z = 1.0;
    if (rule.score == MOE_SCORE_SOFTMAX) {
        uint32_t top = 0;
#pragma unroll 1
        for (int e = lane; e < E; e += 32) top = max(top, to_key(finite_or_0(row[e])));
        m = (double)from_key(warp_max(top));
        z = 0.0;
#pragma unroll 1
        for (int e = lane; e < E; e += 32) z += exp((double)finite_or_0(row[e]) - m);
        z = warp_sum(z);
    }
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        const float l = finite_or_0(row[e]);
        const double p = rule.score == MOE_SCORE_SIGMOID ? sigmoid64(l) : exp((double)l - m) / z;
        key[e] = to_key(bias ? p + (double)finite_or_0(bias[e]) : p);
    }
    __syncwarp();
    uint32_t kept = 0xffffffffu;
    const int size = E / rule.groups;
    if (rule.top_groups < rule.groups) {
        double mine = 0.0;
        if (lane < rule.groups) {
            uint64_t a1 = 0, a2 = 0;
#pragma unroll 1
            for (int e = lane * size; e < (lane + 1) * size; ++e) {
                const uint64_t c = key[e];
                a2 = c > a1 ? a1 : c > a2 ? c : a2;
                a1 = c > a1 ? c : a1;
            }
            mine = from_key(a1) + (size > 1 ? from_key(a2) : 0.0);
        }
        kept = best_groups(mine, rule, lane);
    }
    __syncwarp();
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
        if (!((kept >> (e / size)) & 1u) && rule.top_groups < rule.groups)
            key[e] = 0;
        else if (!bias)
            key[e] = to_key((double)finite_or_0(row[e]));
    }
    __syncwarp();
    int my_idx = 0;
#pragma unroll 1
    for (int s = 0; s < k; ++s) {
        uint64_t best = 0;
        int at = 0x7fffffff;
#pragma unroll 1
        for (int e = lane; e < E; e += 32)
            if (key[e] > best) { best = key[e]; at = e; }
        const uint64_t top = warp_max(best);
        const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? (uint32_t)at : 0x7fffffffu);
        if (lane == s) my_idx = (int)e;
        if ((int)(e & 31) == lane) key[e] = 0;
        __syncwarp();
    }
    return my_idx;
}

// The two largest of a pair and another.
__device__ __forceinline__ void top_two(uint32_t &o1, uint32_t &o2, uint32_t a1, uint32_t a2,
                                        uint32_t b1, uint32_t b2) {
    o2 = max(min(a1, b1), max(a2, b2));
    o1 = max(a1, b1);
}

// The k experts of a row: lane s < k gets the s-th.  l, b: logits and biases of the
// lane's experts, finite.
//
// In 32 bits a sigmoid's c is held as c - 1 = b - (1 - p), which is exact to 5.4e-7 of 1 - p
// and half a step of itself: scores near 1, where the picks are, keep their differences.
// With |c - 1| and the largest |b| no smaller than 1 - p together, two values are told
// apart by more than 6.5e-7 (|x| + |y| + 2 max |b|), and by 2e-15, what 64 bits tell apart.
// Softmax: p is off by p (6 + 2.2 |l - m|) 2^-23, p |l - m| <= 0.37, and 14 half steps of the
// sum, at most 1.7e-6, and c by half a step.  Sums of two: four times and twice that
// (one of them may be positive, up to max |b|, and the other as far below, so the half
// steps of a softmax's two c are up to 2^-23 max |b|, of two sums twice that).
template <int Q>
__device__ __forceinline__ int choose(const float (&l)[Q], const float (&b)[Q],
                                      const float *row, int E, int k, const RouteRule &rule,
                                      int lane, uint64_t *scratch) {
    const bool biased = rule.bias != nullptr, grouped = rule.top_groups < rule.groups;
    const int size = E / rule.groups;
    uint32_t key[Q];
    float base = 0.f, part = 0.f;
    if (biased || grouped) {
        float p[Q];
        if (rule.score == MOE_SCORE_SIGMOID) {
#pragma unroll
            for (int q = 0; q < Q; ++q) p[q] = -rest32(l[q]);
        } else {
            uint32_t top = 0;
#pragma unroll
            for (int q = 0; q < Q; ++q)
                if (lane + 32 * q < E) top = max(top, to_key(l[q]));
            const float m = from_key(warp_max(top));
            float z = 0.f;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                p[q] = lane + 32 * q < E ? __expf(l[q] - m) : 0.f;
                z += p[q];
            }
            const float inv = 1.f / warp_sum(z);
#pragma unroll
            for (int q = 0; q < Q; ++q) p[q] *= inv;
        }
        uint32_t big = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            key[q] = lane + 32 * q < E ? to_key(p[q] + b[q]) : 0u;
            big = max(big, __float_as_uint(b[q]) & 0x7FFFFFFFu);
        }
        if (rule.score == MOE_SCORE_SIGMOID) {
            part = 6.5e-7f;
            base = 1.3e-6f * (biased ? __uint_as_float(warp_max(big)) : 0.f) + 2e-15f;
        } else {
            part = 2.4e-7f;
            base = 1.2e-7f * (biased ? __uint_as_float(warp_max(big)) : 0.f) + 3.6e-6f;
        }
    }
    const bool whole = size % 32 == 0;  // register q is of group 32 q / size
    uint32_t stays = 0xffu;             // bit q: expert lane + 32 q is of a group that stays
    if (grouped) {
        uint32_t v1 = 0, v2 = 0;  // of group `lane`
        if (size == 32 || size == 64 || size == 128) {
            // registers of one group merged, then all groups' two largest at once: a lane
            // keeps half of them a step (a reduction per group and value: one token 5.6
            // us, so 5.3)
            uint32_t a1[Q], a2[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                a1[q] = key[q];
                a2[q] = 0;
            }
#pragma unroll
            for (int span = 64; span <= 128; span *= 2) {
                if (size < span) continue;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    if (i < Q / 2)
                        top_two(a1[i], a2[i], a1[2 * i], a2[2 * i], a1[2 * i + 1], a2[2 * i + 1]);
                    else
                        a1[i] = a2[i] = 0;
                }
            }
            int off = 16;
#pragma unroll
            for (int n = Q / 2; n >= 1; n /= 2, off /= 2) {
                const bool upper = lane & off;
#pragma unroll
                for (int i = 0; i < n; ++i) {
                    const uint32_t g1 = __shfl_xor_sync(0xffffffffu, upper ? a1[i] : a1[i + n], off);
                    const uint32_t g2 = __shfl_xor_sync(0xffffffffu, upper ? a2[i] : a2[i + n], off);
                    const uint32_t k1 = upper ? a1[i + n] : a1[i], k2 = upper ? a2[i + n] : a2[i];
                    top_two(a1[i], a2[i], k1, k2, g1, g2);
                }
            }
            for (; off >= 1; off /= 2) {
                const uint32_t g1 = __shfl_xor_sync(0xffffffffu, a1[0], off);
                const uint32_t g2 = __shfl_xor_sync(0xffffffffu, a2[0], off);
                top_two(a1[0], a2[0], a1[0], a2[0], g1, g2);
            }
            // group g is where the bits of g chose the halves
            int src = 0;
#pragma unroll
            for (int n = Q / 2, bit = 16; n >= 1; n /= 2, bit /= 2) src |= lane & n ? bit : 0;
            v1 = __shfl_sync(0xffffffffu, a1[0], src);
            v2 = __shfl_sync(0xffffffffu, a2[0], src);
        } else {
#pragma unroll 1
            for (int g = 0; g < rule.groups; ++g) {
                const int lo = g * size - lane;  // 32 q of its members: lo .. lo + size - 1
                uint32_t a1 = 0, a2 = 0;
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const uint32_t c = (uint32_t)(32 * q - lo) < (uint32_t)size ? key[q] : 0u;
                    a2 = max(a2, min(a1, c));
                    a1 = max(a1, c);
                }
                const uint32_t t1 = warp_max(a1);
                const int winner = __ffs(__ballot_sync(0xffffffffu, a1 == t1)) - 1;
                const uint32_t t2 = warp_max(lane == winner ? a2 : a1);
                if (lane == g) { v1 = t1; v2 = t2; }
            }
        }
        const float mine = lane < rule.groups ? from_key(v1) + (size > 1 ? from_key(v2) : 0.f) : 0.f;
        const uint32_t kept = best_groups(mine, rule, lane);
        const bool in = (kept >> lane) & 1u;
        const float worst = from_key(__reduce_min_sync(0xffffffffu, in ? to_key(mine) : 0xffffffffu));
        const float best = from_key(warp_max(!in && lane < rule.groups ? to_key(mine) : 0u));
        if (!(worst - best > 4.f * base + 2.f * part * (fabsf(worst) + fabsf(best))))
            return choose_64(row, rule.bias, E, k, rule, lane, scratch);
        stays = 0;
        int g = whole ? 0 : lane / size, left = whole ? size : size - lane % size;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            stays |= ((kept >> (g & 31)) & 1u) << q;
            for (left -= 32; left <= 0; left += size) ++g;
        }
    }
    uint32_t id[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 32 * q;
        if (!biased) key[q] = to_key(l[q]);
        if (e >= E || !((stays >> q) & 1u)) key[q] = 0;
        id[q] = (uint32_t)e;
    }
    // the lane's experts, best first (equal ones by index): an odd-even merge network
#define RVQ_CE(i, j)                                                     \
    {                                                                    \
        const bool s = key[i] < key[j] || (key[i] == key[j] && id[i] > id[j]); \
        const uint32_t x = key[i], y = id[i];                            \
        key[i] = s ? key[j] : x;                                         \
        id[i] = s ? id[j] : y;                                           \
        key[j] = s ? x : key[j];                                         \
        id[j] = s ? y : id[j];                                           \
    }
    if constexpr (Q == 2) {
        RVQ_CE(0, 1)
    } else if constexpr (Q == 4) {
        RVQ_CE(0, 1) RVQ_CE(2, 3) RVQ_CE(0, 2) RVQ_CE(1, 3) RVQ_CE(1, 2)
    } else {
        RVQ_CE(0, 1) RVQ_CE(2, 3) RVQ_CE(4, 5) RVQ_CE(6, 7)
        RVQ_CE(0, 2) RVQ_CE(1, 3) RVQ_CE(4, 6) RVQ_CE(5, 7)
        RVQ_CE(1, 2) RVQ_CE(5, 6)
        RVQ_CE(0, 4) RVQ_CE(1, 5) RVQ_CE(2, 6) RVQ_CE(3, 7)
        RVQ_CE(2, 4) RVQ_CE(3, 5)
        RVQ_CE(1, 2) RVQ_CE(3, 4) RVQ_CE(5, 6)
    }
#undef RVQ_CE
    // lane s takes the s-th pick and its key; with a bias one more than k (up to 32).  (Rows
    // of the lists sorted across the warp and merged instead: 11.4 -> 14 us for 2048 tokens
    // without bias and groups.)
    uint32_t my_id = 0, my_key = 0;
    const int most = biased ? min(k + 1, 32) : k;
    const auto pick = [&](int s) {
        const uint32_t top = warp_max(key[0]);
        const uint32_t e = __reduce_min_sync(0xffffffffu, key[0] == top ? id[0] : 0xffffu);
        if (lane == s) {
            my_id = e;
            my_key = top;
        }
        if (id[0] == e) {
#pragma unroll
            for (int q = 0; q + 1 < Q; ++q) {
                key[q] = key[q + 1];
                id[q] = id[q + 1];
            }
            key[Q - 1] = 0;
        }
    };
#pragma unroll 1
    for (int s = 0; s < most; ++s) pick(s);
    if (!biased) return (int)my_id;
    // bit s: the pick after the s-th is not told apart from it
    const auto open_after = [&](int picked) {
        uint32_t next = __shfl_down_sync(0xffffffffu, my_key, 1);
        if (picked == 32) {  // the one after the last pick
            const uint32_t top = warp_max(key[0]);
            if (lane == 31) next = top;
        }
        const float x = from_key(my_key), y = from_key(next);
        return __ballot_sync(0xffffffffu, lane < picked && next != 0 &&
                                              !(x - y > base + part * (fabsf(x) + fabsf(y))));
    };
    int have = most, cut = k;
    uint32_t open = open_after(have);
    if ((open & (0xffffffffu >> (32 - k))) == 0) return (int)my_id;
    if (rule.score != MOE_SCORE_SIGMOID) return choose_64(row, rule.bias, E, k, rule, lane, scratch);
    // on until a pick is told apart from the next: the first `cut` are the candidates
#pragma unroll 1
    while ((open >> (cut - 1)) & 1u) {
        if (cut == 32) return choose_64(row, rule.bias, E, k, rule, lane, scratch);
        if (++cut == have) {
            if (have < 32) pick(have++);
            open = open_after(have);
        }
    }
    // the first `cut` values again in 64 bits, one per lane, and their order
    const double c = lane < cut ? sigmoid64(finite_or_0(row[my_id])) +
                                      (double)finite_or_0(rule.bias[my_id])
                                : 0.0;
    int place = 0;
#pragma unroll 1
    for (int s = 0; s < cut; ++s) {
        const double o = __shfl_sync(0xffffffffu, c, s);
        const uint32_t e = __shfl_sync(0xffffffffu, my_id, s);
        if (o > c || (o == c && e < my_id)) ++place;
    }
    int idx = 0;
#pragma unroll 1
    for (int s = 0; s < cut; ++s) {
        const int at = __shfl_sync(0xffffffffu, place, s);
        const uint32_t e = __shfl_sync(0xffffffffu, my_id, s);
        if (at == lane) idx = (int)e;
    }
    return idx;
}

// Chosen expert and weight of lane s < k.
template <int Q>
__device__ __forceinline__ void route_row(const float *__restrict__ row, int E, int k,
                                          const RouteRule &rule, const float (&b)[Q], int lane,
                                          uint32_t *status, uint64_t *scratch, int &my_idx,
                                          float &my_w) {
    float l[Q];
    uint32_t big = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int e = lane + 32 * q;
        l[q] = e < E ? row[e] : 0.f;
        big = max(big, __float_as_uint(l[q]) & 0x7FFFFFFFu);
    }
    if (__any_sync(0xffffffffu, big >= 0x7F800000u)) {  // reported; finite values keep the outputs in range
        if (lane == 0) set_dev_error(status, RVQ_DEV_ERR_NONFINITE);
#pragma unroll
        for (int q = 0; q < Q; ++q) l[q] = finite_or_0(l[q]);
    }
    my_idx = choose(l, b, row, E, k, rule, lane, scratch);
    const bool on = lane < k;
    const float mine = finite_or_0(row[on ? my_idx : 0]);
    const float top = from_key(warp_max(on ? to_key(mine) : 0u));
    float e;
    if (rule.score == MOE_SCORE_SIGMOID) {
        // renormalised: sigmoids over e^m, m the largest logit up to 0, so that sums of
        // very negative logits stay away from 0
        const float m = rule.renorm ? fminf(top, 0.f) : 0.f;
        const float t = expf(-fabsf(mine));
        e = mine <= 0.f ? expf(mine - m) / (1.f + t) : 1.f / (1.f + t);
    } else if (rule.renorm) {
        e = expf(mine - top);
    } else {
        uint32_t all = 0;
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (lane + 32 * q < E) all = max(all, to_key(l[q]));
        const float m = from_key(warp_max(all));
#pragma unroll
        for (int q = 0; q < Q; ++q)
            if (lane + 32 * q < E) z += expf(l[q] - m);
        e = expf(mine - m) / warp_sum(z);
    }
    my_w = rule.scale * (rule.renorm ? e / warp_sum(on ? e : 0.f) : e);
}

template <int Q>
__device__ __forceinline__ void load_bias(const RouteRule &rule, int E, int lane, uint32_t *status,
                                          float (&b)[Q]) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
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

// One block, a warp per token: choice and grouping.
template <int Q>
__global__ void __launch_bounds__(RS_NT) route_scored_one_kernel(const RouteScoredJob j) {
    __shared__ uint32_t mask[256];  // tokens of an expert
    __shared__ int cnt[256];
    extern __shared__ uint64_t scratch[];  // [warps][E]
    const int lane = threadIdx.x & 31, t = threadIdx.x >> 5;
    mask[threadIdx.x] = 0u;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    int idx = 0;
    if (t < j.n) {
        float b[Q], w;
        load_bias<Q>(j.rule, j.E, lane, j.status, b);
        route_row<Q>(j.logits + (int64_t)t * j.E, j.E, j.k, j.rule, b, lane, j.status,
                     scratch + t * j.E, idx, w);
        if (lane < j.k) {
            j.idx[t * j.k + lane] = idx;
            j.w[t * j.k + lane] = w;
            atomicOr(&mask[idx], 1u << t);
        }
    }
    __syncthreads();
    cnt[threadIdx.x] = __popc(mask[threadIdx.x]);
    __syncthreads();
    if (t == 0) {
        const int end = scan_counts(cnt, j.E, lane);
        if (lane == 0) j.offsets[j.E] = end;
    }
    __syncthreads();
    if (threadIdx.x < j.E) j.offsets[threadIdx.x] = cnt[threadIdx.x];
    if (t < j.n && lane < j.k)
        j.pairs[cnt[idx] + __popc(mask[idx] & ((1u << t) - 1u))] = t * j.k + lane;
}

// Many tokens, first launch: block b chooses for tokens run * b .. and counts its
// experts into hist[b][E].
template <int Q>
__global__ void __launch_bounds__(1024) route_scored_choose_kernel(const RouteScoredJob j) {
    __shared__ int cnt[256];
    extern __shared__ uint64_t scratch[];  // [warps][E]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < 256; e += blockDim.x) cnt[e] = 0;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    float b[Q];
    load_bias<Q>(j.rule, j.E, lane, j.status, b);
    const int t0 = blockIdx.x * j.run, t1 = min(j.n, t0 + j.run);
    for (int t = t0 + warp; t < t1; t += (int)blockDim.x / 32) {
        int idx;
        float w;
        route_row<Q>(j.logits + (int64_t)t * j.E, j.E, j.k, j.rule, b, lane, j.status,
                  scratch + warp * j.E, idx, w);
        if (lane < j.k) {
            j.idx[(int64_t)t * j.k + lane] = idx;
            j.w[(int64_t)t * j.k + lane] = w;
            atomicAdd(&cnt[idx], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < j.E; e += blockDim.x) j.hist[blockIdx.x * j.E + e] = cnt[e];
}

// Second launch: block b places its run's pairs.
__global__ void __launch_bounds__(RS_PLACE) route_scored_place_kernel(const RouteScoredJob j) {
    extern __shared__ uint32_t mask[];  // [E][words], then [E][words] of 16-bit ranks
    __shared__ int cnt[256], before[256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int words = (j.run + 31) / 32;
    uint16_t *pre = reinterpret_cast<uint16_t *>(mask + j.E * words);
    for (int i = threadIdx.x; i < j.E * words; i += RS_PLACE) mask[i] = 0u;
    if (threadIdx.x < 256) cnt[threadIdx.x] = before[threadIdx.x] = 0;
    dependency_wait();
    dependents_may_start();
    __syncthreads();
    const int t0 = blockIdx.x * j.run, t1 = min(j.n, t0 + j.run);
    const int64_t p0 = (int64_t)t0 * j.k;
    const int np = (t1 - t0) * j.k;
    for (int i = threadIdx.x; i < np; i += RS_PLACE) {
        const int t = i / j.k;
        atomicOr(&mask[j.idx[p0 + i] * words + (t >> 5)], 1u << (t & 31));
    }
    {
        // counts of all runs and of those before this one: a thread per expert and share
        // of the runs, all its loads in flight at once
        const int shares = RS_PLACE / j.E, e = threadIdx.x % j.E, share = threadIdx.x / j.E;
        int all = 0, mine = 0;
        if (share < shares) {
#pragma unroll 16
            for (int r = share; r < (int)gridDim.x; r += shares) {
                const int c = j.hist[r * j.E + e];
                all += c;
                mine += r < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&cnt[e], all);
            atomicAdd(&before[e], mine);
        }
    }
    __syncthreads();
    if (warp == 0) {
        const int end = scan_counts(cnt, j.E, lane);
        if (blockIdx.x == 0 && lane == 0) j.offsets[j.E] = end;
    } else {
        for (int e = threadIdx.x - 32; e < j.E; e += RS_PLACE - 32) {
            int run = 0;
            for (int w = 0; w < words; ++w) {
                pre[e * words + w] = (uint16_t)run;
                run += __popc(mask[e * words + w]);
            }
        }
    }
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < j.E) j.offsets[threadIdx.x] = cnt[threadIdx.x];
    for (int i = threadIdx.x; i < np; i += RS_PLACE) {
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
// A logit that is not finite is 0, as it was for the weights.
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
    const float l = in ? finite_or_0(row[idx]) : 0.f, dw = in ? j.dw[(int64_t)t * j.k + lane] : 0.f;
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
            all[q] = lane + 32 * q < j.E ? finite_or_0(row[lane + 32 * q]) : 0.f;
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

// Q: experts per lane that the kernels are made for (64 experts or fewer: half the
// instructions of 256).
template <int Q>
static rvq_status launch_choice(const RouteScoredJob &job, cudaStream_t stream) {
    static std::atomic<int> attr_done[64];  // per device; setting twice is harmless
    int dev = 0;
    RVQ_CUDA(cudaGetDevice(&dev));
    if (dev < 64 && !attr_done[dev]) {
        RVQ_CUDA(cudaFuncSetAttribute(route_scored_place_kernel,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, 160 << 10));
        RVQ_CUDA(cudaFuncSetAttribute(route_scored_choose_kernel<Q>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, 64 << 10));
        attr_done[dev] = 1;
    }
    if (job.n <= kRouteOneBlock) {
        RVQ_CUDA(launch_after(route_scored_one_kernel<Q>, 1, RS_NT,
                              (size_t)kRouteOneBlock * job.E * 8, stream, job));
        return RVQ_OK;
    }
    RouteScoredJob j = job;
    j.run = route_scored_run(j.n);
    const unsigned blocks = (unsigned)((j.n + j.run - 1) / j.run);
    // a warp per token of a run, up to 32
    const int warps = j.run < 32 ? j.run : 32;
    RVQ_CUDA(launch_after(route_scored_choose_kernel<Q>, blocks, 32 * warps, (size_t)warps * j.E * 8,
                          stream, j));
    const size_t smem = (size_t)j.E * ((j.run + 31) / 32) * 6;
    RVQ_CUDA(launch_after(route_scored_place_kernel, blocks, RS_PLACE, smem, stream, j));
    return RVQ_OK;
}

rvq_status launch_route_scored(const RouteScoredJob &job, cudaStream_t stream) {
    if (job.E <= 64) return launch_choice<2>(job, stream);
    if (job.E <= 128) return launch_choice<4>(job, stream);
    return launch_choice<8>(job, stream);
}

rvq_status launch_route_scored_backward(const RouteScoredJob &job, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((job.n + RS_NT / 32 - 1) / (RS_NT / 32));
    RVQ_CUDA(launch_after(route_scored_backward_kernel, blocks, RS_NT, 0, stream, job));
    return RVQ_OK;
}

}  // namespace rvq
