// route_scores.cu - routing to experts from given logits, and its gradient.
//
// "Appendix C - Acronyms & Symbols", tables "Core MoE symbols" (top-k set and
// gates) and "Balancing" (per-expert selection bias). For a token with logits l:
//   s = softmax(l) or sigmoid(l);  key_e = s_e + b_e, or l_e without bias and groups;
//   a group's score is the sum of its highest one or two keys; the best
//   top_groups groups stay in; the k highest keys in them are selected;
//   w_r = scale s_{e_r} (/ sum_j s_{e_j} when renormalised).
// Equal keys and groups go to the lower index. Experts whose logit or key is
// -inf or NaN are never selected: choices that are left over get index -1 and
// weight 0.
//
// The selection is that of keys computed in 64 bits, so that it does not hang on
// how an exponential rounds. One warp routes one token, in two steps:
//   route_fast   selects on fp32 keys of which the lowest 5 + log2(RE) bits give way
//                to the expert's index, so that one 32-bit maximum finds key and
//                expert, and the lower expert between equal ones; then it looks at
//                the selected experts' whole keys, neighbour by neighbour, and at the
//                highest value that the first one left out can have;
//   route_exact  does it in 64 bits, for the tokens whose fp32 keys do not tell, as two
//                of these (or two groups at the border of the selection) are closer
//                together than their error: 0.1% to 0.5% of the tokens for normal
//                logits and 256 experts.
// Bounds that route_fast relies on, from CUDA's error bounds of the functions:
//   a sigmoid 1 / (1 + x): x = __expf(-l) is off by 2 + 1.173 |l| ulp, the sum by half an
//     ulp, __fdividef by 2. Of itself s is off by (1 - s)(2 + 1.173 |l|) 2^-23 + 2.5 x 2^-23,
//     above e^-16 22.5 x 2^-23 < 2^-18; in all by 1.91 x 2^-23 < 2^-22 (the most, near l = 1);
//   a softmax, 2^-19 of itself (the sum of at most 512 terms in 16 + 5 steps, expf, the
//     division) and, but for the sum, which all keys share, 1.4 x 2^-20 down to e^-16 of the
//     largest (rounding l - m 2^-20, expf 2^-22, the product 2^-24).
// So keys without a bias are in order if 2^-17 (sigmoid) or 2^-18 (softmax) of themselves
// apart; with one the error counts absolutely, twice 2^-22 or 2^-19 of the largest score for
// two keys, and 2^-24 of each key for adding the biases; a group's score has the errors of
// the two keys that it is the sum of, each at its key's size.
// Logits themselves as keys are exact.
//
// What bounds it: the instructions, about 810 a token for 256 experts in 8 groups,
// 8 selected, sigmoids and a bias (32768 tokens: 41 us, the issue slots 66% taken and the
// ALU 58%, where reading the logits takes 7; 17 us for one expert of 256 by its logit).
#include <algorithm>
#include <type_traits>

#include "route_common.cuh"
#include "route_scores.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;   // of the forward
constexpr int kWarps = kThreads / 32;
constexpr int kUndecided = 256;  // undecided tokens that a block puts by
constexpr int kBackThreads = 256;
constexpr int kBackWarps = kBackThreads / 32;

__device__ __forceinline__ double neg_inf() { return __longlong_as_double(0xfff0000000000000ll); }

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <typename XT>
__device__ __forceinline__ float logit(const XT *src, int e) {
    const float l = to_f32(src[e]);
    return l != l ? -INFINITY : l;
}

// What a lane needs to know of the groups, once for all tokens: `width` lanes (a power
// of two) look at each group of experts, this one at those of group g from base on,
// below `end`, `width` apart; every lane takes `steps` steps, which are all inside one group and 32 experts where
// `even`. bit[q]: the first lane of expert lane + 32 q's group.
template <int RE>
struct Groups {
    int width, g, steps, base, end;
    bool even;
    uint32_t bit[RE];

    __device__ __forceinline__ Groups(const RouteArgs &a, int lane) {
        width = a.groups > 16 ? 1 : a.groups > 8 ? 2 : a.groups > 4 ? 4 : a.groups > 2 ? 8 : 16;
        g = lane / width;
        const int gs = a.E / a.groups;
        steps = (gs + width - 1) / width;
        base = g * gs + lane % width;
        end = min(g + 1, a.groups) * gs;
        even = a.groups * width == 32 && 32 % gs == 0 && gs % width == 0;
#pragma unroll
        for (int q = 0; q < RE; ++q) bit[q] = 1u << min((lane + 32 * q) / gs, a.groups - 1) * width;
    }

    // Whether expert lane + 32 q's group has its bit in `lanes`.
    __device__ __forceinline__ bool in(uint32_t lanes, int q) const {
        return (lanes & bit[q]) != 0u;
    }
};

__device__ __forceinline__ float warp_max(float v) {
    return code_key(__reduce_max_sync(0xffffffffu, key_code(v)));
}

// The maximum of a token's logits (src: its row).
template <typename XT>
__device__ __forceinline__ float top_logit(const XT *src, int E, int lane) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, logit(src, e));
    return warp_max(m);
}

// Step 1 of a token in 64 bits, by the whole block: an expert a thread, as the
// exponentials' latency is what these tokens cost. row: what the keys are made of,
// the logit, the sigmoid or exp(l - m); -inf for masked experts.
template <typename XT, int RE>
__device__ __forceinline__ void exact_scores(const XT *src, double *row, const RouteArgs &a, int lane) {
    const bool by_logit = !a.bias && a.groups == 1;
    const float m = a.sigmoid || by_logit ? 0.f : top_logit(src, a.E, lane);
    for (int e = threadIdx.x; e < 32 * RE; e += blockDim.x) {
        const float l = e < a.E ? logit(src, e) : -INFINITY;
        double v = (double)l;
        if (l != -INFINITY && !by_logit) {
            const double x = exp(a.sigmoid ? -v : v - (double)m);
            v = a.sigmoid ? 1.0 / (1.0 + x) : x;
        }
        row[e] = v;
    }
}

// Step 2, by a warp. Lane l holds experts l + 32 q; lane r returns choice r: its
// expert (-1: none) and its weight's bits.
template <typename XT, int RE>
__device__ __forceinline__ int2 route_exact(const XT *src, double *row, const RouteArgs &a, int lane) {
    const bool by_logit = !a.bias && a.groups == 1;
    const float m = a.sigmoid ? 0.f : top_logit(src, a.E, lane);
    double key[RE], z = 1.0;
#pragma unroll
    for (int q = 0; q < RE; ++q) key[q] = row[lane + 32 * q];
    if (!a.sigmoid && !(by_logit && a.renormalize)) {
        z = 0.0;
        for (int q = 0; q < RE; ++q) {
            const double v = row[lane + 32 * q];
            if (v != neg_inf()) z += by_logit ? exp(v - (double)m) : v;
        }
        z = warp_sum(z);
    }
    if (!by_logit) {
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            if (!a.sigmoid && key[q] != neg_inf()) key[q] /= z;
            if (a.bias && lane + 32 * q < a.E) key[q] += (double)a.bias[lane + 32 * q];
            if (key[q] != key[q]) key[q] = neg_inf();
        }
    }
    if (a.groups > 1) {
        const Groups<RE> gr(a, lane);
        __syncwarp();
#pragma unroll
        for (int q = 0; q < RE; ++q) row[lane + 32 * q] = key[q];
        __syncwarp();
        double t1 = neg_inf(), t2 = neg_inf();
        for (int e = gr.base; e < gr.end; e += gr.width) {
            const double v = row[e];
            t2 = v > t1 ? t1 : (v > t2 ? v : t2);
            t1 = v > t1 ? v : t1;
        }
        for (int off = 1; off < gr.width; off <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, t1, off), o2 = __shfl_xor_sync(0xffffffffu, t2, off);
            const double low = o1 > t1 ? t1 : o1, second = o2 > t2 ? o2 : t2;
            t1 = o1 > t1 ? o1 : t1;
            t2 = low > second ? low : second;
        }
        const double mine = a.group_top == 2 && t2 != neg_inf() ? t1 + t2 : t1;
        int before = 0;
        for (int o = 0; o < a.groups; ++o) {
            const double v = __shfl_sync(0xffffffffu, mine, o * gr.width);
            before += v > mine || (v == mine && o < gr.g);
        }
        const uint32_t lanes = __ballot_sync(0xffffffffu, gr.g < a.groups && before < a.top_groups);
#pragma unroll
        for (int q = 0; q < RE; ++q)
            if (!gr.in(lanes, q)) key[q] = neg_inf();
    }
    // Order-preserving codes, as key_code's; those of -inf and below are no choice.
    unsigned long long code[RE];
    constexpr unsigned long long kNone = 0x0010000000000000ull;
#pragma unroll
    for (int q = 0; q < RE; ++q) {
        const long long u = __double_as_longlong(key[q] + 0.0);
        code[q] = static_cast<unsigned long long>(u) ^ (static_cast<unsigned long long>(u >> 63) | (1ull << 63));
    }
    int choice = -1;
#pragma unroll 1
    for (int r = 0; r < a.k; ++r) {
        unsigned long long best = code[0];
        int e = lane;
#pragma unroll
        for (int q = 1; q < RE; ++q) {
            e = code[q] > best ? lane + 32 * q : e;
            best = code[q] > best ? code[q] : best;
        }
        const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
        const uint32_t top_hi = __reduce_max_sync(0xffffffffu, hi);
        const uint32_t top_lo = __reduce_max_sync(0xffffffffu, hi == top_hi ? lo : 0u);
        const uint32_t be = __reduce_min_sync(0xffffffffu, hi == top_hi && lo == top_lo ? static_cast<uint32_t>(e) : 0xffffu);
        if ((static_cast<unsigned long long>(top_hi) << 32 | top_lo) < kNone) break;
        if (lane == r) choice = static_cast<int>(be);
#pragma unroll
        for (int q = 0; q < RE; ++q) code[q] = be == static_cast<uint32_t>(lane + 32 * q) ? 0ull : code[q];
    }
    // The weights: in fp32 as route_fast's, unless they are too small for it.
    const float l = choice >= 0 ? logit(src, choice) : -INFINITY, zf = static_cast<float>(z);
    float sf = choice >= 0 ? (a.sigmoid ? __fdividef(1.f, 1.f + expf(-l)) : __fdividef(expf(l - m), zf)) : 0.f;
    if (__all_sync(0xffffffffu, choice < 0 || sf > 0x1p-80f)) {
        if (a.renormalize) {
            float sum = sf;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            sf = sum > 0.f ? __fdividef(sf, sum) : 0.f;
        }
        return make_int2(choice, __float_as_int(sf * a.scale));
    }
    double s = 0.0;
    if (a.renormalize) {
        // Over e^top, the largest of the selection's e^l (softmax) or e^min(l, 0) (sigmoid, which is that over
        // 1 + e^-|l|): scores that are nothing in 64 bits still have their shares.
        const float x = a.sigmoid ? fminf(l, 0.f) : l, top = warp_max(x);  // l: -inf without a choice
        if (choice >= 0) s = exp((double)x - (double)top) / (a.sigmoid ? 1.0 + exp(-fabs((double)l)) : 1.0);
        const double sum = warp_sum(s);
        s = sum > 0.0 ? s / sum : 0.0;
    } else if (choice >= 0) {
        s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
    }
    return make_int2(choice, __float_as_int(static_cast<float>(s * (double)a.scale)));
}

__device__ __forceinline__ void cas32(uint32_t &x, uint32_t &y) {
    const uint32_t hi = max(x, y), lo = min(x, y);
    x = hi;
    y = lo;
}

// Descending (Batcher's odd-even merge network).
template <int RE>
__device__ __forceinline__ void sort32(uint32_t (&v)[RE]) {
#pragma unroll
    for (int p = 1; p < RE; p *= 2)
#pragma unroll
        for (int k = p; k > 0; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < RE; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < RE && (i + j) / (2 * p) == (i + j + k) / (2 * p)) cas32(v[i + j], v[i + j + k]);
}

__device__ __forceinline__ uint32_t select(uint32_t which, uint32_t x, uint32_t y) {
    uint32_t r;
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tselp.b32 %0, %1, %2, p;\n\t}" : "=r"(r) : "r"(x), "r"(y), "r"(which));
    return r;
}

// What a token's keys are: its logits (no bias, no groups), or its scores with the biases, without and
// with groups.
enum { kByLogit = 0, kByScore = 1, kGrouped = 2 };

// Where expert e's fp32 key lies in a warp's buffer: four places more every 32, so that the lanes that look
// at groups of 32 experts read different banks.
constexpr int kPad = 36;
__device__ __forceinline__ int padded(int e) { return e + (e >> 5) * (kPad - 32); }

// Two highest of two pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge_top2(float &a1, float &a2, float b1, float b2) {
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

// Routes a token on fp32 keys; false if they do not decide it. Lane l holds experts
// l + 32 q: h[q] is the logit, -inf for experts that are not there, -inf or NaN for masked ones;
// bias: the experts' biases. `row` is the warp's shared buffer, holding the logits; keys: a
// second one.
template <int RE, int MODE, bool SIGMOID>
__device__ __forceinline__ bool route_fast(float (&h)[RE], const float *bias, const Groups<RE> &gr,
                                           const float *row, float *keys, const RouteArgs &a, bool exact_codes, int lane,
                                           int &choice, float &weight) {
    constexpr uint32_t kLow = 32 * RE - 1;     // the index bits of a code
    constexpr uint32_t kNone = 0x00800000u;    // codes of finite keys are not below, those of -inf are
    constexpr bool by_logit = MODE == kByLogit;
    choice = -1;
    weight = 0.f;
    float m = 0.f, z = 1.f;
    float key[RE];
    if constexpr (!SIGMOID) {
#pragma unroll
        for (int q = 0; q < RE; ++q) h[q] = fmaxf(h[q], -INFINITY);  // a NaN is a masked logit
        m = h[0];
#pragma unroll
        for (int q = 1; q < RE; ++q) m = fmaxf(m, h[q]);
        m = warp_max(m);
        if (m == -INFINITY) return true;  // nothing to select
        if (!by_logit || !a.renormalize) {  // every score
            float sum = 0.f;
#pragma unroll
            for (int q = 0; q < RE; ++q) {
                key[q] = expf(h[q] - m);
                sum += key[q];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            z = 1.f / sum;
#pragma unroll
            for (int q = 0; q < RE; ++q) key[q] *= z;
        }
    } else if constexpr (!by_logit) {
#pragma unroll
        for (int q = 0; q < RE; ++q) key[q] = __fdividef(1.f, 1.f + __expf(-h[q]));
    }
    bool sure = true;
    const float smax = SIGMOID ? 1.f : z;  // no score is larger (a softmax's largest is exp(0) z)
    const float apart = SIGMOID ? 0x1p-21f : 0x1p-18f * smax;  // what two scores may be off together
    if constexpr (by_logit) {
#pragma unroll
        for (int q = 0; q < RE; ++q) key[q] = fmaxf(h[q] + 0.f, -INFINITY);  // one zero for both signs, NaN masked
    } else {
        // 0 h is NaN for a masked expert (-inf or NaN), and so is its key, and the key of a NaN bias; the
        // maximum with -inf is -inf then.
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            key[q] = fmaxf(fmaf(h[q], 0.f, key[q]) + (a.bias ? bias[lane + 32 * q] : 0.f), -INFINITY);
            keys[lane + kPad * q] = key[q];
        }
        __syncwarp();
    }
    if constexpr (MODE == kGrouped) {
        float t1 = -INFINITY, t2 = -INFINITY;
        auto take = [&](float v) {
            t2 = fmaxf(t2, fminf(t1, v));
            t1 = fmaxf(t1, v);
        };
        if (gr.even) {
            const float *p = keys + padded(gr.base);
#pragma unroll 4
            for (int j = 0; j < gr.steps; ++j, p += gr.width) take(*p);
        } else {
#pragma unroll 4
            for (int j = 0, e = gr.base; j < gr.steps; ++j, e += gr.width) take(e < gr.end ? keys[padded(e)] : -INFINITY);
        }
        __syncwarp();
        for (int off = 1; off < gr.width; off <<= 1)
            merge_top2(t1, t2, __shfl_xor_sync(0xffffffffu, t1, off), __shfl_xor_sync(0xffffffffu, t2, off));
        // Half a group's score, which does not leave the range where the lowest finite numbers are added up.
        const float h1 = 0.5f * t1, h2 = a.group_top == 2 && t2 != -INFINITY ? 0.5f * t2 : 0.f, mine = h1 + h2;
        // Scores with the group's index in the lowest bits: the check below sees to those that this puts out
        // of order.
        const uint32_t rank = (key_code(mine) & ~31u) | (31u - gr.g);
        // Each of a group's lanes compares with every width-th group.
        int before = 0;
#pragma unroll 2
        for (int o = lane & (gr.width - 1), left = a.groups; left > 0; left -= gr.width, o += gr.width)
            before += __shfl_sync(0xffffffffu, rank, o * gr.width) > rank && o < a.groups;
        for (int off = 1; off < gr.width; off <<= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
        const bool there = gr.g < a.groups, chosen = there && before < a.top_groups;
        const uint32_t lanes = __ballot_sync(0xffffffffu, chosen);
        if (a.top_groups < a.groups) {
            // The lowest group inside against the highest one outside, each as far off as it can be: its keys
            // were rounded at their own size, of which their sum says nothing where they have opposite signs. That
            // and the sum's rounding come to 2^-23 (|h1| + |h2|); 2^-22 holds the rounding of the bounds too.
            const float off = fabsf(mine) == INFINITY ? 0.f : 0x1p-22f * (fabsf(h1) + fabsf(h2));
            const float in = -warp_max(chosen ? off - mine : -INFINITY), out = warp_max(there && !chosen ? mine + off : -INFINITY);
            if (out != -INFINITY && !(in - out > apart)) sure = false;
        }
#pragma unroll
        for (int q = 0; q < RE; ++q)
            if (!gr.in(lanes, q)) key[q] = -INFINITY;
    }
    uint32_t code[RE];
    const uint32_t low = 31u & ~static_cast<uint32_t>(lane);
#pragma unroll
    for (int q = 0; q < RE; ++q) {
        const uint32_t u = __float_as_uint(key[q]);
        const uint32_t c = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
        code[q] = (c & ~kLow) | (low + 32u * (RE - 1 - q));  // the complement of the expert's index below
    }
    sort32<RE>(code);
    // A lane that holds more than kDepth of up to 8 choices (0.1% of the tokens, 256 experts) is not followed
    // further: each round costs a select for every key that can come up.
    constexpr int kDepth = RE < 4 ? RE : 4;
    auto rounds = [&](auto depth) {
        constexpr int D = decltype(depth)::value;
#pragma unroll 1
        for (int r = 0; r < a.k; ++r) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, code[0]);
            const uint32_t mine = code[0] == top;
#pragma unroll
            for (int q = 0; q < D; ++q) code[q] = select(mine, q + 1 < D ? code[q + 1] : 0u, code[q]);
            if (lane == r) choice = static_cast<int>(top);
        }
    };
    if (a.k <= 8) rounds(std::integral_constant<int, kDepth>{});
    else rounds(std::integral_constant<int, RE>{});
    choice = lane < a.k && static_cast<uint32_t>(choice) >= kNone ? static_cast<int>(kLow - (choice & kLow)) : -1;
    if (RE > kDepth && a.k <= 8 && __any_sync(0xffffffffu, code[0] == 0u && code[RE > kDepth ? kDepth : 0] >= kNone)) sure = false;
    const uint32_t left = __reduce_max_sync(0xffffffffu, code[0]);  // the first one left out
    float l = row[max(choice, 0)];
    l = choice >= 0 ? l : -INFINITY;
    if constexpr (by_logit) {
        // Equal logits are in the order of their indices; where fp32 logits have equal codes at the
        // border, the ones left out may be higher.
        const float next = __shfl_down_sync(0xffffffffu, l, 1);
        bool fine = lane >= a.k - 1 || l >= next;
        if (!exact_codes && lane == a.k - 1 && choice >= 0 && left >= kNone)
            fine = (key_code(l) & ~kLow) > (left & ~kLow);
        if (!__all_sync(0xffffffffu, fine)) sure = false;
    } else {
        float v = keys[padded(max(choice, 0))];
        v = choice >= 0 ? v : -INFINITY;
        float next = __shfl_down_sync(0xffffffffu, v, 1);
        if (lane == a.k - 1) next = left >= kNone ? code_key(left | kLow) : -INFINITY;
        const float error = a.bias ? apart + 0x1p-23f * fabsf(v) : (SIGMOID ? 0x1p-17f : 0x1p-18f) * v;
        bool fine = lane >= a.k || next == -INFINITY || v - next > error;
        if (!__all_sync(0xffffffffu, fine || lane != a.k - 1)) {
            // The first one left out may be as high as the lowest choice by its code: its whole key counts, if
            // no other one has the same code. Behind the codes that the rounds moved up, a lane has those that they
            // did not reach (code[kDepth], up to 8 choices).
            const uint32_t behind = max(RE > 1 ? code[1] : 0u, RE > kDepth ? code[RE > kDepth ? kDepth : 0] : 0u);
            const uint32_t rest = __reduce_max_sync(0xffffffffu, code[0] == left ? behind : code[0]);
            if (lane == a.k - 1)
                fine = (rest & ~kLow) < (left & ~kLow) && v - keys[padded(static_cast<int>(kLow - (left & kLow)))] > error;
        }
        // Scores without a bias that are too small for the bounds are left to 64 bits.
        const bool small = !a.bias && choice >= 0 && !(v >= 0x1p-23f * smax);
        if (!__all_sync(0xffffffffu, fine && !small)) sure = false;
    }
    if (!sure) return false;
    // The scores of the selection, from its logits.
    float s = 0.f;
    s = SIGMOID ? __fdividef(1.f, 1.f + expf(-l)) : expf(l - m) * z;
    s = choice >= 0 ? s : 0.f;
    if (a.renormalize) {
        float sum = s;
        for (int off = 1; off < a.k; off <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        // Scores so small that fp32 loses them are left to 64 bits.
        if (!__all_sync(0xffffffffu, lane >= a.k || sum > 0x1p-80f)) return __all_sync(0xffffffffu, choice < 0);
        s = __fdividef(s, sum);
    }
    weight = s * a.scale;
    return true;
}

// A grid of one block writes its counts; the blocks of a larger one add theirs to `counts`
// (zeroed before) by atomics.
template <typename XT, int RE, int MODE, bool SIGMOID>
__global__ void __launch_bounds__(kThreads, RE > 8 ? 2 : 3) route_kernel(const __grid_constant__ RouteArgs a) {
    __shared__ int32_t hist[kRouteMaxExperts];
    __shared__ __align__(8) float rows[kWarps][(32 + kPad) * RE];  // logits and keys, or a row of 64-bit keys
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < kRouteMaxExperts; e += kThreads) hist[e] = 0;
    float *row = rows[warp], *keys = rows[warp] + 32 * RE;
    __shared__ float bias[32 * RE];
    __shared__ int undecided[kUndecided], n_undecided;  // tokens of this block left to route_exact
    for (int e = threadIdx.x; e < 32 * RE; e += kThreads) bias[e] = a.bias && e < a.E ? a.bias[e] : 0.f;
    if (threadIdx.x == 0) n_undecided = 0;
    __syncthreads();
    const Groups<RE> gr(a, lane);
    auto token = [&](int i) { return blockIdx.x + (int64_t)gridDim.x * i; };
    float ahead[RE];
    auto load = [&](int64_t t) {
        if (t >= a.T) return;
        const XT *src = static_cast<const XT *>(a.logits) + t * a.ld;
        if (a.E == 32 * RE) {
#pragma unroll
            for (int q = 0; q < RE; ++q) ahead[q] = to_f32(src[lane + 32 * q]);
        } else {
#pragma unroll
            for (int q = 0; q < RE; ++q) ahead[q] = lane + 32 * q < a.E ? to_f32(src[lane + 32 * q]) : -INFINITY;
        }
    };
    auto write = [&](int64_t t, int choice, float weight) {
        if (a.fill && __any_sync(0xffffffffu, lane < a.k && choice < 0)) {
            int n = __popc(__ballot_sync(0xffffffffu, lane < a.k && choice >= 0));  // the choices there are
            for (int e = 0; n < a.k && e < a.E; ++e)
                if (!__any_sync(0xffffffffu, lane < a.k && choice == e)) {
                    if (lane == n) choice = e;
                    ++n;
                }
        }
        if (lane < a.k) {
            a.idx[t * a.k + lane] = choice;
            a.weights[t * a.k + lane] = weight;
            if (a.counts && choice >= 0) atomicAdd(&hist[choice], 1);
        }
    };
    // Block b has tokens b, b + blocks, ..., its warps in turn. Undecided ones are put by and routed, by all
    // warps together, when the block has no others left (or no room for more).
    int i = warp;
    load(token(i));
    do {
        while (token(i) < a.T && *reinterpret_cast<volatile int *>(&n_undecided) <= kUndecided - kWarps) {
            float h[RE];
#pragma unroll
            for (int q = 0; q < RE; ++q) row[lane + 32 * q] = h[q] = ahead[q];
            const int next = i + kWarps;
            load(token(next));  // the next token's logits, while this one is routed
            __syncwarp();
            int choice;
            float weight;
            if (route_fast<RE, MODE, SIGMOID>(h, bias, gr, row, keys, a, sizeof(XT) == 2, lane, choice, weight))
                write(token(i), choice, weight);
            else if (lane == 0)
                undecided[atomicAdd(&n_undecided, 1)] = i;
            i = next;
            __syncwarp();
        }
        __syncthreads();
        const int n = n_undecided;
        for (int j0 = 0; j0 < n; j0 += kWarps) {
            for (int j = j0; j < min(n, j0 + kWarps); ++j)
                exact_scores<XT, RE>(static_cast<const XT *>(a.logits) + token(undecided[j]) * a.ld,
                                     reinterpret_cast<double *>(rows[j - j0]), a, lane);
            __syncthreads();
            if (j0 + warp < n) {
                const int64_t t = token(undecided[j0 + warp]);
                const int2 r = route_exact<XT, RE>(static_cast<const XT *>(a.logits) + t * a.ld,
                                                   reinterpret_cast<double *>(row), a, lane);
                write(t, r.x, __int_as_float(r.y));
            }
            __syncthreads();
        }
        if (threadIdx.x == 0) n_undecided = 0;
    } while (__syncthreads_or(token(i) < a.T));
    if (!a.counts) return;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
        if (gridDim.x == 1) a.counts[e] = hist[e];
        else if (hist[e]) atomicAdd(a.counts + e, hist[e]);
    }
}

// The gradient of a token's weights with respect to its logits. Lane r holds
// choice r; the row is put together in shared memory, so that an expert chosen
// twice adds up (in the order of the choices). Lane l writes (DENSE: also reads)
// experts 4 l .. 4 l + 3 of every 128 in one access where the rows allow it.
//
// The row is written once and read only where every logit has a gradient (the softmax that is
// not renormalised): 32768 x 256 fp32 in 14.4 us then, 16.4 in a loop of calls (4.2 to 4.8 TB/s, the issue slots
// 68% taken: both are near), 9.1 for the renormalised sigmoid.
template <typename XT, int N>
struct alignas(N * sizeof(XT)) Pack {
    XT v[N];
};

template <typename XT, int RE, bool DENSE, bool VEC>
__global__ void __launch_bounds__(kBackThreads) route_backward_kernel(const __grid_constant__ RouteBackwardArgs a) {
    __shared__ __align__(16) float rows[kBackWarps][32 * RE];
    constexpr int V = VEC ? (RE < 4 ? RE : 4) : 1, NV = RE / V;  // elements of an access, accesses
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *buf = rows[warp];
    auto at = [&](int i) { return (i * 32 + lane) * V; };  // the first element of access i
    auto sum = [](float v) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        return v;
    };
    const int64_t stride = (int64_t)gridDim.x * kBackWarps;
#pragma unroll
    for (int q = 0; q < RE; ++q) buf[lane + 32 * q] = 0.f;
    for (int64_t t = (int64_t)blockIdx.x * kBackWarps + warp; t < a.T; t += stride) {
        const XT *row = static_cast<const XT *>(a.logits) + t * a.ld;
        int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
        if (e >= a.E) e = -1;
        e = max(e, -1);
        float g = lane < a.k ? a.grad_weights[t * a.k + lane] * a.scale : 0.f;
        g = e >= 0 ? g : 0.f;
        Pack<XT, V> raw[NV];
        if constexpr (DENSE) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (at(i) < a.E) raw[i] = *reinterpret_cast<const Pack<XT, V> *>(row + at(i));
        }
        float l = e >= 0 ? to_f32(row[e]) : -INFINITY;
        l = fmaxf(l, -INFINITY);  // a NaN is a masked logit
        const bool live = l != -INFINITY;
        float d, mean = 0.f, p[RE];
        if constexpr (DENSE) {
            float m = l;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    p[i * V + j] = at(i) < a.E ? fmaxf(to_f32(raw[i].v[j]), -INFINITY) : -INFINITY;
                    m = fmaxf(m, p[i * V + j]);
                }
            m = warp_max(m);
            if (m == -INFINITY) m = 0.f;  // no logit at all: every probability is 0
            float z = 0.f;
#pragma unroll
            for (int q = 0; q < RE; ++q) {
                p[q] = expf(p[q] - m);
                z += p[q];
            }
            z = sum(z);
            const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
            for (int q = 0; q < RE; ++q) p[q] *= inv;
            mean = sum(live ? g * expf(l - m) * inv : 0.f);
            d = g;
        } else if (a.sigmoid) {
            const float en = expf(-fabsf(l)), r = __fdividef(1.f, 1.f + en);
            const float s = live ? (l >= 0.f ? r : en * r) : 0.f, ds = live ? (l >= 0.f ? en * r : r) : 0.f;  // s, 1 - s
            d = g * s * ds;
            if (a.renormalize) {
                float x = s, total = sum(s);
                if (!(total > 0x1p-80f)) {
                    // Scores so small that fp32 loses them: s is e^min(l, 0) r, here over the largest e^min(l, 0).
                    const float low = fminf(l, 0.f), top = warp_max(low);
                    x = live ? expf(low - top) * r : 0.f;
                    total = sum(x);
                }
                const float w = total > 0.f ? x / total : 0.f;
                d = w * (g - sum(g * w)) * ds;
            }
        } else {  // the softmax over the selection alone
            const float m = warp_max(l), x = live ? expf(l - m) : 0.f, total = sum(x);
            const float w = total > 0.f ? x / total : 0.f;
            d = w * (g - sum(g * w));
        }
        // The first lane of those with the same expert adds their terms up.
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const uint32_t first = __ffs(same) - 1;
        float total = d;
        if (__any_sync(0xffffffffu, e >= 0 && (same & (same - 1)))) {
            total = 0.f;
            for (int r = 0; r < a.k; ++r) {
                const float o = __shfl_sync(0xffffffffu, d, r);
                if ((same >> r) & 1u) total += o;
            }
        }
        const bool put = e >= 0 && lane == static_cast<int>(first);
        if (put) buf[e] = total;
        __syncwarp();
        XT *out = static_cast<XT *>(a.grad_logits) + t * a.grad_ld;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<XT, V> o;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float v = buf[at(i) + j];
                o.v[j] = from_f32<XT>(DENSE ? p[i * V + j] * (v - mean) : v);
            }
            if (at(i) < a.E) *reinterpret_cast<Pack<XT, V> *>(out + at(i)) = o;
        }
        __syncwarp();
        if (put) buf[e] = 0.f;  // the buffer is zero again for the next token
        __syncwarp();
    }
}

template <typename XT, int RE, int MODE, bool SIGMOID>
cudaError_t launch_forward(const RouteArgs &a, int num_sms, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.T + kWarps - 1) / kWarps;
    const int n = static_cast<int>(std::min<int64_t>(blocks, (int64_t)num_sms * (RE > 8 ? 2 : 3)));
    // One block needs no zeroed counts: a call every 5.2 us, 6.1 with the memset. (A cluster of up to 8 blocks
    // could add its counts up without it too: a call every 5.6 us, but its result comes 0.7 us later for 64
    // tokens and 1 to 3 us later for 128 and more.)
    if (a.counts && n > 1) {
        const cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.E, s);
        if (e != cudaSuccess) return e;
    }
    route_kernel<XT, RE, MODE, SIGMOID><<<n, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename XT, int RE>
cudaError_t launch_mode(const RouteArgs &a, int num_sms, cudaStream_t s) {
    if (a.groups > 1)
        return a.sigmoid ? launch_forward<XT, RE, kGrouped, true>(a, num_sms, s)
                         : launch_forward<XT, RE, kGrouped, false>(a, num_sms, s);
    if (a.bias)
        return a.sigmoid ? launch_forward<XT, RE, kByScore, true>(a, num_sms, s)
                         : launch_forward<XT, RE, kByScore, false>(a, num_sms, s);
    return a.sigmoid ? launch_forward<XT, RE, kByLogit, true>(a, num_sms, s)
                     : launch_forward<XT, RE, kByLogit, false>(a, num_sms, s);
}

template <typename XT, int RE>
cudaError_t launch_both(const RouteArgs *f, const RouteBackwardArgs *b, int num_sms, cudaStream_t s) {
    if (f) return launch_mode<XT, RE>(*f, num_sms, s);
    constexpr int V = RE < 4 ? RE : 4;
    auto rows_of = [&](const void *p, int64_t ld) {
        return reinterpret_cast<uintptr_t>(p) % (V * sizeof(XT)) == 0 && ld % V == 0;
    };
    const bool dense = !b->sigmoid && !b->renormalize;
    const bool vec = b->E % V == 0 && rows_of(b->grad_logits, b->grad_ld) && (!dense || rows_of(b->logits, b->ld));
    // As many blocks as fit at once (six an SM with up to 256 experts): 32768 x 256, softmax, in a loop of
    // calls 16.4 us, 17.9 with eight (a second round of a third of them); loading the next row ahead gains
    // nothing more.
    const int grid =
        static_cast<int>(std::min<int64_t>(((int64_t)b->T + kBackWarps - 1) / kBackWarps, (int64_t)num_sms * 6));
    if (dense) {
        if (vec) route_backward_kernel<XT, RE, true, true><<<grid, kBackThreads, 0, s>>>(*b);
        else route_backward_kernel<XT, RE, true, false><<<grid, kBackThreads, 0, s>>>(*b);
    } else {
        if (vec) route_backward_kernel<XT, RE, false, true><<<grid, kBackThreads, 0, s>>>(*b);
        else route_backward_kernel<XT, RE, false, false><<<grid, kBackThreads, 0, s>>>(*b);
    }
    return cudaGetLastError();
}

template <typename XT>
cudaError_t launch_any(const RouteArgs *f, const RouteBackwardArgs *b, int num_sms, cudaStream_t s) {
    const int E = f ? f->E : b->E;
    if (E <= 64) return launch_both<XT, 2>(f, b, num_sms, s);
    if (E <= 128) return launch_both<XT, 4>(f, b, num_sms, s);
    if (E <= 256) return launch_both<XT, 8>(f, b, num_sms, s);
    return launch_both<XT, 16>(f, b, num_sms, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs &a, bool bf16, int num_sms, cudaStream_t s) {
    if (a.T <= 0) return a.counts ? cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.E, s) : cudaSuccess;
    return bf16 ? launch_any<__nv_bfloat16>(&a, nullptr, num_sms, s) : launch_any<float>(&a, nullptr, num_sms, s);
}

cudaError_t launch_route_backward(const RouteBackwardArgs &a, bool bf16, int num_sms, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    return bf16 ? launch_any<__nv_bfloat16>(nullptr, &a, num_sms, s) : launch_any<float>(nullptr, &a, num_sms, s);
}

}  // namespace moe
