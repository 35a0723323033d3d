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
//                together than their error: below 1% of the tokens for logits of
//                variance 2 and 256 experts.
// Bounds that route_fast relies on: above e^-16 of the largest possible one, a
// sigmoid is off by 2^-19 of itself (__expf's 2 + 1.2 |l| ulp), and by 2^-21
// absolutely; a softmax by 2^-19 of itself (the sum of at most 512 terms in 16 + 5
// steps, expf, the division) and, but for the sum, which all keys share, by 2^-20.
// So keys without a bias are in order if 2^-18 of themselves apart; with one the
// error counts absolutely, 2^-18 of the largest score for two, and 2^-23 of the keys
// for adding the biases. Logits themselves as keys are exact.
//
// What bounds it: the instructions, about 450 a token for 256 experts in 8 groups.
#include <algorithm>

#include "route_common.cuh"
#include "route_scores.cuh"

namespace moe {
namespace {

// Threads of a forward block: more in the one-cluster form, where a warp should
// have few tokens; 256 where the rows' buffers or the registers of 16 experts a lane ask for it.
template <int RE, bool CLUSTER>
constexpr int kForwardThreads = CLUSTER && RE <= 8 ? 512 : 256;
constexpr int kMaxCluster = 8;  // blocks that put their counts together without atomics
constexpr int kBackThreads = 256;
constexpr int kBackWarps = kBackThreads / 32;

__device__ __forceinline__ double neg_inf() { return __longlong_as_double(0xfff0000000000000ll); }

// (key, index) of the warp's highest key, the lower index between equal ones.
__device__ __forceinline__ void warp_argmax(double &key, int &e) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const double ok = __shfl_xor_sync(0xffffffffu, key, off);
        const int oe = __shfl_xor_sync(0xffffffffu, e, off);
        if (ok > key || (ok == key && oe < e)) {
            key = ok;
            e = oe;
        }
    }
}

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

// Routes a token with keys in 64 bits, which `key` [E], in shared memory, takes.
// Lane r returns choice r: its expert (-1: none) and its weight.
template <typename XT>
__device__ __noinline__ void route_exact(const XT *src, double *key, const RouteArgs &a, int lane, int &choice,
                                         float &weight) {
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32) m = fmaxf(m, logit(src, e));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    double z = 1.0;
    if (!a.sigmoid) {
        z = 0.0;
        for (int e = lane; e < a.E; e += 32) {
            const float l = logit(src, e);
            if (l != -INFINITY) z += exp((double)l - (double)m);
        }
        z = warp_sum(z);
    }
    auto score = [&](float l) {
        if (l == -INFINITY) return 0.0;
        return a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) / z;
    };
    for (int e = lane; e < a.E; e += 32) {
        const float l = logit(src, e);
        double v = neg_inf();
        if (l != -INFINITY) {
            if (a.bias) v = score(l) + (double)a.bias[e];
            else v = a.groups > 1 ? score(l) : (double)l;
            if (v != v) v = neg_inf();
        }
        key[e] = v;
    }
    __syncwarp();
    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        double mine = neg_inf();  // lane g: the score of group g
        if (lane < a.groups) {
            double t1 = neg_inf(), t2 = neg_inf();
            for (int e = lane * gs; e < (lane + 1) * gs; ++e) {
                const double v = key[e];
                if (v > t1) {
                    t2 = t1;
                    t1 = v;
                } else if (v > t2) {
                    t2 = v;
                }
            }
            mine = a.group_top == 2 && t2 != neg_inf() ? t1 + t2 : t1;
        }
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, mine, g);
            if (o > mine || (o == mine && g < lane)) ++before;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, lane < a.groups && before < a.top_groups);
        __syncwarp();
        for (int e = lane; e < a.E; e += 32)
            if (!((in >> (e / gs)) & 1u)) key[e] = neg_inf();
        __syncwarp();
    }
    choice = -1;
    for (int r = 0; r < a.k; ++r) {
        double best = neg_inf();
        int be = kRouteMaxExperts;
        for (int e = lane; e < a.E; e += 32)
            if (key[e] > best) {
                best = key[e];
                be = e;
            }
        warp_argmax(best, be);
        if (best == neg_inf()) break;
        if (lane == r) choice = be;
        if (lane == (be & 31)) key[be] = neg_inf();
        __syncwarp();
    }
    double s = choice >= 0 ? score(logit(src, choice)) : 0.0;
    if (a.renormalize) {
        const double sum = warp_sum(s);
        s = sum > 0.0 ? s / sum : 0.0;
    }
    weight = static_cast<float>(s * (double)a.scale);
    __syncwarp();
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

// Two highest of two pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge_top2(float &a1, float &a2, float b1, float b2) {
    a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
    a1 = fmaxf(a1, b1);
}

__device__ __forceinline__ float warp_max(float v) {
    return code_key(__reduce_max_sync(0xffffffffu, key_code(v)));
}

// Lanes (a power of two) that look at each group of experts.
__device__ __forceinline__ int lanes_per_group(int groups) {
    return groups > 16 ? 1 : groups > 8 ? 2 : groups > 4 ? 4 : groups > 2 ? 8 : 16;
}

// Routes a token on fp32 keys; false if they do not decide it. Lane l holds experts
// l + 32 q: h[q] is the logit, -inf for experts that are not there or masked. `row`
// is the warp's shared buffer, holding the logits; keys: a second one. bias: the lane's experts' biases; group_lane: in byte q the first lane
// of the group of expert lane + 32 q.
template <int RE>
__device__ __forceinline__ bool route_fast(const float (&h)[RE], const float (&bias)[RE],
                                           const uint32_t (&group_lane)[(RE + 3) / 4], const float *row, float *keys,
                                           const RouteArgs &a, bool exact_codes, int lane, int &choice, float &weight) {
    choice = -1;
    weight = 0.f;
    constexpr uint32_t kLow = 32 * RE - 1;  // the index bits of a code
    const bool by_logit = !a.bias && a.groups == 1;
    const bool need_all = !by_logit || (!a.sigmoid && !a.renormalize);  // every score, or those of the selection alone
    float m = 0.f, z = 1.f;
    float key[RE];
    if (!a.sigmoid) {
        m = h[0];
#pragma unroll
        for (int q = 1; q < RE; ++q) m = fmaxf(m, h[q]);
        m = warp_max(m);
        if (m == -INFINITY) return true;  // nothing to select
    }
    if (need_all) {
        float sum = 0.f;
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            key[q] = a.sigmoid ? __fdividef(1.f, 1.f + __expf(-h[q])) : expf(h[q] - m);
            sum += key[q];
        }
        if (!a.sigmoid) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            z = 1.f / sum;
        }
#pragma unroll
        for (int q = 0; q < RE; ++q) key[q] *= z;
    }
    bool sure = true;
    const float smax = a.sigmoid ? 1.f : z;  // no score is larger (a softmax's largest is exp(0) z)
    if (by_logit) {
#pragma unroll
        for (int q = 0; q < RE; ++q) key[q] = h[q];
    } else {
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            key[q] = h[q] == -INFINITY ? -INFINITY : (a.bias ? key[q] + bias[q] : key[q]);
            if (key[q] != key[q]) key[q] = -INFINITY;
        }
    }
    if (!by_logit) {
#pragma unroll
        for (int q = 0; q < RE; ++q) keys[lane + 32 * q] = key[q];
        __syncwarp();
    }
    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        const int width = lanes_per_group(a.groups), g = lane / width;
        float t1 = -INFINITY, t2 = -INFINITY;
        if (g < a.groups)
            for (int i = lane % width; i < gs; i += width) {
                const float v = keys[g * gs + i];
                t2 = fmaxf(t2, fminf(t1, v));
                t1 = fmaxf(t1, v);
            }
        for (int off = 1; off < width; off <<= 1)
            merge_top2(t1, t2, __shfl_xor_sync(0xffffffffu, t1, off), __shfl_xor_sync(0xffffffffu, t2, off));
        const float mine = t1 == -INFINITY ? -INFINITY : (a.group_top == 2 && t2 != -INFINITY ? t1 + t2 : t1);
        int before = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float v = __shfl_sync(0xffffffffu, mine, o * width);
            if (v > mine || (v == mine && o < g)) ++before;
        }
        const bool chosen = g < a.groups && before < a.top_groups;
        const uint32_t lanes = __ballot_sync(0xffffffffu, chosen);
        if (a.top_groups < a.groups) {
            // The lowest group inside against the highest one outside.
            const float in = -warp_max(chosen ? -mine : -INFINITY), out = warp_max(!chosen && g < a.groups ? mine : -INFINITY);
            if (out != -INFINITY && !(in - out > 0x1p-16f * fmaxf(smax, fmaxf(fabsf(in), fabsf(out))))) sure = false;
        }
#pragma unroll
        for (int q = 0; q < RE; ++q)
            if (!((lanes >> (group_lane[q / 4] >> (8 * (q % 4)) & 31u)) & 1u)) key[q] = -INFINITY;
    }
    uint32_t code[RE];
#pragma unroll
    for (int q = 0; q < RE; ++q)
        code[q] = key[q] == -INFINITY ? 0u : (key_code(key[q]) & ~kLow) | (kLow - (lane + 32 * q));
    sort32<RE>(code);
    for (int r = 0; r < a.k; ++r) {
        const uint32_t top = __reduce_max_sync(0xffffffffu, code[0]);
        if (code[0] == top) {
#pragma unroll
            for (int q = 0; q + 1 < RE; ++q) code[q] = code[q + 1];
            code[RE - 1] = 0u;
        }
        if (lane == r && top != 0u) choice = static_cast<int>(kLow - (top & kLow));
    }
    const uint32_t left = __reduce_max_sync(0xffffffffu, code[0]);  // the first one left out
    if (by_logit) {
        // Equal logits are in the order of their indices; where fp32 logits have equal codes at the
        // border, the ones left out may be higher.
        const float v = choice >= 0 ? row[choice] : -INFINITY;
        const float next = __shfl_down_sync(0xffffffffu, v, 1);
        bool fine = lane >= a.k - 1 || v >= next;
        if (!exact_codes && lane == a.k - 1 && choice >= 0 && left != 0u)
            fine = (key_code(v) & ~kLow) > (left & ~kLow);
        sure = __all_sync(0xffffffffu, fine);
    } else {
        const float v = choice >= 0 ? keys[choice] : -INFINITY;
        float next = __shfl_down_sync(0xffffffffu, v, 1);
        if (lane == a.k - 1) next = left != 0u ? code_key(left | kLow) : -INFINITY;
        const float error = a.bias ? 0x1p-18f * smax + 0x1p-23f * fabsf(v) : 0x1p-18f * v;
        const bool fine = lane >= a.k || next == -INFINITY || v - next > error;
        // Scores without a bias that are too small for the bounds are left to 64 bits.
        const bool small = !a.bias && choice >= 0 && !(v >= 0x1p-23f * smax);
        if (!__all_sync(0xffffffffu, fine && !small)) sure = false;
    }
    if (!sure) return false;
    // The scores of the selection, from its logits.
    const float l = choice >= 0 ? row[choice] : -INFINITY;
    float s;
    if (a.sigmoid) s = choice >= 0 ? 1.f / (1.f + expf(-l)) : 0.f;
    else s = choice >= 0 ? expf(l - m) * z : 0.f;
    if (a.renormalize) {
        float sum = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        // Scores so small that fp32 loses them are left to 64 bits.
        if (!(sum > 0x1p-80f)) return sum == 0.f && __all_sync(0xffffffffu, choice < 0);
        s = s / sum;
    }
    weight = s * a.scale;
    return true;
}

__device__ __forceinline__ int ld_shared_cluster(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// CLUSTER: the whole grid is one cluster, whose blocks add their counts up among
// themselves; otherwise they are added to `counts` (zeroed before) by atomics.
template <typename XT, int RE, bool CLUSTER>
__global__ void __launch_bounds__(kForwardThreads<RE, CLUSTER>, CLUSTER ? 1 : RE > 8 ? 2 : 3)
    route_kernel(const RouteArgs a) {
    constexpr int kThreads = kForwardThreads<RE, CLUSTER>, kWarps = kThreads / 32;
    __shared__ int32_t hist[kRouteMaxExperts];
    __shared__ __align__(8) float rows[kWarps][2][32 * RE];  // logits and keys, or a row of 64-bit keys
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.counts) {
        for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
        __syncthreads();
    }
    float *row = rows[warp][0], *keys = rows[warp][1];
    float bias[RE];
#pragma unroll
    for (int q = 0; q < RE; ++q) bias[q] = a.bias && lane + 32 * q < a.E ? a.bias[lane + 32 * q] : 0.f;
    uint32_t group_lane[(RE + 3) / 4] = {};
#pragma unroll
    for (int q = 0; q < RE; ++q)
        group_lane[q / 4] |= static_cast<uint32_t>(min((lane + 32 * q) / (a.E / a.groups), a.groups - 1) *
                                                   lanes_per_group(a.groups)) << (8 * (q % 4));
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const XT *src = static_cast<const XT *>(a.logits) + t * a.ld;
        float h[RE];
#pragma unroll
        for (int q = 0; q < RE; ++q) h[q] = lane + 32 * q < a.E ? to_f32(src[lane + 32 * q]) : -INFINITY;
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            if (h[q] != h[q]) h[q] = -INFINITY;
            row[lane + 32 * q] = h[q];
        }
        __syncwarp();
        int choice;
        float weight;
        if (!route_fast<RE>(h, bias, group_lane, row, keys, a, sizeof(XT) == 2, lane, choice, weight))
            route_exact<XT>(src, reinterpret_cast<double *>(row), a, lane, choice, weight);
        if (lane < a.k) {
            a.idx[t * a.k + lane] = choice;
            a.weights[t * a.k + lane] = weight;
            if (a.counts && choice >= 0) atomicAdd(&hist[choice], 1);
        }
        __syncwarp();
    }
    if (!a.counts) return;
    if constexpr (CLUSTER) {
        cluster_sync_all();
        for (int e = blockIdx.x + gridDim.x * threadIdx.x; e < a.E; e += gridDim.x * kThreads) {
            int n = 0;
            for (uint32_t b = 0; b < gridDim.x; ++b) n += ld_shared_cluster(mapa_shared(smem_u32(&hist[e]), b));
            a.counts[e] = n;
        }
        cluster_sync_all();  // no block leaves while others read its counts
    } else {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            if (hist[e]) atomicAdd(a.counts + e, hist[e]);
    }
}

// The gradient of a token's weights with respect to its logits. Lane r holds
// choice r; the row is put together in shared memory, so that an expert chosen
// twice adds up (in the order of the choices).
template <typename XT, int RE>
__global__ void __launch_bounds__(kBackThreads) route_backward_kernel(const RouteBackwardArgs a) {
    __shared__ float rows[kBackWarps][32 * RE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *buf = rows[warp];
    const bool dense = !a.sigmoid && !a.renormalize;
    for (int64_t t = (int64_t)blockIdx.x * kBackWarps + warp; t < a.T; t += (int64_t)gridDim.x * kBackWarps) {
        const XT *row = static_cast<const XT *>(a.logits) + t * a.ld;
        int e = lane < a.k ? a.idx[t * a.k + lane] : -1;
        if (e >= a.E) e = -1;
        const float g = e >= 0 ? a.grad_weights[t * a.k + lane] * a.scale : 0.f;
        float l = e >= 0 ? to_f32(row[e]) : -INFINITY;
        float p[RE], m = l;
        if (dense) {
#pragma unroll
            for (int q = 0; q < RE; ++q) {
                p[q] = lane + 32 * q < a.E ? to_f32(row[lane + 32 * q]) : -INFINITY;
                if (p[q] != p[q]) p[q] = -INFINITY;
                m = fmaxf(m, p[q]);
            }
        }
        if (l != l) l = -INFINITY;
        float d, mean = 0.f;
        auto sum = [](float v) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
            return v;
        };
        if (!a.sigmoid) {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        }
        const bool live = l != -INFINITY;
        if (a.sigmoid) {
            const float en = expf(-fabsf(l)), s = live ? (l >= 0.f ? 1.f : en) / (1.f + en) : 0.f;
            const float ds = live ? (l >= 0.f ? en : 1.f) / (1.f + en) : 0.f;  // 1 - s
            if (a.renormalize) {
                const float total = sum(s);
                const float w = total > 0.f ? s / total : 0.f;
                d = w * (g - sum(g * w)) * ds;
            } else {
                d = g * s * ds;
            }
        } else if (a.renormalize) {
            const float x = live ? expf(l - m) : 0.f, total = sum(x);
            const float w = total > 0.f ? x / total : 0.f;
            d = w * (g - sum(g * w));
        } else {
            float z = 0.f;
#pragma unroll
            for (int q = 0; q < RE; ++q) {
                p[q] = p[q] == -INFINITY ? 0.f : expf(p[q] - m);
                z += p[q];
            }
            z = sum(z);
            const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
            for (int q = 0; q < RE; ++q) p[q] *= inv;
            mean = sum(live ? g * expf(l - m) * inv : 0.f);
            d = g;
        }
#pragma unroll
        for (int q = 0; q < RE; ++q) buf[lane + 32 * q] = 0.f;
        __syncwarp();
        // The first lane of those with the same expert adds their terms up.
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        float total = 0.f;
        for (int r = 0; r < a.k; ++r) {
            const float o = __shfl_sync(0xffffffffu, d, r);
            if ((same >> r) & 1u) total += o;
        }
        if (e >= 0 && lane == __ffs(same) - 1) buf[e] = total;
        __syncwarp();
        XT *out = static_cast<XT *>(a.grad_logits) + t * a.grad_ld;
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            const int c = lane + 32 * q;
            const float v = buf[c];
            if (c < a.E) out[c] = from_f32<XT>(dense ? p[q] * (v - mean) : v);
        }
        __syncwarp();
    }
}

template <typename XT, int RE>
cudaError_t launch_forward(const RouteArgs &a, int num_sms, cudaStream_t s) {
    // Up to four tokens a warp of one cluster: no zeroing of the counts before (2 us of host time and a
    // launch less; 128 tokens: 4 against 6 us on the device).
    constexpr int kBig = kForwardThreads<RE, true>, kSmall = kForwardThreads<RE, false>;
    if (a.counts && a.T <= 4 * kMaxCluster * (kBig / 32)) {
        const int blocks = (a.T + kBig / 32 - 1) / (kBig / 32);
        int n = 1;
        while (n < kMaxCluster && n < blocks) n *= 2;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(n, 1, 1);
        cfg.blockDim = dim3(kBig, 1, 1);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = n;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, route_kernel<XT, RE, true>, a);
    }
    if (a.counts) {
        const cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.E, s);
        if (e != cudaSuccess) return e;
    }
    const int64_t blocks = ((int64_t)a.T + kSmall / 32 - 1) / (kSmall / 32);
    const int grid = static_cast<int>(std::min<int64_t>(blocks, (int64_t)num_sms * (RE > 8 ? 2 : 3)));
    route_kernel<XT, RE, false><<<grid, kSmall, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename XT, int RE>
cudaError_t launch_both(const RouteArgs *f, const RouteBackwardArgs *b, int num_sms, cudaStream_t s) {
    if (f) return launch_forward<XT, RE>(*f, num_sms, s);
    const int grid =
        static_cast<int>(std::min<int64_t>(((int64_t)b->T + kBackWarps - 1) / kBackWarps, (int64_t)num_sms * 8));
    route_backward_kernel<XT, RE><<<grid, kBackThreads, 0, s>>>(*b);
    return cudaGetLastError();
}

template <typename XT>
cudaError_t launch_any(const RouteArgs *f, const RouteBackwardArgs *b, int num_sms, cudaStream_t s) {
    const int E = f ? f->E : b->E;
    if (E <= 32) return launch_both<XT, 1>(f, b, num_sms, s);
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
