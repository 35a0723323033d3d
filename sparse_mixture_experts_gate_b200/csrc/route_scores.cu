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
// how an exponential rounds. One warp routes one token.
#include <algorithm>

#include "route_scores.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// Routes a token with keys in 64 bits. Lane l holds experts l + 32 q: h[q] is
// the logit, -inf for experts that are not there or masked. Lane r returns
// choice r: its expert (-1: none) and its weight.
template <int RE>
__device__ __forceinline__ void route_token(const float (&h)[RE], const RouteArgs &a, int lane, int &choice,
                                            float &weight) {
    float m = -INFINITY;
#pragma unroll
    for (int q = 0; q < RE; ++q) m = fmaxf(m, h[q]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    double s[RE], key[RE];
    double z = 0.0;
#pragma unroll
    for (int q = 0; q < RE; ++q) {
        if (h[q] == -INFINITY) s[q] = 0.0;
        else s[q] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)h[q])) : exp((double)h[q] - (double)m);
        z += s[q];
    }
    if (!a.sigmoid) {
        z = warp_sum(z);
#pragma unroll
        for (int q = 0; q < RE; ++q) s[q] = z > 0.0 ? s[q] / z : 0.0;
    }
#pragma unroll
    for (int q = 0; q < RE; ++q) {
        const int e = lane + 32 * q;
        key[q] = neg_inf();
        if (h[q] == -INFINITY) continue;
        if (a.bias) key[q] = s[q] + (double)a.bias[e];
        else key[q] = a.groups > 1 ? s[q] : (double)h[q];
        if (key[q] != key[q]) key[q] = neg_inf();
    }
    if (a.groups > 1) {
        const int gs = a.E / a.groups;
        double mine = neg_inf();  // lane g: the score of group g
        for (int g = 0; g < a.groups; ++g) {
            double total = 0.0;
            int taken = -1;
            bool any = false;
            for (int i = 0; i < a.group_top; ++i) {
                double best = neg_inf();
                int be = kRouteMaxExperts;
#pragma unroll
                for (int q = 0; q < RE; ++q) {
                    const int e = lane + 32 * q;
                    if (e / gs == g && e != taken && key[q] > best) {
                        best = key[q];
                        be = e;
                    }
                }
                warp_argmax(best, be);
                if (best == neg_inf()) break;
                total += best;
                any = true;
                taken = be;
            }
            if (lane == g) mine = any ? total : neg_inf();
        }
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double o = __shfl_sync(0xffffffffu, mine, g);
            if (o > mine || (o == mine && g < lane)) ++before;
        }
        const uint32_t in = __ballot_sync(0xffffffffu, lane < a.groups && before < a.top_groups);
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            const int e = lane + 32 * q;
            if (e < a.E && !((in >> (e / gs)) & 1u)) key[q] = neg_inf();
        }
    }
    choice = -1;
    double ws = 0.0;
    for (int r = 0; r < a.k; ++r) {
        double best = neg_inf();
        int be = kRouteMaxExperts;
#pragma unroll
        for (int q = 0; q < RE; ++q)
            if (key[q] > best) {
                best = key[q];
                be = lane + 32 * q;
            }
        warp_argmax(best, be);
        if (best == neg_inf()) break;
        double sv = 0.0;
#pragma unroll
        for (int q = 0; q < RE; ++q)
            if (lane + 32 * q == be) {
                sv = s[q];
                key[q] = neg_inf();
            }
        sv = __shfl_sync(0xffffffffu, sv, be & 31);
        if (lane == r) {
            choice = be;
            ws = sv;
        }
    }
    if (a.renormalize) {
        const double sum = warp_sum(ws);
        ws = sum > 0.0 ? ws / sum : 0.0;
    }
    weight = static_cast<float>(ws * (double)a.scale);
}

template <typename XT, int RE>
__global__ void __launch_bounds__(kThreads) route_kernel(const RouteArgs a) {
    __shared__ int32_t hist[kRouteMaxExperts];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.counts) {
        for (int e = threadIdx.x; e < a.E; e += kThreads) hist[e] = 0;
        __syncthreads();
    }
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
        const XT *row = static_cast<const XT *>(a.logits) + t * a.ld;
        float h[RE];
#pragma unroll
        for (int q = 0; q < RE; ++q) {
            const int e = lane + 32 * q;
            h[q] = e < a.E ? to_f32(row[e]) : -INFINITY;
            if (h[q] != h[q]) h[q] = -INFINITY;
        }
        int choice;
        float weight;
        route_token<RE>(h, a, lane, choice, weight);
        if (lane < a.k) {
            a.idx[t * a.k + lane] = choice;
            a.weights[t * a.k + lane] = weight;
            if (a.counts && choice >= 0) atomicAdd(&hist[choice], 1);
        }
    }
    if (a.counts) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kThreads)
            if (hist[e]) atomicAdd(a.counts + e, hist[e]);
    }
}

// The gradient of a token's weights with respect to its logits. Lane r holds
// choice r; the row is put together in shared memory, so that an expert chosen
// twice adds up (in the order of the choices).
template <typename XT, int RE>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const RouteBackwardArgs a) {
    __shared__ float rows[kWarps][32 * RE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *buf = rows[warp];
    const bool dense = !a.sigmoid && !a.renormalize;
    for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps) {
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
cudaError_t launch_both(const RouteArgs *f, const RouteBackwardArgs *b, int num_sms, cudaStream_t s) {
    const int64_t T = f ? f->T : b->T;
    const int grid = static_cast<int>(std::min<int64_t>((T + kWarps - 1) / kWarps, (int64_t)num_sms * 8));
    if (f) route_kernel<XT, RE><<<grid, kThreads, 0, s>>>(*f);
    else route_backward_kernel<XT, RE><<<grid, kThreads, 0, s>>>(*b);
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
    if (a.counts) {
        const cudaError_t e = cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.E, s);
        if (e != cudaSuccess) return e;
    }
    if (a.T <= 0) return cudaSuccess;
    return bf16 ? launch_any<__nv_bfloat16>(&a, nullptr, num_sms, s) : launch_any<float>(&a, nullptr, num_sms, s);
}

cudaError_t launch_route_backward(const RouteBackwardArgs &a, bool bf16, int num_sms, cudaStream_t s) {
    if (a.T <= 0) return cudaSuccess;
    return bf16 ? launch_any<__nv_bfloat16>(nullptr, &a, num_sms, s) : launch_any<float>(nullptr, &a, num_sms, s);
}

}  // namespace moe
