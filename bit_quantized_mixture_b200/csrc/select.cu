// Expert selection under a routing rule: softmax or sigmoid scores, a bias
// that takes part in the selection only, groups of experts, top-k, and the
// chosen experts' weights (renormalised or not, times a scale).
//
//   s_e   = softmax over the eligible experts, or 1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e; without a bias the order of the logits
//   group score = largest key, or sum of the two largest; the best groups stay
//   ids   = the k best keys of the groups that stay, key descending, expert
//           ascending on equal keys; w_j = s_j [/ sum s] * scale
//
// The order is that of the exact keys: keys are taken in fp64, in which two
// different fp32 logits or biases give different keys unless they differ by
// less than 1e-15 of a score (fp32 keys would swap about one token's experts
// in a few thousand).
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSelWarps = 4;         // warps (tokens) of a CTA

MOE_DEV double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
MOE_DEV double warp_max_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// NaN, -inf and the lowest finite value (what masks are filled with) switch
// an expert off, as a logit or as a bias; +inf counts as the largest one.
MOE_DEV bool sel_on(float v) { return v > -FLT_MAX; }
MOE_DEV float sel_cap(float v) { return fminf(v, FLT_MAX); }

// Weights of the chosen experts: lane j < k holds the j-th one's logit x (on:
// the slot has an eligible expert).  Renormalised weights are taken relative
// to the largest chosen score, so they hold where every score underflows:
// softmax exp(x - max), sigmoid exp(x - m) / (1 + exp(x)) with m = min(max, 0).
// top / total: the row's largest logit and its sum of exp(x - top).
MOE_DEV void store_weights(const SelectArgs& a, int t, int id, float x, bool on, float top, float total) {
    const int lane = threadIdx.x & 31;
    const bool live = lane < a.k && on;
    float w = 0.0f;
    if (a.renorm) {
        const float mx = warp_max(live ? x : -INFINITY);
        if (live) {
            if (!a.sigmoid) w = expf(x - mx);
            else if (x > 0.0f) w = __fdiv_rn(1.0f, 1.0f + expf(-x));
            else w = __fdiv_rn(expf(x - fminf(mx, 0.0f)), 1.0f + expf(x));
        }
        const float sum = warp_sum(w);
        w = live ? __fdiv_rn(w, sum) : 0.0f;
    } else if (live) {
        w = a.sigmoid ? __fdiv_rn(1.0f, 1.0f + expf(-x)) : __fdiv_rn(expf(x - top), total);
    }
    if (lane < a.k) {
        a.ids[(size_t)t * a.k + lane] = id;
        a.w[(size_t)t * a.k + lane] = w * a.scale;
    }
}

// The whole rule for one token in fp64, one warp, expert e in lane e % 32.
template <int SLOTS>
__device__ __noinline__ void select_exact(const SelectArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    const float* row = a.logits + (size_t)t * a.ld;
    double key[SLOTS];                   // -inf: not eligible
    float top = -INFINITY;
    bool any = false;
    for (int i = 0; i < SLOTS; ++i) {
        const int e = lane + 32 * i;
        key[i] = -INFINITY;
        if (e < a.E) {
            const float l = __ldg(row + e);
            if (sel_on(l) && (!a.bias || sel_on(__ldg(a.bias + e)))) {
                key[i] = (double)sel_cap(l);
                top = fmaxf(top, sel_cap(l));
                any = true;
            }
        }
    }
    any = __any_sync(0xffffffffu, any);
    top = warp_max(top);
    double total = 0.0;
    if (!a.sigmoid && any) {
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) total += exp(key[i] - (double)top);
        total = warp_sum_d(total);
    }
    auto score = [&](double x) { return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / total; };
    const bool scored_groups = a.G > 1 && a.top2 && a.per > 1;
    if (a.bias)
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) key[i] = score(key[i]) + (double)sel_cap(__ldg(a.bias + lane + 32 * i));
    if (a.G > 1) {
        // lane g: group g's score
        double mine = -INFINITY;
        for (int g = 0; g < a.G; ++g) {
            double b1 = -INFINITY, b2 = -INFINITY;
            for (int i = 0; i < SLOTS; ++i) {
                const int e = lane + 32 * i;
                if (e < a.E && e / a.per == g && key[i] > -INFINITY) {
                    const double v = scored_groups && !a.bias ? score(key[i]) : key[i];
                    if (v > b1) { b2 = b1; b1 = v; }
                    else if (v > b2) b2 = v;
                }
            }
            const double m1 = warp_max_d(b1);
            double v = m1;
            if (scored_groups) {
                // the second largest: the first lane holding the largest offers its next one
                const int who = __ffs(__ballot_sync(0xffffffffu, b1 == m1)) - 1;
                const double m2 = warp_max_d(lane == who ? b2 : b1);
                v = m2 > -INFINITY ? m1 + m2 : m1;
            }
            if (lane == g) mine = v;
        }
        int rank = 0;
        for (int g = 0; g < a.G; ++g) {
            const double v = __shfl_sync(0xffffffffu, mine, g);
            rank += (v > mine || (v == mine && g < lane)) ? 1 : 0;
        }
        const unsigned kept = __ballot_sync(0xffffffffu, lane < a.G && rank < a.keep);
        for (int i = 0; i < SLOTS; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / a.per)) & 1u)) key[i] = -INFINITY;
        }
    }
    uint32_t live = 0;
    for (int i = 0; i < SLOTS; ++i) live |= ((lane + 32 * i) < a.E ? 1u : 0u) << i;
    int my_id = 0;
    bool my_on = false;
    for (int j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        int slot = -1;
        for (int i = 0; i < SLOTS; ++i)
            if (((live >> i) & 1u) && (slot < 0 || key[i] > best)) { best = key[i]; slot = i; }
        const double m = warp_max_d(slot >= 0 ? best : -INFINITY);
        const uint32_t e = __reduce_min_sync(0xffffffffu, slot >= 0 && best == m ? (uint32_t)(lane + 32 * slot) : 0xffffffffu);
        if ((int)(e & 31u) == lane) live &= ~(1u << (e >> 5));
        if (lane == j) { my_id = (int)e; my_on = m > -INFINITY; }
    }
    const float x = lane < a.k && my_on ? sel_cap(__ldg(row + my_id)) : 0.0f;
    store_weights(a, t, my_id, x, my_on, top, (float)total);
}

template <int SLOTS>
__global__ void __launch_bounds__(kSelWarps * 32) k_select(SelectArgs a) {
    const int t = blockIdx.x * kSelWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    select_exact<SLOTS>(a, t);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kSelWarps - 1) / kSelWarps);
    if (a.E <= 512) k_select<16><<<grid, kSelWarps * 32, 0, st>>>(a);
    else k_select<32><<<grid, kSelWarps * 32, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
