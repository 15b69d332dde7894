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
// The order is that of the exact keys.  fp32 keys alone would swap about one
// token's experts in a few thousand, and fp64 keys for every expert bind the
// kernel to the fp64 exponentials (123 us for 8192 tokens of 512 experts).  So
// select_fast works in fp32 with a bound on each key's error and hands a token
// in which two keys that matter are nearer than their bounds to select_exact,
// which repeats the whole rule in fp64.  Without a bias, and with group scores
// that are single keys, the logits themselves are compared: nothing is rounded.
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSelWarps = 4;         // warps (tokens) of a CTA
constexpr int kSelCand = 64;         // candidates that a warp's list holds
constexpr int kSelOneKey = 12;       // up to this k one key per lane sets the threshold

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
#pragma unroll 1
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
#pragma unroll 1
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) total += exp(key[i] - (double)top);
        total = warp_sum_d(total);
    }
    auto score = [&](double x) { return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / total; };
    const bool scored_groups = a.G > 1 && a.top2 && a.per > 1;
    if (a.bias)
#pragma unroll 1
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) key[i] = score(key[i]) + (double)sel_cap(__ldg(a.bias + lane + 32 * i));
    if (a.G > 1) {
        // lane g: group g's score
        double mine = -INFINITY;
        for (int g = 0; g < a.G; ++g) {
            double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 1
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
#pragma unroll 1
        for (int i = 0; i < SLOTS; ++i) {
            const int e = lane + 32 * i;
            if (e < a.E && !((kept >> (e / a.per)) & 1u)) key[i] = -INFINITY;
        }
    }
    uint32_t live = 0;
#pragma unroll 1
    for (int i = 0; i < SLOTS; ++i) live |= ((lane + 32 * i) < a.E ? 1u : 0u) << i;
    int my_id = 0;
    bool my_on = false;
    for (int j = 0; j < a.k; ++j) {
        double best = -INFINITY;
        int slot = -1;
#pragma unroll 1
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

// Order-preserving key of a float: larger value, larger key; 0 is below all.
MOE_DEV uint32_t sel_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
MOE_DEV float sel_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// shared memory of one warp
struct SelScratch {
    unsigned long long cand[kSelCand];   // candidates: key, then ~expert
    unsigned long long best[kSelCand];   // by rank
};

// The rule in fp32 for one token, one warp, expert e in lane e % 32.  false:
// two keys that matter are too near (or more candidates than there is room
// for): nothing is written.
//
// Error bounds.  ks: of a score.  sigmoid: __expf is off by 2 + 1.173 |x| ulp,
// which the score sees as at most (4 + 0.37 x 2.4) x 2^-24 absolute, plus 3 ulp
// of the addition and the division: 1e-6 is over twice that.  softmax: expf 2
// ulp, rounding of x - top at most 0.37 x 2^-24 of the largest score 1/S, the
// sum S 32 terms in a row, 5 folds and its terms' own errors (the mean of
// top - x under the softmax is at most ln 1024): 3.5e-6 / S; 5e-6 / S is taken.
// A key adds half a step, 2^-24 of its size.
//
// Threshold: each lane's M largest keys; t is reached by at least k of them, so
// no key below t (less both errors) is among the k best.  t comes from bisecting
// the keys' integer order by ballots, until it is reached by k to k + 2 of them:
// about 12 candidates of 512 for k = 10.  M = 2 for k > 12, where one key per
// lane would leave far more candidates than k (130 for k = 32).  Candidates go
// to the warp's list and each is ranked by counting those ahead of it.
template <int SLOTS>
MOE_DEV bool select_fast(const SelectArgs& a, int t, SelScratch& sc, float* gkey) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const float* row = a.logits + (size_t)t * a.ld;
    float x[SLOTS];
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        const int e = lane + 32 * i;
        x[i] = e < a.E ? __ldg(row + e) : -FLT_MAX;
    }
    uint32_t on = 0;
    float top = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        bool ok = sel_on(x[i]);
        x[i] = sel_cap(x[i]);
        if (a.bias && lane + 32 * i < a.E) ok = ok && sel_on(__ldg(a.bias + lane + 32 * i));
        on |= ok ? 1u << i : 0u;
        if (ok) top = fmaxf(top, x[i]);
    }
    if (!__any_sync(all, on != 0)) {                 // nothing eligible: experts 0 .. k-1, weights 0
        store_weights(a, t, lane, 0.0f, false, 0.0f, 1.0f);
        return true;
    }
    const bool top2 = a.G > 1 && a.top2 && a.per > 1;
    const bool scored = a.bias != nullptr || top2;   // keys or group scores need the scores
    float total = 1.0f, ks = 1e-6f;
    if (!a.sigmoid && (scored || !a.renorm)) {
        top = warp_max(top);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if ((on >> i) & 1u) s += expf(x[i] - top);
        total = warp_sum(s);
        ks = __fdividef(5e-6f, total);
    }
    uint32_t key[SLOTS];                             // 0: not eligible
    if (scored) {
        const float inv = __fdividef(1.0f, total);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int e = lane + 32 * i;
            const bool ok = (on >> i) & 1u;
            float v = a.sigmoid ? __fdividef(1.0f, 1.0f + __expf(-x[i])) : expf(x[i] - top) * inv;
            if (a.bias) v += ok ? sel_cap(__ldg(a.bias + e)) : 0.0f;
            if (a.G > 1 && e < a.E) gkey[e] = ok ? v : -INFINITY;
            key[i] = ok ? sel_key(a.bias ? v : x[i]) : 0u;
        }
    } else {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const int e = lane + 32 * i;
            const bool ok = (on >> i) & 1u;
            if (a.G > 1 && e < a.E) gkey[e] = ok ? x[i] : -INFINITY;
            key[i] = ok ? sel_key(x[i]) : 0u;
        }
    }
    if (a.G > 1) {
        // 2^gl lanes per group, their largest two keys folded together; each
        // group starts at another offset so that the lanes' banks differ
        const int gl = a.group_lanes_log2, L = 1 << gl;
        const int g = lane >> gl, sub = lane & (L - 1);
        const int nit = (a.per + L - 1) >> gl;
        __syncwarp();
        float b1 = -INFINITY, b2 = -INFINITY;
        if (g < a.G) {
            int it = g % nit;
            for (int n = 0; n < nit; ++n) {
                const int j = sub + (it << gl);
                const float v = j < a.per ? gkey[g * a.per + j] : -INFINITY;
                b2 = fmaxf(b2, fminf(b1, v));
                b1 = fmaxf(b1, v);
                it = it + 1 == nit ? 0 : it + 1;
            }
        }
        for (int o = L >> 1; o > 0; o >>= 1) {
            const float c1 = __shfl_xor_sync(all, b1, o), c2 = __shfl_xor_sync(all, b2, o);
            b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
            b1 = fmaxf(b1, c1);
        }
        const float mine = top2 && b2 > -INFINITY ? b1 + b2 : b1;
        // rank of this lane's group: lane g << gl speaks for group g
        int rank = 0;
        for (int q = 0; q < a.G; ++q) {
            const float v = __shfl_sync(all, mine, q << gl);
            rank += (v > mine || (v == mine && q < g)) ? 1 : 0;
        }
        const bool speaks = g < a.G && sub == 0;
        if (scored && a.keep < a.G) {
            // the last group that stays against the first that does not: errors
            // of up to two keys and their sum, at most the largest group score's
            const float big = warp_max(speaks && mine > -INFINITY ? fmaxf(fabsf(b1), fabsf(mine)) : 0.0f);
            const float in = warp_max(speaks && rank == a.keep - 1 ? mine : -INFINITY);
            const float out = warp_max(speaks && rank == a.keep ? mine : -INFINITY);
            if (out > -INFINITY && !(in - out > 4.2f * ks + 7.5e-7f * big)) return false;
        }
        const unsigned speak = __ballot_sync(all, speaks && rank < a.keep);
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) {
            const unsigned ge = ((unsigned)(lane + 32 * i) * a.per_magic) >> 20;      // e / per
            if (!((speak >> ((ge << gl) & 31u)) & 1u)) key[i] = 0u;
        }
        __syncwarp();
    }
    // the lane's largest keys
    uint32_t m1 = 0, m2 = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        m2 = max(m2, min(m1, key[i]));
        m1 = max(m1, key[i]);
    }
    if (a.k <= kSelOneKey) m2 = 0;
    uint32_t lo = __reduce_min_sync(all, m1), hi = __reduce_max_sync(all, m1);
    if (hi == 0) {                                   // no eligible expert in the groups that stay
        return false;
    }
    if (lo == 0) lo = 1;
    auto reached = [&](uint32_t v) { return __popc(__ballot_sync(all, m1 >= v)) + __popc(__ballot_sync(all, m2 >= v)); };
    if (reached(lo) < a.k) {
        lo = 1;                                      // few lanes hold keys: every eligible expert
    } else {
        while (hi - lo > 1) {
            const uint32_t mid = lo + ((hi - lo) >> 1);
            const int c = reached(mid);
            if (c >= a.k) {
                lo = mid;
                if (c <= a.k + 2) break;
            } else {
                hi = mid;
            }
        }
    }
    if (a.bias && lo > 1) {
        const float v = sel_value(lo);
        lo = max(1u, sel_key(v - (2.1f * ks + 3e-7f * fabsf(v))));
    }
    unsigned cm = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) cm |= key[i] >= lo ? 1u << i : 0u;
    const int mineN = __popc(cm);
    int incl = mineN;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(all, incl, o);
        if (lane >= o) incl += u;
    }
    const int C = __shfl_sync(all, incl, 31);
    if (C > kSelCand || C < a.k) return false;
    {
        int p = incl - mineN;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i)
            if ((cm >> i) & 1u) sc.cand[p++] = ((unsigned long long)key[i] << 32) | (uint32_t)~(lane + 32 * i);
    }
    __syncwarp();
    {
        const unsigned long long c0 = lane < C ? sc.cand[lane] : 0ull, c1 = lane + 32 < C ? sc.cand[lane + 32] : 0ull;
        int r0 = 0, r1 = 0;
        if (C <= 32) {
            for (int j = 0; j < C; ++j) r0 += sc.cand[j] > c0 ? 1 : 0;
        } else {
            for (int j = 0; j < C; ++j) {
                const unsigned long long v = sc.cand[j];
                r0 += v > c0 ? 1 : 0;
                r1 += v > c1 ? 1 : 0;
            }
        }
        if (lane < C) sc.best[r0] = c0;
        if (lane + 32 < C) sc.best[r1] = c1;
    }
    __syncwarp();
    const unsigned long long me = lane < a.k ? sc.best[lane] : 0ull;
    const int id = (int)~(uint32_t)me;
    float xs = 0.0f;
    if (lane < a.k) xs = sel_cap(__ldg(row + id));
    if (a.bias) {
        bool near = false;
        if (lane < a.k && lane + 1 < C) {
            const unsigned long long nx = sc.best[lane + 1];
            const float v = sel_value((uint32_t)(me >> 32)), u = sel_value((uint32_t)(nx >> 32));
            if (!(v - u > 2.0f * ks + 2.4e-7f * fmaxf(fabsf(v), fabsf(u)))) {
                // equal logits and biases are equal keys: the lower expert first
                const int e2 = (int)~(uint32_t)nx;
                near = !(xs == sel_cap(__ldg(row + e2)) && sel_cap(__ldg(a.bias + id)) == sel_cap(__ldg(a.bias + e2)));
            }
        }
        if (__any_sync(all, near)) return false;
    }
    store_weights(a, t, id, xs, true, top, total);
    return true;
}

template <int SLOTS>
__global__ void __launch_bounds__(kSelWarps * 32, SLOTS == 32 ? 6 : 8) k_select(SelectArgs a) {
    __shared__ SelScratch scratch[kSelWarps];
    extern __shared__ float gkeys[];                 // [kSelWarps][E] with groups
    const int w = threadIdx.x >> 5;
    const int t = blockIdx.x * kSelWarps + w;
    if (t >= a.T) return;
    if (!select_fast<SLOTS>(a, t, scratch[w], gkeys + (size_t)w * a.E)) select_exact<SLOTS>(a, t);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& args, cudaStream_t st) {
    SelectArgs a = args;
    a.group_lanes_log2 = 0;
    while (a.G > 1 && (a.G << (a.group_lanes_log2 + 1)) <= 32) ++a.group_lanes_log2;
    a.per_magic = ((1u << 20) + a.per - 1) / a.per;  // e * magic >> 20 = e / per for e, per <= 1024
    const unsigned grid = (unsigned)((a.T + kSelWarps - 1) / kSelWarps);
    const size_t smem = a.G > 1 ? sizeof(float) * kSelWarps * (size_t)a.E : 0;
    if (a.E <= 256) k_select<8><<<grid, kSelWarps * 32, smem, st>>>(a);
    else if (a.E <= 512) k_select<16><<<grid, kSelWarps * 32, smem, st>>>(a);
    else k_select<32><<<grid, kSelWarps * 32, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
