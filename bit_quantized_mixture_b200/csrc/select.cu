// Expert selection under a routing rule: softmax or sigmoid scores, a bias
// that takes part in the selection only, groups of experts, top-k, and the
// chosen experts' weights (renormalised or not, times a scale).
//
//   s_e   = softmax over the row's logits, or 1 / (1 + exp(-l_e))
//   key_e = s_e + bias_e; without a bias the order of the logits
//   group score = largest key, or sum of the two largest; the best groups stay
//   ids   = the k best keys of the groups that stay, key descending, then logit
//           descending, then expert ascending; w_j = s_j [/ sum s] * scale
//
// The order is that of the keys in fp64.  Scores rise with their logits, so where
// two keys are equal there (saturated scores, scores far below their biases) the
// logits tell the rest: a bias of one value for all experts changes no order.  fp32
// keys alone would swap about one token's experts in a few thousand, and fp64 keys
// for every expert bind the kernel to the fp64 exponentials (123 us for 8192 tokens
// of 512 experts).  So
// select_fast works in fp32 with a bound on each key's error.  Where the last
// group that stays and the first that does not, or two of the chosen keys, are
// nearer than their bounds, group_rank_exact and rank_exact take the keys that
// can matter again in fp64; select_exact repeats the whole rule in fp64 for the
// rare token whose candidates overflow their list.  Without a bias, and with
// group scores that are single keys, the logits themselves are compared:
// nothing is rounded.
//
// What bounds it: instructions.  32768 tokens of 1024 experts (k = 32) issue about
// 1200 per token and warp, 0.63 per cycle and scheduler, in 50 us, where the
// logits alone stream in 21 us; of 8192 tokens of 512 experts in 8 groups (17 us)
// a quarter goes to the scores, a quarter to the groups.  Warps that walk through
// several tokens and load the next row while they rank one were slower (64 and
// 22 us: a fixed share of tokens per warp against the hardware's own hand-out).
#include <float.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSelWarps = 4;         // warps of a CTA
// Up to so many tokens (four per SM) a CTA per token, whose four warps walk through
// a quarter of its long way of instructions each, then a warp per token.  us, CTA /
// warp per token: 1 token of 512 experts in 8 groups 3.9 / 5.2, 333 of 600 in 24
// groups 6.1 / 9.6, 600 tokens 8.5 / 11.6 and (512 in 8 groups) 6.0 / 6.5; 1200 tokens
// 7.0 / 6.8, 2400 10.8 / 8.6.
constexpr int kSelTeamTokens = 592;
constexpr int kSelCand = 64;         // candidates that a warp's list holds
constexpr int kSelSpare = 4;         // ... and may hold beyond k of the lanes' largest keys

// the largest of a warp's values (redux.sync on fp32: one instruction in place of
// five shuffles and five maxima; volatile, since every lane has to come to it)
MOE_DEV float warp_max1(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
// exp(v) = 2^(v log2 e) by the instruction's approximate power of two: off by at most
// 2 + 1.173 |v| ulp; results below 2^-126 are 0, which is within the bounds below
MOE_DEV float exp_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
    return r;
}
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
// an expert off: as a logit altogether, as a bias for the selection (its score
// stays in the softmax's sum); +inf counts as the largest one.
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
        const float mx = warp_max1(live ? x : -INFINITY);
        if (live) {
            if (!a.sigmoid) {
                w = expf(x - mx);
            } else {
                const float e = expf(-fabsf(x));
                w = __fdiv_rn(x > 0.0f ? 1.0f : (mx < 0.0f ? expf(x - mx) : e), 1.0f + e);
            }
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

// what the W warps of a token tell one another
template <int W>
struct SelTeam {
    float top[W], sum[W];
    int count[W];
    float2 largest[W][32];
    unsigned kept;
    bool fail;
};

// sum of exp(l - top) over the row in fp64 (softmax)
MOE_DEV double softmax_total(const SelectArgs& a, const float* row, float top) {
    double total = 0.0;
    if (!a.sigmoid)
        for (int e = threadIdx.x & 31; e < a.E; e += 32) {
            const float l = __ldg(row + e);
            if (sel_on(l)) total += exp((double)sel_cap(l) - (double)top);
        }
    return warp_sum_d(total);
}
// (called, not inlined: few tokens come here, and one copy stays in the
// instruction caches)
__device__ __noinline__ double exact_score(const SelectArgs& a, double x, float top, double total) {
    return a.sigmoid ? 1.0 / (1.0 + exp(-x)) : exp(x - (double)top) / total;
}

// A group's score by its two largest keys.  Scores and biases are added apart: the
// same two scores and biases in another combination, an exact tie, give the same bits.
MOE_DEV double sum_of_two(double s1, double s2, float b1, float b2) { return (s1 + s2) + ((double)b1 + (double)b2); }

// The whole rule for one token in fp64, one warp, expert e in lane e % 32.
template <int SLOTS>
__device__ __noinline__ void select_exact(const SelectArgs& a, int t) {
    const int lane = threadIdx.x & 31;
    const float* row = a.logits + (size_t)t * a.ld;
    double key[SLOTS];                   // -inf: not eligible
    float top = -INFINITY, low = INFINITY;
    bool any = false;
#pragma unroll 1
    for (int i = 0; i < SLOTS; ++i) {
        const int e = lane + 32 * i;
        key[i] = -INFINITY;
        if (e < a.E) {
            const float l = __ldg(row + e);
            if (sel_on(l)) {
                key[i] = (double)sel_cap(l);
                top = fmaxf(top, sel_cap(l));
                low = fminf(low, sel_cap(l));
                any = true;
            }
        }
    }
    any = __any_sync(0xffffffffu, any);
    top = warp_max1(top);
    const bool differ = top > -warp_max1(-low);      // not all logits of the row are equal
    double total = 0.0;
    if (!a.sigmoid && any) {
#pragma unroll 1
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) total += exp(key[i] - (double)top);
        total = warp_sum_d(total);
    }
    auto score = [&](double x) { return exact_score(a, x, top, total); };
    const bool scored_groups = a.G > 1 && a.top2 && a.per > 1;
    if (a.bias)
#pragma unroll 1
        for (int i = 0; i < SLOTS; ++i)
            if (key[i] > -INFINITY) {
                const float b = __ldg(a.bias + lane + 32 * i);
                key[i] = sel_on(b) ? score(key[i]) + (double)sel_cap(b) : -INFINITY;
            }
    if (a.G > 1) {
        // lane g: group g's score, and the logit of its largest key
        double mine = -INFINITY;
        float minel = -INFINITY;
        int first = 0, second = -1;      // its two experts, where their sum is the score
        for (int g = 0; g < a.G; ++g) {
            double b1 = -INFINITY, b2 = -INFINITY;
            float bl = -INFINITY;
            int e1 = 0, e2 = 0;
            const int lo = g * a.per, hi = lo + a.per;       // its experts (hi <= E)
#pragma unroll 1
            for (int i = lo >> 5; i <= (hi - 1) >> 5; ++i) {
                const int e = lane + 32 * i;
                if (e >= lo && e < hi && key[i] > -INFINITY) {
                    const double v = scored_groups && !a.bias ? score(key[i]) : key[i];
                    if (!scored_groups && v >= b1) {
                        const float l = sel_cap(__ldg(row + e));
                        bl = v > b1 ? l : fmaxf(bl, l);
                    }
                    if (v > b1) { b2 = b1; e2 = e1; b1 = v; e1 = e; }
                    else if (v > b2) { b2 = v; e2 = e; }
                }
            }
            const double m1 = warp_max_d(b1);
            if (scored_groups) {
                // the second largest: the first lane holding the largest offers its next one
                const int who = __ffs(__ballot_sync(0xffffffffu, b1 == m1)) - 1;
                const double next = lane == who ? b2 : b1;
                const double m2 = warp_max_d(next);
                const int other = __ffs(__ballot_sync(0xffffffffu, next == m2)) - 1;
                const int f1 = __shfl_sync(0xffffffffu, e1, who), f2 = __shfl_sync(0xffffffffu, other == who ? e2 : e1, other);
                if (lane == g) { first = f1; second = m2 > -INFINITY ? f2 : -1; }
            }
            const float ml = scored_groups ? 0.0f : warp_max1(b1 == m1 ? bl : -INFINITY);
            if (lane == g) { mine = m1; minel = ml; }
        }
        if (second >= 0)
            mine = sum_of_two(score((double)sel_cap(__ldg(row + first))), score((double)sel_cap(__ldg(row + second))),
                              a.bias ? sel_cap(__ldg(a.bias + first)) : 0.0f, a.bias ? sel_cap(__ldg(a.bias + second)) : 0.0f);
        int rank = 0;
        for (int g = 0; g < a.G; ++g) {
            const double v = __shfl_sync(0xffffffffu, mine, g);
            const float l = __shfl_sync(0xffffffffu, minel, g);
            rank += (v > mine || (v == mine && (l > minel || (l == minel && g < lane)))) ? 1 : 0;
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
        // the largest key, the lowest expert on equal ones
        double best = -INFINITY;
        int slot = -1;
        bool again = false;              // another of this lane's keys equals its best
#pragma unroll 4
        for (int i = 0; i < SLOTS; ++i) {
            const double v = key[i];
            const bool on = (live >> i) & 1u, up = on && (slot < 0 || v > best);
            again = !up && (again || (on && v == best));
            best = up ? v : best;
            slot = up ? i : slot;
        }
        const double m = warp_max_d(slot >= 0 ? best : -INFINITY);
        bool first = slot >= 0 && best == m;
        const unsigned lanes = __ballot_sync(0xffffffffu, first), twice = __ballot_sync(0xffffffffu, first && again);
        if (a.bias && differ && m > -INFINITY && (twice || (lanes & (lanes - 1)))) {
            // ... of equal keys with a bias the largest logit, then the lowest expert
            float l = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < SLOTS; ++i) {
                const float x = first && ((live >> i) & 1u) && key[i] == m ? sel_cap(__ldg(row + lane + 32 * i)) : -INFINITY;
                slot = x > l ? i : slot;
                l = fmaxf(l, x);
            }
            const float ml = warp_max1(l);           // (every lane comes here)
            first = first && l == ml;
        }
        const uint32_t e = __reduce_min_sync(0xffffffffu, first ? (uint32_t)(lane + 32 * slot) : 0xffffffffu);
        if ((int)(e & 31u) == lane) live &= ~(1u << (e >> 5));
        if (lane == j) { my_id = (int)e; my_on = m > -INFINITY; }
    }
    const float x = lane < a.k && my_on ? sel_cap(__ldg(row + my_id)) : 0.0f;
    store_weights(a, t, my_id, x, my_on, top, (float)total);
}

MOE_DEV float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Order-preserving key of a float: larger value, larger key; 0 is below all.
MOE_DEV uint32_t sel_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);            // -0 counts as +0
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
MOE_DEV float sel_value(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}

// shared memory of one warp: the candidates' keys in integer order, their
// experts, and the candidates by rank
struct __align__(16) SelScratch {
    uint32_t key[kSelCand];
    int expert[kSelCand];
    int order[kSelCand];
    double exact[kSelCand];              // fp64 keys, where they are needed
};

// The candidates ranked by their keys in fp64, then by their logits
__device__ __noinline__ void rank_exact(const SelectArgs& a, const float* row, float top, int C, SelScratch& sc) {
    const int lane = threadIdx.x & 31;
    const double total = softmax_total(a, row, top);
    double mine[2] = {0.0, 0.0};
    int rank[2] = {0, 0};
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
        const int j = lane + 32 * u;
        if (j < C) {
            const int e = sc.expert[j];
            const float l = sel_cap(__ldg(row + e));
            mine[u] = exact_score(a, (double)l, top, total) + (double)sel_cap(__ldg(a.bias + e));
            sc.exact[j] = mine[u];
            sc.key[j] = sel_key(l);                  // (the fp32 keys have done their work)
        }
    }
    __syncwarp();
    for (int j = 0; j < C; ++j) {
        const double v = sc.exact[j];
        for (int u = 0; u < 2; ++u) rank[u] += v > mine[u] ? 1 : 0;
    }
    auto place = [&] {
        for (int u = 0; u < 2; ++u)
            if (lane + 32 * u < C) sc.order[rank[u]] = lane + 32 * u;
        __syncwarp();
    };
    place();
    // equal keys meet at one rank, and one of them does not find itself there
    bool met = false;
    for (int u = 0; u < 2; ++u) met = met || (lane + 32 * u < C && sc.order[rank[u]] != lane + 32 * u);
    if (!__any_sync(0xffffffffu, met)) return;
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
        const int i = lane + 32 * u;
        if (i >= C) continue;
        const uint32_t li = sc.key[i];
        const int e = sc.expert[i];
        for (int j = 0; j < C; ++j)
            rank[u] += sc.exact[j] == mine[u] && (sc.key[j] > li || (sc.key[j] == li && sc.expert[j] < e)) ? 1 : 0;
    }
    __syncwarp();
    place();
}

// The candidates ranked by fp32 key, the lower expert first on equal keys.
// The keys alone decide unless two are equal: those meet at one rank, and
// one of them does not find itself there.
MOE_DEV void rank_fast(int C, SelScratch& sc) {
    const int lane = threadIdx.x & 31;
    const bool h0 = lane < C, h1 = lane + 32 < C;
    const uint32_t k0 = h0 ? sc.key[lane] : 0u, k1 = h1 ? sc.key[lane + 32] : 0u;
    const uint4* quads = reinterpret_cast<const uint4*>(sc.key);
    int r0 = 0, r1 = 0;
    if (C <= 32) {
#pragma unroll 4
        for (int j = 0; j < (C + 3) / 4; ++j) {
            const uint4 x = quads[j];
            r0 += (x.x > k0) + (x.y > k0) + (x.z > k0) + (x.w > k0);
        }
    } else {
#pragma unroll 4
        for (int j = 0; j < (C + 3) / 4; ++j) {
            const uint4 x = quads[j];
            r0 += (x.x > k0) + (x.y > k0) + (x.z > k0) + (x.w > k0);
            r1 += (x.x > k1) + (x.y > k1) + (x.z > k1) + (x.w > k1);
        }
    }
    if (h0) sc.order[r0] = lane;
    if (h1) sc.order[r1] = lane + 32;
    __syncwarp();
    const bool met = (h0 && sc.order[r0] != lane) || (h1 && sc.order[r1] != lane + 32);
    if (__any_sync(0xffffffffu, met)) {
        const int e0 = h0 ? sc.expert[lane] : 0, e1 = h1 ? sc.expert[lane + 32] : 0;
        for (int j = 0; j < C; ++j) {
            const uint32_t x = sc.key[j];
            const int o = sc.expert[j];
            r0 += x == k0 && o < e0 ? 1 : 0;
            r1 += x == k1 && o < e1 ? 1 : 0;
        }
        if (h0) sc.order[r0] = lane;
        if (h1) sc.order[r1] = lane + 32;
        __syncwarp();
    }
}

// Twice the relative error of a score s (or exp(l - top)) taken by exp_approx, which is
// off by 2 + 1.173 |x| ulp with |x| at most 1 - ln s; below kSelTiny nothing is
// said of it (scores underflow).
constexpr float kSelTiny = 1e-30f;
MOE_DEV float score_error(float s) { return 3e-6f + 6e-7f * fabsf(__logf(fmaxf(s, 1e-38f))); }

// The rank of the lane's group (lanes as in select_fast) by fp64 scores; -1:
// too many members to list.  Only members whose fp32 key reaches their group's
// second largest (largest: max scores), less both errors, can be among its two
// largest keys: they are listed first, so that the lanes take their fp64 keys
// side by side.
__device__ __noinline__ int group_rank_exact(const SelectArgs& a, const float* row, float top, const float* gkey, float b1, float b2,
                                             float ks, SelScratch& sc) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    const int gl = a.group_lanes_log2, g = lane >> gl, L = 1 << gl;
    const double total = softmax_total(a, row, top);
    const bool top2 = a.top2 && a.per > 1;
    const float last = top2 && b2 > -INFINITY ? b2 : b1;
    const float bar = a.bias ? last - (2.1f * ks + 3e-7f * fabsf(last)) : (last > kSelTiny ? last * (1.0f - score_error(last)) : 0.0f);
    int n = 0;
    for (int j0 = 0; j0 < a.per; j0 += L) {
        const int j = j0 + (lane & (L - 1)), e = g * a.per + j;
        const bool hit = g < a.G && j < a.per && gkey[e] > -INFINITY && gkey[e] >= bar;
        const unsigned who = __ballot_sync(all, hit);
        const int p = n + __popc(who & ((1u << lane) - 1u));
        n += __popc(who);
        if (n > kSelCand) return -1;
        if (hit) { sc.expert[p] = e; sc.order[p] = g; }
    }
    __syncwarp();
    for (int j = lane; j < n; j += 32) {
        const float l = sel_cap(__ldg(row + sc.expert[j])), b = a.bias ? sel_cap(__ldg(a.bias + sc.expert[j])) : 0.0f;
        // sums of two: score and bias apart; single keys: the key, and the logit that
        // decides between equal ones
        const double s = exact_score(a, (double)l, top, total);
        sc.exact[j] = top2 ? s : s + (double)b;
        sc.key[j] = top2 ? __float_as_uint(b) : sel_key(l);
    }
    __syncwarp();
    double d1 = -INFINITY, d2 = -INFINITY;
    uint32_t dl = 0u;                                // the largest key's logit
    int j1 = 0, j2 = 0;
    for (int j = 0; j < n; ++j)
        if (sc.order[j] == g) {
            const uint32_t l = sc.key[j];
            const double x = top2 ? sc.exact[j] + (double)__uint_as_float(l) : sc.exact[j];
            if (!top2) dl = x > d1 || (x == d1 && l > dl) ? l : dl;
            if (x > d1) { d2 = d1; j2 = j1; d1 = x; j1 = j; }
            else if (x > d2) { d2 = x; j2 = j; }
        }
    const double mine = top2 && d2 > -INFINITY ? sum_of_two(sc.exact[j1], sc.exact[j2], __uint_as_float(sc.key[j1]), __uint_as_float(sc.key[j2])) : d1;
    __syncwarp();
    int rank = 0;
    for (int q = 0; q < a.G; ++q) {
        const double x = __shfl_sync(all, mine, q << gl);
        const uint32_t l = __shfl_sync(all, dl, q << gl);
        rank += (x > mine || (x == mine && (l > dl || (l == dl && q < g)))) ? 1 : 0;
    }
    return rank;
}

// The groups that stay, as a mask of the lanes that speak for them (group g's
// first: g << group_lanes_log2); fail: group_rank_exact could not tell.  One warp.
template <bool VEC>
MOE_DEV unsigned choose_groups(const SelectArgs& a, const float* row, float top, const float* gkey, float ks, bool scored, bool top2,
                               SelScratch& sc, bool& fail) {
    const int lane = threadIdx.x & 31;
    const unsigned all = 0xffffffffu;
    // 2^gl lanes per group, their largest two keys folded together; each
    // group starts at another offset so that the lanes' banks differ
    const int gl = a.group_lanes_log2, L = 1 << gl;
    const int g = lane >> gl, sub = lane & (L - 1);
    float b1 = -INFINITY, b2 = -INFINITY;
    auto take = [&](float x) {
        b2 = fmaxf(b2, fminf(b1, x));
        b1 = fmaxf(b1, x);
    };
    if (g < a.G) {
        const bool quads = VEC && (a.per & 3) == 0;
        const int m = quads ? a.per >> 2 : a.per, nit = (m + L - 1) >> gl;
        int it = g % nit;
        if (quads) {
#pragma unroll 4
            for (int n = 0; n < nit; ++n) {
                const int j = sub + (it << gl);
                const float4 x = j < m ? *reinterpret_cast<const float4*>(gkey + g * a.per + 4 * j)
                                       : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                take(x.x); take(x.y); take(x.z); take(x.w);
                it = it + 1 == nit ? 0 : it + 1;
            }
        } else {
#pragma unroll 4
            for (int n = 0; n < nit; ++n) {
                const int j = sub + (it << gl);
                take(j < m ? gkey[g * a.per + j] : -INFINITY);
                it = it + 1 == nit ? 0 : it + 1;
            }
        }
    }
    __syncwarp();
    for (int o = L >> 1; o > 0; o >>= 1) {
        const float c1 = __shfl_xor_sync(all, b1, o), c2 = __shfl_xor_sync(all, b2, o);
        b2 = fmaxf(fmaxf(b2, c2), fminf(b1, c1));
        b1 = fmaxf(b1, c1);
    }
    const float mine = top2 && b2 > -INFINITY ? b1 + b2 : b1;
    // rank of this lane's group: lane g << gl speaks for group g
    int rank = 0;
#pragma unroll 4
    for (int q = 0; q < a.G; ++q) {
        const float x = __shfl_sync(all, mine, q << gl);
        rank += (x > mine || (x == mine && q < g)) ? 1 : 0;
    }
    const bool speaks = g < a.G && sub == 0;
    if (scored && a.keep < a.G) {
        // the last group that stays against the first that does not: errors
        // of up to two keys and their sum, at most the largest group score's
        const float big = warp_max1(speaks && mine > -INFINITY ? fmaxf(fabsf(b1), fabsf(mine)) : 0.0f);
        const float in = warp_max1(speaks && rank == a.keep - 1 ? mine : -INFINITY);
        const float out = warp_max1(speaks && rank == a.keep ? mine : -INFINITY);
        // (without a bias both are sums of scores, whose errors are relative)
        const float near = a.bias ? 4.2f * ks + 7.5e-7f * big : (in > kSelTiny ? score_error(out) * (in + out) : INFINITY);
        if (out > -INFINITY && !(in - out > near)) {
            rank = group_rank_exact(a, row, top, gkey, b1, b2, ks, sc);
            fail = rank < 0;
        }
    }
    return __ballot_sync(all, speaks && rank < a.keep);
}

// The rule in fp32 for one token, W warps; lane l of warp w holds the experts
// 128 c + 4 ((l + 9 c) % 32) + q of chunk c = W i + w in v[4 i + q] (turned from
// chunk to chunk, so that the groups that stay are not all in a few lanes).  With
// W > 1 warp 0 alone chooses the groups and ranks the candidates.  Group scores, and then keys, that are nearer
// than their errors are taken again in fp64.  false: the candidates are more
// than the list holds, or fewer than k; nothing is written.
//
// Error bounds.  ks: of a score.  sigmoid: exp_approx is off by 2 + 1.173 |x| ulp,
// which the score sees as at most (4 + 0.37 x 2.4) x 2^-24 absolute, plus 3 ulp
// of the addition and the division: 1e-6 is over twice that; where the largest
// logit m of the row is negative the same holds relative to exp(m), with 2 + 1.173 |m|
// ulp.  softmax: exp_approx
// (as above, and x - top rounded) 5 x 2^-24 of the largest score 1/S, the
// sum S 32 terms in a row, 5 folds and its terms' own errors (the mean of
// top - x under the softmax is at most ln 1024): 4e-6 / S; 5e-6 / S is taken.
// A key adds half a step, 2^-24 of its size.
//
// Threshold: each lane's two largest keys; t is reached by at least k of them,
// so no key below t (less both errors) is among the k best.  t comes from
// bisecting the keys' integer order by ballots, until it is reached by k to
// k + 4 of them: about 15 candidates of 512 for k = 10 and 40 of 1024 for
// k = 32 (one key per lane would leave 130 there).  The candidates go to the
// warp's list and each is ranked by counting those ahead of it.
template <int CH, bool VEC, int W>
MOE_DEV bool select_fast(const SelectArgs& a, int t, SelScratch& sc, float* gkey, SelTeam<W>& team) {
    constexpr int SLOTS = 4 * CH;
    const int lane = threadIdx.x & 31, wid = W > 1 ? (int)threadIdx.x >> 5 : 0;
    auto sync = [] {
        if (W > 1) __syncthreads();
        else __syncwarp();
    };
    const unsigned all = 0xffffffffu;
    const float* row = a.logits + (size_t)t * a.ld;
    auto first = [&](int i) {
        const int c = W * i + wid;
        return 128 * c + 4 * ((lane + 9 * c) & 31);
    };
    // four consecutive floats from p[e], off: what stands for entries past E
    auto load4 = [&](const float* p, int e, float off, float* d) {
        if (VEC) {
            const float4 q = e < a.E ? __ldg(reinterpret_cast<const float4*>(p + e)) : make_float4(off, off, off, off);
            d[0] = q.x; d[1] = q.y; d[2] = q.z; d[3] = q.w;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = e + q < a.E ? __ldg(p + e + q) : off;
        }
    };
    float v[SLOTS];                                  // on: above -FLT_MAX
#pragma unroll
    for (int i = 0; i < CH; ++i) load4(row, first(i), -FLT_MAX, v + 4 * i);
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) v[i] = fminf(fmaxf(v[i], -FLT_MAX), FLT_MAX);      // NaN and -inf are off, +inf is capped
    const bool top2 = a.G > 1 && a.top2 && a.per > 1;
    const bool scored = a.bias != nullptr || top2;   // keys or group scores need the scores
    // (total also divides unnormalised weights: with expf in place of exp_approx their
    // error over 2000 rows of 600 was 5.8e-8 in place of 6.1e-8 on average and the same
    // at most, for 8192 rows in 37.5 us in place of 36.2)
    float top = -FLT_MAX, total = 1.0f, ks = 1e-6f;
    if (!a.sigmoid && (scored || !a.renorm)) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) top = fmaxf(top, v[i]);
        top = warp_max1(top);
        if (W > 1) {
            if (lane == 0) team.top[wid] = top;
            sync();
            for (int w = 0; w < W; ++w) top = fmaxf(top, team.top[w]);
        }
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) s += exp_approx(v[i] - top);     // 0 for those that are off
        total = warp_sum(s);
        if (W > 1) {
            if (lane == 0) team.sum[wid] = total;
            sync();
            total = 0.0f;
            for (int w = 0; w < W; ++w) total += team.sum[w];
        }
        // without a bias the groups compare exp(l - top) itself, total times the scores
        ks = a.bias ? __fdividef(5e-6f, total) : 5e-6f;
    }
    if (a.sigmoid && a.bias) {
#pragma unroll
        for (int i = 0; i < SLOTS; ++i) top = fmaxf(top, v[i]);
        top = warp_max1(top);
        if (W > 1) {
            if (lane == 0) team.top[wid] = top;
            sync();
            for (int w = 0; w < W; ++w) top = fmaxf(top, team.top[w]);
        }
        if (top < 0.0f) ks = __expf(top) * (1e-6f + 3e-7f * fabsf(top)) + 1e-37f;
    }
    if (scored || a.G > 1) {
        const float inv = a.bias ? __fdividef(1.0f, total) : 1.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int e = first(i);
            float b[4] = {0.0f, 0.0f, 0.0f, 0.0f}, g[4];
            if (a.bias) load4(a.bias, e, -FLT_MAX, b);
#pragma unroll
            for (int q = 0; q < 4; ++q) g[q] = v[4 * i + q];
            if (scored) {
                if (a.sigmoid) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) g[q] = rcp_approx(1.0f + exp_approx(-g[q]));
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) g[q] = exp_approx(g[q] - top) * inv;
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) g[q] = sel_on(v[4 * i + q]) && sel_on(b[q]) ? g[q] + sel_cap(b[q]) : -INFINITY;
            if (a.bias) {
#pragma unroll
                for (int q = 0; q < 4; ++q) v[4 * i + q] = g[q];
            }
            if (VEC) {
                if (e < a.E) *reinterpret_cast<float4*>(gkey + e) = make_float4(g[0], g[1], g[2], g[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (e + q < a.E) gkey[e + q] = g[q];
            }
        }
        sync();
    }
    if (a.G > 1) {
        const int gl = a.group_lanes_log2;
        bool fail = false;
        unsigned kept = wid == 0 ? choose_groups<VEC>(a, row, top, gkey, ks, scored, top2, sc, fail) : 0u;
        if (W > 1) {
            if (wid == 0 && lane == 0) { team.kept = kept; team.fail = fail; }
            sync();
            kept = team.kept;
            fail = team.fail;
        }
        if (fail) return false;
        auto stays = [&](int e) { return (kept >> (((((unsigned)e * a.per_magic) >> 20) << gl) & 31u)) & 1u; };
        if ((a.per & 3) == 0) {                      // four neighbours share their group
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (!stays(first(i))) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[4 * i + q] = -FLT_MAX;
                }
        } else {
#pragma unroll
            for (int i = 0; i < SLOTS; ++i)
                if (!stays(first(i / 4) + (i & 3))) v[i] = -FLT_MAX;
        }
    }
    // the lane's largest keys in their integer order, 0 for none
    float f1 = -FLT_MAX, f2 = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
        f2 = fmaxf(f2, fminf(f1, v[i]));
        f1 = fmaxf(f1, v[i]);
    }
    if (W > 1) {                                     // ... of the whole team: the same experts' lanes together
        team.largest[wid][lane] = make_float2(f1, f2);
        sync();
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wid) continue;
            const float2 o = team.largest[w][lane];
            f2 = fmaxf(fmaxf(f2, o.y), fminf(f1, o.x));
            f1 = fmaxf(f1, o.x);
        }
    }
    const uint32_t m1 = sel_on(f1) ? sel_key(f1) : 0u, m2 = sel_on(f2) ? sel_key(f2) : 0u;
    uint32_t lo = max(__reduce_min_sync(all, m1), 1u), hi = __reduce_max_sync(all, m1);
    if (hi == 0) {                                   // nothing eligible: experts 0 .. k-1, weights 0
        if (wid == 0) store_weights(a, t, lane, 0.0f, false, 0.0f, 1.0f);
        return true;
    }
    auto reached = [&](uint32_t x) { return __popc(__ballot_sync(all, m1 >= x)) + __popc(__ballot_sync(all, m2 >= x)); };
    const float lowest = sel_value(sel_key(-FLT_MAX) + 1u);
    float bar = lowest;                              // few lanes hold keys: every eligible expert
    if (reached(lo) >= a.k) {
        while (hi - lo > 1) {
            const uint32_t mid = lo + ((hi - lo) >> 1);
            const int c = reached(mid);
            if (c >= a.k) {
                lo = mid;
                if (c <= a.k + kSelSpare) break;
            } else {
                hi = mid;
            }
        }
        bar = fmaxf(sel_value(lo), lowest);
        if (a.bias) bar = fmaxf(bar - (2.1f * ks + 3e-7f * fabsf(bar)), lowest);
    }
    unsigned cm = 0;
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) cm |= v[i] >= bar ? 1u << i : 0u;
    const int n = __popc(cm);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(all, incl, o);
        if (lane >= o) incl += u;
    }
    int C = __shfl_sync(all, incl, 31), before = 0;
    if (W > 1) {
        if (lane == 0) team.count[wid] = C;
        sync();
        C = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w == wid) before = C;
            C += team.count[w];
        }
    }
    if (C > kSelCand || C < a.k) return false;
    for (int p = before + incl - n; cm; cm &= cm - 1) {
        const int i = __ffs(cm) - 1;
        sc.expert[p++] = first(i >> 2) + (i & 3);
    }
    sync();
    if (wid != 0) return true;
    // the last four are filled up with 0, which is behind all
    for (int j = lane; j < ((C + 3) & ~3); j += 32)
        sc.key[j] = j < C ? sel_key(a.bias ? gkey[sc.expert[j]] : sel_cap(__ldg(row + sc.expert[j]))) : 0u;
    __syncwarp();
    rank_fast(C, sc);
    if (a.bias) {
        // neighbours in the order, and the k-th against the next one
        bool near = false;
        if (lane < a.k && lane + 1 < C) {
            const int j1 = sc.order[lane], j2 = sc.order[lane + 1];
            const float x = sel_value(sc.key[j1]), y = sel_value(sc.key[j2]);
            if (!(x - y > 2.0f * ks + 2.4e-7f * fmaxf(fabsf(x), fabsf(y)))) {
                // equal logits and biases are equal keys: the lower expert first.  Behind
                // the k-th an equal key says nothing: the one after it may be nearer
                // than fp32 tells, and is not looked at.
                const int e1 = sc.expert[j1], e2 = sc.expert[j2];
                near = !(lane + 1 < a.k && sel_cap(__ldg(row + e1)) == sel_cap(__ldg(row + e2)) && sel_cap(__ldg(a.bias + e1)) == sel_cap(__ldg(a.bias + e2)));
            }
        }
        if (__any_sync(all, near)) rank_exact(a, row, top, C, sc);
    }
    const int j = lane < a.k ? sc.order[lane] : 0;
    const int id = sc.expert[j];
    const float xs = lane < a.k ? (a.bias ? sel_cap(__ldg(row + id)) : sel_value(sc.key[j])) : 0.0f;
    store_weights(a, t, id, xs, true, top, total);
    return true;
}

// One token per warp: kSelWarps tokens of a CTA
template <int CH, bool VEC>
__global__ void __launch_bounds__(kSelWarps * 32, CH == 8 ? 6 : 8) k_select(const __grid_constant__ SelectArgs a) {
    __shared__ SelScratch scratch[kSelWarps];
    extern __shared__ __align__(16) float gkeys[];   // [kSelWarps][key_room] with groups or a bias
    const int w = threadIdx.x >> 5;
    const int t = blockIdx.x * kSelWarps + w;
    if (t >= a.T) return;
    SelTeam<1> alone;
    if (!select_fast<CH, VEC, 1>(a, t, scratch[w], gkeys + w * a.key_room, alone)) select_exact<4 * CH>(a, t);
}

// One token per CTA
template <int CH, bool VEC>
__global__ void __launch_bounds__(kSelWarps * 32) k_select_team(const __grid_constant__ SelectArgs a) {
    __shared__ SelScratch scratch;
    __shared__ SelTeam<kSelWarps> team;
    extern __shared__ __align__(16) float gkeys[];   // [key_room] with groups or a bias
    if (!select_fast<CH, VEC, kSelWarps>(a, blockIdx.x, scratch, gkeys, team) && threadIdx.x < 32) select_exact<32>(a, blockIdx.x);
}

template <int CH, int TEAM_CH>
void launch_ch(const SelectArgs& a, cudaStream_t st) {
    // rows of whole, aligned 16-byte vectors
    const bool vec = a.E % 4 == 0 && (a.T == 1 || a.ld % 4 == 0) && (reinterpret_cast<uintptr_t>(a.logits) & 15u) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0;
    const size_t keys = a.G > 1 || a.bias ? sizeof(float) * (size_t)a.key_room : 0;
    if (a.T <= kSelTeamTokens) {
        if (vec) k_select_team<TEAM_CH, true><<<a.T, kSelWarps * 32, keys, st>>>(a);
        else k_select_team<TEAM_CH, false><<<a.T, kSelWarps * 32, keys, st>>>(a);
        return;
    }
    const unsigned grid = (unsigned)((a.T + kSelWarps - 1) / kSelWarps);
    if (vec) k_select<CH, true><<<grid, kSelWarps * 32, kSelWarps * keys, st>>>(a);
    else k_select<CH, false><<<grid, kSelWarps * 32, kSelWarps * keys, st>>>(a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& args, cudaStream_t st) {
    SelectArgs a = args;
    a.group_lanes_log2 = 0;
    while (a.G > 1 && (a.G << (a.group_lanes_log2 + 1)) <= 32) ++a.group_lanes_log2;
    a.per_magic = ((1u << 20) + a.per - 1) / a.per;  // e * magic >> 20 = e / per for e, per <= 1024
    a.key_room = (a.E + 3) & ~3;
    if (a.E <= 256) launch_ch<2, 1>(a, st);
    else if (a.E <= 512) launch_ch<4, 1>(a, st);
    else launch_ch<8, 2>(a, st);
    return cudaGetLastError();
}

}  // namespace moe
