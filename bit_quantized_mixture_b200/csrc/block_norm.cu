// What lies between two blocks, in one pass over the rows: the norm on a
// block's output, its gate, the scaled residual add and the next block's norm.
//
//   u  = y * rsqrt(mean(y^2) + eps) * (w_post + o)      (u = y without w_post)
//   g  = 1 | gate | sigmoid(gate), per channel, token or element
//   r' = residual_scale * r + branch_scale * g * u
//   x  = r' * rsqrt(mean(r'^2) + eps) * (w_pre + o)     o = 0 or 1
//
// Sums and products are fp32; r' is rounded once to the residual's type, and
// the second norm reads r' before that rounding.
//
// Bound by memory: r, y (and an element gate) in, r' and x out, once each.  The
// row stays in registers between its two sums.  Walking over the rows with the
// next ones on their way into shared memory was slower (8192 x 2048: 41 us
// against 31 of the same arithmetic): its ring leaves room for 16 warps per SM,
// and each row's weights then come from L2.
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 512;    // most threads of a CTA

// Two fp32 values in a 64-bit register: the paired multiply and fused
// multiply-add take one issue slot for both.
typedef unsigned long long f32x2;
MOE_DEV f32x2 pair(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
MOE_DEV void split(f32x2 v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
MOE_DEV f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
MOE_DEV f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// eight bf16 values as four pairs, and back (rounded to nearest even)
MOE_DEV void unpack8(const uint4& q, f32x2 (&v)[4]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pair(bf16_lo(w[i]), bf16_hi(w[i]));
}
MOE_DEV uint4 pack8(const f32x2 (&v)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(v[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// The fast exponential and division: a gate is off by up to 2 + 1.2 |g| units of 2^-23
// of its value (3.3e-6 for |g| up to 65 against 1.9e-7 by expf and a rounded
// division, which take the row's time past the memory's: 4096 x 8192, fp32 residual,
// sigmoid of a channel gate 70 against 89 us, 8192 x 2048, of an element gate 29
// against 42).
MOE_DEV float gate_of(float g, bool sigmoid) { return sigmoid ? __fdividef(1.0f, 1.0f + __expf(-g)) : g; }

// sum over the CTA; buf: one float per warp (zeros behind them up to a multiple
// of four), not to be written again before every thread has passed another
// barrier
MOE_DEV float cta_sum(f32x2 v2, float* buf) {
    float lo, hi;
    split(v2, lo, hi);
    const float v = warp_sum(lo + hi);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; w += 4) {
        const float4 q = *reinterpret_cast<const float4*>(buf + w);
        s += (q.x + q.y) + (q.z + q.w);
    }
    return s;
}

// One row per CTA, V vectors of 8 columns per thread (thread i's are i,
// i + blockDim.x, ...), the row in registers: r, y and the gate are read once,
// and every load is out before the first sum.  WIDE: r fp32.  GATED: a channel
// or element gate.  EXACT: the threads' vectors are the row's, none is past its
// end.
template <int V, bool WIDE, bool GATED, bool EXACT>
__global__ void __launch_bounds__(kNormThreads, V == 4 ? 1 : 2) k_block_norm(const __grid_constant__ NormArgs a) {
    __shared__ __align__(16) float buf[2][kNormThreads / 32];
    const size_t t = blockIdx.x;
    const int nv = a.H / 8;
    constexpr int RV = WIDE ? 2 : 1;
    const uint4 zero = make_uint4(0, 0, 0, 0), ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
    const bool has_y = a.y != nullptr;
    const uint4* rp = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(a.r) + t * a.ld_r * (WIDE ? 4 : 2));
    const uint4* yp = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y);
    const uint4* gp = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.gate) +
                                                     (a.gate_kind == kGateElement ? t * a.ld_gate : 0));
    auto inside = [&](int c) { return EXACT || c < nv; };
    uint4 rq[V][RV], yq[V], gq[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        yq[i] = has_y && inside(c) ? yp[c] : zero;
#pragma unroll
        for (int q = 0; q < RV; ++q) rq[i][q] = inside(c) ? rp[RV * c + q] : zero;
    }
    if (GATED) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            gq[i] = inside(c) ? gp[c] : zero;
        }
    }
    if (threadIdx.x < kNormThreads / 32) buf[0][threadIdx.x] = buf[1][threadIdx.x] = 0.0f;
    __syncthreads();
    auto weight = [&](const void* w, int i) {
        const int c = threadIdx.x + i * blockDim.x;
        return w && inside(c) ? __ldg(reinterpret_cast<const uint4*>(w) + c) : ones;
    };
    const float inv_h = __fdividef(1.0f, (float)a.H);
    float k = a.branch_scale;            // the branch's factors that the row shares
    if (a.gate_kind == kGateToken) k *= gate_of(__ldg(reinterpret_cast<const float*>(a.gate) + t), a.gate_sigmoid);
    float ko = 0.0f;
    if (a.w_post) {
        f32x2 ss = 0ull;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            f32x2 u[4];
            unpack8(yq[i], u);
#pragma unroll
            for (int q = 0; q < 4; ++q) ss = fma2(u[q], u[q], ss);
        }
        k *= rsqrtf(cta_sum(ss, buf[0]) * inv_h + a.eps);
        ko = k * a.offset;
    }
    const f32x2 k2 = pair(k, k), ko2 = pair(ko, ko), rs2 = pair(a.residual_scale, a.residual_scale);
    f32x2 r[V][4];
    f32x2 rr = 0ull;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (WIDE) {
            const uint4 q0 = rq[i][0], q1 = rq[i][RV - 1];
            r[i][0] = pair(__uint_as_float(q0.x), __uint_as_float(q0.y));
            r[i][1] = pair(__uint_as_float(q0.z), __uint_as_float(q0.w));
            r[i][2] = pair(__uint_as_float(q1.x), __uint_as_float(q1.y));
            r[i][3] = pair(__uint_as_float(q1.z), __uint_as_float(q1.w));
        } else {
            unpack8(rq[i][0], r[i]);
        }
        f32x2 u[4], w[4];
        unpack8(yq[i], u);
        unpack8(weight(a.w_post, i), w);
        if (GATED) {
            f32x2 g[4];
            unpack8(gq[i], g);
            if (a.gate_sigmoid) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float lo, hi;
                    split(g[q], lo, hi);
                    g[q] = pair(gate_of(lo, true), gate_of(hi, true));
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) u[q] = mul2(u[q], g[q]);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            r[i][q] = fma2(u[q], fma2(w[q], k2, ko2), mul2(r[i][q], rs2));
            rr = fma2(r[i][q], r[i][q], rr);
        }
        if (a.r_out && inside(c)) {
            if (WIDE) {
                ulonglong2* p = reinterpret_cast<ulonglong2*>(reinterpret_cast<float*>(a.r_out) + t * a.ld_r_out) + 2 * c;
                p[0] = make_ulonglong2(r[i][0], r[i][1]);
                p[1] = make_ulonglong2(r[i][2], r[i][3]);
            } else {
                reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.r_out) + t * a.ld_r_out)[c] = pack8(r[i]);
            }
        }
    }
    if (!a.x_out) return;
    const float pre = rsqrtf(cta_sum(rr, buf[1]) * inv_h + a.eps), po = pre * a.offset;
    const f32x2 pre2 = pair(pre, pre), po2 = pair(po, po);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        f32x2 w[4];
        unpack8(weight(a.w_pre, i), w);
#pragma unroll
        for (int q = 0; q < 4; ++q) w[q] = mul2(r[i][q], fma2(w[q], pre2, po2));
        if (inside(c)) reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.x_out) + t * a.ld_x)[c] = pack8(w);
    }
}

template <int V, bool WIDE, bool GATED>
void launch_vg(const NormArgs& a, int threads, cudaStream_t st) {
    if (V * threads == a.H / 8) k_block_norm<V, WIDE, GATED, true><<<a.T, threads, 0, st>>>(a);
    else k_block_norm<V, WIDE, GATED, false><<<a.T, threads, 0, st>>>(a);
}

template <int V>
void launch_v(const NormArgs& a, cudaStream_t st) {
    const int threads = ((a.H / 8 + V - 1) / V + 31) / 32 * 32;
    const bool gated = a.gate_kind == kGateElement || a.gate_kind == kGateChannel;
    if (a.r_fp32 && gated) launch_vg<V, true, true>(a, threads, st);
    else if (a.r_fp32) launch_vg<V, true, false>(a, threads, st);
    else if (gated) launch_vg<V, false, true>(a, threads, st);
    else launch_vg<V, false, false>(a, threads, st);
}

}  // namespace

// Vectors per thread: threads that wait less for one another against more rows
// on their way per SM.  2048 columns, bf16, 1 / 2 / 4 vectors: 600 rows 3.3 /
// 3.1 / 3.3 us, 2400 rows 9.8 / 9.4 / 9.8, 8192 rows 28.9 / 25.6 / 24.0 (134 MB:
// 5.6 TB/s); one row 2.2 / 2.3 / 2.4.  4096 x 8192 with an fp32 residual: 73 us
// with two, 70 with four (403 MB: 5.8 TB/s).
cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
    const int nv = a.H / 8;
    if (a.T >= 4096 || nv > 2 * kNormThreads) launch_v<4>(a, st);
    else if (a.T >= 592 || nv > kNormThreads) launch_v<2>(a, st);
    else launch_v<1>(a, st);
    return cudaGetLastError();
}

}  // namespace moe
