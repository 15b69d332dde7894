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
#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 512;    // most threads of a CTA
constexpr int kNormManyRows = 592;   // from so many rows on (four per SM) four vectors per thread

MOE_DEV void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
}
MOE_DEV uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
MOE_DEV float gate_of(float g, bool sigmoid) { return sigmoid ? __fdiv_rn(1.0f, 1.0f + expf(-g)) : g; }

// sum over the CTA; buf: one float per warp, used once per launch
MOE_DEV float cta_sum(float v, float* buf) {
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    if (nw == 1) return v;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += buf[w];
    return s;
}

// One row per CTA, V vectors of 8 columns per thread, the row in registers: r
// and y are read once and every load is out before the first sum.
template <int V, bool WIDE>
__global__ void __launch_bounds__(kNormThreads, V == 4 ? 1 : 2) k_block_norm(const __grid_constant__ NormArgs a) {
    __shared__ float buf[2][kNormThreads / 32];
    const size_t t = blockIdx.x;
    const int nv = a.H / 8;
    const float inv_h = __fdividef(1.0f, (float)a.H);
    uint4 rq[V][WIDE ? 2 : 1], yq[V], gq[V];
    const bool has_y = a.y != nullptr, per_el = a.gate_kind == kGateElement;
    const char* rp = reinterpret_cast<const char*>(a.r) + t * a.ld_r * (WIDE ? 4 : 2);
    const uint4* yp = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y);
    const uint4* gp = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.gate) + (per_el ? t * a.ld_gate : 0));
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool in = c < nv;
        yq[i] = in && has_y ? yp[c] : zero;
        const uint4* p = reinterpret_cast<const uint4*>(rp) + (WIDE ? 2 * c : c);
        rq[i][0] = in ? p[0] : zero;
        if (WIDE) rq[i][WIDE ? 1 : 0] = in ? p[1] : zero;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        gq[i] = c < nv && (per_el || a.gate_kind == kGateChannel) ? gp[c] : zero;
    }
    const float tok = a.gate_kind == kGateToken ? gate_of(__ldg(reinterpret_cast<const float*>(a.gate) + t), a.gate_sigmoid) : 1.0f;
    float post = 1.0f;
    if (a.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float u[8];
            unpack8(yq[i], u);
#pragma unroll
            for (int q = 0; q < 8; ++q) ss = fmaf(u[q], u[q], ss);
        }
        post = rsqrtf(cta_sum(ss, buf[0]) * inv_h + a.eps);
    }
    float r[V][8];
    float rr = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (WIDE) {
            const uint4 q0 = rq[i][0], q1 = rq[i][WIDE ? 1 : 0];
            const uint32_t w[8] = {q0.x, q0.y, q0.z, q0.w, q1.x, q1.y, q1.z, q1.w};
#pragma unroll
            for (int q = 0; q < 8; ++q) r[i][q] = __uint_as_float(w[q]);
        } else {
            unpack8(rq[i][0], r[i]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) r[i][q] *= a.residual_scale;
        if (has_y) {
            float u[8];
            unpack8(yq[i], u);
            if (a.w_post) {
                float w[8];
                unpack8(c < nv ? __ldg(reinterpret_cast<const uint4*>(a.w_post) + c) : zero, w);
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] *= (w[q] + a.offset) * post;
            }
            if (per_el || a.gate_kind == kGateChannel) {
                float g[8];
                unpack8(gq[i], g);
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] *= gate_of(g[q], a.gate_sigmoid);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) u[q] *= tok;
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) r[i][q] += a.branch_scale * u[q];
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) rr = fmaf(r[i][q], r[i][q], rr);
        if (a.r_out && c < nv) {
            if (WIDE) {
                float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.r_out) + t * a.ld_r_out) + 2 * c;
                p[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                p[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
            } else {
                reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.r_out) + t * a.ld_r_out)[c] = pack8(r[i]);
            }
        }
    }
    if (!a.x_out) return;
    const float pre = rsqrtf(cta_sum(rr, buf[1]) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nv) continue;
        float w[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(a.w_pre) + c), w);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = r[i][q] * pre * (w[q] + a.offset);
        reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.x_out) + t * a.ld_x)[c] = pack8(w);
    }
}

template <int V>
void launch_v(const NormArgs& a, cudaStream_t st) {
    const int threads = ((a.H / 8 + V - 1) / V + 31) / 32 * 32;
    if (a.r_fp32) k_block_norm<V, true><<<a.T, threads, 0, st>>>(a);
    else k_block_norm<V, false><<<a.T, threads, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
    const int nv = a.H / 8;
    if (a.T >= kNormManyRows || nv > 2 * kNormThreads) launch_v<4>(a, st);
    else if (nv > kNormThreads) launch_v<2>(a, st);
    else launch_v<1>(a, st);
    return cudaGetLastError();
}

}  // namespace moe
