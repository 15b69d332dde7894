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

MOE_DEV void unpack8(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[2 * i] = bf16_lo(w[i]); v[2 * i + 1] = bf16_hi(w[i]); }
}
MOE_DEV uint4 pack8(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
MOE_DEV float gate_of(float g, bool sigmoid) { return sigmoid ? __fdiv_rn(1.0f, 1.0f + expf(-g)) : g; }

// sum over the CTA; buf: one float per warp
MOE_DEV float cta_sum(float v, float* buf) {
    v = warp_sum(v);
    const int nw = blockDim.x >> 5;
    __syncthreads();                     // buf is free again
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int w = 0; w < nw; ++w) s += buf[w];
    return s;
}

// One row per CTA, V vectors of 8 columns per thread.
template <int V>
__global__ void __launch_bounds__(256) k_block_norm(NormArgs a) {
    __shared__ float buf[8];
    const size_t t = blockIdx.x;
    const int nv = a.H / 8;
    const float inv_h = 1.0f / (float)a.H;
    float u[V][8], r[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        const bool in = c < nv;
#pragma unroll
        for (int q = 0; q < 8; ++q) { u[i][q] = 0.0f; r[i][q] = 0.0f; }
        if (!in) continue;
        if (a.r_fp32) {
            const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.r) + t * a.ld_r + (size_t)c * 8);
            const float4 p0 = p[0], p1 = p[1];
            r[i][0] = p0.x; r[i][1] = p0.y; r[i][2] = p0.z; r[i][3] = p0.w;
            r[i][4] = p1.x; r[i][5] = p1.y; r[i][6] = p1.z; r[i][7] = p1.w;
        } else {
            unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.r) + t * a.ld_r + (size_t)c * 8), r[i]);
        }
        if (a.y) unpack8(*reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.y) + t * a.ld_y + (size_t)c * 8), u[i]);
#pragma unroll
        for (int q = 0; q < 8; ++q) ss = fmaf(u[i][q], u[i][q], ss);
    }
    float post = 1.0f;
    if (a.y && a.w_post) post = rsqrtf(cta_sum(ss, buf) * inv_h + a.eps);
    const float tok = a.y && a.gate_kind == kGateToken ? gate_of(__ldg(reinterpret_cast<const float*>(a.gate) + t), a.gate_sigmoid) : 1.0f;
    float rr = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nv) continue;
        float w[8], g[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) { w[q] = 1.0f; g[q] = tok; }
        if (a.y && a.w_post) {
            unpack8(reinterpret_cast<const uint4*>(a.w_post)[c], w);
#pragma unroll
            for (int q = 0; q < 8; ++q) w[q] = (w[q] + a.offset) * post;
        }
        if (a.y && (a.gate_kind == kGateChannel || a.gate_kind == kGateElement)) {
            const __nv_bfloat16* gp = reinterpret_cast<const __nv_bfloat16*>(a.gate) + (a.gate_kind == kGateElement ? t * a.ld_gate : 0);
            unpack8(*reinterpret_cast<const uint4*>(gp + (size_t)c * 8), g);
#pragma unroll
            for (int q = 0; q < 8; ++q) g[q] = gate_of(g[q], a.gate_sigmoid);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            r[i][q] = a.residual_scale * r[i][q];
            if (a.y) r[i][q] += a.branch_scale * (g[q] * (u[i][q] * w[q]));
            rr = fmaf(r[i][q], r[i][q], rr);
        }
        if (a.r_out) {
            if (a.r_fp32) {
                float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.r_out) + t * a.ld_r_out + (size_t)c * 8);
                p[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
                p[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
            } else {
                *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.r_out) + t * a.ld_r_out + (size_t)c * 8) = pack8(r[i]);
            }
        }
    }
    if (!a.x_out) return;
    const float pre = rsqrtf(cta_sum(rr, buf) * inv_h + a.eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= nv) continue;
        float w[8];
        unpack8(reinterpret_cast<const uint4*>(a.w_pre)[c], w);
#pragma unroll
        for (int q = 0; q < 8; ++q) w[q] = r[i][q] * pre * (w[q] + a.offset);
        *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.x_out) + t * a.ld_x + (size_t)c * 8) = pack8(w);
    }
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, cudaStream_t st) {
    const int nv = a.H / 8;
    if (nv <= 256) k_block_norm<1><<<a.T, 256, 0, st>>>(a);
    else if (nv <= 512) k_block_norm<2><<<a.T, 256, 0, st>>>(a);
    else if (nv <= 1024) k_block_norm<4><<<a.T, 256, 0, st>>>(a);
    else k_block_norm<8><<<a.T, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace moe
