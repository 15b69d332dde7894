// Low-rank adapters of many requests beside a shared projection:
//   out_t = y_t + scale_i * B_i (A_i x_t),   i = adapter of token t,
// A_i [R, K], B_i [N, R] (bf16, the first rank_i rows / columns in use), x
// bf16, y and out bf16 or fp32.  Tokens without an adapter keep y_t.
//
// One cluster of CTAs per token: CTA c sums A_i x_t over its share of the K
// columns (a warp per row of A, lanes along K), the shares meet through
// distributed shared memory, and CTA c then writes its share of the N
// outputs, a thread per output.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

constexpr int kAdThreads = 256;
constexpr int kAdCluster = 8;

MOE_DEV float dot8(const uint4& p, const uint4& q, float s) {
    const uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(bf16_lo(a[i]), bf16_lo(b[i]), s);
        s = fmaf(bf16_hi(a[i]), bf16_hi(b[i]), s);
    }
    return s;
}

__global__ void __launch_bounds__(kAdThreads) k_adapter_token(AdapterArgs a) {
    __shared__ float part[kAdapterMaxRank];      // this CTA's share of z
    __shared__ float z[kAdapterMaxRank];
    cg::cluster_group cl = cg::this_cluster();
    const int c = (int)cl.block_rank();
    const size_t t = blockIdx.x / kAdCluster;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int id = __ldg(a.ids + t);
    const bool has = id >= 0 && id < a.n;
    int rank = has ? (a.ranks ? __ldg(a.ranks + id) : a.R) : 0;
    rank = min(max(rank, 0), a.R);
    // K in vectors of 8 columns, shares of whole vectors
    const int kv = a.K / 8;
    const int k0 = (int)((long long)kv * c / kAdCluster), k1 = (int)((long long)kv * (c + 1) / kAdCluster);
    const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.x) + t * a.ld_x);
    for (int r = warp; r < rank; r += kAdThreads / 32) {
        const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.a) + ((size_t)id * a.R + r) * a.K);
        float s = 0.0f;
        for (int v = k0 + lane; v < k1; v += 32) s = dot8(__ldg(row + v), __ldg(x + v), s);
        s = warp_sum(s);
        if (lane == 0) part[r] = s;
    }
    cl.sync();
    const float scale = rank ? __ldg(a.scales + id) : 0.0f;
    for (int r = threadIdx.x; r < rank; r += kAdThreads) {
        float s = 0.0f;
#pragma unroll
        for (int q = 0; q < kAdCluster; ++q) s += cl.map_shared_rank(part, q)[r];
        z[r] = s * scale;
    }
    cl.sync();                                   // z is written; nobody reads part any more
    const int n0 = (int)((long long)a.N * c / kAdCluster), n1 = (int)((long long)a.N * (c + 1) / kAdCluster);
    for (int j = n0 + (int)threadIdx.x; j < n1; j += kAdThreads) {
        const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(a.b) + ((size_t)(has ? id : 0) * a.N + j) * a.R;
        float s = 0.0f;
        for (int r0 = 0; r0 < rank; r0 += 8) {
            const uint4 q = __ldg(reinterpret_cast<const uint4*>(b + r0));
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (r0 + i < rank) s = fmaf((i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]), z[r0 + i], s);
        }
        if (a.wide) {
            const float y = reinterpret_cast<const float*>(a.y)[t * a.ld_y + j];
            reinterpret_cast<float*>(a.out)[t * a.ld_out + j] = rank ? y + s : y;
        } else {
            const __nv_bfloat16 y = reinterpret_cast<const __nv_bfloat16*>(a.y)[t * a.ld_y + j];
            reinterpret_cast<__nv_bfloat16*>(a.out)[t * a.ld_out + j] = rank ? __float2bfloat16_rn(bf16_to_f(y) + s) : y;
        }
    }
}

}  // namespace

cudaError_t launch_add_adapters(const AdapterArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.T * kAdCluster);
    cfg.blockDim = dim3(kAdThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kAdCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_token, a);
}

}  // namespace moe
