// Low-rank adapters of many requests beside a shared projection:
//   out_t = y_t + scale_i * B_i (A_i x_t),   i = adapter of token t,
// A_i [R, K], B_i [N, R] (bf16, the first rank_i rows / columns in use), x
// bf16, y and out bf16 or fp32.  Tokens without an adapter keep y_t.
//
// Few tokens: a cluster of CTAs per token.  CTA c sums A_i x_t over its share of
// the K columns (a warp per four rows of A, lanes along K), writes the sums into
// every CTA's shared memory, and then has its share of the N outputs, R / 8 lanes
// per output; the rows of B are on their way meanwhile.
#include <cooperative_groups.h>

#include "adapters.cuh"
#include "kernels.h"

namespace moe {

namespace {

namespace cg = cooperative_groups;

// Which kernel takes a call is a matter of its tokens: whose they are is known on
// the device alone.  A cluster per token reads each token's whole adapter; tiles
// share it among the tokens of one request, but go through a tile's adapters one
// after another.  2048 -> 2048, us, tokens of 64 requests mixed / of 12 requests in
// order: 128 tokens rank 16, by token 6.4 / 6.4, in tiles of 16 33 / 12; 256 tokens
// 9.4 / 9.8 and 34 / 11; 512 tokens 17 / 17 and 35 / 11; rank 64, 128 tokens 22 / 15
// and 58 / 16; 256 tokens 40 / 25 and 57 / 16: there tokens of many requests lose 17 us
// by the rule, tokens in order would lose 9 by the other.
constexpr int kAdTokenMax = 256, kAdTokenWork = 8192;        // most tokens, most tokens x R, of a cluster per token
// CTAs per token: rank 16, 1 token 3.8 us with 8, 4.6 with 4, 6.9 with 2; 64 tokens
// 5.6 / 5.4 / 7.1; 128 tokens 9.8 / 6.4 / 7.6; 256 tokens 18 / 11.4 / 9.4.
constexpr int kAdCluster8 = 32, kAdCluster4 = 192;           // up to so many tokens 8, 4 CTAs
// 2048 -> 2048, 12 requests in order, us, tiles of 16 tokens / of 128 on tcgen05
// (adapters_tc.cu), bf16: rank 16, 2500 tokens 20.4 / 23.2, 2800 tokens 22.3 / 21.9, 8192
// tokens 58 / 34; rank 32, 3200 tokens 25.6 / 26.7, 3700 tokens 30.8 / 30.3, 8192 tokens
// 60 / 36; rank 64, 2500 tokens 31.2 / 33.5, 2800 tokens 34 / 31.7, 8192 tokens 82 / 45;
// rank 128, 1300 tokens 42 / 44, 1600 tokens 53 / 41, 8192 tokens 200 / 78.  fp32
// outputs, tiles of 16 / of 64 / tcgen05: rank 16, 3700 tokens 33 / 36 / 31, 4500
// tokens 37 / 32 / 39, 6000 tokens 49 / 49 / 41, 8192 tokens 65 / 55 / 42; rank 32, 3700
// tokens 35 / 37 / 41, 6000 tokens 50 / 50 / 54, 8192 tokens 66 / 56 / 51; rank 64, 4500
// tokens 51 / 52 / 63, 6000 tokens 67 / 77 / 59, 8192 tokens 88 / 83 / 61; rank 128
// (no tcgen05), 3200 tokens 90 / 94, 3700 tokens 102 / 87, 8192 tokens 202 / 152.
constexpr int kAdTc16 = 2800, kAdTc32 = 3500, kAdTc64 = 2700, kAdTc128 = 1400;   // from so many tokens on tcgen05: ranks to 16, 32, 64, 128
constexpr int kAdTcWide16 = 5000, kAdTcWide32 = 7000, kAdTcWide64 = 5000;        // fp32, likewise
constexpr int kAdTile64Wide32 = 4000, kAdTile64Wide128 = 3600;   // fp32: from so many on tiles of 64 (ranks 33 to 64: never)
constexpr int kAdThreads = 256;

MOE_DEV float dot8(const uint4& p, const uint4& q, float s) {
    const uint32_t a[4] = {p.x, p.y, p.z, p.w}, b[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = fmaf(bf16_lo(a[i]), bf16_lo(b[i]), s);
        s = fmaf(bf16_hi(a[i]), bf16_hi(b[i]), s);
    }
    return s;
}

MOE_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
MOE_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// LL: log2 of the lanes that share an output (8 of B's columns each).
template <int CL, int LL>
__global__ void __launch_bounds__(kAdThreads) k_adapter_token(const __grid_constant__ AdapterArgs a) {
    constexpr int WARPS = kAdThreads / 32, L = 1 << LL, PER = 32 / L, BATCH = 4;
    __shared__ float part[CL][kAdapterMaxRank];  // every CTA's share of z, written by them
    __shared__ __align__(16) float z[kAdapterMaxRank];
    cg::cluster_group cl = cg::this_cluster();
    const int c = (int)cl.block_rank();
    const size_t t = blockIdx.x / CL;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & (L - 1);
    const int id = __ldg(a.ids + t);
    const bool has = id >= 0 && id < a.n;
    const int rank = has ? min(max(a.ranks ? __ldg(a.ranks + id) : a.R, 0), a.R) : 0;
    const float scale = rank ? __ldg(a.scales + id) : 0.0f;
    // this CTA's outputs, and the first batch of their rows of B: they need no z
    const int n0 = (int)((long long)a.N * c / CL), n1 = (int)((long long)a.N * (c + 1) / CL);
    const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(a.b) + (size_t)(has ? id : 0) * a.N * a.R + 8 * sub;
    const bool cols = 8 * sub < rank;
    auto output = [&](int i) { return n0 + (i * WARPS + warp) * PER + lane / L; };
    uint4 q[BATCH];
    auto fetch = [&](int i0) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int j = output(i0 + u);
            q[u] = cols && j < n1 ? ldg_nc_v4(b + (size_t)j * a.R) : make_uint4(0, 0, 0, 0);
        }
    };
    fetch(0);
    // K in vectors of 8 columns, shares of whole vectors
    const int kv = a.K / 8;
    const int k0 = (int)((long long)kv * c / CL), k1 = (int)((long long)kv * (c + 1) / CL);
    const uint4* x = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.x) + t * a.ld_x);
    cluster_arrive();                            // everyone is here: its shared memory may be written
    bool here = false;
    for (int r0 = warp; r0 < rank; r0 += 4 * WARPS) {
        const uint4* row = reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.a) + ((size_t)id * a.R + r0) * a.K);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int v = k0 + lane; v < k1; v += 32) {
            uint4 p[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) p[u] = r0 + u * WARPS < rank ? ldg_nc_v4(row + (size_t)u * WARPS * kv + v) : make_uint4(0, 0, 0, 0);
            const uint4 xv = __ldg(x + v);
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] = dot8(p[u], xv, s[u]);
        }
        if (!here) cluster_wait();
        here = true;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            s[u] = warp_sum(s[u]);
            if (lane < CL && r0 + u * WARPS < rank) *cl.map_shared_rank(&part[c][r0 + u * WARPS], lane) = s[u];
        }
    }
    if (!here) cluster_wait();
    cluster_arrive();
    cluster_wait();
    for (int r = threadIdx.x; r < kAdapterMaxRank; r += kAdThreads) {
        float s = 0.0f;
        if (r < rank) {
#pragma unroll
            for (int u = 0; u < CL; ++u) s += part[u][r];
        }
        z[r] = r < rank ? s * scale : 0.0f;
    }
    __syncthreads();
    float zv[8];
    uint32_t keep[4];                            // columns behind the rank may hold anything
#pragma unroll
    for (int i = 0; i < 8; ++i) zv[i] = z[8 * sub + i];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        keep[i] = (8 * sub + 2 * i < rank ? 0xffffu : 0u) | (8 * sub + 2 * i + 1 < rank ? 0xffff0000u : 0u);
    for (int i0 = 0; output(i0) - lane / L < n1; i0 += BATCH) {
        if (i0) fetch(i0);
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const uint32_t w[4] = {q[u].x & keep[0], q[u].y & keep[1], q[u].z & keep[2], q[u].w & keep[3]};
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s = fmaf(bf16_lo(w[i]), zv[2 * i], s);
                s = fmaf(bf16_hi(w[i]), zv[2 * i + 1], s);
            }
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            const int j = output(i0 + u);
            if (sub != 0 || j >= n1) continue;
            if (a.wide) {
                const float y = reinterpret_cast<const float*>(a.y)[t * a.ld_y + j];
                reinterpret_cast<float*>(a.out)[t * a.ld_out + j] = rank ? y + s : y;
            } else {
                const __nv_bfloat16 y = reinterpret_cast<const __nv_bfloat16*>(a.y)[t * a.ld_y + j];
                reinterpret_cast<__nv_bfloat16*>(a.out)[t * a.ld_out + j] = rank ? __float2bfloat16_rn(bf16_to_f(y) + s) : y;
            }
        }
    }
}

template <int CL, int LL>
cudaError_t launch_token(const AdapterArgs& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.T * CL);
    cfg.blockDim = dim3(kAdThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = CL;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_token<CL, LL>, a);
}

template <int CL>
cudaError_t launch_tokens(const AdapterArgs& a, cudaStream_t st) {
    if (a.R <= 8) return launch_token<CL, 0>(a, st);
    if (a.R <= 16) return launch_token<CL, 1>(a, st);
    if (a.R <= 32) return launch_token<CL, 2>(a, st);
    if (a.R <= 64) return launch_token<CL, 3>(a, st);
    return launch_token<CL, 4>(a, st);
}

// D (16 x 8, fp32) += A (16 x 16, bf16) B (16 x 8, bf16)
MOE_DEV void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Many tokens: a cluster of kTileCluster CTAs takes BT = 16 MT MG consecutive
// tokens.  Both products run on mma.sync m16n8k16 straight from global memory.
//
//   1. z = A_i x: the cluster's 8 / MG x kTileCluster column shares of x, a warp
//      per share and 16 MT rows; the shares meet in shared memory, then across
//      the cluster.  A warp repeats this for each adapter among its rows and
//      keeps each row's own.
//   2. out = y + B_i (scale z): the same split over the N outputs.
//
// Fragments.  A sum over k may take k in any order, so lane (g, c) (g = lane / 4,
// c = lane % 4) loads 16 bytes, columns 8c .. 8c+7 of a 32-column chunk, from
// row g of either operand: words 0, 1 are its k pairs of the chunk's first
// mma, words 2, 3 of the second.  Likewise column 2c + i of the n-tile j of a
// group of four stands for 8c + 2j + i, so that a lane's results of the four
// tiles are eight neighbours (16-byte loads of y and stores of out), and z's
// results are, without any exchange, the first operand of step 2 with B's
// 16-byte loads.
//
// RG: groups of 32 rank rows.  WIDE: y and out fp32.  z is held in three bf16
// parts (adapters.cuh), one product each.  Ranks that are not in use have z = 0,
// whatever x holds.
constexpr int kTileCluster = 4;
constexpr int kTileWarps = 8;

template <int RG, int MT, int MG>
constexpr size_t tile_smem_bytes() {
    // [parts][MG][MT][4 RG tiles][2 row halves][32 lanes] float2
    return (size_t)(kTileWarps / MG) * MG * MT * 4 * RG * 2 * 32 * sizeof(float2);
}

// Eight outputs of a row, taken again in fp32 (a NaN among them whose z parts cannot
// tell, see adapters.cuh; rare, so not inlined).  zrow: the row's words of z, part q
// at q * stride (see zf below).
template <int RG, bool WIDE>
__device__ __noinline__ void tile_repair(const AdapterArgs& a, int t, int col, int id, int rank, const uint32_t* zrow, int stride) {
    auto z_of = [&](int r) {
        const int j = 4 * (r >> 5) + ((r >> 1) & 3);
        const uint32_t* w = zrow + (j >> 1) * 128 + ((r >> 3) & 3) * 4 + (j & 1) * 2;
        float v = 0.0f;
        for (int q = kZParts - 1; q >= 0; --q) v += r & 1 ? bf16_hi(w[q * stride]) : bf16_lo(w[q * stride]);
        return v;
    };
    const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(a.b) + ((size_t)id * a.N + col) * a.R;
    for (int u = 0; u < 8; ++u, b += a.R) {
        const float s = whole_product(z_of, b, rank);
        const size_t yo = (size_t)t * a.ld_y + col + u, oo = (size_t)t * a.ld_out + col + u;
        if (WIDE) reinterpret_cast<float*>(a.out)[oo] = reinterpret_cast<const float*>(a.y)[yo] + s;
        else reinterpret_cast<__nv_bfloat16*>(a.out)[oo] = __float2bfloat16_rn(bf16_to_f(reinterpret_cast<const __nv_bfloat16*>(a.y)[yo]) + s);
    }
}

template <int RG, int MT, int MG, bool WIDE>
__global__ void __launch_bounds__(kTileWarps * 32, RG == 4 ? 1 : 2) k_adapter_tile(const __grid_constant__ AdapterArgs a) {
    constexpr int BT = 16 * MT * MG, PARTS = kTileWarps / MG, TJ = 4 * RG, NPASS = RG == 4 ? 2 : 1, PJ = TJ / NPASS;
    constexpr int ZN = MG * MT * TJ * 2 * 32;             // float2 values of z
    extern __shared__ __align__(16) float2 part_s[];      // [PARTS][ZN]; later zf in place of part 1 on
    __shared__ float s_scale[BT];
    __shared__ int s_rank[BT];                            // 0: no adapter
    __shared__ int s_unsure[BT];                          // the row has a z that its parts may not stand for
    cg::cluster_group cl = cg::this_cluster();
    const int crank = (int)cl.block_rank();
    const int t0 = (int)(blockIdx.x / kTileCluster) * BT;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int mg = warp % MG, part = warp / MG;
    const int r0 = t0 + 16 * MT * mg;                     // the warp's first row
    auto rank_of = [&](int id) { return min(a.ranks ? __ldg(a.ranks + id) : a.R, a.R); };
    // the adapters of the warp's rows (lane: row), -1 for none
    int myid = -1;
    if (lane < 16 * MT && r0 + lane < a.T) {
        const int id = __ldg(a.ids + r0 + lane);
        if (id >= 0 && id < a.n && rank_of(id) > 0) myid = id;
    }
    const int myrank = myid >= 0 ? rank_of(myid) : 0;
    if (part == 0 && lane < 16 * MT) {
        s_scale[16 * MT * mg + lane] = myid >= 0 ? __ldg(a.scales + myid) : 0.0f;
        s_rank[16 * MT * mg + lane] = myrank;
        s_unsure[16 * MT * mg + lane] = 0;
    }
    const unsigned with = __ballot_sync(0xffffffffu, myid >= 0);
    const int share = crank * PARTS + part;
    constexpr int SHARES = kTileCluster * PARTS;
    {
        // ------------------------------------------------ z, this warp's columns
        const int nch = (a.K + 31) / 32;
        const int lo = (int)((long long)nch * share / SHARES), hi = (int)((long long)nch * (share + 1) / SHARES);
        float2* mine = part_s + (size_t)part * ZN + mg * (MT * TJ * 2 * 32) + lane;
        const __nv_bfloat16* xr[2 * MT];
#pragma unroll
        for (int u = 0; u < 2 * MT; ++u)
            xr[u] = reinterpret_cast<const __nv_bfloat16*>(a.x) + (size_t)min(r0 + g + 8 * u, a.T - 1) * a.ld_x + 8 * c;
        if (with == 0) {
#pragma unroll
            for (int i = 0; i < MT * TJ * 2; ++i) mine[i * 32] = make_float2(0.0f, 0.0f);
        }
        for (unsigned todo = with; todo;) {
            const int id = __shfl_sync(0xffffffffu, myid, __ffs(todo) - 1);
            const unsigned mem = __ballot_sync(0xffffffffu, myid == id);
            const bool first = todo == with;
            todo &= ~mem;
            const int rk = rank_of(id);
            const __nv_bfloat16* arow = reinterpret_cast<const __nv_bfloat16*>(a.a) + ((size_t)id * a.R + 8 * (g >> 1) + (g & 1)) * a.K + 8 * c;
#pragma unroll 1
            for (int p = 0; p < NPASS; ++p) {
                float acc[MT][PJ][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < PJ; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[m][j][q] = 0.0f;
#pragma unroll 2
                for (int ch = lo; ch < hi; ++ch) {
                    const bool in = 32 * ch + 8 * c < a.K;
                    uint4 xv[2 * MT], av[PJ];
#pragma unroll
                    for (int u = 0; u < 2 * MT; ++u) xv[u] = in ? ldg_stream_v4(xr[u] + 32 * ch) : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int j = 0; j < PJ; ++j) {
                        const int ro = 32 * (j / 4) + 2 * (j & 3) + 32 * (PJ / 4) * p;    // row: ro + 8 (g / 2) + g % 2
                        av[j] = in && ro + 8 * (g >> 1) + (g & 1) < rk ? ldg_nc_v4(arow + (size_t)ro * a.K + 32 * ch) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int j = 0; j < PJ; ++j)
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            mma_16816(acc[m][j], xv[2 * m].x, xv[2 * m + 1].x, xv[2 * m].y, xv[2 * m + 1].y, av[j].x, av[j].y);
                            mma_16816(acc[m][j], xv[2 * m].z, xv[2 * m + 1].z, xv[2 * m].w, xv[2 * m + 1].w, av[j].z, av[j].w);
                        }
                }
                // each row's own adapter; rows without one get zeros
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool own = (mem >> (16 * m + 8 * h + g)) & 1u;
                        const bool none = !((with >> (16 * m + 8 * h + g)) & 1u);
                        if (own || (first && none)) {
#pragma unroll
                            for (int j = 0; j < PJ; ++j)
                                mine[((m * TJ + PJ * p + j) * 2 + h) * 32] = own ? make_float2(acc[m][j][2 * h], acc[m][j][2 * h + 1])
                                                                                 : make_float2(0.0f, 0.0f);
                        }
                    }
            }
        }
    }
    __syncthreads();
    // ------------------------------------- the CTA's shares, then the cluster's
    for (int i = threadIdx.x; i < ZN; i += kTileWarps * 32) {
        float2 v = part_s[i];
#pragma unroll
        for (int q = 1; q < PARTS; ++q) {
            const float2 o = part_s[(size_t)q * ZN + i];
            v.x += o.x;
            v.y += o.y;
        }
        part_s[i] = v;
    }
    cl.sync();
    // z * scale as the second product's first operand: [MG][MT][2 RG steps][32
    // lanes][4 words] for each of its parts
    uint32_t* zf = reinterpret_cast<uint32_t*>(part_s + ZN);
    for (int i = threadIdx.x; i < ZN; i += kTileWarps * 32) {
        float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int q = 0; q < kTileCluster; ++q) {
            const float2 o = cl.map_shared_rank(part_s, q)[i];
            v.x += o.x;
            v.y += o.y;
        }
        const int l = i & 31, h = (i >> 5) & 1, j = (i >> 6) % TJ, mm = (i >> 6) / TJ;     // mm: 16-row tile of the block
        const float sc = s_scale[16 * mm + 8 * h + (l >> 2)];
        const int left = s_rank[16 * mm + 8 * h + (l >> 2)] - (32 * (j >> 2) + 8 * (l & 3) + 2 * (j & 3));     // ranks in use from this pair on
        v.x = left > 0 ? v.x * sc : 0.0f;
        v.y = left > 1 ? v.y * sc : 0.0f;
        const int w = ((mm * 2 * RG + (j >> 1)) * 32 + l) * 4 + (j & 1) * 2 + h;
        uint32_t p[kZParts];
        split_z2(v.x, v.y, p);
#pragma unroll
        for (int q = 0; q < kZParts; ++q) zf[q * ZN + w] = p[q];
        if (z_unsure(v.x) || z_unsure(v.y)) s_unsure[16 * mm + 8 * h + (l >> 2)] = 1;
    }
    // the others may still read this CTA's sums: waited for at the end
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();
    {
        // ------------------------------------------- out, this warp's columns
        const int ng = (a.N + 31) / 32;
        const int lo = (int)((long long)ng * share / SHARES), hi = (int)((long long)ng * (share + 1) / SHARES);
        const uint4* zq = reinterpret_cast<const uint4*>(zf) + (size_t)(mg * MT) * 2 * RG * 32 + lane;
        for (int cgp = lo; cgp < hi; ++cgp) {
            const int col = 32 * cgp + 8 * c;                         // this lane's eight outputs
            float delta[MT][4][4];
            uint4 yv[2 * MT][WIDE ? 2 : 1];
#pragma unroll
            for (int u = 0; u < 2 * MT; ++u) {
                const bool in = r0 + g + 8 * u < a.T && col < a.N;
                const size_t off = (size_t)(r0 + g + 8 * u) * a.ld_y + col;
                if (WIDE) {
                    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(a.y) + off);
                    yv[u][0] = in ? p[0] : make_uint4(0, 0, 0, 0);
                    yv[u][WIDE ? 1 : 0] = in ? p[1] : make_uint4(0, 0, 0, 0);
                } else {
                    yv[u][0] = in ? *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(a.y) + off) : make_uint4(0, 0, 0, 0);
                }
            }
            for (unsigned todo = with; todo;) {
                const int id = __shfl_sync(0xffffffffu, myid, __ffs(todo) - 1);
                const unsigned mem = __ballot_sync(0xffffffffu, myid == id);
                todo &= ~mem;
                const int rk = rank_of(id);
                float acc[MT][4][4];
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[m][j][q] = 0.0f;
#pragma unroll
                for (int G = 0; G < RG; ++G) {
                    const int left = rk - (32 * G + 8 * c);           // columns of this lane's eight in use
                    uint4 bv[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int n = 32 * cgp + 8 * (g >> 1) + 2 * j + (g & 1);
                        bv[j] = left > 0 && n < a.N ? ldg_nc_v4(reinterpret_cast<const __nv_bfloat16*>(a.b) + ((size_t)id * a.N + n) * a.R + 32 * G + 8 * c)
                                                    : make_uint4(0, 0, 0, 0);
                        if (left > 0 && left < 8) {
                            uint32_t* wd = &bv[j].x;
#pragma unroll
                            for (int q = 0; q < 4; ++q) wd[q] &= left >= 2 * q + 2 ? 0xffffffffu : (left == 2 * q + 1 ? 0xffffu : 0u);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int q = kZParts - 1; q >= 0; --q) {
                            const uint4* zp = zq + (size_t)(m * 2 * RG + 2 * G) * 32 + q * (ZN / 4);
                            const uint4 z0 = zp[0], z1 = zp[32];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                mma_16816(acc[m][j], z0.x, z0.y, z0.z, z0.w, bv[j].x, bv[j].y);
                                mma_16816(acc[m][j], z1.x, z1.y, z1.z, z1.w, bv[j].z, bv[j].w);
                            }
                        }
                }
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if ((mem >> (16 * m + 8 * h + g)) & 1u) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                delta[m][j][2 * h] = acc[m][j][2 * h];
                                delta[m][j][2 * h + 1] = acc[m][j][2 * h + 1];
                            }
                        }
            }
#pragma unroll
            for (int u = 0; u < 2 * MT; ++u) {
                if (r0 + g + 8 * u >= a.T || col >= a.N) continue;
                const int m = u >> 1, h = u & 1;
                const bool own = (with >> (8 * u + g)) & 1u;          // rows without an adapter keep y's bits
                const int row = r0 + g + 8 * u - t0;
                if (own && s_unsure[row]) {
                    bool nan = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) nan = nan || delta[m][j][2 * h] != delta[m][j][2 * h] || delta[m][j][2 * h + 1] != delta[m][j][2 * h + 1];
                    if (nan) {
                        tile_repair<RG, WIDE>(a, t0 + row, col, __ldg(a.ids + t0 + row), s_rank[row], zf + ((row >> 4) * 2 * RG * 32 + 4 * g) * 4 + h, ZN);
                        continue;
                    }
                }
                const size_t off = (size_t)(r0 + g + 8 * u) * a.ld_out + col;
                uint32_t* y = &yv[u][0].x;
                if (WIDE) {
                    uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<float*>(a.out) + off);
                    uint32_t* y1 = &yv[u][WIDE ? 1 : 0].x;
                    if (own) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            y[q] = __float_as_uint(__uint_as_float(y[q]) + delta[m][q >> 1][2 * h + (q & 1)]);
                            y1[q] = __float_as_uint(__uint_as_float(y1[q]) + delta[m][2 + (q >> 1)][2 * h + (q & 1)]);
                        }
                    }
                    p[0] = yv[u][0];
                    p[1] = yv[u][WIDE ? 1 : 0];
                } else {
                    if (own) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) y[j] = pack_bf16x2(bf16_lo(y[j]) + delta[m][j][2 * h], bf16_hi(y[j]) + delta[m][j][2 * h + 1]);
                    }
                    *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(a.out) + off) = yv[u][0];
                }
            }
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <int RG, int MT, int MG, bool WIDE>
cudaError_t launch_tile(const AdapterArgs& a, cudaStream_t st) {
    constexpr int BT = 16 * MT * MG;
    constexpr size_t smem = tile_smem_bytes<RG, MT, MG>();
    cudaError_t e = cudaFuncSetAttribute(k_adapter_tile<RG, MT, MG, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((a.T + BT - 1) / BT) * kTileCluster);
    cfg.blockDim = dim3(kTileWarps * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kTileCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_adapter_tile<RG, MT, MG, WIDE>, a);
}

template <bool WIDE>
cudaError_t launch_tiles(const AdapterArgs& a, cudaStream_t st) {
    if (a.R <= 32) return launch_tile<1, 1, 1, WIDE>(a, st);
    if (a.R <= 64) return launch_tile<2, 1, 1, WIDE>(a, st);
    return launch_tile<4, 1, 1, WIDE>(a, st);
}

}  // namespace

cudaError_t launch_add_adapters(const AdapterArgs& a, cudaStream_t st) {
    if (a.T <= kAdTokenMax && (long long)a.T * a.R <= kAdTokenWork) {
        if (a.T <= kAdCluster8) return launch_tokens<8>(a, st);
        return a.T <= kAdCluster4 ? launch_tokens<4>(a, st) : launch_tokens<2>(a, st);
    }
    const int tc = a.R <= 16 ? (a.wide ? kAdTcWide16 : kAdTc16) : a.R <= 32 ? (a.wide ? kAdTcWide32 : kAdTc32)
                 : a.R <= 64 ? (a.wide ? kAdTcWide64 : kAdTc64) : kAdTc128;
    if (a.T >= tc) {
        const cudaError_t e = launch_add_adapters_tc(a, st);
        if (e != cudaErrorNotSupported) return e;
    }
    if (!a.wide) return launch_tiles<false>(a, st);
    if (a.R <= 32 && a.T >= kAdTile64Wide32) return launch_tile<1, 2, 2, true>(a, st);
    if (a.R > 64 && a.T >= kAdTile64Wide128) return launch_tile<4, 2, 2, true>(a, st);
    return launch_tiles<true>(a, st);
}

}  // namespace moe
