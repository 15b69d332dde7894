// Low-rank adapters of many requests for many tokens, on the tensor cores:
//   out_t = y_t + B_i (scale_i A_i x_t),   i = adapter of token t.
//
// A cluster of CTAs takes 128 consecutive tokens; CTA c has its share of the K
// columns of x for the first product and of the N columns of y for the second.
//
//   1. z: tcgen05.mma, M = the 128 tokens, N = the rank, over 64-column chunks of
//      x and of the tile's adapters' A (TMA, 128-byte swizzle).  As many adapters
//      as 256 accumulator columns hold share one pass over x; each row keeps its
//      own adapter's columns (a tile of one adapter, or of two neighbours, needs
//      one pass).
//   2. The cluster's partial sums: each CTA owns 128 / CL of the rows; the others
//      write their sums for these into its shared memory, it adds them (in the
//      CTAs' order), and writes z times its scale as the operand of step 3 (three
//      bf16 parts, adapters.cuh) into every CTA's: at ranks above 16 in the place of
//      the sums, when all CTAs have read theirs (operand and sums side by side leave
//      the rings of x and y two slots in place of three: 8192 tokens of one
//      request, rank 16, 29 us against 27).  All remote traffic is stores, whose
//      latency nobody waits for (reading the others' sums took 5 to 8 us of a tile's
//      30).
//   3. out: per chunk of 64 (fp32: 32) output columns and adapter of the tile, one
//      accumulator of Z B_i^T; rows of that adapter add it to their y, which TMA
//      brought into the same ring that x came through (it fills while the sums
//      of step 2 meet), and TMA stores the chunk.
//
// A row's results come from its own adapter's accumulators alone, so weights that
// are not finite spoil no other adapter's tokens.
//
// Warps: 0 loads x and y, 11-12 A and B (TMA; one thread for all of it spends longer on
// its waits and loads than a chunk takes), 1-2 MMA issuers, 3-10 epilogue (two groups
// of a thread per row), 13 and 15 clean B's unused columns, 14 stores.
// Bound by memory: x and y in, out once; the adapters come from L2.
#include <cooperative_groups.h>
#include <cuda.h>

#include "adapters.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace moe {

namespace {

using namespace sm100;
namespace cg = cooperative_groups;

constexpr int kTcRows = 128;
constexpr int kTcEpiWarps = 8;           // 4 per stream
constexpr int kTcSmall = 11, kTcCleaner = 13, kTcStore = 14, kTcCleaner1 = 15;     // warps
constexpr int kTcThreads = 32 * (kTcCleaner1 + 1);
// Two of everything per chunk: an MMA issuer's waits and commits, and an epilogue
// group's chain from accumulator to store, each take about as long as a chunk's way
// from memory.  So two issuers and two epilogue groups take turns by chunk, each
// with rings and accumulators of its own (a parity wait tells only a slot's next use
// from the last: whoever waits has to see every use).
constexpr int kTcStreams = 2;
constexpr int kTcTmemCols = 512;
constexpr int kTcZCols = 256;            // z: adapters of a pass x streams x rank
constexpr int kTcDBufs = 2;              // output accumulators of a stream (64 columns each)
constexpr int kTcCtas = 148;             // SMs of the device: what the tile split aims at

// RB: blocks of 64 rank columns; WIDE: y and out fp32
template <int RB, bool WIDE>
struct TcCfg {
    static constexpr int NC = WIDE ? 32 : 64;               // output columns of a chunk: 128 bytes of a row
    static constexpr int BIG = kTcRows * 128;               // a chunk of x or y
    static constexpr int SMALL = RB * 64 * 128;             // a chunk of one A, or of one B
    // slots of each stream's rings
    static constexpr int NBIG = RB == 1 ? 3 : 2, NSMALL = RB == 1 ? 4 : 1;
    static constexpr int OFF_SMALL = kTcStreams * NBIG * BIG;
    // fp32 sums of the rows that this CTA owns, by source CTA; the second product's
    // operand lies behind as many of them as there is room for, and otherwise in
    // their place once they are read
    static constexpr int OFF_Z = OFF_SMALL + kTcStreams * NSMALL * SMALL, OFF_OP = OFF_Z + (RB == 1 ? 15 * 1024 : 0);
    static constexpr int SUMS = RB * 64 * kTcRows * 4;
    static constexpr int ZBLOCK = kTcRows * 128;                    // 64 columns of a part of the operand
    static constexpr int OPERAND = RB * kZParts * ZBLOCK;
    static_assert(OFF_OP + OPERAND >= OFF_Z + SUMS, "the sums end within the operand");
    static constexpr size_t BYTES = OFF_OP + OPERAND + 1024;        // base rounded up to the swizzle's 1024
};

struct TcMaps {
    CUtensorMap x, y, out, a, b;
};

MOE_DEV void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                 ::"r"(smem_u32(dst)), "l"((uint64_t)map), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2) : "memory");
}
// arrive on the barrier at the same place in CTA `rank` of the cluster,
// releasing this thread's earlier writes to the cluster
MOE_DEV void mbar_arrive_cluster(uint64_t* bar, int rank) {
    asm volatile("{ .reg .b32 ra; mapa.shared::cluster.u32 ra, %0, %1;\n"
                 "  mbarrier.arrive.release.cluster.shared::cluster.b64 _, [ra]; }"
                 ::"r"(smem_u32(bar)), "r"(rank) : "memory");
}
// 16 bytes to the same place in CTA `rank` of the cluster
MOE_DEV void st_cluster_v4(void* p, int rank, uint4 v) {
    asm volatile("{ .reg .b32 ra; mapa.shared::cluster.u32 ra, %0, %1;\n"
                 "  st.shared::cluster.v4.b32 [ra], {%2, %3, %4, %5}; }"
                 ::"r"(smem_u32(p)), "r"(rank), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
MOE_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
MOE_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// bounded wait that acquires what the cluster's arrivals released
MOE_DEV bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code, long long limit) {
    const long long t0 = clock64();
    while (true) {
        uint32_t ok;
        asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                     : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
        if (ok) return true;
        if (*abort_flag) return false;
        if (clock64() - t0 > limit) {
            *abort_flag = 1;
            if (err) atomicCAS(err, 0, code);
            return false;
        }
    }
}
MOE_DEV bool all_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* err, int code, long long limit) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, code, limit));
}
// 16-byte piece j of row r of a 128-byte-swizzled tile
MOE_DEV uint32_t sw_piece(int r, int j) { return (uint32_t)(r * 128 + ((j ^ (r & 7)) << 4)); }

// The chunks lo .. hi - 1 in order, started at another one (any integer turn)
struct Turned {
    int at, lo, hi;
    MOE_DEV Turned(int l, int h, int turn) : at(l + turn % max(h - l, 1)), lo(l), hi(h) {}
    MOE_DEV void next() {
        if (++at == hi) at = lo;
    }
};

// A place in a ring of N slots and the parity of its use
template <int N>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    MOE_DEV void next() {
        if (++slot == N) { slot = 0; phase ^= 1u; }
    }
};
// a wait that ends by itself after a while, whatever the barrier does
MOE_DEV void wait_some(uint64_t* bar, uint32_t parity) {
    for (int q = 0; q < 1000 && !mbar_try_wait(bar, parity); ++q) {}
}

// Calls without an error word of their own: how many CTAs have given up a wait on
// this device, and the last one's site.  It only grows, so that no report is lost to
// another stream's and every stream can ask for itself.
struct WaitErrors {
    unsigned count;
    int code;
};
__device__ WaitErrors g_wait_errors;

// 32 output columns of a row, taken again in fp32 (a NaN among them whose z parts
// cannot tell, see adapters.cuh; rare, so not inlined).  n: the first column's
// number, c: its place in the chunk at `tile` (which holds y), op: z's parts
template <int RB, bool WIDE>
__device__ __noinline__ void tc_repair(const AdapterArgs& a, int id, int rank, int n, int row, uint8_t* tile, int c, const uint8_t* op) {
    using C = TcCfg<RB, WIDE>;
    auto z_of = [&](int r) {
        float v = 0.0f;
        for (int h = kZParts - 1; h >= 0; --h)
            v += bf16_to_f(*reinterpret_cast<const __nv_bfloat16*>(op + (h * RB + (r >> 6)) * C::ZBLOCK + sw_piece(row, (r & 63) >> 3) + (r & 7) * 2));
        return v;
    };
    const __nv_bfloat16* b = reinterpret_cast<const __nv_bfloat16*>(a.b) + ((size_t)id * a.N + n) * a.R;
    for (int u = 0; u < 32 && n + u < a.N; ++u, b += a.R) {
        const float s = whole_product(z_of, b, rank);
        if (WIDE) {
            float* p = reinterpret_cast<float*>(tile + sw_piece(row, (c + u) >> 2)) + ((c + u) & 3);
            *p += s;
        } else {
            __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(tile + sw_piece(row, (c + u) >> 3)) + ((c + u) & 7);
            *p = __float2bfloat16_rn(bf16_to_f(*p) + s);
        }
    }
}

template <int RB, bool WIDE>
__global__ void __launch_bounds__(kTcThreads, 1)
k_adapter_tc(const __grid_constant__ AdapterArgs a, const __grid_constant__ TcMaps maps, int rows_a, int per_pass) {
    using C = TcCfg<RB, WIDE>;
    constexpr int NBIG = C::NBIG, NSMALL = C::NSMALL, NC = C::NC;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t big_full[kTcStreams][NBIG], big_empty[kTcStreams][NBIG], chunk_done[kTcStreams][NBIG];
    __shared__ uint64_t small_full[kTcStreams][NSMALL], small_empty[kTcStreams][NSMALL], small_clean[kTcStreams][NSMALL];
    __shared__ uint64_t z_full, z_free, z_ready, z_read, op_full, mma_done[kTcStreams];
    __shared__ uint64_t d_full[kTcStreams][kTcDBufs], d_empty[kTcStreams][kTcDBufs];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag, s_err;
    __shared__ int s_sent[2 * kTcStreams];       // loads of x and y, of A and B by stream
    __shared__ int s_id[kTcRows], s_list[kTcRows], s_rank[kTcRows];
    __shared__ unsigned s_first[4];
    __shared__ float s_scale[kTcRows];
    // the swizzle and its descriptors count from 1024-byte boundaries
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    cg::cluster_group cl = cg::this_cluster();
    int* const err = a.err ? a.err : &s_err;
    const long long limit = a.wait_limit > 0 ? a.wait_limit : kWaitLimitCycles;
    const int CL = (int)cl.num_blocks(), crank = (int)cl.block_rank();
    const int t0 = (int)(blockIdx.x / CL) * kTcRows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nk = (a.K + 63) / 64, nn = (a.N + NC - 1) / NC;
    const int k0 = (int)((long long)nk * crank / CL), k1 = (int)((long long)nk * (crank + 1) / CL);
    const int n0 = (int)((long long)nn * crank / CL), n1 = (int)((long long)nn * (crank + 1) / CL);
    const int early = min(kTcStreams * NBIG, k1 - k0);
    // each tile starts its chunks elsewhere, so that not all CTAs ask for the
    // same lines of A and B at once
    const int turn = t0 / kTcRows * 5 % 4096;

    auto rank_of = [&](int id) { return min(a.ranks ? __ldg(a.ranks + id) : a.R, a.R); };
    // The start: four warps list the tile's adapters while others make the
    // barriers, send for the first chunks of x (which need no adapter) and take
    // the tensor memory.
    if (warp < 4) {
        // the adapters in order of their first row
        const int t = t0 + (int)threadIdx.x;
        const int id = t < a.T ? __ldg(a.ids + t) : -1;
        const int my_id = id >= 0 && id < a.n && rank_of(id) > 0 ? id : -1;
        s_id[threadIdx.x] = my_id;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const unsigned same = __match_any_sync(0xffffffffu, my_id);
        bool leads = my_id >= 0 && lane == __ffs(same) - 1;          // the first row of its adapter
        for (unsigned todo = __ballot_sync(0xffffffffu, leads); todo; todo &= todo - 1) {
            const int l = __ffs(todo) - 1, lid = __shfl_sync(0xffffffffu, my_id, l);
            bool seen = false;               // in an earlier warp's rows
            for (int w = 0; w < warp; ++w) seen = seen || s_id[32 * w + lane] == lid;
            if (__any_sync(0xffffffffu, seen) && lane == l) leads = false;
        }
        const unsigned mine = __ballot_sync(0xffffffffu, leads);
        if (lane == 0) s_first[warp] = mine;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        int at = __popc(mine & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) at += __popc(s_first[w]);
        if (leads) {
            s_list[at] = my_id;
            s_rank[at] = rank_of(my_id);
        }
    } else if (warp == kTcStore && lane == 0) {
        for (int w = 0; w < kTcStreams; ++w) {
            for (int i = 0; i < NBIG; ++i) {
                mbar_init(&big_full[w][i], 1);
                mbar_init(&big_empty[w][i], 1);
                mbar_init(&chunk_done[w][i], kTcEpiWarps / kTcStreams);
            }
            for (int i = 0; i < NSMALL; ++i) {
                mbar_init(&small_full[w][i], 1);
                mbar_init(&small_empty[w][i], 1);
                mbar_init(&small_clean[w][i], 1);
            }
            for (int i = 0; i < kTcDBufs; ++i) { mbar_init(&d_full[w][i], 1); mbar_init(&d_empty[w][i], kTcEpiWarps / kTcStreams); }
        }
        mbar_init(&z_full, (uint32_t)min(kTcStreams, k1 - k0));
        mbar_init(&z_free, kTcEpiWarps);
        mbar_init(&z_ready, (uint32_t)(kTcEpiWarps * CL));
        mbar_init(&z_read, (uint32_t)(kTcEpiWarps * CL));
        mbar_init(&op_full, (uint32_t)(kTcEpiWarps * CL));
        for (int w = 0; w < kTcStreams; ++w) mbar_init(&mma_done[w], 1);
        abort_flag = 0;
        s_err = 0;
        fence_barrier_init();
        fence_proxy_async_smem();
        Turned kc(k0, k1, turn);
        for (int i = 0; i < early; ++i, kc.next()) {
            const int w = i & (kTcStreams - 1), slot = i / kTcStreams;
            mbar_arrive_expect_tx(&big_full[w][slot], C::BIG);
            tma_load_2d(smem + (w * NBIG + slot) * C::BIG, &maps.x, 64 * kc.at, t0, &big_full[w][slot]);
        }
    } else if (warp == kTcCleaner) {
        tmem_alloc(&tmem_slot, kTcTmemCols);
    } else if (warp == 4 && lane < 3) {
        const CUtensorMap* p = lane == 0 ? &maps.a : (lane == 1 ? &maps.b : &maps.y);
        asm volatile("prefetch.tensormap [%0];" ::"l"((uint64_t)p) : "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this CTA's barriers are there for remote arrivals (waited for before the
    // first; their initialisation was released to the cluster where they were made)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    int D = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) D += __popc(s_first[w]);
    const uint32_t tmem = tmem_slot;

    const int passes = max(1, (D + per_pass - 1) / per_pass);      // without an adapter x is let through all the same

    // stream w's chunks: lo + w, lo + w + 2, ...
    auto count = [](int lo, int hi, int w) { return (hi - lo - w + kTcStreams - 1) / kTcStreams; };

    if (warp == 0) {
        // ------------------------------ producer of x and y (one thread)
        if (lane == 0) {
            Ring<NBIG> ring[kTcStreams];
            int sent[kTcStreams] = {0, 0};
            bool ok = true;
            auto send = [&](int i, const CUtensorMap* map, int col, bool out) {
                Ring<NBIG>& r = ring[i & (kTcStreams - 1)];
                const int w = i & (kTcStreams - 1);
                if (!out) {
                    ok = mbar_wait(&big_empty[w][r.slot], r.phase ^ 1u, &abort_flag, err, 41, limit);
                    if (!ok) return;
                    mbar_arrive_expect_tx(&big_full[w][r.slot], C::BIG);
                    tma_load_2d(smem + (w * NBIG + r.slot) * C::BIG, map, col, t0, &big_full[w][r.slot]);
                }
                ++sent[w];
                r.next();
            };
            for (int p = 0; ok && p < passes; ++p) {
                Turned kc(k0, k1, turn);
                // the first ones went out at the start, into slots not used before
                for (int i = 0; ok && i < k1 - k0; ++i, kc.next()) send(i, &maps.x, 64 * kc.at, p == 0 && i < early);
            }
            Turned nc(n0, n1, turn);
            for (int i = 0; ok && i < n1 - n0; ++i, nc.next()) send(i, &maps.y, NC * nc.at, false);
            for (int w = 0; w < kTcStreams; ++w) s_sent[w] = max(sent[w], count(0, early, w));
        }
        __syncwarp();
    } else if (warp == kTcSmall || warp == kTcSmall + 1) {
        // ------------------ producers of A and B, one stream each (one thread)
        if (lane == 0) {
            const int w = warp - kTcSmall;
            Ring<NSMALL> r;
            int sent = 0;
            bool ok = true;
            uint8_t* slots = smem + C::OFF_SMALL + w * NSMALL * C::SMALL;
            for (int p = 0; ok && p < passes; ++p) {
                const int d0 = p * per_pass, d1 = min(D, d0 + per_pass);
                Turned kc(k0, k1, turn);
                for (int i = 0; ok && i < k1 - k0; ++i, kc.next()) {
                    if ((i & (kTcStreams - 1)) != w) continue;
                    for (int d = d0; d < d1; ++d, r.next(), ++sent) {
                        if (!(ok = mbar_wait(&small_empty[w][r.slot], r.phase ^ 1u, &abort_flag, err, 42, limit))) break;
                        mbar_arrive_expect_tx(&small_full[w][r.slot], (uint32_t)rows_a * 128u);
                        tma_load_3d(slots + r.slot * C::SMALL, &maps.a, 64 * kc.at, 0, s_list[d], &small_full[w][r.slot]);
                    }
                }
            }
            Turned nc(n0, n1, turn);
            for (int i = 0; ok && i < n1 - n0; ++i, nc.next()) {
                if ((i & (kTcStreams - 1)) != w) continue;
                for (int d = 0; d < D; ++d, r.next(), ++sent) {
                    if (!(ok = mbar_wait(&small_empty[w][r.slot], r.phase ^ 1u, &abort_flag, err, 44, limit))) break;
                    const int nb = (s_rank[d] + 63) / 64;
                    mbar_arrive_expect_tx(&small_full[w][r.slot], (uint32_t)(nb * NC * 128));
                    for (int b = 0; b < nb; ++b)
                        tma_load_3d(slots + r.slot * C::SMALL + b * NC * 128, &maps.b, 64 * b, NC * nc.at, s_list[d], &small_full[w][r.slot]);
                }
            }
            s_sent[kTcStreams + w] = sent;
        }
        __syncwarp();
    } else if (warp <= kTcStreams) {
        // --------------------------------------- MMA issuers (one thread)
        if (lane == 0) {
            const int w = warp - 1;
            Ring<NBIG> big;
            Ring<NSMALL> small;
            int unit = 0;                            // this stream's B tiles so far
            bool ok = true;
            const uint32_t base = smem_u32(smem);
            // descriptors of the rings' starts; an address counts in 16 bytes
            const uint64_t dx = desc_kmajor_sw128(base + w * NBIG * C::BIG), ds = desc_kmajor_sw128(base + C::OFF_SMALL + w * NSMALL * C::SMALL);
            const uint64_t dz = desc_kmajor_sw128(base + C::OFF_OP);
            const uint32_t idz = idesc_bf16_f32(kTcRows, rows_a), ido = idesc_bf16_f32(kTcRows, NC);
            for (int p = 0; ok && p < passes; ++p) {
                const int nd = min(D - p * per_pass, per_pass);
                if (p > 0 && !(ok = mbar_wait(&z_free, (uint32_t)(p - 1) & 1u, &abort_flag, err, 45, limit))) break;
                tc_fence_after();
                for (int kc = k0 + w; ok && kc < k1; kc += kTcStreams, big.next()) {
                    if (!(ok = mbar_wait(&big_full[w][big.slot], big.phase, &abort_flag, err, 46, limit))) break;
                    const uint64_t xd = dx + (uint64_t)(big.slot * (C::BIG >> 4));
                    for (int d = 0; d < nd; ++d, small.next()) {
                        if (!(ok = mbar_wait(&small_full[w][small.slot], small.phase, &abort_flag, err, 47, limit))) break;
                        const uint64_t ad = ds + (uint64_t)(small.slot * (C::SMALL >> 4));
                        const uint32_t dst = tmem + (uint32_t)((d * kTcStreams + w) * rows_a);
#pragma unroll
                        for (int q = 0; q < 4; ++q) mma_bf16(dst, xd + 2 * q, ad + 2 * q, idz, kc > k0 + w || q > 0 ? 1u : 0u);
                        mma_commit(&small_empty[w][small.slot]);
                    }
                    if (ok) mma_commit(&big_empty[w][big.slot]);
                }
                if (ok && w < k1 - k0) mma_commit(&z_full);
            }
            if (ok && D > 0) {
                ok = mbar_wait_cluster(&op_full, 0u, &abort_flag, err, 48, limit);
                fence_proxy_async_smem();            // the operand came by ordinary stores
            }
            for (int nc = n0 + w; ok && nc < n1; nc += kTcStreams)
                for (int d = 0; d < D; ++d, small.next(), ++unit) {
                    const int buf = unit & 1, steps = (s_rank[d] + 15) / 16;
                    ok = a.ranks ? mbar_wait(&small_clean[w][small.slot], (uint32_t)(unit / NSMALL) & 1u, &abort_flag, err, 49, limit)
                                 : mbar_wait(&small_full[w][small.slot], small.phase, &abort_flag, err, 49, limit);
                    ok = ok && mbar_wait(&d_empty[w][buf], ((uint32_t)(unit >> 1) & 1u) ^ 1u, &abort_flag, err, 50, limit);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t bd = ds + (uint64_t)(small.slot * (C::SMALL >> 4));
                    const uint32_t dst = tmem + kTcZCols + 64u * (uint32_t)(w * kTcDBufs + buf);
                    // (unrolled, 8192 tokens of 16 requests, rank 64: 49.7 -> 44.8 us; the first
                    // step by itself, 4096 tokens of 12 requests, rank 16: 25.8 -> 24.4 us)
                    auto step = [&](int q) {
#pragma unroll
                        for (int h = 0; h < kZParts; ++h)
                            mma_bf16(dst, dz + (uint64_t)((h * RB + (q >> 2)) * (C::ZBLOCK >> 4) + 2 * (q & 3)),
                                     bd + (uint64_t)((q >> 2) * (NC * 128 >> 4) + 2 * (q & 3)), ido, h + q > 0 ? 1u : 0u);
                    };
                    step(0);
                    if (steps > 1) {
#pragma unroll
                        for (int q = 1; q < 4 * RB; ++q)
                            if (q < steps) step(q);
                    }
                    mma_commit(&small_empty[w][small.slot]);
                    mma_commit(&d_full[w][buf]);
                }
            mma_commit(&mma_done[w]);                // nothing of this thread's runs on when the CTA ends
            wait_some(&mma_done[w], 0u);
        }
        __syncwarp();
    } else if (warp == kTcStore) {
        // -------------------------------------------- stores (one thread)
        if (lane == 0) {
            Ring<NBIG> ring[kTcStreams];                         // phase: of the slot's chunk_done
            for (int w = 0; w < kTcStreams; ++w) ring[w].slot = passes * count(k0, k1, w) % NBIG;
            int first[kTcStreams] = {ring[0].slot, ring[1].slot};
            Turned at(n0, n1, turn);
            bool ok = true;
            for (int i = 0; ok && i < n1 - n0; ++i, at.next()) {
                const int w = i & (kTcStreams - 1), s = ring[w].slot;
                if (!(ok = mbar_wait(&chunk_done[w][s], ring[w].phase, &abort_flag, err, 59, limit))) break;
                tma_store_2d(&maps.out, NC * at.at, t0, smem + (w * NBIG + s) * C::BIG);
                bulk_commit();
                bulk_wait_read<0>();
                mbar_arrive(&big_empty[w][s]);
                // the ring's round, counted from where the stream's chunks began
                ring[w].slot = s + 1 == NBIG ? 0 : s + 1;
                if (ring[w].slot == first[w]) ring[w].phase ^= 1u;
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp == kTcCleaner || warp == kTcCleaner1) {
        // With ranks of their own, adapters' B columns behind the rank may hold
        // anything: those of the last k step are zeroed where they arrived, whole
        // pieces by a warp per stream (rank <= 16, 16 requests, 8192 tokens: column by
        // column and one warp 61 us, by pieces 41, two warps 37; without ranks of
        // their own 31).
        if (a.ranks) {
            // the first product's uses of the slots are over then, and the slots
            // go on where it left off
            bool ok = D == 0 || __all_sync(0xffffffffu, mbar_wait_cluster(&op_full, 0u, &abort_flag, err, 57, limit));
            const int w = warp == kTcCleaner ? 0 : 1;
            int used = D * count(k0, k1, w);
            for (int nc = n0 + w; ok && nc < n1; nc += kTcStreams) {
                for (int d = 0; d < D; ++d, ++used) {
                    const int slot = used % NSMALL;
                    if (!(ok = all_wait(&small_full[w][slot], (uint32_t)(used / NSMALL) & 1u, &abort_flag, err, 56, limit))) break;
                    const int rank = s_rank[d], steps = (rank + 15) / 16;
                    if (rank & 15) {
                        uint8_t* bt = smem + C::OFF_SMALL + (w * NSMALL + slot) * C::SMALL;
                        // a row of the step is two pieces of eight columns: the one
                        // that the rank ends in keeps `left` of them, one behind it none
                        const int col = rank & ~7, left = rank & 7, end = 16 * steps;
                        uint32_t keep[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) keep[q] = (left > 2 * q ? 0xffffu : 0u) | (left > 2 * q + 1 ? 0xffff0000u : 0u);
                        uint8_t* block = bt + (col >> 6) * NC * 128;
#pragma unroll
                        for (int r = lane; r < NC; r += 32) {
                            uint4* piece = reinterpret_cast<uint4*>(block + sw_piece(r, (col & 63) >> 3));
                            uint4 v = make_uint4(0, 0, 0, 0);
                            if (left) v = *piece;
                            *piece = make_uint4(v.x & keep[0], v.y & keep[1], v.z & keep[2], v.w & keep[3]);
                            if (end - col > 8)
                                *reinterpret_cast<uint4*>(block + sw_piece(r, ((col & 63) >> 3) + 1)) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&small_clean[w][slot]);
                }
            }
        }
    } else {
        // --------------------------------------------------------- epilogue
        const int quarter = warp & 3, group = (warp - 3) >> 2, row = quarter * 32 + lane;
        const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
        const int id = s_id[row];
        int mine = -1;
        for (int d = 0; id >= 0 && mine < 0; ++d) mine = s_list[d] == id ? d : -1;
        if (group == 0) s_scale[row] = id >= 0 ? __ldg(a.scales + id) : 0.0f;     // read behind z_ready
        bool ok = true;
        cluster_wait();
        if (D > 0) {
            // [source CTA][rank / 4][own row]
            const int own_rows = kTcRows / CL, owner = row / own_rows, quads = rows_a / 4;
            float4* zp = reinterpret_cast<float4*>(smem + C::OFF_Z);
            for (int p = 0; ok && p < passes; ++p) {
                if (!(ok = all_wait(&z_full, (uint32_t)p & 1u, &abort_flag, err, 51, limit))) break;
                tc_fence_after();
                const int nd = min(D - p * per_pass, per_pass);
                for (int d = 0; d < nd; ++d) {
                    const bool own = mine == p * per_pass + d;
                    if (!__any_sync(0xffffffffu, own)) continue;
                    for (int c = 16 * group; c < rows_a; c += 32) {
                        float v[16];
                        const uint32_t src = tmem + lane_base + (uint32_t)(d * kTcStreams * rows_a + c);
                        tmem_ld16(src, v);
                        if (k1 - k0 > 1) {               // the second issuer's chunks
                            float u[16];
                            tmem_ld16(src + (uint32_t)rows_a, u);
#pragma unroll
                            for (int e = 0; e < 16; ++e) v[e] += u[e];
                        }
                        if (own) {
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                st_cluster_v4(zp + (crank * quads + c / 4 + q) * own_rows + row % own_rows, owner,
                                              make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                                         __float_as_uint(v[4 * q + 3])));
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&z_free);
            }
            __syncwarp();
            if (ok) {
                if (lane < CL && !((int)blockIdx.x == a.withhold && warp == 3)) mbar_arrive_cluster(&z_ready, lane);
                ok = __all_sync(0xffffffffu, mbar_wait_cluster(&z_ready, 0u, &abort_flag, err, 52, limit));
            }
            if (ok) {
                // this CTA's rows, eight columns of one at a time
                constexpr int ITEMS = kTcRows * RB * 8 / (kTcEpiWarps * 32);
                const int items = own_rows * (rows_a / 8), i0 = (int)threadIdx.x - 96;
                auto sum = [&](int i, float (&v)[8]) {
                    const int rl = i % own_rows, j = i / own_rows, r = crank * own_rows + rl;     // row, eight columns
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = 0.0f;
                    if (s_id[r] < 0) return;
                    const int rank = rank_of(s_id[r]);
                    const float scale = s_scale[r];
#pragma unroll 1
                    for (int q = 0; q < CL; ++q) {
                        const float4 v0 = zp[(q * quads + 2 * j) * own_rows + rl], v1 = zp[(q * quads + 2 * j + 1) * own_rows + rl];
                        v[0] += v0.x; v[1] += v0.y; v[2] += v0.z; v[3] += v0.w;
                        v[4] += v1.x; v[5] += v1.y; v[6] += v1.z; v[7] += v1.w;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[q] = 8 * j + q < rank ? v[q] * scale : 0.0f;
                };
                auto put = [&](int i, const float (&v)[8]) {
                    const int j = i / own_rows, r = crank * own_rows + i % own_rows;
                    uint32_t w[4][kZParts];
#pragma unroll
                    for (int q = 0; q < 4; ++q) split_z2(v[2 * q], v[2 * q + 1], w[q]);
                    uint8_t* d = smem + C::OFF_OP + (j >> 3) * C::ZBLOCK + sw_piece(r, j & 7);
#pragma unroll 1
                    for (int q = 0; q < CL; ++q)
#pragma unroll
                        for (int h = 0; h < kZParts; ++h) st_cluster_v4(d + h * RB * C::ZBLOCK, q, make_uint4(w[0][h], w[1][h], w[2][h], w[3][h]));
                };
                if (C::OFF_Z + rows_a * kTcRows * 4 <= C::OFF_OP) {
#pragma unroll 1
                    for (int i = i0; i < items; i += kTcEpiWarps * 32) {
                        float z[8];
                        sum(i, z);
                        put(i, z);
                    }
                } else {
                    // the operand takes the sums' place: it is written when nobody
                    // needs them any more
                    float z[ITEMS][8];
#pragma unroll
                    for (int u = 0; u < ITEMS; ++u)
                        if (i0 + u * kTcEpiWarps * 32 < items) sum(i0 + u * kTcEpiWarps * 32, z[u]);
                    __syncwarp();
                    if (lane < CL) mbar_arrive_cluster(&z_read, lane);
                    ok = __all_sync(0xffffffffu, mbar_wait_cluster(&z_read, 0u, &abort_flag, err, 53, limit));
#pragma unroll
                    for (int u = 0; u < ITEMS; ++u)
                        if (ok && i0 + u * kTcEpiWarps * 32 < items) put(i0 + u * kTcEpiWarps * 32, z[u]);
                }
            }
            if (ok) {
                asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
                __syncwarp();
                if (lane < CL) mbar_arrive_cluster(&op_full, lane);
            }
        }
        // The first product's uses of the slots are over (a parity tells only one
        // use from the next), and this group's chunks, every other one, go on
        // where its stream left off.
        if (D == 0) ok = all_wait(&z_full, 0u, &abort_flag, err, 58, limit);
        bool unsure = false;                 // this row has a z that its parts may not stand for
        if (ok && D > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait_cluster(&op_full, 0u, &abort_flag, err, 60, limit));
            for (int j = 0; ok && j < rows_a / 8; ++j) {
                const uint4 p = *reinterpret_cast<const uint4*>(smem + C::OFF_OP + (j >> 3) * C::ZBLOCK + sw_piece(row, j & 7));
                const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) unsure = unsure || z_unsure(bf16_lo(w[q])) || z_unsure(bf16_hi(w[q]));
            }
        }
        int unit = 0, big = passes * count(k0, k1, group);
        Turned at(n0, n1, turn);
        if (group) at.next();
        for (int nc = n0 + group; ok && nc < n1; nc += kTcStreams, ++big, at.next(), at.next()) {
            const int s = big % NBIG;
            if (!(ok = all_wait(&big_full[group][s], (uint32_t)(big / NBIG) & 1u, &abort_flag, err, 54, limit))) break;
            uint8_t* tile = smem + (group * NBIG + s) * C::BIG;
            for (int d = 0; d < D; ++d, ++unit) {
                const int buf = unit & 1;
                if (!(ok = all_wait(&d_full[group][buf], (uint32_t)(unit >> 1) & 1u, &abort_flag, err, 55, limit))) break;
                tc_fence_after();
                if (__any_sync(0xffffffffu, mine == d)) {
                    const uint32_t src = tmem + lane_base + kTcZCols + 64u * (uint32_t)(group * kTcDBufs + buf);
                    // 32 output columns at a time: 64 (fp32: 128) bytes of the row
#pragma unroll
                    for (int c = 0; c < NC; c += 32) {
                        uint32_t r[32];
                        tmem_ld_x32c(src + (uint32_t)c, r);
                        bool nan = false;
                        if (unsure)
#pragma unroll
                            for (int e = 0; e < 32; ++e) nan = nan || __uint_as_float(r[e]) != __uint_as_float(r[e]);
                        if (mine == d && nan) {
                            tc_repair<RB, WIDE>(a, id, s_rank[d], NC * at.at + c, row, tile, c, smem + C::OFF_OP);
                        } else if (mine == d) {
#pragma unroll
                            for (int j = 0; j < (WIDE ? 8 : 4); ++j) {
                                uint4* p = reinterpret_cast<uint4*>(tile + sw_piece(row, c / 8 + j));
                                uint4 v = *p;
                                uint32_t* w = &v.x;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    if (WIDE) w[q] = __float_as_uint(__uint_as_float(w[q]) + __uint_as_float(r[4 * j + q]));
                                    else w[q] = pack_bf16x2(bf16_lo(w[q]) + __uint_as_float(r[(8 * j + 2 * q) & 31]),
                                                            bf16_hi(w[q]) + __uint_as_float(r[(8 * j + 2 * q + 1) & 31]));
                                }
                                *p = v;
                            }
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&d_empty[group][buf]);
            }
            if (!ok) break;
            fence_proxy_async_smem();        // the chunk is stored from where it lies
            __syncwarp();
            if (lane == 0) mbar_arrive(&chunk_done[group][s]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (abort_flag && threadIdx.x == 0) {
        // given up: what is in flight lands first (bounded).  A slot of n loads has
        // had n - 1 whole phases before the last one's.
        for (int w = 0; w < kTcStreams; ++w) {
            for (int i = 0; i < NBIG; ++i)
                if (s_sent[w] > i) wait_some(&big_full[w][i], (uint32_t)((s_sent[w] - i - 1) / NBIG) & 1u);
            for (int i = 0; i < NSMALL; ++i)
                if (s_sent[kTcStreams + w] > i) wait_some(&small_full[w][i], (uint32_t)((s_sent[kTcStreams + w] - i - 1) / NSMALL) & 1u);
        }
        if (s_err) {
            atomicExch(&g_wait_errors.code, s_err);
            __threadfence();
            atomicAdd(&g_wait_errors.count, 1u);
        }
    }
    if (warp == kTcCleaner) tmem_dealloc(tmem, kTcTmemCols);
    if (warp <= kTcStreams || warp >= kTcSmall) cluster_wait();     // of the first arrival
    cluster_arrive();                        // nobody leaves while others may write to its shared memory
    cluster_wait();
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeTiledFn>(p);
    }();
    return fn;
}

// rows of `cols` elements, `ld` elements apart; boxes of 128 bytes x box_rows
bool map_rows(CUtensorMap* m, const void* base, bool fp32, int rows, int cols, long long ld, int box_rows) {
    const int es = fp32 ? 4 : 2;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld * es};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)box_rows}, one[2] = {1, 1};
    return encode_fn()(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
                       one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// contiguous bf16 [n][rows][cols]; boxes of 64 columns x box_rows of one matrix, zeros past its edges
bool map_stack(CUtensorMap* m, const void* base, int n, int rows, int cols, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)rows * cols * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1}, one[3] = {1, 1, 1};
    return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int RB, bool WIDE>
cudaError_t launch_tc(const AdapterArgs& a, cudaStream_t st) {
    using C = TcCfg<RB, WIDE>;
    if (!encode_fn()) return cudaErrorNotSupported;
    const int rows_a = (a.R + 15) / 16 * 16;
    TcMaps m;
    if (!map_rows(&m.x, a.x, false, a.T, a.K, a.ld_x, kTcRows) || !map_rows(&m.y, a.y, WIDE, a.T, a.N, a.ld_y, kTcRows) ||
        !map_rows(&m.out, a.out, WIDE, a.T, a.N, a.ld_out, kTcRows) || !map_stack(&m.a, a.a, a.n, a.R, a.K, rows_a) ||
        !map_stack(&m.b, a.b, a.n, a.N, a.R, C::NC))
        return cudaErrorNotSupported;
    // CTAs for about one wave; no share of K or N is empty
    const int tiles = (a.T + kTcRows - 1) / kTcRows;
    const int nk = (a.K + 63) / 64, nn = (a.N + C::NC - 1) / C::NC;
    auto k = k_adapter_tc<RB, WIDE>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // The largest cluster with which all tiles run at once: its CTAs share a GPC,
    // so fewer of the larger ones fit (here 74 of 2, 33 of 4, 15 of 8).
    int cluster = 8;
    for (; cluster > 1; cluster /= 2) {
        if (cluster > nk || cluster > nn || tiles * cluster > kTcCtas) continue;
        at[0].val.clusterDim.x = (unsigned)cluster;
        cfg.gridDim = dim3((unsigned)(tiles * cluster));
        int fit = 0;
        e = cudaOccupancyMaxActiveClusters(&fit, k, &cfg);
        if (e != cudaSuccess) return e;
        if (tiles <= fit) break;
    }
    at[0].val.clusterDim.x = (unsigned)cluster;
    cfg.gridDim = dim3((unsigned)(tiles * cluster));
    return cudaLaunchKernelEx(&cfg, k, a, m, rows_a, kTcZCols / (kTcStreams * rows_a));
}

}  // namespace

cudaError_t read_wait_errors(unsigned* count, int* code, cudaStream_t st) {
    WaitErrors w{};
    cudaError_t e = cudaMemcpyFromSymbolAsync(&w, g_wait_errors, sizeof w, 0, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    *count = w.count;
    *code = w.code;
    return e;
}

// the next launch's test of the bounded waits, on this host thread
static thread_local int t_withhold = -1;
static thread_local long long t_wait_limit = 0;
void set_adapter_wait_test(int withhold, long long limit) {
    t_withhold = withhold;
    t_wait_limit = withhold < 0 ? 0 : limit;
}

cudaError_t launch_add_adapters_tc(const AdapterArgs& args, cudaStream_t st) {
    AdapterArgs a = args;
    a.withhold = t_withhold;
    a.wait_limit = t_wait_limit;
    set_adapter_wait_test(-1, 0);
    if (a.R <= 64) return a.wide ? launch_tc<1, true>(a, st) : launch_tc<1, false>(a, st);
    // ranks above 64 with fp32 outputs have no variant here
    return a.wide ? cudaErrorNotSupported : launch_tc<2, false>(a, st);
}

}  // namespace moe
