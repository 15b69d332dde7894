// What the adapter kernels with tensor-core products share: z, an fp32 sum, as
// bf16 operands of the second product, and the outputs where that splitting
// shows.
#pragma once

#include "common.cuh"

namespace moe {

// z's parts: bf16 values of 8 significant bits each, largest first, by truncation
// (z - part is exact, no part is past the largest finite bf16).  Three hold all 24
// bits.  In one part an output lost up to 2^-8 of each term, more than its own
// rounding where y and the terms nearly cancel; in two, 2^-16.  8192 tokens, 2048 ->
// 2048, 16 requests, rank 64: one part 38 us, two 42, three 44.
constexpr int kZParts = 3;

// An infinite weight times a part that is zero would be a NaN where z is not zero.
// So parts of nothing hold 2^-126 with z's sign where that is below z's last bit
// (2^-28 of it); below kZSmall they stay zero, and whoever adds the outputs looks at
// them (z_unsure).
constexpr float kZSmall = 0x1p-98f;
MOE_DEV void split_z(float v, uint32_t (&part)[kZParts]) {
    const uint32_t fill = fabsf(v) < kZSmall ? 0u : (__float_as_uint(v) & 0x80000000u) | 0x00800000u;
#pragma unroll
    for (int q = 0; q < kZParts; ++q) {
        const uint32_t p = __float_as_uint(v) & 0xffff0000u;
        v = fabsf(v) < INFINITY ? v - __uint_as_float(p) : 0.0f;     // nothing is left of an infinity
        part[q] = q > 0 && (p << 1) == 0 ? fill : p;
    }
}
// two neighbours' parts as bf16 pairs
MOE_DEV void split_z2(float lo, float hi, uint32_t (&pair)[kZParts]) {
    uint32_t l[kZParts], h[kZParts];
    split_z(lo, l);
    split_z(hi, h);
#pragma unroll
    for (int q = 0; q < kZParts; ++q) pair[q] = __byte_perm(l[q], h[q], 0x7632);
}
MOE_DEV bool z_unsure(float v) { return v != 0.0f && fabsf(v) < kZSmall; }

// One output's second product in fp32, term by term: sum over r < rank of b[r] times
// what z_of(r) gives; a NaN in z spoils it.
template <typename Z>
MOE_DEV float whole_product(Z z_of, const __nv_bfloat16* b, int rank) {
    float s = 0.0f;
    for (int r = 0; r < rank; ++r) s = fmaf(bf16_to_f(b[r]), z_of(r), s);
    return s;
}

}  // namespace moe
