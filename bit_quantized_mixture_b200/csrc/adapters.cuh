// What the adapter kernels with tensor-core products share: z, an fp32 sum, as
// bf16 operands of the second product, and the outputs where that splitting
// shows.
#pragma once

#include "common.cuh"

namespace moe {

// The upper halves of two fp32 values as a bf16 pair (truncated), and in their
// place what is left of them.  Three such parts hold the 24 significant bits of a
// value exactly; truncation never goes past the largest finite bf16, and nothing
// is left of an infinity or a NaN (inf - inf would make a NaN of the whole).
MOE_DEV uint32_t take_bf16x2(float& lo, float& hi) {
    const uint32_t p = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
    lo = fabsf(lo) < INFINITY ? lo - bf16_lo(p) : 0.0f;
    hi = fabsf(hi) < INFINITY ? hi - bf16_hi(p) : 0.0f;
    return p;
}

// One output's second product in fp32, term by term: sum over r < rank of b[r] times
// what z_of(r) gives.  The products of z's parts are a NaN where an infinite weight
// meets a part that is zero or of the other sign; this tells whether the value
// itself is one.
template <typename Z>
MOE_DEV float whole_product(Z z_of, const __nv_bfloat16* b, int rank) {
    float s = 0.0f;
    for (int r = 0; r < rank; ++r) s = fmaf(bf16_to_f(b[r]), z_of(r), s);
    return s;
}
template <typename Z>
MOE_DEV bool any_nan(Z z_of, int rank) {
    bool nan = false;
    for (int r = 0; r < rank; ++r) nan = nan || z_of(r) != z_of(r);
    return nan;
}

// Is one of 32 fp32 values a NaN?  By their sum, two at a time (opposite infinities
// and overflows say yes as well, and are taken again for nothing).
MOE_DEV bool sum_is_nan(const uint32_t (&v)[32]) {
    unsigned long long s[4];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        unsigned long long p;
        asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(v[2 * i]), "r"(v[2 * i + 1]));
        if (i < 4) s[i] = p;
        else asm("add.rn.f32x2 %0, %1, %2;" : "=l"(s[i & 3]) : "l"(s[i & 3]), "l"(p));
    }
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(s[i]));
        t += __uint_as_float(lo) + __uint_as_float(hi);
    }
    return t != t;
}

}  // namespace moe
