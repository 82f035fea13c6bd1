// rb_epilogue.cuh -- the activations of the linear product's epilogue, their
// slopes, and the argument checks that its entry points share.
#pragma once

#include "rbw_internal.cuh"

namespace rbw {

// The activation is a template argument throughout: a run-time switch inside
// the element loops would keep every variant's registers live.  The divisions
// are the fast ones (2 ulp; a denominator past 2^126 gives 0, which is the
// limit here) and so are the exponentials: their error, a few 2^-23, is far
// below the bf16 rounding of what is stored, and the kernels that use them
// are bound by memory or by the tensor cores.

// The normal distribution function for GELU, from e = exp(-p^2 / 2):
//   Phi(-|p|) = e t Q(t),   t = 1 / (1 + 0.3 |p|),
// Q of degree 7, fitted to 1.4e-7 relative for |p| up to 13.5 (an exchange algorithm on erfc's scaled form; with
// the roundings 4.5e-7), where e leaves fp32.  (1 + erf(p / sqrt 2)) / 2 would cancel below zero: 4 % off at -5.
// erfcf has the accuracy, at a price (gradient of gelu(x + b) .* u, 2048 x 14336, in a graph: 77.1 us by erfcf, 60.4 by
// erff, 53.7 by this, which shares e with the slope).
__device__ __forceinline__ float normal_cdf(float p, float e)
{
    const float t = __fdividef(1.0f, fmaf(0.3f, fabsf(p), 1.0f));
    float q = 0.035892046988010406f;
    q = fmaf(q, t, -0.15811005234718323f);
    q = fmaf(q, t, 0.20791947841644287f);
    q = fmaf(q, t, -0.05512828379869461f);
    q = fmaf(q, t, 0.1293278932571411f);
    q = fmaf(q, t, 0.09968061000108719f);
    q = fmaf(q, t, 0.12079139053821564f);
    q = fmaf(q, t, 0.11962684988975525f);
    q *= t * e;
    return p > 0.0f ? 1.0f - q : q;
}

template <int ACT>
__device__ __forceinline__ float activate(float p)
{
    if constexpr (ACT == RB_ACT_RELU) {
        return p > 0.0f ? p : (p == p ? 0.0f : p);               // NaN stays
    } else if constexpr (ACT == RB_ACT_SILU) {
        return __fdividef(p, 1.0f + __expf(-p));
    } else if constexpr (ACT == RB_ACT_GELU) {
        return p * normal_cdf(p, __expf(-0.5f * p * p));
    } else if constexpr (ACT == RB_ACT_GELU_TANH) {
        // (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        const float u = 0.79788456080286536f * (p + 0.044715f * p * p * p);
        return __fdividef(p, 1.0f + __expf(-2.0f * u));
    } else {
        return p;
    }
}

// activate() and its slope together
template <int ACT>
__device__ __forceinline__ void activate_slope(float p, float& a, float& d)
{
    if constexpr (ACT == RB_ACT_RELU) {
        a = activate<ACT>(p);
        d = p > 0.0f ? 1.0f : (p == p ? 0.0f : p);
    } else if constexpr (ACT == RB_ACT_SILU) {
        const float q = __fdividef(1.0f, 1.0f + __expf(-p));
        a = p * q;
        d = q + a * (1.0f - q);
    } else if constexpr (ACT == RB_ACT_GELU) {
        const float e = __expf(-0.5f * p * p);
        const float c = normal_cdf(p, e);
        a = p * c;
        d = c + p * 0.39894228040143268f * e;
    } else if constexpr (ACT == RB_ACT_GELU_TANH) {
        const float p2 = p * p;
        const float u = 0.79788456080286536f * (p + 0.044715f * p2 * p);
        const float q = __fdividef(1.0f, 1.0f + __expf(-2.0f * u));
        a = p * q;
        const float w = a * (1.0f - q);                          // 0 long before p2 overflows
        d = w == 0.0f ? q : q + w * (2.0f * 0.79788456080286536f) * (1.0f + 3.0f * 0.044715f * p2);
    } else {
        a = p;
        d = 1.0f;
    }
}

inline bool good_act(int act) { return act >= RB_ACT_NONE && act <= RB_ACT_GELU_TANH; }

// Addresses of a [M][N] array with row stride ld (elements of `bytes`).
struct MatRange {
    uintptr_t lo, hi, pitch, width;
};
inline MatRange mat_range(const void* p, int64_t M, int64_t N, int64_t ld, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return MatRange{a, a + (uintptr_t)(((M - 1) * ld + N) * bytes), (uintptr_t)(ld * bytes), (uintptr_t)(N * bytes)};
}
// Arrays of one pitch may lie beside each other in the same rows (the halves of a [M][2N] buffer); with
// different pitches, ranges that meet count as an overlap.
inline bool overlaps(const MatRange& a, const MatRange& b)
{
    if (a.lo >= b.hi || b.lo >= a.hi) return false;
    if (a.pitch != b.pitch) return true;
    const uintptr_t d = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}

// Whether an array meets n bytes at p (nothing at null).
inline bool meets(const MatRange& a, const void* p, size_t n)
{
    return p && n && overlaps(a, mat_range(p, 1, (int64_t)n, (int64_t)n, 1));
}

}  // namespace rbw
