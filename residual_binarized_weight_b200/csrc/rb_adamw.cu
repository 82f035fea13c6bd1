// rb_adamw.cu -- one AdamW step over many tensors at once (rb_adamw_step): the
// latent weights, scales and biases that rb_qat_backward and
// rb_epilogue_backward leave gradients for.
//
//   m = b1 m + (1 - b1) g;   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// all in fp32, every product and sum rounded on its own (no contraction), so the
// states do not depend on which variant of the kernel computed them.
//
// 8-bit states: 256 consecutive elements share one fp32 scale per moment, the
// block's largest magnitude / 448, and hold e4m3 codes.  exp_avg is rounded to
// the nearest code (b1 moves it by a tenth a step, more than half a code's
// step of 1/16).  The second moment is held as its square root, which halves
// the octaves that the code has to span, and rounded stochastically: b2 moves
// it by 0.05 % a step, far less than half a code's step, so rounding to nearest
// would never move it.  A nonzero root never becomes code 0 (its quotient would
// be m / eps).  p is updated from the unrounded moments.
//
// One pass: 28 bytes per element (fp32 parameter, gradient and states) or
// 16.06 (8-bit states), HBM-bound.  A warp owns a block of 256 elements, eight per
// lane as two groups of four (16-byte loads and stores of fp32, 8-byte of
// bf16, 4-byte of codes), so a block's maximum is one warp reduction.  With fp32
// states that runs at the copy rate.  With 8-bit states instruction issue bounds it
// (two codes each way, the hash, a root): 127 us for 45 M elements in a graph, 112 at the copy
// rate.  Products and sums go two at a time (5 us less), and it wants warps: five CTAs of 48
// registers per SM are as fast as six of 40 (but 5.1 us against 6.0 for 120 small tensors),
// seven and eight of 32 take 16 us longer.
#include "rbw_internal.cuh"

#include <algorithm>
#include <cmath>

#include <cuda_fp8.h>

namespace rbw {
namespace {

constexpr int kBlock = 256;            // elements per scale of the 8-bit states, and per warp and step
constexpr int kWarps = 8;
constexpr int kChunk = kBlock * kWarps;        // elements per CTA: one block per warp (a loop over two measured 3 to 8 % slower)
constexpr float kE4m3Max = 448.0f;
constexpr float kTiny = 0x1p-100f;     // a block whose largest magnitude is below this is stored as zero

struct AdamwEntry {
    int64_t n;
    void* p;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    double lr;
    double wd;
    float step_size, decay;            // lr / (1 - b1^t) and 1 - lr wd, when both are known on the host
    int32_t kind;                      // 1: bf16 parameter, 2: bf16 gradient, 4: 8-bit states
    int32_t chunk0;                    // first chunk of this tensor in the launch
    int32_t index;                     // position in the call
    uint32_t key;                      // random bits of (seed, step, index), when the step is known on the host
};

struct AdamwArgs {
    double beta1, beta2;
    float b1, ob1, b2, ob2, eps, inv_bc2, one;     // one: 1, for add2
    uint32_t seed, step;
    const int32_t* step_dev;
    const float* lr_scale;
    const float* grad_scale;
    int32_t* dev_status;
    int32_t count;
};

template <int CAP>
struct AdamwTable {
    AdamwArgs a;
    AdamwEntry e[CAP];
};

__host__ __device__ inline double power(double b, int64_t t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

__host__ __device__ inline uint32_t mix32(uint32_t x)
{
    x ^= x >> 16;
    x *= 0x7A3D95F5u;
    x ^= x >> 15;
    x *= 0x5C6B2E3Bu;
    return x ^ (x >> 16);
}

// Two products or sums in one instruction, each rounded as __fmul_rn and __fadd_rn round.  A sum is a + b * one with a 1
// that the compiler does not know: it contracts a pair's product and sum, which would round once instead of twice.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ void unpair(float& a, float& b, uint64_t v) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b, uint64_t one) { return fma2(a, one, b); }
__device__ __forceinline__ uint64_t both(float a) { return pair(a, a); }
// x[j] = x[j] * s
__device__ __forceinline__ void scale8(float (&x)[8], float s)
{
    const uint64_t t = both(s);
#pragma unroll
    for (int j = 0; j < 8; j += 2) unpair(x[j], x[j + 1], mul2(pair(x[j], x[j + 1]), t));
}

// Eight elements of a lane: 4 lane .. + 3 and 128 + 4 lane .. + 3 of the block.
__device__ __forceinline__ int elem(int lane, int j) { return (j >> 2) * 128 + 4 * lane + (j & 3); }

template <bool BF16>
__device__ __forceinline__ void load8(float (&x)[8], const void* src, int64_t base, int lane, int left)
{
    if constexpr (BF16) {
        const uint16_t* s = static_cast<const uint16_t*>(src) + base;
        if (left >= kBlock) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint2 u = __ldcs(reinterpret_cast<const uint2*>(s + h * 128 + 4 * lane));
                x[4 * h] = bf16_bits_to_f32(u.x & 0xffffu);
                x[4 * h + 1] = __uint_as_float(u.x & 0xffff0000u);
                x[4 * h + 2] = bf16_bits_to_f32(u.y & 0xffffu);
                x[4 * h + 3] = __uint_as_float(u.y & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = elem(lane, j) < left ? bf16_bits_to_f32(s[elem(lane, j)]) : 0.0f;
        }
    } else {
        const float* s = static_cast<const float*>(src) + base;
        if (left >= kBlock) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 u = __ldcs(reinterpret_cast<const float4*>(s + h * 128 + 4 * lane));
                x[4 * h] = u.x; x[4 * h + 1] = u.y; x[4 * h + 2] = u.z; x[4 * h + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = elem(lane, j) < left ? s[elem(lane, j)] : 0.0f;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* dst, const float (&x)[8], int64_t base, int lane, int left)
{
    if constexpr (BF16) {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(dst) + base;
        if (left >= kBlock) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                __nv_bfloat162 a = __floats2bfloat162_rn(x[4 * h], x[4 * h + 1]);
                __nv_bfloat162 b = __floats2bfloat162_rn(x[4 * h + 2], x[4 * h + 3]);
                uint2 u;
                u.x = *reinterpret_cast<uint32_t*>(&a);
                u.y = *reinterpret_cast<uint32_t*>(&b);
                __stcs(reinterpret_cast<uint2*>(d + h * 128 + 4 * lane), u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (elem(lane, j) < left) d[elem(lane, j)] = __float2bfloat16_rn(x[j]);
        }
    } else {
        float* d = static_cast<float*>(dst) + base;
        if (left >= kBlock) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                __stcs(reinterpret_cast<float4*>(d + h * 128 + 4 * lane),
                       make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (elem(lane, j) < left) d[elem(lane, j)] = x[j];
        }
    }
}

__device__ __forceinline__ void load_codes(uint32_t (&c)[2], const void* src, int64_t base, int lane, int left)
{
    const uint8_t* s = static_cast<const uint8_t*>(src) + base;
    if (left >= kBlock) {
#pragma unroll
        for (int h = 0; h < 2; ++h) c[h] = __ldcs(reinterpret_cast<const uint32_t*>(s + h * 128 + 4 * lane));
    } else {
        c[0] = c[1] = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (elem(lane, j) < left) c[j >> 2] |= (uint32_t)s[elem(lane, j)] << (8 * (j & 3));
    }
}

__device__ __forceinline__ void store_codes(void* dst, const uint32_t (&c)[2], int64_t base, int lane, int left)
{
    uint8_t* d = static_cast<uint8_t*>(dst) + base;
    if (left >= kBlock) {
#pragma unroll
        for (int h = 0; h < 2; ++h) __stcs(reinterpret_cast<uint32_t*>(d + h * 128 + 4 * lane), c[h]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (elem(lane, j) < left) d[elem(lane, j)] = (uint8_t)(c[j >> 2] >> (8 * (j & 3)));
    }
}

__device__ __forceinline__ void decode(float (&x)[8], const uint32_t (&c)[2], float scale)
{
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        const __half2_raw r =
            __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(r));
        x[2 * h] = f.x;
        x[2 * h + 1] = f.y;
    }
    scale8(x, scale);
}

__device__ __forceinline__ void encode(uint32_t (&c)[2], const float (&y)[8])
{
    c[0] = c[1] = 0;
#pragma unroll
    for (int h = 0; h < 4; ++h)
        c[h >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y[2 * h], y[2 * h + 1]), __NV_SATFINITE, __NV_E4M3)
                     << (16 * (h & 1));
}

// Largest magnitude of the warp's block (NaN ignored), 0 below kTiny.
__device__ __forceinline__ float block_top(const float (&x)[8])
{
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) t = fmaxf(t, fabsf(x[j]));
#pragma unroll
    for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
    return t < kTiny ? 0.0f : t;
}

// Up to the next e4m3 code with the chance of the remainder: adding 20 random
// bits below the three kept mantissa bits and cutting them off.  Below 2^-6 the
// codes are evenly spaced; 2^-6 more puts them into the binade of that spacing.
// What is above 0 becomes code 1 (2^-9) at least; NaN, which the random bits would carry into a zero,
// stays (45 M elements, in a graph: 126.9 us; 125.7 without that, 129.6 where a maximum of the block's looks for it).
__device__ __forceinline__ float stochastic_e4m3(float y, uint32_t rnd20)
{
    y = fmaxf(y, y > 0.0f ? 0x1p-9f : y);
    const float lift = y < 0x1p-6f ? 0x1p-6f : 0.0f;
    const float z = __uint_as_float((__float_as_uint(__fadd_rn(y, lift)) + rnd20) & 0xfff00000u) - lift;
    return y == y ? fminf(z, kE4m3Max) : y;
}

// a / b within two units of the last place: the update is a small part of p, whose own rounding
// hides that.  (The fast quotient is 0 for b past 2^126, which no root of an fp32 number reaches.)
__device__ __forceinline__ float quotient(float a, float b) { return __fdividef(a, b); }

template <int KIND>
__device__ __forceinline__ void adamw_block(const AdamwEntry& e, const AdamwArgs& a, int64_t blk, int lane,
                                            float step_size, float decay, float inv_bc2, float gscale,
                                            uint32_t key, bool& bad)
{
    constexpr bool kP16 = (KIND & 1) != 0, kG16 = (KIND & 2) != 0, kS8 = (KIND & 4) != 0;
    const int64_t base = blk * kBlock;
    const int left = (int)min((int64_t)kBlock, e.n - base);
    float p[8], g[8], m[8], v[8];
    load8<kG16>(g, e.g, base, lane, left);
    load8<kP16>(p, e.p, base, lane, left);
    if constexpr (kS8) {
        uint32_t cm[2], cv[2];
        load_codes(cm, e.m, base, lane, left);
        load_codes(cv, e.v, base, lane, left);
        decode(m, cm, e.ms[blk]);
        decode(v, cv, e.vs[blk]);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const uint64_t t = pair(v[j], v[j + 1]);
            unpair(v[j], v[j + 1], mul2(t, t));
        }
    } else {
        load8<false>(m, e.m, base, lane, left);
        load8<false>(v, e.v, base, lane, left);
    }
    float r[8];
    const uint64_t one = both(a.one);
    uint64_t odd = 0;                              // 0 times every gradient: NaN once one is not finite
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint64_t gj = mul2(pair(g[j], g[j + 1]), both(gscale));
        odd = fma2(gj, 0, odd);
        const uint64_t mj = add2(mul2(pair(m[j], m[j + 1]), both(a.b1)), mul2(gj, both(a.ob1)), one);
        const uint64_t vj = add2(mul2(pair(v[j], v[j + 1]), both(a.b2)), mul2(mul2(gj, gj), both(a.ob2)), one);
        unpair(m[j], m[j + 1], mj);
        unpair(v[j], v[j + 1], vj);
        r[j] = __fsqrt_rn(v[j]);
        r[j + 1] = __fsqrt_rn(v[j + 1]);
        float n0, n1, d0, d1;
        unpair(n0, n1, mul2(mj, both(-step_size)));
        unpair(d0, d1, add2(mul2(pair(r[j], r[j + 1]), both(inv_bc2)), both(a.eps), one));
        unpair(p[j], p[j + 1], add2(mul2(pair(p[j], p[j + 1]), both(decay)), pair(quotient(n0, d0), quotient(n1, d1)), one));
    }
    {
        float o0, o1;
        unpair(o0, o1, odd);
        bad |= o0 != o0 || o1 != o1;
    }
    store8<kP16>(e.p, p, base, lane, left);
    if constexpr (kS8) {
        uint32_t c[2];
        float y[8];
        const float tm = block_top(m);
        const float im = tm > 0.0f ? __fmul_rn(__frcp_rn(tm), kE4m3Max) : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = m[j];
        scale8(y, im);
        encode(c, y);
        store_codes(e.m, c, base, lane, left);
        const float tr = block_top(r);
        const float ir = tr > 0.0f ? __fmul_rn(__frcp_rn(tr), kE4m3Max) : 0.0f;
        key = mix32(key + (uint32_t)blk);
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = r[j];
        scale8(y, ir);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            y[j] = stochastic_e4m3(y[j], mix32(key + (uint32_t)elem(lane, j) * 0x9E3779B1u) >> 12);
        encode(c, y);
        store_codes(e.v, c, base, lane, left);
        if (lane == 0) {
            e.ms[blk] = __fmul_rn(tm, 1.0f / kE4m3Max);
            e.vs[blk] = __fmul_rn(tr, 1.0f / kE4m3Max);
        }
    } else {
        store8<false>(e.m, m, base, lane, left);
        store8<false>(e.v, v, base, lane, left);
    }
}

template <int CAP, bool S8>
__global__ void __launch_bounds__(kWarps * 32, 5)
adamw_kernel(const __grid_constant__ AdamwTable<CAP> t)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = t.a.count - 1;                 // the tensor whose chunks include this CTA's
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.e[mid].chunk0 <= (int)blockIdx.x) lo = mid;
        else hi = mid - 1;
    }
    const AdamwEntry& e = t.e[lo];
    pdl_launch_dependents();
    pdl_wait();
    float step_size = e.step_size, decay = e.decay, inv_bc2 = t.a.inv_bc2;
    uint32_t key = e.key;                           // random bits of this tensor and step
    if (t.a.step_dev || t.a.lr_scale) {             // known on the device only
        __shared__ float s[3];
        const uint32_t step = t.a.step_dev ? (uint32_t)*t.a.step_dev : t.a.step;
        key = mix32(mix32(mix32(t.a.seed) + step) + (uint32_t)e.index);
        if (threadIdx.x == 0) {
            const double lr = t.a.lr_scale ? e.lr * (double)*t.a.lr_scale : e.lr;
            s[0] = (float)(lr / (1.0 - power(t.a.beta1, step)));
            s[1] = (float)(1.0 - lr * e.wd);
            s[2] = (float)(1.0 / sqrt(1.0 - power(t.a.beta2, step)));
        }
        __syncthreads();
        step_size = s[0];
        decay = s[1];
        inv_bc2 = s[2];
    }
    const float gscale = t.a.grad_scale ? *t.a.grad_scale : 1.0f;
    const int64_t nblk = (e.n + kBlock - 1) / kBlock;
    const int64_t blk = (int64_t)((int)blockIdx.x - e.chunk0) * kWarps + warp;
    if (blk >= nblk) return;
    bool bad = false;
    constexpr int K0 = S8 ? 4 : 0;
    switch (e.kind & 3) {
        case 0: adamw_block<K0>(e, t.a, blk, lane, step_size, decay, inv_bc2, gscale, key, bad); break;
        case 1: adamw_block<K0 + 1>(e, t.a, blk, lane, step_size, decay, inv_bc2, gscale, key, bad); break;
        case 2: adamw_block<K0 + 2>(e, t.a, blk, lane, step_size, decay, inv_bc2, gscale, key, bad); break;
        default: adamw_block<K0 + 3>(e, t.a, blk, lane, step_size, decay, inv_bc2, gscale, key, bad); break;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_dev_status(t.a.dev_status, RB_DEV_NONFINITE);
}

// ---------------------------------------------------------------- host side
constexpr int kSmallCap = 16, kLargeCap = 128;    // tensors per launch: the table is a kernel argument

struct Range {
    uintptr_t lo, hi;
};

bool good_dtype(int d) { return d == RB_F32 || d == RB_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
int elem_bytes(int dtype) { return dtype == RB_BF16 ? 2 : 4; }

rb_status check_tensor(const rb_adamw_tensor_t& t)
{
    if (t.n < 0 || t.reserved != 0) return RB_ERR_ARG;
    if (!good_dtype(t.param_dtype) || !good_dtype(t.grad_dtype)) return RB_ERR_ARG;
    if (t.state_bits != 32 && t.state_bits != 8) return RB_ERR_ARG;
    if (!(t.lr >= 0.0) || !std::isfinite(t.lr) || !std::isfinite(t.weight_decay)) return RB_ERR_ARG;
    if (t.n == 0) return RB_OK;
    if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return RB_ERR_ARG;
    if (t.state_bits == 8 && (!t.exp_avg_scale || !t.exp_avg_sq_scale)) return RB_ERR_ARG;
    if (t.n > (int64_t)1 << 40) return RB_ERR_SHAPE;
    if (!aligned16(t.param) || !aligned16(t.grad) || !aligned16(t.exp_avg) || !aligned16(t.exp_avg_sq))
        return RB_ERR_ALIGN;
    if (t.state_bits == 8 && (!aligned4(t.exp_avg_scale) || !aligned4(t.exp_avg_sq_scale))) return RB_ERR_ALIGN;
    return RB_OK;
}

Range range_of(const void* p, int64_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{a, a + (uintptr_t)bytes};
}

bool gradient_overlaps(const rb_adamw_tensor_t& t)
{
    if (t.n == 0) return false;
    const Range g = range_of(t.grad, t.n * elem_bytes(t.grad_dtype));
    auto over = [&](const void* p, int64_t bytes) {
        const Range o = range_of(p, bytes);
        return g.lo < o.hi && o.lo < g.hi;
    };
    const int64_t state = t.n * (t.state_bits / 8), scales = (t.n + kBlock - 1) / kBlock * 4;
    return over(t.param, t.n * elem_bytes(t.param_dtype)) || over(t.exp_avg, state) || over(t.exp_avg_sq, state) ||
           (t.state_bits == 8 && (over(t.exp_avg_scale, scales) || over(t.exp_avg_sq_scale, scales)));
}

// What the tensors of one launch write must not overlap (they would race).  Five lists: parameters, both
// moments, both scales.  Where each is in order and their extents are apart, as with states kept in
// buffers of their own, nothing is sorted; and where the gradients' extent is apart from them, no
// gradient is looked at by itself.
bool launch_overlaps(const rb_adamw_tensor_t* t, int n)
{
    Range r[5 * kLargeCap];
    int c = 0, from[6] = {};
    bool plain = true;
    Range g = {UINTPTR_MAX, 0};
    for (int i = 0; i < n; ++i) {
        if (t[i].n == 0) continue;
        const Range x = range_of(t[i].grad, t[i].n * elem_bytes(t[i].grad_dtype));
        g.lo = std::min(g.lo, x.lo);
        g.hi = std::max(g.hi, x.hi);
    }
    for (int k = 0; k < 5; ++k) {
        for (int i = 0; i < n; ++i) {
            if (t[i].n == 0 || (k >= 3 && t[i].state_bits != 8)) continue;
            const int64_t scales = (t[i].n + kBlock - 1) / kBlock * 4;
            r[c] = k == 0   ? range_of(t[i].param, t[i].n * elem_bytes(t[i].param_dtype))
                   : k == 1 ? range_of(t[i].exp_avg, t[i].n * (t[i].state_bits / 8))
                   : k == 2 ? range_of(t[i].exp_avg_sq, t[i].n * (t[i].state_bits / 8))
                   : k == 3 ? range_of(t[i].exp_avg_scale, scales)
                            : range_of(t[i].exp_avg_sq_scale, scales);
            plain &= c == from[k] || r[c - 1].hi <= r[c].lo;
            ++c;
        }
        from[k + 1] = c;
        for (int j = 0; j < k && plain; ++j)       // this list's extent against the earlier ones'
            if (from[j] < from[j + 1] && from[k] < c)
                plain = r[c - 1].hi <= r[from[j]].lo || r[from[j + 1] - 1].hi <= r[from[k]].lo;
    }
    bool apart = plain;
    for (int k = 0; k < 5 && apart; ++k)
        if (from[k] < from[k + 1]) apart = g.hi <= r[from[k]].lo || r[from[k + 1] - 1].hi <= g.lo;
    for (int i = 0; i < n && !apart; ++i)
        if (gradient_overlaps(t[i])) return true;
    if (plain) return false;
    std::sort(r, r + c, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    for (int i = 1; i < c; ++i)
        if (r[i].lo < r[i - 1].hi) return true;
    return false;
}

template <int CAP, bool S8>
rb_status launch_group(const rb_adamw_tensor_t* t, int first, int n, const AdamwArgs& base, double bc1, bool pdl,
                       cudaStream_t stream)
{
    AdamwTable<CAP> tab;
    tab.a = base;
    int c = 0;
    int64_t chunks = 0;
    for (int i = first; i < first + n; ++i) {
        if (t[i].n == 0 || (t[i].state_bits == 8) != S8) continue;
        AdamwEntry& e = tab.e[c++];
        e.n = t[i].n;
        e.p = t[i].param;
        e.g = t[i].grad;
        e.m = t[i].exp_avg;
        e.v = t[i].exp_avg_sq;
        e.ms = t[i].exp_avg_scale;
        e.vs = t[i].exp_avg_sq_scale;
        e.lr = t[i].lr;
        e.wd = t[i].weight_decay;
        e.step_size = (float)(t[i].lr / bc1);
        e.decay = (float)(1.0 - t[i].lr * t[i].weight_decay);
        e.kind = (t[i].param_dtype == RB_BF16 ? 1 : 0) | (t[i].grad_dtype == RB_BF16 ? 2 : 0) |
                 (t[i].state_bits == 8 ? 4 : 0);
        e.chunk0 = (int32_t)chunks;
        e.index = i;
        e.key = mix32(mix32(mix32(base.seed) + base.step) + (uint32_t)i);
        chunks += (t[i].n + kChunk - 1) / kChunk;
    }
    if (c == 0) return RB_OK;
    tab.a.count = c;
    cudaLaunchConfig_t cfg = {};                // the table is up to 12 KB: passed by address, copied once
    cfg.gridDim = dim3((unsigned)chunks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    void* args[] = {&tab};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&adamw_kernel<CAP, S8>), args) == cudaSuccess
               ? RB_OK : RB_ERR_CUDA;
}

}  // namespace
}  // namespace rbw

using namespace rbw;

extern "C" rb_status rb_adamw_step(const rb_adamw_tensor_t* tensors, int count, const rb_adamw_t* hyper,
                                   int32_t* dev_status, unsigned flags, cudaStream_t stream)
{
    if (!tensors || !hyper || count < 1 || (flags & ~RB_LAUNCH_PDL)) return RB_ERR_ARG;
    if (!(hyper->beta1 >= 0.0 && hyper->beta1 < 1.0) || !(hyper->beta2 >= 0.0 && hyper->beta2 < 1.0)) return RB_ERR_ARG;
    if (!(hyper->eps >= 0.0) || !std::isfinite(hyper->eps) || hyper->reserved != 0) return RB_ERR_ARG;
    if (!hyper->step_dev && (hyper->step < 1 || hyper->step > INT32_MAX)) return RB_ERR_ARG;
    if (!aligned4(hyper->step_dev) || !aligned4(hyper->lr_scale) || !aligned4(hyper->grad_scale)) return RB_ERR_ALIGN;
    if (dev_status && !aligned16(dev_status)) return RB_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {
        const rb_status st = check_tensor(tensors[i]);
        if (st != RB_OK) return st;
    }
    // Launches of up to kLargeCap tensors and fewer than 2^31 chunks; a whole
    // call is checked before the first is made.
    int64_t chunks = 0;
    for (int first = 0, n = 0; first < count; first += n) {
        for (n = 0, chunks = 0; n < kLargeCap && first + n < count; ++n) {
            const int64_t c = (tensors[first + n].n + kChunk - 1) / kChunk;
            if (n && chunks + c > INT32_MAX) break;
            chunks += c;
        }
        if (launch_overlaps(tensors + first, n)) return RB_ERR_ARG;
    }
    if (!device_is_sm100()) return RB_ERR_UNSUPPORTED;
    AdamwArgs a = {};
    a.beta1 = hyper->beta1;
    a.beta2 = hyper->beta2;
    a.b1 = (float)hyper->beta1;
    a.ob1 = (float)(1.0 - hyper->beta1);
    a.b2 = (float)hyper->beta2;
    a.ob2 = (float)(1.0 - hyper->beta2);
    a.eps = (float)hyper->eps;
    a.one = 1.0f;
    a.seed = hyper->seed;
    a.step = (uint32_t)hyper->step;
    a.step_dev = hyper->step_dev;
    a.lr_scale = hyper->lr_scale;
    a.grad_scale = hyper->grad_scale;
    a.dev_status = dev_status;
    const double bc1 = hyper->step_dev ? 1.0 : 1.0 - power(hyper->beta1, hyper->step);
    a.inv_bc2 = hyper->step_dev ? 1.0f : (float)(1.0 / std::sqrt(1.0 - power(hyper->beta2, hyper->step)));
    const bool pdl = (flags & RB_LAUNCH_PDL) != 0;
    for (int first = 0, n = 0; first < count; first += n) {
        for (n = 0, chunks = 0; n < kLargeCap && first + n < count; ++n) {
            const int64_t c = (tensors[first + n].n + kChunk - 1) / kChunk;
            if (n && chunks + c > INT32_MAX) break;
            chunks += c;
        }
        rb_status st = n <= kSmallCap ? launch_group<kSmallCap, false>(tensors, first, n, a, bc1, pdl, stream)
                                      : launch_group<kLargeCap, false>(tensors, first, n, a, bc1, pdl, stream);
        if (st != RB_OK) return st;
        st = n <= kSmallCap ? launch_group<kSmallCap, true>(tensors, first, n, a, bc1, pdl, stream)
                            : launch_group<kLargeCap, true>(tensors, first, n, a, bc1, pdl, stream);
        if (st != RB_OK) return st;
    }
    return RB_OK;
}
