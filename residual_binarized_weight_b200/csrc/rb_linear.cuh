// rb_linear.cuh -- what the two kernels of the linear product share: the
// conversion of X, the epilogue on eight columns of a token, tensor maps.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "rb_epilogue.cuh"
#include "rb_tcgen05.cuh"

namespace rbw {
namespace {

struct LinEp {
    const float* bias;
    const uint16_t* mul;
    const void* res;
    uint16_t* pre;
    void* Y;
    int64_t ld_mul, ld_res, ld_pre, ld_y;
    int act, res_bf16, y_bf16;
    const float* xs;                           // [M] what a token's accumulators are multiplied by (X in fp16, below)
    int vec;                                   // 1, 2, 4, 8: rows of mul, residual, preact, Y start on 16 bytes
};

// ---------------------------------------------------------------- waits of a whole warp
// Bounded as mbar_wait (rb_tcgen05.cuh), but every lane waits, in steps of up to 10 us that the
// hardware sleeps through: a polling warp would take issue slots from the warps that expand the
// weights, and a loop that only one lane runs keeps the MMA operands out of the uniform registers
// (16 tokens: 900 to 1000 cycles from one k-block's MMAs to the next's, 600 with the whole warp in the loop).
__device__ __forceinline__ bool try_wait_asleep(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.b32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(bar), "r"(parity), "r"(10000u) : "memory");
    return ok != 0;
}
// IDLE: a wait that may be late (a ring's refill), with a pause between the looks.
template <bool IDLE = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* dev_status)
{
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
    if (__all_sync(0xffffffffu, try_wait_asleep(bar, parity))) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (IDLE) __nanosleep(100);
        if (__all_sync(0xffffffffu, try_wait_asleep(bar, parity))) return true;
        if ((it & 15u) == 0u) {
            const bool late = globaltimer_ns() - t0 > kTimeoutNs;
            const bool told = *abort_flag || (dev_status && (*reinterpret_cast<volatile int32_t*>(dev_status) & RB_DEV_TIMEOUT));
            if (__any_sync(0xffffffffu, late || told)) {
                *abort_flag = 1;
                set_dev_status(dev_status, RB_DEV_TIMEOUT);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ---------------------------------------------------------------- X in fp16
// X16[m][32 q + 2 j + e] = fp16(X[m][32 q + j + 16 e] 2^s),   xs[m] = 2^-s,
// s by row, so that its largest value comes to lie in [2^14, 2^15): a token's accumulators times xs are its products,
// exactly, and gradients of 1e-9 or outliers of 1e6 lose nothing against values of 1.  A value keeps all its bits
// down to 2^-31 of the row's largest, and is off by at most 2^-39 of that below.  A row with an infinity or NaN,
// of which no product is finite, takes the smallest s.
//
// T of a CTA's B threads take a row, with H vectors of eight columns each in flight; of a row longer than those
// (K > 16384) the second look comes from L2.  In a vector's group of four lanes (32 columns), a lane and its neighbour
// two further on exchange half of theirs.
__device__ __forceinline__ uint32_t scaled_f16x2(uint32_t v, float s)
{
    const __half2 h = __floats2half2_rn(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint4 interleave(const uint4& in, int lane, float s)
{
    const uint32_t c0 = scaled_f16x2(in.x, s), c1 = scaled_f16x2(in.y, s);
    const uint32_t c2 = scaled_f16x2(in.z, s), c3 = scaled_f16x2(in.w, s);
    const bool hi = lane & 2;                  // columns 16.. of the group
    const uint32_t p0 = __shfl_xor_sync(0xffffffffu, hi ? c0 : c2, 2);
    const uint32_t p1 = __shfl_xor_sync(0xffffffffu, hi ? c1 : c3, 2);
    const uint32_t a0 = hi ? p0 : c0, a1 = hi ? p1 : c1, b0 = hi ? c2 : p0, b1 = hi ? c3 : p1;
    return make_uint4(prmt(a0, b0, 0x5410), prmt(a0, b0, 0x7632), prmt(a1, b1, 0x5410), prmt(a1, b1, 0x7632));
}

constexpr uint32_t kOverF16 = 0x4780u, kInfBf16 = 0x7f80u;     // bf16 65536, the first that fp16 has not, and infinity
__device__ __forceinline__ bool any_over(const uint4& v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    bool r = false;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        r |= (w[q] & 0x7fffu) - kOverF16 <= kInfBf16 - kOverF16 || ((w[q] >> 16) & 0x7fffu) - kOverF16 <= kInfBf16 - kOverF16;
    return r;
}

template <int B, int T, int H>
__device__ __forceinline__ void convert_rows(const uint16_t* __restrict__ X, int64_t ldx, int M, int K, int block, int blocks,
                                             uint16_t* __restrict__ X16, float* __restrict__ xs, bool& range)
{
    __shared__ uint32_t tops[B / 32];
    constexpr int R = B / T, W = T / 32;     // rows per CTA, warps per row
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tr = threadIdx.x % T, vecs = K / 8;   // vecs: a multiple of 4
    for (int64_t m0 = (int64_t)block * R; m0 < M; m0 += (int64_t)blocks * R) {
        const int64_t m = m0 + threadIdx.x / T;
        const int mine = m < M ? vecs : 0;
        const uint16_t* src = X + m * ldx;
        uint4 in[H];
        auto load = [&](int b) {
#pragma unroll
            for (int u = 0; u < H; ++u) {
                const int v = b + u * T + tr;
                in[u] = v < mine ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)v * 8)) : make_uint4(0, 0, 0, 0);
            }
        };
        uint32_t two = 0;                      // the largest |bf16|, of even and of odd columns
        for (int b = 0; b < vecs; b += T * H) {
            load(b);
#pragma unroll
            for (int u = 0; u < H; ++u) {
                two = __vmaxu2(two, __vmaxu2(in[u].x & 0x7fff7fffu, in[u].y & 0x7fff7fffu));
                two = __vmaxu2(two, __vmaxu2(in[u].z & 0x7fff7fffu, in[u].w & 0x7fff7fffu));
            }
        }
        uint32_t top = __reduce_max_sync(0xffffffffu, max(two & 0xffffu, two >> 16));
        if constexpr (W > 1) {
            __syncthreads();                   // the row before has been read
            if (lane == 0) tops[warp] = top;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < W; ++w) top = max(top, tops[warp / W * W + w]);
        }
        // biased exponents: 2^s brings the largest's to 127 + 14; 2^127 at most (values below 2^-113)
        const uint32_t up = min(268u - min(top >> 7, 254u), 254u), down = 254u - up;
        const float s = __uint_as_float(up << 23);
        if (tr == 0 && m < M) xs[m] = __uint_as_float(down ? down << 23 : 0x00400000u);
        const bool nan = top > kInfBf16;       // (hides what else there is)
        range |= top >= kOverF16 && !nan;
        for (int b = 0; b < vecs; b += T * H) {
            if (vecs > T * H) load(b);
#pragma unroll
            for (int u = 0; u < H; ++u) {
                if (nan) range |= any_over(in[u]);
                const uint4 o = interleave(in[u], lane, s);
                const int v = b + u * T + tr;
                if (v < mine)                  // lanes 0, 2, 1, 3 of four hold cells 0-3, 4-7, 8-11, 12-15
                    *reinterpret_cast<uint4*>(X16 + m * K + (int64_t)((v & ~3) | ((v >> 1) & 1) | ((v & 1) << 1)) * 8) = o;
            }
        }
    }
}

inline size_t x16_bytes(int M, int K) { return ((size_t)M * K * 2 + 255) / 256 * 256; }
inline size_t xs_bytes(int M) { return ((size_t)M * 4 + 255) / 256 * 256; }

// ---------------------------------------------------------------- epilogue
template <int ACT, int CNT>
__device__ __forceinline__ void act_all(float (&y)[CNT])
{
#pragma unroll
    for (int e = 0; e < CNT; ++e) y[e] = activate<ACT>(y[e]);
}
template <int CNT>
__device__ __forceinline__ void act_switch(int act, float (&y)[CNT])
{
    switch (act) {
        case RB_ACT_RELU: act_all<RB_ACT_RELU>(y); break;
        case RB_ACT_SILU: act_all<RB_ACT_SILU>(y); break;
        case RB_ACT_GELU: act_all<RB_ACT_GELU>(y); break;
        case RB_ACT_GELU_TANH: act_all<RB_ACT_GELU_TANH>(y); break;
        default: break;
    }
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight columns n .. n + 7 of token m (n a multiple of 8); cnt of them exist.
// Vector accesses where the row's stride keeps them on 16 bytes (ep.vec).
struct Eight {
    uint4 mul;
    uint4 res[2];
};
// Addresses of element (m, n) in the epilogue's arrays, and what a number of tokens further is, in bytes.
struct EpAt {
    const char* mul;
    const char* res;
    char* pre;
    char* y;
};
struct EpStep {
    int64_t mul, res, pre, y;
};
__device__ __forceinline__ EpAt ep_at(const LinEp& ep, int64_t m, int64_t n)
{
    EpAt p;
    p.mul = reinterpret_cast<const char*>(ep.mul) + (m * ep.ld_mul + n) * 2;
    p.res = static_cast<const char*>(ep.res) + (m * ep.ld_res + n) * (ep.res_bf16 ? 2 : 4);
    p.pre = reinterpret_cast<char*>(ep.pre) + (m * ep.ld_pre + n) * 2;
    p.y = static_cast<char*>(ep.Y) + (m * ep.ld_y + n) * (ep.y_bf16 ? 2 : 4);
    return p;
}
__device__ __forceinline__ EpStep ep_tokens(const LinEp& ep, int tokens)
{
    return EpStep{tokens * ep.ld_mul * 2, tokens * ep.ld_res * (ep.res_bf16 ? 2 : 4), tokens * ep.ld_pre * 2,
                  tokens * ep.ld_y * (ep.y_bf16 ? 2 : 4)};
}
__device__ __forceinline__ EpAt ep_down(const EpAt& p, const EpStep& s)
{
    return EpAt{p.mul + s.mul, p.res + s.res, p.pre + s.pre, p.y + s.y};
}
__device__ __forceinline__ EpAt ep_right(const LinEp& ep, const EpAt& p, int columns)
{
    return EpAt{p.mul + columns * 2, p.res + columns * (ep.res_bf16 ? 2 : 4), p.pre + columns * 2,
                p.y + columns * (ep.y_bf16 ? 2 : 4)};
}

__device__ __forceinline__ uint4 fetch_bf16(const char* at, bool vec, int cnt)
{
    if (vec && cnt == 8) return *reinterpret_cast<const uint4*>(at);
    const uint16_t* p = reinterpret_cast<const uint16_t*>(at);
    uint32_t w[4] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < cnt) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void ep_fetch(const LinEp& ep, const EpAt& at, int cnt, Eight& f)
{
    if (ep.mul) f.mul = fetch_bf16(at.mul, ep.vec & 1, cnt);
    if (ep.res) {
        if (ep.res_bf16) {
            f.res[0] = fetch_bf16(at.res, ep.vec & 2, cnt);
        } else if ((ep.vec & 2) && cnt == 8) {
            f.res[0] = reinterpret_cast<const uint4*>(at.res)[0];
            f.res[1] = reinterpret_cast<const uint4*>(at.res)[1];
        } else {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(at.res);
            uint32_t w[8] = {};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < cnt) w[e] = p[e];
            f.res[0] = make_uint4(w[0], w[1], w[2], w[3]);
            f.res[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
}

__device__ __forceinline__ void store_bf16(char* at, bool vec, int cnt, const float (&y)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = pack_bf16(y[2 * q], y[2 * q + 1]);
    if (vec && cnt == 8) {
        *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(at);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// y: P of the eight columns
__device__ __forceinline__ void ep_finish(const LinEp& ep, const EpAt& at, int cnt, const Eight& f, float (&y)[8])
{
    if (ep.pre) store_bf16(at.pre, ep.vec & 4, cnt, y);
    act_switch(ep.act, y);
    if (ep.mul) {
        const uint32_t w[4] = {f.mul.x, f.mul.y, f.mul.z, f.mul.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            y[2 * q] *= __uint_as_float(w[q] << 16);
            y[2 * q + 1] *= __uint_as_float(w[q] & 0xffff0000u);
        }
    }
    if (ep.res) {
        if (ep.res_bf16) {
            const uint32_t w[4] = {f.res[0].x, f.res[0].y, f.res[0].z, f.res[0].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                y[2 * q] += __uint_as_float(w[q] << 16);
                y[2 * q + 1] += __uint_as_float(w[q] & 0xffff0000u);
            }
        } else {
            const uint32_t w[8] = {f.res[0].x, f.res[0].y, f.res[0].z, f.res[0].w,
                                   f.res[1].x, f.res[1].y, f.res[1].z, f.res[1].w};
#pragma unroll
            for (int q = 0; q < 8; ++q) y[q] += __uint_as_float(w[q]);
        }
    }
    if (ep.y_bf16) {
        store_bf16(at.y, ep.vec & 8, cnt, y);
    } else if ((ep.vec & 8) && cnt == 8) {
        reinterpret_cast<float4*>(at.y)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4*>(at.y)[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        float* p = reinterpret_cast<float*>(at.y);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < cnt) p[e] = y[e];
    }
}

// Rows that start anywhere: one column per lane, R tokens of it, so that a warp's accesses are consecutive.
// `at`: the first token's place; the first `tokens` of the R exist.
__device__ __forceinline__ bool ep_vectors(const LinEp& ep)
{
    const int need = (ep.mul ? 1 : 0) | (ep.res ? 2 : 0) | (ep.pre ? 4 : 0) | 8;
    return (ep.vec & need) == need;
}
template <int R>
struct Column {
    uint16_t mul[R];
    uint32_t res[R];
};
template <int R>
__device__ __forceinline__ void ep_fetch_column(const LinEp& ep, const EpAt& at, int tokens, Column<R>& f)
{
    if (ep.mul) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(at.mul);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_mul)
            if (j < tokens) f.mul[j] = *p;
    }
    if (ep.res && ep.res_bf16) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(at.res);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_res)
            if (j < tokens) f.res[j] = *p;
    } else if (ep.res) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(at.res);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_res)
            if (j < tokens) f.res[j] = *p;
    }
}
// y: P
template <int R>
__device__ __forceinline__ void ep_finish_column(const LinEp& ep, const EpAt& at, int tokens, const Column<R>& f, float (&y)[R])
{
    if (ep.pre) {
        uint16_t* p = reinterpret_cast<uint16_t*>(at.pre);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_pre)
            if (j < tokens) *p = __bfloat16_as_ushort(__float2bfloat16_rn(y[j]));
    }
    act_switch(ep.act, y);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        if (ep.mul) y[j] *= bf16_bits_to_f32(f.mul[j]);
        if (ep.res) y[j] += ep.res_bf16 ? bf16_bits_to_f32(f.res[j]) : __uint_as_float(f.res[j]);
    }
    if (ep.y_bf16) {
        uint16_t* p = reinterpret_cast<uint16_t*>(at.y);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_y)
            if (j < tokens) *p = __bfloat16_as_ushort(__float2bfloat16_rn(y[j]));
    } else {
        float* p = reinterpret_cast<float*>(at.y);
#pragma unroll
        for (int j = 0; j < R; ++j, p += ep.ld_y)
            if (j < tokens) *p = y[j];
    }
}

// ---------------------------------------------------------------- tensor maps
inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cache{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = cache.load(std::memory_order_acquire);
    if (!fn) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess) {
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
            cache.store(fn, std::memory_order_release);
        }
    }
    return fn;
}

// fp16 [rows][K], boxes of 64 columns x `box_rows` rows, 128-byte swizzle
inline bool encode_fp16(CUtensorMap* map, const void* base, int64_t rows, int K, int box_rows)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t gdim[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t gstride[1] = {(cuuint64_t)K * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), gdim, gstride, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// rb_pack's sign planes, with a next launch that may start beside it (rb_pack.cu).
rb_status pack_planes_early(const float* W, const float* g, const float* h, int N, int K, int kp, uint32_t* planes,
                            int32_t* dev_status, bool early, cudaStream_t stream);

// One token on the byte tables of rb_gemv (rb_gemv.cu); `epilogue` is a LinEp.
rb_status lut_linear(const rb_layer_t* L, const uint16_t* X, const void* epilogue, bool pdl, cudaStream_t stream);

// The product on weights expanded to fp16 in the workspace (rb_linear_dense.cu).
struct DenseArgs {
    const uint16_t* X;
    int64_t ldx;
    const uint32_t* planes;
    const uint16_t* g16;
    const uint16_t* h16;
    const float* g32;              // not null: the scales of a training forward, instead of g16 and h16
    const float* h32;
    int N, K, M, kp;
    int32_t* dev_status;
};
struct DensePlan {
    int bn, tiles;                 // rows per tile; 0 tiles: not served
    double cost;                   // SM cycles
};
DensePlan dense_plan(int N, int K, int M);
size_t dense_workspace(int N, int K, int M);
rb_status dense_run(const DenseArgs& d, const void* epilogue, void* workspace, bool pdl, cudaStream_t stream);

}  // namespace rbw
