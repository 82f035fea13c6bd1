// rb_linear.cu -- the binarized linear product with its epilogue (rb_linear,
// rb_qat_linear):
//
//   P = X What^T + bias;  Y = act(P) .* mul + residual,
//   What[n][c] = sum_i g_i[n] B_i[n][c] h_i[c].
//
// The k planes are summed BEFORE the product: each weight becomes one fp16
//   a[n][c] = B_f h_f + sum_{i != f} r_i[n] (B_i[n][c] h_i[c]),   r_i = fp16(g_i / g_f),
// f the row's plane of the largest |g| (k = 1: a = +-h exactly), and the
// accumulator is scaled by g_f[n] in fp32.  That is k times fewer MMAs than one
// product per plane.  The price is a rounding of each ratio and each sum, 2^-11 at
// most of sum_i |r_i h_i| each, random in sign over c; on a dot product of a few
// thousand columns that is about 2^-12 of the result, an eighth of the bf16
// rounding of Y.
//
// A CTA computes 128 output rows x bt tokens (any multiple of 16 up to 256),
// its weights as the MMA's A operand in tensor memory, the tokens as B in shared
// memory, D = 128 lanes x bt columns in tensor memory.
//   warps 0..15 expansion: warp w has rows 32 (w % 4) .. + 31 (one per lane) and
//               k-block w / 4 of each 256-column slice (four of 64 columns); sign
//               words from shared memory (conflict-free in the storage order), h
//               pairs from shared memory (broadcast), tcgen05.st of 16 cells
//               at a time.  Afterwards the epilogue.
//   warp 16     issues the MMAs.
//   warp 17     loads sign words (one thread, bulk copies, 4 KB per plane and slice) and
//               lays out the slice's h as pairs of columns (j, j + 16).  The expansion
//               then need not wait for the pre-pass, which prepared the pairs before (0.5 us
//               of 11.2 for 4096 x 4096, k = 2, 8 tokens; 0.6 of 19.4 for 5003 x 4128, k = 3, 64 tokens;
//               1.1 of 75.6 for 11008 x 4096, k = 2, 777 tokens, in a graph).  It
//               shares a scheduler with expansion warps, so it is kept short: the range
//               is looked at once, on the largest |h|.
//   warp 18     one thread loads X tiles (TMA, 128-byte swizzle), prepared by a pre-pass.
// A pre-pass converts X to fp16, each row at a power of two of its own (rb_linear.cuh), which the
// accumulators take back (0.1 us of 19.0 for 11008 x 4096, 8 tokens, 0.8 of 19.3 for 4096 x 11008, 64 tokens,
// against one conversion for all rows), and each 32-column group interleaved so that columns (j, j + 16) are
// neighbours: then one shift brings the sign bits of a pair to the sign bits of an fp16x2.
//
// Three rings: X (shared memory, up to 8 k-blocks), sign words and h pairs (by slice), and A (tensor memory, 8
// k-blocks).  Two k-blocks make a unit, whose MMAs are issued and whose stages are
// freed together: the issuing warp's bookkeeping costs as much as four narrow MMAs.
// X and A have rings of their own so that the expansion runs ahead while X is still on
// its way.  Every wait is bounded (rb_tcgen05.cuh).
//
// gridDim.z > 1 splits K over a cluster: each CTA pushes its scaled partial rows to
// the rank that owns them, which adds them in rank order (deterministic).
#include <atomic>
#include <cmath>
#include <initializer_list>

#include "rbw_internal.cuh"
#include "rb_epilogue.cuh"
#include "rb_linear.cuh"
#include "rb_tcgen05.cuh"

namespace rbw {
namespace {

constexpr int kBR = 128;                       // output rows per CTA
constexpr int kBK = 64;                        // columns per k-block (128 bytes of fp16)
constexpr int kEW = 16;                        // expansion warps
constexpr int kThreads = 32 * (kEW + 3);
constexpr int kMaxStages = 8;                  // X stages, and A stages
constexpr int kUnitsA = kMaxStages / 2;
constexpr int kMaxWStages = 4;
constexpr int kWBlock = 4096;                  // sign words of 128 rows x 256 columns, one plane
constexpr int kHBlock = 128;                   // h pairs of a k-block, one plane
__host__ __device__ constexpr int w_stage_bytes(int kp) { return kp * (kWBlock + 4 * kHBlock); }
constexpr int kTile = 16 * 36 * 4;             // a warp's transpose tile: 16 tokens x 32 rows (+ 4 pad), fp32
constexpr int kMaxSmem = 227 * 1024;
constexpr int kBarBytes = 320;                // barriers, then at 272 the TMEM address and the abort flag

struct LinArgs {
    const uint32_t* planes;
    const uint16_t* g16;
    const float* g32;                          // not null: the row scales (training forward)
    const uint16_t* h16;
    const float* h32;                          // (training forward)
    float limit;                               // |h| above it is reported: 65504 / k, where the sum of k planes (k = 1: an fp32 scale) may leave fp16
    const uint16_t* X;                         // read by the pre-pass
    int64_t ldx;
    LinEp ep;
    int32_t* dev_status;
    int N, K, M;
    int bt, stages, wstages, kb_per;
};

// ---------------------------------------------------------------- pre-pass
// beside: the launch before this one derives the planes of a training forward, which it does not read: it runs
// beside it, and waits for it only before it ends (2048 x 4096 -> 4096: 97.4 us against 99.1 one after the other).
template <int B, int T, int H>
__global__ void __launch_bounds__(B)
linear_prepass_kernel(const uint16_t* __restrict__ X, int64_t ldx, int M, int K, uint16_t* __restrict__ X16,
                      float* __restrict__ xs, int32_t* dev_status, bool beside)
{
    pdl_launch_dependents();
    if (!beside) pdl_wait();
    bool range = false;
    convert_rows<B, T, H>(X, ldx, M, K, (int)blockIdx.x, (int)gridDim.x, X16, xs, range);
    if (range) set_dev_status(dev_status, RB_DEV_RANGE);
    if (beside) pdl_wait();                    // so that whoever waits for this grid has waited for the planes too
}
template <int B, int T, int H>
rb_status launch_prepass(const LinArgs& a, uint16_t* x16, float* xs, bool pdl, cudaStream_t stream)
{
    const int64_t blocks = ((int64_t)a.M + B / T - 1) / (B / T), most = 8 * 148 * 256 / B;
    return launch(linear_prepass_kernel<B, T, H>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(B), 0, stream, pdl, a.X,
                  a.ldx, a.M, a.K, x16, xs, a.dev_status, a.g32 != nullptr);
}

// ---------------------------------------------------------------- main kernel
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ __half2 as_h2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }

// Shared memory: X stages, W stages (sign words and h pairs of a slice), barriers, the receive area of a K split.
__host__ __device__ inline int rows_per_rank(int ks) { return 8 * ((16 + ks - 1) / ks); }      // at most
__host__ __device__ inline int recv_pitch(int bt) { return bt + 4; }
__host__ __device__ inline int recv_bytes(int bt, int ks) { return ks > 1 ? ks * rows_per_rank(ks) * recv_pitch(bt) * 4 : 0; }
__host__ inline int linear_smem(int kp, int bt, int stages, int wstages, int ks)
{
    int ring = stages * bt * 128;
    if (ring < kEW * kTile) ring = kEW * kTile;                // the transpose tiles reuse it
    return 1024 + ring + wstages * w_stage_bytes(kp) + kBarBytes + recv_bytes(bt, ks);
}

// xs of the sixteen tokens from c on: lane j % 16 holds the jth's.
__device__ __forceinline__ float token_xs(const LinEp& ep, int64_t m0, int c, int tokens, int lane)
{
    return c + (lane & 15) < tokens ? ep.xs[m0 + c + (lane & 15)] : 0.0f;
}

__device__ __forceinline__ void sts128(uint32_t a, const uint4& v)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" :: "r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ bool above(const uint2& v, float limit)     // any of four |fp16| (NaN: no)
{
    const float2 a = __half22float2(as_h2(v.x)), b = __half22float2(as_h2(v.y));
    return fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))) > limit;
}
__device__ __forceinline__ uint2 h_to_fp16(const float4& h)
{
    return make_uint2(as_u32(__floats2half2_rn(h.x, h.y)), as_u32(__floats2half2_rn(h.z, h.w)));
}

// The 16 cells (fp16 pairs) of one 32-column word: the first plane's +-h, and the others' times their ratio.
// (Shifts as multiplications, to take them off the ALU pipe, measured 9 % slower.)
template <int KP>
__device__ __forceinline__ void expand_word(uint32_t (&a)[16], const uint32_t (&w)[KP], const uint32_t (&ratio)[KP],
                                            const uint32_t (&hoff)[KP], uint32_t h)
{
#pragma unroll
    for (int v = 0; v < 4; ++v) {
        uint4 H[KP];
#pragma unroll
        for (int i = 0; i < KP; ++i) H[i] = lds128(h + hoff[i] + v * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int j = 4 * v + e;
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const uint32_t hw = e == 0 ? H[i].x : e == 1 ? H[i].y : e == 2 ? H[i].z : H[i].w;
                const uint32_t sh = lop3_sign(w[i] << (15 - j), hw);
                a[j] = i == 0 ? sh : as_u32(__hfma2(as_h2(ratio[i]), as_h2(sh), as_h2(a[j])));
            }
        }
    }
}
template <int KP>
__device__ __forceinline__ float pl_select(const float (&g)[KP], int i)
{
    float v = g[0];
#pragma unroll
    for (int j = 1; j < KP; ++j) v = i == j ? g[j] : v;
    return v;
}

// Tensor memory: D in columns [0, 256), the A stages of 32 columns from 256 on.
template <int KP>
__global__ void __launch_bounds__(kThreads, 1)
linear_tc_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ LinArgs A)
{
    constexpr uint32_t NC = 512, DC = 256;
    static_assert(DC + kMaxStages * 32 <= NC, "tensor memory");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (sbase - smem_u32(smem_raw));
    const int bt = A.bt, stages = A.stages, units = A.stages / 2, wstages = A.wstages;   // stages: even
    const uint32_t xstage = (uint32_t)bt * 128u;
    uint32_t ring = (uint32_t)stages * xstage;
    if (ring < (uint32_t)(kEW * kTile)) ring = kEW * kTile;
    const uint32_t ws0 = sbase + ring;
    const uint32_t bar0 = ws0 + (uint32_t)(wstages * w_stage_bytes(KP));
    uint8_t* tail = gbase + (bar0 - sbase);
    auto full_x = [&](int u) { return bar0 + 8u * u; };                                     // by unit
    auto full_a = [&](int u) { return bar0 + 8u * (kMaxStages + u); };                      // by unit
    auto empty_a = [&](int u) { return bar0 + 8u * (kMaxStages + kUnitsA + u); };
    auto empty_x = [&](int u) { return bar0 + 8u * (kMaxStages + 2 * kUnitsA + u); };
    auto full_w = [&](int s) { return bar0 + 8u * (2 * kMaxStages + kUnitsA + s); };
    auto empty_w = [&](int s) { return bar0 + 8u * (2 * kMaxStages + kUnitsA + kMaxWStages + s); };
    const bool same_ring = units == kUnitsA;      // X and A stages in step: one barrier frees both
    const uint32_t acc_full = bar0 + 8u * (2 * kMaxStages + kUnitsA + 2 * kMaxWStages);
    static_assert(8 * (2 * kMaxStages + kUnitsA + 2 * kMaxWStages) + 8 <= 272 && kBarBytes >= 280, "barrier area");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + 272);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 276);
    float* recv = reinterpret_cast<float*>(tail + kBarBytes);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n0 = blockIdx.x * kBR, m0 = blockIdx.y * bt;
    const int nkb = (A.K + kBK - 1) / kBK;
    const int ks = (int)gridDim.z, rank = (int)blockIdx.z;
    const int kb0 = rank * A.kb_per;                              // a multiple of 4: whole slices
    const int kb1 = min(kb0 + A.kb_per, nkb);
    const int nloc = kb1 - kb0;                                   // >= 1 (host guarantees)
    const int64_t S = num_slices(A.K), Nt = num_row_tiles(A.N);
    const int64_t tile0 = n0 >> 5;
    const int sl0 = kb0 >> 2, nsl = (nloc + 3) >> 2;

    if (threadIdx.x == 0) {
        for (int u = 0; u < kUnitsA; ++u) {
            mbar_init(full_x(u), 1);
            mbar_init(full_a(u), kEW / 2);
            mbar_init(empty_a(u), 1);
            mbar_init(empty_x(u), 1);
        }
        for (int s = 0; s < kMaxWStages; ++s) {
            mbar_init(full_w(s), 2);              // sign words, h pairs
            mbar_init(empty_w(s), kEW);
        }
        mbar_init(acc_full, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(&tmap_x) : "memory");
    }
    if (warp == kEW) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(NC) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // The next launch may read packed planes before it waits: not while the planes of a training forward, which are
    // derived beside the pre-pass and left for the caller, are still being written.
    if (!A.g32) pdl_launch_dependents();
    if (ks > 1) cluster_arrive();                 // waited for before the first store to a peer

    bool ok = true;
    float scale = 0.0f;                           // of this thread's row
    if (warp == kEW + 1) {
        // ---------------- sign words and h pairs by slice
        const uint32_t wbytes = (uint32_t)(Nt - tile0 < 4 ? Nt - tile0 : 4) * 1024u;
        const int word = lane >> 2, j4 = 4 * (lane & 3);          // this lane's columns: four, and the four 16 further on
        int issued = 0, sw = 0;
        uint32_t wph = 1;                         // of the stage's last release
        __half2 top = __half2half2(__float2half_rn(0.0f)), nan = top;      // the largest |h|, and NaN (of fp32 scales) once there is one
        const uint32_t pair_at = (uint32_t)(KP * kWBlock + ((word >> 1) * KP * 32 + (word & 1) * 16 + j4) * 4);
        const uint32_t* planes = A.planes + block_index(0, sl0, tile0, S, Nt) * 256;
        const int64_t plane = S * Nt * 256;
        if (A.g32) {                              // packed planes do not depend on what ran before
            pdl_wait();
            pdl_launch_dependents();
        }
        for (; issued < nsl; ++issued) {
            const int c = (sl0 + issued) * 256 + word * 32 + j4;
            uint2 lo[KP], hi[KP];
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                lo[i] = hi[i] = make_uint2(0, 0);
                if (c >= A.K) continue;           // K % 32 == 0: the columns 16 further on exist as well
                const int64_t at = (int64_t)i * A.K + c;
                if (A.h32) {
                    lo[i] = h_to_fp16(*reinterpret_cast<const float4*>(A.h32 + at));
                    hi[i] = h_to_fp16(*reinterpret_cast<const float4*>(A.h32 + at + 16));
                } else {
                    lo[i] = *reinterpret_cast<const uint2*>(A.h16 + at);
                    hi[i] = *reinterpret_cast<const uint2*>(A.h16 + at + 16);
                }
            }
            if (issued >= wstages &&
                !wait_warp(empty_w(sw), wph, abort_flag, A.dev_status))
                break;
            const uint32_t stage = ws0 + (uint32_t)(sw * w_stage_bytes(KP));
            if (lane == 0) {
                mbar_arrive_expect_tx(full_w(sw), wbytes * KP);
                for (int i = 0; i < KP; ++i)
                    bulk_load(stage + (uint32_t)(i * kWBlock), planes + i * plane, wbytes, full_w(sw));
            }
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                sts128(stage + pair_at + (uint32_t)(i * 128),
                       make_uint4(prmt(lo[i].x, hi[i].x, 0x5410), prmt(lo[i].x, hi[i].x, 0x7632),
                                  prmt(lo[i].y, hi[i].y, 0x5410), prmt(lo[i].y, hi[i].y, 0x7632)));
                top = __hmax2(__hmax2(top, __habs2(as_h2(lo[i].x))), __habs2(as_h2(lo[i].y)));
                top = __hmax2(__hmax2(top, __habs2(as_h2(hi[i].x))), __habs2(as_h2(hi[i].y)));
                if (A.h32)
                    nan = __hmax2_nan(__hmax2_nan(__hmax2_nan(nan, as_h2(lo[i].x)), __hmax2_nan(as_h2(lo[i].y), as_h2(hi[i].x))),
                                      as_h2(hi[i].y));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full_w(sw));
            planes += Nt * 256;
            if (++sw == wstages) { sw = 0; wph ^= 1u; }
        }
        const int flags = (above(make_uint2(as_u32(top), 0), A.limit) ? RB_DEV_RANGE : 0) |
                          (__hisnan(__low2half(nan)) || __hisnan(__high2half(nan)) ? RB_DEV_NONFINITE : 0);
        if (flags) set_dev_status(A.dev_status, flags);
        if (lane == 0 && *abort_flag) {           // drain the loads this thread issued: they always land
            const uint64_t t0 = globaltimer_ns();
            for (int b = max(issued - wstages, 0); b < issued; ++b)
                mbar_drain(full_w(b % wstages), (b / wstages) & 1, t0);
        }
    } else if (warp == kEW + 2) {
        if (lane == 0) {                          // ---------------- X tiles
            pdl_wait();                           // X16
            int issued = 0, u = 0, j = 0;         // units
            for (int kb = kb0; kb < kb1; kb += 2) {
                if (j > 0 && !mbar_wait(empty_x(u), (j - 1) & 1, abort_flag, A.dev_status, kTimeoutNs)) break;
                const int n = min(kb1 - kb, 2);
                mbar_arrive_expect_tx(full_x(u), (uint32_t)n * xstage);
                for (int i = 0; i < n; ++i)
                    tma_load_2d(sbase + (2 * u + i) * xstage, &tmap_x, full_x(u), (kb + i) * kBK, m0);
                ++issued;
                if (++u == units) { u = 0; ++j; }
            }
            if (*abort_flag) {
                const uint64_t t0 = globaltimer_ns();
                for (int b = max(issued - units, 0); b < issued; ++b) mbar_drain(full_x(b % units), (b / units) & 1, t0);
            }
        }
    } else if (warp == kEW) {
        // ---------------- MMAs: the whole warp runs the loop, one elected lane issues
        const uint32_t idesc = (1u << 4) | ((uint32_t)(bt >> 3) << 17) | ((uint32_t)(kBR >> 4) << 24);
        const uint64_t bd0 = smem_desc_sw128(sbase);
        int ux = 0, ua = 0;                       // the unit's place in the two rings
        uint32_t px = 0, pa = 0;
        for (int it = 0; it < nloc; it += 2) {
            if (!wait_warp(full_x(ux), px, abort_flag, A.dev_status)) break;
            if (!wait_warp(full_a(ua), pa, abort_flag, A.dev_status)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t bd = bd0 + (uint32_t)(2 * ux * (xstage >> 4));
                const uint32_t at = tmem + DC + (uint32_t)(2 * ua * 32);
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk)
                    tc_mma_f16_ts(tmem, at + kk * 8, bd + kk * 2, idesc, (it > 0 || kk > 0) ? 1u : 0u);
                if (it + 1 < nloc) {
#pragma unroll
                    for (int kk = 0; kk < kBK / 16; ++kk)
                        tc_mma_f16_ts(tmem, at + 32 + kk * 8, bd + (xstage >> 4) + kk * 2, idesc, 1u);
                }
                tc_commit(empty_x(ux));
                if (!same_ring) tc_commit(empty_a(ua));
            }
            __syncwarp();
            if (++ux == units) { ux = 0; px ^= 1u; }
            if (++ua == kUnitsA) { ua = 0; pa ^= 1u; }
        }
        if (elect_one()) tc_commit(acc_full);     // arrives once every MMA issued above is done
        __syncwarp();
    } else {                                      // ---------------- expansion, then epilogue
        const int q = warp & 3, g4 = warp >> 2;   // rows, and which of a slice's four k-blocks
        const int r = q * 32 + lane;
        const int64_t n = (int64_t)n0 + r;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        if (A.g32) pdl_wait();                    // (weights otherwise: no dependence)
        // The row's plane of the largest |g| goes first, as it is; its g scales the row.
        float gi[KP];
        int first = 0;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            gi[i] = n >= A.N ? 0.0f : A.g32 ? A.g32[(int64_t)i * A.N + n]
                                            : __half2float(__ushort_as_half(A.g16[(int64_t)i * A.N + n]));
            if (i > 0 && fabsf(gi[i]) > fabsf(scale)) first = i;
            if (first == i) scale = gi[i];
        }
        uint32_t ratio[KP], hoff[KP], woff[KP];   // of the planes in the row's order
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const int pl = i == 0 ? first : i <= first ? i - 1 : i;
            const float gp = pl_select<KP>(gi, pl);
            ratio[i] = as_u32(__half2half2(__float2half_rn(scale != 0.0f ? __fdiv_rn(gp, scale) : gp)));
            hoff[i] = (uint32_t)(pl * 128);
            woff[i] = (uint32_t)(pl * kWBlock);
        }
        // word w of row `lane` of tile q in the stage: slot w ^ (lane / 4)
        const uint32_t wrow = ws0 + (uint32_t)(q * 1024 + lane * 4);
        const uint32_t slot0 = (uint32_t)(((2 * g4) ^ (lane >> 2)) * 128), slot1 = (uint32_t)(((2 * g4 + 1) ^ (lane >> 2)) * 128);
        int sw = 0;
        uint32_t wph = 0;
        for (int sl = 0; sl < nsl; ++sl) {
            if (!wait_warp(full_w(sw), wph, abort_flag, A.dev_status)) { ok = false; break; }
            uint32_t w[2][KP];
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                w[0][i] = lds32(wrow + (uint32_t)(sw * w_stage_bytes(KP)) + woff[i] + slot0);
                w[1][i] = lds32(wrow + (uint32_t)(sw * w_stage_bytes(KP)) + woff[i] + slot1);
            }
            const int ua = 2 * (sl & 1) + (g4 >> 1);          // the A unit, used for the (sl / 2)th time
            const bool unit = sl * 4 + (g4 & 2) < nloc, mine = sl * 4 + g4 < nloc;
            if (unit && sl >= 2) {
                if (!wait_warp(same_ring ? empty_x(ua) : empty_a(ua), ((sl >> 1) - 1) & 1, abort_flag, A.dev_status)) { ok = false; break; }
                tc_fence_after();
            }
            if (mine) {
                const uint32_t h = ws0 + (uint32_t)(sw * w_stage_bytes(KP) + KP * kWBlock + g4 * KP * kHBlock);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t a[16];
                    expand_word<KP>(a, w[hh], ratio, hoff, h + (uint32_t)(hh * 64));
                    tc_st_32x32b_x16(tmem + lane_base + DC + (uint32_t)((2 * ua + (g4 & 1)) * 32 + hh * 16), a);
                }
                tc_wait_st();
                tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(empty_w(sw));
                if (unit) mbar_arrive(full_a(ua));            // also for a unit's second k-block that does not exist
            }
            if (++sw == wstages) { sw = 0; wph ^= 1u; }
        }
    }
    __syncwarp();
    if (ks > 1) cluster_wait();                   // the peers run: their shared memory may be written

    if (warp < kEW) {                             // ---------------- epilogue
        const int q = warp & 3, part = warp >> 2, r = q * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q * 32) << 16;
        if (ok) {
            const int tokens = min(bt, A.M - m0);
            pdl_wait();                           // xs, what mul and residual hold
            float xs = ks == 1 ? token_xs(A.ep, m0, part * 16, tokens, lane) : 0.0f;    // of a block's tokens, one block ahead
            if (ks == 1 && !ep_vectors(A.ep)) {
                const float bias = A.ep.bias && n0 + r < A.N ? A.ep.bias[n0 + r] : 0.0f;
                Column<16> f;                     // the next block's operands are fetched while this one is finished
                EpAt at = ep_at(A.ep, (int64_t)m0 + part * 16, (int64_t)n0 + r);
                const EpStep block = ep_tokens(A.ep, 4 * kEW);
                int left = n0 + r < A.N ? tokens - part * 16 : 0;             // tokens from this lane's first on
                ep_fetch_column(A.ep, at, left, f);
                ok = wait_warp(acc_full, 0, abort_flag, A.dev_status);
                tc_fence_after();
                for (int c = part * 16; ok && c < tokens; c += 4 * kEW) {
                    uint32_t v[16];
                    tc_ld_32x32b_x16(tmem + lane_base + (uint32_t)c, v);
                    tc_wait_ld();
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        y[j] = fmaf(scale, __uint_as_float(v[j]) * __shfl_sync(0xffffffffu, xs, j), bias);
                    xs = token_xs(A.ep, m0, c + 4 * kEW, tokens, lane);
                    ep_finish_column(A.ep, at, left, f, y);
                    at = ep_down(at, block);
                    left -= 4 * kEW;
                    ep_fetch_column(A.ep, at, left, f);
                }
            } else if (ks == 1) {
                // 16 tokens at a time through a tile of this warp's own in the (now idle) ring, so
                // that four lanes take 32 consecutive columns of a token
                float* tile = reinterpret_cast<float*>(gbase + warp * kTile);
                const int64_t nn = (int64_t)n0 + q * 32 + 8 * (lane & 3);
                const int cnt = A.N - nn >= 8 ? 8 : (int)max((int64_t)0, A.N - nn);
                float bias[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) bias[e] = A.ep.bias && e < cnt ? A.ep.bias[nn + e] : 0.0f;
                Eight f[2];                       // of the block's tokens 8 u + lane / 4; the next block's are
                                                  // fetched while this one is finished
                EpAt at = ep_at(A.ep, (int64_t)m0 + part * 16 + (lane >> 2), nn);
                const EpStep eight = ep_tokens(A.ep, 8), block = ep_tokens(A.ep, 4 * kEW);
                int left = cnt > 0 ? tokens - part * 16 - (lane >> 2) : 0;    // tokens from this lane's first on
                if (left > 0) ep_fetch(A.ep, at, cnt, f[0]);
                if (left > 8) ep_fetch(A.ep, ep_down(at, eight), cnt, f[1]);
                ok = wait_warp(acc_full, 0, abort_flag, A.dev_status);
                tc_fence_after();
                for (int c = part * 16; ok && c < tokens; c += 4 * kEW) {
                    uint32_t v[16];
                    tc_ld_32x32b_x16(tmem + lane_base + (uint32_t)c, v);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) tile[j * 36 + lane] = scale * __uint_as_float(v[j]);
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float* src = tile + (u * 8 + (lane >> 2)) * 36 + 8 * (lane & 3);
                        const float4 lo = *reinterpret_cast<const float4*>(src);
                        const float4 hi = *reinterpret_cast<const float4*>(src + 4);
                        float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                        const float back = __shfl_sync(0xffffffffu, xs, u * 8 + (lane >> 2));
#pragma unroll
                        for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], back, bias[e]);
                        const EpAt pu = u == 0 ? at : ep_down(at, eight);
                        if (left > 8 * u) ep_finish(A.ep, pu, cnt, f[u], y);
                        if (left > 4 * kEW + 8 * u) ep_fetch(A.ep, ep_down(pu, block), cnt, f[u]);
                    }
                    xs = token_xs(A.ep, m0, c + 4 * kEW, tokens, lane);
                    at = ep_down(at, block);
                    left -= 4 * kEW;
                    __syncwarp();
                }
            } else {
                // slot (this rank, row, token) at the row's owner: rank j owns the groups of eight rows
                // [16 j / ks, 16 (j + 1) / ks)
                const int owner = ((r >> 3) * ks + ks - 1) / 16, lr = r - 8 * (16 * owner / ks);
                ok = wait_warp(acc_full, 0, abort_flag, A.dev_status);
                tc_fence_after();
                for (int c = part * 16; ok && c < tokens; c += 4 * kEW) {
                    uint32_t v[16];
                    tc_ld_32x32b_x16(tmem + lane_base + (uint32_t)c, v);
                    tc_wait_ld();
                    const uint32_t dst = smem_u32(recv) + (uint32_t)(((rank * rows_per_rank(ks) + lr) * recv_pitch(bt) + c) * 4);
#pragma unroll
                    for (int j = 0; j < 16; j += 4)
                        st_dsmem_v4(dst + (uint32_t)(j * 4), (uint32_t)owner, scale * __uint_as_float(v[j]),
                                    scale * __uint_as_float(v[j + 1]), scale * __uint_as_float(v[j + 2]),
                                    scale * __uint_as_float(v[j + 3]));
                }
            }
        }
    }

    if (ks > 1) {                                 // every CTA arrives, also one that gave up
        // one item per token and group of eight rows; consecutive threads take consecutive tokens, so that the
        // sums read shared memory without conflicts
        const int g0 = 16 * rank / ks, groups = 16 * (rank + 1) / ks - g0;
        const int tokens = min(bt, A.M - m0), items = groups * tokens, pitch = recv_pitch(bt);
        Eight f;
        float back = 0.0f;                        // the token's xs
        auto item = [&](int x, bool finish) {
            const int g = x / tokens, tok = x - g * tokens;
            const int64_t n = (int64_t)n0 + 8 * (g0 + g);
            const int cnt = A.N - n >= 8 ? 8 : (int)(A.N - n);
            if (cnt <= 0) return;
            const EpAt at = ep_at(A.ep, (int64_t)m0 + tok, n);
            if (!finish) {
                back = A.ep.xs[m0 + tok];
                ep_fetch(A.ep, at, cnt, f);
                return;
            }
            float y[8] = {};
            for (int j = 0; j < ks; ++j) {
                const float* src = recv + (j * rows_per_rank(ks) + 8 * g) * pitch + tok;
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] += src[e * pitch];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = fmaf(y[e], back, A.ep.bias && e < cnt ? A.ep.bias[n + e] : 0.0f);
            ep_finish(A.ep, at, cnt, f, y);
        };
        __syncwarp();
        if ((int)threadIdx.x < items) {           // the first item's operands are in flight over the barrier
            pdl_wait();
            item((int)threadIdx.x, false);
        }
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (!*abort_flag)
            for (int x = threadIdx.x; x < items; x += kThreads) {
                if (x != (int)threadIdx.x) item(x, false);
                item(x, true);
            }
    }

    // ---- teardown: every MMA has completed (acc_full) or the CTA gave up
    if (warp == kEW && lane == 0 && *abort_flag)    // no MMA may still run when TMEM is freed
        mbar_drain(acc_full, 0, globaltimer_ns());
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) set_dev_status(A.dev_status, RB_DEV_TIMEOUT);
    if (warp == kEW) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(NC) : "memory");
    }
}

// ---------------------------------------------------------------- host side
struct LinPlan {
    int bt, ks, kb_per;
    bool dense;
};
// Tokens per tile and K split, and whether the weights are expanded once for all tokens instead
// (rb_linear_dense.cu): the least time by a model in SM cycles.  Here: waves of CTAs, one per SM, each
// with a k-block's MMAs (2 cycles per token) or its expansion, whichever is longer, and a start and an
// epilogue that nothing overlaps.  `slots` clusters of ks CTAs are resident (a cluster stays within a GPC).
// There: see dense_plan.  Measured against each other, this / that in us: 4096 x 4096, k = 2,
// M = 1024: 30.8 / 39.7, M = 2048: 57.3 / 66.2, M = 2560: 82.1 / 72.5; k = 4, M = 1536: 64.2 / 57.2;
// 14336 x 4096, M = 1536: 141 / 152, M = 2048: 203 / 187; 4096 x 11008, M = 2048: 145 / 182.
// Below 768 tokens the model favours the other form too early and is not asked: 4096 x 4096, k = 4,
// M = 384: 29.9 / 33.0, M = 512: 30.5 / 33.3; 14336 x 4096, k = 4, M = 752: 102 / 121; 4096 x 14336, k = 4, M = 450:
// 86.7 / 108; 8192 x 1024, k = 2, M = 640: 22.7 / 27.3; 20000 x 160, k = 2, M = 512: 26.4 / 27.7.  That costs
// where k is large: 4096 x 4096, k = 6, M = 512: 41.0 / 40.3, k = 8, M = 384: 50.9 / 44.0, M = 752: 53.0 / 49.4.
LinPlan plan(int N, int K, int kp, int M)
{
    const int nkb = (K + kBK - 1) / kBK, nt = (N + kBR - 1) / kBR;
    LinPlan best = {0, 1, nkb, false};
    double cost = 0;
    for (int bt = 16; bt <= 256; bt += 16) {
        const int mt = (M + bt - 1) / bt;
        if (bt > 16 && (M + bt - 17) / (bt - 16) == mt) continue;    // a narrower tile does with as many
        if (mt > 65535) continue;                                    // the grid's second dimension
        const int64_t tiles = (int64_t)nt * mt;
        int last = 0;
        for (int ks = 1; ks <= 8; ++ks) {
            if (ks > 1 && tiles >= 148) break;
            const int kb_per = ((nkb + ks - 1) / ks + 3) / 4 * 4;      // whole 256-column slices
            const int z = (nkb + kb_per - 1) / kb_per;
            if (z == last || recv_bytes(bt, z) > 72 * 1024) continue;
            last = z;
            static const int slots[8] = {148, 74, 48, 35, 26, 24, 18, 16};
            const double waves = (double)((tiles + slots[z - 1] - 1) / slots[z - 1]);
            const double mma = 2.0 * bt, expand = 70.0 * kp + 300.0;
            const double c = waves * (1.1 * kb_per * (mma > expand ? mma : expand) + 9000 + 20.0 * bt +
                                      (z > 1 ? 2500 + 16.0 * bt : 0)) + 9000;
            if (best.bt == 0 || c < cost) {
                cost = c;
                best.bt = bt;
                best.kb_per = kb_per;
                best.ks = z;
            }
        }
    }
    best.dense = best.bt == 0 || (M >= 768 && dense_plan(N, K, M).cost < cost);
    return best;
}

template <int KP>
rb_status launch_tc(const LinArgs& args, const uint16_t* x16, int ks, cudaStream_t stream)
{
    LinArgs a = args;
    CUtensorMap map = {};
    if (!encode_fp16(&map, x16, a.M, a.K, a.bt)) return RB_ERR_CUDA;
    static std::atomic<bool> attr_set[64];       // per device; setting the attributes twice is harmless
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RB_ERR_CUDA;
    auto* kern = linear_tc_kernel<KP>;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem) != cudaSuccess)
            return RB_ERR_CUDA;
        if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
    }
    a.wstages = KP <= 2 ? 3 : 2;
    a.stages = kMaxStages;
    while (a.stages > 2 && linear_smem(KP, a.bt, a.stages, a.wstages, ks) > kMaxSmem) a.stages -= 2;
    if (linear_smem(KP, a.bt, a.stages, a.wstages, ks) > kMaxSmem) return RB_ERR_UNSUPPORTED;
    // A whole SM's shared memory, always: a CTA of a cluster must not share its SM with another kernel
    // that holds tensor memory, or two clusters could each wait for the columns the other's peer holds.
    const int smem = kMaxSmem;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + kBR - 1) / kBR), (unsigned)((a.M + a.bt - 1) / a.bt), (unsigned)ks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (ks > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = 1;
        attr[na].val.clusterDim.y = 1;
        attr[na].val.clusterDim.z = (unsigned)ks;
        ++na;
    }
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;   // after the pre-pass
    attr[na].val.programmaticStreamSerializationAllowed = 1;
    ++na;
    cfg.attrs = attr;
    cfg.numAttrs = (unsigned)na;
    return cudaLaunchKernelEx(&cfg, kern, map, a) == cudaSuccess ? RB_OK : RB_ERR_CUDA;
}

size_t run_workspace(int N, int K, int kp, int M)
{
    return plan(N, K, kp, M).dense ? dense_workspace(N, K, M) : x16_bytes(M, K) + xs_bytes(M);
}

// a: planes, row scales, X, h, epilogue, sizes
rb_status linear_run(LinArgs a, int kp, void* workspace, bool pdl, cudaStream_t stream)
{
    const LinPlan p = plan(a.N, a.K, kp, a.M);
    if (p.dense) {
        const DenseArgs d = {a.X, a.ldx, a.planes, a.g16, a.h16, a.g32, a.h32, a.N, a.K, a.M, kp, a.dev_status};
        return dense_run(d, &a.ep, workspace, pdl, stream);
    }
    a.bt = p.bt;
    a.kb_per = p.kb_per;
    a.limit = kp > 1 || a.h32 ? 65504.0f / (float)kp : HUGE_VALF;
    uint16_t* x16 = static_cast<uint16_t*>(workspace);
    float* xs = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + x16_bytes(a.M, a.K));
    a.ep.xs = xs;
    const bool dependent = pdl || a.g32;
    const rb_status st = a.K <= 1024   ? launch_prepass<256, 32, 4>(a, x16, xs, dependent, stream)
                         : a.K <= 4096 ? launch_prepass<256, 128, 4>(a, x16, xs, dependent, stream)
                                       : launch_prepass<512, 512, 4>(a, x16, xs, dependent, stream);
    if (st != RB_OK) return st;
    switch (kp) {
        case 1: return launch_tc<1>(a, x16, p.ks, stream);
        case 2: return launch_tc<2>(a, x16, p.ks, stream);
        case 3: return launch_tc<3>(a, x16, p.ks, stream);
        case 4: return launch_tc<4>(a, x16, p.ks, stream);
        case 5: return launch_tc<5>(a, x16, p.ks, stream);
        case 6: return launch_tc<6>(a, x16, p.ks, stream);
        case 7: return launch_tc<7>(a, x16, p.ks, stream);
        default: return launch_tc<8>(a, x16, p.ks, stream);
    }
}

constexpr int kMaxRows = 1 << 30, kMaxColumns = 1 << 24;      // M and N, K: the kernels' 32-bit coordinates

// Checks of the epilogue and the outputs, shared by both entry points; fills `out`.
rb_status check_epilogue(const rb_epilogue_t* ep, const uint16_t* X, int64_t ldx, int M, int64_t N, int64_t K, void* Y,
                         int64_t ldy, rb_dtype y_dtype, LinEp& out)
{
    if (!X || !Y || (y_dtype != RB_F32 && y_dtype != RB_BF16)) return RB_ERR_ARG;
    rb_epilogue_t e = {};
    if (ep) e = *ep;
    if (e.reserved != 0 || !good_act(e.act) || (e.residual_dtype != RB_F32 && e.residual_dtype != RB_BF16))
        return RB_ERR_ARG;
    if (M < 1 || M > kMaxRows || N > kMaxRows || K > kMaxColumns || ldx < K || ldx % 8 != 0 || ldy < N || (e.mul && e.ld_mul < N) || (e.residual && e.ld_residual < N) ||
        (e.preact && e.ld_preact < N))
        return RB_ERR_SHAPE;
    const void* ptrs[] = {X, Y, e.bias, e.mul, e.residual, e.preact};
    for (const void* q : ptrs)
        if (!aligned16(q)) return RB_ERR_ALIGN;
    const int yb = y_dtype == RB_BF16 ? 2 : 4, rb = e.residual_dtype == RB_BF16 ? 2 : 4;
    const MatRange y = mat_range(Y, M, N, ldy, yb);
    const MatRange x = mat_range(X, M, K, ldx, 2);
    const bool in_place = e.residual == Y && e.ld_residual == ldy && rb == yb;
    if (overlaps(y, x) || (e.bias && overlaps(y, mat_range(e.bias, 1, N, N, 4)))) return RB_ERR_ARG;
    if (e.mul && overlaps(y, mat_range(e.mul, M, N, e.ld_mul, 2))) return RB_ERR_ARG;
    if (e.residual && !in_place && overlaps(y, mat_range(e.residual, M, N, e.ld_residual, rb))) return RB_ERR_ARG;
    if (e.preact) {
        const MatRange p = mat_range(e.preact, M, N, e.ld_preact, 2);
        if (overlaps(p, y) || overlaps(p, x) || (e.bias && overlaps(p, mat_range(e.bias, 1, N, N, 4))) || (e.mul && overlaps(p, mat_range(e.mul, M, N, e.ld_mul, 2))) ||
            (e.residual && overlaps(p, mat_range(e.residual, M, N, e.ld_residual, rb))))
            return RB_ERR_ARG;
    }
    out.bias = e.bias;
    out.mul = e.mul;
    out.res = e.residual;
    out.pre = e.preact;
    out.Y = Y;
    out.ld_mul = e.ld_mul;
    out.ld_res = e.ld_residual;
    out.ld_pre = e.ld_preact;
    out.ld_y = ldy;
    out.act = e.act;
    out.res_bf16 = e.residual_dtype == RB_BF16;
    out.y_bf16 = y_dtype == RB_BF16;
    out.vec = (e.ld_mul % 8 == 0 ? 1 : 0) | (e.ld_residual % 8 == 0 ? 2 : 0) | (e.ld_preact % 8 == 0 ? 4 : 0) |
              (ldy % 8 == 0 ? 8 : 0);
    return RB_OK;
}

// Whether Y or the pre-activation meets one of the call's other arrays.
struct Bytes {
    const void* p;
    size_t n;
};
bool outputs_meet(const LinEp& ep, int64_t M, int64_t N, std::initializer_list<Bytes> others)
{
    const MatRange y = mat_range(ep.Y, M, N, ep.ld_y, ep.y_bf16 ? 2 : 4);
    for (const Bytes& b : others)
        if (meets(y, b.p, b.n) || (ep.pre && meets(mat_range(ep.pre, M, N, ep.ld_pre, 2), b.p, b.n))) return true;
    return false;
}

// One token goes through the byte tables (4096 x 4096, k = 2: 5.8 us against 10.6 us on the tensor cores, and exact).
bool one_token(int k_planes, int M) { return M == 1 && k_planes <= 4; }

bool good_shape(int n_out, int k_in, int k_planes, int M)
{
    return n_out >= 1 && n_out <= kMaxRows && k_in >= 32 && k_in <= kMaxColumns && k_in % 32 == 0 && k_planes >= 1 &&
           k_planes <= 8 && M >= 1 && M <= kMaxRows;
}
size_t planes_bytes(int n_out, int k_in, int k_planes)
{
    return (rb_packed_words(n_out, k_in, k_planes) * 4 + 255) / 256 * 256;
}

}  // namespace
}  // namespace rbw

using namespace rbw;

extern "C" size_t rb_linear_workspace_bytes(int n_out, int k_in, int k_planes, int M)
{
    if (!good_shape(n_out, k_in, k_planes, M) || one_token(k_planes, M)) return 0;
    return run_workspace(n_out, k_in, k_planes, M);
}

extern "C" rb_status rb_linear(const rb_layer_t* layer, const uint16_t* X, int64_t ldx, int M, const rb_epilogue_t* ep,
                               void* Y, int64_t ldy, rb_dtype y_dtype, void* workspace, size_t workspace_bytes,
                               int32_t* dev_status, unsigned flags, cudaStream_t stream)
{
    rb_status st = check_apply_args(layer, X, M, Y, y_dtype, flags);
    if (st != RB_OK) return st;
    LinArgs a = {};
    st = check_epilogue(ep, X, ldx, M, layer->n_out, layer->k_in, Y, ldy, y_dtype, a.ep);
    if (st != RB_OK) return st;
    if (dev_status && !aligned16(dev_status)) return RB_ERR_ALIGN;
    const size_t need = rb_linear_workspace_bytes(layer->n_out, layer->k_in, layer->k_planes, M);
    if (need) {
        if (!workspace || workspace_bytes < need) return RB_ERR_WORKSPACE;
        if (!aligned16(workspace)) return RB_ERR_ALIGN;
    }
    const size_t kp = (size_t)layer->k_planes;
    if (outputs_meet(a.ep, M, layer->n_out,
                     {{layer->planes, rb_packed_words(layer->n_out, layer->k_in, layer->k_planes) * 4},
                      {layer->g16, kp * layer->n_out * 2}, {layer->h16, kp * layer->k_in * 2}, {workspace, need}}))
        return RB_ERR_ARG;
    if (!device_is_sm100()) return RB_ERR_UNSUPPORTED;
    if (one_token(layer->k_planes, M)) return lut_linear(layer, X, &a.ep, (flags & RB_LAUNCH_PDL) != 0, stream);
    a.planes = layer->planes;
    a.g16 = layer->g16;
    a.dev_status = dev_status;
    a.N = layer->n_out;
    a.K = layer->k_in;
    a.M = M;
    a.X = X;
    a.ldx = ldx;
    a.h16 = layer->h16;
    return linear_run(a, layer->k_planes, workspace, (flags & RB_LAUNCH_PDL) != 0, stream);
}

extern "C" size_t rb_qat_linear_workspace_bytes(int n_out, int k_in, int k_planes, int M)
{
    if (!good_shape(n_out, k_in, k_planes, M)) return 0;
    return planes_bytes(n_out, k_in, k_planes) + run_workspace(n_out, k_in, k_planes, M);
}

extern "C" rb_status rb_qat_linear(const float* W, const float* g, const float* h, int n_out, int k_in, int k_planes,
                                   const uint16_t* X, int64_t ldx, int M, const rb_epilogue_t* ep, void* Y, int64_t ldy,
                                   rb_dtype y_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   unsigned flags, cudaStream_t stream)
{
    if (!W || !g || !h || k_planes < 1 || k_planes > 8 || (flags & ~RB_LAUNCH_PDL)) return RB_ERR_ARG;
    if (n_out < 1 || k_in < 32 || k_in % 32 != 0) return RB_ERR_SHAPE;
    if (!aligned16(W) || !aligned16(g) || !aligned16(h)) return RB_ERR_ALIGN;
    LinArgs a = {};
    rb_status st = check_epilogue(ep, X, ldx, M, n_out, k_in, Y, ldy, y_dtype, a.ep);
    if (st != RB_OK) return st;
    if (dev_status && !aligned16(dev_status)) return RB_ERR_ALIGN;
    if (!workspace || workspace_bytes < rb_qat_linear_workspace_bytes(n_out, k_in, k_planes, M)) return RB_ERR_WORKSPACE;
    if (!aligned16(workspace)) return RB_ERR_ALIGN;
    const size_t kp = (size_t)k_planes;
    if (outputs_meet(a.ep, M, n_out,
                     {{W, (size_t)n_out * k_in * 4}, {g, kp * n_out * 4}, {h, kp * k_in * 4},
                      {workspace, rb_qat_linear_workspace_bytes(n_out, k_in, k_planes, M)}}))
        return RB_ERR_ARG;
    if (!device_is_sm100()) return RB_ERR_UNSUPPORTED;
    uint32_t* planes = static_cast<uint32_t*>(workspace);
    const bool beside = !plan(n_out, k_in, k_planes, M).dense;    // (the dense form's first pass reads the planes)
    st = pack_planes_early(W, g, h, n_out, k_in, k_planes, planes, dev_status, beside, stream);
    if (st != RB_OK) return st;
    a.planes = planes;
    a.g32 = g;
    a.dev_status = dev_status;
    a.N = n_out;
    a.K = k_in;
    a.M = M;
    a.X = X;
    a.ldx = ldx;
    a.h32 = h;
    return linear_run(a, k_planes, static_cast<uint8_t*>(workspace) + planes_bytes(n_out, k_in, k_planes),
                      (flags & RB_LAUNCH_PDL) != 0, stream);
}
