// rb_linear_dense.cu -- the linear product for many tokens: the weights are
// expanded to fp16 once, then multiplied as a dense matrix.
//
// A weight's expansion costs instructions for every token tile that repeats it
// (rb_linear.cu); from some hundred tokens on it is cheaper to write the expanded
// matrix once, 2 bytes per weight, and let TMA bring both operands.
//
// Pass 1 (expand_kernel): X16 = fp16(X), each row at a power of two of its own (rb_linear.cuh),
// and W16[n][c] = fp16(sum_i (g_i[n] 2^-e) (B_i h_i[c])),
// scale[n] = 2^e with k max_i |g_i| <= 2^e, so that no sum overflows and the
// ratios of fp16 scales are exact; k = 1: W16 = +-h, scale = g, exact.  Both
// matrices hold each 32-column group in the order 0, 16, 1, 17, ..: the signs of
// columns j and j + 16 are 16 bits apart in a sign word, where an fp16x2 has its
// two sign bits, and the order of the columns does not matter to a dot product.
//
// Pass 2 (dense_kernel): D[m][n] = X16 W16^T on pairs of CTAs (tcgen05
// cta_group::2).  A pair computes 256 tokens x bn rows n (bn a multiple of 32 up to
// 256): each CTA holds its 128 tokens (A) and half of the bn rows (B) in shared memory
// and 128 lanes x bn columns of D; the MMA reads both halves of B, which halves
// what each SM loads.  Persistent: pair p takes tiles p, p + pairs, ..; D is
// double-buffered in tensor memory, so that the eight epilogue warps finish one
// tile while the MMAs of the next run.
//   warps 0..7  epilogue: warp w has tokens 32 (w % 4) .. + 31 and every other 32 columns.
//               A 32 x 32 block goes through a tile in shared memory, so that four
//               lanes take 32 consecutive columns of a token; the factor and
//               the residual of a block are fetched while the one before is finished
//   warp 8      the pair's even CTA issues the MMAs of both
//   warp 9      TMA of this CTA's halves; both CTAs' loads count on the even
//               CTA's barrier
// Waits are bounded (rb_tcgen05.cuh); a CTA that gives up still meets the cluster
// barrier, after its loads and MMAs have had time to land.
#include "rbw_internal.cuh"
#include "rb_epilogue.cuh"
#include "rb_linear.cuh"
#include "rb_tcgen05.cuh"

namespace rbw {
namespace {

constexpr int kDK = 64;                        // columns per stage (128 bytes of fp16)
constexpr int kDTok = 128;                     // tokens per CTA (tensor-memory lanes)
constexpr int kDEW = 8;                        // epilogue warps
constexpr int kDThreads = 32 * (kDEW + 2);
constexpr int kDStages = 5;
constexpr uint32_t kDHalf = kDTok * 128;       // bytes of a stage's A, and at most of its B
constexpr int kDPitch = 36;                    // floats per row of a warp's 32 x 32 transpose tile
constexpr int kDTile = 32 * kDPitch * 4;
constexpr int kDSmem = 227 * 1024;             // a whole SM's: no other kernel's CTA beside it may hold tensor memory
static_assert(kDStages * 2 * (int)kDHalf + 1024 + 256 + kDEW * kDTile <= kDSmem, "shared memory");
constexpr uint32_t kLeadMask = 0xFEFFFFFFu;    // shared::cluster address of the pair's even CTA

struct DenseKernelArgs {
    LinEp ep;
    const float* scale;
    int32_t* dev_status;
    int N, K, M, bn, mt, tiles;                // tiles = mt x (row tiles), token tiles fastest
};

// ---------------------------------------------------------------- pass 1
// Rows of tile t (128 of them), slice s: warp w expands word w of the slice; a
// lane takes four cells (8 columns) of one row, eight rows per warp and step, so
// that the sign words and the 64-byte runs of W16 are read and written whole.
template <int KP>
__device__ __forceinline__ void expand_block(const DenseArgs& d, int64_t blk, uint16_t* __restrict__ W16,
                                             float* __restrict__ scale, int& flags)
{
    __shared__ uint32_t rho[KP][128];
    const int64_t S = num_slices(d.K), Nt = num_row_tiles(d.N);
    const int64_t s = blk % S, t = blk / S;
    if (threadIdx.x < 128) {
        const int64_t n = t * 128 + threadIdx.x;
        float g[KP], top = 0.0f;
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            g[i] = n >= d.N ? 0.0f : d.g32 ? d.g32[(int64_t)i * d.N + n]
                                           : __half2float(__ushort_as_half(d.g16[(int64_t)i * d.N + n]));
            top = fmaxf(top, fabsf(g[i]));
        }
        float sc = g[0];
        if constexpr (KP > 1) {
            // 2^e >= KP top (as a power of two above it); 0 and non-finite scales: 1, so that NaN and inf stay
            int e = 0;
            if (top > 0.0f && top <= 3.0e38f) (void)frexpf(top, &e);
            e += KP > 4 ? 3 : KP > 2 ? 2 : 1;
            if (e > 126) e = 126;
            if (e < -120) e = -120;
            sc = __int_as_float((e + 127) << 23);
            const float inv = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int i = 0; i < KP; ++i) {
                const __half2 r = __half2half2(__float2half_rn(g[i] * inv));
                rho[i][threadIdx.x] = *reinterpret_cast<const uint32_t*>(&r);
            }
        }
        if (s == 0 && n < d.N) scale[n] = sc;
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, t4 = lane & 3;
    const int64_t c0 = s * 256 + w * 32;
    if (c0 >= d.K) return;                     // (no barrier follows)
    uint32_t h[KP][4];
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t c = (int64_t)i * d.K + c0 + 4 * t4 + e;
            uint32_t lo, hi;
            if (d.h32) {
                const __half a = __float2half_rn(d.h32[c]), b = __float2half_rn(d.h32[c + 16]);
                if (__hisnan(a) || __hisnan(b)) flags |= RB_DEV_NONFINITE;
                else if (__hisinf(a) || __hisinf(b)) flags |= RB_DEV_RANGE;
                lo = __half_as_ushort(a);
                hi = __half_as_ushort(b);
            } else {
                lo = d.h16[c];
                hi = d.h16[c + 16];
            }
            h[i][e] = lo | (hi << 16);
        }
    // Row r = 8 it + lane / 4 of the block: tile it / 4, and in it row 8 (it % 4) + lane / 4, whose slot
    // for word w is w ^ (2 (it % 4) + lane / 16).
    const int sh = 12 - 4 * t4;                // cell 4 t4 + e: its signs come to bits 15 and 31 by sh + 3 - e
    const int rows = (int)min((int64_t)128, d.N - t * 128);
    const uint32_t* pl[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) pl[i] = d.planes + block_index(i, s, t * 4, S, Nt) * 256 + (lane >> 2);
    int off[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) off[j] = (w ^ (2 * j + (lane >> 4))) * 32 + 8 * j;
    uint16_t* out = W16 + (t * 128 + (lane >> 2)) * d.K + c0 + t4 * 8;
    const int64_t step = (int64_t)d.K * 8;
#pragma unroll 1
    for (int tile = 0; tile < 4; ++tile) {
        uint32_t words[4][KP];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < KP; ++i)
                words[j][i] = tile * 32 + j * 8 + (lane >> 2) < rows ? __ldg(pl[i] + tile * 256 + off[j]) << sh : 0u;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = tile * 32 + j * 8 + (lane >> 2);
            uint32_t q[KP], o[4];
            if constexpr (KP > 1) {
#pragma unroll
                for (int i = 0; i < KP; ++i) q[i] = rho[i][r];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                __half2 acc;
#pragma unroll
                for (int i = 0; i < KP; ++i) {
                    o[e] = lop3_sign(words[j][i] << (3 - e), h[i][e]);
                    if constexpr (KP > 1) {
                        const __half2 v = *reinterpret_cast<const __half2*>(&o[e]);
                        const __half2 g = *reinterpret_cast<const __half2*>(&q[i]);
                        acc = i == 0 ? __hmul2(g, v) : __hfma2(g, v, acc);
                    }
                }
                if constexpr (KP > 1) o[e] = *reinterpret_cast<const uint32_t*>(&acc);
            }
            if (r < rows) *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
            out += step;
        }
    }
}

template <int KP>
__global__ void __launch_bounds__(256)
expand_kernel(const __grid_constant__ DenseArgs d, int xblocks, int64_t wblocks, uint16_t* __restrict__ X16,
              uint16_t* __restrict__ W16, float* __restrict__ scale, float* __restrict__ xs)
{
    pdl_launch_dependents();
    pdl_wait();
    int flags = 0;
    if ((int)blockIdx.x < xblocks) {
        bool range = false;
        if (d.K <= 1024) convert_rows<256, 32, 4>(d.X, d.ldx, d.M, d.K, (int)blockIdx.x, xblocks, X16, xs, range);
        else if (d.K <= 4096) convert_rows<256, 128, 4>(d.X, d.ldx, d.M, d.K, (int)blockIdx.x, xblocks, X16, xs, range);
        else convert_rows<256, 256, 8>(d.X, d.ldx, d.M, d.K, (int)blockIdx.x, xblocks, X16, xs, range);
        if (range) flags |= RB_DEV_RANGE;
    } else {
        expand_block<KP>(d, (int64_t)blockIdx.x - xblocks, W16, scale, flags);
    }
    if (flags) set_dev_status(d.dev_status, flags);
}

// ---------------------------------------------------------------- pass 2
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%2, %3}], [%4];"
                 :: "r"(dst), "l"(map), "r"(x), "r"(y), "r"(bar) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued before are done.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(bar), "h"((uint16_t)3) : "memory");
}
// Arrive on the even CTA's barrier at this offset.
__device__ __forceinline__ void arrive_lead(uint32_t bar)
{
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(remote) : "r"(bar));
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(remote) : "memory");
}

// A warp's part of the epilogue of all tiles of this CTA.  VEC: the arrays' rows start on 16 bytes, a lane takes
// eight columns of rows rr + 8 i; otherwise one column of sixteen rows at a time.
template <bool VEC>
__device__ __forceinline__ void dense_epilogue(const DenseKernelArgs& A, uint8_t* tiles, uint32_t tmem, uint32_t acc_full,
                                               uint32_t acc_empty, volatile int* abort_flag)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = warp & 3, hh = warp >> 2;
    const int rank = (int)cluster_rank(), pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1), bn = A.bn;
    const uint32_t lane_base = (uint32_t)(q * 32) << 16;
    float* tile = reinterpret_cast<float*>(tiles + warp * kDTile);
    const int rr = VEC ? lane >> 2 : 0, cc = VEC ? 8 * (lane & 3) : lane;
    const EpStep step = ep_tokens(A.ep, VEC ? 8 : 16);
    int it = 0;
    for (int t = pair; t < A.tiles; t += pairs, ++it) {
        const int buf = it & 1;
        const int64_t m = (int64_t)(t % A.mt) * 2 * kDTok + rank * kDTok + q * 32 + rr;
        const int64_t n0 = (int64_t)(t / A.mt) * bn;
        const int cend = A.N - n0 < bn ? (int)(A.N - n0) : bn;
        const int left = A.M - m > 32 ? 32 : (int)(A.M - m);              // tokens from this lane's first on
        auto columns = [&](int c) {               // existing columns of this lane in the block at c
            const int n = cend - c - cc, most = VEC ? 8 : 1;
            return n >= most ? most : n > 0 ? n : 0;
        };
        EpAt at = ep_at(A.ep, m, n0 + hh * 32 + cc);
        Eight f[VEC ? 4 : 1];                     // operands of the block; the next one's are fetched as they are used
        Column<16> col[VEC ? 1 : 2];
        {
            const int cnt = columns(hh * 32);
            EpAt p = at;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (cnt > 0 && left > 8 * i) ep_fetch(A.ep, p, cnt, f[i]);
                    p = ep_down(p, step);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    ep_fetch_column(A.ep, p, cnt ? left - 16 * h : 0, col[h]);
                    p = ep_down(p, step);
                }
            }
        }
        const int64_t token = m - rr + lane;      // whose accumulators this lane reads
        const float xs = token < A.M ? __ldg(A.ep.xs + token) : 0.0f;
        if (!wait_warp(acc_full + 8u * buf, (it >> 1) & 1, abort_flag, A.dev_status)) break;
        tc_fence_after();
        for (int c = hh * 32; c < cend; c += 64) {
            const int cnt = columns(c), next = columns(c + 64);
            const float* scp = A.scale + n0 + c + cc;
            const float* bip = A.ep.bias + n0 + c + cc;
            alignas(16) float sc[VEC ? 8 : 4], bi[VEC ? 8 : 4];
            if (VEC && cnt == 8) {
                *reinterpret_cast<float4*>(sc) = __ldg(reinterpret_cast<const float4*>(scp));
                *reinterpret_cast<float4*>(sc + (VEC ? 4 : 0)) = __ldg(reinterpret_cast<const float4*>(scp) + 1);
                const float4 zero = make_float4(0, 0, 0, 0);
                *reinterpret_cast<float4*>(bi) = A.ep.bias ? __ldg(reinterpret_cast<const float4*>(bip)) : zero;
                *reinterpret_cast<float4*>(bi + (VEC ? 4 : 0)) = A.ep.bias ? __ldg(reinterpret_cast<const float4*>(bip) + 1) : zero;
            } else {
#pragma unroll
                for (int e = 0; e < (VEC ? 8 : 1); ++e) {
                    sc[e] = e < cnt ? __ldg(scp + e) : 0.0f;
                    bi[e] = A.ep.bias && e < cnt ? __ldg(bip + e) : 0.0f;
                }
            }
            uint32_t v[32];
            tc_ld_32x32b_x32(tmem + lane_base + (uint32_t)(buf * 256 + c), v);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e)
                *reinterpret_cast<float4*>(tile + lane * kDPitch + 4 * e) =
                    make_float4(__uint_as_float(v[4 * e]) * xs, __uint_as_float(v[4 * e + 1]) * xs,
                                __uint_as_float(v[4 * e + 2]) * xs, __uint_as_float(v[4 * e + 3]) * xs);
            __syncwarp();
            EpAt p = at;
            if constexpr (VEC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* src = tile + (rr + 8 * i) * kDPitch + cc;
                    const float4 lo = *reinterpret_cast<const float4*>(src), hi = *reinterpret_cast<const float4*>(src + 4);
                    float y[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = fmaf(sc[e], y[e], bi[e]);
                    if (left > 8 * i) {
                        if (cnt > 0) ep_finish(A.ep, p, cnt, f[i], y);
                        if (next > 0) ep_fetch(A.ep, ep_right(A.ep, p, 64), next, f[i]);
                    }
                    p = ep_down(p, step);
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float y[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) y[j] = fmaf(sc[0], tile[(16 * h + j) * kDPitch + lane], bi[0]);
                    ep_finish_column(A.ep, p, cnt ? left - 16 * h : 0, col[h], y);
                    ep_fetch_column(A.ep, ep_right(A.ep, p, 64), next ? left - 16 * h : 0, col[h]);
                    p = ep_down(p, step);
                }
            }
            at = ep_right(A.ep, at, 64);
            __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead(acc_empty + 8u * buf);
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDThreads, 1)
dense_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
             const __grid_constant__ DenseKernelArgs A)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t bar0 = sbase + kDStages * 2 * kDHalf;
    auto full = [&](int s) { return bar0 + 8u * s; };                     // even CTA's: both CTAs' loads
    auto empty = [&](int s) { return bar0 + 8u * (kDStages + s); };
    auto acc_full = [&](int b) { return bar0 + 8u * (2 * kDStages + b); };
    auto acc_empty = [&](int b) { return bar0 + 8u * (2 * kDStages + 2 + b); };   // even CTA's: both CTAs' warps
    static_assert(8 * (2 * kDStages + 4) + 8 <= 256, "barrier area");
    uint8_t* tail = smem_raw + (bar0 - smem_u32(smem_raw)) + 8 * (2 * kDStages + 4);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tail + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int nkb = (A.K + kDK - 1) / kDK;
    const int bn = A.bn;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kDStages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full(b), 1);
            mbar_init(acc_empty(b), 2 * kDEW);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(&tmap_x) : "memory");
        asm volatile("prefetch.tensormap [%0];" :: "l"(&tmap_w) : "memory");
    }
    if (warp == kDEW) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(tmem_slot)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();                           // both CTAs' barriers are ready
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    pdl_wait();                                   // X16, W16, scale, xs

    if (warp == kDEW + 1) {
        if (lane == 0) {                          // ---------------- TMA
            const uint32_t bytes = 2u * (kDHalf + (uint32_t)bn * 64u);       // both CTAs'
            int s = 0, j = 0, issued = 0;
            for (int t = pair; t < A.tiles && !*abort_flag; t += pairs) {
                const int m0 = (t % A.mt) * 2 * kDTok + (int)rank * kDTok;
                const int n0 = (t / A.mt) * bn + (int)rank * (bn / 2);
                for (int kb = 0; kb < nkb; ++kb) {
                    if (j > 0 && !mbar_wait(empty(s), (j - 1) & 1, abort_flag, A.dev_status, kTimeoutNs)) break;
                    const uint32_t a = sbase + (uint32_t)s * 2 * kDHalf, bar = full(s) & kLeadMask;
                    if (rank == 0) mbar_arrive_expect_tx(full(s), bytes);
                    tma_load_pair(a, &tmap_x, bar, kb * kDK, m0);
                    tma_load_pair(a + kDHalf, &tmap_w, bar, kb * kDK, n0);
                    ++issued;
                    if (++s == kDStages) { s = 0; ++j; }
                }
            }
            const uint64_t t0 = globaltimer_ns();
            if (*abort_flag) {
                while (globaltimer_ns() - t0 < 5000000ull) {}              // 5 ms: what was issued has landed
            } else {
                // every stage read: the last commits' arrivals have reached this CTA before it can leave
                for (int b = max(issued - kDStages, 0); b < issued; ++b)
                    mbar_drain(empty(b % kDStages), (b / kDStages) & 1, t0);
            }
        }
    } else if (warp == kDEW) {
        if (rank == 0) {                          // ---------------- MMAs of the pair
            const uint32_t idesc = (1u << 4) | ((uint32_t)(bn >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
            const uint64_t ad0 = smem_desc_sw128(sbase), bd0 = smem_desc_sw128(sbase + kDHalf);
            int s = 0, it = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int t = pair; t < A.tiles && ok; t += pairs, ++it) {
                const int buf = it & 1;
                if (it >= 2) ok = wait_warp(acc_empty(buf), ((it >> 1) - 1) & 1, abort_flag, A.dev_status);
                if (!ok) break;
                tc_fence_after();
                for (int kb = 0; kb < nkb; ++kb) {
                    if (!wait_warp(full(s), ph, abort_flag, A.dev_status)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad = ad0 + (uint32_t)(s * (2 * kDHalf >> 4)), bd = bd0 + (uint32_t)(s * (2 * kDHalf >> 4));
#pragma unroll
                        for (int kk = 0; kk < kDK / 16; ++kk)
                            mma_pair(tmem + (uint32_t)buf * 256u, ad + kk * 2, bd + kk * 2, idesc, (kb > 0 || kk > 0) ? 1u : 0u);
                        commit_pair(empty(s));
                    }
                    __syncwarp();
                    if (++s == kDStages) { s = 0; ph ^= 1u; }
                }
                if (elect_one()) commit_pair(acc_full(buf));
                __syncwarp();
            }
            if (!ok) {                            // MMAs already issued complete well within this
                const uint64_t t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 5000000ull) {}
            }
        }
    } else if (ep_vectors(A.ep)) {                // ---------------- epilogue
        dense_epilogue<true>(A, smem_raw + (bar0 - smem_u32(smem_raw)) + 256, tmem, acc_full(0), acc_empty(0), abort_flag);
    } else {
        dense_epilogue<false>(A, smem_raw + (bar0 - smem_u32(smem_raw)) + 256, tmem, acc_full(0), acc_empty(0), abort_flag);
    }

    // ---- both CTAs are done with each other's shared and tensor memory
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (*abort_flag && threadIdx.x == 0) set_dev_status(A.dev_status, RB_DEV_TIMEOUT);
    if (warp == kDEW) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
    }
}

// ---------------------------------------------------------------- host side
struct DenseWs {
    uint16_t* x16;
    uint16_t* w16;
    float* scale;
    float* xs;
    size_t bytes;
};
DenseWs dense_layout(int N, int K, int M, void* base)
{
    const size_t xb = x16_bytes(M, K), wb = ((size_t)N * K * 2 + 255) / 256 * 256;
    const size_t sb = ((size_t)N * 4 + 255) / 256 * 256;
    char* p = static_cast<char*>(base);
    return DenseWs{reinterpret_cast<uint16_t*>(p), reinterpret_cast<uint16_t*>(p + xb),
                   reinterpret_cast<float*>(p + xb + wb), reinterpret_cast<float*>(p + xb + wb + sb), xb + wb + sb + xs_bytes(M)};
}

template <int KP>
rb_status launch_expand(const DenseArgs& d, const DenseWs& ws, bool pdl, cudaStream_t stream)
{
    const int rows = d.K <= 1024 ? 8 : d.K <= 4096 ? 2 : 1;
    int64_t xblocks = ((int64_t)d.M + rows - 1) / rows;
    if (xblocks > 4 * 148) xblocks = 4 * 148;
    const int64_t wblocks = (((int64_t)d.N + 127) / 128) * num_slices(d.K);
    if (xblocks + wblocks > INT32_MAX) return RB_ERR_UNSUPPORTED;
    return launch(expand_kernel<KP>, dim3((unsigned)(xblocks + wblocks)), dim3(256), 0, stream, pdl, d, (int)xblocks,
                  wblocks, ws.x16, ws.w16, ws.scale, ws.xs);
}

}  // namespace

// Rows per tile (a multiple of 32), by the least time over the 74 pairs of SMs: a k-block's MMAs take 2 bn cycles
// (8 % more measured); besides, both passes' starts and the last tile's epilogue, and pass 1, which
// writes at 3.9 TB/s (as fast as a fill of the same size does).
DensePlan dense_plan(int N, int K, int M)
{
    const int64_t mt = ((int64_t)M + 255) / 256, nkb = ((int64_t)K + kDK - 1) / kDK;
    DensePlan best = {0, 0, 0.0};
    for (int bn = 256; bn >= 96; bn -= 32) {
        const int64_t tiles = mt * (((int64_t)N + bn - 1) / bn);
        if (tiles > INT32_MAX) continue;
        const double c = (double)((tiles + 73) / 74) * (1.08 * (double)nkb * 2 * bn + 2500) + 22000 +
                         4.6e-4 * 2.0 * (double)K * ((double)N + (double)M);
        if (best.tiles == 0 || c < best.cost) best = DensePlan{bn, (int)tiles, c};
    }
    return best;
}

size_t dense_workspace(int N, int K, int M) { return dense_layout(N, K, M, nullptr).bytes; }

rb_status dense_run(const DenseArgs& d, const void* epilogue, void* workspace, bool pdl, cudaStream_t stream)
{
    const DensePlan p = dense_plan(d.N, d.K, d.M);
    if (p.tiles == 0) return RB_ERR_UNSUPPORTED;
    const DenseWs ws = dense_layout(d.N, d.K, d.M, workspace);
    rb_status st;
    switch (d.kp) {
        case 1: st = launch_expand<1>(d, ws, pdl, stream); break;
        case 2: st = launch_expand<2>(d, ws, pdl, stream); break;
        case 3: st = launch_expand<3>(d, ws, pdl, stream); break;
        case 4: st = launch_expand<4>(d, ws, pdl, stream); break;
        case 5: st = launch_expand<5>(d, ws, pdl, stream); break;
        case 6: st = launch_expand<6>(d, ws, pdl, stream); break;
        case 7: st = launch_expand<7>(d, ws, pdl, stream); break;
        default: st = launch_expand<8>(d, ws, pdl, stream); break;
    }
    if (st != RB_OK) return st;
    DenseKernelArgs a;
    a.ep = *static_cast<const LinEp*>(epilogue);
    a.ep.xs = ws.xs;
    a.scale = ws.scale;
    a.dev_status = d.dev_status;
    a.N = d.N;
    a.K = d.K;
    a.M = d.M;
    a.mt = (int)(((int64_t)d.M + 255) / 256);
    a.bn = p.bn;
    a.tiles = p.tiles;
    const int pairs = num_sms() / 2;
    CUtensorMap mx, mw;
    if (!encode_fp16(&mx, ws.x16, d.M, d.K, kDTok) || !encode_fp16(&mw, ws.w16, d.N, d.K, a.bn / 2)) return RB_ERR_CUDA;
    static std::atomic<bool> attr_set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return RB_ERR_CUDA;
    if (dev >= 64 || !attr_set[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(dense_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDSmem) != cudaSuccess)
            return RB_ERR_CUDA;
        if (dev < 64) attr_set[dev].store(true, std::memory_order_release);
    }
    const int np = a.tiles < pairs ? a.tiles : pairs;
    return launch(dense_kernel, dim3((unsigned)(2 * np)), dim3(kDThreads), (size_t)kDSmem, stream, true, mx, mw, a);
}

}  // namespace rbw
