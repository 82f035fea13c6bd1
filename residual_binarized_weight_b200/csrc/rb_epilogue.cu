// rb_epilogue.cu -- gradient of the linear product's epilogue
// Y = act(P) .* mul + residual (rb_epilogue_backward):
//
//   dP = dY .* mul .* act'(P);   dmul = dY .* act(P);   dbias[n] = sum_m dP[m][n]
//
// One elementwise pass with column sums on the side, HBM-bound: with mul and
// dmul 10 bytes per element (2048 x 14336: 294 MB in 51.9 us with the second launch, in
// a graph: 88 % of the measured copy rate).  A CTA takes a strip of 32 vectors of 8 columns
// (one per lane) and a chunk of rows (warp w the rows w, w + 8, ...), so each
// warp reads and writes 512 consecutive bytes of a row, and each lane keeps the
// sums of its eight columns in registers.
//
// Rows whose stride is no multiple of 8 elements start at varying distances
// from a 16-byte boundary, but rows 8 apart at the same one.  A warp's vectors
// are therefore laid from the boundary at or before its rows' start, the
// same one for all its rows, and only a row's first and last vector are taken
// element by element.  That needs one stride modulo 8 for all arrays; arrays
// that differ there are read one element per lane.
//
// dbias: each CTA adds its warps' sums in warp order and writes one partial per
// column; a second launch adds the chunks in a fixed order (no atomics).  For a
// short batch the chunks are a cluster of at most 8 CTAs instead, whose first adds
// them from distributed shared memory: it is bound by its launches (eb_short).
#include "rbw_internal.cuh"
#include "rb_epilogue.cuh"

namespace rbw {
namespace {

constexpr int kEbWarps = 8;
constexpr int kStrip = 256;                        // columns per strip (32 lanes x 8)
constexpr int kStripSums = kStrip + 8;             // a strip's vectors may begin up to 7 columns before it
constexpr int kEbCluster = 8;                      // chunks of a short batch, at most
constexpr int kEbAhead = 4;                        // its rows in flight per thread

struct EbArgs {
    const uint16_t* dY;
    const uint16_t* P;
    const uint16_t* U;
    uint16_t* dP;
    uint16_t* dU;
    float* part;                                   // [chunks][strips][kStripSums], or null
    float* dbias;                                  // (short batches)
    int64_t ld_dy, ld_p, ld_u, ld_dp, ld_du;
    int M, N, rows;                                // rows per chunk, a multiple of 8
    int shift;                                     // common stride modulo 8, or -1: element by element
};

__device__ __forceinline__ void unpack8(float (&x)[8], const uint4& u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        x[2 * q] = __uint_as_float(w[q] << 16);
        x[2 * q + 1] = __uint_as_float(w[q] & 0xffff0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
        w[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int ACT, bool MUL>
__device__ __forceinline__ void eb_element(float dy, float p, float u, float& dp, float& du)
{
    float a, d;
    activate_slope<ACT>(p, a, d);
    du = dy * a;
    dp = (MUL ? dy * u : dy) * d;
}

// R rows of one vector: all their loads are made before the first is used.
template <int ACT, bool MUL, int R>
__device__ __forceinline__ void eb_rows(const EbArgs& A, int r0, int c, float (&sum)[8])
{
    uint4 y[R], p[R], u[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + i * kEbWarps;
        y[i] = __ldcs(reinterpret_cast<const uint4*>(A.dY + r * A.ld_dy + c));
        p[i] = __ldcs(reinterpret_cast<const uint4*>(A.P + r * A.ld_p + c));
        if constexpr (MUL) u[i] = __ldcs(reinterpret_cast<const uint4*>(A.U + r * A.ld_u + c));
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = r0 + i * kEbWarps;
        float fy[8], fp[8], fu[8], dp[8], du[8];
        unpack8(fy, y[i]);
        unpack8(fp, p[i]);
        if constexpr (MUL) unpack8(fu, u[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            eb_element<ACT, MUL>(fy[j], fp[j], MUL ? fu[j] : 1.0f, dp[j], du[j]);
            sum[j] += dp[j];
        }
        __stcs(reinterpret_cast<uint4*>(A.dP + r * A.ld_dp + c), pack8(dp));
        if (MUL && A.dU) __stcs(reinterpret_cast<uint4*>(A.dU + r * A.ld_du + c), pack8(du));
    }
}

// Element (r, c), which is inside the matrix.
template <int ACT, bool MUL>
__device__ __forceinline__ float eb_one(const EbArgs& A, int64_t r, int c)
{
    float dp, du;
    eb_element<ACT, MUL>(bf16_bits_to_f32(A.dY[r * A.ld_dy + c]), bf16_bits_to_f32(A.P[r * A.ld_p + c]),
                         MUL ? bf16_bits_to_f32(A.U[r * A.ld_u + c]) : 1.0f, dp, du);
    A.dP[r * A.ld_dp + c] = __bfloat16_as_ushort(__float2bfloat16_rn(dp));
    if (MUL && A.dU) A.dU[r * A.ld_du + c] = __bfloat16_as_ushort(__float2bfloat16_rn(du));
    return dp;
}

template <int ACT, bool MUL>
__global__ void __launch_bounds__(kEbWarps * 32)
epilogue_backward_kernel(const __grid_constant__ EbArgs A)
{
    __shared__ float sums[kEbWarps][kStripSums];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int strip = blockIdx.x, chunk = blockIdx.y;
    const int r0 = chunk * A.rows;
    const int r1 = min(r0 + A.rows, A.M);
    const int off = A.shift > 0 ? (warp * A.shift) & 7 : 0;   // the warp's rows start so far after a boundary
    float sum[8] = {};
    if (A.shift >= 0) {
        const int c = strip * kStrip + lane * 8 - off;
        if (c >= 0 && c + 8 <= A.N) {
            int r = r0 + warp;
            for (; r + kEbWarps < r1; r += 2 * kEbWarps) eb_rows<ACT, MUL, 2>(A, r, c, sum);
            if (r < r1) eb_rows<ACT, MUL, 1>(A, r, c, sum);
        } else if (c < A.N) {                      // a row's first or last vector
            for (int r = r0 + warp; r < r1; r += kEbWarps)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j >= 0 && c + j < A.N) sum[j] += eb_one<ACT, MUL>(A, r, c + j);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[warp][8 * lane + j - off + 8] = sum[j];
    } else {
        for (int r = r0 + warp; r < r1; r += kEbWarps)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = strip * kStrip + j * 32 + lane;
                if (c < A.N) sum[j] += eb_one<ACT, MUL>(A, r, c);
            }
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[warp][32 * j + lane + 8] = sum[j];
    }
    if (!A.part) return;
    __syncthreads();
    float* out = A.part + ((int64_t)chunk * gridDim.x + strip) * kStripSums;
    for (int x = threadIdx.x; x < kStripSums; x += kEbWarps * 32) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kEbWarps; ++w) {
            const int o = A.shift > 0 ? (w * A.shift) & 7 : 0;
            if (x >= 8 - o && x < kStripSums - o) t += sums[w][x];
        }
        out[x] = t;
    }
}

// A short batch: one column per lane, rows as above, the chunks of a column block a cluster whose first CTA
// adds their sums in order.
template <int ACT, bool MUL>
__global__ void __launch_bounds__(kEbWarps * 32)
epilogue_backward_short_kernel(const __grid_constant__ EbArgs A)
{
    __shared__ float sums[kEbWarps][32];
    __shared__ __align__(16) float recv[kEbCluster][32];
    cluster_arrive();                              // waited for before the first store to a peer
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, chunk = blockIdx.y;
    const int r1 = min((chunk + 1) * A.rows, A.M);
    float sum = 0.0f;
    if (c < A.N)
        for (int r0 = chunk * A.rows + warp; r0 < r1; r0 += kEbAhead * kEbWarps) {
            uint16_t y[kEbAhead], p[kEbAhead], u[kEbAhead];
#pragma unroll
            for (int i = 0; i < kEbAhead; ++i) {
                const int64_t r = min(r0 + i * kEbWarps, r1 - 1);
                y[i] = A.dY[r * A.ld_dy + c];
                p[i] = A.P[r * A.ld_p + c];
                if (MUL) u[i] = A.U[r * A.ld_u + c];
            }
#pragma unroll
            for (int i = 0; i < kEbAhead; ++i) {
                const int64_t r = r0 + i * kEbWarps;
                if (r >= r1) break;
                float dp, du;
                eb_element<ACT, MUL>(bf16_bits_to_f32(y[i]), bf16_bits_to_f32(p[i]), MUL ? bf16_bits_to_f32(u[i]) : 1.0f,
                                     dp, du);
                A.dP[r * A.ld_dp + c] = __bfloat16_as_ushort(__float2bfloat16_rn(dp));
                if (MUL && A.dU) A.dU[r * A.ld_du + c] = __bfloat16_as_ushort(__float2bfloat16_rn(du));
                sum += dp;
            }
        }
    sums[warp][lane] = sum;
    __syncthreads();
    cluster_wait();
    if (warp == 0) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kEbWarps; ++w) t += sums[w][lane];
        st_dsmem_f32(smem_u32(&recv[chunk][lane]), 0, t);
    }
    cluster_sync_all();
    if (chunk == 0 && warp == 0 && c < A.N) {
        float t = 0.0f;
        for (int k = 0; k < (int)gridDim.y; ++k) t += recv[k][lane];
        A.dbias[c] = t;
    }
}

// dbias[c] = the chunks' partials of column c, which lie in its strip and, for
// the strip's last columns, in the next one (whose vectors may begin before it).
// 32 columns per CTA; warp w adds chunks w, w + 8, ..., then the warps in order.
__global__ void __launch_bounds__(kEbWarps * 32)
dbias_kernel(const float* __restrict__ part, float* __restrict__ dbias, int N, int strips, int chunks, int shifted)
{
    __shared__ float s[kEbWarps][32];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int st = c / kStrip, x = c - st * kStrip + 8;
    const bool next = shifted && x - kStrip >= 1 && st + 1 < strips;
    float t = 0.0f;
    if (c < N)
#pragma unroll 4
        for (int k = warp; k < chunks; k += kEbWarps) {
            const float* p = part + ((int64_t)k * strips + st) * kStripSums;
            t += p[x];
            if (next) t += p[kStripSums + x - kStrip];
        }
    s[warp][lane] = t;
    __syncthreads();
    if (warp == 0 && c < N) {
        float u = 0.0f;
#pragma unroll
        for (int w = 0; w < kEbWarps; ++w) u += s[w][lane];
        dbias[c] = u;
    }
}

// Strips (one more where shifted vectors reach past the last), and chunks of a
// multiple of 8 rows: about eight CTAs for each of the 148 SMs where there are
// rows enough (16 and 32 write more partials: 53.9, 56.0 and 59.4 us at 2048 x 14336),
// at least 16 rows each.
struct EbPlan {
    int strips, rows, chunks;
};
EbPlan eb_plan(int M, int N, bool shifted)
{
    EbPlan p;
    p.strips = (int)(((int64_t)N + (shifted ? 7 : 0) + kStrip - 1) / kStrip);
    int64_t rows = ((int64_t)M * (((int64_t)N + kStrip - 1) / kStrip) / (148 * 8) + 7) / 8 * 8;
    const int64_t least = ((int64_t)M + 65534) / 65535;       // the grid's second dimension
    if (rows < least) rows = (least + 7) / 8 * 8;
    if (rows < 16) rows = 16;
    if (rows > M) rows = ((int64_t)M + 7) / 8 * 8;
    p.rows = (int)rows;
    p.chunks = (int)(((int64_t)M + p.rows - 1) / p.rows);
    return p;
}

// Whether one launch does.  One launch / two, us in a graph: 8 x 4096 2.4 / 3.7, 64 x 1027 2.5 / 5.9, 333 x 1027
// 3.6 / 6.7, 512 x 1024 3.9 / 4.6, 1024 x 512 4.9 / 4.9; many rows to a CTA lose (2048 x 256 6.3 / 5.5, 16384 x 32
// 35 / 21), and so do many CTAs (16 x 14336, 896 of them: 4.5 / 4.4, 32 x 16384 7.7 / 4.6).
bool eb_short(int M, int64_t N)
{
    const int64_t chunks = ((int64_t)M + 7) / 8 < kEbCluster ? ((int64_t)M + 7) / 8 : kEbCluster;
    return M <= 1024 && M * N <= (1 << 19) && (N + 31) / 32 * chunks <= 4 * 148;
}

template <int ACT>
rb_status eb_launch(const EbArgs& a, const EbPlan& p, bool pdl, cudaStream_t stream)
{
    const dim3 grid((unsigned)p.strips, (unsigned)p.chunks);
    if (a.dbias) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)((a.N + 31) / 32), (unsigned)p.chunks);
        cfg.blockDim = dim3(kEbWarps * 32);
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 1;
        attr[0].val.clusterDim.y = (unsigned)p.chunks;
        attr[0].val.clusterDim.z = 1;
        attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = pdl ? 2 : 1;
        const cudaError_t e = a.U ? cudaLaunchKernelEx(&cfg, epilogue_backward_short_kernel<ACT, true>, a)
                                  : cudaLaunchKernelEx(&cfg, epilogue_backward_short_kernel<ACT, false>, a);
        return e == cudaSuccess ? RB_OK : RB_ERR_CUDA;
    }
    return a.U ? launch(epilogue_backward_kernel<ACT, true>, grid, dim3(kEbWarps * 32), 0, stream, pdl, a)
               : launch(epilogue_backward_kernel<ACT, false>, grid, dim3(kEbWarps * 32), 0, stream, pdl, a);
}

}  // namespace
}  // namespace rbw

using namespace rbw;

extern "C" size_t rb_epilogue_backward_workspace_bytes(int M, int n_out)
{
    if (M < 1 || M > (1 << 30) || n_out < 1 || n_out > (1 << 30)) return 0;
    const EbPlan p = eb_plan(M, n_out, true);
    return (size_t)p.strips * (size_t)p.chunks * kStripSums * sizeof(float);
}

extern "C" rb_status rb_epilogue_backward(const rb_epilogue_grad_t* grad, int M, int n_out, void* workspace,
                                          size_t workspace_bytes, unsigned flags, cudaStream_t stream)
{
    if (!grad || grad->reserved != 0 || !good_act(grad->act) || (flags & ~RB_LAUNCH_PDL)) return RB_ERR_ARG;
    const rb_epilogue_grad_t& g = *grad;
    if (!g.dY || !g.preact || !g.dP || (g.dmul && !g.mul)) return RB_ERR_ARG;
    const int64_t N = n_out;
    if (M < 1 || M > (1 << 30) || N < 1 || N > (1 << 30) || g.ld_dy < N || g.ld_preact < N || g.ld_dp < N || (g.mul && g.ld_mul < N) ||
        (g.dmul && g.ld_dmul < N))
        return RB_ERR_SHAPE;
    const void* ptrs[] = {g.dY, g.preact, g.mul, g.dP, g.dmul, g.dbias};
    for (const void* q : ptrs)
        if (!aligned16(q)) return RB_ERR_ALIGN;
    if (g.dbias) {
        if (!workspace || workspace_bytes < rb_epilogue_backward_workspace_bytes(M, n_out)) return RB_ERR_WORKSPACE;
        if (!aligned16(workspace)) return RB_ERR_ALIGN;
    }
    // outputs against inputs and each other: only the same array, element for element
    struct Arr {
        const void* p;
        int64_t ld;
    };
    const Arr in[] = {{g.dY, g.ld_dy}, {g.preact, g.ld_preact}, {g.mul, g.ld_mul}};
    const Arr out[] = {{g.dP, g.ld_dp}, {g.dmul, g.ld_dmul}};
    for (int o = 0; o < 2; ++o) {
        if (!out[o].p) continue;
        const MatRange ro = mat_range(out[o].p, M, N, out[o].ld, 2);
        for (int i = 0; i < 3; ++i) {
            if (!in[i].p) continue;
            const bool may = o == 0 ? i < 2 : i == 2;
            if (may && out[o].p == in[i].p && out[o].ld == in[i].ld) continue;
            if (overlaps(ro, mat_range(in[i].p, M, N, in[i].ld, 2))) return RB_ERR_ARG;
        }
        if (o == 1 && overlaps(ro, mat_range(g.dP, M, N, g.ld_dp, 2))) return RB_ERR_ARG;
    }
    if (g.dbias) {
        const MatRange rb = mat_range(g.dbias, 1, N, N, 4);
        for (const Arr& q : in)
            if (q.p && overlaps(rb, mat_range(q.p, M, N, q.ld, 2))) return RB_ERR_ARG;
        const size_t need = rb_epilogue_backward_workspace_bytes(M, n_out);
        if (meets(rb, workspace, need)) return RB_ERR_ARG;
        for (const Arr& q : out)
            if (q.p && (overlaps(rb, mat_range(q.p, M, N, q.ld, 2)) || meets(mat_range(q.p, M, N, q.ld, 2), workspace, need)))
                return RB_ERR_ARG;
    }
    if (!device_is_sm100()) return RB_ERR_UNSUPPORTED;
    EbArgs a;
    a.dY = g.dY;
    a.P = g.preact;
    a.U = g.mul;
    a.dP = g.dP;
    a.dU = g.dmul;
    a.part = g.dbias ? static_cast<float*>(workspace) : nullptr;    // (unused by a short batch)
    a.ld_dy = g.ld_dy;
    a.ld_p = g.ld_preact;
    a.ld_u = g.ld_mul;
    a.ld_dp = g.ld_dp;
    a.ld_du = g.ld_dmul;
    a.M = M;
    a.N = n_out;
    a.shift = (int)(g.ld_dy & 7);
    const bool same = (g.ld_preact & 7) == a.shift && (g.ld_dp & 7) == a.shift &&
                      (!g.mul || (g.ld_mul & 7) == a.shift) && (!g.dmul || (g.ld_dmul & 7) == a.shift);
    const bool small = g.dbias && eb_short(M, N);
    if (!same) a.shift = -1;
    EbPlan p = eb_plan(M, n_out, a.shift > 0);
    if (small) {
        p.rows = (int)((((int64_t)M + kEbCluster - 1) / kEbCluster + 7) / 8 * 8);
        p.chunks = (int)(((int64_t)M + p.rows - 1) / p.rows);
    }
    a.dbias = small ? g.dbias : nullptr;
    a.rows = p.rows;
    const bool pdl = (flags & RB_LAUNCH_PDL) != 0;
    rb_status st;
    switch (g.act) {
        case RB_ACT_RELU: st = eb_launch<RB_ACT_RELU>(a, p, pdl, stream); break;
        case RB_ACT_SILU: st = eb_launch<RB_ACT_SILU>(a, p, pdl, stream); break;
        case RB_ACT_GELU: st = eb_launch<RB_ACT_GELU>(a, p, pdl, stream); break;
        case RB_ACT_GELU_TANH: st = eb_launch<RB_ACT_GELU_TANH>(a, p, pdl, stream); break;
        default: st = eb_launch<RB_ACT_NONE>(a, p, pdl, stream); break;
    }
    if (st != RB_OK || !g.dbias || small) return st;
    return launch(dbias_kernel, dim3((unsigned)((n_out + 31) / 32)), dim3(kEbWarps * 32), 0, stream, true,
                  (const float*)a.part, g.dbias, n_out, p.strips, p.chunks, a.shift > 0 ? 1 : 0);
}
