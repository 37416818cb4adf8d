// Root-mean-square norm of the residual stream: s = x + residual (stored in
// bf16), y = s r gamma with r = 1 / sqrt(mean s^2 + eps); output in bf16 or in
// e4m3 with one scale a row; backward.
//
// All three kernels read every input once and write every output once, with
// the row held in registers between the statistics and the output: HBM bounds
// them.  Rows of up to 1024 channels lie on part of a warp (a power of two of
// lanes, at most four 16-byte pieces each: their loads are all in flight at
// once and the statistics need shuffles only); longer rows take a block each.
// (The backward, with three inputs, at most two pieces a lane.)
#include <cmath>
#include <cuda_fp8.h>
#include <new>

#include "swin_rms.h"
#include "common.cuh"
#include "ptx.cuh"

using namespace swin;

namespace {

constexpr int MAX_C = 16384;
constexpr float E4M3_MAX = 448.f;
constexpr float MIN_AMAX = 1e-30f;   // floor of a row's largest magnitude under its scale

struct RmsArgs {
    const bf16 *x, *residual, *gamma;
    bf16 *out_sum;
    void *out;       // bf16 [rows, C], or e4m3 codes
    float *scales;   // e4m3: [rows]
    int rows, chunks;   // chunks = C / 8
    float inv_c, eps;
    int lpr;         // lanes per row (rows on part of a warp)
};

// Maximum that returns NaN if either argument is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

struct AddOp {
    static __device__ __forceinline__ float run(float a, float b) { return a + b; }
};
struct MaxOp {
    static __device__ __forceinline__ float run(float a, float b) { return max_nan(a, b); }
};

// Reduces v over the lanes of a row: lpr lanes of a warp, or the whole block
// (BLOCK; `red` holds a float a warp, and the call ends with every thread past
// its reads of it).
template <class Op, bool BLOCK>
__device__ __forceinline__ float row_reduce(float v, int lpr, float *red)
{
    const int lanes = BLOCK ? 32 : lpr;
    for (int o = lanes >> 1; o > 0; o >>= 1) v = Op::run(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (BLOCK) {
        const int warps = blockDim.x >> 5;
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = red[0];
        for (int w = 1; w < warps; ++w) v = Op::run(v, red[w]);
        __syncthreads();
    }
    return v;
}

// The sums of a and b over the lanes of a row.
template <bool BLOCK>
__device__ __forceinline__ void row_sum2(float &a, float &b, int lpr, float2 *red)
{
    const int lanes = BLOCK ? 32 : lpr;
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (BLOCK) {
        const int warps = blockDim.x >> 5;
        __syncthreads();   // (the previous row's sums have been read)
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        a = b = 0.f;
        for (int w = 0; w < warps; ++w) {
            a += red[w].x;
            b += red[w].y;
        }
    }
}

__device__ __forceinline__ void unpack8(const uint4 &u, float (&v)[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = unpack_bf16x2(w[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
    }
}

// The compiler takes u for a new value from here on.
__device__ __forceinline__ void forget(uint4 &u) { asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w)); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

__device__ __forceinline__ const uint4 &ld16(const bf16 *p) { return *reinterpret_cast<const uint4 *>(p); }

template <int CPL, bool BLOCK, bool Q8>
__global__ void __launch_bounds__(BLOCK ? 512 : 256) rms_forward_kernel(RmsArgs a)
{
    __shared__ float red[16];
    griddep_launch_dependents();
    griddep_wait();   // (nothing is read before the kernels queued earlier are done)
    const int lane = threadIdx.x & 31;
    const int step = BLOCK ? (int)blockDim.x : a.lpr;
    const int li = BLOCK ? (int)threadIdx.x : lane % a.lpr;
    const int64_t row = BLOCK ? (int64_t)blockIdx.x
                              : ((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * (32 / a.lpr) +
                                    lane / a.lpr;
    const bool row_ok = row < a.rows;
    const int64_t base = row * a.chunks * 8;
    uint4 s[CPL], t[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        const bool ok = row_ok && c < a.chunks;
        s[k] = ok ? ld16(a.x + base + c * 8) : make_uint4(0, 0, 0, 0);
        if (a.residual) t[k] = ok ? ld16(a.residual + base + c * 8) : make_uint4(0, 0, 0, 0);
    }
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        float v[8];
        unpack8(s[k], v);
        if (a.residual) {
            float w[8];
            unpack8(t[k], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += w[e];
            s[k] = pack8(v);
            unpack8(s[k], v);   // the stored (rounded) sum is what the norm sees
            if (a.out_sum && row_ok && c < a.chunks) *reinterpret_cast<uint4 *>(a.out_sum + base + c * 8) = s[k];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sq = fmaf(v[e], v[e], sq);
    }
    uint4 gm[CPL];   // (asked for before the row's sum is known)
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        gm[k] = row_ok && c < a.chunks ? ld16(a.gamma + c * 8) : make_uint4(0, 0, 0, 0);
    }
    sq = row_reduce<AddOp, BLOCK>(sq, a.lpr, red);
    const float r = rsqrtf(fmaf(sq, a.inv_c, a.eps));
    if (!Q8) {
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            if (!(row_ok && c < a.chunks)) continue;
            float v[8], g[8];
            unpack8(s[k], v);
            unpack8(gm[k], g);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * r * g[e];
            *reinterpret_cast<uint4 *>((bf16 *)a.out + base + c * 8) = pack8(v);
        }
        return;
    }
    float y[CPL][8];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        const bool ok = row_ok && c < a.chunks;
        float g[8];
        unpack8(s[k], y[k]);
        unpack8(gm[k], g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            y[k][e] = y[k][e] * r * g[e];
            if (ok) amax = max_nan(amax, fabsf(y[k][e]));
        }
    }
    amax = row_reduce<MaxOp, BLOCK>(amax, a.lpr, red);
    const float scale = max_nan(amax, MIN_AMAX) / E4M3_MAX, inv = 1.f / scale;
    if (row_ok && li == 0) a.scales[row] = scale;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        if (!(row_ok && c < a.chunks)) continue;
        uint32_t w[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const float *v = &y[k][4 * q];
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[0] * inv, v[1] * inv), __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[2] * inv, v[3] * inv), __NV_SATFINITE, __NV_E4M3);
            w[q] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2 *>((uint8_t *)a.out + base + c * 8) = make_uint2(w[0], w[1]);
    }
}

struct RmsBwdArgs {
    const bf16 *s, *dy, *dsum, *gamma;
    bf16 *dx;
    float *partial;   // [gridDim.x, C]: each block's share of dgamma
    int rows, chunks;
    float inv_c, eps;
    int lpr;
};

// dx = r (a - n mean(a n)) + dsum with n = s r, a = dy gamma.  A block walks
// rows blockIdx.x, blockIdx.x + gridDim.x, ... (groups of rows where a row is
// part of a warp); each thread keeps the columns it owns of dgamma in
// registers over its rows, and the block writes one partial row at the end.
template <int CPL, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : 256, BLOCK ? (CPL > 2 ? 1 : 2) : 3) rms_backward_kernel(RmsBwdArgs a)
{
    extern __shared__ float part[];   // !BLOCK: [8 warps][C]
    __shared__ float2 red[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int step = BLOCK ? (int)blockDim.x : a.lpr;
    const int li = BLOCK ? (int)threadIdx.x : lane % a.lpr;
    griddep_launch_dependents();
    griddep_wait();
    const int rpw = BLOCK ? 1 : 32 / a.lpr, rpb = BLOCK ? 1 : rpw * (int)(blockDim.x >> 5);
    float acc[CPL][8];
    uint4 g[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        g[k] = c < a.chunks ? ld16(a.gamma + c * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[k][e] = 0.f;
    }
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.rows; r0 += (int64_t)gridDim.x * rpb) {
        const int64_t row = BLOCK ? r0 : r0 + warp * rpw + lane / a.lpr;
        const bool row_ok = row < a.rows;
        const int64_t base = row * a.chunks * 8;
        uint4 s[CPL], d[CPL], m[CPL];
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            const bool ok = row_ok && c < a.chunks;
            s[k] = ok ? ld16(a.s + base + c * 8) : make_uint4(0, 0, 0, 0);
            d[k] = ok ? ld16(a.dy + base + c * 8) : make_uint4(0, 0, 0, 0);
            m[k] = ok && a.dsum ? ld16(a.dsum + base + c * 8) : make_uint4(0, 0, 0, 0);
        }
        float sq = 0.f, dot = 0.f;   // sum s^2, sum a s
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            float v[8], y[8], w[8];
            unpack8(s[k], v);
            unpack8(d[k], y);
            unpack8(g[k], w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                sq = fmaf(v[e], v[e], sq);
                dot = fmaf(y[e] * w[e], v[e], dot);
            }
        }
        row_sum2<BLOCK>(sq, dot, a.lpr, red);
        // (the packed values stay, their fp32 forms are made again: registers
        // kept across the sums would halve the rows in flight)
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            forget(s[k]);
            forget(d[k]);
            forget(g[k]);
            forget(m[k]);
        }
        const float r = rsqrtf(fmaf(sq, a.inv_c, a.eps));
        const float q = dot * a.inv_c * r * r;   // mean(a n) / s-scale: n mean(a n) = s q
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            float v[8], y[8], w[8], b[8];
            unpack8(s[k], v);
            unpack8(d[k], y);
            unpack8(g[k], w);
            unpack8(m[k], b);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[k][e] = fmaf(y[e], v[e] * r, acc[k][e]);
                b[e] = fmaf(r, y[e] * w[e] - v[e] * q, b[e]);
            }
            if (row_ok && c < a.chunks) *reinterpret_cast<uint4 *>(a.dx + base + c * 8) = pack8(b);
        }
    }
    const int C = a.chunks * 8;
    float *mine = a.partial + (int64_t)blockIdx.x * C;
    if constexpr (BLOCK) {
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            if (c >= a.chunks) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *reinterpret_cast<float4 *>(mine + c * 8 + 4 * q) =
                    make_float4(acc[k][4 * q], acc[k][4 * q + 1], acc[k][4 * q + 2], acc[k][4 * q + 3]);
        }
    } else {
        // the warp's rows, then the block's warps
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float v = acc[k][e];
                for (int o = 16; o >= step; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (lane < step && c < a.chunks) part[warp * C + c * 8 + e] = v;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < C; i += blockDim.x) {
            float v = 0.f;
            for (int w = 0; w < (int)(blockDim.x >> 5); ++w) v += part[w * C + i];
            mine[i] = v;
        }
    }
}

// out[c] = the sum of n partial rows, in a fixed order: 32 columns a block, 32
// threads a column.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, int n, int C, float *out)
{
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    griddep_launch_dependents();
    griddep_wait();
    float v = 0.f;
    if (c < C) {
#pragma unroll 8
        for (int i = w; i < n; i += 32) v += partial[(int64_t)i * C + c];
    }
    part[w][lane] = v;
    __syncthreads();
    // warp w adds column w of the block
    v = part[lane][w];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && blockIdx.x * 32 + w < C) out[blockIdx.x * 32 + w] = v;
}

// How a row of `chunks` 16-byte pieces is laid out: on the fewest lanes of a
// warp that leave each at most `most` pieces, or on a block of as few warps as
// leave each thread at most `most` (more, up to four, where 512 threads are
// not enough for that).
struct RowPlan {
    bool block;
    int lpr, threads, cpl;
};
RowPlan plan_row(int chunks, int most)
{
    RowPlan p{};
    if (chunks <= 32 * most) {
        p.lpr = 1;
        while (p.lpr * most < chunks) p.lpr <<= 1;
        p.threads = 256;
    } else {
        p.block = true;
        p.lpr = 32;
        p.threads = ((chunks + most - 1) / most + 31) / 32 * 32;
        if (p.threads > 512) p.threads = 512;
    }
    const int per = p.block ? p.threads : p.lpr;
    p.cpl = (chunks + per - 1) / per;
    return p;
}
// The backward keeps three inputs and a sum a column: two pieces a thread
// take 127 registers, four would spill.
constexpr int FWD_PIECES = 4, BWD_PIECES = 2;

template <bool Q8>
cudaError_t launch_rms_forward(RmsArgs a, cudaStream_t stream)
{
    // rows that leave SMs idle take as many threads as pieces: the latency of
    // one row counts then (1 x 2048: 5.6 us on 64 threads)
    const RowPlan p = plan_row(a.chunks, a.rows < sm_count() ? 1 : FWD_PIECES);
    a.lpr = p.lpr;
    const int64_t rpb = p.block ? 1 : (p.threads / 32) * (32 / p.lpr);
    const unsigned grid = (unsigned)((a.rows + rpb - 1) / rpb);
#define SWIN_RMS_CASE(n)                                                                      \
    case n:                                                                                   \
        return launch_maybe_overlapped(p.block ? rms_forward_kernel<n, true, Q8>              \
                                               : rms_forward_kernel<n, false, Q8>,            \
                                       dim3(grid), dim3(p.threads), 0, stream, 1, a);
    switch (p.cpl) {
        SWIN_RMS_CASE(1)
        SWIN_RMS_CASE(2)
        SWIN_RMS_CASE(3)
        SWIN_RMS_CASE(4)
    default:
        return cudaErrorInvalidValue;
    }
#undef SWIN_RMS_CASE
}

// Blocks of the backward: as many as the SMs hold at once, each walking its
// share of the rows.
int backward_grid(const RowPlan &p, int rows)
{
    const int64_t rpb = p.block ? 1 : (p.threads / 32) * (32 / p.lpr);
    const int64_t want = (rows + rpb - 1) / rpb, per_sm = !p.block ? 3 : p.cpl <= 2 ? 1024 / p.threads : 1;
    const int64_t most = sm_count() * per_sm;
    return (int)(want < most ? want : most);
}

cudaError_t launch_rms_backward(RmsBwdArgs a, int grid, const RowPlan &p, float *dgamma, cudaStream_t stream)
{
    a.lpr = p.lpr;
    const int C = a.chunks * 8;
    const size_t smem = p.block ? 0 : (size_t)(p.threads / 32) * C * sizeof(float);
    void (*kern)(RmsBwdArgs) = nullptr;
    if (p.block) kern = p.cpl <= 2 ? rms_backward_kernel<2, true> : p.cpl == 3 ? rms_backward_kernel<3, true> : rms_backward_kernel<4, true>;
    else kern = p.cpl == 1 ? rms_backward_kernel<1, false> : rms_backward_kernel<2, false>;
    const cudaError_t e = launch_maybe_overlapped(kern, dim3(grid), dim3(p.threads), smem, stream, 1, a);
    if (e != cudaSuccess) return e;
    return launch_maybe_overlapped(column_sum_kernel, dim3((C + 31) / 32), dim3(1024), 0, stream, 1,
                                   (const float *)a.partial, grid, C, dgamma);
}

bool bad_pointer(const void *p, bool required)
{
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) != 0 : required;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SWIN_WATTN_OK : SWIN_WATTN_ECUDA; }

} // namespace

struct swin_block_rms_s {
    int C;
    float eps;
    int device;   // -1: not bound yet
    int last_launches;
    OrderedWorkspace ws;   // the backward's partial sums of dgamma
};

namespace {

// Checks shared by the two forward forms; `out_bytes` of one output element.
int check_forward(const swin_block_rms_s *h, const void *x, const void *residual, int rows, const void *gamma,
                  const void *out_sum, const void *out, int64_t out_bytes)
{
    if (!h || rows < 0) return SWIN_WATTN_EINVAL;
    if (rows == 0) return SWIN_WATTN_OK;   // (an empty tensor may have no address)
    if (bad_pointer(x, true) || bad_pointer(residual, false) || bad_pointer(gamma, true) ||
        bad_pointer(out_sum, false) || bad_pointer(out, true) || (out_sum && !residual))
        return SWIN_WATTN_EINVAL;
    const int64_t n = (int64_t)rows * h->C, in = 2 * n, on = out_bytes * n;
    const bool same_type = out_bytes == 2;
    // in place (the very same tensor) is fine, any other overlap is not
    for (const void *p : {x, residual}) {
        if (!p) continue;
        if (overlaps(p, in, out, on) && !(same_type && p == out)) return SWIN_WATTN_EINVAL;
        if (out_sum && overlaps(p, in, out_sum, in) && p != out_sum) return SWIN_WATTN_EINVAL;
    }
    if (overlaps(gamma, 2 * (int64_t)h->C, out, on)) return SWIN_WATTN_EINVAL;
    if (out_sum && (overlaps(out_sum, in, out, on) || overlaps(gamma, 2 * (int64_t)h->C, out_sum, in)))
        return SWIN_WATTN_EINVAL;
    return SWIN_WATTN_OK;
}

RmsArgs forward_args(const swin_block_rms_s *h, const void *x, const void *residual, int rows, const void *gamma,
                     void *out_sum, void *out, float *scales)
{
    RmsArgs a{};
    a.x = (const bf16 *)x;
    a.residual = (const bf16 *)residual;
    a.gamma = (const bf16 *)gamma;
    a.out_sum = (bf16 *)out_sum;
    a.out = out;
    a.scales = scales;
    a.rows = rows;
    a.chunks = h->C / 8;
    a.inv_c = 1.f / (float)h->C;
    a.eps = h->eps;
    return a;
}

} // namespace

extern "C" {

int swin_block_rms_create(swin_block_rms_t *out, int C, float eps)
{
    if (!out) return SWIN_WATTN_EINVAL;
    *out = nullptr;
    if (C <= 0 || C % 8 || C > MAX_C || !(eps >= 0.f) || std::isinf(eps)) return SWIN_WATTN_EINVAL;
    swin_block_rms_s *h = new (std::nothrow) swin_block_rms_s{};
    if (!h) return SWIN_WATTN_ENOMEM;
    h->C = C;
    h->eps = eps;
    h->device = -1;
    *out = h;
    return SWIN_WATTN_OK;
}

int swin_block_rms_destroy(swin_block_rms_t h)
{
    if (!h) return SWIN_WATTN_OK;
    ows_free(&h->ws);
    delete h;
    return SWIN_WATTN_OK;
}

int swin_block_rms_last_launches(swin_block_rms_t h) { return h ? h->last_launches : 0; }

int swin_block_rms_forward(swin_block_rms_t h, const void *x, const void *residual, int rows, const void *gamma,
                           void *out_sum, void *out, swin_stream_t stream)
{
    int rc = check_forward(h, x, residual, rows, gamma, out_sum, out, 2);
    if (rc != SWIN_WATTN_OK || rows == 0) return rc;
    if ((rc = bind_device(&h->device)) != SWIN_WATTN_OK) return rc;
    h->last_launches = 1;
    return cuda_status(launch_rms_forward<false>(forward_args(h, x, residual, rows, gamma, out_sum, out, nullptr),
                                                 (cudaStream_t)stream));
}

int swin_block_rms_forward_q8(swin_block_rms_t h, const void *x, const void *residual, int rows, const void *gamma,
                              void *out_sum, void *out8, float *scales, swin_stream_t stream)
{
    int rc = check_forward(h, x, residual, rows, gamma, out_sum, out8, 1);
    if (rc != SWIN_WATTN_OK || rows == 0) return rc;
    if (bad_pointer(scales, true)) return SWIN_WATTN_EINVAL;
    const int64_t n = (int64_t)rows * h->C, sn = 4 * (int64_t)rows;
    if (overlaps(scales, sn, x, 2 * n) || overlaps(scales, sn, residual, residual ? 2 * n : 0) ||
        overlaps(scales, sn, out_sum, out_sum ? 2 * n : 0) || overlaps(scales, sn, out8, n) ||
        overlaps(scales, sn, gamma, 2 * (int64_t)h->C))
        return SWIN_WATTN_EINVAL;
    if ((rc = bind_device(&h->device)) != SWIN_WATTN_OK) return rc;
    h->last_launches = 1;
    return cuda_status(launch_rms_forward<true>(forward_args(h, x, residual, rows, gamma, out_sum, out8, scales),
                                                (cudaStream_t)stream));
}

int swin_block_rms_backward(swin_block_rms_t h, const void *s, int rows, const void *gamma, const void *dy,
                            const void *dsum, void *dx, float *dgamma, swin_stream_t stream)
{
    if (!h || rows < 0) return SWIN_WATTN_EINVAL;
    if (rows == 0) {
        if (bad_pointer(dgamma, true)) return SWIN_WATTN_EINVAL;
        const int rc = bind_device(&h->device);
        return rc != SWIN_WATTN_OK ? rc : cuda_status(cudaMemsetAsync(dgamma, 0, 4 * (size_t)h->C, (cudaStream_t)stream));
    }
    if (bad_pointer(s, true) || bad_pointer(gamma, true) || bad_pointer(dy, true) || bad_pointer(dsum, false) ||
        bad_pointer(dx, true) || bad_pointer(dgamma, true))
        return SWIN_WATTN_EINVAL;
    const int64_t n = 2 * (int64_t)rows * h->C, gn = 2 * (int64_t)h->C;
    if (overlaps(s, n, dx, n) || (overlaps(dy, n, dx, n) && dy != dx) ||
        (dsum && overlaps(dsum, n, dx, n) && dsum != dx) || overlaps(gamma, gn, dx, n))
        return SWIN_WATTN_EINVAL;
    for (const void *p : {s, dy, dsum, (const void *)dx})
        if (p && overlaps(p, n, dgamma, 2 * gn)) return SWIN_WATTN_EINVAL;
    if (overlaps(gamma, gn, dgamma, 2 * gn)) return SWIN_WATTN_EINVAL;
    int rc = bind_device(&h->device);
    if (rc != SWIN_WATTN_OK) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    const RowPlan p = plan_row(h->C / 8, BWD_PIECES);
    const int grid = backward_grid(p, rows);
    void *ws = nullptr;
    bool captured = false;
    if ((rc = ows_begin(&h->ws, (size_t)grid * h->C * sizeof(float), st, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    RmsBwdArgs a{};
    a.s = (const bf16 *)s;
    a.dy = (const bf16 *)dy;
    a.dsum = (const bf16 *)dsum;
    a.gamma = (const bf16 *)gamma;
    a.dx = (bf16 *)dx;
    a.partial = (float *)ws;
    a.rows = rows;
    a.chunks = h->C / 8;
    a.inv_c = 1.f / (float)h->C;
    a.eps = h->eps;
    h->last_launches = 2;
    rc = cuda_status(launch_rms_backward(a, grid, p, dgamma, st));
    const int rc2 = ows_end(&h->ws, st, ws, captured);
    return rc != SWIN_WATTN_OK ? rc : rc2;
}

} // extern "C"
