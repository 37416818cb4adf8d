// What the kernels of the row norms (rms.cu, layernorm.cu) share: a row in
// pieces of eight channels on part of a warp or on a block, its sums, its e4m3
// codes, and the sum of partial rows.
#pragma once

#include <cfloat>
#include <climits>
#include <cuda_fp8.h>

#include "common.cuh"
#include "gelu.cuh"
#include "ptx.cuh"

namespace swin {

constexpr int NORM_MAX_C = 16384;
constexpr float E4M3_MAX = 448.f;
constexpr float MIN_AMAX = 1e-30f;   // floor of a row's largest magnitude under its scale

// Maximum that returns NaN if either argument is one.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The same of three magnitudes.
__device__ __forceinline__ float max_abs(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
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

// The sums of a and b over `lanes` lanes of a warp.
__device__ __forceinline__ void lane_sum2(float &a, float &b, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
}
__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr) : "memory");
    return u;
}

// The compiler takes u for a new value from here on.
__device__ __forceinline__ void forget(uint4 &u) { asm volatile("" : "+r"(u.x), "+r"(u.y), "+r"(u.z), "+r"(u.w)); }

__device__ __forceinline__ const uint4 &ld16(const bf16 *p) { return *reinterpret_cast<const uint4 *>(p); }

// One thread's piece of a row, eight channels, as pairs.
struct Piece {
    f2 v[4];
};
__device__ __forceinline__ Piece piece(const uint4 &u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Piece p;
#pragma unroll
    for (int e = 0; e < 4; ++e) p.v[e] = pack2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
    return p;
}
__device__ __forceinline__ uint4 pack(const Piece &p)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float lo, hi;
        unpack2(p.v[e], lo, hi);
        w[e] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum2(f2 v)
{
    float a, b;
    unpack2(v, a, b);
    return a + b;
}

// y / b for two values, correctly rounded, with inv = 1 / b correctly rounded:
// y inv is within 1.5 units of the last place; one correction by the remainder y
// - q b makes that less than one, and the next is then exact (P. W. Markstein,
// Computation of elementary functions on the IBM RISC System/6000 processor,
// 1990).  For b from 1e-24, where the remainder of every quotient that is not
// rounded to zero is a number with all of its bits, to the largest finite one.
// (A product with inv alone gives a neighbouring code once in 20,000 values, 36.9
// us at 8191 x 4096; with the corrections 37.4, with divisions 46.5.)
__device__ __forceinline__ f2 quotient2(f2 y, f2 minus_b, f2 inv)
{
    f2 q = mul2(y, inv);
    q = fma2(fma2(q, minus_b, y), inv, q);
    return fma2(fma2(q, minus_b, y), inv, q);
}
// A row's values y, of largest magnitude amax, as e4m3 codes with the scale
// max(amax, MIN_AMAX) / 448 (NaN if a value is one).
template <int CPL>
__device__ __forceinline__ void store_codes(f2 (&y)[CPL][4], float amax, float *scale_out, bool row_ok, int li, int step,
                                            int chunks, uint8_t *out)
{
    float scale = max_nan(amax, MIN_AMAX) / E4M3_MAX;
    if (row_ok && li == 0) *scale_out = scale;
    // (outside quotient2's range: a small scale and its row times 2^64, exactly; an
    // infinite scale makes finite values zero, NaN everything NaN)
    if (!(scale >= 1e-24f && scale <= FLT_MAX)) {
        const bool small = scale < 1e-24f;
        const f2 up = pack2(small ? 0x1p64f : scale > FLT_MAX ? 0.f : scale);
#pragma unroll
        for (int k = 0; k < CPL; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[k][e] = mul2(y[k][e], up);
        scale = small ? scale * 0x1p64f : 1.f;
    }
    const f2 minus_b = pack2(-scale), inv = pack2(1.f / scale);
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        if (!(row_ok && c < chunks)) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 q;
            unpack2(quotient2(y[k][e], minus_b, inv), q.x, q.y);
            w[e] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
        }
        *reinterpret_cast<uint2 *>(out + c * 8) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
}

// out[c] = the sum of n partial rows, in a fixed order: 32 columns a block, 32
// threads a column.  Columns from `first` on go to `rest`.
static __global__ void __launch_bounds__(1024) column_sum_kernel(const float *partial, int n, int C, float *out, int first,
                                                                 float *rest)
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
    const int d = blockIdx.x * 32 + w;
    if (lane == 0 && d < C) (d < first ? out + d : rest + (d - first))[0] = v;
}
// How a row of `chunks` 16-byte pieces is laid out: on part of a warp where at
// most `most` pieces a lane suffice, by the count of pieces that leaves the
// fewest lanes idle (the larger of equals: more loads in flight a thread); else on as few warps as leave each thread at most `most`
// (more, up to four, where 512 threads are not enough for that).
struct RowPlan {
    bool block;
    int lanes;     // of a row: of a warp, or threads
    int cpl;
};
inline RowPlan plan_row(int chunks, int most, int block_most)
{
    RowPlan p{};
    if (chunks <= 32 * most) {
        int idle = INT_MAX;
        for (int cpl = 1; cpl <= most; ++cpl) {
            int lanes = 1;
            while (lanes * cpl < chunks) lanes <<= 1;
            if (lanes > 32 || lanes * cpl - chunks > idle) continue;
            idle = lanes * cpl - chunks;
            p.lanes = lanes;
            p.cpl = cpl;
        }
        return p;
    }
    p.block = true;
    p.lanes = ((chunks + block_most - 1) / block_most + 31) / 32 * 32;
    if (p.lanes > 512) p.lanes = 512;
    p.cpl = (chunks + p.lanes - 1) / p.lanes;
    return p;
}
} // namespace swin
