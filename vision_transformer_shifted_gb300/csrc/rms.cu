// Root-mean-square norm of the residual stream: s = x + residual (stored in
// bf16), y = s r gamma with r = 1 / sqrt(mean s^2 + eps); output in bf16 or in
// e4m3 with one scale a row; backward.
//
// All three kernels read every input once and write every output once, with
// the row held in registers between the statistics and the output: HBM bounds
// them.  Rows of up to 1024 channels lie on part of a warp (a power of two of
// lanes, at most four 16-byte pieces each: their loads are all in flight at
// once and the statistics need shuffles only); longer rows take a block each.
// (The backward, with three inputs, at most three pieces a lane.)  With residual,
// 200704 x 96: 23.6 us, 6.5 TB/s; to e4m3, 8191 x 4096: 37.4 us, 6.3 TB/s;
// backward 589824 x 192 with dsum: 135 us, 6.7 TB/s.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cuda_fp8.h>
#include <new>

#include "swin_rms.h"
#include "common.cuh"
#include "gelu.cuh"
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
// The same over group `group` of a block, of `threads` threads that meet at a
// barrier of their own; red: two rows of 16 sums a group, used in turn.
__device__ __forceinline__ void group_sum2(float &a, float &b, int threads, int group, int turn, float2 *red)
{
    lane_sum2(a, b, 32);
    const int warps = threads >> 5, warp = (threadIdx.x - group * threads) >> 5;
    red += (2 * group + (turn & 1)) * 16;
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    a = b = 0.f;
    for (int w = 0; w < warps; ++w) {
        a += red[w].x;
        b += red[w].y;
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
    f2 sq2 = 0;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        Piece v = piece(s[k]);
        if (a.residual) {
            const Piece w = piece(t[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v.v[e] = add2(v.v[e], w.v[e]);
            s[k] = pack(v);
            v = piece(s[k]);   // the stored (rounded) sum is what the norm sees
            if (a.out_sum && row_ok && c < a.chunks) *reinterpret_cast<uint4 *>(a.out_sum + base + c * 8) = s[k];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sq2 = fma2(v.v[e], v.v[e], sq2);
    }
    float sq = sum2(sq2);
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
            Piece v = piece(s[k]);
            const Piece g = piece(gm[k]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v.v[e] = mul2(mul2(v.v[e], pack2(r)), g.v[e]);
            *reinterpret_cast<uint4 *>((bf16 *)a.out + base + c * 8) = pack(v);
        }
        return;
    }
    f2 y[CPL][4];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {   // (pieces behind the row are zeros)
        const Piece v = piece(s[k]), g = piece(gm[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[k][e] = mul2(mul2(v.v[e], pack2(r)), g.v[e]);
            float lo, hi;
            unpack2(y[k][e], lo, hi);
            amax = max_abs(amax, lo, hi);
        }
    }
    amax = row_reduce<MaxOp, BLOCK>(amax, a.lpr, red);
    float scale = max_nan(amax, MIN_AMAX) / E4M3_MAX;
    if (row_ok && li == 0) a.scales[row] = scale;
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
        if (!(row_ok && c < a.chunks)) continue;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float2 q;
            unpack2(quotient2(y[k][e], minus_b, inv), q.x, q.y);
            w[e] = __nv_cvt_float2_to_fp8x2(q, __NV_SATFINITE, __NV_E4M3);
        }
        *reinterpret_cast<uint2 *>((uint8_t *)a.out + base + c * 8) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
}

struct RmsBwdArgs {
    const bf16 *s, *dy, *dsum, *gamma;
    bf16 *dx;
    float *partial;   // [gridDim.x, C]: each block's share of dgamma (one block: dgamma itself)
    int rows, chunks;
    float inv_c, eps;
    int lanes;        // of a row: of a warp, or (wide rows) threads
};

// The backward, dx = r (a - n mean(a n)) + dsum with n = s r, a = dy gamma, of a
// thread's piece of a row.  First its shares of sum s^2 and sum a s:
__device__ __forceinline__ void piece_sums(const Piece &s, const Piece &d, const Piece &g, f2 &sq, f2 &dot)
{
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        sq = fma2(s.v[e], s.v[e], sq);
        dot = fma2(mul2(d.v[e], g.v[e]), s.v[e], dot);
    }
}
// then, with q = mean(a n) r^2 (so that r n mean(a n) = s q), dx and its terms of
// dgamma (dy r s).
template <bool DSUM>
__device__ __forceinline__ uint4 piece_grad(const Piece &s, const Piece &d, const Piece &g, const Piece &m, f2 r, f2 minus_q,
                                            Piece &acc)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 dr = mul2(d.v[e], r);
        acc.v[e] = fma2(dr, s.v[e], acc.v[e]);
        const f2 t = DSUM ? fma2(dr, g.v[e], m.v[e]) : mul2(dr, g.v[e]);
        float lo, hi;
        unpack2(fma2(s.v[e], minus_q, t), lo, hi);
        w[e] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
// Blocks of 256 threads on an SM: enough bytes of loads in flight, and no more
// (200000 x 512 with dsum, two pieces a lane: 130.5 us with two blocks, 131.5
// with three, 142 with four; without dsum 114, 103 and 96; 589824 x 192 without
// dsum, three pieces: 112 with two, 125 with three).
constexpr int blocks_per_sm(int cpl, bool dsum) { return cpl > 2 || (cpl == 2 && dsum) ? 2 : 4; }

// Rows on part of a warp: a block takes 8 * (32 / lanes) rows together, then the
// ones gridDim.x on.  Each thread keeps the columns it owns of dgamma in
// registers over its rows; the block writes one partial row at the end.
template <int CPL, bool DSUM>
__global__ void __launch_bounds__(256, blocks_per_sm(CPL, DSUM)) rms_backward_kernel(RmsBwdArgs a)
{
    extern __shared__ float part[];   // [8 warps][C]
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = a.lanes, li = lane % step;
    const int rpw = 32 / step, rpb = 8 * rpw;
    Piece acc[CPL];
    uint4 g[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        g[k] = c < a.chunks ? ld16(a.gamma + c * 8) : make_uint4(0, 0, 0, 0);
        acc[k] = Piece{};
    }
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.rows; r0 += (int64_t)gridDim.x * rpb) {
        const int64_t row = r0 + warp * rpw + lane / step;
        const bool row_ok = row < a.rows;
        const int64_t base = row * a.chunks * 8;
        uint4 s[CPL], d[CPL], m[CPL];
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            const bool ok = row_ok && c < a.chunks;
            s[k] = ok ? ld16(a.s + base + c * 8) : make_uint4(0, 0, 0, 0);
            d[k] = ok ? ld16(a.dy + base + c * 8) : make_uint4(0, 0, 0, 0);
            if (DSUM) m[k] = ok ? ld16(a.dsum + base + c * 8) : make_uint4(0, 0, 0, 0);
        }
        f2 sq2 = 0, dot2 = 0;
#pragma unroll
        for (int k = 0; k < CPL; ++k) piece_sums(piece(s[k]), piece(d[k]), piece(g[k]), sq2, dot2);
        float sq = sum2(sq2), dot = sum2(dot2);
        lane_sum2(sq, dot, step);
        // (the packed values stay, their fp32 forms are made again: registers
        // kept across the sums would halve the rows in flight)
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            forget(s[k]);
            forget(d[k]);
            forget(g[k]);
            if (DSUM) forget(m[k]);
        }
        // (no row: r = 0, since its columns' sums get zero times r, and with eps = 0
        // one over the root of its mean is infinite)
        const float r = row_ok ? rsqrtf(fmaf(sq, a.inv_c, a.eps)) : 0.f, q = dot * a.inv_c * r * r * r;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            const uint4 o = piece_grad<DSUM>(piece(s[k]), piece(d[k]), piece(g[k]), DSUM ? piece(m[k]) : Piece{}, pack2(r),
                                             pack2(-q), acc[k]);
            if (row_ok && c < a.chunks) *reinterpret_cast<uint4 *>(a.dx + base + c * 8) = o;
        }
    }
    // the warp's rows, then the block's warps
    const int C = a.chunks * 8;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        float sums[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack2(acc[k].v[e], sums[2 * e], sums[2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = sums[e];
            for (int o = 16; o >= step; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane < step && c < a.chunks) part[warp * C + c * 8 + e] = v;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < C; i += 256) {
        float v = 0.f;
        for (int w = 0; w < 8; ++w) v += part[w * C + i];
        a.partial[(int64_t)blockIdx.x * C + i] = v;
    }
}

// Wider rows: a group of warps a row, several groups a block (few blocks, since
// each writes a partial row of dgamma that is read again).  Every thread
// fetches its own pieces of the next row by asynchronous copies into its own
// place in shared memory, so that the latency of HBM is paid once, not once a
// row (3001 x 2744: 15.5 us; 20.8 with the rows loaded as they come, and 30010
// rows: 84.7 us one row ahead, 91 two).
template <int CPL, bool DSUM>
__global__ void __launch_bounds__(512, 1) rms_backward_wide_kernel(RmsBwdArgs a)
{
    constexpr int ARRAYS = DSUM ? 3 : 2, DEPTH = 2;   // stages: a row, and the next
    extern __shared__ __align__(16) float part[];   // the pieces; at the end [C]
    __shared__ float2 red[2 * 16 * 16];
    griddep_launch_dependents();
    griddep_wait();
    const int step = a.lanes, group = (int)threadIdx.x / step, li = (int)threadIdx.x - group * step;
    const int rpb = (int)blockDim.x / step, C = a.chunks * 8;
    // this thread's piece k of array i in a stage at `at`: place(at, i, k)
    const uint32_t stride = blockDim.x * 16, stage = ARRAYS * CPL * stride;
    const uint32_t ring = smem_u32(part) + threadIdx.x * 16, ring_end = ring + DEPTH * stage;
    auto place = [&](uint32_t at, int i, int k) { return at + (uint32_t)(i * CPL + k) * stride; };
    bool have[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) have[k] = li + k * step < a.chunks;
    const int64_t first = (int64_t)blockIdx.x * rpb + group, hop = (int64_t)gridDim.x * rpb;
    int64_t ahead = first;   // the next row to fetch, and its stage
    uint32_t ahead_at = ring;
    auto fetch = [&]() {
        if (ahead < a.rows) {
            const int64_t off = ahead * C + li * 8;
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                if (!have[k]) continue;
                cp_async16(place(ahead_at, 0, k), a.s + off + k * step * 8, 16);
                cp_async16(place(ahead_at, 1, k), a.dy + off + k * step * 8, 16);
                if (DSUM) cp_async16(place(ahead_at, 2, k), a.dsum + off + k * step * 8, 16);
            }
        }
        cp_async_commit();
        ahead += hop;
        ahead_at += stage;
        if (ahead_at == ring_end) ahead_at = ring;
    };
#pragma unroll
    for (int d = 0; d < DEPTH - 1; ++d) fetch();
    Piece acc[CPL], g[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        g[k] = piece(have[k] ? ld16(a.gamma + (li + k * step) * 8) : make_uint4(0, 0, 0, 0));
        acc[k] = Piece{};
    }
    uint32_t at = ring;
    int turn = 0;
#pragma unroll 1
    for (int64_t row = first; row < a.rows; row += hop) {   // (the same for a group's threads)
        fetch();
        cp_async_wait<DEPTH - 1>();
        f2 sq2 = 0, dot2 = 0;
#pragma unroll
        for (int k = 0; k < CPL; ++k)
            if (have[k]) piece_sums(piece(lds16(place(at, 0, k))), piece(lds16(place(at, 1, k))), g[k], sq2, dot2);
        float sq = sum2(sq2), dot = sum2(dot2);
        group_sum2(sq, dot, step, group, turn++, red);
        const float r = rsqrtf(fmaf(sq, a.inv_c, a.eps)), q = dot * a.inv_c * r * r * r;
        bf16 *dx = a.dx + row * C + li * 8;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            if (!have[k]) continue;
            const Piece m = DSUM ? piece(lds16(place(at, 2, k))) : Piece{};
            *reinterpret_cast<uint4 *>(dx + k * step * 8) = piece_grad<DSUM>(
                piece(lds16(place(at, 0, k))), piece(lds16(place(at, 1, k))), g[k], m, pack2(r), pack2(-q), acc[k]);
        }
        at += stage;
        if (at == ring_end) at = ring;
    }
    __syncthreads();   // (every group is done with its pieces)
    // the groups add theirs in turn
    for (int t = 0; t < rpb; ++t) {
        if (group == t)
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                const int c = li + k * step;
                if (c >= a.chunks) continue;
                float4 *p = reinterpret_cast<float4 *>(part + c * 8);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float4 v;
                    unpack2(acc[k].v[2 * h], v.x, v.y);
                    unpack2(acc[k].v[2 * h + 1], v.z, v.w);
                    const float4 old = t ? p[h] : make_float4(0.f, 0.f, 0.f, 0.f);
                    p[h] = make_float4(old.x + v.x, old.y + v.y, old.z + v.z, old.w + v.w);
                }
            }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < C; i += blockDim.x) a.partial[(int64_t)blockIdx.x * C + i] = part[i];
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

// How a row of `chunks` 16-byte pieces is laid out: on part of a warp where at
// most `most` pieces a lane suffice, by the count of pieces that leaves the
// fewest lanes idle (the larger of equals: more loads in flight a thread); else on as few warps as leave each thread at most `most`
// (more, up to four, where 512 threads are not enough for that).
struct RowPlan {
    bool block;
    int lanes;     // of a row: of a warp, or threads
    int cpl;
};
RowPlan plan_row(int chunks, int most, int block_most)
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
constexpr int FWD_PIECES = 4, BWD_PIECES = 3, BWD_BLOCK_PIECES = 4;
constexpr int MAX_GROUPS = 15;   // row groups of a block: a block has 16 barriers, and one is everybody's

template <bool Q8>
cudaError_t launch_rms_forward(RmsArgs a, cudaStream_t stream)
{
    // rows that leave SMs idle take as many threads as pieces: the latency of
    // one row counts then (1 x 2048: 5.6 us on 64 threads)
    const int most = a.rows < sm_count() ? 1 : FWD_PIECES;
    const RowPlan p = plan_row(a.chunks, most, most);
    a.lpr = p.block ? 32 : p.lanes;
    const int threads = p.block ? p.lanes : 256;
    const int64_t rpb = p.block ? 1 : 8 * (32 / p.lanes);
    const unsigned grid = (unsigned)((a.rows + rpb - 1) / rpb);
#define SWIN_RMS_CASE(n)                                                                      \
    case n:                                                                                   \
        return launch_maybe_overlapped(p.block ? rms_forward_kernel<n, true, Q8>              \
                                               : rms_forward_kernel<n, false, Q8>,            \
                                       dim3(grid), dim3(threads), 0, stream, 1, a);
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

// The backward's launch: as many blocks as the SMs hold at once, each walking
// its share of the rows.  (A wide row's block is an SM's only one, of up to 512
// threads with three or four pieces each: with two on 1024 threads, what a
// thread spends on a row beside its pieces took 1 of 18 us.)
struct BwdPlan {
    RowPlan row;
    int threads, grid;
    size_t smem;
};
BwdPlan plan_backward(int rows, int C, bool with_dsum)
{
    const int chunks = C / 8;
    BwdPlan p{};
    p.row = plan_row(chunks, BWD_PIECES, BWD_BLOCK_PIECES);
    const RowPlan &r = p.row;
    int64_t rpb, per_sm;
    if (r.block) {
        const int groups = 512 / r.lanes;
        rpb = groups < MAX_GROUPS ? groups : MAX_GROUPS;
        per_sm = 1;
        p.threads = (int)rpb * r.lanes;
        p.smem = (size_t)p.threads * (with_dsum ? 3 : 2) * 2 * r.cpl * 16;   // (at most 192 KB)
        if (p.smem < (size_t)C * sizeof(float)) p.smem = (size_t)C * sizeof(float);
    } else {
        rpb = 8 * (32 / r.lanes);
        per_sm = blocks_per_sm(r.cpl, with_dsum);
        p.threads = 256;
        p.smem = (size_t)8 * C * sizeof(float);
    }
    const int64_t want = (rows + rpb - 1) / rpb, most = sm_count() * per_sm;
    // few rows: one block, whose sums are dgamma (two turns at most: less than what
    // the second launch would cost)
    p.grid = want <= 2 ? 1 : (int)(want < most ? want : most);
    return p;
}

cudaError_t launch_rms_backward(RmsBwdArgs a, const BwdPlan &p, float *dgamma, cudaStream_t stream)
{
    const RowPlan &r = p.row;
    a.lanes = r.lanes;
    const int C = a.chunks * 8;
    void (*kern)(RmsBwdArgs) = nullptr;
    if (r.block)
        kern = a.dsum ? (r.cpl == 3 ? rms_backward_wide_kernel<3, true> : rms_backward_wide_kernel<4, true>)
                      : (r.cpl == 3 ? rms_backward_wide_kernel<3, false> : rms_backward_wide_kernel<4, false>);
    else if (a.dsum)
        kern = r.cpl == 1 ? rms_backward_kernel<1, true> : r.cpl == 2 ? rms_backward_kernel<2, true> : rms_backward_kernel<3, true>;
    else
        kern = r.cpl == 1 ? rms_backward_kernel<1, false>
                          : r.cpl == 2 ? rms_backward_kernel<2, false> : rms_backward_kernel<3, false>;
    cudaError_t e;
    // (always the most any call needs: another thread may be between its setting
    // and its launch)
    if (r.block &&
        (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 512 * 6 * r.cpl * 16)) != cudaSuccess)
        return e;
    e = launch_maybe_overlapped(kern, dim3(p.grid), dim3(p.threads), p.smem, stream, 1, a);
    if (e != cudaSuccess || p.grid == 1) return e;
    return launch_maybe_overlapped(column_sum_kernel, dim3((C + 31) / 32), dim3(1024), 0, stream, 1,
                                   (const float *)a.partial, p.grid, C, dgamma);
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
    const BwdPlan p = plan_backward(rows, h->C, dsum != nullptr);
    void *ws = nullptr;
    bool captured = false;
    if (p.grid > 1 &&
        (rc = ows_begin(&h->ws, (size_t)p.grid * h->C * sizeof(float), st, &ws, &captured)) != SWIN_WATTN_OK)
        return rc;
    RmsBwdArgs a{};
    a.s = (const bf16 *)s;
    a.dy = (const bf16 *)dy;
    a.dsum = (const bf16 *)dsum;
    a.gamma = (const bf16 *)gamma;
    a.dx = (bf16 *)dx;
    a.partial = p.grid > 1 ? (float *)ws : dgamma;
    a.rows = rows;
    a.chunks = h->C / 8;
    a.inv_c = 1.f / (float)h->C;
    a.eps = h->eps;
    h->last_launches = p.grid > 1 ? 2 : 1;
    rc = cuda_status(launch_rms_backward(a, p, dgamma, st));
    const int rc2 = ows_end(&h->ws, st, ws, captured);
    return rc != SWIN_WATTN_OK ? rc : rc2;
}

} // extern "C"
