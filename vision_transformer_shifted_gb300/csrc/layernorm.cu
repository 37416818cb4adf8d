// Layer norm of the residual stream: s = x + residual (stored in bf16), y = (s -
// mu) r gamma + beta with r = 1 / sqrt(var + eps); output in bf16, in e4m3 with
// one scale a row, or added to the residual (post-norm); backward.
//
// As the root-mean-square norm (rms.cu): every input is read once and every
// output written once, the row stays in registers (the backward: shared memory)
// between the statistics and the output, and HBM bounds it: 200704 x 96 with the
// residual 23.9 us, 6.5 TB/s; post-norm 589824 x 192 97.4 us, 7.0 TB/s; e4m3 8191 x
// 4096 40.0 us, 5.9 TB/s; backward 589824 x 192 with dsum 137 us, 6.6 TB/s (half of the
// issue slots).  The statistics are one sum a row, of s - p and of its square, p being
// the mean of the row's first eight values: sum s^2 - C mu^2 (p = 0) would lose what a
// row's mean has above its spread; of values around p the variance keeps all but
// log2(1 + k^2) of fp32's bits, p lying k standard deviations from the mean, and a row
// of one value gives exact zeros.  k is some 0.35 as a rule, but sqrt(C / 8) beside a
// large channel among the eight: above sqrt 2 (one random row in 16,000) the row's sums
// are taken again about the mean, from registers or shared memory (a large channel
// there in every row: e4m3 8191 x 4096 44.1 us, backward 30010 x 2744 124 for 91.5).
// (Always two sums one after the other, the mean first: e4m3 8191 x 4096 43.0 us,
// backward 589824 x 192 151; each thread about its own values' mean, the threads'
// variances joined: 40.7 us, backward 30010 x 2744 112.6.)
#include <cmath>
#include <new>

#include "swin_layernorm.h"
#include "norm.cuh"

using namespace swin;

namespace {

enum { FORM_BF16 = 0, FORM_POST = 1, FORM_Q8 = 2 };

struct LnArgs {
    const bf16 *x, *residual, *gamma, *beta;
    bf16 *out_sum;
    void *out;       // bf16 [rows, C], or e4m3 codes
    float *scales;   // e4m3: [rows]
    int rows, chunks;   // chunks = C / 8
    float inv_c, eps;
    int lpr;         // lanes per row (rows on part of a warp)
};

// The sums of a and b over a row's lanes (a block: red holds a pair a warp).
template <bool BLOCK>
__device__ __forceinline__ void row_sum2(float &a, float &b, int lpr, float2 *red)
{
    lane_sum2(a, b, BLOCK ? 32 : lpr);
    if (!BLOCK) return;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
    for (int w = 0; w < warps; ++w) {
        a += red[w].x;
        b += red[w].y;
    }
}

// The sum of a piece's eight values.
__device__ __forceinline__ float piece_sum(const Piece &v) { return sum2(add2(add2(v.v[0], v.v[1]), add2(v.v[2], v.v[3]))); }

// Whether a row's sums of s - p and of its square say that p lies more than sqrt 2
// standard deviations from the mean: they are then taken again about the mean.
__device__ __forceinline__ bool far_pivot(float sum, float squares, float inv_c)
{
    const float mean = sum * inv_c;
    return 1.5f * mean * mean > squares * inv_c;   // (not for a NaN, nor for infinite squares)
}

// 1 / sqrt(var + eps) from the row's sums of s - p and of its square; mean: of s - p.
__device__ __forceinline__ float deviation(float sum, float squares, float inv_c, float eps, float &mean)
{
    mean = sum * inv_c;
    return rsqrtf(max_nan(fmaf(-mean, mean, squares * inv_c), 0.f) + eps);   // (infinite squares: r = 0)
}

// Threads of a block whose rows lie on part of a warp.  Post-norm: few, whose loads and
// stores mix with other blocks' (589824 x 192 97.1 us, by 256 threads 102.8; 200000 x 512,
// a power of two, 96.0 and 105 to 108 us).
constexpr int forward_threads(int form) { return form == FORM_POST ? 64 : 256; }

// (Blocks of a row: registers for two of 512 threads an SM, more in flight: post-norm
// 20000 x 6000 117 us, 204 without.  Rows on part of a warp: no such request, the
// compiler's own count.)
template <int CPL, bool BLOCK, int FORM>
__global__ void __launch_bounds__(BLOCK ? 512 : forward_threads(FORM), BLOCK ? 2 : 0) layernorm_forward_kernel(LnArgs a)
{
    __shared__ float2 red[16];
    __shared__ float amaxes[16];
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
    // post-norm: the residual, used last, by asynchronous copies into the thread's
    // own places (as plain loads the compiler puts them off until they are used:
    // 589824 x 192 113 us)
    extern __shared__ uint4 later[];   // a block's row: [CPL][blockDim.x]
    constexpr int THREADS = forward_threads(FORM);
    __shared__ uint4 warps_later[FORM == FORM_POST && !BLOCK ? CPL * THREADS : 1];
    const uint32_t own = smem_u32(BLOCK ? later : warps_later) + threadIdx.x * 16;
    const uint32_t own_step = (BLOCK ? blockDim.x : THREADS) * 16;
    uint4 s[CPL], t[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        const bool ok = row_ok && c < a.chunks;
        s[k] = ok ? ld16(a.x + base + c * 8) : make_uint4(0, 0, 0, 0);
        if (FORM == FORM_POST) {
            if (ok) cp_async16(own + k * own_step, a.residual + base + c * 8, 16);
        } else if (a.residual) {
            t[k] = ok ? ld16(a.residual + base + c * 8) : make_uint4(0, 0, 0, 0);
        }
    }
    // the stored (rounded) sum is what the norm sees
    auto stored = [&](const uint4 &x, const uint4 &res) {
        Piece v = piece(x);
        const Piece w = piece(res);
#pragma unroll
        for (int e = 0; e < 4; ++e) v.v[e] = add2(v.v[e], w.v[e]);
        return pack(v);
    };
    const bool add = FORM != FORM_POST && a.residual;
    uint4 head = make_uint4(0, 0, 0, 0);   // the row's first piece (a block: read by every thread)
    if (BLOCK) {
        head = ld16(a.x + base);
        if (add) head = stored(head, ld16(a.residual + base));
    }
    auto store_sum = [&]() {
        if (!add || !a.out_sum || !row_ok) return;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            if (c < a.chunks) *reinterpret_cast<uint4 *>(a.out_sum + base + c * 8) = s[k];
        }
    };
    if (add)
#pragma unroll
        for (int k = 0; k < CPL; ++k) s[k] = stored(s[k], t[k]);
    if (!BLOCK) store_sum();
    float p = piece_sum(piece(BLOCK ? head : s[0])) * 0.125f;
    if (!BLOCK) p = __shfl_sync(0xffffffffu, p, lane - li);
    auto minus_p = [&](int k) { return li + k * step < a.chunks ? pack2(-p) : pack2(0.f); };   // (behind the row: zeros)
    auto sums = [&](float &sum, float &sq) {
        f2 sum2v = 0, sq2v = 0;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const Piece v = piece(s[k]);
            const f2 m = minus_p(k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 d = add2(v.v[e], m);
                sum2v = add2(sum2v, d);
                sq2v = fma2(d, d, sq2v);
            }
        }
        sum = sum2(sum2v);
        sq = sum2(sq2v);
    };
    float sum, sq;
    sums(sum, sq);
    uint4 gm[CPL], bt[CPL];   // (asked for before the row's sums are known)
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        const int c = li + k * step;
        const bool ok = row_ok && c < a.chunks;
        gm[k] = ok ? ld16(a.gamma + c * 8) : make_uint4(0, 0, 0, 0);
        bt[k] = ok && a.beta ? ld16(a.beta + c * 8) : make_uint4(0, 0, 0, 0);
    }
    row_sum2<BLOCK>(sum, sq, a.lpr, red);
#pragma unroll
    for (int k = 0; k < CPL; ++k) {   // (kept packed: fewer registers, more rows in flight)
        forget(s[k]);
        forget(gm[k]);
        forget(bt[k]);
    }
    if (FORM == FORM_POST) {
        cp_async_commit();
        cp_async_wait<0>();
    }
    const bool far = far_pivot(sum, sq, a.inv_c);   // (the same for a row's threads)
    if (BLOCK ? far : __any_sync(0xffffffffu, far)) {
        if (far) p += sum * a.inv_c;
        sums(sum, sq);
#pragma unroll
        for (int k = 0; k < CPL; ++k) forget(s[k]);
        if (BLOCK) __syncthreads();   // (the first sums have been read)
        row_sum2<BLOCK>(sum, sq, a.lpr, red);
    }
    if (BLOCK) store_sum();   // (in place: only now has every thread read the row's first piece)
    float mean;
    const float r = deviation(sum, sq, a.inv_c, a.eps, mean);
    const f2 r2 = pack2(r), shift = pack2(-mean * r);
    if (FORM != FORM_Q8) {
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            if (!(row_ok && c < a.chunks)) continue;
            Piece v = piece(s[k]);
            const Piece g = piece(gm[k]), b = piece(bt[k]), w = FORM == FORM_POST ? piece(lds16(own + k * own_step)) : Piece{};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v.v[e] = fma2(fma2(add2(v.v[e], pack2(-p)), r2, shift), g.v[e], b.v[e]);
                if (FORM == FORM_POST) v.v[e] = add2(v.v[e], w.v[e]);
            }
            *reinterpret_cast<uint4 *>((bf16 *)a.out + base + c * 8) = pack(v);
        }
        return;
    }
    f2 y[CPL][4];
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) {   // (pieces behind the row: gamma and beta are zeros)
        const Piece v = piece(s[k]), g = piece(gm[k]), b = piece(bt[k]);
        const f2 m = minus_p(k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[k][e] = fma2(fma2(add2(v.v[e], m), r2, shift), g.v[e], b.v[e]);
            float lo, hi;
            unpack2(y[k][e], lo, hi);
            amax = max_abs(amax, lo, hi);
        }
    }
    amax = row_reduce<MaxOp, BLOCK>(amax, a.lpr, amaxes);
    store_codes<CPL>(y, amax, a.scales + row, row_ok, li, step, a.chunks, (uint8_t *)a.out + base);
}

struct LnBwdArgs {
    const bf16 *s, *dy, *dsum, *gamma;
    bf16 *dx;
    float *partial;   // [gridDim.x, cols]: each block's shares of dgamma and (from column C) dbeta
    float *dgamma, *dbeta;   // one block: written by it
    int rows, chunks;
    float inv_c, eps;
    int lanes;        // of a row: of a warp, or (wide rows) threads
};

// The backward, dx = r (a - mean a - n mean(a n)) + dsum with a = dy gamma, of a
// thread's piece of a row: its shares of the row's sums of s - p, its square, a and
// a (s - p),
struct RowSums {
    f2 sum, sq, a, dot;
};
__device__ __forceinline__ void piece_sums(const uint4 &su, const uint4 &du, const uint4 &gu, f2 minus_p, RowSums &w)
{
    const uint32_t s[4] = {su.x, su.y, su.z, su.w}, d[4] = {du.x, du.y, du.z, du.w}, g[4] = {gu.x, gu.y, gu.z, gu.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 v = add_bf16x2(s[e], minus_p), x = mul_bf16x2(d[e], g[e]);
        w.sum = add2(w.sum, v);
        w.sq = fma2(v, v, w.sq);
        w.a = add2(w.a, x);
        w.dot = fma2(x, v, w.dot);
    }
}
// and, from the row's sums, dx and the terms of dgamma and dbeta.
struct RowGrad {
    f2 minus_p, r, shift;         // n = (s - p) r + shift
    f2 minus_ra, minus_rn;        // -r mean a, -r mean(a n)
};
__device__ __forceinline__ RowGrad row_grad(float p, const float4 &w, float inv_c, float eps)
{
    float mean;
    const float r = deviation(w.x, w.y, inv_c, eps, mean);
    const float ma = w.z * inv_c, mn = r * fmaf(-mean, ma, w.w * inv_c);
    return {pack2(-p), pack2(r), pack2(-mean * r), pack2(-r * ma), pack2(-r * mn)};
}
template <bool DSUM>
__device__ __forceinline__ uint4 piece_grad(const uint4 &su, const uint4 &du, const uint4 &gu, const uint4 &mu, const RowGrad &w,
                                            Piece &dg, Piece &db)
{
    const uint32_t s[4] = {su.x, su.y, su.z, su.w}, d[4] = {du.x, du.y, du.z, du.w}, g[4] = {gu.x, gu.y, gu.z, gu.w},
                   m[4] = {mu.x, mu.y, mu.z, mu.w};
    const Piece y = piece(du);
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 n = fma2(add_bf16x2(s[e], w.minus_p), w.r, w.shift);
        dg.v[e] = fma2(y.v[e], n, dg.v[e]);
        db.v[e] = add2(db.v[e], y.v[e]);
        f2 t = fma2(mul_bf16x2(d[e], g[e]), w.r, w.minus_ra);
        t = fma2(n, w.minus_rn, t);
        if (DSUM) t = add_bf16x2(m[e], t);
        float lo, hi;
        unpack2(t, lo, hi);
        o[e] = pack_bf16x2(lo, hi);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// A block's columns of dgamma and dbeta: partial rows, or (one block) the result.
__device__ __forceinline__ float *block_columns(const LnBwdArgs &a, int which)
{
    const int C = a.chunks * 8;
    if (gridDim.x == 1) return which ? a.dbeta : a.dgamma;
    return a.partial + (int64_t)blockIdx.x * C * (a.dbeta ? 2 : 1) + which * C;
}

// Blocks of 256 threads on an SM: enough bytes of loads in flight, and no more
// (200000 x 512, two pieces a lane: with dsum 120 us with two blocks, 129 with
// three; without 102 and 99).
constexpr int blocks_per_sm(int cpl, bool dsum) { return cpl > 2 || (cpl == 2 && dsum) ? 2 : cpl == 2 ? 3 : 4; }

// Rows on part of a warp: a block takes 8 * (32 / lanes) rows together, then the
// ones gridDim.x on.  Every thread fetches its pieces of the rows after these by
// asynchronous copies into its own place in shared memory, so that loads are in
// flight while it computes.  It keeps the columns it owns of dgamma and dbeta in
// registers over its rows; the block writes one partial row at the end.
template <int CPL, bool DSUM>
__global__ void __launch_bounds__(256, blocks_per_sm(CPL, DSUM)) layernorm_backward_kernel(LnBwdArgs a)
{
    constexpr uint32_t STAGE = (DSUM ? 3 : 2) * CPL * 4096;   // two: these rows, and the next
    extern __shared__ __align__(16) float part[];   // the pieces; at the end [8 warps][C]
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, step = a.lanes, li = lane % step;
    const int rpw = 32 / step, rpb = 8 * rpw;
    // this thread's piece k of array i in a stage at `at`: at + (i CPL + k) 4 KB
    uint32_t at = smem_u32(part) + threadIdx.x * 16, other = at + STAGE;
    bool have[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) have[k] = li + k * step < a.chunks;
    auto fetch = [&](int64_t row, uint32_t to) {
        if (row < a.rows) {
            const int64_t off = (row * a.chunks + li) * 8;
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                if (!have[k]) continue;
                cp_async16(to + k * 4096, a.s + off + k * step * 8, 16);
                cp_async16(to + (CPL + k) * 4096, a.dy + off + k * step * 8, 16);
                if (DSUM) cp_async16(to + (2 * CPL + k) * 4096, a.dsum + off + k * step * 8, 16);
            }
        }
        cp_async_commit();
    };
    const int64_t hop = (int64_t)gridDim.x * rpb;
    int64_t row = (int64_t)blockIdx.x * rpb + warp * rpw + lane / step;
    fetch(row, at);
    Piece acc[2][CPL];
    uint4 g[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        g[k] = have[k] ? ld16(a.gamma + (li + k * step) * 8) : make_uint4(0, 0, 0, 0);
        acc[0][k] = acc[1][k] = Piece{};
    }
#pragma unroll 1
    for (int64_t r0 = (int64_t)blockIdx.x * rpb; r0 < a.rows; r0 += hop, row += hop) {
        fetch(row + hop, other);
        cp_async_wait<1>();
        const bool row_ok = row < a.rows;   // (no row: its pieces hold whatever was there, and count for nothing)
        float p = __shfl_sync(0xffffffffu, piece_sum(piece(lds16(at))) * 0.125f, lane - li);
        auto row_sums = [&]() {
            RowSums w{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                forget(g[k]);   // (kept packed)
                if (have[k]) piece_sums(lds16(at + k * 4096), lds16(at + (CPL + k) * 4096), g[k], pack2(-p), w);
            }
            float4 v = make_float4(sum2(w.sum), sum2(w.sq), sum2(w.a), sum2(w.dot));
            lane_sum2(v.x, v.y, step);
            lane_sum2(v.z, v.w, step);
            return v;
        };
        float4 sums = row_sums();
        const bool far = row_ok && far_pivot(sums.x, sums.y, a.inv_c);   // (the same for a row's lanes)
        if (__any_sync(0xffffffffu, far)) {
            if (far) p += sums.x * a.inv_c;
            sums = row_sums();
        }
        if (row_ok) {
            const RowGrad grad = row_grad(p, sums, a.inv_c, a.eps);
            bf16 *dx = a.dx + (row * a.chunks + li) * 8;
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                forget(g[k]);
                if (!have[k]) continue;
                *reinterpret_cast<uint4 *>(dx + k * step * 8) =
                    piece_grad<DSUM>(lds16(at + k * 4096), lds16(at + (CPL + k) * 4096), g[k],
                                     DSUM ? lds16(at + (2 * CPL + k) * 4096) : uint4{}, grad, acc[0][k], acc[1][k]);
            }
        }
        const uint32_t was = at;
        at = other;
        other = was;
    }
    __syncthreads();   // (every thread is done with its pieces)
    // the warp's rows, then the block's warps
    const int C = a.chunks * 8;
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        if (z && !a.dbeta) break;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            const int c = li + k * step;
            float v[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) unpack2(acc[z][k].v[e], v[2 * e], v[2 * e + 1]);
            // (two lanes share the piece's values between them, each a half, then
            // quarters: seven shuffles for three steps, not 24; 4873 x 96 9.2 us and 6.7)
            int first = 0, n = 8;
#pragma unroll
            for (int s = 0; s < 5; ++s) {
                const int o = 16 >> s;
                if (o < step) break;
                const bool upper = lane & o;
                if (s < 3) {
                    const int half = 4 >> s;
#pragma unroll
                    for (int e = 0; e < half; ++e) {
                        const float give = upper ? v[e] : v[e + half];
                        v[e] = (upper ? v[e + half] : v[e]) + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                    first += upper ? half : 0;
                    n = half;
                } else {
                    v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                    if (upper) n = 0;
                }
            }
            if (c >= a.chunks) continue;
            float *to = part + warp * C + c * 8 + first;
            if (n >= 4) *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
            if (n == 8) *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (n == 2) *reinterpret_cast<float2 *>(to) = make_float2(v[0], v[1]);
            if (n == 1) to[0] = v[0];
        }
        __syncthreads();
        float *out = block_columns(a, z);
        for (int i = threadIdx.x; i < C; i += 256) {
            float v = 0.f;
            for (int w = 0; w < 8; ++w) v += part[w * C + i];
            out[i] = v;
        }
        __syncthreads();
    }
}

// A row's sums over a group of a block, of `threads` threads that meet at a
// barrier of their own; red: two rows of 16 a group, used in turn.
__device__ __forceinline__ void group_sum4(float4 &v, int threads, int group, int turn, float4 *red)
{
    lane_sum2(v.x, v.y, 32);
    lane_sum2(v.z, v.w, 32);
    const int warps = threads >> 5, warp = (threadIdx.x - group * threads) >> 5;
    red += (2 * group + (turn & 1)) * 16;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = 0; w < warps; ++w) {
        const float4 u = red[w];
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
    }
}

// Wider rows: a group of warps a row, several groups a block (few blocks, since
// each writes partial rows that are read again).  Every thread fetches its own
// pieces of the next row by asynchronous copies into its own place in shared
// memory, so that the latency of HBM is paid once, not once a row.
template <int CPL, bool DSUM>
__global__ void __launch_bounds__(512, 1) layernorm_backward_wide_kernel(LnBwdArgs a)
{
    constexpr int ARRAYS = DSUM ? 3 : 2, DEPTH = 2;   // stages: a row, and the next
    extern __shared__ __align__(16) float part[];   // the pieces; at the end the columns' sums
    __shared__ float4 red[2 * 16 * 16];
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
    uint4 head = make_uint4(0, 0, 0, 0);   // its first piece, for every thread
    auto fetch = [&]() {
        if (ahead < a.rows) {
            const int64_t off = ahead * C + li * 8;
            head = ld16(a.s + ahead * C);
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
    Piece acc[2][CPL];
    uint4 g[CPL];
#pragma unroll
    for (int k = 0; k < CPL; ++k) {
        g[k] = have[k] ? ld16(a.gamma + (li + k * step) * 8) : make_uint4(0, 0, 0, 0);
        acc[0][k] = acc[1][k] = Piece{};
    }
    uint32_t at = ring;
    int turn = 0;
#pragma unroll 1
    for (int64_t row = first; row < a.rows; row += hop) {   // (the same for a group's threads)
        float p = piece_sum(piece(head)) * 0.125f;
        fetch();
        cp_async_wait<DEPTH - 1>();
        auto row_sums = [&]() {
            RowSums w{0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < CPL; ++k) {
                forget(g[k]);   // (kept packed)
                if (have[k]) piece_sums(lds16(place(at, 0, k)), lds16(place(at, 1, k)), g[k], pack2(-p), w);
            }
            float4 v = make_float4(sum2(w.sum), sum2(w.sq), sum2(w.a), sum2(w.dot));
            group_sum4(v, step, group, turn++, red);
            return v;
        };
        float4 sums = row_sums();
        if (far_pivot(sums.x, sums.y, a.inv_c)) {   // (the same for the group's threads)
            p += sums.x * a.inv_c;
            sums = row_sums();
        }
        const RowGrad grad = row_grad(p, sums, a.inv_c, a.eps);
        bf16 *dx = a.dx + row * C + li * 8;
#pragma unroll
        for (int k = 0; k < CPL; ++k) {
            forget(g[k]);
            if (!have[k]) continue;
            *reinterpret_cast<uint4 *>(dx + k * step * 8) =
                piece_grad<DSUM>(lds16(place(at, 0, k)), lds16(place(at, 1, k)), g[k],
                                 DSUM ? lds16(place(at, 2, k)) : uint4{}, grad, acc[0][k], acc[1][k]);
        }
        at += stage;
        if (at == ring_end) at = ring;
    }
    __syncthreads();   // (every group is done with its pieces)
    // each thread's columns into its own places, [z][k][half][thread]; then a column
    // piece a thread over the groups
    float4 *own = reinterpret_cast<float4 *>(part) + threadIdx.x;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int k = 0; k < CPL; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 v;
                unpack2(acc[z][k].v[2 * h], v.x, v.y);
                unpack2(acc[z][k].v[2 * h + 1], v.z, v.w);
                own[((z * CPL + k) * 2 + h) * blockDim.x] = v;
            }
    __syncthreads();
    const int pieces = 2 * a.chunks;   // halves of the columns' pieces
    for (int i = threadIdx.x; i < (a.dbeta ? 2 : 1) * pieces; i += blockDim.x) {
        const int z = i >= pieces, c = (i - z * pieces) >> 1, h = i & 1;
        const float4 *from = reinterpret_cast<const float4 *>(part) + ((z * CPL + c / step) * 2 + h) * blockDim.x + c % step;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int t = 0; t < rpb; ++t) {
            const float4 u = from[t * step];
            v.x += u.x;
            v.y += u.y;
            v.z += u.z;
            v.w += u.w;
        }
        *reinterpret_cast<float4 *>(block_columns(a, z) + c * 8 + h * 4) = v;
    }
}

constexpr int FWD_PIECES = 4, BWD_PIECES = 3, BWD_BLOCK_PIECES = 4;
constexpr int MAX_GROUPS = 15;   // row groups of a block: a block has 16 barriers, and one is everybody's

template <int FORM>
cudaError_t launch_forward(LnArgs a, cudaStream_t stream)
{
    // rows that leave SMs idle take as many threads as pieces: the latency of
    // one row counts then
    const int most = a.rows < sm_count() ? 1 : FWD_PIECES;
    const RowPlan p = plan_row(a.chunks, most, most);
    a.lpr = p.block ? 32 : p.lanes;
    const int threads = p.block ? p.lanes : forward_threads(FORM);
    const int64_t rpb = p.block ? 1 : threads / 32 * (32 / p.lanes);
    const unsigned grid = (unsigned)((a.rows + rpb - 1) / rpb);
#define SWIN_LN_CASE(n)                                                                       \
    case n:                                                                                   \
        return launch_maybe_overlapped(p.block ? layernorm_forward_kernel<n, true, FORM>      \
                                               : layernorm_forward_kernel<n, false, FORM>,    \
                                       dim3(grid), dim3(threads), smem, stream, 1, a);
    const size_t smem = FORM == FORM_POST && p.block ? (size_t)p.cpl * threads * 16 : 0;   // (at most 32 KB)
    switch (p.cpl) {
        SWIN_LN_CASE(1)
        SWIN_LN_CASE(2)
        SWIN_LN_CASE(3)
        SWIN_LN_CASE(4)
    default:
        return cudaErrorInvalidValue;
    }
#undef SWIN_LN_CASE
}

// The backward's launch: as many blocks as the SMs hold at once, each walking
// its share of the rows.
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
    // (three pieces a thread rather than four where no more lanes idle so: 30010 x 2744
    // 94.1 us by 96 threads a row, 91.1 by 128, with dsum 118.4 and 112.3, 10000 x 8448
    // 134.4 and 107.4; not 16384 x 4096, by 128 threads 72, by 192 80)
    const RowPlan three = plan_row(chunks, BWD_PIECES, BWD_PIECES);
    if (p.row.block && three.cpl == 3 && three.lanes * 3 <= p.row.lanes * p.row.cpl) p.row = three;
    const RowPlan &r = p.row;
    int64_t rpb, per_sm;
    if (r.block) {
        const int groups = 512 / r.lanes;
        rpb = groups < MAX_GROUPS ? groups : MAX_GROUPS;
        per_sm = 1;
        p.threads = (int)rpb * r.lanes;
        p.smem = (size_t)p.threads * (with_dsum ? 3 : 2) * 2 * r.cpl * 16;   // (at most 192 KB; the sums need 64 B a piece)
    } else {
        rpb = 8 * (32 / r.lanes);
        per_sm = blocks_per_sm(r.cpl, with_dsum);
        p.threads = 256;
        p.smem = (size_t)(with_dsum ? 3 : 2) * r.cpl * 2 * 4096;   // (at most 72 KB)
        if (p.smem < (size_t)8 * C * sizeof(float)) p.smem = (size_t)8 * C * sizeof(float);
    }
    const int64_t want = (rows + rpb - 1) / rpb, most = sm_count() * per_sm;
    // few rows: one block, whose sums are the result, for as many turns as cost less than
    // a second launch (190 x 96, three turns, 6.7 us by two launches, 5.6; 250 x 96, four, 6.6
    // both; wide rows' take longer: 15 x 2744, three, 6.7 and 9.4)
    p.grid = want <= (r.block ? 2 : 4) ? 1 : (int)(want < most ? want : most);
    return p;
}

cudaError_t launch_backward(LnBwdArgs a, const BwdPlan &p, cudaStream_t stream)
{
    const RowPlan &r = p.row;
    a.lanes = r.lanes;
    const int C = a.chunks * 8, cols = a.dbeta ? 2 * C : C;
    void (*kern)(LnBwdArgs) = nullptr;
    if (r.cpl < (r.block ? 3 : 1) || r.cpl > (r.block ? 4 : 3)) return cudaErrorInvalidValue;
    if (r.block)
        kern = a.dsum ? (r.cpl == 3 ? layernorm_backward_wide_kernel<3, true> : layernorm_backward_wide_kernel<4, true>)
                      : (r.cpl == 3 ? layernorm_backward_wide_kernel<3, false> : layernorm_backward_wide_kernel<4, false>);
    else if (a.dsum)
        kern = r.cpl == 1 ? layernorm_backward_kernel<1, true>
                          : r.cpl == 2 ? layernorm_backward_kernel<2, true> : layernorm_backward_kernel<3, true>;
    else
        kern = r.cpl == 1 ? layernorm_backward_kernel<1, false>
                          : r.cpl == 2 ? layernorm_backward_kernel<2, false> : layernorm_backward_kernel<3, false>;
    cudaError_t e;
    // (always the most any call needs: another thread may be between its setting
    // and its launch)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (r.block ? 512 : 256) * 6 * r.cpl * 16);
    if (e != cudaSuccess) return e;
    e = launch_maybe_overlapped(kern, dim3(p.grid), dim3(p.threads), p.smem, stream, 1, a);
    if (e != cudaSuccess || p.grid == 1) return e;
    return launch_maybe_overlapped(column_sum_kernel, dim3((cols + 31) / 32), dim3(1024), 0, stream, 1,
                                   (const float *)a.partial, p.grid, cols, a.dgamma, C, a.dbeta);
}

bool bad_pointer(const void *p, bool required)
{
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) != 0 : required;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SWIN_WATTN_OK : SWIN_WATTN_ECUDA; }

} // namespace

struct swin_block_layernorm_s {
    int C;
    float eps;
    int device;   // -1: not bound yet
    int last_launches;
    OrderedWorkspace ws;   // the backward's partial sums of dgamma and dbeta
};

namespace {

// Checks shared by the forward forms; `out_bytes` of one output element.
int check_forward(const swin_block_layernorm_s *h, const void *x, const void *residual, int rows, const void *gamma,
                  const void *beta, const void *out_sum, const void *out, int64_t out_bytes)
{
    if (!h || rows < 0) return SWIN_WATTN_EINVAL;
    if (rows == 0) return SWIN_WATTN_OK;   // (an empty tensor may have no address)
    if (bad_pointer(x, true) || bad_pointer(residual, false) || bad_pointer(gamma, true) || bad_pointer(beta, false) ||
        bad_pointer(out_sum, false) || bad_pointer(out, true) || (out_sum && !residual))
        return SWIN_WATTN_EINVAL;
    const int64_t n = (int64_t)rows * h->C, in = 2 * n, on = out_bytes * n, vec = 2 * (int64_t)h->C;
    const bool same_type = out_bytes == 2;
    // in place (the very same tensor) is fine, any other overlap is not
    for (const void *p : {x, residual}) {
        if (!p) continue;
        if (overlaps(p, in, out, on) && !(same_type && p == out)) return SWIN_WATTN_EINVAL;
        if (out_sum && overlaps(p, in, out_sum, in) && p != out_sum) return SWIN_WATTN_EINVAL;
    }
    for (const void *p : {gamma, beta})
        if (p && (overlaps(p, vec, out, on) || (out_sum && overlaps(p, vec, out_sum, in)))) return SWIN_WATTN_EINVAL;
    if (out_sum && overlaps(out_sum, in, out, on)) return SWIN_WATTN_EINVAL;
    return SWIN_WATTN_OK;
}

LnArgs forward_args(const swin_block_layernorm_s *h, const void *x, const void *residual, int rows, const void *gamma,
                    const void *beta, void *out_sum, void *out, float *scales)
{
    LnArgs a{};
    a.x = (const bf16 *)x;
    a.residual = (const bf16 *)residual;
    a.gamma = (const bf16 *)gamma;
    a.beta = (const bf16 *)beta;
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

int swin_block_layernorm_create(swin_block_layernorm_t *out, int C, float eps)
{
    if (!out) return SWIN_WATTN_EINVAL;
    *out = nullptr;
    if (C <= 0 || C % 8 || C > NORM_MAX_C || !(eps >= 0.f) || std::isinf(eps)) return SWIN_WATTN_EINVAL;
    swin_block_layernorm_s *h = new (std::nothrow) swin_block_layernorm_s{};
    if (!h) return SWIN_WATTN_ENOMEM;
    h->C = C;
    h->eps = eps;
    h->device = -1;
    *out = h;
    return SWIN_WATTN_OK;
}

int swin_block_layernorm_destroy(swin_block_layernorm_t h)
{
    if (!h) return SWIN_WATTN_OK;
    ows_free(&h->ws);
    delete h;
    return SWIN_WATTN_OK;
}

int swin_block_layernorm_last_launches(swin_block_layernorm_t h) { return h ? h->last_launches : 0; }

int swin_block_layernorm_forward(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                 const void *gamma, const void *beta, void *out_sum, void *out, swin_stream_t stream)
{
    int rc = check_forward(h, x, residual, rows, gamma, beta, out_sum, out, 2);
    if (rc != SWIN_WATTN_OK || rows == 0) return rc;
    if ((rc = bind_device(&h->device)) != SWIN_WATTN_OK) return rc;
    h->last_launches = 1;
    return cuda_status(launch_forward<FORM_BF16>(forward_args(h, x, residual, rows, gamma, beta, out_sum, out, nullptr),
                                                 (cudaStream_t)stream));
}

int swin_block_layernorm_forward_post(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                      const void *gamma, const void *beta, void *out, swin_stream_t stream)
{
    int rc = check_forward(h, x, residual, rows, gamma, beta, nullptr, out, 2);
    if (rc != SWIN_WATTN_OK || rows == 0) return rc;
    if (!residual) return SWIN_WATTN_EINVAL;
    if ((rc = bind_device(&h->device)) != SWIN_WATTN_OK) return rc;
    h->last_launches = 1;
    return cuda_status(launch_forward<FORM_POST>(forward_args(h, x, residual, rows, gamma, beta, nullptr, out, nullptr),
                                                 (cudaStream_t)stream));
}

int swin_block_layernorm_forward_q8(swin_block_layernorm_t h, const void *x, const void *residual, int rows,
                                    const void *gamma, const void *beta, void *out_sum, void *out8, float *scales,
                                    swin_stream_t stream)
{
    int rc = check_forward(h, x, residual, rows, gamma, beta, out_sum, out8, 1);
    if (rc != SWIN_WATTN_OK || rows == 0) return rc;
    if (bad_pointer(scales, true)) return SWIN_WATTN_EINVAL;
    const int64_t n = (int64_t)rows * h->C, sn = 4 * (int64_t)rows, vec = 2 * (int64_t)h->C;
    if (overlaps(scales, sn, x, 2 * n) || overlaps(scales, sn, residual, residual ? 2 * n : 0) ||
        overlaps(scales, sn, out_sum, out_sum ? 2 * n : 0) || overlaps(scales, sn, out8, n) ||
        overlaps(scales, sn, gamma, vec) || overlaps(scales, sn, beta, beta ? vec : 0))
        return SWIN_WATTN_EINVAL;
    if ((rc = bind_device(&h->device)) != SWIN_WATTN_OK) return rc;
    h->last_launches = 1;
    return cuda_status(launch_forward<FORM_Q8>(forward_args(h, x, residual, rows, gamma, beta, out_sum, out8, scales),
                                               (cudaStream_t)stream));
}

int swin_block_layernorm_backward(swin_block_layernorm_t h, const void *s, int rows, const void *gamma, const void *dy,
                                  const void *dsum, void *dx, float *dgamma, float *dbeta, swin_stream_t stream)
{
    if (!h || rows < 0 || bad_pointer(dgamma, true) || bad_pointer(dbeta, false)) return SWIN_WATTN_EINVAL;
    const int64_t n = 2 * (int64_t)rows * h->C, vec = 2 * (int64_t)h->C;
    if (dbeta && overlaps(dgamma, 2 * vec, dbeta, 2 * vec)) return SWIN_WATTN_EINVAL;
    cudaStream_t st = (cudaStream_t)stream;
    if (rows == 0) {
        const int rc = bind_device(&h->device);
        if (rc != SWIN_WATTN_OK) return rc;
        const cudaError_t e = cudaMemsetAsync(dgamma, 0, 2 * (size_t)vec, st);
        return cuda_status(e != cudaSuccess || !dbeta ? e : cudaMemsetAsync(dbeta, 0, 2 * (size_t)vec, st));
    }
    if (bad_pointer(s, true) || bad_pointer(gamma, true) || bad_pointer(dy, true) || bad_pointer(dsum, false) ||
        bad_pointer(dx, true))
        return SWIN_WATTN_EINVAL;
    if (overlaps(s, n, dx, n) || (overlaps(dy, n, dx, n) && dy != dx) ||
        (dsum && overlaps(dsum, n, dx, n) && dsum != dx) || overlaps(gamma, vec, dx, n))
        return SWIN_WATTN_EINVAL;
    for (const void *o : {(const void *)dgamma, (const void *)dbeta}) {
        if (!o) continue;
        for (const void *p : {s, dy, dsum, (const void *)dx})
            if (p && overlaps(p, n, o, 2 * vec)) return SWIN_WATTN_EINVAL;
        if (overlaps(gamma, vec, o, 2 * vec)) return SWIN_WATTN_EINVAL;
    }
    int rc = bind_device(&h->device);
    if (rc != SWIN_WATTN_OK) return rc;
    const BwdPlan p = plan_backward(rows, h->C, dsum != nullptr);
    void *ws = nullptr;
    bool captured = false;
    if (p.grid > 1 && (rc = ows_begin(&h->ws, (size_t)p.grid * h->C * (dbeta ? 2 : 1) * sizeof(float), st, &ws, &captured)) !=
                          SWIN_WATTN_OK)
        return rc;
    LnBwdArgs a{};
    a.s = (const bf16 *)s;
    a.dy = (const bf16 *)dy;
    a.dsum = (const bf16 *)dsum;
    a.gamma = (const bf16 *)gamma;
    a.dx = (bf16 *)dx;
    a.partial = (float *)ws;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.rows = rows;
    a.chunks = h->C / 8;
    a.inv_c = 1.f / (float)h->C;
    a.eps = h->eps;
    h->last_launches = p.grid > 1 ? 2 : 1;
    rc = cuda_status(launch_backward(a, p, st));
    const int rc2 = ows_end(&h->ws, st, ws, captured);
    return rc != SWIN_WATTN_OK ? rc : rc2;
}

} // extern "C"
