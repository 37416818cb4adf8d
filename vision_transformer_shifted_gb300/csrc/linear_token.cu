// The linear operator for a single token: the weights' trip from HBM and the
// latency around it are all there is.  On the few-row kernel (gated_few.cu) a token
// pays for tensor memory, barriers and two cluster barriers; here a warp takes two
// output channels and their whole K, or a block's warps share K, with the loads of
// four steps in flight a lane; exact products of 16-bit values are summed in fp32
// (one instruction each, no conversion; e4m3 values go through f16, which holds
// them all), and the lanes' sums added by shuffles.  1 x 2048 x 8192: 7.0 us (4.8
// TB/s) and 9.4 on the few-row kernel, 1 x 4096 x 16384 20.6 us (6.5 TB/s) and 24.6,
// e4m3 1 x 4096 x 11264 11.0 and 12.4.  (Two rows: 9.6 and 9.5, four: 11.8 and 9.6.)
#include "linear.cuh"

namespace swin {

namespace {

constexpr int TOKEN_WARPS = 8, TOKEN_OUT = 2, TOKEN_STEPS = 4;   // outputs of a warp; steps of loads in flight

struct TokenArgs {
    const void *x, *w;
    const bf16 *bias, *residual;
    const float *sx, *sw;
    bf16 *out, *z;
    int N, act;
    int pieces;      // of a row: 16 bytes each
    int64_t pitch;   // bytes of a row
    int split;       // warps that share an output's K
};

// Loads in the order they are written (as plain ones the compiler spreads them out
// between the products, four steps no longer in flight: 1 x 2048 x 8192 8.3 us).
__device__ __forceinline__ uint4 load_once(const void *p)
{
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}
__device__ __forceinline__ uint4 load_kept(const void *p)
{
    uint4 u;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
    return u;
}
// acc += the products of two pairs of 16-bit values.
__device__ __forceinline__ void dot2_bf16(float &acc, uint32_t a, uint32_t b)
{
    asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\t"
        "fma.rn.f32.bf16 %0, l, m, %0;\n\tfma.rn.f32.bf16 %0, h, n, %0;\n\t}"
        : "+f"(acc)
        : "r"(a), "r"(b));
}
__device__ __forceinline__ void dot2_f16(float &acc, uint32_t a, uint32_t b)
{
    asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\t"
        "fma.rn.f32.f16 %0, l, m, %0;\n\tfma.rn.f32.f16 %0, h, n, %0;\n\t}"
        : "+f"(acc)
        : "r"(a), "r"(b));
}
// Two e4m3 values, of a word's lower and upper half, as f16.
__device__ __forceinline__ void e4m3_pairs(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// (bf16: registers for the loads in flight; e4m3, whose conversions bind: as many
// warps as there are, e4m3 1 x 4096 x 11264 11.9 us with 64 registers)
template <bool Q8>
__global__ void __launch_bounds__(32 * TOKEN_WARPS, Q8 ? 0 : 4) token_kernel(const TokenArgs a)
{
    __shared__ float part[TOKEN_WARPS][TOKEN_OUT];
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int groups = TOKEN_WARPS / a.split, share = warp % a.split;
    const int n0 = ((int)blockIdx.x * groups + warp / a.split) * TOKEN_OUT;
    const char *w = (const char *)a.w + (n0 < a.N ? n0 : 0) * a.pitch, *x = (const char *)a.x;
    float acc[TOKEN_OUT] = {};
    const int step = a.split * 32;
#pragma unroll 1
    for (int c0 = share * 32 + lane; c0 < a.pieces; c0 += TOKEN_STEPS * step) {
        uint4 wv[TOKEN_STEPS][TOKEN_OUT], xv[TOKEN_STEPS];
#pragma unroll
        for (int i = 0; i < TOKEN_STEPS; ++i) {
            const int c = c0 + i * step;
            const bool in = c < a.pieces;
#pragma unroll
            for (int o = 0; o < TOKEN_OUT; ++o)   // (N is even: both outputs are there)
                wv[i][o] = in ? load_once(w + o * a.pitch + (int64_t)c * 16) : make_uint4(0, 0, 0, 0);
            xv[i] = in ? load_kept(x + (int64_t)c * 16) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < TOKEN_STEPS; ++i) {
            const uint32_t xw[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
            uint32_t x0[4], x1[4];
            if (Q8) {
#pragma unroll
                for (int e = 0; e < 4; ++e) e4m3_pairs(xw[e], x0[e], x1[e]);
            }
#pragma unroll
            for (int o = 0; o < TOKEN_OUT; ++o) {
                const uint32_t ww[4] = {wv[i][o].x, wv[i][o].y, wv[i][o].z, wv[i][o].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (Q8) {
                        uint32_t w0, w1;
                        e4m3_pairs(ww[e], w0, w1);
                        dot2_f16(acc[o], w0, x0[e]);
                        dot2_f16(acc[o], w1, x1[e]);
                    } else {
                        dot2_bf16(acc[o], ww[e], xw[e]);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int o = 0; o < TOKEN_OUT; ++o) {
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) acc[o] += __shfl_xor_sync(0xffffffffu, acc[o], s);
        if (lane == 0) part[warp][o] = acc[o];
    }
    __syncthreads();
    // a thread an output value
    const int t = threadIdx.x, n = (int)blockIdx.x * groups * TOKEN_OUT + t;
    if (t >= groups * TOKEN_OUT || n >= a.N) return;
    float v = 0.f;
    for (int s = 0; s < a.split; ++s) v += part[t / TOKEN_OUT * a.split + s][t % TOKEN_OUT];
    if (Q8) v *= a.sx[0] * a.sw[n];
    if (a.bias) v += __bfloat162float(a.bias[n]);
    if (a.z) a.z[n] = __float2bfloat16_rn(v);
    float other;
    if (a.act != ACT_NONE)
        unpack2(a.act == ACT_SILU ? activate2<ACT_SILU>(pack2(v)) : activate2<ACT_GELU>(pack2(v)), v, other);
    if (a.residual) v += __bfloat162float(a.residual[n]);
    a.out[n] = __float2bfloat16_rn(v);
}

} // namespace

cudaError_t launch_token_linear(const FewLinear &u, cudaStream_t stream)
{
    TokenArgs a{};
    const bool q8 = u.sx != nullptr;
    a.x = u.x;
    a.w = u.w;
    a.bias = u.bias;
    a.residual = u.residual;
    a.sx = u.sx;
    a.sw = u.sw;
    a.out = u.out;
    a.z = u.z;
    a.N = u.N;
    a.act = u.act;
    a.pitch = (int64_t)u.C * (q8 ? 1 : 2);
    a.pieces = (int)(a.pitch / 16);
    // warps that share K: until there are 24 an SM, each lane left two pieces at least
    const int outs = u.N / TOKEN_OUT;
    a.split = 1;
    while (a.split < TOKEN_WARPS && (int64_t)outs * a.split < 24ll * sm_count() && a.pieces >= 64 * a.split) a.split *= 2;
    const int groups = TOKEN_WARPS / a.split;
    return launch_maybe_overlapped(q8 ? token_kernel<true> : token_kernel<false>,
                                   dim3((unsigned)((outs + groups - 1) / groups)), dim3(32 * TOKEN_WARPS), 0, stream, 1, a);
}

} // namespace swin
