// The gated block's forward for few rows (single tokens, small batches), where
// the weights' one trip from HBM is the work: each product with the weights as
// the MMA's A operand (128 weight rows) and the rows of x as its narrow B (16 to
// 128 columns), so that no row of the tensor-core tile is idle weight traffic.
//
// A CTA takes one tile of 128 weight rows (64 of Wg and the same 64 of Wu, or
// 128 of Wd) and a share of K; the CTAs of a cluster share a tile's K (up to
// eight), which spreads few tiles over the SMs without partial sums in global
// memory: each CTA leaves its fp32 tile in shared memory and the cluster's CTAs
// add their shares of it through distributed shared memory, in rank order.
// Weights stream through a TMA ring of about 100 KB a CTA, two CTAs an SM: HBM
// bounds it, and the latency of two launches (9 us + bytes / 7.07 TB/s over the
// sizes; 1 x 2048 x 5632: 20 us, 24 rows from e4m3 4096 x 11264: 37).
#include <atomic>
#include <cstring>

#include "gated.cuh"

namespace swin {

namespace {

constexpr int FEW_THREADS = 192;   // four draining warps, a loading and an issuing one
constexpr int ACT_NONE = -1;
constexpr int FEW_MAX_STAGES = 6;

struct FewArgs {
    CUtensorMap w0, w1, x;         // ACT: Wg, Wu (boxes of 64 rows); else Wd (128 rows); x: np rows
    const bf16 *b0, *b1;           // ACT: bg, bu; else bd
    const float *sx, *s0, *s1;     // 8-bit: scales of x, Wg, Wu
    const bf16 *residual;
    bf16 *out;                     // [rows, ld]: h, or the block's output
    int rows, np;                  // np: rows rounded up to 16
    int cols, ld;                  // columns of out
    int k, kb, split, stages, stage_bytes;
    DeviceStatus st;
};

__device__ __forceinline__ float4 ld_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ void add4(float (&s)[4], const float4 &v)
{
    s[0] += v.x;
    s[1] += v.y;
    s[2] += v.z;
    s[3] += v.w;
}
__device__ __forceinline__ void add4(float (&s)[4], const bf16 *p)
{
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
    add4(s, make_float4(a.x, a.y, b.x, b.y));
}

template <int KIND>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    if (KIND == MMA_BF16)
        mma_bf16(d, adesc, bdesc, idesc, acc);
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
            : "memory");
}

template <int ACT, bool Q8>
__global__ void __launch_bounds__(FEW_THREADS) few_rows_kernel(const __grid_constant__ FewArgs a)
{
    constexpr int ELEMS = Q8 ? 128 : 64;            // K elements of a block
    constexpr int W = ACT == ACT_NONE ? 128 : 64;   // output columns of a tile
    constexpr bool EARLY = ACT == ACT_NONE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align(smem_raw, 1024);
    __shared__ uint64_t bars[2 * FEW_MAX_STAGES + 1];
    __shared__ uint32_t tslot;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * FEW_MAX_STAGES, done = empty + 8 * FEW_MAX_STAGES;
    const int split = a.split, rank = (int)(blockIdx.x % split), tile = (int)(blockIdx.x / split);
    const int kb0 = (int)((int64_t)a.kb * rank / split), kb1 = (int)((int64_t)a.kb * (rank + 1) / split);
    const uint32_t tcols = a.np <= 32 ? 32 : a.np <= 64 ? 64 : 128;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        mbar_init(done, 1);
        mbar_init_fence();
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(&tslot), tcols);
        tmem_relinquish();
    }
    if (warp == 4 && elect_one()) {
        prefetch_map(&a.w0);
        prefetch_map(&a.x);
        if (ACT != ACT_NONE) prefetch_map(&a.w1);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tslot;
    bool failed = false;
    if (!EARLY) {
        griddep_wait();
        griddep_launch_dependents();   // (after the wait: see the loads below)
    }

    if (warp == 4) {
        const uint32_t ring = smem_u32(smem);
        int s = 0;
        uint32_t ph = 0;
        auto load_w = [&](int kb, uint32_t dst, uint32_t bar) {
            if (ACT == ACT_NONE) {
                tma_load_2d(dst, &a.w0, kb * ELEMS, tile * 128, bar);
            } else {
                tma_load_2d(dst, &a.w0, kb * ELEMS, tile * 64, bar);
                tma_load_2d(dst + 8192, &a.w1, kb * ELEMS, tile * 64, bar);
            }
        };
        // The last product's weights are asked for before the kernel ahead has
        // finished: that kernel let this one start only after its own wait, so
        // whatever wrote the weights is done; its output h is waited for.
        const int ahead = EARLY ? (kb1 - kb0 < a.stages ? kb1 - kb0 : a.stages) : 0;
        if (EARLY) {
            if (elect_one())
                for (int i = 0; i < ahead; ++i) {
                    mbar_arrive_expect_tx(full + 8 * i, a.stage_bytes);
                    load_w(kb0 + i, ring + i * a.stage_bytes, full + 8 * i);
                }
            griddep_wait();
            griddep_launch_dependents();
        }
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, pair_wait(empty + 8 * s, ph ^ 1u, a.st.wait_ns))) {
                failed = true;
                break;
            }
            if (elect_one()) {
                const uint32_t dst = ring + s * a.stage_bytes, bar = full + 8 * s;
                if (kb - kb0 >= ahead) {
                    mbar_arrive_expect_tx(bar, a.stage_bytes);
                    load_w(kb, dst, bar);
                }
                tma_load_2d(dst + 16384, &a.x, kb * ELEMS, 0, bar);
            }
            if (++s == a.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
        if (failed) {
            // (copies in flight land before the memory is given back)
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000) __nanosleep(1000);
        }
    } else if (warp == 5) {
        const uint32_t ring16 = smem_u32(smem) >> 4;
        const uint32_t idesc = idesc_pair(Q8 ? MMA_E4M3 : MMA_BF16, false, false, 128, 0) | (uint32_t)(a.np >> 3) << 17;
        int s = 0;
        uint32_t ph = 0;
#pragma unroll 1
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, pair_wait(full + 8 * s, ph, a.st.wait_ns))) {
                failed = true;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint32_t a16 = ring16 + s * (a.stage_bytes >> 4);
                const int steps = kblock_steps(a.k, kb, ELEMS);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < steps)
                        mma_one<Q8 ? MMA_E4M3 : MMA_BF16>(tmem, PairOperand<false>::desc(a16, k),
                                                          PairOperand<false>::desc(a16 + 1024, k), idesc,
                                                          (kb != kb0) | (k != 0));
                mma_commit(empty + 8 * s);
                if (kb == kb1 - 1) mma_commit(done);
            }
            if (++s == a.stages) {
                s = 0;
                ph ^= 1u;
            }
        }
    } else {
        // this CTA's sums to shared memory, [np][128] (the ring is free then:
        // every load has been consumed)
        failed = !__all_sync(0xffffffffu, pair_wait(done, 0, a.st.wait_ns));
        if (!failed) {
            tc_fence_after();
            float *part = reinterpret_cast<float *>(smem) + warp * 32 + lane;
            const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
            for (int n = 0; n < a.np; n += 16) {
                float v[16];
                tmem_ld16(t_lane + n, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(n + i) * 128] = v[i];
            }
        }
    }
    if (EARLY && warp != 4) griddep_wait();   // (out may be what an earlier kernel still reads)
    if (failed && lane == 0) atomicOr(a.st.err, ERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_sync_all();
    // the cluster's CTAs finish every split-th group of output values, four
    // neighbours a thread
    const uint32_t base = smem_u32(smem);
    const int items = a.rows * (W / 4);
    for (int e = rank * FEW_THREADS + (int)threadIdx.x; e < items; e += split * FEW_THREADS) {
        const int t = e / (W / 4), i = e % (W / 4) * 4, c = tile * W + i;
        if (c >= a.cols) continue;   // (cols is a multiple of 8)
        float v[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int r = 0; r < split; ++r) {
            const uint32_t at = map_rank(base + (uint32_t)(t * 128 + i) * 4, r);
            add4(v, ld_cluster(at));
            if (ACT != ACT_NONE) add4(u, ld_cluster(at + 64 * 4));
        }
        if (Q8) {
            const float sx = a.sx[t];
            const float4 p = *reinterpret_cast<const float4 *>(a.s0 + c), q = *reinterpret_cast<const float4 *>(a.s1 + c);
            v[0] *= sx * p.x; v[1] *= sx * p.y; v[2] *= sx * p.z; v[3] *= sx * p.w;
            u[0] *= sx * q.x; u[1] *= sx * q.y; u[2] *= sx * q.z; u[3] *= sx * q.w;
        }
        if (a.b0) add4(v, a.b0 + c);
        if (ACT == ACT_NONE) {
            if (a.residual) add4(v, a.residual + (int64_t)t * a.ld + c);
        } else {
            if (a.b1) add4(u, a.b1 + c);
#pragma unroll
            for (int k = 0; k < 4; k += 2)
                unpack2(mul2(activate2<ACT>(pack2(v[k], v[k + 1])), pack2(u[k], u[k + 1])), v[k], v[k + 1]);
        }
        *reinterpret_cast<uint2 *>(a.out + (int64_t)t * a.ld + c) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
    if (split > 1) cluster_sync_all();   // (the others have read this CTA's sums)
    if (warp == 5) tmem_dealloc(tmem, tcols);
}

template <int ACT, bool Q8>
cudaError_t launch_few(FewArgs &a, int width, cudaStream_t stream)
{
    constexpr int W = ACT == ACT_NONE ? 128 : 64;
    a.kb = (a.k + (Q8 ? 127 : 63)) / (Q8 ? 128 : 64);
    // CTAs a tile: until there is one for every SM, with two K blocks each at least
    const int tiles = (width + W - 1) / W;
    a.split = 1;
    while (a.split < 8 && tiles * a.split < sm_count() && a.kb >= 4 * a.split) a.split *= 2;
    // two CTAs an SM (three stages with 128 rows, up to six with 16)
    a.stage_bytes = 16384 + a.np * 128;
    a.stages = 110 * 1024 / a.stage_bytes;
    static_assert(110 * 1024 / (16384 + 16 * 128) <= FEW_MAX_STAGES && 3 * (16384 + 128 * 128) <= 110 * 1024, "ring");
    const size_t smem = 1024 + (size_t)a.stages * a.stage_bytes;
    static std::atomic<uint64_t> ready;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(few_rows_kernel<ACT, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize, 111 * 1024);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(tiles * a.split));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.split;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, few_rows_kernel<ACT, Q8>, a);
}

} // namespace

cudaError_t launch_few_up(const FewUp &u, DeviceStatus st, cudaStream_t stream)
{
    FewArgs a;
    memset(&a, 0, sizeof(a));
    const int e8 = u.sx ? 1 : 2;
    const CUtensorMapDataType type = u.sx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    a.rows = u.rows;
    a.np = (u.rows + 15) / 16 * 16;
    cudaError_t e;
    if ((e = make_tensor_map(&a.w0, type, u.wg, u.C, u.F, (int64_t)u.C * e8, 128 / e8, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.w1, type, u.wu, u.C, u.F, (int64_t)u.C * e8, 128 / e8, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.x, type, u.x, u.C, u.rows, (int64_t)u.C * e8, 128 / e8, a.np, 128)) != cudaSuccess) return e;
    a.b0 = u.bg;
    a.b1 = u.bu;
    a.sx = u.sx;
    a.s0 = u.sg;
    a.s1 = u.su;
    a.out = u.h;
    a.cols = u.F;
    a.ld = u.ldh;
    a.k = u.C;
    a.st = st;
    if (u.gelu) return u.sx ? launch_few<ACT_GELU, true>(a, u.F, stream) : launch_few<ACT_GELU, false>(a, u.F, stream);
    return u.sx ? launch_few<ACT_SILU, true>(a, u.F, stream) : launch_few<ACT_SILU, false>(a, u.F, stream);
}

cudaError_t launch_few_down(const bf16 *h, int ldh, int rows, const bf16 *wd, const bf16 *bd, const bf16 *residual,
                            bf16 *out, int C, int F, DeviceStatus st, cudaStream_t stream)
{
    FewArgs a;
    memset(&a, 0, sizeof(a));
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    a.rows = rows;
    a.np = (rows + 15) / 16 * 16;
    cudaError_t e;
    if ((e = make_tensor_map(&a.w0, type, wd, F, C, (int64_t)F * 2, 64, 128, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.x, type, h, F, rows, (int64_t)ldh * 2, 64, a.np, 128)) != cudaSuccess) return e;
    a.b0 = bd;
    a.residual = residual;
    a.out = out;
    a.cols = a.ld = C;
    a.k = F;
    a.st = st;
    return launch_few<ACT_NONE, false>(a, C, stream);
}

} // namespace swin
