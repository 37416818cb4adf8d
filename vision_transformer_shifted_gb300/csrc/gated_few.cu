// The gated block's forward, the linear operator's and its dx for few rows (single
// tokens, small batches), where the weights' one trip from HBM is the work: each
// product with the weights as the MMA's A operand (128 weight rows) and the rows of
// x as its narrow B (16 to 128 columns), so that no row of the tensor-core tile is
// idle weight traffic.
//
// A CTA takes one tile of 128 weight rows (64 of Wg and the same 64 of Wu, or
// 128 of Wd) and a share of K; the CTAs of a cluster share a tile's K (up to
// eight, the linear operator's few tiles sixteen), which spreads few tiles over
// the SMs without partial sums in global memory: each CTA leaves its fp32 tile in
// shared memory and the cluster's CTAs add their shares of it through distributed
// shared memory, in rank order.
// Weights stream through a TMA ring of about 100 KB a CTA, two CTAs an SM: HBM
// bounds it, and the latency of two launches (9 us + bytes / 7.07 TB/s over the
// sizes; 1 x 2048 x 5632: 20 us, 24 rows from e4m3 4096 x 11264: 37).
//
// The linear operator's dx = dz W has the same form with W as stored, [K, 128
// columns], MN-major (30 x 3992 to 1296, with dW and db: 16.3 us, 28.2 by pairs of
// CTAs).  A few hundred rows with a long K go through in chunks of 128, each with
// its own pass over the weights, the later ones from L2.
#include <atomic>
#include <cstring>
#include <type_traits>

#include "gated.cuh"

namespace swin {

namespace {

constexpr int FEW_THREADS = 192;   // four draining warps, a loading and an issuing one
// What a launch computes: the gated block's first products with the activation
// (FORM_UP + ACT_*), its last product, the linear operator, or its dx (these two in
// chunks of 128 rows).
enum { FORM_UP = 0, FORM_DOWN = -1, FORM_LINEAR = -2, FORM_DX = -3 };
constexpr int FEW_MAX_STAGES = 11;
constexpr int FEW_RING = 110 * 1024, FEW_RING_ALONE = 200 * 1024;   // bytes, of two CTAs an SM and of one

struct FewArgs {
    CUtensorMap w0, w1, x;         // up: Wg, Wu (boxes of 64 rows); else Wd or W (128 rows); x: np rows
    const bf16 *b0, *b1;           // up: bg, bu; else bd or b
    const float *sx, *s0, *s1;     // 8-bit: scales of x, Wg (W), Wu
    const bf16 *residual;
    bf16 *out;                     // [rows, ld]: h, or the output
    bf16 *z;                       // linear: as out, the value before the activation, or null
    int act;                       // linear: ACT_*
    int rows, np;                  // np: rows rounded up to 16 (linear: of a chunk, 128 of more rows)
    int tiles;                     // of weight rows, in each chunk of rows
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
__device__ __forceinline__ void add4(float (&s)[4], const uint2 &u)   // (bf16)
{
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

template <int FORM, bool Q8>
__global__ void __launch_bounds__(FEW_THREADS) few_rows_kernel(const __grid_constant__ FewArgs a)
{
    constexpr int ELEMS = Q8 ? 128 : 64;            // K elements of a block
    constexpr int W = FORM < FORM_UP ? 128 : 64;   // output columns of a tile
    constexpr bool EARLY = FORM == FORM_DOWN, CHUNKS = FORM <= FORM_LINEAR, A_MN = FORM == FORM_DX;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align(smem_raw, 1024);
    __shared__ uint64_t bars[2 * FEW_MAX_STAGES + 1];
    __shared__ uint32_t tslot;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * FEW_MAX_STAGES, done = empty + 8 * FEW_MAX_STAGES;
    const int split = a.split, rank = (int)(blockIdx.x % split);
    const int tile = (int)(blockIdx.x / split) % a.tiles, row0 = CHUNKS ? (int)(blockIdx.x / split) / a.tiles * FEW_ROWS : 0;
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
        if (FORM >= FORM_UP) prefetch_map(&a.w1);
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
            if (A_MN) {
                tma_load_2d(dst, &a.w0, tile * 128, kb * ELEMS, bar);
                tma_load_2d(dst + 8192, &a.w0, tile * 128 + 64, kb * ELEMS, bar);
            } else if (FORM < FORM_UP) {
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
                tma_load_2d(dst + 16384, &a.x, kb * ELEMS, row0, bar);
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
        // (without the CTA's rank in the cluster, which a shared-memory address holds above
        // its 18 bits: it would end up in the descriptor's leading byte offset)
        const uint32_t ring16 = (smem_u32(smem) & 0x3ffffu) >> 4;
        const uint32_t idesc = idesc_pair(Q8 ? MMA_E4M3 : MMA_BF16, A_MN, false, 128, 0) | (uint32_t)(a.np >> 3) << 17;
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
                        mma_one<Q8 ? MMA_E4M3 : MMA_BF16>(tmem, PairOperand<A_MN>::desc(a16, k),
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
    // the cluster's CTAs finish every split-th group of output values, four
    // neighbours a thread, always of the same columns
    const uint32_t base = smem_u32(smem);
    const int rows = CHUNKS && a.rows - row0 > FEW_ROWS ? FEW_ROWS : a.rows - row0;
    const int first = rank * FEW_THREADS + (int)threadIdx.x, i = first % (W / 4) * 4, c = tile * W + i;
    const bool in = c < a.cols;   // (cols is a multiple of 8)
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 s0 = Q8 && in ? *reinterpret_cast<const float4 *>(a.s0 + c) : zero,
                 s1 = Q8 && FORM >= FORM_UP && in ? *reinterpret_cast<const float4 *>(a.s1 + c) : zero;
    const uint2 none = make_uint2(0, 0);
    const uint2 b0 = a.b0 && in ? *reinterpret_cast<const uint2 *>(a.b0 + c) : none,
                b1 = FORM >= FORM_UP && a.b1 && in ? *reinterpret_cast<const uint2 *>(a.b1 + c) : none;
    if (split > 1) cluster_sync_all();
    const int step = split * FEW_THREADS / (W / 4);   // rows between a thread's
    auto finish = [&](auto at_once) {
        constexpr int N = decltype(at_once)::value;
#pragma unroll 1
        for (int r0 = first / (W / 4); in && r0 < rows; r0 += N * step) {
            float v[N][4], u[N][4], sx[N];
            uint2 res[N];
            int row[N];   // (past the end the first one again)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                row[j] = r0 + j * step < rows ? r0 + j * step : r0;
                const int64_t t = row0 + row[j];
                res[j] = FORM < FORM_UP && a.residual ? *reinterpret_cast<const uint2 *>(a.residual + t * a.ld + c) : none;
                sx[j] = Q8 ? a.sx[t] : 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) v[j][k] = u[j][k] = 0.f;
            }
#pragma unroll(N == 1 ? 4 : 1)
            for (int r = 0; r < split; ++r) {
                float4 w[N], x[N];
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const uint32_t at = map_rank(base + (uint32_t)(row[j] * 128 + i) * 4, r);
                    w[j] = ld_cluster(at);
                    if (FORM >= FORM_UP) x[j] = ld_cluster(at + 64 * 4);
                }
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    add4(v[j], w[j]);
                    if (FORM >= FORM_UP) add4(u[j], x[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (j && r0 + j * step >= rows) break;
                const int64_t at = (int64_t)(row0 + row[j]) * a.ld + c;
                float *p = v[j], *q = u[j];
                if (Q8) {
                    p[0] *= sx[j] * s0.x; p[1] *= sx[j] * s0.y; p[2] *= sx[j] * s0.z; p[3] *= sx[j] * s0.w;
                    if (FORM >= FORM_UP) {
                        q[0] *= sx[j] * s1.x; q[1] *= sx[j] * s1.y; q[2] *= sx[j] * s1.z; q[3] *= sx[j] * s1.w;
                    }
                }
                if (a.b0) add4(v[j], b0);
                if (FORM == FORM_LINEAR) {
                    if (a.z) *reinterpret_cast<uint2 *>(a.z + at) = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
#pragma unroll
                    for (int k = 0; k < 4; k += 2) {
                        const f2 g = pack2(p[k], p[k + 1]);
                        unpack2(a.act == ACT_SILU ? activate2<ACT_SILU>(g) : a.act == ACT_GELU ? activate2<ACT_GELU>(g) : g, p[k],
                                p[k + 1]);
                    }
                }
                if (FORM < FORM_UP) {
                    if (a.residual) add4(v[j], res[j]);
                } else {
                    if (a.b1) add4(u[j], b1);
#pragma unroll
                    for (int k = 0; k < 4; k += 2)
                        unpack2(mul2(activate2<(FORM < FORM_UP ? ACT_NONE : FORM)>(pack2(p[k], p[k + 1])), pack2(q[k], q[k + 1])),
                                p[k], p[k + 1]);
                }
                *reinterpret_cast<uint2 *>(a.out + at) = make_uint2(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]));
            }
        }
    };
    // The linear operator's few CTAs a tile take their many rows several at a time, so
    // that the latencies of shared memory, the residual and the scales pass together
    // (126 x 256 x 768 9.1 us and 6.3, 128 x 512 x 512 9.2 and 7.3; clusters of eight or
    // sixteen have the loads of their ranks in flight: 100 x 4096 x 4096 14.5 and 20.9).
    if (CHUNKS && split <= 2) finish(std::integral_constant<int, 4>{});
    else finish(std::integral_constant<int, 1>{});
    if (split > 1) cluster_sync_all();   // (the others have read this CTA's sums)
    if (warp == 5) tmem_dealloc(tmem, tcols);
}

// Clusters of `split` CTAs that find room at once, of one CTA an SM or two: the
// device's processor clusters differ in size, and a cluster lies in one of them
// (clusters of eight, two CTAs an SM: 36, not 38; of sixteen, one an SM: 7).
// The question is put for a kernel of its own, never launched, with this one's threads
// and shared memory: of one that allocates tensor memory the answer is one CTA an SM,
// whatever it allocates.
__global__ void __launch_bounds__(FEW_THREADS) few_room() {}
int ask_clusters(int split, bool alone)   // (0: no device, a plan is asked for)
{
    int n = 0;
    const void *kern = (const void *)few_room;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr;
    cfg.gridDim = dim3((unsigned)(split * 2 * sm_count()));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = 2048 + (alone ? FEW_RING_ALONE : FEW_RING);   // (and the barriers)
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 2048 + FEW_RING_ALONE) == cudaSuccess &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0)
        return n;
    cudaGetLastError();
    return 0;
}
// ask()'s answer for a device, kept (0: asked again).
template <class Ask>
int clusters_of(int dev, int split, bool alone, Ask &&ask)
{
    static std::atomic<int> known[64][2][17];
    const bool keep = dev >= 0 && dev < 64;
    int n = keep ? known[dev][alone][split].load() : 0;
    if (n) return n;
    n = ask();
    if (keep && n) known[dev][alone][split].store(n);
    return n;
}
int current_device()   // (-1: none)
{
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
    return dev;
}
int few_clusters(int dev, int split, bool alone)
{
    const int n = clusters_of(dev, split, alone, [&] { return ask_clusters(split, alone); });
    return n ? n : (alone ? 1 : 2) * sm_count() / split;
}

template <int FORM, bool Q8>
cudaError_t launch_few(FewArgs &a, int width, cudaStream_t stream)
{
    constexpr int W = FORM < FORM_UP ? 128 : 64;
    a.kb = (a.k + (Q8 ? 127 : 63)) / (Q8 ? 128 : 64);
    // CTAs a tile: until there is one for every SM, with two K blocks each at least
    a.tiles = (width + W - 1) / W;
    const int chunks = FORM <= FORM_LINEAR ? (a.rows + FEW_ROWS - 1) / FEW_ROWS : 1, tiles = a.tiles * chunks;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    a.split = 1;
    while (a.split < 8 && tiles * a.split < sm_count() && a.kb >= 4 * a.split) a.split *= 2;
    if (FORM <= FORM_LINEAR) a.split = few_split(tiles, a.kb);
    // Two CTAs an SM (three stages with 128 rows, up to six with 16), or, from 64 rows,
    // where all clusters find room so, one with twice the ring (128 x 8192 x 512, 32 CTAs,
    // 12.4 us and 11.3; 16 rows no change, and the next kernel starts later; sixteen
    // clusters of eight, of which fifteen fit: 385 x 2968 x 400 9.7 and 12.4).
    const bool alone = FORM <= FORM_LINEAR && a.np >= 64 && tiles <= few_clusters(dev, a.split, true);
    a.stage_bytes = 16384 + a.np * 128;
    a.stages = (alone ? FEW_RING_ALONE : FEW_RING) / a.stage_bytes;
    static_assert(FEW_RING_ALONE / (16384 + 16 * 128) <= FEW_MAX_STAGES && 3 * (16384 + 128 * 128) <= FEW_RING, "ring");
    const size_t smem = 1024 + (size_t)a.stages * a.stage_bytes;
    static std::atomic<uint64_t> ready;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(few_rows_kernel<FORM, Q8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 1024 + (FORM <= FORM_LINEAR ? FEW_RING_ALONE : FEW_RING));
        if (e == cudaSuccess && FORM <= FORM_LINEAR)
            e = cudaFuncSetAttribute(few_rows_kernel<FORM, Q8>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    return cudaLaunchKernelEx(&cfg, few_rows_kernel<FORM, Q8>, a);
}

} // namespace

// As many as two an SM hold in one round (24 rows from e4m3 4096 x 11264, 88 tiles,
// 12.9 us with two, 12.3 with three; one cluster in a second round: 100 x 4096 x 4800, 38
// tiles by eight, 21.6, by six 14.3; 24 x 4096 x 9600, 75 by four, 23.3, by three 17.9),
// up to sixteen where the tiles are so few that one an SM does (128 x 8192 x 512 12.3 us
// by eight, 10.1; 64 x 8192 x 896, seven tiles, 10.4 and 8.9; eight tiles, 128 x 4096 x
// 1024, 9.8 and 12.3), with four K blocks each at least.
int few_split(int64_t tiles, int kb)
{
    const int dev = current_device(), most = tiles <= few_clusters(dev, 16, true) ? 16 : 8;
    int split = 1;
    for (int s = 2; s <= most && kb >= 4 * s; ++s)
        if (tiles <= few_clusters(dev, s, false)) split = s;
    return split;
}

int test_few_clusters_of(int dev, int split, bool alone, int answer)
{
    return clusters_of(dev, split, alone, [&] { return answer; });
}

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
    if (u.gelu) return u.sx ? launch_few<FORM_UP + ACT_GELU, true>(a, u.F, stream) : launch_few<FORM_UP + ACT_GELU, false>(a, u.F, stream);
    return u.sx ? launch_few<FORM_UP + ACT_SILU, true>(a, u.F, stream) : launch_few<FORM_UP + ACT_SILU, false>(a, u.F, stream);
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
    return launch_few<FORM_DOWN, false>(a, C, stream);
}

cudaError_t launch_few_linear(const FewLinear &u, DeviceStatus st, cudaStream_t stream)
{
    FewArgs a;
    memset(&a, 0, sizeof(a));
    const int e8 = u.sx ? 1 : 2;
    const CUtensorMapDataType type = u.sx ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    a.rows = u.rows;
    a.np = u.rows < FEW_ROWS ? (u.rows + 15) / 16 * 16 : FEW_ROWS;
    cudaError_t e;
    if ((e = make_tensor_map(&a.w0, type, u.w, u.C, u.N, (int64_t)u.C * e8, 128 / e8, 128, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.x, type, u.x, u.C, u.rows, (int64_t)u.C * e8, 128 / e8, a.np, 128)) != cudaSuccess) return e;
    a.b0 = u.bias;
    a.sx = u.sx;
    a.s0 = u.sw;
    a.residual = u.residual;
    a.out = u.out;
    a.z = u.z;
    a.act = u.act;
    a.cols = a.ld = u.N;
    a.k = u.C;
    a.st = st;
    return u.sx ? launch_few<FORM_LINEAR, true>(a, u.N, stream) : launch_few<FORM_LINEAR, false>(a, u.N, stream);
}

cudaError_t launch_few_dx(const bf16 *dz, int ld, int rows, const bf16 *w, bf16 *dx, int C, int N, DeviceStatus st,
                          cudaStream_t stream)
{
    FewArgs a;
    memset(&a, 0, sizeof(a));
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    a.rows = rows;
    a.np = rows < FEW_ROWS ? (rows + 15) / 16 * 16 : FEW_ROWS;
    cudaError_t e;
    if ((e = make_tensor_map(&a.w0, type, w, C, N, (int64_t)C * 2, 64, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.x, type, dz, N, rows, (int64_t)ld * 2, 64, a.np, 128)) != cudaSuccess) return e;
    a.out = dx;
    a.cols = a.ld = C;
    a.k = N;
    a.st = st;
    return launch_few<FORM_DX, false>(a, C, stream);
}

} // namespace swin
