// The weight gradient of a linear layer with an activation, dW = dz^T x with dz =
// dy act'(z), from z and dy themselves: a tile has up to 512 columns of dW, so that
// few pairs (up to 512 input channels: one) read an element of z and dy; dz is
// formed in shared memory, where the MMAs read it, and written once for dx's
// product.  As a kernel of its own (act_grad_kernel) dz costs a trip of z and dy
// through the SMs that feeds nothing, and another one of dz.
//
// A CTA pair takes a tile of 256 output channels (128 a CTA, the rows of dW) x up to
// 512 input channels and a slice of the tokens; TMEM holds the tile (up to 512
// columns), the slices' partial tiles are joined by dx's epilogue warps or
// finish_kernel.  Per K block of 64 tokens a CTA loads its 64 x 128 of z and of dy
// (its own barrier) and its half of x's columns (the leader's); sixteen warps turn z
// into dz in place, a 1 KB atom of the swizzled tile (8 tokens x 64 channels) each,
// add up their channels for db, store dz, and release the block to the MMAs.  What
// binds it: up to 256 columns HBM (50176 x 128 x 2048, 617 MB, 96 us: 6.4 TB/s); 512
// columns, 1.1 us a block, both that (without the stores of dz 92 of 111 us at 50176 x
// 512 x 2048) and the formation's instructions (42 a pair of values; without the
// activation 104 us, at 12544 x 1024 x 4096, read from L2 by the second tile, 77 of
// 106).  (z and dy by plain loads into registers, two blocks ahead: 43 us at 12544 x
// 512 x 2048, 36 by TMA; two groups of eight warps at alternate blocks: 36.)
#include <atomic>
#include <cstring>

#include "linear.cuh"

namespace swin {

namespace {

constexpr int WG_WARPS = 16, WG_THREADS = 96 + 32 * WG_WARPS;
constexpr int WG_TILE = 16384;   // z or dy of a block (two boxes of 64 channels x 64 tokens)
// Rings of their own: z's place (then dz's) is free when the MMAs are done, dy's as
// soon as dz is formed, x's comes from L2 and needs the fewest.
template <bool WIDE>   // more than 256 columns
struct WgradRings {
    static constexpr int Z = WIDE ? 4 : 5, Y = WIDE ? 3 : 4, X = WIDE ? 3 : 4, X_BYTES = WIDE ? 32768 : 16384;
    static constexpr int BYTES = (Z + Y) * WG_TILE + X * X_BYTES;
};
// A place in a ring and the parity of its phase.
struct RingAt {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int stages)
    {
        if (++s == stages) {
            s = 0;
            ph ^= 1u;
        }
    }
};

struct WgradArgs {
    CUtensorMap z, dy, x, part;   // part: partial tiles [pairs][256][n] fp32
    bf16 *dz;                     // [rows, ld], or null
    float *sums;                  // [slices, N]: shares of db, or null
    int rows, N, ld;
    int n;                        // columns of a tile, a multiple of 32
    int mt, nt;                   // tiles of dW
    int slices, kb, slice_kb;     // K blocks of all tokens, of a slice
    DeviceStatus st;
};

__device__ __forceinline__ uint32_t b_boxes(int n) { return n / 2 > 64 ? 2 : 1; }   // of a CTA's half of n columns
__device__ __forceinline__ void sts16(uint32_t addr, const uint4 &u)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(u.x), "r"(u.y), "r"(u.z), "r"(u.w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t addr)
{
    uint4 u;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr) : "memory");
    return u;
}

template <int ACT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WG_THREADS, 1)
act_wgrad_kernel(const __grid_constant__ WgradArgs a)
{
    using R = WgradRings<WIDE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align(smem_raw, 1024);
    __shared__ uint64_t bars[3 * R::Z + R::Y + 2 * R::X + 1];
    __shared__ uint32_t tslot;
    __shared__ float red[WG_WARPS][64];
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, slice = pair % a.slices;
    int mtile, ntile;
    tile_order(pair / a.slices, a.mt, a.nt, mtile, ntile);
    const int kb0 = slice * a.slice_kb, kb_n = (a.kb - kb0 < a.slice_kb ? a.kb - kb0 : a.slice_kb);
    const int ch0 = mtile * 256 + (int)rank * 128;   // this CTA's first output channel
    const bool first = ntile == 0;                   // (dz and db are the first column tile's)
    // z and dy have landed (own), dz is formed (the leader's), the MMAs are done with
    // it (both); dy has been read (own); x has landed (the leader's, of both CTAs), the
    // MMAs are done with it (both); the tile is complete (both)
    const uint32_t afull = smem_u32(bars), ready = afull + 8 * R::Z, zempty = ready + 8 * R::Z, yempty = zempty + 8 * R::Z,
                   xfull = yempty + 8 * R::Y, xempty = xfull + 8 * R::X, done = xempty + 8 * R::X;
    if (threadIdx.x == 0) {
        for (int s = 0; s < R::Z; ++s) {
            mbar_init(afull + 8 * s, 1);
            mbar_init(ready + 8 * s, 2 * WG_WARPS);
            mbar_init(zempty + 8 * s, 1);
        }
        for (int s = 0; s < R::Y; ++s) mbar_init(yempty + 8 * s, WG_WARPS);
        for (int s = 0; s < R::X; ++s) {
            mbar_init(xfull + 8 * s, 1);
            mbar_init(xempty + 8 * s, 1);
        }
        mbar_init(done, 1);
        mbar_init_fence();
    }
    if (warp == 0 && elect_one()) {
        prefetch_map(&a.z);
        prefetch_map(&a.dy);
        prefetch_map(&a.x);
        prefetch_map(&a.part);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&tslot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tslot;
    bool failed = false;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t zring = smem_u32(smem), yring = zring + R::Z * WG_TILE, xring = yring + R::Y * WG_TILE;
    const int n0 = a.n < 256 ? a.n : 256, n1 = a.n - n0;   // columns of the one or two MMAs

    if (warp == 0) {
        RingAt z, y;
        int issued = 0;
#pragma unroll 1
        for (int i = 0; i < kb_n; ++i, ++issued, z.next(R::Z), y.next(R::Y)) {
            if (!warp_pair_wait(zempty + 8 * z.s, z.ph ^ 1u, a.st.wait_ns) ||
                !warp_pair_wait(yempty + 8 * y.s, y.ph ^ 1u, a.st.wait_ns)) {
                failed = true;
                break;
            }
            if (elect_one()) {
                const uint32_t zd = zring + z.s * WG_TILE, yd = yring + y.s * WG_TILE, bar = afull + 8 * z.s;
                const int k = (kb0 + i) * 64;
                mbar_arrive_expect_tx(bar, 2 * WG_TILE);
                tma_load_2d(zd, &a.z, ch0, k, bar);
                tma_load_2d(zd + 8192, &a.z, ch0 + 64, k, bar);
                tma_load_2d(yd, &a.dy, ch0, k, bar);
                tma_load_2d(yd + 8192, &a.dy, ch0 + 64, k, bar);
            }
        }
        // every place given back: no commit is on its way to this CTA's barriers
        for (int k = 0; k < R::Z && k < issued && !failed; ++k) {
            const RingUse u = last_use(R::Z, issued, k);
            failed = !warp_pair_wait(zempty + 8 * u.stage, u.parity, a.st.wait_ns);
        }
        if (failed) {
            // (copies in flight land before the memory is given back)
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000) __nanosleep(1000);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t idesc = idesc_pair(MMA_BF16, true, true, 256, 0);
            const uint32_t idesc0 = idesc | (uint32_t)(n0 >> 3) << 17, idesc1 = idesc | (uint32_t)(n1 >> 3) << 17;
            RingAt z, x;
#pragma unroll 1
            for (int i = 0; i < kb_n; ++i, z.next(R::Z), x.next(R::X)) {
                if (!warp_pair_wait(xfull + 8 * x.s, x.ph, a.st.wait_ns) || !warp_pair_wait(ready + 8 * z.s, z.ph, a.st.wait_ns)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t a16 = (zring + z.s * WG_TILE) >> 4, b16 = (xring + x.s * R::X_BYTES) >> 4;
                    const int steps = kblock_steps(a.rows, kb0 + i, 64);
                    mma_kblock<MMA_BF16, true, true>(tmem, a16, b16, idesc0, steps, i == 0);
                    if (WIDE) mma_kblock<MMA_BF16, true, true>(tmem + 256, a16, b16 + 1024, idesc1, steps, i == 0);
                    mma_commit_pair(zempty + 8 * z.s);
                    mma_commit_pair(xempty + 8 * x.s);
                    if (i == kb_n - 1) mma_commit_pair(done);
                }
            }
        }
    } else if (warp == 2) {
        const uint32_t lead = map_rank(xfull, 0), bytes = (b_boxes(n0) + (WIDE ? b_boxes(n1) : 0)) * 8192;
        const int c0 = ntile * a.n + (int)rank * (n0 / 2), c1 = ntile * a.n + 256 + (int)rank * (n1 / 2);
        RingAt x;
        int issued = 0;
#pragma unroll 1
        for (int i = 0; i < kb_n; ++i, ++issued, x.next(R::X)) {
            if (!warp_pair_wait(xempty + 8 * x.s, x.ph ^ 1u, a.st.wait_ns)) {
                failed = true;
                break;
            }
            if (elect_one()) {
                const uint32_t dst = xring + x.s * R::X_BYTES, bar = lead + 8 * x.s;
                const int k = (kb0 + i) * 64;
                if (rank == 0) mbar_arrive_expect_tx(xfull + 8 * x.s, 2 * bytes);
                tma_load_2d_pair(dst, &a.x, c0, k, bar);
                if (b_boxes(n0) > 1) tma_load_2d_pair(dst + 8192, &a.x, c0 + 64, k, bar);
                if (WIDE) {
                    tma_load_2d_pair(dst + 16384, &a.x, c1, k, bar);
                    if (b_boxes(n1) > 1) tma_load_2d_pair(dst + 24576, &a.x, c1 + 64, k, bar);
                }
            }
        }
        for (int k = 0; k < R::X && k < issued && !failed; ++k) {
            const RingUse u = last_use(R::X, issued, k);
            failed = !warp_pair_wait(xempty + 8 * u.stage, u.parity, a.st.wait_ns);
        }
        if (failed) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000) __nanosleep(1000);
        }
    } else {
        const int w = warp - 3;
        // this lane's two 16-byte pieces of the warp's atom: tokens t, t + 4, eight
        // channels (one logical chunk, so that its sums are of fixed channels)
        const int box = w & 1, chunk = lane & 7, t = lane >> 3;
        const uint32_t at0 = (uint32_t)box * 8192 + sw128_offset((w >> 1) * 8 + t, chunk),
                       at1 = (uint32_t)box * 8192 + sw128_offset((w >> 1) * 8 + t + 4, chunk);
        const uint32_t lead_ready = map_rank(ready, 0);
        const int c = ch0 + box * 64 + chunk * 8;
        const bool stored = first && a.dz && c < a.N;
        f2 sum[4] = {0, 0, 0, 0};
        RingAt z, y;
        int64_t row = (int64_t)kb0 * 64 + (w >> 1) * 8 + t;
#pragma unroll 1
        for (int i = 0; i < kb_n; ++i, row += 64, z.next(R::Z), y.next(R::Y)) {
            if (!warp_pair_wait(afull + 8 * z.s, z.ph, a.st.wait_ns)) {
                failed = true;
                break;
            }
            const uint32_t zat = zring + z.s * WG_TILE, yat = yring + y.s * WG_TILE;
            auto grad = [&](uint32_t at, int64_t r) {
                const uint4 zu = lds16(zat + at), du = lds16(yat + at);
                const uint32_t zw[4] = {zu.x, zu.y, zu.z, zu.w}, dw[4] = {du.x, du.y, du.z, du.w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 zf = unpack_bf16x2(zw[e]), df = unpack_bf16x2(dw[e]);
                    f2 act, slope;
                    activate_grad2<ACT>(pack2(zf.x, zf.y), act, slope);
                    const f2 v = mul2(pack2(df.x, df.y), slope);
                    sum[e] = add2(sum[e], v);   // (behind the last token: dy is zero)
                    float lo, hi;
                    unpack2(v, lo, hi);
                    o[e] = pack_bf16x2(lo, hi);
                }
                const uint4 u = make_uint4(o[0], o[1], o[2], o[3]);
                sts16(zat + at, u);
                if (stored && r < a.rows) *reinterpret_cast<uint4 *>(a.dz + r * a.ld + c) = u;
            };
            grad(at0, row);
            grad(at1, row + 4);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_cluster(lead_ready + 8 * z.s);
                mbar_arrive(yempty + 8 * y.s);
            }
        }
        // the lanes' sums, then those of the eight warps of the same channels
        if (first && a.sums) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[2];
                unpack2(sum[e], v[0], v[1]);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[h] += __shfl_xor_sync(0xffffffffu, v[h], 8);
                    v[h] += __shfl_xor_sync(0xffffffffu, v[h], 16);
                    if (lane < 8) red[w][chunk * 8 + 2 * e + h] = v[h];
                }
            }
            asm volatile("bar.sync 1, %0;" ::"n"(32 * WG_WARPS) : "memory");
            const int i = (int)threadIdx.x - 96;
            if (i < 128 && ch0 + i < a.N) {
                float v = 0.f;
                for (int k = 0; k < WG_WARPS / 2; ++k) v += red[2 * k + (i >> 6)][i & 63];
                a.sums[(int64_t)slice * a.N + ch0 + i] = v;
            }
        }
        // the tile's fp32 values, boxes of 16 columns through the free stages
        if (!failed) failed = !warp_pair_wait(done, 0, a.st.wait_ns);
        if (!failed) {
            tc_fence_after();
            const int quad = warp & 3, share = w >> 2;   // (share: of the columns)
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16);
            uint8_t *stage = smem + w * 4096;
            int turn = 0;
#pragma unroll 1
            for (int j = share * 16; j < a.n; j += 64, ++turn) {
                float v[16];
                tmem_ld16(acc + j, v);
                if (lane == 0) bulk_wait_read1();   // (the box written two before)
                __syncwarp();
                tmem_wait_ld();
                uint8_t *to = stage + (turn & 1) * 2048;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4 *>(to + sw64_offset(lane, q)) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                store_box(&a.part, j, pair * 256 + (int)rank * 128 + quad * 32, true, to, lane);
            }
            if (lane == 0) bulk_wait_all();
        }
    }
    if (failed && lane == 0) atomicOr(a.st.err, ERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <int ACT, bool WIDE>
cudaError_t launch(const WgradArgs &a, int pairs, cudaStream_t stream)
{
    constexpr size_t smem = 1024 + WgradRings<WIDE>::BYTES;
    static std::atomic<uint64_t> ready;   // devices whose copy of the kernel may use this much shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(act_wgrad_kernel<ACT, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    return launch_maybe_overlapped(act_wgrad_kernel<ACT, WIDE>, dim3(2u * (unsigned)pairs), dim3(WG_THREADS), smem, stream, 1, a);
}

} // namespace

ActWgradPlan plan_act_wgrad(int C, int N, int rows, const ProductsPlan &apart)
{
    ActWgradPlan p{};
    const int pairs = sm_count() / 2, mt = ceil_div(N, 256), nt = ceil_div(C, 512), tiles = mt * nt, kb = ceil_div(rows, 64);
    if (nt > 4 || tiles > pairs) return p;
    p.n = C < 64 ? 64 : ceil_div(ceil_div(C, nt), 32) * 32;
    p.mt = mt;
    p.nt = nt;
    p.tiles = tiles;
    p.kb = kb;
    p.slice_kb = ceil_div(kb, pairs / tiles);
    p.slices = ceil_div(kb, p.slice_kb);
    p.part_bytes = (size_t)tiles * p.slices * 256 * p.n * sizeof(float);
    // Estimates in us: the trips of z, dy and dz at 6 TB/s (as a launch of their own
    // worse), a K block of a tile here and of a whole tile in dW's own product, launches
    // and joins.  Measured, whole backwards, dz apart and here: 12544 x 512 x 2048 89.2
    // and 61.9, 12544 x 768 x 768 54.2 and 40.7, 5000 x 1000 x 1000 55.7 and 36.0, 3136
    // x 384 x 1536 40.9 and 31.4, 12544 x 1024 x 4096 188 and 182; not taken: 8192 x 2048
    // x 2048 114.5 and 123.1, 3000 x 1024 x 4096 57.2 and 64.6, 2000 x 2048 x 2048 36.7
    // and 54.8, 1500 x 512 x 512 20.4 and 28.1; 40 sizes: 0.8% above the better of both
    // on average.
    const double trips = 6.0 * rows * N / 6.0e6, blocks = p.slice_kb * (0.6 + 0.5 * p.n / 512);
    p.chosen = 14 + (blocks > trips ? blocks : trips) < 10 + 1.25 * trips + 0.00283 * (double)apart.cost;
    return p;
}

cudaError_t launch_act_wgrad(const ActWgrad &w, const ActWgradPlan &p, DeviceStatus st, cudaStream_t stream, JoinArgs *join,
                             int *join_blocks)
{
    WgradArgs a;
    memset(&a, 0, sizeof(a));
    const int pairs = p.tiles * p.slices;
    cudaError_t e;
    if ((e = map_mn(&a.z, w.z, w.rows, w.N)) != cudaSuccess) return e;
    if ((e = map_mn(&a.dy, w.dy, w.rows, w.N)) != cudaSuccess) return e;
    if ((e = map_mn(&a.x, w.x, w.rows, w.C)) != cudaSuccess) return e;
    e = make_tensor_map(&a.part, T_F32, w.part, p.n, (int64_t)pairs * 256, (int64_t)p.n * 4, 16, 32, 64);
    if (e != cudaSuccess) return e;
    a.dz = w.dz;
    a.sums = w.sums;
    a.rows = w.rows;
    a.N = w.N;
    a.ld = w.ld;
    a.n = p.n;
    a.mt = p.mt;
    a.nt = p.nt;
    a.slices = p.slices;
    a.kb = p.kb;
    a.slice_kb = p.slice_kb;
    a.st = st;
    PairSplit &s = join->split;
    s = PairSplit{};
    s.tiles = s.cut = p.tiles;
    s.np = pairs;
    s.k_blocks = p.kb;
    s.q = (uint32_t)p.slice_kb;
    s.kb = p.slice_kb * p.slices;
    join->part = w.part;
    join->slots = 1;
    join->single = true;
    join->tn = p.n;
    join->blocks = p.tiles >= 16 ? 16 : 64;
    join->p[0] = {nullptr, nullptr, w.dW, w.N, w.C, p.mt, p.nt, 0};
    join->p[1].first = join->p[2].first = 0x7fffffff;
    *join_blocks = p.tiles * join->blocks;
    if (p.n > 256) return w.act == ACT_SILU ? launch<ACT_SILU, true>(a, pairs, stream) : launch<ACT_GELU, true>(a, pairs, stream);
    return w.act == ACT_SILU ? launch<ACT_SILU, false>(a, pairs, stream) : launch<ACT_GELU, false>(a, pairs, stream);
}

} // namespace swin
