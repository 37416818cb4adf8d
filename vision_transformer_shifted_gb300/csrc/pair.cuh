// The CTA-pair GEMM skeleton of the gated feed-forward kernels: persistent
// clusters of two CTAs, each pair computing 256-row tiles with
// tcgen05.mma.cta_group::2 (each CTA holds half of the rows of A, half of the
// rows of B and the accumulators of its 128 rows), operands staged by TMA in a
// ring of shared-memory stages, accumulators handed to 8 or 16 epilogue warps.
//
// Why pairs: a 256 x 256 x 64 step reads 32 KB of shared memory a CTA for 2 x
// 256 x 256 x 64 FLOPs a pair, half of what two independent 128 x 256 tiles
// read, which is what lets the tensor cores run at their rate.
//
// Roles: warp 0 loads (one thread in each CTA, its own halves, signalling the
// leader's barrier), warp 1 of the leader issues the MMAs, the other warps of
// both CTAs drain (warp w owns TMEM lane quarter w % 4 and a share of the
// columns).  Every wait is bounded; on expiry the error word is set, the
// roles leave, and the CTAs meet at the closing cluster barrier.
//
// A policy P describes the kernel:
//   Args                    kernel parameters (np: pairs launched; st: DeviceStatus)
//   Unit, count(a, pair), decode(a, pair, n)   a pair's work items (a tile, or
//                           a range of a tile's K blocks)
//   STAGES, STAGE_BYTES     the ring
//   EPI, GROUPS             epilogue warps; they drain units all together, or as
//                           two groups in turn (GROUPS = 2): where the epilogue
//                           binds, one group's latencies pass under the other's work
//   STAGING                 bytes of shared memory per epilogue warp, laid out by
//                           the epilogue (staged stores, vectors)
//   CHAIN                   its Args have a `chain` (CHAIN_*): the kernel may be one that
//                           runs beside the kernel before it
//   SEGS                    accumulation segments of a unit (each a K loop
//                           into one slot of TMEM columns)
//   slot(seg, n), slot_col(slot), slot_use(seg, n)   the slot of the n-th unit
//                           of this pair, its first column, how often it was used
//   kblocks(a, u, seg), tx(a, u, seg), load(...), mma(...)
//   prefetch_maps(a, pair, rank)   fetches the tensor maps this CTA begins with
//   side(a, w, lane)        what epilogue warp w of the launch does before its first
//                           accumulators are ready, if anything
//   Pre, prefetch(...), epilogue(...)   what an epilogue thread fetches before
//                           the accumulators are ready, and the epilogue
#pragma once

#include <atomic>

#include "common.cuh"
#include "ptx.cuh"

namespace swin {

constexpr int PAIR_SLOTS = 3;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Cluster address of the shared-memory location `addr` in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Arrival on a barrier of either CTA.  What is handed over so lies in TMEM
// (ordered by the tcgen05 fences) or is read by the MMAs through the async
// proxy (ordered by the proxy fence): no generic access of the other CTA hangs
// on it, and the cluster-wide release, which waits for all of a thread's
// earlier writes, is not needed (it cost the narrow forward 20 of 117 us).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// Bounded wait as mbar_wait, for waits that are rarely over before they begin:
// the suspending form at once, the clock (slow to read) only if it ran out.
__device__ __forceinline__ bool pair_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    uint64_t t0 = 0;
#pragma unroll 1
    while (true) {
        if (mbar_try_wait_hint(bar, parity, 1000000u)) return true;
        const uint64_t t = global_timer_ns();
        if (!t0) t0 = t;
        else if (t - t0 > limit_ns) return false;
    }
}
// The same for a whole warp, with one outcome.
__device__ __forceinline__ bool warp_pair_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns)
{
    return __all_sync(0xffffffffu, pair_wait(bar, parity, limit_ns));
}
// True in one lane of a converged warp (the same one every time).
__device__ __forceinline__ bool elect_one()
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}
// 2-D TMA load into this CTA's shared memory, completing on a barrier that may
// be the peer's (cluster address).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const void *tmap, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Brings a tensor map (a kernel parameter) to where the copy engine reads it.
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(ncols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Arrives on the barrier at this offset in both CTAs when the MMAs issued so
// far have completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

enum { MMA_BF16 = 0, MMA_E4M3 = 1 };
template <int KIND>
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc)
{
    if (KIND == MMA_BF16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
            : "memory");
}
// Instruction descriptor: fp32 accumulator, bf16 or e4m3 operands, each K-major
// or MN-major (bf16 only), M x N.
__host__ __device__ constexpr uint32_t idesc_pair(int kind, bool a_mn, bool b_mn, int M, int N)
{
    return (1u << 4) | (kind == MMA_BF16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) |
           (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// Operand tiles, 128-byte swizzle.  K-major: rows of 128 bytes of K, 8-row
// atoms stacked densely; a step of 32 bytes of K moves the start by 32.
// MN-major: boxes of 64 MN elements (128 bytes) x 64 k, boxes 8 KB apart; a step
// of 16 k moves the start by 16 rows.  Descriptors as two words: the upper is a
// constant, the lower a constant plus the address in 16-byte units, so that the
// issuing thread spends an addition per operand and MMA.
template <bool MN>
struct PairOperand {
    static constexpr uint32_t STEP = MN ? 128 : 2;
    static constexpr uint32_t LO = (MN ? 8192u >> 4 : 1u) << 16;
    static constexpr uint32_t HI = (1024u >> 4) | 1u << 14 | (uint32_t)SWZ_128B << 29;
    static __device__ __forceinline__ uint64_t desc(uint32_t addr16, int k)
    {
        return (uint64_t)HI << 32 | (uint64_t)((addr16 | LO) + STEP * k);
    }
};
// The MMAs of one K block: operands at a16, b16 (16-byte units), `steps` of its
// four steps (fewer in the last block of a K that ends inside it).
template <int KIND, bool A_MN, bool B_MN>
__device__ __forceinline__ void mma_kblock(uint32_t d, uint32_t a16, uint32_t b16, uint32_t idesc, int steps, bool first)
{
    mma_pair<KIND>(d, PairOperand<A_MN>::desc(a16, 0), PairOperand<B_MN>::desc(b16, 0), idesc, !first);
    if (steps == 4) {
#pragma unroll
        for (int k = 1; k < 4; ++k)
            mma_pair<KIND>(d, PairOperand<A_MN>::desc(a16, k), PairOperand<B_MN>::desc(b16, k), idesc, 1);
    } else {
#pragma unroll 1
        for (int k = 1; k < steps; ++k)
            mma_pair<KIND>(d, PairOperand<A_MN>::desc(a16, k), PairOperand<B_MN>::desc(b16, k), idesc, 1);
    }
}
// MMA steps of K block kb of a K of `k` elements (block: 128 bytes, four steps).
__device__ __forceinline__ int kblock_steps(int k, int kb, int elems)
{
    const int left = k - kb * elems, per = elems / 4;
    return left >= elems ? 4 : (left + per - 1) / per;
}

template <class P>
struct PairSmem {
    static constexpr int BARS = 2 * P::STAGES + 2 * PAIR_SLOTS;
    static constexpr size_t ring = (size_t)P::STAGES * P::STAGE_BYTES;
    static constexpr size_t bytes = 1024 + ring + P::EPI * P::STAGING + BARS * 8 + 16;
    static_assert(bytes <= 227 * 1024, "shared memory");
};

// Order of an mt x nt grid of tiles: bands of eight row tiles, column by column
// inside a band, so that the tiles in flight share rows of A and of B in L2.
__device__ __forceinline__ void tile_order(int t, int mt, int nt, int &m, int &n)
{
    const int band = t / (8 * nt), r = t - band * 8 * nt;
    const int h = mt - band * 8 < 8 ? mt - band * 8 : 8;
    n = r / h;
    m = band * 8 + (r - n * h);
}

// Tiles dealt out in turn: pair, pair + np, ...
__device__ __forceinline__ int deal_count(int tiles, int np, int pair)
{
    return pair < tiles ? (tiles - pair + np - 1) / np : 0;
}

// The same with a last round that would leave half of the pairs idle or more
// dealt out as halves or quarters of its tiles' columns (`parts`): unit n of a
// pair is tile t, from column `col` on, `width` of 128 columns.
struct PairDeal {
    int tiles, np;
    int full, parts;   // rounds of whole tiles; parts of a tile in the round after them
    __device__ __forceinline__ int count(int pair) const
    {
        return parts == 1 ? deal_count(tiles, np, pair) : full + (pair < (tiles - full * np) * parts);
    }
    __device__ __forceinline__ int tile(int pair, int n, int &col, int &width) const
    {
        const bool whole = parts == 1 || n < full;
        width = whole ? 128 : 128 / parts;
        col = whole ? 0 : pair % parts * width;
        return whole ? pair + n * np : full * np + pair / parts;
    }
};
inline PairDeal deal_tiles(int tiles, int pairs)
{
    PairDeal d{};
    d.tiles = tiles;
    d.full = tiles / pairs;
    const int rest = tiles - d.full * pairs;
    d.parts = rest == 0 ? 1 : 4 * rest <= pairs ? 4 : 2 * rest <= pairs ? 2 : 1;
    d.np = d.full ? pairs : rest * d.parts;
    return d;
}

// The k-th of the last min(stages, issued) uses of a ring's stages by `issued` K
// blocks: its stage, and the parity of the phase that its release completes.
struct RingUse {
    int stage;
    uint32_t parity;
};
__host__ __device__ inline RingUse last_use(int stages, int issued, int k)
{
    const int i = issued - (issued < stages ? issued : stages) + k;
    return {i % stages, (uint32_t)(i / stages) & 1u};
}

// A kernel that reads nothing of the one before it need not wait but at its end, if
// that one let it start only after its own wait: all that it reads was then written by
// kernels which had completed, their writes performed, before this one's first block
// began.  That is the order of completion; griddepcontrol.wait promises visibility to
// the grid that waits, which is the one before.  So an early kernel reads global memory
// through L2 only, where those writes are: tiles by TMA, everything else by loads that
// pass L1 over (load_l2), in which lines from before them could lie.
enum { CHAIN_NONE = 0, CHAIN_EARLY = 1 };

template <class P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(64 + 32 * P::EPI, 1)
pair_kernel(const __grid_constant__ typename P::Args a)
{
    using L = PairSmem<P>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align(smem_raw, 1024);
    uint8_t *staging = smem + L::ring;
    uint64_t *bars = reinterpret_cast<uint64_t *>(staging + P::EPI * P::STAGING);
    const uint32_t full = smem_u32(bars), empty = full + 8 * P::STAGES, tfull = empty + 8 * P::STAGES,
                   tempty = tfull + 8 * PAIR_SLOTS;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + L::BARS);
    // (from one lane: the compiler then knows it for the same in all of them)
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, units = P::count(a, pair);

    if (threadIdx.x == 0) {
        for (int s = 0; s < P::STAGES; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int s = 0; s < PAIR_SLOTS; ++s) {
            mbar_init(tfull + 8 * s, 1);
            mbar_init(tempty + 8 * s, 2 * P::EPI / P::GROUPS);   // (the leader's: a group's warps in both CTAs)
        }
        mbar_init_fence();
    }
    if (warp == 0 && elect_one()) P::prefetch_maps(a, pair, rank);
    if (warp == 1) tmem_alloc_pair(smem_u32(tslot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    bool failed = false;
    // launched while the kernel before it drains: no global memory is touched
    // until that kernel, and so every earlier one, has completed
    bool late = false;
    if constexpr (P::CHAIN) late = a.chain == CHAIN_EARLY;
    if (late) {
        griddep_launch_dependents();
    } else if (P::CHAIN) {   // (after the wait: the next kernel may be an early one)
        griddep_wait();
        griddep_launch_dependents();
    } else {
        griddep_launch_dependents();
        griddep_wait();
    }

    // The two issuing warps run their loops as whole warps and let one lane
    // issue: addresses and descriptors then stay in uniform registers.  (With
    // the loops inside a one-lane branch, a K block cost its issuing thread
    // some 500 cycles, more than the MMAs of a 256 x 128 tile take.)
    if (warp == 0) {
        const uint32_t ring = smem_u32(smem), lead_full = map_rank(full, 0);
        int s = 0, issued = 0;
        uint32_t ph = 0;
#pragma unroll 1
        for (int n = 0; n < units && !failed; ++n) {
            const typename P::Unit un = P::decode(a, pair, n);
#pragma unroll 1
            for (int seg = 0; seg < P::SEGS && !failed; ++seg) {
                const int kb_n = P::kblocks(a, un, seg);
                const uint32_t tx = P::tx(a, un, seg);
#pragma unroll 1
                for (int kb = 0; kb < kb_n; ++kb) {
                    if (!warp_pair_wait(empty + 8 * s, ph ^ 1u, a.st.wait_ns)) {
                        failed = true;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, tx);
                        P::load(a, un, seg, kb, rank, ring + s * P::STAGE_BYTES, lead_full + 8 * s);
                    }
                    ++issued;
                    if (++s == P::STAGES) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        // every stage given back: no commit is on its way to this CTA's
        // barriers when it ends
        for (int k = 0; k < P::STAGES && k < issued && !failed; ++k) {
            const RingUse u = last_use(P::STAGES, issued, k);
            failed = !warp_pair_wait(empty + 8 * u.stage, u.parity, a.st.wait_ns);
        }
        if (failed) {
            // copies in flight land before this CTA's memory is given back:
            // the leader's barriers say so for both CTAs
            if (rank == 0)
                for (int k = 0; k < P::STAGES && k < issued; ++k) {
                    if (--s < 0) {
                        s = P::STAGES - 1;
                        ph ^= 1u;
                    }
                    pair_wait(full + 8 * s, ph, a.st.wait_ns);
                }
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000) __nanosleep(1000);
        }
    } else if (warp == 1) {
        if (rank == 0) {
            const uint32_t ring16 = smem_u32(smem) >> 4;
            int s = 0, n = 0;
            uint32_t ph = 0;
#pragma unroll 1
            for (; n < units && !failed; ++n) {
                const typename P::Unit un = P::decode(a, pair, n);
#pragma unroll 1
                for (int seg = 0; seg < P::SEGS && !failed; ++seg) {
                    const int slot = P::slot(seg, n), kb_n = P::kblocks(a, un, seg);
                    if (!warp_pair_wait(tempty + 8 * slot, (P::slot_use(seg, n) & 1) ^ 1,
                                                                 a.st.wait_ns)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + P::slot_col(slot);
#pragma unroll 1
                    for (int kb = 0; kb < kb_n; ++kb) {
                        if (!warp_pair_wait(full + 8 * s, ph, a.st.wait_ns)) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            P::mma(a, un, seg, kb, ring16 + s * (P::STAGE_BYTES >> 4), d);
                            mma_commit_pair(empty + 8 * s);
                            if (kb == kb_n - 1) mma_commit_pair(tfull + 8 * slot);
                        }
                        if (++s == P::STAGES) {
                            s = 0;
                            ph ^= 1u;
                        }
                    }
                }
            }
        }
    } else {
        constexpr int TEAM = P::EPI / P::GROUPS;
        const int quad = warp & 3, part = (warp - 2) % TEAM >> 2;   // (part: of the columns)
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
        P::side(a, (int)blockIdx.x * P::EPI + warp - 2, lane);
        for (int n = (warp - 2) / TEAM; n < units && !failed; n += P::GROUPS) {
            const typename P::Unit un = P::decode(a, pair, n);
            // (warp-uniform outcome: the TMEM loads below are warp-collective)
            const typename P::Pre pre = P::prefetch(a, un, rank, warp - 2, quad, part, lane, staging);
            for (int seg = 0; seg < P::SEGS && !failed; ++seg)
                failed = !warp_pair_wait(tfull + 8 * P::slot(seg, n), P::slot_use(seg, n) & 1, a.st.wait_ns);
            if (failed) break;
            tc_fence_after();
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    for (int seg = 0; seg < P::SEGS; ++seg)
                        mbar_arrive_cluster(map_rank(tempty + 8 * P::slot(seg, n), 0));
            };
            P::epilogue(a, un, pre, n, rank, warp - 2, quad, part, lane, t_lane, staging, release);
        }
        // the staged stores have read shared memory, and are complete
        if (lane == 0) bulk_wait_all();
    }
    if (failed && lane == 0) atomicOr(a.st.err, ERR_TIMEOUT);
    if (late) griddep_wait();   // (whoever waits for this kernel waits for the one beside it too)
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

template <class P>
cudaError_t launch_pair(const typename P::Args &a, cudaStream_t stream)
{
    constexpr size_t smem = PairSmem<P>::bytes;
    static std::atomic<uint64_t> ready;   // devices whose copy of the kernel may use this much shared memory
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load() & bit)) {
        e = cudaFuncSetAttribute(pair_kernel<P>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit);
    }
    return launch_maybe_overlapped(pair_kernel<P>, dim3(2u * (unsigned)a.np), dim3(64 + 32 * P::EPI), smem, stream, 1, a);
}

} // namespace swin
