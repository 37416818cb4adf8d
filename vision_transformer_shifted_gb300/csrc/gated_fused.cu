// The gated block's forward as one kernel for narrow tokens (C <= 128): out =
// residual + (act(x Wg^T + bg) * (x Wu^T + bu)) Wd^T + bd with the hidden
// activation kept on the SM.  At C = 96, F = 256 the hidden activation is 2.7
// times as wide as a token: written and read back it would be 206 of 283 MB of
// traffic for 200,704 tokens; here x, the residual and out remain.
//
// A CTA pair walks 256-row tiles.  The hidden units go in chunks of 64: one 256
// x 128 x C MMA group leaves g in columns 0..63 and u in 64..127 of one of two
// TMEM buffers (the halves of B again from Wg and Wu); one of two groups of
// eight warps forms h and writes it to shared memory as the K-major A operand
// of the last product, whose 256 x C accumulator sums over the chunks in one of
// two more TMEM buffers.  The groups take alternate chunks, and group t mod 2
// drains tile t's output after its first chunk of tile t + 1: neither waits for
// the MMAs of its own last chunk.  Weights stream through a ring of chunks, or
// stay (loaded once) where all chunks fit it.  The activation warps bind, not HBM:
// four a scheduler, some 21 instructions a hidden value with the drain, waiting
// on TMEM and on their own chains in 39% of the issue slots.  200704 x 96 x 256
// with biases and residual takes 49.9 us, 70.5 as two kernels.
#include <atomic>
#include <cstring>

#include "gated.cuh"

namespace swin {

namespace {

constexpr int FUSED_GROUPS = 2, FUSED_GROUP_WARPS = 8;
constexpr int FUSED_THREADS = 128 + 32 * FUSED_GROUPS * FUSED_GROUP_WARPS;   // a loading warp, two issuing ones, one idle
constexpr int FUSED_CHUNK = 64;
constexpr int FUSED_SLOTS = 12;   // most weight chunks in the ring

struct FusedArgs {
    CUtensorMap x, wg, wu, wd, out;
    const bf16 *bg, *bu, *bd, *residual;
    int rows, C, F, tiles, np;
    int xb, n2;              // K blocks of a token; N of the last product (C rounded up to 32: a pair's step)
    int chunks, slots, slot_bytes;
    bool resident;           // every chunk has its slot: loaded once
    bool shared_staging;     // the two groups drain through one staging, in turn
    DeviceStatus st;
};

struct FusedBars {
    uint64_t xfull[2], xempty[2], gfull[2], gempty[2], hready[2], hfree[2], yfull[2], yempty[2];
    uint64_t wfull[FUSED_SLOTS], wempty[FUSED_SLOTS];
    uint64_t sfree[FUSED_GROUP_WARPS];   // a staging's tiles, in turn by the two groups
};

// (position, phase) in a ring.
struct RingPos {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++s == n) {
            s = 0;
            ph ^= 1u;
        }
    }
};

template <int ACT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(FUSED_THREADS, 1)
gated_fused_kernel(const __grid_constant__ FusedArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_align(smem_raw, 1024);
    __shared__ FusedBars bars;
    __shared__ uint32_t tslot;
    __shared__ __align__(16) float vecs[FUSED_GROUPS * FUSED_GROUP_WARPS][64];   // a warp's biases of its 32 hidden units
    // [x 2][h 2][weights slots][staging a warp of a group]
    const uint32_t x_bytes = (uint32_t)a.xb * 16384u;
    uint8_t *sx = smem, *sh = sx + 2 * x_bytes, *sw = sh + 2 * 16384, *stg = sw + (size_t)a.slots * a.slot_bytes;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, my = deal_count(a.tiles, a.np, pair);
    const uint64_t limit = a.st.wait_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.xfull[i]), 1);
            mbar_init(smem_u32(&bars.xempty[i]), 1);
            mbar_init(smem_u32(&bars.gfull[i]), 1);
            mbar_init(smem_u32(&bars.gempty[i]), 2 * FUSED_GROUP_WARPS);
            mbar_init(smem_u32(&bars.hready[i]), 2 * FUSED_GROUP_WARPS);
            mbar_init(smem_u32(&bars.hfree[i]), 1);
            mbar_init(smem_u32(&bars.yfull[i]), 1);
            mbar_init(smem_u32(&bars.yempty[i]), 2 * FUSED_GROUP_WARPS);
        }
        for (int i = 0; i < FUSED_GROUP_WARPS; ++i) mbar_init(smem_u32(&bars.sfree[i]), 1);
        for (int i = 0; i < a.slots; ++i) {
            mbar_init(smem_u32(&bars.wfull[i]), 1);
            mbar_init(smem_u32(&bars.wempty[i]), 1);
        }
        mbar_init_fence();
    }
    if (warp == 0 && elect_one()) {
        prefetch_map(&a.x);
        prefetch_map(rank ? &a.wu : &a.wg);
        prefetch_map(&a.wd);
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&tslot), 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = tslot;
    const uint32_t TY = tmem + 256;   // (output accumulators; g | u at columns 0 and 128)
    bool failed = false;
    griddep_launch_dependents();
    griddep_wait();

    if (warp == 0) {
        // ---------------- loads ----------------
        const uint32_t xfull0 = map_rank(smem_u32(&bars.xfull[0]), 0), wfull0 = map_rank(smem_u32(&bars.wfull[0]), 0);
        RingPos w;
#pragma unroll 1
        for (int i = 0; i < my && !failed; ++i) {
            const int row = (pair + i * a.np) * 256 + (int)rank * 128, b = i & 1;
            if (!warp_pair_wait(smem_u32(&bars.xempty[b]), ((uint32_t)(i >> 1) & 1u) ^ 1u, limit)) {
                failed = true;
                break;
            }
            if (elect_one()) {
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.xfull[b]), 2 * x_bytes);
                for (int k = 0; k < a.xb; ++k)
                    tma_load_2d_pair(smem_u32(sx) + b * x_bytes + k * 16384, &a.x, k * 64, row, xfull0 + 8 * b);
            }
            if (a.resident && i > 0) continue;
#pragma unroll 1
            for (int c = 0; c < a.chunks; ++c) {
                if (!warp_pair_wait(smem_u32(&bars.wempty[w.s]), w.ph ^ 1u, limit)) {
                    failed = true;
                    break;
                }
                if (elect_one()) {
                    const uint32_t dst = smem_u32(sw) + w.s * a.slot_bytes, bar = wfull0 + 8 * w.s;
                    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars.wfull[w.s]), 2 * a.slot_bytes);
                    for (int k = 0; k < a.xb; ++k)
                        tma_load_2d_pair(dst + k * 8192, rank ? &a.wu : &a.wg, k * 64, c * FUSED_CHUNK, bar);
                    tma_load_2d_pair(dst + a.xb * 8192, &a.wd, c * FUSED_CHUNK, (int)rank * (a.n2 / 2), bar);
                }
                w.next(a.slots);
            }
        }
        // every commit on its way to this CTA's barriers has arrived
        for (int i = my > 1 ? my - 2 : 0; i < my && !failed; ++i)
            failed = !warp_pair_wait(smem_u32(&bars.xempty[i & 1]), (uint32_t)(i >> 1) & 1u, limit);
        for (int k = 0; !a.resident && k < a.slots && k < my * a.chunks && !failed; ++k, w.next(a.slots))
            failed = !warp_pair_wait(smem_u32(&bars.wempty[w.s]), w.ph ^ 1u, limit);
        if (failed) {
            // (copies in flight land before the memory is given back)
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < 200000) __nanosleep(1000);
        }
    } else if (warp == 1) {
        // ---------------- g | u MMAs (the leader's) ----------------
        // A warp of their own: their buffer is free as soon as its group has read
        // it, and the group's next chunk is ready when it is done with this one,
        // whatever the last product waits for.
        if (rank == 0) {
            const uint32_t idesc = idesc_pair(MMA_BF16, false, false, 256, 128);
            const uint32_t x16 = smem_u32(sx) >> 4, w16 = smem_u32(sw) >> 4;
            int q = 0;
            RingPos w;
#pragma unroll 1
            for (int i = 0; i < my && !failed; ++i) {
                if (!warp_pair_wait(smem_u32(&bars.xfull[i & 1]), (uint32_t)(i >> 1) & 1u, limit)) failed = true;
                if (a.resident) w = RingPos();
#pragma unroll 1
                for (int c = 0; c < a.chunks && !failed; ++c, ++q, w.next(a.slots)) {
                    const int b = q & 1;
                    if (!warp_pair_wait(smem_u32(&bars.wfull[w.s]), a.resident ? 0u : w.ph, limit) ||
                        !warp_pair_wait(smem_u32(&bars.gempty[b]), ((uint32_t)(q >> 1) & 1u) ^ 1u, limit)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        for (int k = 0; k < a.xb; ++k)
                            mma_kblock<MMA_BF16, false, false>(tmem + 128 * b, x16 + (i & 1) * (x_bytes >> 4) + k * 1024,
                                                               w16 + w.s * (a.slot_bytes >> 4) + k * 512, idesc,
                                                               kblock_steps(a.C, k, 64), k == 0);
                        mma_commit_pair(smem_u32(&bars.gfull[b]));
                        if (c == a.chunks - 1) mma_commit_pair(smem_u32(&bars.xempty[i & 1]));
                    }
                }
            }
        }
    } else if (warp == 2) {
        // ---------------- the last product's MMAs (the leader's) ----------------
        if (rank == 0) {
            const uint32_t idesc = idesc_pair(MMA_BF16, false, false, 256, 0) | (uint32_t)(a.n2 >> 3) << 17;
            const uint32_t h16 = smem_u32(sh) >> 4, w16 = (smem_u32(sw) >> 4) + a.xb * 512;
            int q = 0;
            RingPos w;
#pragma unroll 1
            for (int i = 0; i < my && !failed; ++i) {
                const int y = i & 1;
                if (!warp_pair_wait(smem_u32(&bars.yempty[y]), ((uint32_t)(i >> 1) & 1u) ^ 1u, limit)) failed = true;
                if (a.resident) w = RingPos();
#pragma unroll 1
                for (int c = 0; c < a.chunks && !failed; ++c, ++q, w.next(a.slots)) {
                    const int b = q & 1;
                    if (!warp_pair_wait(smem_u32(&bars.wfull[w.s]), a.resident ? 0u : w.ph, limit) ||
                        !warp_pair_wait(smem_u32(&bars.hready[b]), (uint32_t)(q >> 1) & 1u, limit)) {
                        failed = true;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        mma_kblock<MMA_BF16, false, false>(TY + 128 * y, h16 + b * 1024, w16 + w.s * (a.slot_bytes >> 4),
                                                           idesc, 4, c == 0);
                        mma_commit_pair(smem_u32(&bars.hfree[b]));
                        // (g and u of this chunk were done before its h was)
                        if (!a.resident) mma_commit_pair(smem_u32(&bars.wempty[w.s]));
                        if (c == a.chunks - 1) mma_commit_pair(smem_u32(&bars.yfull[y]));
                    }
                }
            }
        }
    } else if (warp >= 4) {
        // ---------------- activations and output ----------------
        const int e = warp - 4, grp = e / FUSED_GROUP_WARPS, quad = warp & 3, half = (e % FUSED_GROUP_WARPS) >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        uint8_t *hbuf = sh + grp * 16384, *stage = stg + (a.shared_staging ? e % FUSED_GROUP_WARPS : e) * 4096;
        const uint32_t gempty = map_rank(smem_u32(&bars.gempty[grp]), 0), hready = map_rank(smem_u32(&bars.hready[grp]), 0);
        const int total = my * a.chunks;
        float *vec = vecs[e];

        // The staging (two boxes of 32 columns), where it is shared, goes from group
        // to group with the tiles they drain: tile i's warp takes it when tile i -
        // 1's stores have read it (over a tile ago, as a rule).
        const int boxes = half * 64 + 32 < a.C ? 2 : half * 64 < a.C;
        const uint32_t sfree = smem_u32(&bars.sfree[e % FUSED_GROUP_WARPS]);
        bool owed = false;   // this warp's last stores may still read the staging
        auto pass_on = [&]() {
            if (!owed || !a.shared_staging) return;
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(sfree);
            }
            owed = false;
        };
        auto take = [&](int i) {
            if (!a.shared_staging) staging_free(lane);
            else if (i > 0 && boxes && !warp_pair_wait(sfree, (uint32_t)(i - 1) & 1u, limit)) failed = true;
        };
        // the residual's boxes of this pair's i-th tile on their way into the
        // staging, four lanes a row (a row a lane, 32 lines an instruction, took
        // 16 us of 67 at 200,704 x 96)
        auto fetch_residual = [&](int i) {
            take(i);
            if (failed) return;
            const int row0 = (pair + i * a.np) * 256 + (int)rank * 128 + quad * 32;
#pragma unroll 1
            for (int j = 0; j < boxes; ++j) {
                const int col = half * 64 + 32 * j + 8 * (lane & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2);
                    const bool ok = row0 + r < a.rows && col < a.C;
                    cp_async16(smem_u32(stage) + j * 2048 + sw64_offset(r, lane & 3),
                               ok ? a.residual + (int64_t)(row0 + r) * a.C + col : a.residual, ok ? 16u : 0u);
                }
            }
            cp_async_commit();
        };
        // output rows of this pair's i-th tile: bias, residual, store
        auto drain = [&](int i) {
            const int y = i & 1;
            if (!a.residual) take(i);
            if (failed || !warp_pair_wait(smem_u32(&bars.yfull[y]), (uint32_t)(i >> 1) & 1u, limit)) {
                failed = true;
                return;
            }
            tc_fence_after();
            const int row0 = (pair + i * a.np) * 256 + (int)rank * 128 + quad * 32;
            if (a.residual) cp_async_wait<0>();
            __syncwarp();   // (the vector's last readers are done; the residual is there)
#pragma unroll 1
            for (int j = 0; j < boxes; ++j) {
                const int c0 = half * 64 + 32 * j;
                float v[32];
                tmem_ld32(TY + 128 * y + lanes + c0, v);
                vec[32 * j + lane] = lane_value(a.bd, c0 + lane, a.C);
                __syncwarp();
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float b[8];
                    if (a.bd) {
                        spread8(vec + 32 * j, q, b);
                        add8(v + 8 * q, b);
                    }
                    uint4 *at = reinterpret_cast<uint4 *>(stage + j * 2048 + sw64_offset(lane, q));
                    if (a.residual) {
                        load8(reinterpret_cast<const bf16 *>(at), 0, 8, b);
                        add8(v + 8 * q, b);
                    }
                    *at = pack8f(v + 8 * q);
                }
                store_box(&a.out, c0, row0, row0 < a.rows, stage + j * 2048, lane);
            }
            owed = boxes > 0;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(map_rank(smem_u32(&bars.yempty[y]), 0));
        };

        int pending = -1;   // tile whose output this group has yet to drain
        int i = grp / a.chunks, c = grp % a.chunks;
        float bg = 0.f, bu = 0.f;   // of this lane's hidden unit in this group's next chunk
        const bool biased = a.bg || a.bu;
        auto fetch_biases = [&](int chunk) {
            if (!biased) return;
            const int f = chunk * FUSED_CHUNK + half * 32 + lane;
            bg = lane_value(a.bg, f, a.F);
            bu = lane_value(a.bu, f, a.F);
        };
        fetch_biases(c);
#pragma unroll 1
        for (int q = grp; q < total && !failed; q += FUSED_GROUPS) {
            const uint32_t use = (uint32_t)(q >> 1) & 1u;
            pass_on();
            if (!warp_pair_wait(smem_u32(&bars.gfull[grp]), use, limit)) {
                failed = true;
                break;
            }
            tc_fence_after();
            float g[32], v[32];
            tmem_ld32(tmem + 128 * grp + lanes + half * 32, g);
            tmem_ld32(tmem + 128 * grp + lanes + 64 + half * 32, v);
            __syncwarp();
            vec[lane] = bg;
            vec[32 + lane] = bu;
            // (the next chunk's, a chunk ahead)
            int next = c + FUSED_GROUPS;
            while (next >= a.chunks) next -= a.chunks;
            fetch_biases(next);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(gempty);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float *gq = g + 8 * s, *vq = v + 8 * s;
                float b[8];
                if (a.bg) {
                    spread8(vec, s, b);
                    add8(gq, b);
                }
                if (a.bu) {
                    spread8(vec + 32, s, b);
                    add8(vq, b);
                }
                gate8<ACT>(gq, vq);
            }
            // the MMAs that read this buffer two chunks ago are done
            if (!warp_pair_wait(smem_u32(&bars.hfree[grp]), use ^ 1u, limit)) {
                failed = true;
                break;
            }
#pragma unroll
            for (int s = 0; s < 4; ++s)
                *reinterpret_cast<uint4 *>(hbuf + sw128_offset(quad * 32 + lane, half * 4 + s)) = pack8f(v + 8 * s);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(hready);

            if (pending >= 0) {
                drain(pending);
                pending = -1;
            }
            const int tile = i;
            c += FUSED_GROUPS;
            while (c >= a.chunks) {
                c -= a.chunks;
                ++i;
            }
            // (this group's last chunk of an own tile: drained after its next chunk)
            if (i > tile)
                for (int t = tile; t < i; ++t)
                    if ((t & 1) == grp) pending = t;
            if (pending >= 0 && a.residual) {
                pass_on();   // (the other group may need it to get to where it passes on the one awaited here)
                fetch_residual(pending);
            }
        }
        if (!failed && pending >= 0) {
            pass_on();
            drain(pending);
        }
        pass_on();
        const int mine = (total - grp + 1) / FUSED_GROUPS;   // chunks of this group
        if (!failed && mine > 0) failed = !warp_pair_wait(smem_u32(&bars.hfree[grp]), (uint32_t)(mine - 1) & 1u, limit);
        if (lane == 0) bulk_wait_all();
    }
    if (failed && lane == 0) atomicOr(a.st.err, ERR_TIMEOUT);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// N of the last product: C rounded up to a pair's step.
int last_n(int C) { return (C + 31) / 32 * 32; }
// Bytes of a CTA's part of a chunk's weights.
int slot_bytes(int C) { return (C + 63) / 64 * 8192 + last_n(C) * 64; }

} // namespace

// Tokens narrow enough for the accumulators to fit TMEM, and not so few tiles of
// such a long F that the pairs that have none would be missed.  Both forms' times,
// in hundredths of a us beyond what they share, from 60 sizes (129 to 200704 rows,
// F from 88 to 16384; the choice costs 0.5% against the better of each): a chunk
// 0.85 and a tile 0.6 a round; two kernels 8 more and 2.3 for a pair's tile of 256
// rows x 128 hidden units.  (129 x 128 x 4096: 52 us as one kernel, 15.9 as two;
// 20000 x 128 x 4096, two rounds of which the second has three tiles: 107, 90;
// 100000 x 128 x 4096: 357, 421; 200704 x 96 x 256: 49.9, 70.5.)
bool gated_fused_chosen(int C, int F, int rows)
{
    if (C > 128) return false;
    const FusedPlan p = plan_gated_fused(C, F, rows);
    const int64_t pairs = sm_count() / 2, rounds = (p.tiles + pairs - 1) / pairs;
    const int64_t units = (int64_t)p.tiles * ((F + 127) / 128);
    return rounds * (85 * p.chunks + 60) <= 800 + 230 * units / pairs;
}

FusedPlan plan_gated_fused(int C, int F, int rows)
{
    FusedPlan p{};
    p.tiles = (int)(((int64_t)rows + 255) / 256);
    p.np = p.tiles < sm_count() / 2 ? p.tiles : sm_count() / 2;
    p.chunks = (F + FUSED_CHUNK - 1) / FUSED_CHUNK;
    // A staging a group where it leaves room for every chunk's weights (400000 x 64
    // x 128 with biases and residual: 52 us, 62 shared), else one for both (200704
    // x 96 x 256: 49.9 us; 52.4 with halves of it, where the second box waits for
    // the first one's store).
    constexpr int STAGING = FUSED_GROUP_WARPS * 4096;
    const int most = 222 * 1024 - 1024;   // (5 KB for the barriers and biases, 1 KB of alignment)
    int fixed = 2 * ((C + 63) / 64) * 16384 + 2 * 16384 + FUSED_GROUPS * STAGING;
    p.shared_staging = p.chunks > FUSED_SLOTS || fixed + p.chunks * slot_bytes(C) > most;
    if (p.shared_staging) fixed -= STAGING;
    p.slots = (most - fixed) / slot_bytes(C);
    if (p.slots > FUSED_SLOTS) p.slots = FUSED_SLOTS;
    if (p.slots > p.chunks) p.slots = p.chunks;
    p.resident = p.slots == p.chunks;   // (three slots at least otherwise: g | u run two chunks ahead)
    p.smem = 1024 + (size_t)fixed + (size_t)p.slots * slot_bytes(C);
    return p;
}

cudaError_t launch_gated_fused(const bf16 *x, int rows, int C, int F, bool gelu, const bf16 *wg, const bf16 *bg,
                               const bf16 *wu, const bf16 *bu, const bf16 *wd, const bf16 *bd, const bf16 *residual,
                               bf16 *out, DeviceStatus st, cudaStream_t stream)
{
    FusedArgs a;
    memset(&a, 0, sizeof(a));
    const CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const FusedPlan pl = plan_gated_fused(C, F, rows);
    a.n2 = last_n(C);
    a.xb = (C + 63) / 64;
    a.chunks = pl.chunks;
    a.slot_bytes = slot_bytes(C);
    a.slots = pl.slots;
    a.resident = pl.resident;
    a.shared_staging = pl.shared_staging;
    a.tiles = pl.tiles;
    a.np = pl.np;
    cudaError_t e;
    if ((e = make_tensor_map(&a.x, type, x, C, rows, (int64_t)C * 2, 64, 128, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.wg, type, wg, C, F, (int64_t)C * 2, 64, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.wu, type, wu, C, F, (int64_t)C * 2, 64, 64, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.wd, type, wd, F, C, (int64_t)F * 2, 64, a.n2 / 2, 128)) != cudaSuccess) return e;
    if ((e = make_tensor_map(&a.out, type, out, C, rows, (int64_t)C * 2, 32, 32, 64)) != cudaSuccess) return e;
    a.bg = bg;
    a.bu = bu;
    a.bd = bd;
    a.residual = residual;
    a.rows = rows;
    a.C = C;
    a.F = F;
    a.st = st;
    auto *kern = gelu ? gated_fused_kernel<ACT_GELU> : gated_fused_kernel<ACT_SILU>;
    static std::atomic<uint64_t> ready[2];
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready[gelu].load() & bit)) {
        if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 222 * 1024)) != cudaSuccess) return e;
        ready[gelu].fetch_or(bit);
    }
    return launch_maybe_overlapped(kern, dim3(2u * (unsigned)a.np), dim3(FUSED_THREADS), pl.smem, stream, 1, a);
}

} // namespace swin
