// Kernels of the gated feed-forward block on the CTA-pair skeleton: the two
// first projections with the activation and the product, and the backward's
// recompute.
#pragma once

#include "products.cuh"

namespace swin {

// ---- h = act(x Wg^T + bg) * (x Wu^T + bu) --------------------------------------
//
// A unit is 256 rows x 128 hidden columns.  CTA 0 of the pair loads 128 rows of
// Wg as its half of B, CTA 1 the same rows of Wu: one 256 x 256 MMA then
// leaves g in accumulator columns 0..127 and u in 128..255 of the same rows, so
// that the thread that drains a row holds both and forms h without exchange.
// The tensor cores bind it (8192 x 2048 x 8192: 271 us alone, 2.03 PFLOP/s, busy in
// 96% of the cycles) until K is short (118162 x 192 x 672: 67 us, 57% of the issue
// slots with the activation).
template <int ACT, bool Q8>
struct UpPolicy {
    struct Args {
        CUtensorMap x, wg, wu, h;
        CUtensorMap wg_part, wu_part;   // boxes of a part of a tile's columns
        const bf16 *bg, *bu;
        const float *sx, *sg, *su;   // Q8
        int rows, C, F, mt, nt, kb, np;
        PairDeal deal;
        DeviceStatus st;
    };
    struct Unit {
        int m, col, width;   // row tile, first hidden column, columns
    };
    static constexpr int ELEMS = Q8 ? 128 : 64;   // K elements of a block (128 bytes)
    static constexpr bool CHAIN = false;
    static constexpr int STAGES = 5, STAGE_BYTES = 32768, EPI = 16, GROUPS = 2, STAGING = 2560, SEGS = 1;
    static constexpr uint32_t IDESC = idesc_pair(Q8 ? MMA_E4M3 : MMA_BF16, false, false, 256, 0);   // (N: 2 width)

    static __device__ __forceinline__ int slot(int, int n) { return n & 1; }
    static __device__ __forceinline__ int slot_use(int, int n) { return n >> 1; }
    static __device__ __forceinline__ int slot_col(int s) { return s * 256; }
    static __device__ __forceinline__ int count(const Args &a, int pair) { return a.deal.count(pair); }
    static __device__ __forceinline__ Unit decode(const Args &a, int pair, int n)
    {
        Unit r;
        int col, nt;
        const int t = a.deal.tile(pair, n, col, r.width);
        tile_order(t, a.mt, a.nt, r.m, nt);
        r.col = nt * 128 + col;
        return r;
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &a, int, uint32_t rank)
    {
        prefetch_map(&a.x);
        prefetch_map(rank ? &a.wu : &a.wg);
        prefetch_map(&a.h);
    }
    static __device__ __forceinline__ void side(const Args &, int, int) {}
    static __device__ __forceinline__ int kblocks(const Args &a, const Unit &, int) { return a.kb; }
    static __device__ __forceinline__ uint32_t tx(const Args &, const Unit &u, int) { return 2 * (16384 + 128 * u.width); }
    static __device__ __forceinline__ void load(const Args &a, const Unit &u, int, int kb, uint32_t rank, uint32_t dst,
                                                uint32_t bar)
    {
        tma_load_2d_pair(dst, &a.x, kb * ELEMS, u.m * 256 + (int)rank * 128, bar);
        tma_load_2d_pair(dst + 16384, weight_map(a, u, rank), kb * ELEMS, u.col, bar);
    }
    static __device__ __forceinline__ const CUtensorMap *weight_map(const Args &a, const Unit &u, uint32_t rank)
    {
        return u.width == 128 ? (rank ? &a.wu : &a.wg) : (rank ? &a.wu_part : &a.wg_part);
    }
    static __device__ __forceinline__ void mma(const Args &a, const Unit &u, int, int kb, uint32_t src16, uint32_t d)
    {
        mma_kblock<Q8 ? MMA_E4M3 : MMA_BF16, false, false>(d, src16, src16 + 1024, IDESC | (uint32_t)(u.width >> 2) << 17,
                                                           kblock_steps(a.C, kb, ELEMS), kb == 0);
    }
    struct Pre {
        float bg[2], bu[2], sg[2], su[2], sx;   // of this lane's column of each box of 32, and its row's scale
    };
    // a part's columns of the unit (64; in a narrower unit 32): its first, boxes of 32
    static __device__ __forceinline__ int part_col(const Unit &u, int part) { return part * (u.width == 128 ? 64 : 32); }
    static __device__ __forceinline__ int col_of(const Unit &u, int part, int j) { return u.col + part_col(u, part) + 32 * j; }
    static __device__ __forceinline__ Pre prefetch(const Args &a, const Unit &u, uint32_t rank, int, int quad, int part,
                                                   int lane, uint8_t *)
    {
        Pre p{};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int c = col_of(u, part, j) + lane;
            p.bg[j] = lane_value(a.bg, c, a.F);
            p.bu[j] = lane_value(a.bu, c, a.F);
            if (Q8) {
                p.sg[j] = c < a.F ? a.sg[c] : 0.f;
                p.su[j] = c < a.F ? a.su[c] : 0.f;
            }
        }
        const int row = u.m * 256 + (int)rank * 128 + quad * 32 + lane;
        if (Q8) p.sx = row < a.rows ? a.sx[row] : 0.f;
        return p;
    }
    template <class Release>
    static __device__ __forceinline__ void epilogue(const Args &a, const Unit &u, const Pre &pre, int n, uint32_t rank,
                                                    int warp, int quad, int part, int lane, uint32_t t_lane,
                                                    uint8_t *staging, Release &&release)
    {
        const int row0 = u.m * 256 + (int)rank * 128 + quad * 32;
        const uint32_t acc = t_lane + slot_col(slot(0, n)) + part_col(u, part);
        const int boxes = u.width == 128 ? 2 : part_col(u, part) < u.width;
        if (boxes == 0) {
            release();
            return;
        }
        // the warps' boxes (aligned for their swizzle), then the warps' vectors
        uint8_t *stage = staging + warp * 2048;
        float *vec = reinterpret_cast<float *>(staging + EPI * 2048 + warp * 512);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (j == boxes) break;
            float g[32], v[32];
            tmem_ld32(acc + 32 * j, g);
            tmem_ld32(acc + u.width + 32 * j, v);
            __syncwarp();
            vec[lane] = pre.bg[j];
            vec[32 + lane] = pre.bu[j];
            if (Q8) {
                vec[64 + lane] = pre.sg[j];
                vec[96 + lane] = pre.su[j];
            }
            staging_free(lane);   // (and the vectors are there)
            tmem_wait_ld();
            if (j == boxes - 1) release();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float *gq = g + 8 * q, *vq = v + 8 * q;
                float s[8];
                if (Q8) {
                    spread8(vec + 64, q, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) gq[e] *= pre.sx * s[e];
                    spread8(vec + 96, q, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) vq[e] *= pre.sx * s[e];
                }
                if (a.bg) {
                    spread8(vec, q, s);
                    add8(gq, s);
                }
                if (a.bu) {
                    spread8(vec + 32, q, s);
                    add8(vq, s);
                }
                gate8<ACT>(gq, vq);
                *reinterpret_cast<uint4 *>(stage + sw64_offset(lane, q)) = pack8f(vq);
            }
            const int col0 = col_of(u, part, j);
            store_box(&a.h, col0, row0, row0 < a.rows && col0 < a.F, stage, lane);
        }
    }
};

// Column sums of a warp's 32 rows x 16 columns (a row a lane): lane l returns
// column l % 16's.  Each exchange halves the columns a lane still sums.  (Of the
// rounded values, by MMAs with ones, they took a tenth of the instructions, but
// 1.4 to 1.7 times the error, and little less time where L2 binds: backward
// 12544 x 512 x 1368 125 against 126 us, 200704 x 96 x 256 204 against 212.)
__device__ __forceinline__ float column_sum16(float (&v)[16], int lane)
{
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
        for (int i = 0; i < o; ++i) {
            const bool up = lane & o;
            const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// ---- the backward's recompute: h, dg, du -----------------------------------------
//
// A unit is 256 rows x 128 hidden columns: dh = dy Wd (K = C; Wd [C, F] as an
// MN-major B) into 128 accumulator columns, then g | u as in the forward into
// 256.  384 of the 512 TMEM columns do not fit twice; dh alternates between
// two places of 128 columns, so that the next unit's dh (a third of its MMAs)
// runs under this unit's epilogue.  At 12544 x 512 x 1368 it takes 50 us, 37
// without its epilogue, 41 without the stores alone: its operands (518 MB) and
// outputs (103 MB) on their way from and to L2 bind it, not the arithmetic.
template <int ACT>
struct GradPolicy {
    struct Args {
        CUtensorMap x, wg, wu, dy, wd, h, dg, du;
        CUtensorMap wg_part, wu_part;   // boxes of a part of a tile's columns
        const bf16 *bg, *bu;
        float *dg_sums, *du_sums;   // [row blocks of 32][F]: sums of dg and du, or null
        int rows, C, F, mt, nt, kb, np;
        PairDeal deal;
        DeviceStatus st;
    };
    struct Unit {
        int m, col, width;   // row tile, first hidden column, columns
    };
    static constexpr bool CHAIN = false;
    static constexpr int STAGES = 5, STAGE_BYTES = 32768, EPI = 16, GROUPS = 1, STAGING = 4096 + 64, SEGS = 2;
    static constexpr uint32_t IDESC_H = idesc_pair(MMA_BF16, false, true, 256, 0);    // (N: width)
    static constexpr uint32_t IDESC_GU = idesc_pair(MMA_BF16, false, false, 256, 0);  // (N: 2 width)

    // segment 0 (dh): slots 1 and 2 in turn; segment 1 (g | u): slot 0
    static __device__ __forceinline__ int slot(int seg, int n) { return seg ? 0 : 1 + (n & 1); }
    static __device__ __forceinline__ int slot_use(int seg, int n) { return seg ? n : n >> 1; }
    static __device__ __forceinline__ int slot_col(int s) { return s == 0 ? 0 : 128 + 128 * s; }
    static __device__ __forceinline__ int count(const Args &a, int pair) { return a.deal.count(pair); }
    static __device__ __forceinline__ Unit decode(const Args &a, int pair, int n)
    {
        Unit r;
        int col, nt;
        const int t = a.deal.tile(pair, n, col, r.width);
        tile_order(t, a.mt, a.nt, r.m, nt);
        r.col = nt * 128 + col;
        return r;
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &a, int, uint32_t rank)
    {
        prefetch_map(&a.dy);
        prefetch_map(&a.wd);
        prefetch_map(&a.x);
        prefetch_map(rank ? &a.wu : &a.wg);
    }
    static __device__ __forceinline__ void side(const Args &, int, int) {}
    static __device__ __forceinline__ int kblocks(const Args &a, const Unit &, int) { return a.kb; }
    static __device__ __forceinline__ uint32_t tx(const Args &, const Unit &u, int seg)
    {
        return 2 * (16384 + (seg ? 128 * u.width : 8192));   // (Wd: 64 columns are loaded whatever the unit uses)
    }
    static __device__ __forceinline__ void load(const Args &a, const Unit &u, int seg, int kb, uint32_t rank,
                                                uint32_t dst, uint32_t bar)
    {
        const int row = u.m * 256 + (int)rank * 128;
        if (seg == 0) {
            tma_load_2d_pair(dst, &a.dy, kb * 64, row, bar);
            tma_load_2d_pair(dst + 16384, &a.wd, u.col + (int)rank * (u.width / 2), kb * 64, bar);
        } else {
            tma_load_2d_pair(dst, &a.x, kb * 64, row, bar);
            tma_load_2d_pair(dst + 16384, u.width == 128 ? (rank ? &a.wu : &a.wg) : (rank ? &a.wu_part : &a.wg_part), kb * 64,
                             u.col, bar);
        }
    }
    static __device__ __forceinline__ void mma(const Args &a, const Unit &u, int seg, int kb, uint32_t src16, uint32_t d)
    {
        const int steps = kblock_steps(a.C, kb, 64);
        const uint32_t w = (uint32_t)(u.width >> 3) << 17;
        if (seg == 0) mma_kblock<MMA_BF16, false, true>(d, src16, src16 + 1024, IDESC_H | w, steps, kb == 0);
        else mma_kblock<MMA_BF16, false, false>(d, src16, src16 + 1024, IDESC_GU | 2 * w, steps, kb == 0);
    }
    struct Pre {
        bf16 bg, bu;   // of this lane's column
    };
    static __device__ __forceinline__ Pre prefetch(const Args &a, const Unit &u, uint32_t, int, int, int part, int lane,
                                                   uint8_t *)
    {
        const int c = u.col + part * 32 + lane;
        Pre p;
        p.bg = a.bg && c < a.F ? a.bg[c] : __float2bfloat16_rn(0.f);
        p.bu = a.bu && c < a.F ? a.bu[c] : __float2bfloat16_rn(0.f);
        return p;
    }
    template <class Release>
    static __device__ __forceinline__ void epilogue(const Args &a, const Unit &u, const Pre &pre, int n, uint32_t rank,
                                                    int warp, int quad, int part, int lane, uint32_t t_lane,
                                                    uint8_t *staging, Release &&release)
    {
        if (part * 32 >= u.width) {   // (a narrow unit: the last of its pair)
            release();
            return;
        }
        const int row0 = u.m * 256 + (int)rank * 128 + quad * 32, col0 = u.col + part * 32;
        const uint32_t gu = t_lane + part * 32, dh = t_lane + slot_col(slot(0, n)) + part * 32;
        const bool inside = row0 < a.rows && col0 < a.F;
        uint4 du[4];
        // the boxes, then the biases (bf16: a KB is all that is left), shared by
        // the four warps of the same columns, which write the same values; by
        // units in turn, since a warp can be one unit ahead of another (not two:
        // the MMAs of the second wait for every warp's release of the first)
        uint8_t *stage = staging + warp * 4096;
        bf16 *vec = reinterpret_cast<bf16 *>(staging + EPI * 4096) + ((n & 1) * 4 + part) * 64;
        vec[lane] = pre.bg;
        vec[32 + lane] = pre.bu;
        staging_free(lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float g[16], v[16], d[16];
            tmem_ld16(gu + 16 * j, g);
            tmem_ld16(gu + u.width + 16 * j, v);
            tmem_ld16(dh + 16 * j, d);
            tmem_wait_ld();
            if (j == 1) release();
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float *gq = g + 8 * q, *vq = v + 8 * q, *dq = d + 8 * q;
                float s[8];
                if (a.bg) {
                    load8(vec, 8 * (2 * j + q), 32, s);
                    add8(gq, s);
                }
                if (a.bu) {
                    load8(vec + 32, 8 * (2 * j + q), 32, s);
                    add8(vq, s);
                }
                float hh[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const f2 u2 = pack2(vq[e], vq[e + 1]), dh2 = pack2(dq[e], dq[e + 1]);
                    f2 act2, grad2;
                    activate_grad2<ACT>(pack2(gq[e], gq[e + 1]), act2, grad2);
                    unpack2(mul2(act2, u2), hh[e], hh[e + 1]);
                    unpack2(mul2(mul2(dh2, u2), grad2), gq[e], gq[e + 1]);   // dg = dh u act'(g)
                    unpack2(mul2(dh2, act2), dq[e], dq[e + 1]);              // du = dh act(g)
                }
                const uint32_t off = sw64_offset(lane, 2 * j + q);
                *reinterpret_cast<uint4 *>(stage + off) = pack8f(hh);
                *reinterpret_cast<uint4 *>(stage + 2048 + off) = pack8f(gq);
                du[2 * j + q] = pack8f(dq);
            }
            if (a.dg_sums) {
                if (row0 + lane >= a.rows) {   // (no token: zero times an infinite parameter is not zero)
#pragma unroll
                    for (int e = 0; e < 16; ++e) g[e] = d[e] = 0.f;
                }
                const int c = col0 + 16 * j + (lane & 15);
                const float sg = column_sum16(g, lane), su = column_sum16(d, lane);
                if (lane < 16 && c < a.F) {
                    const int64_t at = (int64_t)(u.m * 8 + (int)rank * 4 + quad) * a.F + c;
                    a.dg_sums[at] = sg;
                    a.du_sums[at] = su;
                }
            }
        }
        // two boxes of staging for three outputs: du takes h's when it is read
        store_box(&a.h, col0, row0, inside, stage, lane);
        if (lane == 0 && inside) {
            tma_store_2d(&a.dg, col0, row0, smem_u32(stage + 2048));
            bulk_commit();
            bulk_wait_read1();
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(stage + sw64_offset(lane, q)) = du[q];
        store_box(&a.du, col0, row0, inside, stage, lane);
    }
};

// ---- few rows (gated_few.cu) -------------------------------------------------------

struct FewUp {
    const void *x, *wg, *wu;
    const bf16 *bg, *bu;
    const float *sx, *sg, *su;   // 8-bit form, else null
    bf16 *h;
    int rows, C, F, ldh;
    bool gelu;
};
// h = act(x Wg^T + bg) * (x Wu^T + bu) into rows of stride ldh.
cudaError_t launch_few_up(const FewUp &u, DeviceStatus st, cudaStream_t stream);
// out = residual + h Wd^T + bd; queued directly behind launch_few_up.
cudaError_t launch_few_down(const bf16 *h, int ldh, int rows, const bf16 *wd, const bf16 *bd, const bf16 *residual,
                            bf16 *out, int C, int F, DeviceStatus st, cudaStream_t stream);

// ---- narrow tokens (gated_fused.cu) ---------------------------------------------------

// The whole forward as one kernel, without a workspace.
bool gated_fused_chosen(int C, int F, int rows);   // rather than two kernels
struct FusedPlan {
    int tiles, np;           // of 256 rows, pairs that walk them
    int chunks, slots;       // of hidden units, weight chunks in the ring
    bool resident;           // every chunk has its slot: loaded once
    bool shared_staging;     // the two groups drain through one staging, in turn
    size_t smem;
};
FusedPlan plan_gated_fused(int C, int F, int rows);
cudaError_t launch_gated_fused(const bf16 *x, int rows, int C, int F, bool gelu, const bf16 *wg, const bf16 *bg,
                               const bf16 *wu, const bf16 *bu, const bf16 *wd, const bf16 *bd, const bf16 *residual,
                               bf16 *out, DeviceStatus st, cudaStream_t stream);

} // namespace swin
