// The linear operator's forward product on the CTA-pair skeleton: D = act(A B^T +
// bias) + residual, A and B K-major, in bf16 or e4m3 with scales of rows and
// columns, the value before the activation kept beside if asked for.
#pragma once

#include "products.cuh"

namespace swin {

// A unit is 256 rows x wn (256, 192 or 128) columns, a half of that in the last
// round, or a range of its K blocks (PairSplit).  Two groups of eight warps drain
// units in turn, each warp 32 rows x half of the columns in boxes of 32: at small
// K the epilogue binds, and one group's latencies pass under the other's work.
template <int ACT, bool Q8>
struct LinearPolicy {
    struct Args {
        CUtensorMap x, w, w_half, out, z, part;   // part: partial tiles [2 np][256][wn] fp32
        PairSplit split;
        const bf16 *bias, *residual;
        const float *sx, *sw;   // Q8
        int rows, cols, k;
        int mt, nt, wn, np;
        uint32_t per_band;      // 2^32 / (8 nt) rounded up, where that divides every tile's number exactly, else 0
        bool keep;              // z
        DeviceStatus st;
    };
    struct Unit {
        int m, col, width;   // row tile, first column, columns
        int kb0, kbn;        // K blocks
        int slot;            // partial tile to write (-1: the whole K, to D)
    };
    static constexpr int ELEMS = Q8 ? 128 : 64;   // K elements of a block (128 bytes)
    static constexpr bool CHAIN = false;
    static constexpr int STAGES = Q8 ? 4 : 5, STAGE_BYTES = 32768, EPI = 16, GROUPS = 2, SEGS = 1;
    static constexpr int BOX = 4096, VEC = Q8 ? 192 : 64;   // a warp's two boxes; its bias (bf16) and scales (fp32)
    static constexpr int STAGING = BOX + VEC;
    static constexpr int KIND = Q8 ? MMA_E4M3 : MMA_BF16;
    static constexpr uint32_t IDESC = idesc_pair(KIND, false, false, 256, 0);   // (N: width)

    static __device__ __forceinline__ int slot(int, int n) { return n & 1; }
    static __device__ __forceinline__ int slot_use(int, int n) { return n >> 1; }
    static __device__ __forceinline__ int slot_col(int s) { return s * 256; }
    static __device__ __forceinline__ int count(const Args &a, int pair) { return split_count(a.split, pair); }
    static __device__ __forceinline__ Unit decode(const Args &a, int pair, int n)
    {
        const SplitUnit s = split_unit(a.split, pair, n);
        Unit r;
        int nt;
        // (tile_order without its divisions, which took a tenth of the instructions at
        // K = 96: all bands but the last are of eight)
        const int band = (int)__umulhi((uint32_t)s.tile, a.per_band);
        if (a.per_band && band * 8 + 8 <= a.mt) {
            const int t = s.tile - band * 8 * a.nt;
            nt = t >> 3;
            r.m = band * 8 + (t & 7);
        } else {
            tile_order(s.tile, a.mt, a.nt, r.m, nt);
        }
        r.width = s.half >= 0 ? a.wn / 2 : a.wn;
        r.col = nt * a.wn + (s.half > 0 ? r.width : 0);
        r.kb0 = s.kb0;
        r.kbn = s.kbn;
        r.slot = s.slot;
        return r;
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &a, int pair, uint32_t)
    {
        const Unit u = decode(a, pair, 0);
        prefetch_map(&a.x);
        prefetch_map(u.width == a.wn ? &a.w : &a.w_half);
        prefetch_map(u.slot >= 0 ? &a.part : &a.out);
        if (a.keep) prefetch_map(&a.z);
    }
    static __device__ __forceinline__ void side(const Args &, int, int) {}
    static __device__ __forceinline__ int kblocks(const Args &, const Unit &u, int) { return u.kbn; }
    static __device__ __forceinline__ uint32_t tx(const Args &, const Unit &u, int) { return 2 * (16384 + u.width * 64); }
    static __device__ __forceinline__ void load(const Args &a, const Unit &u, int, int i, uint32_t rank, uint32_t dst,
                                                uint32_t bar)
    {
        const int k = (u.kb0 + i) * ELEMS;
        tma_load_2d_pair(dst, &a.x, k, u.m * 256 + (int)rank * 128, bar);
        tma_load_2d_pair(dst + 16384, u.width == a.wn ? &a.w : &a.w_half, k, u.col + (int)rank * (u.width / 2), bar);
    }
    static __device__ __forceinline__ void mma(const Args &a, const Unit &u, int, int i, uint32_t src16, uint32_t d)
    {
        mma_kblock<KIND, false, false>(d, src16, src16 + 1024, IDESC | (uint32_t)(u.width >> 3) << 17,
                                       kblock_steps(a.k, u.kb0 + i, ELEMS), i == 0);
    }

    // First row of a warp, first column of its box j, and its boxes inside the matrix.
    static __device__ __forceinline__ int row_of(const Unit &u, uint32_t rank, int quad)
    {
        return u.m * 256 + (int)rank * 128 + quad * 32;
    }
    static __device__ __forceinline__ int col_of(const Unit &u, int part, int j) { return u.col + part * (u.width / 2) + 32 * j; }
    static __device__ __forceinline__ int boxes(const Args &a, const Unit &u, int part)
    {
        const int left = (a.cols - col_of(u, part, 0) + 31) / 32, all = u.width / 64;
        return left < 0 ? 0 : left < all ? left : all;
    }
    // Box j of the residual into the warp's staging, asynchronously (one group of
    // copies a call, also where there is nothing to fetch).
    static __device__ __forceinline__ void fetch_residual(const Args &a, const Unit &u, int row0, int part, int j, bool any,
                                                          int lane, uint32_t box)
    {
        if (any) {
            const int col = col_of(u, part, j) + 8 * (lane & 3);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = 8 * k + (lane >> 2);
                const bool ok = row0 + r < a.rows && col < a.cols;
                cp_async16(box + sw64_offset(r, lane & 3), ok ? a.residual + (int64_t)(row0 + r) * a.cols + col : a.residual,
                           ok ? 16u : 0u);
            }
        }
        cp_async_commit();
    }
    // p += the eight bf16 values of u; and p's eight rounded.
    static __device__ __forceinline__ void add_words(f2 *p, const uint4 &u)
    {
        p[0] = add_bf16x2(u.x, p[0]);
        p[1] = add_bf16x2(u.y, p[1]);
        p[2] = add_bf16x2(u.z, p[2]);
        p[3] = add_bf16x2(u.w, p[3]);
    }
    static __device__ __forceinline__ uint4 pack_words(const f2 *p)
    {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) unpack2(p[e], v[2 * e], v[2 * e + 1]);
        return pack8f(v);
    }
    struct Pre {
        float bias, sw, sx;   // of this lane's column of the first box, and its row's scale
    };
    static __device__ __forceinline__ Pre prefetch(const Args &a, const Unit &u, uint32_t rank, int warp, int quad,
                                                   int part, int lane, uint8_t *staging)
    {
        Pre p{};
        staging_free(lane);   // (of the unit before)
        if (u.slot >= 0) return p;
        const int c = col_of(u, part, 0) + lane, row0 = row_of(u, rank, quad), n = boxes(a, u, part);
        p.bias = lane_value(a.bias, c, a.cols);
        if (Q8) {
            p.sw = c < a.cols ? a.sw[c] : 0.f;
            p.sx = row0 + lane < a.rows ? a.sx[row0 + lane] : 0.f;
        }
        if (a.residual && !a.keep) {
            const uint32_t box = smem_u32(staging + warp * BOX);
            fetch_residual(a, u, row0, part, 0, n > 0, lane, box);
            fetch_residual(a, u, row0, part, 1, n > 1, lane, box + 2048);
        }
        return p;
    }
    template <class Release>
    static __device__ __forceinline__ void epilogue(const Args &a, const Unit &u, const Pre &pre, int n, uint32_t rank,
                                                    int warp, int quad, int part, int lane, uint32_t t_lane,
                                                    uint8_t *staging, Release &&release)
    {
        uint8_t *stage = staging + warp * BOX;
        const uint32_t acc = t_lane + slot_col(slot(0, n)) + part * (u.width / 2);
        if (u.slot >= 0) {   // fp32 boxes of 16 columns, the two stagings in turn
            const int count = u.width / 32;
#pragma unroll 1
            for (int j = 0; j < count; ++j) {
                float v[16];
                tmem_ld16(acc + 16 * j, v);
                if (lane == 0) bulk_wait_read1();   // (the box written two before)
                __syncwarp();
                tmem_wait_ld();
                if (j == count - 1) release();
                uint8_t *box = stage + (j & 1) * 2048;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4 *>(box + sw64_offset(lane, q)) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                store_box(&a.part, part * (u.width / 2) + 16 * j, u.slot * 256 + (int)rank * 128 + quad * 32, true, box, lane);
            }
            return;
        }
        const int count = boxes(a, u, part), row0 = row_of(u, rank, quad);
        if (count == 0) {
            release();
            return;
        }
        bf16 *vec = reinterpret_cast<bf16 *>(staging + EPI * BOX + warp * VEC);
        float *scales = reinterpret_cast<float *>(vec + 32);
        const bool inside = row0 < a.rows, ahead = a.residual && !a.keep;
        float bias = pre.bias, sw = pre.sw;
#pragma unroll 1
        for (int j = 0; j < count; ++j) {
            float v[32];
            tmem_ld32(acc + 32 * j, v);
            if (ahead && j) {   // the next residual, in the place of the box stored last
                if (lane == 0) bulk_wait_read();
                __syncwarp();
                fetch_residual(a, u, row0, part, j + 1, j + 1 < count, lane, smem_u32(stage) + (j + 1) % 2 * 2048);
            }
            // with z: its box and out's, else the two in turn
            uint8_t *box = stage + (a.keep || (j & 1) ? 2048 : 0);
            if (!ahead && lane == 0) bulk_wait_read1();
            __syncwarp();   // (and the vectors of the box before have been read)
            if (a.bias) vec[lane] = __float2bfloat16_rn(bias);
            if (Q8) scales[lane] = sw;
            if (j + 1 < count) {
                const int c = col_of(u, part, j + 1) + lane;
                bias = lane_value(a.bias, c, a.cols);
                if (Q8) sw = c < a.cols ? a.sw[c] : 0.f;
            }
            uint4 res[4];
            const bool own = a.residual && a.keep;
            if (own) {
                const int col = col_of(u, part, j);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    res[q] = row0 + lane < a.rows && col + 8 * q < a.cols
                                 ? *reinterpret_cast<const uint4 *>(a.residual + (int64_t)(row0 + lane) * a.cols + col + 8 * q)
                                 : make_uint4(0, 0, 0, 0);
            }
            if (ahead) cp_async_wait<1>();
            __syncwarp();
            tmem_wait_ld();
            if (j == count - 1) release();
            const int col0 = col_of(u, part, j);
            f2 p[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = pack2(v[2 * e], v[2 * e + 1]);
            if (Q8) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float s[8];
                    spread8(scales, q, s);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[4 * q + e] = mul2(p[4 * q + e], mul2(pack2(pre.sx), pack2(s[2 * e], s[2 * e + 1])));
                }
            }
            if (a.bias) {
#pragma unroll
                for (int q = 0; q < 4; ++q) add_words(p + 4 * q, *reinterpret_cast<const uint4 *>(vec + 8 * q));
            }
            if (a.keep) {
#pragma unroll
                for (int q = 0; q < 4; ++q) *reinterpret_cast<uint4 *>(stage + sw64_offset(lane, q)) = pack_words(p + 4 * q);
                store_box(&a.z, col0, row0, inside, stage, lane);
                if (lane == 0) bulk_wait_read1();   // (out's box before)
                __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) p[e] = activate2<ACT>(p[e]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 *at = reinterpret_cast<uint4 *>(box + sw64_offset(lane, q));
                if (a.residual) add_words(p + 4 * q, own ? res[q] : *at);
                *at = pack_words(p + 4 * q);
            }
            store_box(&a.out, col0, row0, inside, box, lane);
        }
        if (ahead) cp_async_wait<0>();
    }
};

// ---- the weight gradient through an activation (linear_grad.cu) ----------------------

// dW = dz^T x, dz = dy act'(z) (written to dz unless null, rows of stride ld) and
// the slices' shares of db [slices, N] (null: not computed).
struct ActWgrad {
    const bf16 *z, *dy, *x;
    bf16 *dz, *dW;
    float *sums, *part;   // part: plan.part_bytes
    int rows, C, N, ld, act;
};
struct ActWgradPlan {
    bool chosen;          // rather than dz by a kernel of its own
    int n, tiles, slices; // columns of a tile, tiles of 256 rows of dW, slices of the tokens
    int mt, nt;           // the tiles' rows and columns
    int kb, slice_kb;
    size_t part_bytes;
};
ActWgradPlan plan_act_wgrad(int C, int N, int rows, const ProductsPlan &apart);
// Queues the kernel; the join of its partial tiles is left to launch_finish.
cudaError_t launch_act_wgrad(const ActWgrad &w, const ActWgradPlan &p, DeviceStatus st, cudaStream_t stream, JoinArgs *join,
                             int *join_blocks);

} // namespace swin
