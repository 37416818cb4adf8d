// Kernels of the gated feed-forward block on the CTA-pair skeleton: the two
// first projections with the activation and the product, the general GEMM of
// the other products, and the backward's recompute.
#pragma once

#include "gelu.cuh"
#include "pair.cuh"

namespace swin {

enum { ACT_SILU = 0, ACT_GELU = 1 };

// 1 / (1 + 2^z).
__device__ __forceinline__ f2 logistic2(f2 z)
{
    float a, b;
    unpack2(z, a, b);
    unpack2(add2(pack2(ex2_approx(a), ex2_approx(b)), pack2(1.f)), a, b);
    return pack2(rcp_approx(a), rcp_approx(b));
}

// What stands in front of g in act(g) = g P(g), for two values.
//
// GELU's P as 1 / (1 + 2^(x Q(x^2))): the logit of the normal distribution function
// is odd and smooth, and Q, of degree 6, was fitted to it here by reweighted
// least squares for the smallest largest error of x Phi(x) on [0, 9] (6.6e-8;
// 5.9e-7 evaluated in fp32, as good as gelu_exact's 4.7e-7).  Ten two-lane
// operations and no sign handling against fourteen and four more; its last
// coefficient is negative, so that far from zero Phi goes to 0 and 1.
template <int ACT>
__device__ __forceinline__ f2 gate2(f2 g)
{
    if (ACT == ACT_SILU) return logistic2(mul2(g, pack2(-1.4426950408889634f)));
    const f2 t = mul2(g, g);
    f2 z = fma2(t, pack2(-5.23388088e-9f), pack2(3.860164099e-7f));
    z = fma2(z, t, pack2(-1.1466739124e-5f));
    z = fma2(z, t, pack2(1.59485251061e-4f));
    z = fma2(z, t, pack2(9.5295035863e-5f));
    z = fma2(z, t, pack2(-0.10483819246f));
    z = fma2(z, t, pack2(-2.30220746994f));
    return logistic2(mul2(z, g));
}
template <int ACT>
__device__ __forceinline__ f2 activate2(f2 g)
{
    return mul2(g, gate2<ACT>(g));
}
// act of two values and its derivative d = P + g P'(g).
template <int ACT>
__device__ __forceinline__ void activate_grad2(f2 g, f2 &a, f2 &d)
{
    const f2 p = gate2<ACT>(g);
    a = mul2(g, p);
    if (ACT == ACT_SILU) {   // p + g p (1 - p) = p + p (g - a)
        d = fma2(p, fma2(a, pack2(-1.f), g), p);
        return;
    }
    // g P'(g): g times the density exp(-g^2 / 2) / sqrt(2 pi)
    float e0, e1;
    unpack2(mul2(mul2(g, g), pack2(-0.72134752044448170f)), e0, e1);
    d = fma2(mul2(g, pack2(0.3989422804014327f)), pack2(ex2_approx(e0), ex2_approx(e1)), p);
}

// Eight values of a bf16 vector at column c (zero past n, and for NULL).
__device__ __forceinline__ void load8(const bf16 *v, int c, int n, float (&f)[8])
{
    uint4 u = make_uint4(0, 0, 0, 0);
    if (v && c < n) u = *reinterpret_cast<const uint4 *>(v + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 p = unpack_bf16x2(w[e]);
        f[2 * e] = p.x;
        f[2 * e + 1] = p.y;
    }
}

// A vector over the columns of a warp's accumulators (a bias, a scale): each lane
// fetches its column's value, early; the warp spreads them through 32 floats of
// its shared memory, and every lane reads them back eight at a time.  (Eight
// values of the vector loaded from global memory by every lane at every use
// took 21 us of the narrow forward's 97.)
__device__ __forceinline__ float lane_value(const bf16 *v, int c, int n)
{
    return v && c < n ? __bfloat162float(v[c]) : 0.f;
}
__device__ __forceinline__ void spread8(const float *vec, int q, float (&f)[8])
{
    const float4 x = *reinterpret_cast<const float4 *>(vec + 8 * q), y = *reinterpret_cast<const float4 *>(vec + 8 * q + 4);
    f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
}
__device__ __forceinline__ void add8(float *d, const float (&s)[8])
{
#pragma unroll
    for (int e = 0; e < 8; e += 2) unpack2(add2(pack2(d[e], d[e + 1]), pack2(s[e], s[e + 1])), d[e], d[e + 1]);
}
// v = act(g) v, eight values.
template <int ACT>
__device__ __forceinline__ void gate8(const float *g, float *v)
{
#pragma unroll
    for (int e = 0; e < 8; e += 2)
        unpack2(mul2(activate2<ACT>(pack2(g[e], g[e + 1])), pack2(v[e], v[e + 1])), v[e], v[e + 1]);
}

__device__ __forceinline__ uint4 pack8f(const float *v)
{
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
}

// A warp's staged box to global memory: every lane has written its row; one
// lane stores it unless it lies outside.
__device__ __forceinline__ void store_box(const CUtensorMap *map, int x, int y, bool inside, uint8_t *stage, int lane)
{
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && inside) {
        tma_store_2d(map, x, y, smem_u32(stage));
        bulk_commit();
    }
}
// The staging may be written again.
__device__ __forceinline__ void staging_free(int lane)
{
    if (lane == 0) bulk_wait_read();
    __syncwarp();
}

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

// ---- general product --------------------------------------------------------------
//
// D = A B^T over up to two K segments (dx = dg Wg + du Wu), A and B each K-major
// or MN-major as stored: no operand is ever transposed in memory.  Up to three
// problems run as one launch (the three weight gradients).  The tensor cores bind
// it (8192 x 8192 x 2048 with the residual: 156 us, 1.76 PFLOP/s); with K of a few
// hundred its operands' way from L2 does (12544 x 2736 x 512: 30 us at 10 TB/s).
//
// Tiles are dealt to the pairs in rounds; a last round that would leave pairs
// idle is instead dealt out as half tiles, or cut along K: its tiles' K blocks, laid end to end, are split
// evenly over the pairs, and a pair's ranges that hold only a part of a tile go
// to fp32 partial tiles that a second kernel adds in the order of K.  (4096 x
// 2048 x 5632's dx: 128 tiles on 76 pairs, 2 rounds of 176 blocks; cut, 1.68: at
// the board's power limit no gain, the backward took 494 us cut and 481 whole;
// 12544 x 512 x 1368, below it: 131 cut, 147 whole.)
struct PairProblem {
    CUtensorMap a[2], b[2], d;
    CUtensorMap b_half[2];         // K-major B: boxes for a half tile
    const bf16 *bias, *residual;   // [cols] / [rows, cols] or null
    int rows, cols, k[2], kb[2];
    int mt, nt, first;             // first: this problem's first tile
};
// The division of `tiles` tiles of kb K blocks each over np pairs.
struct PairSplit {
    int tiles, np;
    int halves;      // the round after the whole ones is tiles' halves (of their columns): how many
    int k_blocks;    // of a tile
    int kb;          // the same, or (equal slices) a multiple of the slices a little above
    int full;        // rounds of whole tiles
    int cut;         // tiles cut along K (0: the last round is whole tiles too)
    uint32_t q, r;   // blocks a pair of the cut tiles: q, the first r pairs q + 1
    __device__ __forceinline__ uint32_t begin(int pair) const
    {
        return q * pair + ((uint32_t)pair < r ? (uint32_t)pair : r);
    }
    __device__ __forceinline__ int owner(uint32_t block) const
    {
        return block < r * (q + 1) ? (int)(block / (q + 1)) : (int)(r + (block - r * (q + 1)) / q);
    }
    // the partial tile of a pair's range in cut tile t
    __device__ __forceinline__ int slot(int pair, int t) const
    {
        return 2 * pair + ((int)(begin(pair) / (uint32_t)kb) != t);
    }
};

// Column sums of up to three matrices [rows, cols], bf16 or fp32 (the bias
// gradients): a warp adds every slices-th row of 256 or 128 columns (16 bytes a
// lane) into a partial row, eight rows in flight; the partial rows are added
// later, all in a fixed order.  The weight gradients' epilogue warps do it, which
// wait for their first tile's MMAs.
struct ColumnSums {
    struct {
        const bf16 *b;    // bf16, or
        const float *f;   // fp32
        bf16 *out;
        float *part;      // [slices, cols]
        int64_t rows;
        int cols, slices, tasks;   // tasks: slices of every group of columns
    } m[3];
    int n;
};
template <class T>
__device__ __forceinline__ void column_slice(const T *p, int64_t rows, int cols, int c, int slice, int slices, float *part)
{
    constexpr int V = 16 / sizeof(T);
    if (c >= cols) return;
    float v[V] = {};
    int64_t i = slice;
    auto add = [&](const uint4 &u) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (V == 4) {
                v[e] += __uint_as_float(w[e]);
            } else {
                v[2 * e % V] += __uint_as_float(w[e] << 16);
                v[(2 * e + 1) % V] += __uint_as_float(w[e] & 0xffff0000u);
            }
        }
    };
#pragma unroll 1
    for (; i + 7 * (int64_t)slices < rows; i += 8 * (int64_t)slices) {
        uint4 u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = *reinterpret_cast<const uint4 *>(p + (i + k * (int64_t)slices) * cols + c);
#pragma unroll
        for (int k = 0; k < 8; ++k) add(u[k]);
    }
#pragma unroll 1
    for (; i < rows; i += slices) add(*reinterpret_cast<const uint4 *>(p + i * cols + c));
#pragma unroll
    for (int e = 0; e < V; e += 4)
        *reinterpret_cast<float4 *>(part + (int64_t)slice * cols + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}
// Warp w's share, of `warps`.
__device__ __forceinline__ void column_partials(const ColumnSums &a, int w, int warps, int lane)
{
    int t = w;
    for (int z = 0; z < a.n; ++z) {
        const auto &m = a.m[z];
        for (; t < m.tasks; t += warps) {
            const int slice = t % m.slices, g = t / m.slices;
            if (m.b) column_slice(m.b, m.rows, m.cols, g * 256 + lane * 8, slice, m.slices, m.part);
            else column_slice(m.f, m.rows, m.cols, g * 128 + lane * 4, slice, m.slices, m.part);
        }
        t -= m.tasks;
    }
}

// Place in the order of tiles of the t-th tile worked on.  Products of the hidden
// activations' rows (not their weight gradients) go through the rows from the
// last: the kernel before wrote those last, and L2 still has them (118162 x 192 x
// 672 forward 104.3 us from the first, 101.8; 200704 x 96 x 256 backward 210.7, 207.6).
__host__ __device__ inline int tile_place(int t, int mt, int nt, bool from_last) { return from_last ? mt * nt - 1 - t : t; }

template <int TN, bool A_MN, bool B_MN>
struct GemmPolicy {
    struct Args {
        PairProblem p[3];
        CUtensorMap part;   // partial tiles [2 np][256][TN] fp32
        PairSplit split;
        ColumnSums sums;    // with A_MN: summed under the first tile's MMAs
        int wn;             // columns of a tile: TN, or 192 of 256
        int np;
        DeviceStatus st;
    };
    struct Unit {
        int p, m, col, kb0, kbn;
        int width;          // columns, from col: a tile's, or half of them
        int slot;           // partial tile to write (-1: the whole K, to D)
        int k0, kb_first;   // the first segment's K, and its blocks
    };
    static constexpr int STAGE_BYTES = 16384 + TN * 64, EPI = 16, GROUPS = 1, STAGING = 4096, SEGS = 1;
    static constexpr int STAGES = TN == 256 ? 5 : 6;
    static constexpr int BOXES = TN / 128;   // a warp's share of the columns: boxes of 32
    static constexpr uint32_t IDESC = idesc_pair(MMA_BF16, A_MN, B_MN, 256, 0);   // (N: width)

    static __device__ __forceinline__ int slot(int, int n) { return n & 1; }
    static __device__ __forceinline__ int slot_use(int, int n) { return n >> 1; }
    static __device__ __forceinline__ int slot_col(int s) { return s * 256; }
    static __device__ __forceinline__ int count(const Args &a, int pair)
    {
        const PairSplit &s = a.split;
        if (s.cut == 0) return s.full + (pair < s.halves) + (s.halves ? 0 : deal_count(s.tiles - s.full * s.np, s.np, pair));
        const uint32_t b0 = s.begin(pair), b1 = s.begin(pair + 1);
        return s.full + (b1 > b0 ? (int)((b1 - 1) / s.kb - b0 / s.kb) + 1 : 0);
    }
    static __device__ __forceinline__ Unit decode(const Args &a, int pair, int n)
    {
        const PairSplit &s = a.split;
        Unit r;
        int t = pair + n * s.np;
        r.kb0 = 0;
        r.kbn = s.k_blocks;
        r.slot = -1;
        if (s.cut && n >= s.full) {
            const uint32_t b0 = s.begin(pair), b1 = s.begin(pair + 1), kb = s.kb;
            const int c = (int)(b0 / kb) + n - s.full;   // cut tile
            const uint32_t lo = c * kb > b0 ? c * kb : b0, hi = (c + 1) * kb < b1 ? (c + 1) * kb : b1;
            r.kb0 = (int)(lo - c * kb);
            r.kbn = (int)((hi - c * kb < (uint32_t)s.k_blocks ? hi - c * kb : (uint32_t)s.k_blocks)) - r.kb0;
            if (hi - lo < kb) r.slot = 2 * pair + (n > s.full);
            t = s.full * s.np + c;
        }
        const bool half = s.halves && n >= s.full;
        if (half) t = s.full * s.np + pair / 2;
        r.p = t >= a.p[2].first ? 2 : t >= a.p[1].first ? 1 : 0;
        const PairProblem &p = a.p[r.p];
        int nt;
        tile_order(tile_place(t - p.first, p.mt, p.nt, !A_MN), p.mt, p.nt, r.m, nt);
        r.width = half ? TN / 2 : a.wn;
        r.col = nt * a.wn + (half ? pair % 2 * (TN / 2) : 0);
        r.k0 = p.k[0];
        r.kb_first = p.kb[0];
        return r;
    }
    static __device__ __forceinline__ void prefetch_maps(const Args &a, int pair, uint32_t)
    {
        const Unit u = decode(a, pair, 0);
        const int seg = u.kb0 >= u.kb_first;
        prefetch_map(&a.p[u.p].a[seg]);
        prefetch_map(&a.p[u.p].b[seg]);
        prefetch_map(u.slot >= 0 ? &a.part : &a.p[u.p].d);
    }
    static __device__ __forceinline__ void side(const Args &a, int w, int lane)
    {
        if (A_MN) column_partials(a.sums, w, 2 * a.np * EPI, lane);   // (the weight gradients)
    }
    static __device__ __forceinline__ int kblocks(const Args &, const Unit &u, int) { return u.kbn; }
    static __device__ __forceinline__ uint32_t tx(const Args &, const Unit &u, int)
    {
        return 2 * (16384 + (B_MN ? mn_boxes(u.width / 2) * 8192 : u.width * 64));
    }
    static __device__ __forceinline__ int mn_boxes(int rows) { return rows > 64 ? 2 : 1; }
    template <bool MN>
    static __device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap *map, int row, int rows, int k,
                                                        uint32_t bar)
    {
        if (MN) {
            tma_load_2d_pair(dst, map, row, k, bar);
            if (mn_boxes(rows) > 1) tma_load_2d_pair(dst + 8192, map, row + 64, k, bar);
        } else {
            tma_load_2d_pair(dst, map, k, row, bar);
        }
    }
    static __device__ __forceinline__ void load(const Args &a, const Unit &u, int, int i, uint32_t rank, uint32_t dst,
                                                uint32_t bar)
    {
        const PairProblem &p = a.p[u.p];
        int kb = u.kb0 + i;
        const int seg = kb >= u.kb_first;
        if (seg) kb -= u.kb_first;
        load_operand<A_MN>(dst, &p.a[seg], u.m * 256 + (int)rank * 128, 128, kb * 64, bar);
        load_operand<B_MN>(dst + 16384, B_MN || u.width == a.wn ? &p.b[seg] : &p.b_half[seg],
                           u.col + (int)rank * (u.width / 2), u.width / 2, kb * 64, bar);
    }
    static __device__ __forceinline__ void mma(const Args &a, const Unit &u, int, int i, uint32_t src16, uint32_t d)
    {
        // (two segments are of one K: dg and du)
        int kb = u.kb0 + i;
        if (kb >= u.kb_first) kb -= u.kb_first;
        mma_kblock<MMA_BF16, A_MN, B_MN>(d, src16, src16 + 1024, IDESC | (uint32_t)(u.width >> 3) << 17,
                                         kblock_steps(u.k0, kb, 64), i == 0);
    }
    // Of a warp's two 2 KB boxes of staging, box j takes its columns 32 j ...:
    // before the accumulators are ready, the residual.
    struct Pre {
        float bias[BOXES];   // of this lane's column of each box
    };
    // columns of a warp's part of the unit, and boxes of 32 of them
    static __device__ __forceinline__ int part_cols(const Unit &u) { return u.width > 128 ? 64 : 32; }
    static __device__ __forceinline__ int boxes(const Unit &u, int part)
    {
        return part * part_cols(u) < u.width ? part_cols(u) / 32 : 0;
    }
    static __device__ __forceinline__ int row_of(const Unit &u, uint32_t rank, int quad)
    {
        return u.m * 256 + (int)rank * 128 + quad * 32;
    }
    static __device__ __forceinline__ int col_of(const Unit &u, int part, int j) { return u.col + part * part_cols(u) + 32 * j; }
    static __device__ __forceinline__ Pre prefetch(const Args &a, const Unit &u, uint32_t rank, int warp, int quad,
                                                   int part, int lane, uint8_t *staging)
    {
        const PairProblem &p = a.p[u.p];
        Pre pre{};
        if (u.slot >= 0) return pre;
        if (p.residual) {
            const int row0 = row_of(u, rank, quad);
            staging_free(lane);
#pragma unroll
            for (int j = 0; j < BOXES; ++j) {
                if (j == boxes(u, part)) break;
                const int col = col_of(u, part, j) + 8 * (lane & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = 8 * k + (lane >> 2);
                    const bool ok = row0 + r < p.rows && col < p.cols;
                    cp_async16(smem_u32(staging + warp * STAGING + j * 2048) + sw64_offset(r, lane & 3),
                               ok ? p.residual + (int64_t)(row0 + r) * p.cols + col : p.residual, ok ? 16u : 0u);
                }
            }
            cp_async_commit();
        }
#pragma unroll
        for (int j = 0; j < BOXES; ++j) pre.bias[j] = lane_value(p.bias, col_of(u, part, j) + lane, p.cols);
        return pre;
    }
    template <class Release>
    static __device__ __forceinline__ void epilogue(const Args &a, const Unit &u, const Pre &pre, int n, uint32_t rank,
                                                    int warp, int quad, int part, int lane, uint32_t t_lane,
                                                    uint8_t *staging, Release &&release)
    {
        const PairProblem &p = a.p[u.p];
        uint8_t *stage = staging + warp * STAGING;
        const uint32_t acc = t_lane + slot_col(slot(0, n)) + part * part_cols(u);
        if (u.slot >= 0) {   // fp32 boxes of 16 columns, the two stagings in turn
#pragma unroll 1
            for (int j = 0; j < 2 * BOXES; ++j) {
                float v[16];
                tmem_ld16(acc + 16 * j, v);
                if (lane == 0) {   // (the box written two before; at first, whatever an earlier unit stored)
                    if (j) bulk_wait_read1();
                    else bulk_wait_read();
                }
                __syncwarp();
                tmem_wait_ld();
                if (j == 2 * BOXES - 1) release();
                uint8_t *box = stage + (j & 1) * 2048;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<float4 *>(box + sw64_offset(lane, q)) =
                        make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
                store_box(&a.part, part * (TN / 4) + 16 * j, u.slot * 256 + (int)rank * 128 + quad * 32, true, box, lane);
            }
            return;
        }
        if (boxes(u, part) == 0) {
            release();
            return;
        }
        const int row0 = row_of(u, rank, quad);
        if (p.residual) {
            cp_async_wait<0>();
            __syncwarp();
        } else {
            staging_free(lane);
        }
#pragma unroll
        for (int j = 0; j < BOXES; ++j) {
            if (j == boxes(u, part)) break;
            float v[32];
            tmem_ld32(acc + 32 * j, v);
            tmem_wait_ld();
            if (j == boxes(u, part) - 1) release();
            uint8_t *box = stage + j * 2048;
            if (p.bias) {
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xffffffffu, pre.bias[j], i);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 *at = reinterpret_cast<uint4 *>(box + sw64_offset(lane, q));
                if (p.residual) {
                    float b[8];
                    load8(reinterpret_cast<const bf16 *>(at), 0, 8, b);
                    add8(v + 8 * q, b);
                }
                *at = pack8f(v + 8 * q);
            }
            store_box(&p.d, col_of(u, part, j), row0, row0 < p.rows && col_of(u, part, j) < p.cols, box, lane);
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

constexpr int FEW_ROWS = 128;   // most rows of these kernels
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
