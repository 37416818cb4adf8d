// Matrix products on the CTA-pair skeleton (pair.cuh), shared by the gated block
// and the linear operator: what their epilogues are made of, the general product
// with its plans, and the kernel that finishes cut tiles and column sums.
#pragma once

#include "gelu.cuh"
#include "pair.cuh"

namespace swin {

enum { ACT_SILU = 0, ACT_GELU = 1, ACT_NONE = 2 };

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
    return ACT == ACT_NONE ? g : mul2(g, gate2<ACT>(g));
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

// ---- general product --------------------------------------------------------------
//
// D = A B^T over up to two K segments (dx = dg Wg + du Wu), A and B each K-major
// or MN-major as stored: no operand is ever transposed in memory.  Up to three
// problems run as one launch (the three weight gradients).  The tensor cores bind
// it (8192 x 8192 x 2048 with the residual: 173 to 178 us a call at the board's power
// limit, 1.55 to 1.59 PFLOP/s; one launch alone 158); with K of a few
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

// A pair's units of a split, and the n-th of them.
struct SplitUnit {
    int tile, half;      // half: 0 or 1, of its columns; -1: all
    int kb0, kbn;        // K blocks
    int slot;            // partial tile to write (-1: the whole K)
};
__device__ __forceinline__ int split_count(const PairSplit &s, int pair)
{
    if (s.cut == 0) return s.full + (pair < s.halves) + (s.halves ? 0 : deal_count(s.tiles - s.full * s.np, s.np, pair));
    const uint32_t b0 = s.begin(pair), b1 = s.begin(pair + 1);
    return s.full + (b1 > b0 ? (int)((b1 - 1) / s.kb - b0 / s.kb) + 1 : 0);
}
__device__ __forceinline__ SplitUnit split_unit(const PairSplit &s, int pair, int n)
{
    SplitUnit r{pair + n * s.np, -1, 0, s.k_blocks, -1};
    if (s.cut && n >= s.full) {
        const uint32_t b0 = s.begin(pair), b1 = s.begin(pair + 1), kb = s.kb;
        const int c = (int)(b0 / kb) + n - s.full;   // cut tile
        const uint32_t lo = c * kb > b0 ? c * kb : b0, hi = (c + 1) * kb < b1 ? (c + 1) * kb : b1;
        r.kb0 = (int)(lo - c * kb);
        r.kbn = (int)((hi - c * kb < (uint32_t)s.k_blocks ? hi - c * kb : (uint32_t)s.k_blocks)) - r.kb0;
        if (hi - lo < kb) r.slot = 2 * pair + (n > s.full);
        r.tile = s.full * s.np + c;
    } else if (s.halves && n >= s.full) {
        r.tile = s.full * s.np + pair / 2;
        r.half = pair % 2;
    }
    return r;
}

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
        float *part;      // [slices, cols], or (few rows) null: added to the end, to out
        int64_t rows;
        int cols, slices, tasks;   // tasks: slices of every group of columns
    } m[3];
    int n;
};
// Adds to v the values of 16 bytes.
template <class T, int V>
__device__ __forceinline__ void add16(float (&v)[V], const uint4 &u)
{
    static_assert(V == 16 / sizeof(T), "16 bytes");
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
}
// 16 bytes from L2 (the kernel may be an early one: CHAIN_EARLY).
__device__ __forceinline__ uint4 load_l2(const void *p) { return __ldcg(static_cast<const uint4 *>(p)); }
template <class T>
__device__ __forceinline__ void column_slice(const T *p, int64_t rows, int cols, int c, int slice, int slices, float *part)
{
    constexpr int V = 16 / sizeof(T);
    if (c >= cols) return;
    float v[V] = {};
    int64_t i = slice;
#pragma unroll 1
    for (; i + 7 * (int64_t)slices < rows; i += 8 * (int64_t)slices) {
        uint4 u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) u[k] = load_l2(p + (i + k * (int64_t)slices) * cols + c);
#pragma unroll
        for (int k = 0; k < 8; ++k) add16<T>(v, u[k]);
    }
#pragma unroll 1
    for (; i < rows; i += slices) add16<T>(v, load_l2(p + i * cols + c));
#pragma unroll
    for (int e = 0; e < V; e += 4)
        *reinterpret_cast<float4 *>(part + (int64_t)slice * cols + c + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
}
// Few rows to the end: four lanes across the columns, eight rows at a time.
template <class T>
__device__ __forceinline__ void column_few(const T *p, int rows, int cols, int c, int lane, bf16 *out)
{
    constexpr int V = 16 / sizeof(T);
    c += (lane & 3) * V;
    const bool in = c < cols;
    float v[V] = {};
#pragma unroll 1
    for (int i = lane >> 2; i < rows; i += 64) {
        uint4 u[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            u[k] = in && i + 8 * k < rows ? load_l2(p + (int64_t)(i + 8 * k) * cols + c) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) add16<T>(v, u[k]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    if (!in || lane >= 4) return;
#pragma unroll
    for (int e = 0; e < V; e += 4)
        *reinterpret_cast<uint2 *>(out + c + e) = make_uint2(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]));
}
// Warp w's share, of `warps`.
__device__ __forceinline__ void column_partials(const ColumnSums &a, int w, int warps, int lane)
{
    int t = w;
    for (int z = 0; z < a.n; ++z) {
        const auto &m = a.m[z];
        for (; t < m.tasks; t += warps) {
            if (!m.part) {
                if (m.b) column_few(m.b, (int)m.rows, m.cols, t * 32, lane, m.out);
                else column_few(m.f, (int)m.rows, m.cols, t * 16, lane, m.out);
                continue;
            }
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

// What the linear operator's tiles go through beside bias and residual.
struct LinearJoin {
    bool on;
    int act;                // ACT_*, after the bias
    const float *sx, *sw;   // 8 bits: scales of rows and columns, else null
    bf16 *z;                // where the value before the activation is kept, or null
};
// The cut tiles of a launch: out = the sum of a tile's partial tiles in the order
// of K (+ bias + residual).  `blocks` blocks a tile and VEC values a thread at a
// time: 16 and eight, or (few tiles, of many partial tiles each) 64 and four;
// 3 tiles of 25 partial tiles: 9 us, 15 by sixteen blocks.
struct JoinArgs {
    const float *part;
    PairSplit split;
    int tn, blocks;
    bool from_last;   // (tile_place)
    int slots;        // partial tiles a pair has: 2, or 1 (its range lies in one tile)
    bool single;      // a tile of one partial tile is joined too
    LinearJoin linear;
    struct {
        const bf16 *bias, *residual;
        bf16 *out;
        int rows, cols, mt, nt, first;
    } p[3];
};
template <int VEC>
__device__ __forceinline__ void add_vec(float (&v)[VEC], const float *p)
{
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(p + k);
        v[k] += w.x;
        v[k + 1] += w.y;
        v[k + 2] += w.z;
        v[k + 3] += w.w;
    }
}
template <int VEC>
__device__ __forceinline__ void add_vec(float (&v)[VEC], const bf16 *p)
{
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
        const uint2 u = *reinterpret_cast<const uint2 *>(p + k);
        const float2 x = unpack_bf16x2(u.x), y = unpack_bf16x2(u.y);
        v[k] += x.x;
        v[k + 1] += x.y;
        v[k + 2] += y.x;
        v[k + 3] += y.y;
    }
}
template <int VEC>
__device__ __forceinline__ void store_vec(bf16 *p, const float (&v)[VEC])
{
#pragma unroll
    for (int k = 0; k < VEC; k += 4)
        *reinterpret_cast<uint2 *>(p + k) = make_uint2(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]));
}
// Values e0, e0 + step, ... (VEC at a time) of cut tile c.
template <int VEC>
__device__ __forceinline__ void join_tile(const JoinArgs &a, int c, int e0, int step)
{
    const PairSplit &s = a.split;
    const int t = s.full * s.np + c;
    const int p0 = s.owner((uint32_t)c * s.kb), p1 = s.owner((uint32_t)(c + 1) * s.kb - 1);
    if (p0 == p1 && !a.single) return;   // (one pair had the whole tile and wrote it)
    const int i = t >= a.p[2].first ? 2 : t >= a.p[1].first ? 1 : 0;
    int m, n;
    tile_order(tile_place(t - a.p[i].first, a.p[i].mt, a.p[i].nt, a.from_last), a.p[i].mt, a.p[i].nt, m, n);
    const int rows = a.p[i].rows, cols = a.p[i].cols, per = a.tn / VEC;
    const int64_t size = 256 * a.tn;
    const int first = a.slots == 1 ? p0 : s.slot(p0, c);
    for (int e = e0; e < 256 * per; e += step) {
        const int row = m * 256 + e / per, col = n * a.tn + e % per * VEC;
        if (row >= rows || col >= cols) continue;
        const float *src = a.part + (int64_t)e * VEC;
        float v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        add_vec<VEC>(v, src + first * size);
#pragma unroll 8
        for (int p = p0 + 1; p <= p1; ++p)   // (these begin inside the tile: their first range)
            add_vec<VEC>(v, src + a.slots * p * size);
        const int64_t at = (int64_t)row * cols + col;
        if (a.linear.sx) {
            const float sx = a.linear.sx[row];
#pragma unroll
            for (int k = 0; k < VEC; ++k) v[k] *= sx * a.linear.sw[col + k];
        }
        if (a.p[i].bias) add_vec<VEC>(v, a.p[i].bias + col);
        if (a.linear.on) {
            if (a.linear.z) store_vec<VEC>(a.linear.z + at, v);
#pragma unroll
            for (int k = 0; k < VEC; k += 2) {
                const f2 g = pack2(v[k], v[k + 1]);
                unpack2(a.linear.act == ACT_SILU ? activate2<ACT_SILU>(g)
                                                 : a.linear.act == ACT_GELU ? activate2<ACT_GELU>(g) : g,
                        v[k], v[k + 1]);
            }
        }
        if (a.p[i].residual) add_vec<VEC>(v, a.p[i].residual + at);
        store_vec<VEC>(a.p[i].out + at, v);
    }
}

template <int TN, bool A_MN, bool B_MN>
struct GemmPolicy {
    struct Args {
        PairProblem p[3];
        CUtensorMap part;   // partial tiles [2 np][256][TN] fp32
        PairSplit split;
        ColumnSums sums;    // with A_MN: summed under the first tile's MMAs; else their last additions are
        JoinArgs side;      // another product's cut tiles, joined there too (joined: how many)
        int joined;
        int wn;             // columns of a tile: TN, or 192 of 256
        int np;
        int chain;          // CHAIN_*
        DeviceStatus st;
    };
    struct Unit {
        int p, m, col, kb0, kbn;
        int width;          // columns, from col: a tile's, or half of them
        int slot;           // partial tile to write (-1: the whole K, to D)
        int k0, kb_first;   // the first segment's K, and its blocks
    };
    static constexpr int STAGE_BYTES = 16384 + TN * 64, EPI = 16, GROUPS = 1, STAGING = 4096, SEGS = 1;
    static constexpr bool CHAIN = B_MN;   // (the backwards' products)
    static constexpr int STAGES = TN == 256 ? 5 : 6;
    static constexpr int BOXES = TN / 128;   // a warp's share of the columns: boxes of 32
    static constexpr uint32_t IDESC = idesc_pair(MMA_BF16, A_MN, B_MN, 256, 0);   // (N: width)

    static __device__ __forceinline__ int slot(int, int n) { return n & 1; }
    static __device__ __forceinline__ int slot_use(int, int n) { return n >> 1; }
    static __device__ __forceinline__ int slot_col(int s) { return s * 256; }
    static __device__ __forceinline__ int count(const Args &a, int pair) { return split_count(a.split, pair); }
    static __device__ __forceinline__ Unit decode(const Args &a, int pair, int n)
    {
        const SplitUnit s = split_unit(a.split, pair, n);
        Unit r;
        r.kb0 = s.kb0;
        r.kbn = s.kbn;
        r.slot = s.slot;
        r.p = s.tile >= a.p[2].first ? 2 : s.tile >= a.p[1].first ? 1 : 0;
        const PairProblem &p = a.p[r.p];
        int nt;
        tile_order(tile_place(s.tile - p.first, p.mt, p.nt, !A_MN), p.mt, p.nt, r.m, nt);
        r.width = s.half >= 0 ? TN / 2 : a.wn;
        r.col = nt * a.wn + (s.half > 0 ? TN / 2 : 0);
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
        if (A_MN) {
            column_partials(a.sums, w, 2 * a.np * EPI, lane);   // (the weight gradients)
            return;
        }
        if (!a.joined && !a.sums.n) return;
        // (neighbouring warps' shares go to different CTAs: there may be few)
        const int ctas = 2 * a.np, first = (w % EPI * ctas + w / EPI) * 32 + lane, threads = ctas * EPI * 32,
                  per = 64 * a.side.tn;   // fours of a tile
#pragma unroll 1
        for (int i = first; i < a.joined * per; i += threads) join_tile<4>(a.side, i / per, i % per, per);
        if (a.sums.n) {   // (a warp eight columns, four lanes a column)
            const auto &m = a.sums.m[0];
#pragma unroll 1
            for (int c = first / 32 * 8 + (lane & 7); c - (lane & 7) < m.cols; c += threads / 32 * 8) {
                float v = 0.f;
#pragma unroll 8
                for (int s = lane >> 3; s < m.slices; s += 4) v += m.part[(int64_t)s * m.cols + c];
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (lane < 8) m.out[c] = __float2bfloat16_rn(v);   // (cols is a multiple of 8)
            }
        }
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

// ---- host side ---------------------------------------------------------------------

constexpr CUtensorMapDataType T_BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, T_U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8,
                              T_F32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// K-major operand [rows, k] (row stride ld elements, 0: k): boxes of 128 bytes
// of K x box_rows.
inline cudaError_t map_k(CUtensorMap *m, const void *p, int64_t rows, int k, int box_rows, bool q8 = false, int ld = 0)
{
    const int e = q8 ? 1 : 2;
    return make_tensor_map(m, q8 ? T_U8 : T_BF16, p, k, rows, (int64_t)(ld ? ld : k) * e, 128 / e, box_rows, 128);
}
// MN-major operand, stored [k, mn] (row stride ld, 0: mn): boxes of 64 MN
// elements x 64 k.
inline cudaError_t map_mn(CUtensorMap *m, const void *p, int64_t k, int mn, int ld = 0)
{
    return make_tensor_map(m, T_BF16, p, mn, k, (int64_t)(ld ? ld : mn) * 2, 64, 64, 128);
}
// Output [rows, cols]: a warp's boxes of 32 columns x 32 rows.
inline cudaError_t map_out(CUtensorMap *m, const void *p, int64_t rows, int cols)
{
    return make_tensor_map(m, T_BF16, p, cols, rows, (int64_t)cols * 2, 32, 32, 64);
}
// Hidden activations in the workspace, [rows, F] with rows padded to 128 bytes:
// a box's rows are whole lines.  (F = 1368 unpadded: five sectors in two lines
// where four in one would do: its weight gradients took 47.7 us instead of 43.0.)
inline int hidden_ld(int F) { return (F + 63) / 64 * 64; }
// The kernels that write them: boxes of 32 columns x 32 rows.
inline cudaError_t map_hidden(CUtensorMap *m, const void *p, int64_t rows, int cols)
{
    return make_tensor_map(m, T_BF16, p, cols, rows, (int64_t)hidden_ld(cols) * 2, 32, 32, 64);
}

// One product of a launch_products call: D [rows, cols] = sum over K segments of
// A B^T (+ bias + residual).
struct Product {
    const void *a[2], *b[2];
    int k[2];
    int lda, ldb;   // row strides as stored (0: dense)
    bf16 *d;
    const bf16 *bias, *residual;
    int64_t rows;
    int cols;
};

// What is left of a call when its products are done, as one launch: the cut
// tiles of up to two of them, and the last additions of the column sums, eight
// columns a block and 32 threads a column.
struct FinishArgs {
    JoinArgs join[2];
    int joins[2];   // blocks of each
    ColumnSums cs;
};
// Partial rows of a column sum: 16 rows or more each, and not more than 98 (a
// warp takes them eight at a time, some 12 us for 98) up to 2048 partial rows.
inline int column_slices(int64_t rows)
{
    const int few = rows < 128 * 16 ? ceil_div(rows, 16) : 128, many = rows < 2048 * 98 ? ceil_div(rows, 98) : 2048;
    return few > many ? few : many;
}

struct ProductsPlan {
    int n;
    bool wide;            // 256-column tiles (else 128)
    int wn;               // columns of a tile: 256, 192 or 128
    PairSplit split;
    size_t part_bytes;    // of the partial tiles
    int64_t cost;         // estimated, hundredths of a whole tile's K block
};

// The plan of n products as one launch (elems: K elements of a block).
ProductsPlan plan_products(const Product *p, int n, int elems = 64);
// Queues the products (operands K- or MN-major: A, B both K; B MN; both MN); what
// is left to do for their cut tiles goes into fin->join[slot].  With A_MN their
// epilogue warps begin fin's column sums.  Without, they can do what `side` leaves
// to do of a kernel queued before, joins (of slot 1) and sums of few slices: under
// their first tile's MMAs, so that no launch is needed for it.  chain: CHAIN_EARLY
// behind a kernel whose results this one does not read and that lets the next kernel
// start only after its own wait (B MN, or the few-row kernel).
template <bool A_MN, bool B_MN>
cudaError_t launch_products(const Product *ps, const ProductsPlan &pl, float *part, DeviceStatus st,
                            cudaStream_t stream, int *launches, FinishArgs *fin, int slot, const FinishArgs *side = nullptr,
                            int chain = CHAIN_NONE);
cudaError_t launch_finish(const FinishArgs &a, cudaStream_t stream, int *launches);

// Workspace layout: bytes of each part, 1 KB aligned.
struct Carve {
    char *base;
    size_t used = 0;
    explicit Carve(void *p) : base((char *)p) {}
    void *take(size_t bytes)
    {
        void *p = base + used;
        used += (bytes + 1023) / 1024 * 1024;
        return p;
    }
};

// ---- few rows (gated_few.cu) -------------------------------------------------------

constexpr int FEW_ROWS = 128;   // most rows of the few-row kernels
// CTAs that share the K (kb blocks) of each of the linear operator's tiles.
int few_split(int64_t tiles, int kb);
// A device's count of clusters as it is kept, if `answer` is what the device says (tests).
int test_few_clusters_of(int dev, int split, bool alone, int answer);
// The linear operator for few rows, one launch.
struct FewLinear {
    const void *x, *w;
    const bf16 *bias, *residual;
    const float *sx, *sw;   // 8-bit form, else null
    bf16 *out, *z;          // z: or null
    int rows, C, N, act;    // act: ACT_*
};
cudaError_t launch_few_linear(const FewLinear &u, DeviceStatus st, cudaStream_t stream);
// dx = dz W for W [N, C], rows of dz of stride ld; any number of rows, as the above.
cudaError_t launch_few_dx(const bf16 *dz, int ld, int rows, const bf16 *w, bf16 *dx, int C, int N, DeviceStatus st,
                          cudaStream_t stream);
// The same for one row (linear_token.cu).
cudaError_t launch_token_linear(const FewLinear &u, cudaStream_t stream);

} // namespace swin
