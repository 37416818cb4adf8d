// The gated feed-forward block: C ABI, plans and launches of the kernels in
// gated.cuh, and the two small kernels that finish sums over rows.
//   forward   h = act(x Wg^T + bg) * (x Wu^T + bu)        (one kernel)
//             out = residual + h Wd^T + bd                 (one kernel)
//   backward  h, dg, du from x and dy (one kernel), dx = dg Wg + du Wu, then
//             dWg, dWu, dWd in one launch, and the bias gradients' column sums
#include <climits>
#include <cstring>
#include <new>

#include "swin_gated.h"
#include "swin_wattn_test.h"
#include "common.cuh"
#include "gated.cuh"

using namespace swin;

struct swin_block_gated_s {
    int C, F, act;
    int device;   // -1: created without one
    int *d_err;
    int last_launches;
    OrderedWorkspace ws;
};

namespace {

constexpr int MAX_WIDTH = 65536;
constexpr int MAX_ROWS = INT_MAX - 512;   // row coordinates of the last tile stay below 2^31
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr CUtensorMapDataType T_BF16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, T_U8 = CU_TENSOR_MAP_DATA_TYPE_UINT8,
                              T_F32 = CU_TENSOR_MAP_DATA_TYPE_FLOAT32;

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SWIN_WATTN_OK : SWIN_WATTN_ECUDA; }

bool bad_pointer(const void *p, bool required)
{
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) != 0 : required;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// K-major operand [rows, k] (row stride ld elements, 0: k): boxes of 128 bytes
// of K x box_rows.
cudaError_t map_k(CUtensorMap *m, const void *p, int64_t rows, int k, int box_rows, bool q8 = false, int ld = 0)
{
    const int e = q8 ? 1 : 2;
    return make_tensor_map(m, q8 ? T_U8 : T_BF16, p, k, rows, (int64_t)(ld ? ld : k) * e, 128 / e, box_rows, 128);
}
// MN-major operand, stored [k, mn] (row stride ld, 0: mn): boxes of 64 MN
// elements x 64 k.
cudaError_t map_mn(CUtensorMap *m, const void *p, int64_t k, int mn, int ld = 0)
{
    return make_tensor_map(m, T_BF16, p, mn, k, (int64_t)(ld ? ld : mn) * 2, 64, 64, 128);
}
// Output [rows, cols]: a warp's boxes of 32 columns x 32 rows.
cudaError_t map_out(CUtensorMap *m, const void *p, int64_t rows, int cols)
{
    return make_tensor_map(m, T_BF16, p, cols, rows, (int64_t)cols * 2, 32, 32, 64);
}
// Hidden activations in the workspace, [rows, F] with rows padded to 128 bytes:
// a box's rows are whole lines.  (F = 1368 unpadded: five sectors in two lines
// where four in one would do: its weight gradients took 47.7 us instead of 43.0.)
int hidden_ld(int F) { return (F + 63) / 64 * 64; }
// The kernels that write them: boxes of 32 columns x 32 rows.
cudaError_t map_hidden(CUtensorMap *m, const void *p, int64_t rows, int cols)
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

// The shapes of a call's products: the forward's last one, dx, and dWg, dWu, dWd.
Product down_product(int C, int F, int rows)
{
    Product p{};
    p.k[0] = F;
    p.lda = hidden_ld(F);
    p.rows = rows;
    p.cols = C;
    return p;
}
Product dx_product(int C, int F, int rows)
{
    Product p = down_product(C, F, rows);
    p.k[1] = F;
    return p;
}
void weight_products(int C, int F, int rows, Product (&p)[3])
{
    for (int i = 0; i < 3; ++i) {
        p[i] = Product{};
        p[i].k[0] = rows;
        p[i].rows = i < 2 ? F : C;
        p[i].cols = i < 2 ? C : F;
        (i < 2 ? p[i].lda : p[i].ldb) = hidden_ld(F);
    }
}

// What joining the tiles of a cut round costs, in K blocks of a whole tile: the
// launch, the partial tiles' traffic and their second epilogue, some 10 us.
// (Forward 1537 x 1536 x 4104, 42 tiles: 57.5 us with their 65 blocks cut to 36,
// 53.3 whole; 3000 x 1024 x 4096: 63.7 cut, 55.5 whole; 12544 x 512 x 1368
// backward: 147 whole, 131 with the cuts that this cost allows, 135 with every cut
// that saves a block.)
constexpr int WIDE_JOIN = 32, NARROW_JOIN = 36;
// A K block of a 256 x 192 tile in hundredths of a whole one's: tiles of that width
// where they come out cheaper, as a round that leaves a third of the pairs idle
// with 256 columns (1300 x 2048 x 5632 forward: 48 tiles 70.5 us, 66 of them 69.5;
// e4m3 1537 x 1536 x 4104 41.1 and 39.1; 3000 x 1024 x 2736 backward 105 and 103.8).
constexpr int COST_192 = 82;
// A K block of half a tile (256 x 128) in hundredths of a whole one's, with
// `halves` pairs at it: half of the MMAs and a little, or (many pairs) its share
// of what L2 delivers, three quarters of a whole tile's operands a pair.
int half_cost(int halves, int pairs) { return halves * 75 > 55 * pairs ? halves * 75 / pairs : 55; }

// The cut tiles of a launch: out = the sum of a tile's partial tiles in the order
// of K (+ bias + residual).  `blocks` blocks a tile and VEC values a thread at a
// time: 16 and eight, or (few tiles, of many partial tiles each) 64 and four;
// 3 tiles of 25 partial tiles: 9 us, 15 by sixteen blocks.
struct JoinArgs {
    const float *part;
    PairSplit split;
    int tn, blocks;
    bool from_last;   // (tile_place)
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
__device__ __forceinline__ void join_tiles(const JoinArgs &a, int block)
{
    const PairSplit &s = a.split;
    const int c = block / a.blocks, t = s.full * s.np + c;
    const int p0 = s.owner((uint32_t)c * s.kb), p1 = s.owner((uint32_t)(c + 1) * s.kb - 1);
    if (p0 == p1) return;   // (one pair had the whole tile and wrote it)
    const int i = t >= a.p[2].first ? 2 : t >= a.p[1].first ? 1 : 0;
    int m, n;
    tile_order(tile_place(t - a.p[i].first, a.p[i].mt, a.p[i].nt, a.from_last), a.p[i].mt, a.p[i].nt, m, n);
    const int rows = a.p[i].rows, cols = a.p[i].cols, per = a.tn / VEC;
    const int64_t size = 256 * a.tn;
    const int first = s.slot(p0, c);
    for (int e = block % a.blocks * 256 + threadIdx.x; e < 256 * per; e += a.blocks * 256) {
        const int row = m * 256 + e / per, col = n * a.tn + e % per * VEC;
        if (row >= rows || col >= cols) continue;
        const float *src = a.part + (int64_t)e * VEC;
        float v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = 0.f;
        add_vec<VEC>(v, src + first * size);
#pragma unroll 4
        for (int p = p0 + 1; p <= p1; ++p)   // (these begin inside the tile: their first range)
            add_vec<VEC>(v, src + 2 * p * size);
        const int64_t at = (int64_t)row * cols + col;
        if (a.p[i].bias) add_vec<VEC>(v, a.p[i].bias + col);
        if (a.p[i].residual) add_vec<VEC>(v, a.p[i].residual + at);
#pragma unroll
        for (int k = 0; k < VEC; k += 4)
            *reinterpret_cast<uint2 *>(a.p[i].out + at + k) =
                make_uint2(pack_bf16x2(v[k], v[k + 1]), pack_bf16x2(v[k + 2], v[k + 3]));
    }
}

// What is left of a call when its products are done, as one launch: the cut
// tiles of up to two of them, and the last additions of the column sums, eight
// columns a block and 32 threads a column.
struct FinishArgs {
    JoinArgs join[2];
    int joins[2];   // blocks of each
    ColumnSums cs;
};
__host__ __device__ inline int column_blocks(const ColumnSums &cs, int i) { return (cs.m[i].cols + 7) / 8; }
// Partial rows of a column sum: 16 rows or more each, and not more than 98 (a
// warp takes them eight at a time, some 12 us for 98) up to 2048 partial rows.
int column_slices(int64_t rows)
{
    const int few = rows < 128 * 16 ? ceil_div(rows, 16) : 128, many = rows < 2048 * 98 ? ceil_div(rows, 98) : 2048;
    return few > many ? few : many;
}
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs a)
{
    __shared__ float sum[32][8];
    griddep_launch_dependents();
    griddep_wait();
    int b = blockIdx.x;
    for (int i = 0; i < 2; ++i) {
        if (b < a.joins[i]) {
            if (a.join[i].blocks == 16) join_tiles<8>(a.join[i], b);
            else join_tiles<4>(a.join[i], b);
            return;
        }
        b -= a.joins[i];
    }
    int z = 0;
    for (; z + 1 < a.cs.n && b >= column_blocks(a.cs, z); ++z) b -= column_blocks(a.cs, z);
    const auto &m = a.cs.m[z];
    const int k = threadIdx.x & 7, w = threadIdx.x >> 3, c = b * 8 + k;   // (cols is a multiple of 8)
    float v = 0.f;
#pragma unroll 8
    for (int s = w; s < m.slices; s += 32) v += m.part[(int64_t)s * m.cols + c];
    sum[w][k] = v;
    __syncthreads();
    if (threadIdx.x >= 8) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) v += sum[i][k];
    m.out[c] = __float2bfloat16_rn(v);
}
cudaError_t launch_finish(const FinishArgs &a, cudaStream_t stream, int *launches)
{
    int blocks = a.joins[0] + a.joins[1];
    for (int i = 0; i < a.cs.n; ++i) blocks += column_blocks(a.cs, i);
    if (!blocks) return cudaSuccess;
    ++*launches;
    return launch_maybe_overlapped(finish_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, 1, a);
}
struct ProductsPlan {
    int n;
    bool wide;            // 256-column tiles (else 128)
    int wn;               // columns of a tile: 256, 192 or 128
    PairSplit split;
    size_t part_bytes;    // of the partial tiles
};

// Tiles of 256 x 256 where every product has more than 128 columns, else 256 x
// 128.  The last round is cut along K where that saves more K blocks than the
// join costs; few blocks in all go to as many pairs as leave each at least four.
// A last round of at most half of the pairs goes out as half tiles where that
// costs less than either: no join (1024 x 2048 x 5632 forward 61 us cut or whole,
// 57 in halves; 12544 x 512 x 1368 backward, dx's last 22 tiles, 131 cut, 129; its
// weight gradients' 36 tiles of 196 blocks stay cut: in halves 9 us more).
ProductsPlan plan_products(const Product *p, int n)
{
    ProductsPlan pl{};
    pl.n = n;
    pl.wide = true;
    for (int i = 0; i < n; ++i)
        if (p[i].cols <= 128) pl.wide = false;
    const int tn = pl.wn = pl.wide ? 256 : 128;
    auto count = [&](int wn) {
        int64_t tiles = 0;
        for (int i = 0; i < n; ++i) tiles += (int64_t)ceil_div(p[i].rows, 256) * ceil_div(p[i].cols, wn);
        return tiles;
    };
    int64_t tiles = count(tn);
    PairSplit &s = pl.split;
    s.tiles = (int)tiles;
    s.k_blocks = s.kb = ceil_div(p[0].k[0], 64) + (p[0].k[1] ? ceil_div(p[0].k[1], 64) : 0);
    const int pairs = sm_count() / 2;
    s.np = (int)(tiles < pairs ? tiles : pairs);
    const int full = (int)(tiles / pairs), rest = (int)(tiles - (int64_t)full * pairs);
    const int64_t blocks = (int64_t)rest * s.kb;
    int64_t np = full || blocks / 4 >= pairs ? pairs : blocks / 4 > rest ? blocks / 4 : rest;
    const int cut_cost = ceil_div(blocks, np) + (pl.wide ? WIDE_JOIN : NARROW_JOIN), least = s.kb < cut_cost ? s.kb : cut_cost;
    const bool halves = pl.wide && rest && 2 * rest <= pairs && (int64_t)half_cost(2 * rest, pairs) * s.kb <= 100ll * least;
    const int64_t here = 100ll * full * s.kb + (halves ? (int64_t)half_cost(2 * rest, pairs) * s.kb : rest ? 100ll * least : 0);
    const int64_t tiles192 = count(192);
    if (pl.wide && (int64_t)ceil_div(tiles192, pairs) * COST_192 * s.kb < here) {
        pl.wn = 192;
        s.tiles = (int)tiles192;
        s.np = (int)(tiles192 < pairs ? tiles192 : pairs);
    } else if (halves) {
        s.full = full;
        s.halves = 2 * rest;
        s.np = full ? pairs : s.halves;
    } else if (rest && s.kb > cut_cost) {
        // Equal slices of every tile, where they cost at most a tenth more blocks:
        // pairs that share rows of an operand then walk K side by side, and each
        // reads what another has brought into L2.  (36 tiles, the weight gradients
        // of 44821 x 336 x 1288: the backward takes 330 us, 400 by even ranges.  A
        // slice is longer than what rounding K up to equal slices adds, so that none
        // is empty.)
        const int slices = pairs / rest;
        if (!full && slices > 1 && s.kb >= 16 * slices && s.kb >= slices * slices &&
            (int64_t)ceil_div(s.kb, slices) * 10 <= (int64_t)ceil_div(blocks, np) * 11) {
            np = rest * slices;
            s.kb = ceil_div(s.kb, slices) * slices;
        }
        const int64_t all = (int64_t)rest * s.kb;
        s.np = (int)np;
        s.full = full;
        s.cut = rest;
        s.q = (uint32_t)(all / np);
        s.r = (uint32_t)(all % np);
        pl.part_bytes = (size_t)np * 2 * 256 * tn * sizeof(float);
    }
    return pl;
}

template <int TN, bool A_MN, bool B_MN>
cudaError_t launch_products_t(const Product *ps, const ProductsPlan &pl, float *part, DeviceStatus st,
                              cudaStream_t stream, int *launches, FinishArgs *fin, int slot)
{
    typename GemmPolicy<TN, A_MN, B_MN>::Args a;
    memset(&a, 0, sizeof(a));
    JoinArgs &r = fin->join[slot];
    cudaError_t e;
    int first = 0;
    for (int i = 0; i < 3; ++i) {
        PairProblem &q = a.p[i];
        q.first = r.p[i].first = INT_MAX;
        if (i >= pl.n) continue;
        const Product &p = ps[i];
        q.rows = (int)p.rows;
        q.cols = p.cols;
        q.mt = ceil_div(p.rows, 256);
        q.nt = ceil_div(p.cols, pl.wn);
        q.first = first;
        first += q.mt * q.nt;
        q.bias = p.bias;
        q.residual = p.residual;
        r.p[i] = {p.bias, p.residual, p.d, q.rows, q.cols, q.mt, q.nt, q.first};
        for (int s = 0; s < 2; ++s) {
            q.k[s] = p.k[s];
            q.kb[s] = p.k[s] ? ceil_div(p.k[s], 64) : 0;
            if (!p.k[s]) continue;
            e = A_MN ? map_mn(&q.a[s], p.a[s], p.k[s], (int)p.rows, p.lda)
                     : map_k(&q.a[s], p.a[s], p.rows, p.k[s], 128, false, p.lda);
            if (e != cudaSuccess) return e;
            e = B_MN ? map_mn(&q.b[s], p.b[s], p.k[s], p.cols, p.ldb)
                     : map_k(&q.b[s], p.b[s], p.cols, p.k[s], pl.wn / 2, false, p.ldb);
            if (e != cudaSuccess) return e;
            if (!B_MN && pl.split.halves) {
                e = map_k(&q.b_half[s], p.b[s], p.cols, p.k[s], TN / 4, false, p.ldb);
                if (e != cudaSuccess) return e;
            }
        }
        if ((e = map_out(&q.d, p.d, p.rows, p.cols)) != cudaSuccess) return e;
    }
    a.split = r.split = pl.split;
    if (A_MN) a.sums = fin->cs;
    a.wn = pl.wn;
    a.np = pl.split.np;
    a.st = st;
    if (pl.split.cut) {
        e = make_tensor_map(&a.part, T_F32, part, TN, (int64_t)a.np * 2 * 256, TN * 4, 16, 32, 64);
        if (e != cudaSuccess) return e;
    }
    ++*launches;
    r.part = part;
    r.tn = TN;
    r.from_last = !A_MN;
    r.blocks = pl.split.cut >= 16 ? 16 : 64;
    fin->joins[slot] = pl.split.cut * r.blocks;
    return launch_pair<GemmPolicy<TN, A_MN, B_MN>>(a, stream);
}

// Queues the products; what is left to do for their cut tiles goes into
// fin->join[slot].
template <bool A_MN, bool B_MN>
cudaError_t launch_products(const Product *ps, const ProductsPlan &pl, float *part, DeviceStatus st,
                            cudaStream_t stream, int *launches, FinishArgs *fin, int slot)
{
    return pl.wide ? launch_products_t<256, A_MN, B_MN>(ps, pl, part, st, stream, launches, fin, slot)
                   : launch_products_t<128, A_MN, B_MN>(ps, pl, part, st, stream, launches, fin, slot);
}

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

// UpPolicy whose loads never come: a test of the bounded waits.
struct StallPolicy : UpPolicy<ACT_SILU, false> {
    static __device__ __forceinline__ void load(const Args &, const Unit &, int, int, uint32_t, uint32_t, uint32_t) {}
};

// (stall: with StallPolicy)
template <bool Q8>
cudaError_t launch_up(const swin_block_gated_s *h, const void *x, const float *sx, int rows, const void *wg,
                      const float *sg, const void *bg, const void *wu, const float *su, const void *bu, bf16 *hidden,
                      DeviceStatus st, cudaStream_t stream, bool stall = false)
{
    if (rows <= FEW_ROWS) {
        FewUp u{};
        u.x = x;
        u.wg = wg;
        u.wu = wu;
        u.bg = (const bf16 *)bg;
        u.bu = (const bf16 *)bu;
        u.sx = sx;
        u.sg = sg;
        u.su = su;
        u.h = hidden;
        u.rows = rows;
        u.C = h->C;
        u.F = h->F;
        u.ldh = hidden_ld(h->F);
        u.gelu = h->act == SWIN_BLOCK_GATED_GELU;
        return launch_few_up(u, st, stream);
    }
    auto run = [&](auto policy) -> cudaError_t {
        using P = decltype(policy);
        typename P::Args a;
        memset(&a, 0, sizeof(a));
        cudaError_t e;
        if ((e = map_k(&a.x, x, rows, h->C, 128, Q8)) != cudaSuccess) return e;
        if ((e = map_k(&a.wg, wg, h->F, h->C, 128, Q8)) != cudaSuccess) return e;
        if ((e = map_k(&a.wu, wu, h->F, h->C, 128, Q8)) != cudaSuccess) return e;
        if ((e = map_hidden(&a.h, hidden, rows, h->F)) != cudaSuccess) return e;
        a.bg = (const bf16 *)bg;
        a.bu = (const bf16 *)bu;
        a.sx = sx;
        a.sg = sg;
        a.su = su;
        a.rows = rows;
        a.C = h->C;
        a.F = h->F;
        a.mt = ceil_div(rows, 256);
        a.nt = ceil_div(h->F, 128);
        a.kb = ceil_div(h->C, P::ELEMS);
        a.deal = deal_tiles(a.mt * a.nt, sm_count() / 2);
        a.np = a.deal.np;
        if (a.deal.parts > 1) {
            if ((e = map_k(&a.wg_part, wg, h->F, h->C, 128 / a.deal.parts, Q8)) != cudaSuccess) return e;
            if ((e = map_k(&a.wu_part, wu, h->F, h->C, 128 / a.deal.parts, Q8)) != cudaSuccess) return e;
        }
        a.st = st;
        return launch_pair<P>(a, stream);
    };
    if (stall) return run(StallPolicy{});
    return h->act == SWIN_BLOCK_GATED_SILU ? run(UpPolicy<ACT_SILU, Q8>{}) : run(UpPolicy<ACT_GELU, Q8>{});
}

// The handle's device is the current one.
int check_device(const swin_block_gated_s *h)
{
    int dev = h->device;
    if (dev < 0) return SWIN_WATTN_ECUDA;
    return bind_device(&dev);
}

struct Span {
    const void *p;
    int64_t bytes;
};
bool any_overlap(Span o, std::initializer_list<Span> in)
{
    for (const Span &s : in)
        if (s.p && overlaps(o.p, o.bytes, s.p, s.bytes)) return true;
    return false;
}

// The forward's checks, the hidden activation by `up` (into the workspace) and
// the last product.
template <class Up>
int forward(swin_block_gated_s *h, int rows, const void *Wd, const void *bd, const void *residual, void *out,
            cudaStream_t stream, Up &&up)
{
    int rc = check_device(h);
    if (rc != SWIN_WATTN_OK) return rc;
    Product down = down_product(h->C, h->F, rows);
    down.b[0] = Wd;
    down.d = (bf16 *)out;
    down.bias = (const bf16 *)bd;
    down.residual = (const bf16 *)residual;
    const bool few = rows <= FEW_ROWS;
    const ProductsPlan pl = few ? ProductsPlan{} : plan_products(&down, 1);
    Carve size(nullptr);
    size.take((size_t)rows * hidden_ld(h->F) * 2);
    size.take(pl.part_bytes);
    void *ws = nullptr;
    bool captured = false;
    if ((rc = ows_begin(&h->ws, size.used, stream, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    Carve carve(ws);
    bf16 *hidden = (bf16 *)carve.take((size_t)rows * hidden_ld(h->F) * 2);
    float *part = (float *)carve.take(pl.part_bytes);
    down.a[0] = hidden;
    const DeviceStatus st{h->d_err, WAIT_NS};
    h->last_launches = 1;
    cudaError_t e = up(hidden, st);
    if (e == cudaSuccess && few) {
        ++h->last_launches;
        e = launch_few_down(hidden, hidden_ld(h->F), rows, (const bf16 *)Wd, (const bf16 *)bd, (const bf16 *)residual,
                            (bf16 *)out, h->C, h->F, st, stream);
    } else if (e == cudaSuccess) {
        FinishArgs fin{};
        e = launch_products<false, false>(&down, pl, part, st, stream, &h->last_launches, &fin, 0);
        if (e == cudaSuccess) e = launch_finish(fin, stream, &h->last_launches);
    }
    const int rc2 = ows_end(&h->ws, stream, ws, captured);
    return e != cudaSuccess ? SWIN_WATTN_ECUDA : rc2;
}

} // namespace

extern "C" {

int swin_block_gated_create(swin_block_gated_t *out, int C, int F, int act)
{
    if (!out) return SWIN_WATTN_EINVAL;
    *out = nullptr;
    if (C <= 0 || C % 8 || C > MAX_WIDTH || F <= 0 || F % 8 || F > MAX_WIDTH) return SWIN_WATTN_EINVAL;
    if (act != SWIN_BLOCK_GATED_SILU && act != SWIN_BLOCK_GATED_GELU) return SWIN_WATTN_EINVAL;
    swin_block_gated_s *h = new (std::nothrow) swin_block_gated_s{};
    if (!h) return SWIN_WATTN_ENOMEM;
    h->C = C;
    h->F = F;
    h->act = act;
    h->device = -1;
    if (bind_device(&h->device) != SWIN_WATTN_OK) h->device = -1;
    if (h->device >= 0 &&
        (cudaMalloc(&h->d_err, sizeof(int)) != cudaSuccess || cudaMemset(h->d_err, 0, sizeof(int)) != cudaSuccess)) {
        cudaGetLastError();
        if (h->d_err) cudaFree(h->d_err);
        delete h;
        return SWIN_WATTN_ENOMEM;
    }
    *out = h;
    return SWIN_WATTN_OK;
}

int swin_block_gated_destroy(swin_block_gated_t h)
{
    if (!h) return SWIN_WATTN_OK;
    if (h->d_err) {
        cudaDeviceSynchronize();
        cudaFree(h->d_err);
    }
    ows_free(&h->ws);
    delete h;
    return SWIN_WATTN_OK;
}

int swin_block_gated_last_launches(swin_block_gated_t h) { return h ? h->last_launches : 0; }

int swin_block_gated_sync_status(swin_block_gated_t h, swin_stream_t stream)
{
    if (!h) return SWIN_WATTN_EINVAL;
    if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return SWIN_WATTN_ECUDA;
    if (!h->d_err) return SWIN_WATTN_OK;
    int err = 0;
    if (cudaMemcpy(&err, h->d_err, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SWIN_WATTN_ECUDA;
    if (!err) return SWIN_WATTN_OK;
    if (cudaMemset(h->d_err, 0, sizeof(int)) != cudaSuccess) return SWIN_WATTN_ECUDA;
    return SWIN_WATTN_ETIMEOUT;
}

int swin_block_gated_forward(swin_block_gated_t h, const void *x, int rows, const swin_block_gated_params *p,
                             const void *residual, void *out, swin_stream_t stream)
{
    if (!h || !p || rows < 0 || rows > MAX_ROWS) return SWIN_WATTN_EINVAL;
    if (rows == 0) return SWIN_WATTN_OK;   // (an empty tensor may have no address)
    for (const void *q : {x, p->Wg, p->Wu, p->Wd, (const void *)out})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {p->bg, p->bu, p->bd, residual})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const int64_t n = 2 * (int64_t)rows * h->C, w = 2 * (int64_t)h->C * h->F, f = 2 * (int64_t)h->F, c = 2 * (int64_t)h->C;
    if (any_overlap({out, n}, {{x, n}, {p->Wg, w}, {p->Wu, w}, {p->Wd, w}, {p->bg, f}, {p->bu, f}, {p->bd, c},
                               {residual == out ? nullptr : residual, n}}))
        return SWIN_WATTN_EINVAL;
    if (rows > FEW_ROWS && gated_fused_chosen(h->C, h->F, rows)) {
        const int rc = check_device(h);
        if (rc != SWIN_WATTN_OK) return rc;
        h->last_launches = 1;
        return cuda_status(launch_gated_fused((const bf16 *)x, rows, h->C, h->F, h->act == SWIN_BLOCK_GATED_GELU,
                                              (const bf16 *)p->Wg, (const bf16 *)p->bg, (const bf16 *)p->Wu,
                                              (const bf16 *)p->bu, (const bf16 *)p->Wd, (const bf16 *)p->bd,
                                              (const bf16 *)residual, (bf16 *)out, DeviceStatus{h->d_err, WAIT_NS},
                                              (cudaStream_t)stream));
    }
    return forward(h, rows, p->Wd, p->bd, residual, out, (cudaStream_t)stream, [&](bf16 *hidden, DeviceStatus st) {
        return launch_up<false>(h, x, nullptr, rows, p->Wg, nullptr, p->bg, p->Wu, nullptr, p->bu, hidden, st,
                                (cudaStream_t)stream);
    });
}

int swin_block_gated_forward_q8(swin_block_gated_t h, const void *x8, const float *sx, int rows,
                                const swin_block_gated_params_q8 *p, const void *residual, void *out,
                                swin_stream_t stream)
{
    if (!h || !p || rows < 0 || rows > MAX_ROWS) return SWIN_WATTN_EINVAL;
    if (h->C % 16) return SWIN_WATTN_EUNSUPPORTED;
    if (rows == 0) return SWIN_WATTN_OK;
    for (const void *q : {x8, (const void *)sx, p->Wg8, (const void *)p->sg, p->Wu8, (const void *)p->su, p->Wd,
                          (const void *)out})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {p->bg, p->bu, p->bd, residual})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const int64_t m = (int64_t)rows * h->C, w = (int64_t)h->C * h->F, f = 2 * (int64_t)h->F, c = 2 * (int64_t)h->C;
    if (any_overlap({out, 2 * m}, {{x8, m}, {sx, 4 * (int64_t)rows}, {p->Wg8, w}, {p->Wu8, w}, {p->sg, 2 * f},
                                   {p->su, 2 * f}, {p->Wd, 2 * w}, {p->bg, f}, {p->bu, f}, {p->bd, c},
                                   {residual == out ? nullptr : residual, 2 * m}}))
        return SWIN_WATTN_EINVAL;
    return forward(h, rows, p->Wd, p->bd, residual, out, (cudaStream_t)stream, [&](bf16 *hidden, DeviceStatus st) {
        return launch_up<true>(h, x8, sx, rows, p->Wg8, p->sg, p->bg, p->Wu8, p->su, p->bu, hidden, st,
                               (cudaStream_t)stream);
    });
}

int swin_block_gated_backward(swin_block_gated_t h, const void *x, int rows, const swin_block_gated_params *p,
                              const void *dy, void *dx, const swin_block_gated_grads *g, swin_stream_t stream)
{
    if (!h || !p || !g || rows < 0 || rows > MAX_ROWS) return SWIN_WATTN_EINVAL;
    const int64_t n = 2 * (int64_t)rows * h->C, w = 2 * (int64_t)h->C * h->F, f = 2 * (int64_t)h->F, c = 2 * (int64_t)h->C;
    for (const void *q : {x, dy, (const void *)dx})
        if (bad_pointer(q, rows > 0)) return SWIN_WATTN_EINVAL;
    for (const void *q : {p->Wg, p->Wu, p->Wd, (const void *)g->dWg, (const void *)g->dWu, (const void *)g->dWd})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {p->bg, p->bu, p->bd, (const void *)g->dbg, (const void *)g->dbu, (const void *)g->dbd})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const Span outs[] = {{dx, n}, {g->dWg, w}, {g->dWu, w}, {g->dWd, w}, {g->dbg, f}, {g->dbu, f}, {g->dbd, c}};
    for (int i = 0; i < 7; ++i) {
        if (!outs[i].p) continue;
        if (any_overlap(outs[i], {{x, n}, {dy, n}, {p->Wg, w}, {p->Wu, w}, {p->Wd, w}, {p->bg, f}, {p->bu, f}, {p->bd, c}}))
            return SWIN_WATTN_EINVAL;
        for (int j = 0; j < i; ++j)
            if (any_overlap(outs[i], {outs[j]})) return SWIN_WATTN_EINVAL;
    }
    int rc = check_device(h);
    if (rc != SWIN_WATTN_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        for (int i = 1; i < 7; ++i)
            if (outs[i].p && cudaMemsetAsync(const_cast<void *>(outs[i].p), 0, outs[i].bytes, s) != cudaSuccess)
                return SWIN_WATTN_ECUDA;
        return SWIN_WATTN_OK;
    }

    Product dxp = dx_product(h->C, h->F, rows), dw[3];
    weight_products(h->C, h->F, rows, dw);
    dxp.b[0] = p->Wg;
    dxp.b[1] = p->Wu;
    dxp.d = (bf16 *)dx;
    dw[0].b[0] = dw[1].b[0] = x;
    dw[2].a[0] = dy;
    dw[0].d = (bf16 *)g->dWg;
    dw[1].d = (bf16 *)g->dWu;
    dw[2].d = (bf16 *)g->dWd;
    const ProductsPlan px = plan_products(&dxp, 1), pw = plan_products(dw, 3);
    // bias gradients: dg's and du's sums over each warp's 32 rows come from the
    // recompute kernel
    FinishArgs fin{};
    ColumnSums &cs = fin.cs;
    const int row_blocks = ceil_div(rows, 256) * 8;
    const size_t row_sums = g->dbg || g->dbu ? (size_t)row_blocks * h->F * sizeof(float) : 0;
    void *const bias_grads[3] = {g->dbg, g->dbu, g->dbd};
    size_t sum_bytes = 0;
    for (int i = 0; i < 3; ++i) {
        if (!bias_grads[i]) continue;
        auto &m = cs.m[cs.n++];
        m.out = (bf16 *)bias_grads[i];
        m.b = i < 2 ? nullptr : (const bf16 *)dy;
        m.rows = i < 2 ? row_blocks : rows;
        m.cols = i < 2 ? h->F : h->C;
        m.slices = column_slices(m.rows);
        m.tasks = ceil_div(m.cols, m.b ? 256 : 128) * m.slices;
        sum_bytes += (size_t)m.slices * m.cols * sizeof(float);
    }
    const size_t hid = (size_t)rows * hidden_ld(h->F) * 2;
    Carve size(nullptr);
    for (int i = 0; i < 3; ++i) size.take(hid);
    size.take(px.part_bytes);
    size.take(pw.part_bytes);
    for (int i = 0; i < 2; ++i) size.take(row_sums);
    size.take(sum_bytes);
    void *ws = nullptr;
    bool captured = false;
    if ((rc = ows_begin(&h->ws, size.used, s, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    Carve carve(ws);
    bf16 *hidden = (bf16 *)carve.take(hid), *dg = (bf16 *)carve.take(hid), *du = (bf16 *)carve.take(hid);
    float *x_part = (float *)carve.take(px.part_bytes), *w_part = (float *)carve.take(pw.part_bytes);
    float *dg_sums = (float *)carve.take(row_sums), *du_sums = (float *)carve.take(row_sums);
    float *sum_part = (float *)carve.take(sum_bytes);
    dxp.a[0] = dw[0].a[0] = dg;
    dxp.a[1] = dw[1].a[0] = du;
    dw[2].b[0] = hidden;
    for (int i = 0; i < cs.n; ++i) {
        auto &m = cs.m[i];
        if (!m.b) m.f = m.out == g->dbg ? dg_sums : du_sums;
        m.part = sum_part;
        sum_part += (size_t)m.slices * m.cols;
    }
    const DeviceStatus st{h->d_err, WAIT_NS};

    auto grad = [&](auto policy) -> cudaError_t {
        using P = decltype(policy);
        typename P::Args a;
        memset(&a, 0, sizeof(a));
        cudaError_t e;
        if ((e = map_k(&a.x, x, rows, h->C, 128)) != cudaSuccess) return e;
        if ((e = map_k(&a.dy, dy, rows, h->C, 128)) != cudaSuccess) return e;
        if ((e = map_k(&a.wg, p->Wg, h->F, h->C, 128)) != cudaSuccess) return e;
        if ((e = map_k(&a.wu, p->Wu, h->F, h->C, 128)) != cudaSuccess) return e;
        if ((e = map_mn(&a.wd, p->Wd, h->C, h->F)) != cudaSuccess) return e;
        bf16 *o[3] = {hidden, dg, du};
        CUtensorMap *m[3] = {&a.h, &a.dg, &a.du};
        for (int i = 0; i < 3; ++i)
            if ((e = map_hidden(m[i], o[i], rows, h->F)) != cudaSuccess) return e;
        a.bg = (const bf16 *)p->bg;
        a.bu = (const bf16 *)p->bu;
        if (row_sums) {
            a.dg_sums = dg_sums;
            a.du_sums = du_sums;
        }
        a.rows = rows;
        a.C = h->C;
        a.F = h->F;
        a.mt = ceil_div(rows, 256);
        a.nt = ceil_div(h->F, 128);
        a.kb = ceil_div(h->C, 64);
        a.deal = deal_tiles(a.mt * a.nt, sm_count() / 2);
        a.np = a.deal.np;
        if (a.deal.parts > 1) {
            if ((e = map_k(&a.wg_part, p->Wg, h->F, h->C, 128 / a.deal.parts)) != cudaSuccess) return e;
            if ((e = map_k(&a.wu_part, p->Wu, h->F, h->C, 128 / a.deal.parts)) != cudaSuccess) return e;
        }
        a.st = st;
        return launch_pair<P>(a, s);
    };
    h->last_launches = 1;
    cudaError_t e = h->act == SWIN_BLOCK_GATED_SILU ? grad(GradPolicy<ACT_SILU>{}) : grad(GradPolicy<ACT_GELU>{});
    if (e == cudaSuccess) e = launch_products<false, true>(&dxp, px, x_part, st, s, &h->last_launches, &fin, 0);
    if (e == cudaSuccess) e = launch_products<true, true>(dw, pw, w_part, st, s, &h->last_launches, &fin, 1);
    if (e == cudaSuccess) e = launch_finish(fin, s, &h->last_launches);
    const int rc2 = ows_end(&h->ws, s, ws, captured);
    return e != cudaSuccess ? SWIN_WATTN_ECUDA : rc2;
}

// ---- test hooks (swin_wattn_test.h) ------------------------------------------------

int swin_block_gated_test_stall(swin_block_gated_t h, const void *x, int rows, const swin_block_gated_params *p,
                                int64_t wait_limit_us, swin_stream_t stream)
{
    if (!h || !p || rows <= FEW_ROWS || rows > MAX_ROWS || wait_limit_us < 1 || wait_limit_us > 1000000)
        return SWIN_WATTN_EINVAL;
    for (const void *q : {x, p->Wg, p->Wu})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    int rc = check_device(h);
    if (rc != SWIN_WATTN_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    void *ws = nullptr;
    bool captured = false;
    if ((rc = ows_begin(&h->ws, (size_t)rows * hidden_ld(h->F) * 2, s, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    const cudaError_t e = launch_up<false>(h, x, nullptr, rows, p->Wg, nullptr, nullptr, p->Wu, nullptr, nullptr, (bf16 *)ws,
                                           DeviceStatus{h->d_err, (uint64_t)wait_limit_us * 1000}, s, true);
    const int rc2 = ows_end(&h->ws, s, ws, captured);
    return e != cudaSuccess ? SWIN_WATTN_ECUDA : rc2;
}

int swin_block_gated_test_last_use(int stages, int issued, int k, int *stage, int *parity)
{
    if (stages < 1 || issued < 0 || k < 0 || k >= stages || k >= issued || !stage || !parity) return SWIN_WATTN_EINVAL;
    const RingUse u = last_use(stages, issued, k);
    *stage = u.stage;
    *parity = (int)u.parity;
    return SWIN_WATTN_OK;
}

int swin_block_gated_test_plan(int C, int F, int rows, int which, int *plan)
{
    if (C <= 0 || C % 8 || C > MAX_WIDTH || F <= 0 || F % 8 || F > MAX_WIDTH || rows <= FEW_ROWS || rows > MAX_ROWS || !plan)
        return SWIN_WATTN_EINVAL;
    if (which == SWIN_BLOCK_GATED_PLAN_NARROW) {
        if (!gated_fused_chosen(C, F, rows)) return SWIN_WATTN_EINVAL;
        const FusedPlan f = plan_gated_fused(C, F, rows);
        const int v[] = {f.tiles, f.np, f.chunks, f.slots, f.resident, f.shared_staging};
        memcpy(plan, v, sizeof(v));
        return SWIN_WATTN_OK;
    }
    Product p[3];
    int n = 1;
    if (which == SWIN_BLOCK_GATED_PLAN_DOWN) p[0] = down_product(C, F, rows);
    else if (which == SWIN_BLOCK_GATED_PLAN_DX) p[0] = dx_product(C, F, rows);
    else if (which == SWIN_BLOCK_GATED_PLAN_WEIGHTS) weight_products(C, F, rows, p), n = 3;
    else return SWIN_WATTN_EINVAL;
    const ProductsPlan pl = plan_products(p, n);
    const int v[] = {pl.split.tiles, pl.split.np, pl.wn, pl.split.halves, pl.split.cut, pl.split.kb != pl.split.k_blocks};
    memcpy(plan, v, sizeof(v));
    return SWIN_WATTN_OK;
}

int swin_block_gated_test_corrupt_workspace(swin_block_gated_t h, int side)
{
    if (!h || side < 0 || side > 1) return SWIN_WATTN_EINVAL;
    return ws_test_corrupt(h->ws.buf, side);
}

} // extern "C"
