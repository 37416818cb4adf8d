// The general products: plans, launches, and the kernel that finishes their cut
// tiles and the column sums.
#include <climits>
#include <cstring>

#include "products.cuh"

namespace swin {

namespace {

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

__host__ __device__ inline int column_blocks(const ColumnSums &cs, int i) { return (cs.m[i].cols + 7) / 8; }
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ FinishArgs a)
{
    __shared__ float sum[32][8];
    griddep_launch_dependents();
    griddep_wait();
    int b = blockIdx.x;
    for (int i = 0; i < 2; ++i) {
        if (b < a.joins[i]) {
            const JoinArgs &j = a.join[i];
            const int first = b % j.blocks * 256 + (int)threadIdx.x;
            if (j.blocks == 16) join_tile<8>(j, b / 16, first, 16 * 256);
            else join_tile<4>(j, b / 64, first, 64 * 256);
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
} // namespace

cudaError_t launch_finish(const FinishArgs &a, cudaStream_t stream, int *launches)
{
    int blocks = a.joins[0] + a.joins[1];
    for (int i = 0; i < a.cs.n; ++i) blocks += column_blocks(a.cs, i);
    if (!blocks) return cudaSuccess;
    ++*launches;
    return launch_maybe_overlapped(finish_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, 1, a);
}

// Tiles of 256 x 256 where every product has more than 128 columns, else 256 x
// 128.  The last round is cut along K where that saves more K blocks than the
// join costs; few blocks in all go to as many pairs as leave each at least four.
// A last round of at most half of the pairs goes out as half tiles where that
// costs less than either: no join (1024 x 2048 x 5632 forward 61 us cut or whole,
// 57 in halves; 12544 x 512 x 1368 backward, dx's last 22 tiles, 131 cut, 129; its
// weight gradients' 36 tiles of 196 blocks stay cut: in halves 9 us more).
ProductsPlan plan_products(const Product *p, int n, int elems)
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
    s.k_blocks = s.kb = ceil_div(p[0].k[0], elems) + (p[0].k[1] ? ceil_div(p[0].k[1], elems) : 0);
    const int pairs = sm_count() / 2;
    s.np = (int)(tiles < pairs ? tiles : pairs);
    const int full = (int)(tiles / pairs), rest = (int)(tiles - (int64_t)full * pairs);
    const int64_t blocks = (int64_t)rest * s.kb;
    int64_t np = full || blocks / 4 >= pairs ? pairs : blocks / 4 > rest ? blocks / 4 : rest;
    const int cut_cost = ceil_div(blocks, np) + (pl.wide ? WIDE_JOIN : NARROW_JOIN), least = s.kb < cut_cost ? s.kb : cut_cost;
    const bool halves = pl.wide && rest && 2 * rest <= pairs && (int64_t)half_cost(2 * rest, pairs) * s.kb <= 100ll * least;
    const int64_t here = 100ll * full * s.kb + (halves ? (int64_t)half_cost(2 * rest, pairs) * s.kb : rest ? 100ll * least : 0);
    const int64_t tiles192 = count(192), cost192 = (int64_t)ceil_div(tiles192, pairs) * COST_192 * s.kb;
    pl.cost = (pl.wide && cost192 < here ? cost192 : here) * (pl.wide ? 100 : 55) / 100;   // (128 columns: as half a tile)
    if (pl.wide && cost192 < here) {
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

namespace {

template <int TN, bool A_MN, bool B_MN>
cudaError_t launch_products_t(const Product *ps, const ProductsPlan &pl, float *part, DeviceStatus st,
                              cudaStream_t stream, int *launches, FinishArgs *fin, int slot,
                              const FinishArgs *side, int chain)
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
    if (!A_MN && side) {
        a.side = side->join[1];
        a.joined = side->joins[1] ? a.side.split.cut : 0;
        a.sums = side->cs;
    }
    a.wn = pl.wn;
    a.np = pl.split.np;
    a.chain = chain;
    a.st = st;
    if (pl.split.cut) {
        e = make_tensor_map(&a.part, T_F32, part, TN, (int64_t)a.np * 2 * 256, TN * 4, 16, 32, 64);
        if (e != cudaSuccess) return e;
    }
    ++*launches;
    r.part = part;
    r.slots = 2;
    r.tn = TN;
    r.from_last = !A_MN;
    r.blocks = pl.split.cut >= 16 ? 16 : 64;
    fin->joins[slot] = pl.split.cut * r.blocks;
    return launch_pair<GemmPolicy<TN, A_MN, B_MN>>(a, stream);
}

} // namespace

template <bool A_MN, bool B_MN>
cudaError_t launch_products(const Product *ps, const ProductsPlan &pl, float *part, DeviceStatus st,
                            cudaStream_t stream, int *launches, FinishArgs *fin, int slot,
                            const FinishArgs *side, int chain)
{
    return pl.wide ? launch_products_t<256, A_MN, B_MN>(ps, pl, part, st, stream, launches, fin, slot, side, chain)
                   : launch_products_t<128, A_MN, B_MN>(ps, pl, part, st, stream, launches, fin, slot, side, chain);
}
template cudaError_t launch_products<false, false>(const Product *, const ProductsPlan &, float *, DeviceStatus, cudaStream_t,
                                                   int *, FinishArgs *, int, const FinishArgs *, int);
template cudaError_t launch_products<false, true>(const Product *, const ProductsPlan &, float *, DeviceStatus, cudaStream_t,
                                                  int *, FinishArgs *, int, const FinishArgs *, int);
template cudaError_t launch_products<true, true>(const Product *, const ProductsPlan &, float *, DeviceStatus, cudaStream_t,
                                                 int *, FinishArgs *, int, const FinishArgs *, int);

} // namespace swin
