// The linear operator: C ABI, launches, and the kernel of an activation's
// gradient.
//   forward   out = residual + act(x W^T + b)      (one kernel; linear.cuh, or for
//             few rows gated_few.cu; a second joins tiles cut along K)
//   backward  dz = dy act'(z) with its column sums (one kernel, where there is an
//             activation), dx = dz W, dW = dz^T x, and the sums' last additions
#include <climits>
#include <cstring>
#include <new>

#include "swin_linear.h"
#include "swin_wattn_test.h"
#include "linear.cuh"

using namespace swin;

struct swin_block_linear_s {
    int C, N, act;   // act: ACT_*
    int device;      // -1: created without one
    int *d_err;
    int last_launches;
    OrderedWorkspace ws;
};

namespace {

constexpr int MAX_WIDTH = 65536;
constexpr int MAX_ROWS = INT_MAX - 512;   // row coordinates of the last tile stay below 2^31
constexpr uint64_t WAIT_NS = 2000000000ull;

bool bad_pointer(const void *p, bool required)
{
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) != 0 : required;
}

struct Span {
    const void *p;
    int64_t bytes;
};
bool any_overlap(Span o, std::initializer_list<Span> in)
{
    if (!o.p) return false;
    for (const Span &s : in)
        if (s.p && overlaps(o.p, o.bytes, s.p, s.bytes)) return true;
    return false;
}

// The handle's device is the current one.
int check_device(const swin_block_linear_s *h)
{
    int dev = h->device;
    if (dev < 0) return SWIN_WATTN_ECUDA;
    return bind_device(&dev);
}

// ---- forward -----------------------------------------------------------------------

struct Forward {
    const void *x, *w;
    const float *sx, *sw;   // 8-bit form, else null
    const bf16 *bias, *residual;
    bf16 *z, *out;
    int rows;
};
constexpr int elems(bool q8) { return q8 ? 128 : 64; }
Product forward_product(int C, int N, int rows)
{
    Product p{};
    p.k[0] = C;
    p.rows = rows;
    p.cols = N;
    return p;
}

// Whether a product of more than 128 rows goes to the few-row kernel, chunks of 128
// rows with K shared by a cluster, rather than to pairs of CTAs: few tiles of a long
// K.  Estimates in us, from both ways at 25 sizes: there 6.5 and its operands at 13
// TB/s from L2 or half a microsecond a K block of a CTA, here 4.5 and 0.25 to 0.29 a K
// block of the pairs' longest way, 13 for a join (385 x 2968 x 400 17.7 us by pairs, 9.7;
// 800 x 8192 x 1024 26.4, 20.3; 700 x 4096 x 120 12.5, 9.0; not taken: 300 x 1032 x 2056
// 10.2, 11.3; 3779 x 2832 x 424 16.7, 21.5).
bool few_chosen(const Product &p, const ProductsPlan &pl, int elems)
{
    const int64_t tiles = (int64_t)ceil_div(p.cols, 128) * ceil_div(p.rows, FEW_ROWS);
    if (tiles > 2 * sm_count()) return false;
    const int kb = ceil_div(p.k[0], elems);
    const double bytes = tiles * kb * 32768 / 13e6, blocks = 0.5 * ceil_div(kb, few_split(tiles, kb));
    const PairSplit &s = pl.split;
    const double whole = pl.wn == 256 ? 1.0 : pl.wn == 192 ? 0.82 : 0.55;
    const double pairs = s.cut ? 17.5 + 0.283 * whole * ((double)s.full * kb + s.q)
                               : 4.5 + kb * (0.29 * whole * (s.halves ? s.full : ceil_div(s.tiles, s.np)) + (s.halves ? 0.25 : 0.0));
    return 6.5 + (bytes > blocks ? bytes : blocks) < pairs;
}

template <int ACT, bool Q8>
cudaError_t launch_linear(const Forward &f, int C, int N, const ProductsPlan &pl, float *part, DeviceStatus st,
                          cudaStream_t stream, FinishArgs *fin)
{
    using P = LinearPolicy<ACT, Q8>;
    typename P::Args a;
    memset(&a, 0, sizeof(a));
    cudaError_t e;
    if ((e = map_k(&a.x, f.x, f.rows, C, 128, Q8)) != cudaSuccess) return e;
    if ((e = map_k(&a.w, f.w, N, C, pl.wn / 2, Q8)) != cudaSuccess) return e;
    if (pl.split.halves && (e = map_k(&a.w_half, f.w, N, C, pl.wn / 4, Q8)) != cudaSuccess) return e;
    if ((e = map_out(&a.out, f.out, f.rows, N)) != cudaSuccess) return e;
    if (f.z && (e = map_out(&a.z, f.z, f.rows, N)) != cudaSuccess) return e;
    a.split = pl.split;
    a.bias = f.bias;
    a.residual = f.residual;
    a.sx = f.sx;
    a.sw = f.sw;
    a.rows = f.rows;
    a.cols = N;
    a.k = C;
    a.mt = ceil_div(f.rows, 256);
    a.nt = ceil_div(N, pl.wn);
    a.wn = pl.wn;
    // (t d < 2^32 for all tiles t: the product's error is then below 1 / d)
    const int64_t d = 8ll * a.nt;
    a.per_band = (int64_t)a.mt * a.nt * d < (1ll << 32) ? (uint32_t)(((1ll << 32) + d - 1) / d) : 0;
    a.np = pl.split.np;
    a.keep = f.z != nullptr;
    a.st = st;
    if (pl.split.cut) {
        e = make_tensor_map(&a.part, T_F32, part, pl.wn, (int64_t)a.np * 2 * 256, (int64_t)pl.wn * 4, 16, 32, 64);
        if (e != cudaSuccess) return e;
        JoinArgs &j = fin->join[0];
        j.part = part;
        j.slots = 2;
        j.split = pl.split;
        j.tn = pl.wn;
        j.blocks = pl.split.cut >= 16 ? 16 : 64;
        j.linear = {true, ACT, f.sx, f.sw, f.z};
        j.p[0] = {f.bias, f.residual, f.out, f.rows, N, a.mt, a.nt, 0};
        j.p[1].first = j.p[2].first = INT_MAX;
        fin->joins[0] = pl.split.cut * j.blocks;
    }
    return launch_pair<P>(a, stream);
}

int forward(swin_block_linear_s *h, const Forward &f, cudaStream_t stream)
{
    int rc = check_device(h);
    if (rc != SWIN_WATTN_OK) return rc;
    const DeviceStatus st{h->d_err, WAIT_NS};
    const bool q8 = f.sx != nullptr;
    const Product p = forward_product(h->C, h->N, f.rows);
    const ProductsPlan pl = f.rows <= FEW_ROWS ? ProductsPlan{} : plan_products(&p, 1, elems(q8));
    if (f.rows <= FEW_ROWS || few_chosen(p, pl, elems(q8))) {
        h->last_launches = 1;
        const FewLinear u{f.x, f.w, f.bias, f.residual, f.sx, f.sw, f.out, f.z, f.rows, h->C, h->N, h->act};
        const cudaError_t e = f.rows == 1 ? launch_token_linear(u, stream) : launch_few_linear(u, st, stream);
        return e == cudaSuccess ? SWIN_WATTN_OK : SWIN_WATTN_ECUDA;
    }
    void *ws = nullptr;
    bool captured = false;
    if (pl.part_bytes && (rc = ows_begin(&h->ws, pl.part_bytes, stream, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    FinishArgs fin{};
    auto run = [&](auto act) {
        constexpr int A = decltype(act)::value;
        return q8 ? launch_linear<A, true>(f, h->C, h->N, pl, (float *)ws, st, stream, &fin)
                  : launch_linear<A, false>(f, h->C, h->N, pl, (float *)ws, st, stream, &fin);
    };
    h->last_launches = 1;
    cudaError_t e = h->act == ACT_SILU   ? run(std::integral_constant<int, ACT_SILU>{})
                    : h->act == ACT_GELU ? run(std::integral_constant<int, ACT_GELU>{})
                                         : run(std::integral_constant<int, ACT_NONE>{});
    if (e == cudaSuccess) e = launch_finish(fin, stream, &h->last_launches);
    const int rc2 = ows_end(&h->ws, stream, ws, captured);
    return e != cudaSuccess ? SWIN_WATTN_ECUDA : rc2;
}

// ---- dz = dy act'(z) ------------------------------------------------------------------
//
// Elementwise, HBM (or, from a layer just run, L2) bounds it.  A thread takes
// eight columns and every rows_at_once * slices-th row, four rows of loads in
// flight, and adds up its columns of the unrounded dz; a block's sums are a
// partial row.
struct GradArgs {
    const bf16 *z, *dy;
    bf16 *dz;
    float *part;   // [slices, N], or null
    int64_t rows;
    int N, ld;     // ld: of dz
    int across, at_once, slices;   // threads across a row (of eight columns each), rows a block takes at once
};
template <int ACT>
__global__ void __launch_bounds__(256) act_grad_kernel(const GradArgs a)
{
    __shared__ float sums[256][9];
    griddep_launch_dependents();
    griddep_wait();
    const int t = (int)threadIdx.x % a.across, r = (int)threadIdx.x / a.across;
    const int c = ((int)blockIdx.x * a.across + t) * 8;
    const bool on = r < a.at_once && c < a.N;
    f2 sum[4] = {0, 0, 0, 0};
    if (on) {
        const int64_t step = (int64_t)a.at_once * a.slices;
        auto grad = [&](int64_t row, const uint4 &zu, const uint4 &du) {
            const uint32_t zw[4] = {zu.x, zu.y, zu.z, zu.w}, dw[4] = {du.x, du.y, du.z, du.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 zf = unpack_bf16x2(zw[e]), df = unpack_bf16x2(dw[e]);
                f2 act, slope;
                activate_grad2<ACT>(pack2(zf.x, zf.y), act, slope);
                const f2 v = mul2(pack2(df.x, df.y), slope);
                sum[e] = add2(sum[e], v);
                float lo, hi;
                unpack2(v, lo, hi);
                o[e] = pack_bf16x2(lo, hi);
            }
            *reinterpret_cast<uint4 *>(a.dz + row * a.ld + c) = make_uint4(o[0], o[1], o[2], o[3]);
        };
        int64_t row = (int64_t)blockIdx.y * a.at_once + r;
#pragma unroll 1
        for (; row + 3 * step < a.rows; row += 4 * step) {
            uint4 z[4], d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                z[k] = *reinterpret_cast<const uint4 *>(a.z + (row + k * step) * a.N + c);
                d[k] = *reinterpret_cast<const uint4 *>(a.dy + (row + k * step) * a.N + c);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) grad(row + k * step, z[k], d[k]);
        }
#pragma unroll 1
        for (; row < a.rows; row += step)
            grad(row, *reinterpret_cast<const uint4 *>(a.z + row * a.N + c),
                 *reinterpret_cast<const uint4 *>(a.dy + row * a.N + c));
    }
    if (!a.part) return;
#pragma unroll
    for (int e = 0; e < 4; ++e) unpack2(sum[e], sums[threadIdx.x][2 * e], sums[threadIdx.x][2 * e + 1]);
    __syncthreads();
    if (r > 0 || !on) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = sums[t][e];
    for (int i = 1; i < a.at_once; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += sums[i * a.across + t][e];
    float *out = a.part + (int64_t)blockIdx.y * a.N + c;
    *reinterpret_cast<float4 *>(out) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
// Threads across a row: all of its pieces where a block holds them, else even
// shares; rows: about six blocks an SM in all, at least four rows a thread.
struct GradPlan {
    int across, at_once, columns, slices;   // columns: blocks across a row
};
GradPlan plan_grad(int N, int64_t rows)
{
    GradPlan p{};
    const int pieces = N / 8;
    p.columns = ceil_div(pieces, 256);
    p.across = ceil_div(pieces, p.columns);
    p.at_once = 256 / p.across;
    const int64_t most = ceil_div(6 * sm_count(), p.columns), want = ceil_div(rows, 4 * (int64_t)p.at_once);
    p.slices = (int)(want < most ? want : most);
    return p;
}

constexpr int SIDE_SLICES = 512;   // partial rows of db that dx's warps add
// Rows that one warp adds to the end, no launch for a join: 34 x 336 x 576 GELU 15.5 us
// and 13.8, 250 x 512 x 128 without activation 13.1 and 10.1, 130 x 2048 x 2048 19.4 and
// 17.5, 600 x 512 x 1024 GELU (over 64 partial rows of dz's kernel) 22.8 and 19.1.  More
// would keep the warp, and the tile it drains next, longer than a launch takes.
constexpr int FEW_SUMS = 256;

// The shapes of the backward's products.
Product dx_product(int C, int N, int rows, int ld)
{
    Product p{};
    p.k[0] = N;
    p.lda = ld;
    p.rows = rows;
    p.cols = C;
    return p;
}
Product weight_product(int C, int N, int rows, int ld)
{
    Product p{};
    p.k[0] = rows;
    p.lda = ld;
    p.rows = N;
    p.cols = C;
    return p;
}

// What a backward call queues, and which kernel finishes what.
struct BackwardPlan {
    int ld;                 // of dz
    ProductsPlan dx, dw;
    ActWgradPlan through;   // dW through an activation
    GradPlan grad;
    bool few;               // dx by the few-row kernel
    bool side;              // dx's epilogue warps finish what dW's kernel leaves
    bool direct;            // db is added to the end by dW's epilogue warps
    bool dx_adds;           // db's partial rows are added by dx's epilogue warps
    int slices;             // partial rows of db
    size_t dz_bytes, dw_bytes, sum_bytes;   // of the workspace, beside dx.part_bytes
};
BackwardPlan plan_backward(int C, int N, int rows, bool act, bool dx, bool dW, bool db)
{
    BackwardPlan p{};
    p.ld = act ? hidden_ld(N) : N;
    const Product px = dx_product(C, N, rows, p.ld), pw = weight_product(C, N, rows, p.ld);
    if (dx) p.dx = plan_products(&px, 1);
    if (dW) p.dw = plan_products(&pw, 1);
    // few rows: dx by the few-row kernel
    p.few = dx && (rows <= FEW_ROWS || few_chosen(px, p.dx, 64));
    if (p.few) p.dx.part_bytes = 0;
    if (act && dW) p.through = plan_act_wgrad(C, N, rows, p.dw);
    p.grad = plan_grad(N, rows);
    p.slices = p.through.chosen ? p.through.slices : act ? p.grad.slices : rows <= FEW_SUMS ? 1 : column_slices(rows);
    // Few rows of dy are added to the end by the weight gradient's waiting warps, and
    // leave nothing of db to any other kernel.
    const bool dy_direct = db && !act && rows <= FEW_SUMS, sums_left = db && !dy_direct;
    // What dW's kernel leaves, cut tiles and db's partial rows, is finished by dx's
    // epilogue warps under their first tile's MMAs: where they are on most SMs, db's
    // rows are few, and no launch is left to save otherwise (dx's own cut tiles).
    // 12544 x 512 x 2048 GELU 60.2 us, 69.7 by a launch of its own, 50000 x 256 x 1024
    // 80 and 91, 2000 x 2048 x 2048 36.4 and 42.3; 300 x 512 x 1024, on 16 SMs, 48.6
    // and 24.
    p.side = dx && !p.few && dW && (p.through.chosen || p.dw.split.cut || sums_left) &&
             (!sums_left || p.slices <= SIDE_SLICES) && !p.dx.split.cut && 8 * p.dx.split.np >= 3 * sm_count();
    p.dx_adds = p.side && sums_left;
    // So are few rows of dz's kernel's partial sums.
    p.direct = dy_direct || (db && act && !p.through.chosen && !p.side && !p.dw.split.cut && p.slices <= FEW_SUMS);
    p.dz_bytes = act && (dx || !p.through.chosen) ? (size_t)rows * p.ld * 2 : 0;
    p.dw_bytes = p.through.chosen ? p.through.part_bytes : p.dw.part_bytes;
    p.sum_bytes = db && (act || !p.direct) ? (size_t)p.slices * N * sizeof(float) : 0;
    return p;
}

} // namespace

extern "C" {

int swin_block_linear_create(swin_block_linear_t *out, int C, int N, int act)
{
    if (!out) return SWIN_WATTN_EINVAL;
    *out = nullptr;
    if (C <= 0 || C % 8 || C > MAX_WIDTH || N <= 0 || N % 8 || N > MAX_WIDTH) return SWIN_WATTN_EINVAL;
    if (act != SWIN_BLOCK_LINEAR_NONE && act != SWIN_BLOCK_LINEAR_SILU && act != SWIN_BLOCK_LINEAR_GELU)
        return SWIN_WATTN_EINVAL;
    swin_block_linear_s *h = new (std::nothrow) swin_block_linear_s{};
    if (!h) return SWIN_WATTN_ENOMEM;
    h->C = C;
    h->N = N;
    h->act = act == SWIN_BLOCK_LINEAR_SILU ? ACT_SILU : act == SWIN_BLOCK_LINEAR_GELU ? ACT_GELU : ACT_NONE;
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

int swin_block_linear_destroy(swin_block_linear_t h)
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

int swin_block_linear_last_launches(swin_block_linear_t h) { return h ? h->last_launches : 0; }

int swin_block_linear_sync_status(swin_block_linear_t h, swin_stream_t stream)
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

int swin_block_linear_forward(swin_block_linear_t h, const void *x, int rows, const void *W, const void *b,
                              const void *residual, void *z, void *out, swin_stream_t stream)
{
    if (!h || rows < 0 || rows > MAX_ROWS || (z && h->act == ACT_NONE)) return SWIN_WATTN_EINVAL;
    if (rows == 0) return SWIN_WATTN_OK;   // (an empty tensor may have no address)
    for (const void *q : {x, W, (const void *)out})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {b, residual, (const void *)z})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const int64_t in = 2 * (int64_t)rows * h->C, on = 2 * (int64_t)rows * h->N, w = 2 * (int64_t)h->C * h->N, v = 2 * (int64_t)h->N;
    if (any_overlap({out, on}, {{x, in}, {W, w}, {b, v}, {z, on}, {residual == out ? nullptr : residual, on}}) ||
        any_overlap({z, on}, {{x, in}, {W, w}, {b, v}, {residual, on}}))
        return SWIN_WATTN_EINVAL;
    return forward(h, {x, W, nullptr, nullptr, (const bf16 *)b, (const bf16 *)residual, (bf16 *)z, (bf16 *)out, rows},
                   (cudaStream_t)stream);
}

int swin_block_linear_forward_q8(swin_block_linear_t h, const void *x8, const float *sx, int rows, const void *W8,
                                 const float *sw, const void *b, const void *residual, void *out, swin_stream_t stream)
{
    if (!h || rows < 0 || rows > MAX_ROWS) return SWIN_WATTN_EINVAL;
    if (h->C % 16) return SWIN_WATTN_EUNSUPPORTED;
    if (rows == 0) return SWIN_WATTN_OK;
    for (const void *q : {x8, (const void *)sx, W8, (const void *)sw, (const void *)out})
        if (bad_pointer(q, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {b, residual})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const int64_t in = (int64_t)rows * h->C, on = 2 * (int64_t)rows * h->N, w = (int64_t)h->C * h->N, v = 2 * (int64_t)h->N;
    if (any_overlap({out, on}, {{x8, in}, {sx, 4 * (int64_t)rows}, {W8, w}, {sw, 2 * v}, {b, v},
                                {residual == out ? nullptr : residual, on}}))
        return SWIN_WATTN_EINVAL;
    return forward(h, {x8, W8, sx, sw, (const bf16 *)b, (const bf16 *)residual, nullptr, (bf16 *)out, rows},
                   (cudaStream_t)stream);
}

int swin_block_linear_backward(swin_block_linear_t h, const void *x, int rows, const void *W, const void *z,
                               const void *dy, void *dx, void *dW, void *db, swin_stream_t stream)
{
    if (!h || rows < 0 || rows > MAX_ROWS || (!dx && !dW) || (db && !dW) || (z && h->act == ACT_NONE))
        return SWIN_WATTN_EINVAL;
    const bool act = h->act != ACT_NONE;
    const int64_t in = 2 * (int64_t)rows * h->C, on = 2 * (int64_t)rows * h->N, w = 2 * (int64_t)h->C * h->N, v = 2 * (int64_t)h->N;
    for (const void *q : {x, dy})
        if (bad_pointer(q, rows > 0)) return SWIN_WATTN_EINVAL;
    if (bad_pointer(z, act && rows > 0) || bad_pointer(W, true)) return SWIN_WATTN_EINVAL;
    for (const void *q : {dx, dW, db})
        if (bad_pointer(q, false)) return SWIN_WATTN_EINVAL;
    const Span outs[] = {{dx, in}, {dW, w}, {db, v}};
    for (int i = 0; i < 3; ++i) {
        if (any_overlap(outs[i], {{x, in}, {W, w}, {z, on}, {dy, on}})) return SWIN_WATTN_EINVAL;
        for (int j = 0; j < i; ++j)
            if (any_overlap(outs[i], {outs[j]})) return SWIN_WATTN_EINVAL;
    }
    int rc = check_device(h);
    if (rc != SWIN_WATTN_OK) return rc;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        for (int i = 1; i < 3; ++i)
            if (outs[i].p && cudaMemsetAsync(const_cast<void *>(outs[i].p), 0, outs[i].bytes, s) != cudaSuccess)
                return SWIN_WATTN_ECUDA;
        return SWIN_WATTN_OK;
    }
    const BackwardPlan pl = plan_backward(h->C, h->N, rows, act, dx != nullptr, dW != nullptr, db != nullptr);
    const int ld = pl.ld;
    Product px = dx_product(h->C, h->N, rows, ld), pw = weight_product(h->C, h->N, rows, ld);
    FinishArgs fin{};
    Carve size(nullptr);
    size.take(pl.dz_bytes);
    size.take(pl.dx.part_bytes);
    size.take(pl.dw_bytes);
    size.take(pl.sum_bytes);
    void *ws = nullptr;
    bool captured = false;
    if (size.used && (rc = ows_begin(&h->ws, size.used, s, &ws, &captured)) != SWIN_WATTN_OK) return rc;
    Carve carve(ws);
    bf16 *dz = (bf16 *)carve.take(pl.dz_bytes);
    float *x_part = (float *)carve.take(pl.dx.part_bytes), *w_part = (float *)carve.take(pl.dw_bytes);
    float *sum_part = (float *)carve.take(pl.sum_bytes);
    if (db) {
        auto &m = fin.cs.m[fin.cs.n++];
        m.out = (bf16 *)db;
        m.cols = h->N;
        m.part = pl.direct ? nullptr : sum_part;
        m.b = act ? nullptr : (const bf16 *)dy;
        m.f = act ? sum_part : nullptr;
        m.rows = act ? pl.slices : rows;
        m.slices = pl.direct ? 1 : pl.slices;
        m.tasks = pl.direct ? ceil_div(h->N, act ? 16 : 32) : act ? 0 : ceil_div(h->N, 256) * m.slices;
    }
    px.a[0] = pw.a[0] = act ? (const void *)dz : dy;
    px.b[0] = W;
    px.d = (bf16 *)dx;
    pw.b[0] = x;
    pw.d = (bf16 *)dW;
    const DeviceStatus st{h->d_err, WAIT_NS};
    h->last_launches = 0;
    cudaError_t e = cudaSuccess;
    if (pl.through.chosen) {
        const ActWgrad w{(const bf16 *)z, (const bf16 *)dy, (const bf16 *)x, dx ? dz : nullptr, (bf16 *)dW, db ? sum_part : nullptr,
                         w_part, rows, h->C, h->N, ld, h->act};
        ++h->last_launches;
        e = launch_act_wgrad(w, pl.through, st, s, &fin.join[1], &fin.joins[1]);
    } else if (act) {
        const GradArgs a{(const bf16 *)z, (const bf16 *)dy, dz, db ? sum_part : nullptr, rows, h->N, ld, pl.grad.across,
                         pl.grad.at_once, pl.grad.slices};
        ++h->last_launches;
        e = launch_maybe_overlapped(h->act == ACT_SILU ? act_grad_kernel<ACT_SILU> : act_grad_kernel<ACT_GELU>,
                                    dim3((unsigned)pl.grad.columns, (unsigned)pl.grad.slices), dim3(256), 0, s, 1, a);
    }
    // (behind dx, whose results it does not read, it runs beside it, reading through L2
    // what was complete before dx's kernel let it start: see CHAIN_EARLY; 60 x 152 x 1736 11.1
    // us one after the other, 8.2; 300 x 1032 x 256 GELU 13.8 and 11.2)
    auto weight = [&]() {
        if (e == cudaSuccess && dW && !pl.through.chosen)
            e = launch_products<true, true>(&pw, pl.dw, w_part, st, s, &h->last_launches, &fin, 1, nullptr,
                                            dx && !pl.side ? CHAIN_EARLY : CHAIN_NONE);
    };
    if (pl.side) weight();
    if (e == cudaSuccess && dx) {
        FinishArgs left = fin;
        if (!pl.dx_adds) left.cs.n = 0;
        if (pl.side) fin.joins[1] = fin.cs.n = 0;
        if (pl.few) {
            ++h->last_launches;
            e = launch_few_dx((const bf16 *)px.a[0], ld, rows, (const bf16 *)W, (bf16 *)dx, h->C, h->N, st, s);
        } else {
            e = launch_products<false, true>(&px, pl.dx, x_part, st, s, &h->last_launches, &fin, 0, pl.side ? &left : nullptr);
        }
    }
    if (!pl.side) weight();
    if (pl.direct) fin.cs.n = 0;   // (done)
    if (e == cudaSuccess) e = launch_finish(fin, s, &h->last_launches);
    const int rc2 = ows_end(&h->ws, s, ws, captured);
    return e != cudaSuccess ? SWIN_WATTN_ECUDA : rc2;
}

// ---- test hooks (swin_wattn_test.h) ------------------------------------------------

int swin_block_linear_test_plan(int C, int N, int rows, int which, int *plan)
{
    if (C <= 0 || C % 8 || C > MAX_WIDTH || N <= 0 || N % 8 || N > MAX_WIDTH || rows <= 0 || rows > MAX_ROWS || !plan)
        return SWIN_WATTN_EINVAL;
    Product p;
    if (which == SWIN_BLOCK_LINEAR_PLAN_ACT_WEIGHT) {
        p = weight_product(C, N, rows, N);
        const ActWgradPlan a = plan_act_wgrad(C, N, rows, plan_products(&p, 1));
        const int v[] = {a.tiles, a.tiles * a.slices, a.n, a.nt, a.slices, a.chosen};
        memcpy(plan, v, sizeof(v));
        return SWIN_WATTN_OK;
    }
    if (which == SWIN_BLOCK_LINEAR_PLAN_FORWARD || which == SWIN_BLOCK_LINEAR_PLAN_FORWARD_Q8) p = forward_product(C, N, rows);
    else if (which == SWIN_BLOCK_LINEAR_PLAN_DX) p = dx_product(C, N, rows, N);
    else if (which == SWIN_BLOCK_LINEAR_PLAN_WEIGHT) p = weight_product(C, N, rows, N);
    else return SWIN_WATTN_EINVAL;
    const int block = elems(which == SWIN_BLOCK_LINEAR_PLAN_FORWARD_Q8);
    const ProductsPlan pl = plan_products(&p, 1, block);
    const bool few = which != SWIN_BLOCK_LINEAR_PLAN_WEIGHT && (rows <= FEW_ROWS || few_chosen(p, pl, block));
    const int v[] = {pl.split.tiles, few ? 0 : pl.split.np, pl.wn, pl.split.halves, pl.split.cut, pl.split.kb != pl.split.k_blocks};
    memcpy(plan, v, sizeof(v));
    return SWIN_WATTN_OK;
}

int swin_block_linear_test_backward_plan(int C, int N, int rows, int act, int which, int *plan)
{
    if (C <= 0 || C % 8 || C > MAX_WIDTH || N <= 0 || N % 8 || N > MAX_WIDTH || rows <= 0 || rows > MAX_ROWS || !plan)
        return SWIN_WATTN_EINVAL;
    const bool dx = which & SWIN_BLOCK_LINEAR_GRAD_DX, dW = which & SWIN_BLOCK_LINEAR_GRAD_DW, db = which & SWIN_BLOCK_LINEAR_GRAD_DB;
    if (which < 0 || which > 7 || (!dx && !dW) || (db && !dW)) return SWIN_WATTN_EINVAL;
    const BackwardPlan p = plan_backward(C, N, rows, act != SWIN_BLOCK_LINEAR_NONE, dx, dW, db);
    const int v[] = {p.few, p.side, p.direct, p.dx_adds, p.slices, p.sum_bytes != 0, p.through.chosen,
                     p.through.chosen ? p.through.tiles : p.dw.split.cut, p.few ? 0 : p.dx.split.cut};
    memcpy(plan, v, sizeof(v));
    return SWIN_WATTN_OK;
}

int swin_block_linear_test_clusters_of(int device, int split, int alone, int answer)
{
    if (split < 1 || split > 16 || answer < 0) return SWIN_WATTN_EINVAL;
    return test_few_clusters_of(device, split, alone != 0, answer);
}

int swin_block_linear_test_corrupt_workspace(swin_block_linear_t h, int side)
{
    if (!h || side < 0 || side > 1) return SWIN_WATTN_EINVAL;
    return ws_test_corrupt(h->ws.buf, side);
}

} // extern "C"
