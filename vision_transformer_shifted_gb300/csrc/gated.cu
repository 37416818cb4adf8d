// The gated feed-forward block: C ABI and launches of the kernels in gated.cuh
// and of its products (products.cuh).
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

int cuda_status(cudaError_t e) { return e == cudaSuccess ? SWIN_WATTN_OK : SWIN_WATTN_ECUDA; }

bool bad_pointer(const void *p, bool required)
{
    return p ? (reinterpret_cast<uintptr_t>(p) & 15u) != 0 : required;
}

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
