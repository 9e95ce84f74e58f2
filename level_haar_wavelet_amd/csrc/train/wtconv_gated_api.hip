// wtconv_gated_api.hip -- the gated product's plan and entry points
// (include/wtconv.h): argument checks, all before any HIP call.
#include "wtconv_check.h"
#include "wtconv_gated.h"

namespace wtc_gated {

namespace {

constexpr int kUnits = 256;     // compute units
constexpr int64_t kMostSlices = 64;

size_t esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

// Tiles of bm x bn over m x n; where they are fewer than the compute units, each is
// cut along `stages` of the sum.  (Cutting the tiles of a last round that does not fill
// the chip too brought nothing: 8192x2048x5632 bf16 backward, 352 tiles of the weights'
// gradients: 1085 us with it, 1081 and 1114 without.)
Tiles tiles_of(int64_t m, int64_t n, int bm, int bn, int64_t stages, bool cut)
{
    Tiles t = {};
    t.bm = bm;
    t.bn = bn;
    t.tm = (m + bm - 1) / bm;
    t.tn = (int)((n + bn - 1) / bn);
    const int64_t all = t.tm * t.tn;
    int64_t slices = 1;
    if (cut && all < kUnits) {
        // a slice of at least 4 stages
        const int64_t most = stages / 4 < kMostSlices ? stages / 4 : kMostSlices;
        slices = kUnits / all < most ? kUnits / all : most;
        slices = slices < 1 ? 1 : slices;
    }
    t.cut = (stages + slices - 1) / slices;
    t.slices = (int)((stages + t.cut - 1) / t.cut);
    return t;
}

}  // namespace

Plan make_plan(const wtconv_gated_desc_t &d)
{
    Plan p = {};
    p.planes = d.dtype == WTCONV_F32 ? 3 : 1;
    p.pack = p.planes > 1 || d.c % 8;
    p.cp = (int)((d.c + 7) / 8 * 8);
    p.fp = (int)((d.f + 7) / 8 * 8);
    const bool one = p.planes == 1;
    const int bk = one ? 64 : 32;  // of a stage along c and f; along the rows 32
    const int64_t kc = (d.c + bk - 1) / bk, kf = (2 * p.fp + bk - 1) / bk, km = (d.rows + 31) / 32;
    // the large tile where there are enough of them (of fewer, some compute units would have
    // nothing to do)
    auto pick = [&](int64_t m, int64_t n, int64_t stages, bool cut, int half) {
        const Tiles t = tiles_of(m, n, 256, 256 / half, stages, cut);
        if (one && t.tm * t.tn >= kUnits) return t;
        return tiles_of(m, n, 128, 128 / half, stages, cut);
    };
    p.dual = pick(d.rows, d.f, kc, false, 2);
    p.dx = pick(d.rows, d.c, kf, true, 1);
    p.dw = pick(2 * p.fp, d.c, km, true, 1);
    if (p.cp <= (one ? 256 : 192) && d.c % (one ? 8 : 4) == 0 && d.f % 4 == 0) {
        p.steps = 2;
        for (int k : {2, 4, 6, 8, 12, 16})
            if (k * 16 >= p.cp) {
                p.steps = k;
                break;
            }
        p.waves = short_waves(p.planes, p.steps);
        const int64_t rows = p.waves * 32, chunks = (d.f + 63) / 64;
        p.row_tiles = (d.rows + rows - 1) / rows;
        // workgroups for several rounds: 200704x96x384 fp32 225 us with one for a tile of rows,
        // 198 to 207 with three; 50176x192x768 fp16 backward 247 with one, 210 with six
        int64_t parts = (16 * kUnits + p.row_tiles - 1) / p.row_tiles;
        parts = parts > chunks ? chunks : parts;
        p.part_cut = (int)((chunks + parts - 1) / parts);
        p.parts = (int)((chunks + p.part_cut - 1) / p.part_cut);
    }
    // rows of partial sums: at most four waves along a tile's rows, eight of the short kernel's
    const int64_t bias_rows = p.dual.tm * 4 > p.row_tiles * 8 ? p.dual.tm * 4 : p.row_tiles * 8;
    if (p.pack) {
        p.x = align256((size_t)(d.rows * p.cp) * p.planes * 2);
        p.w = align256((size_t)(d.f * 2 * p.cp) * p.planes * 2);
    }
    p.grads = align256((size_t)(d.rows * 2 * p.fp) * p.planes * 2);
    p.bias = align256((size_t)(bias_rows * 2 * p.fp) * 4);
    auto part = [](const Tiles &t) { return t.slices > 1 ? (size_t)(t.groups() * t.bm * t.bn) * 4 : 0; };
    p.part = align256(part(p.dx) > part(p.dw) ? part(p.dx) : part(p.dw));
    return p;
}

size_t workspace_bytes(const wtconv_gated_desc_t &d, bool backward)
{
    const Plan p = make_plan(d);
    if (backward) return p.x + p.w + p.grads + p.bias + p.part;
    return d.rows <= kFewRows ? 0 : p.x + p.w;
}

}  // namespace wtc_gated

namespace {

using namespace wtc_gated;

wtconv_status_t check_desc(const wtconv_gated_desc_t *d)
{
    if (!d) return WTCONV_ERR_NULL;
    if (d->rows < 1 || d->c < 1 || d->f < 1) return WTCONV_ERR_SHAPE;
    // a launch has fewer than 2^32 threads
    if (d->rows >= (int64_t)1 << 30 || d->c > 65536 || d->f > 65536) return WTCONV_ERR_SHAPE;
    if (d->rows * d->c >= (int64_t)1 << 36 || d->rows * d->f >= (int64_t)1 << 36) return WTCONV_ERR_SHAPE;
    if (d->dtype != WTCONV_F32 && d->dtype != WTCONV_F16 && d->dtype != WTCONV_BF16) return WTCONV_ERR_UNSUPPORTED;
    if (d->act < WTCONV_ACT_NONE || d->act > WTCONV_ACT_GELU) return WTCONV_ERR_UNSUPPORTED;
    return WTCONV_OK;
}

struct Sizes {
    size_t x, w, h, b;
};

Sizes sizes_of(const wtconv_gated_desc_t &d)
{
    const size_t e = esize(d.dtype);
    return {(size_t)(d.rows * d.c) * e, (size_t)(d.f * d.c) * e, (size_t)(d.rows * d.f) * e, (size_t)d.f * 4};
}

// x and the weights are read in whole accesses where they are not laid out anew.
size_t factor_alignment(const wtconv_gated_desc_t &d)
{
    return d.dtype != WTCONV_F32 && d.c % 8 == 0 ? 16 : esize(d.dtype);
}

wtconv_status_t check_workspace(size_t need, const void *ws, size_t have)
{
    if (!need) return WTCONV_OK;
    if (!ws || have < need) return WTCONV_ERR_WORKSPACE;
    return aligned_to(ws, 256) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

// dw_f32: the weights' gradients are fp32.
wtconv_status_t backward_of(const wtconv_gated_desc_t *desc, const void *x, const void *dh, const void *w_gate,
                            const void *w_up, const float *b_gate, const float *b_up, void *dx, void *dw_gate,
                            void *dw_up, bool dw_f32, float *db_gate, float *db_up, void *workspace,
                            size_t workspace_bytes, hipStream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!x || !dh || !w_gate || !w_up || !dw_gate != !dw_up || !db_gate != !db_up || (!dx && !dw_gate && !db_gate))
        return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), we = dw_f32 ? 4 : e, fa = factor_alignment(*desc);
    if (!aligned_to(x, fa) || !aligned_to(w_gate, fa) || !aligned_to(w_up, fa) || !aligned_to(dh, e) ||
        !aligned_to(b_gate, 4) || !aligned_to(b_up, 4) || !aligned_to(dx, e) || !aligned_to(dw_gate, we) ||
        !aligned_to(dw_up, we) || !aligned_to(db_gate, 4) || !aligned_to(db_up, 4))
        return WTCONV_ERR_UNSUPPORTED;
    const Sizes s = sizes_of(*desc);
    const size_t need = wtc_gated::workspace_bytes(*desc, true), dw = s.w / e * we;
    const Span in[] = {{x, s.x}, {dh, s.h}, {w_gate, s.w}, {w_up, s.w}, {b_gate, s.b}, {b_up, s.b}},
               out[] = {{dx, s.x}, {dw_gate, dw}, {dw_up, dw}, {db_gate, s.b}, {db_up, s.b}, {workspace, need}};
    if (any_alias(in, 6, out, 5)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(need, workspace, workspace_bytes)) != WTCONV_OK) return st;
    if (any_alias(in, 6, out, 6)) return WTCONV_ERR_ALIAS;
    const Backward a = {x, dh, w_gate, w_up, b_gate, b_up, dx, dw_gate, dw_up, dw_f32, db_gate, db_up};
    hipError_t err;
    if (desc->dtype == WTCONV_F32)
        err = backward<float>(*desc, a, workspace, stream);
    else if (desc->dtype == WTCONV_F16)
        err = backward<_Float16>(*desc, a, workspace, stream);
    else
        err = backward<__bf16>(*desc, a, workspace, stream);
    return err == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

}  // namespace

extern "C" wtconv_status_t wtconv_gated_workspace_size(const wtconv_gated_desc_t *desc, wtconv_op_t op, size_t *bytes)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!bytes) return WTCONV_ERR_NULL;
    if (op != WTCONV_OP_FWD && op != WTCONV_OP_BWD) return WTCONV_ERR_UNSUPPORTED;
    *bytes = workspace_bytes(*desc, op == WTCONV_OP_BWD);
    return WTCONV_OK;
}

extern "C" wtconv_status_t wtconv_gated_forward(const wtconv_gated_desc_t *desc, const void *x, const void *w_gate,
                                                const void *w_up, const float *b_gate, const float *b_up, void *h,
                                                void *workspace, size_t workspace_bytes, wtconv_stream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!x || !w_gate || !w_up || !h) return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), fa = factor_alignment(*desc);
    if (!aligned_to(x, fa) || !aligned_to(w_gate, fa) || !aligned_to(w_up, fa) || !aligned_to(h, e) ||
        !aligned_to(b_gate, 4) || !aligned_to(b_up, 4))
        return WTCONV_ERR_UNSUPPORTED;
    const Sizes s = sizes_of(*desc);
    const size_t need = wtc_gated::workspace_bytes(*desc, false);
    const Span in[] = {{x, s.x}, {w_gate, s.w}, {w_up, s.w}, {b_gate, s.b}, {b_up, s.b}},
               out[] = {{h, s.h}, {workspace, need}};
    if (any_alias(in, 5, out, 1)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(need, workspace, workspace_bytes)) != WTCONV_OK) return st;
    if (any_alias(in, 5, out, 2)) return WTCONV_ERR_ALIAS;
    const Forward a = {x, w_gate, w_up, b_gate, b_up, h};
    hipError_t err;
    if (desc->dtype == WTCONV_F32)
        err = forward<float>(*desc, a, workspace, (hipStream_t)stream);
    else if (desc->dtype == WTCONV_F16)
        err = forward<_Float16>(*desc, a, workspace, (hipStream_t)stream);
    else
        err = forward<__bf16>(*desc, a, workspace, (hipStream_t)stream);
    return err == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

extern "C" wtconv_status_t wtconv_gated_backward(const wtconv_gated_desc_t *desc, const void *x, const void *dh,
                                                 const void *w_gate, const void *w_up, const float *b_gate,
                                                 const float *b_up, void *dx, void *dw_gate, void *dw_up,
                                                 float *db_gate, float *db_up, void *workspace, size_t workspace_bytes,
                                                 wtconv_stream_t stream)
{
    return backward_of(desc, x, dh, w_gate, w_up, b_gate, b_up, dx, dw_gate, dw_up, false, db_gate, db_up, workspace,
                       workspace_bytes, (hipStream_t)stream);
}

extern "C" wtconv_status_t wtconv_gated_backward_f32_grads(const wtconv_gated_desc_t *desc, const void *x,
                                                           const void *dh, const void *w_gate, const void *w_up,
                                                           const float *b_gate, const float *b_up, void *dx,
                                                           float *dw_gate, float *dw_up, float *db_gate,
                                                           float *db_up, void *workspace, size_t workspace_bytes,
                                                           wtconv_stream_t stream)
{
    return backward_of(desc, x, dh, w_gate, w_up, b_gate, b_up, dx, dw_gate, dw_up, true, db_gate, db_up, workspace,
                       workspace_bytes, (hipStream_t)stream);
}
