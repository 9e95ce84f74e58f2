// wtconv_muon_api.hip -- the Newton-Schulz and Muon entry points of the C ABI
// (include/wtconv.h): argument checks, all before any HIP call.
#include <cmath>

#include "wtconv_check.h"
#include "wtconv_muon.h"

namespace {

size_t esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

wtconv_status_t check_desc(const wtconv_ortho_desc_t *d)
{
    if (!d) return WTCONV_ERR_NULL;
    const int64_t lim = ((int64_t)1 << 31) - 1;
    if (d->batch < 1 || d->batch > 65535 || d->rows < 1 || d->cols < 1) return WTCONV_ERR_SHAPE;
    if (d->rows > (1 << 22) || d->cols > (1 << 22) || d->rows * d->cols > lim) return WTCONV_ERR_SHAPE;
    const int64_t r = d->rows < 64 ? 64 : d->rows, c = d->cols < 64 ? 64 : d->cols;
    if (d->batch * r * c >= (int64_t)1 << 36) return WTCONV_ERR_SHAPE;
    if (d->rows > WTCONV_ORTHO_MAX_SIDE && d->cols > WTCONV_ORTHO_MAX_SIDE) return WTCONV_ERR_SHAPE;
    if (d->steps < 1 || d->steps > WTCONV_ORTHO_MAX_STEPS) return WTCONV_ERR_SHAPE;
    if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return WTCONV_ERR_SHAPE;
    if (d->dtype != WTCONV_F32 && d->dtype != WTCONV_F16 && d->dtype != WTCONV_BF16) return WTCONV_ERR_UNSUPPORTED;
    return WTCONV_OK;
}

wtconv_status_t check_workspace(const wtconv_ortho_desc_t &d, const void *ws, size_t have)
{
    const size_t need = wtc_ortho_workspace(d);
    if (!need) return WTCONV_OK;
    if (!ws || have < need) return WTCONV_ERR_WORKSPACE;
    return aligned_to(ws, 256) ? WTCONV_OK : WTCONV_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" wtconv_status_t wtconv_orthogonalize_workspace_size(const wtconv_ortho_desc_t *desc, size_t *bytes)
{
    const wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = wtc_ortho_workspace(*desc);
    return WTCONV_OK;
}

extern "C" wtconv_status_t wtconv_orthogonalize(const wtconv_ortho_desc_t *desc, const void *g, void *out,
                                                void *workspace, size_t workspace_bytes, wtconv_stream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!g || !out) return WTCONV_ERR_NULL;
    const size_t e = esize(desc->dtype), b = (size_t)(desc->batch * desc->rows * desc->cols) * e;
    if (!aligned_to(g, e) || !aligned_to(out, e)) return WTCONV_ERR_UNSUPPORTED;
    if (overlaps(g, out, b)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(*desc, workspace, workspace_bytes)) != WTCONV_OK) return st;
    const size_t wb = wtc_ortho_workspace(*desc);
    if (overlaps2(workspace, wb, g, b) || overlaps2(workspace, wb, out, b)) return WTCONV_ERR_ALIAS;
    const WtcOrthoArgs a = {g, out, nullptr, nullptr, nullptr, nullptr, nullptr};
    return wtc_launch_ortho(*desc, a, workspace, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

extern "C" wtconv_status_t wtconv_muon_step(const wtconv_ortho_desc_t *desc, const wtconv_muon_t *hyper,
                                            const float *weight, const void *grad, const float *momentum,
                                            float *weight_out, float *momentum_out, void *workspace,
                                            size_t workspace_bytes, wtconv_stream_t stream)
{
    wtconv_status_t st = check_desc(desc);
    if (st != WTCONV_OK) return st;
    if (!hyper || !weight || !grad || !momentum || !weight_out || !momentum_out) return WTCONV_ERR_NULL;
    if (hyper->nesterov != 0 && hyper->nesterov != 1) return WTCONV_ERR_UNSUPPORTED;
    const size_t e = esize(desc->dtype), n = (size_t)(desc->batch * desc->rows * desc->cols);
    if (!aligned_to(grad, e) || !aligned_to(weight, 4) || !aligned_to(momentum, 4) || !aligned_to(weight_out, 4) ||
        !aligned_to(momentum_out, 4))
        return WTCONV_ERR_UNSUPPORTED;
    const void *in[] = {weight, momentum}, *out[] = {weight_out, momentum_out};
    for (int i = 0; i < 2; ++i) {
        if (overlaps2(out[i], 4 * n, grad, e * n) || overlaps(out[i], in[1 - i], 4 * n)) return WTCONV_ERR_ALIAS;
        if (out[i] != in[i] && overlaps(out[i], in[i], 4 * n)) return WTCONV_ERR_ALIAS;
    }
    if (overlaps(weight_out, momentum_out, 4 * n)) return WTCONV_ERR_ALIAS;
    if ((st = check_workspace(*desc, workspace, workspace_bytes)) != WTCONV_OK) return st;
    const size_t wb = wtc_ortho_workspace(*desc);
    for (int i = 0; i < 2; ++i)
        if (overlaps2(workspace, wb, in[i], 4 * n) || overlaps2(workspace, wb, out[i], 4 * n)) return WTCONV_ERR_ALIAS;
    if (overlaps2(workspace, wb, grad, e * n)) return WTCONV_ERR_ALIAS;
    const WtcOrthoArgs a = {grad, nullptr, hyper, weight, momentum, weight_out, momentum_out};
    return wtc_launch_ortho(*desc, a, workspace, (hipStream_t)stream) == hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}
