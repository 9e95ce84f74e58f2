// wtconv_clip_api.hip -- the entry points of the gradient norm and clipping
// (include/wtconv.h): argument checks, all before any HIP call.
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "wtconv_check.h"
#include "wtconv_clip.h"

namespace {

constexpr int64_t kMostTensors = 65536;

size_t esize(int dtype) { return dtype == WTCONV_F32 ? 4 : 2; }

struct Range {
    uintptr_t at, end;
    bool out;
};

// Whether an output overlaps another tensor (its own gradient apart, where it is
// the same memory).  In ascending order, every range has to end before the next
// begins, unless both are only read: so the furthest end of those before, of all
// and of the outputs alone, are what the next is held against.
bool any_overlap(Range *r, size_t n)
{
    const auto less = [](const Range &a, const Range &b) { return a.at < b.at; };
    if (!std::is_sorted(r, r + n, less)) std::sort(r, r + n, less);
    uintptr_t all = 0, outs = 0;
    for (size_t i = 0; i < n; ++i) {
        if (r[i].at < (r[i].out ? all : outs)) return true;
        all = std::max(all, r[i].end);
        if (r[i].out) outs = std::max(outs, r[i].end);
    }
    return false;
}

wtconv_status_t check(const wtconv_tensor_t *t, int64_t count, bool clip, const float *norm, const void *ws, size_t have)
{
    if (count < 0 || count > kMostTensors) return WTCONV_ERR_SHAPE;
    if ((count && !t) || !norm) return WTCONV_ERR_NULL;
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (t[i].elems < 0 || t[i].elems >= (int64_t)1 << 40) return WTCONV_ERR_SHAPE;
        if ((all += t[i].elems) >= (int64_t)1 << 40) return WTCONV_ERR_SHAPE;
        if (t[i].dtype != WTCONV_F32 && t[i].dtype != WTCONV_F16 && t[i].dtype != WTCONV_BF16)
            return WTCONV_ERR_UNSUPPORTED;
        if (!t[i].elems) continue;
        if (!t[i].grad || (clip && !t[i].out)) return WTCONV_ERR_NULL;
        const size_t e = esize(t[i].dtype);
        if (!aligned_to(t[i].grad, e) || (clip && !aligned_to(t[i].out, e))) return WTCONV_ERR_UNSUPPORTED;
    }
    if (!aligned_to(norm, 4)) return WTCONV_ERR_UNSUPPORTED;
    const size_t need = wtc_clip::workspace_bytes(count);
    if (!ws || have < need) return WTCONV_ERR_WORKSPACE;
    if (!aligned_to(ws, 256)) return WTCONV_ERR_UNSUPPORTED;
    if (overlaps2(ws, need, norm, 4)) return WTCONV_ERR_ALIAS;
    const size_t n = (size_t)count * (clip ? 2 : 1) + 2;
    std::unique_ptr<Range[]> r(new (std::nothrow) Range[n]);
    if (!r) return WTCONV_ERR_HIP;
    size_t k = 0;
    r[k++] = {(uintptr_t)norm, (uintptr_t)norm + 4, true};
    r[k++] = {(uintptr_t)ws, (uintptr_t)ws + need, true};
    for (int64_t i = 0; i < count; ++i) {
        if (!t[i].elems) continue;
        const size_t b = (size_t)t[i].elems * esize(t[i].dtype);
        const uintptr_t g = (uintptr_t)t[i].grad, o = (uintptr_t)t[i].out;
        if (clip) r[k++] = {o, o + b, true};
        if (!clip || o != g) r[k++] = {g, g + b, false};
    }
    return any_overlap(r.get(), k) ? WTCONV_ERR_ALIAS : WTCONV_OK;
}

}  // namespace

extern "C" wtconv_status_t wtconv_grad_norm_workspace_size(int64_t count, size_t *bytes)
{
    if (count < 0 || count > kMostTensors) return WTCONV_ERR_SHAPE;
    if (!bytes) return WTCONV_ERR_NULL;
    *bytes = wtc_clip::workspace_bytes(count);
    return WTCONV_OK;
}

extern "C" wtconv_status_t wtconv_grad_norm(const wtconv_tensor_t *tensors, int64_t count, float *norm,
                                            void *workspace, size_t workspace_bytes, wtconv_stream_t stream)
{
    const wtconv_status_t st = check(tensors, count, false, norm, workspace, workspace_bytes);
    if (st != WTCONV_OK) return st;
    return wtc_launch_clip(tensors, count, false, 0.f, 0.f, norm, (double *)workspace, (hipStream_t)stream) ==
                   hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}

extern "C" wtconv_status_t wtconv_clip_grad_norm(const wtconv_tensor_t *tensors, int64_t count, float max_norm,
                                                 float eps, float *norm, void *workspace, size_t workspace_bytes,
                                                 wtconv_stream_t stream)
{
    if (!(max_norm >= 0.f) || !(eps >= 0.f) || !std::isfinite(max_norm) || !std::isfinite(eps) ||
        (max_norm == 0.f && eps == 0.f))
        return WTCONV_ERR_SHAPE;
    const wtconv_status_t st = check(tensors, count, true, norm, workspace, workspace_bytes);
    if (st != WTCONV_OK) return st;
    return wtc_launch_clip(tensors, count, true, max_norm, eps, norm, (double *)workspace, (hipStream_t)stream) ==
                   hipSuccess ? WTCONV_OK : WTCONV_ERR_HIP;
}
