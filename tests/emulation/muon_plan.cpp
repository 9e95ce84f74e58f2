// muon_plan.cpp -- the plans of the tiled Newton-Schulz path, compiled for the
// host (test tool): which kernel instances a call launches.
#include "../../level_haar_wavelet_amd/csrc/train/wtconv_muon_plan.h"

// 1 and, for the Gram product, the polynomial and P X: {tile, deep, full tiles,
// tiles cut along k, slices of those, 32-blocks of k in a slice, padded rows,
// padded columns}; 0 where one workgroup holds a matrix.  `bytes`: of the workspace.
extern "C" int emu_muon_plan(int64_t batch, int64_t rows, int64_t cols, int64_t *out, int64_t *bytes)
{
    using namespace wtc_muon;
    const wtconv_ortho_desc_t d = {batch, rows, cols, WTCONV_F32, 5, 1e-7f};
    const Plan p = make_plan(d);
    *bytes = (int64_t)workspace_bytes(p, batch);
    if (p.one) return 0;
    const Deal *deals[] = {&p.gram, &p.poly, &p.apply};
    const int lp[] = {p.np, p.np, p.np}, rp[] = {p.np, p.np, p.mp}, kp[] = {p.mp, p.np, p.np};
    for (int i = 0; i < 3; ++i) {
        const Deal &e = *deals[i];
        const int64_t rest = (int64_t)e.tiles * batch - e.full, groups = e.full + rest * e.slices;
        const int64_t v[] = {e.tile, is_deep(groups, e.slices > 1 ? e.cut : kp[i] / 32, e.tile), e.full, rest,
                             e.slices, e.cut, lp[i], rp[i]};
        for (int k = 0; k < 8; ++k) out[8 * i + k] = v[k];
    }
    return 1;
}
