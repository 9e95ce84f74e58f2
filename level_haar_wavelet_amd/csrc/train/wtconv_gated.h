// wtconv_gated.h -- plan and launch entry points of the gated product's kernels.
#ifndef WTCONV_GATED_H
#define WTCONV_GATED_H

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../../include/wtconv.h"

namespace wtc_gated {

// Rows up to which the forward call takes the weights straight into registers: us with it, and
// with tiles of 128 rows or more in its place:
//   rows              1        16        32        64
//   4096x4096 bf16   17, 39   19, 40   25, 40   40, 40
//   2048x5632 bf16   13, 23   14, 23   18, 23   25, 23
//   4096x512  bf16   12, 29   14, 30   17, 30   26, 30
//   4096x4096 fp32   38, 203  42, 209  64, 215  100, 229
constexpr int kFewRows = 64;

struct Forward {
    const void *x, *w_gate, *w_up;
    const float *b_gate, *b_up;
    void *h;
};

struct Backward {
    const void *x, *dh, *w_gate, *w_up;
    const float *b_gate, *b_up;
    void *dx, *dw_gate, *dw_up;
    bool dw_f32;  // the weights' gradients are fp32, whatever the activations' type
    float *db_gate, *db_up;
};

// A product's tile (side of the rows, of the columns), and its cut along the sum's
// index into `slices` of `cut` stages, whose sums are joined.
struct Tiles {
    int bm, bn;
    int64_t tm;
    int tn, slices;
    int64_t cut;
    int64_t groups() const { return tm * tn * slices; }
};

// The calls' plan, a function of the sizes and types alone.
struct Plan {
    int planes;          // 16-bit numbers of a factor: 1, fp32: 3
    bool pack;           // x and the weights are laid out anew (fp32, or rows of no whole accesses)
    int cp, fp;          // row lengths in the workspace: c and f up to a multiple of 8
    Tiles dual, dx, dw;  // g and u; dx; the weights' gradients
    int64_t row_tiles;   // of the kernel for short rows (0: rows are too long for it)
    int steps, waves;    // its steps of 16 in a row, its waves of 32 rows
    int parts, part_cut; // its workgroups for a tile of rows, and their chunks of 64 columns
    // bytes
    size_t x, w, grads, bias, part;
};

// Waves of a workgroup of the kernel for short rows.
constexpr int short_waves(int planes, int steps)
{
    return planes > 1 && steps > 6 ? 8 : 4;
}

Plan make_plan(const wtconv_gated_desc_t &d);
size_t workspace_bytes(const wtconv_gated_desc_t &d, bool backward);

template <typename T>
hipError_t forward(const wtconv_gated_desc_t &d, const Forward &a, void *workspace, hipStream_t stream);
template <typename T>
hipError_t backward(const wtconv_gated_desc_t &d, const Backward &a, void *workspace, hipStream_t stream);

}  // namespace wtc_gated

#endif  // WTCONV_GATED_H
