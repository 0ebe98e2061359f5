// The two conversions that leave a DFP-8 tensor: of a floating tensor, and of
// a Linear layer's error behind its activation.  Shared by their entry points.
#pragma once

#include "float_ops.h"

namespace ionn {
namespace dfp8 {

// Workgroups that a maximum is taken by, and maxima that the rounding pass
// reads back.
constexpr int kMaxParts = 1024;

// The errors' pass works on column strips and row ranges; its layout for
// B x OUT errors of es bytes.
struct ActLayout {
    int lanes;        // lanes that share a row (a power of two up to 64)
    int strips;       // column strips of lanes * (16 / es) columns
    int chunks;       // row ranges
    int64_t rows;     // rows of a range
};

ActLayout act_layout(int64_t B, int64_t OUT, size_t es);

// Bytes of the maxima and of the column sums' partial rows.
size_t act_workspace_bytes(int64_t B, int64_t OUT);

// dZ = dY act'(Z): its column sums gb (nullable), its DFP-8 form and status
// (nullable).  B, OUT >= 1.  One launch for small errors, else two.
int launch_act_bwd(const void *dY, const void *Z, int act, int dtype, int64_t B, int64_t OUT, int8_t *dZ8,
                   int32_t *edZ, float *gb, int32_t *status, void *workspace, hipStream_t st);

}  // namespace dfp8
}  // namespace ionn
