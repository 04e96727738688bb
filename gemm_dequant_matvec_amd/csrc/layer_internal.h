// Internal declarations of the many-token layer operators (qmv_layer.h).
#pragma once

#include "../../include/qmv_layer.h"
#include "qmv_internal.h"

namespace qmv {

// How the backward pass cuts its product: tile 0 (128 columns x 64 tokens), 1 (128 x 128) or
// 2 (256 x 256), the depth in `splits` of `steps` stages, and what it needs of the workspace:
// f32 partial sums (splits > 1), then 16-bit copies of dG and dU with rows of ld values (N % 8 != 0),
// then their low parts in rows of ld values (wide: dX from the unrounded dG and dU).
struct GluBwdPlan {
  int tile, splits, steps, ld;
  int64_t tiles;
  int64_t part_bytes, copy_bytes, low_bytes;  // copy_bytes, low_bytes: of each of the two
};
GluBwdPlan glu_backward_plan(int64_t N, int64_t K, int64_t M, bool wide);

// Launchers: hipSuccess or the launch error; arguments are already validated.
hipError_t launch_glu_fwd(int fmt, int64_t N, int64_t K, int64_t M, const uint8_t* Wg, const uint8_t* Wu,
                          const uint16_t* X, bool f16, int act, uint16_t* H, uint16_t* G, uint16_t* U, hipStream_t s);
hipError_t launch_glu_bwd(int fmt, int64_t N, int64_t K, int64_t M, const uint8_t* Wg, const uint8_t* Wu,
                          const uint16_t* G, const uint16_t* U, const uint16_t* dH, bool f16, int act,
                          const GluBwdPlan& plan, uint16_t* dG, uint16_t* dU, uint16_t* dX, uint8_t* ws, hipStream_t s);
hipError_t launch_rope(int64_t T, int D, int R, int layout, int count, const qmv_rope_tensor* t, int dtype,
                       const int64_t* pos, const float* freqs, float amplitude, int inverse, hipStream_t s);

}  // namespace qmv
