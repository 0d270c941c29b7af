// Shared by the selective scan's files: the arguments of its kernels and the
// step size's map.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "linattn.h"

namespace la {
namespace scan {

// Rows at p + b bs + n ts (+ h P, + g S, + h): x, z, y [B, N, H, P], B and C
// [B, N, G, S], step [B, N, H].
struct ScanArgs {
    const void *x, *step, *Bm, *Cm, *z;
    void* y;
    int64_t x_bs, x_ts, step_bs, step_ts, b_bs, b_ts, c_bs, c_ts, z_bs, z_ts, y_bs, y_ts;
    const float *A, *D, *step_bias, *S0;
    float* S_out;               // [B, H, S, P]
    const int32_t* lengths;     // [B] or null
    float* seeds;               // [B H, nseg, S, P]: end states, then the segments' start states
    float* seg_decay;           // [B H, nseg]: sum of d A over the segment
    int N, H, G, S, P, softplus;
    int nseg, seg_len;
};

// softplus(v) = max(v, 0) + log(1 + e^-|v|), or v as it is.
__device__ __forceinline__ float step_size(float v, int softplus) {
    return softplus ? fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))) : v;
}

// Tensor-core path (csrc/scan_tc.cu): whether these arguments can take it, its
// segments, and the launches.
bool tc_supported(const ScanArgs& a, int B, la_dtype dt);
int tc_segments(int64_t B, int H, int G, int N, int P);
cudaError_t tc_scan(ScanArgs& a, int B, void* ws_header, cudaStream_t st);

int recurrence_segments(int64_t BH, int N);
cudaError_t launch_seeds(const ScanArgs& a, int64_t BH, cudaStream_t st);

}  // namespace scan
}  // namespace la
