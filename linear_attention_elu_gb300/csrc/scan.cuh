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

// softplus(v) = max(v, 0) + log(1 + e^-|v|), or v as it is. With e = e^-|v| the
// logarithm is 2 artanh(s), s = e / (2 + e) <= 1/3, by its odd power series to s^13
// (truncation below 2^-26 of the value), which keeps small step sizes accurate
// relative to themselves; e^-|v| is 2^t with the rounding of t = -|v| log2 e put back.
// |v| is held within 128, where e^-|v| is 0 in fp32 already: the lowest values of a type and
// minus infinity, which mask a token, give 0 (t and its rounding would be infinities that
// cancel to NaN). A comparison, not a minimum, so that NaN stays NaN.
__device__ __forceinline__ float step_size(float v, int softplus) {
    if (!softplus) return v;
    constexpr double kLog2e = 1.44269504088896340736;
    constexpr float kL = (float)kLog2e, kLLo = (float)(kLog2e - (double)kL);
    const float m = fabsf(v), x = m > 128.f ? -128.f : -m, t = x * kL;
    const float r = fmaf(x, kL, -t) + x * kLLo;
    float e, q;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = fmaf(e, r * 0.6931471805599453f, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(2.f + e));
    const float s = e * q, u = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, u, 1.f / 11.f);
    p = fmaf(p, u, 1.f / 9.f);
    p = fmaf(p, u, 1.f / 7.f);
    p = fmaf(p, u, 1.f / 5.f);
    p = fmaf(p, u, 1.f / 3.f);
    p = fmaf(p, u, 1.f);
    return fmaxf(v, 0.f) + 2.f * s * p;
}

// Tensor-core path (csrc/scan_tc.cu): whether these arguments can take it, its
// segments, and the launches.
bool tc_supported(const ScanArgs& a, int B, la_dtype dt);
int tc_segments(int64_t B, int H, int G, int N, int P);
cudaError_t tc_scan(ScanArgs& a, int B, void* ws_header, cudaStream_t st);

// Launches a kernel, with `dependent` as a programmatic dependent of the one before
// it in the stream (it must call griddepcontrol.wait before it reads that one's results).
template <typename... P, typename... V>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                         bool dependent, V&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

int recurrence_segments(int64_t BH, int N, int S, int P);
cudaError_t launch_seeds(const ScanArgs& a, int64_t BH, cudaStream_t st);

}  // namespace scan
}  // namespace la
