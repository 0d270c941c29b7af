// Shared by the files of linear attention with a decay per head: the arguments of
// its kernels and the decay's factors.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "linattn.h"

namespace la {
namespace decay {

// Rows at p + b bs + h hs + n ts (elements), values adjacent.
struct Tensor {
    const void* p;
    int64_t bs, hs, ts;
};

// One sum over tokens, per head with l = decay[h]:
//   o_t = scale sum_{u <= t} e^{l (t - u)} (a_t . b_u) c_u  + scale e^{l (t + 1)} a_t^T S0
// (rev: over u >= t, e^{l (u - t)}, without states). a, b [B, H, N, Da]; c, o [B, H, N, Dc].
// The forward pass is (q, k, v); the gradients are (dout, v, k), reversed (v, dout, q) and
// reversed (k, q, dout).
struct Args {
    Tensor a, b, c, o;
    const float* decay;         // [H], the logarithm of the factor per token
    const int32_t* lengths;     // [B] or null
    const float* S0;            // [B, H, Da, Dc] or null
    float* S_out;               // the same or null
    float* seeds;               // [B H, nseg, Da, Dc]: the segments' end states from zero; chained: their start states
    int B, H, N, Da, Dc, rev;
    int nseg, seg_len;          // segments and their tokens (a multiple of the chunk)
    int fold;                   // the main pass joins the end states before its segment itself: they are not chained
    int seeds_t;                // seeds are [.., Dc, Da]: those of the sum with b and c exchanged
    float scale;
};

// e^x as a value and what its rounding leaves of it, for factors that a state passes many
// times: near 1 the rounding of the factor itself (2^-25) would add up over the passes.
struct Factor {
    float hi, lo;
};
__device__ __forceinline__ Factor factor(float x) {
    if (x > -0.1f && x < 0.1f) {
        const float e = expm1f(x), hi = 1.f + e;
        return {hi, e - (hi - 1.f)};
    }
    return {expf(x), 0.f};
}

// The head's decay as a power of two per token. Held within -400, where one token's factor
// is 0 in fp32 already, so that 0 times it is 0 and not NaN (a factor of exactly 0 has the
// logarithm minus infinity). A comparison, so that NaN stays NaN.
__device__ __forceinline__ float log2_decay(float l) {
    const float v = l * 1.4426950408889634f;
    return v < -400.f ? -400.f : v;
}
__device__ __forceinline__ float log_decay(float l) { return l < -277.f ? -277.f : l; }

__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ int tokens_of(const Args& a, int b) {
    return a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
}

// Chains the segments' end states of one or two sums into their start states, in place
// (csrc/decay.cu). chunk: the tensor-core path's states of reversed sums stand at whole chunks.
cudaError_t launch_chain(const Args* sums, int count, int chunk, cudaStream_t st);

// The cut of a sequence into `nseg` segments or fewer of whole chunks.
inline void cut(Args* a, int nseg, int chunk) {
    const int chunks = (a->N + chunk - 1) / chunk, per = (chunks + nseg - 1) / nseg;
    a->nseg = (chunks + per - 1) / per;
    a->seg_len = per * chunk;
}

// Tokens of segment i of a sequence that ends after n.
__device__ __forceinline__ int seg_tokens(const Args& a, int n, int i) {
    return min(max(n - i * a.seg_len, 0), a.seg_len);
}

// Tensor-core path (csrc/decay_tc.cu): whether a sum can take it; one sum; the three sums of
// the backward pass, dq, dk, dv in this order, and the floats of seeds of either.
bool tc_supported(const Args& a, la_dtype dt);
size_t tc_seeds(int64_t BH, int N, int Dk, int Dv, bool backward);
int tc_launches(int64_t BH, int N, int Dk, int Dv, bool backward);
cudaError_t tc_run(Args a, void* ws_header, cudaStream_t st);
cudaError_t tc_backward(Args dq, Args dk, Args dv, void* ws_header, cudaStream_t st);

}  // namespace decay
}  // namespace la
