// Causal linear attention whose state decays by a factor of its head per token:
//   S_t = e^{l_h} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
// ("Why Replace Attention? The Softmax Bottleneck and the Path to Linear Time",
// section 7.2, steps 1-4, with a decay of the state; features are the caller's and
// there is no denominator: a norm of the outputs takes its place).
//
// With o = F(q, k, v), F(a, b, c)_t = scale sum_{u <= t} e^{l (t - u)} (a_t . b_u) c_u,
// the gradients are sums of the same form:
//   dq = F(dout, v, k),  dk = F'(v, dout, q),  dv = F'(k, q, dout)
// with F' the sum over u >= t: so one kernel, run forwards or backwards in time, is
// the forward pass and its whole gradient, and no state is stored.
//
// This file: fp32 arithmetic on the CUDA cores for every type, width and stride, the
// single-token step, the chaining of segments and the entry points. bf16 with whole
// 16-byte rows runs on the tensor cores instead (csrc/decay_tc.cu).
//
// Chunks of 64 tokens in shared memory, 64 or 128 columns of c per block, 256 threads of
// 4 x 4 or 8 x 4 outputs each:
//   O = e^{l (i + 1)} A S;   P = weighted, masked A B^T (in A's place);   O += P C;
//   S = e^{64 l} S + B^T (w C)
// with S in registers between chunks. What bounds it: the operands' reads from shared
// memory, 128 bytes per cycle and SM whether lanes share them or not, so 3 reads of 16
// bytes for 32 multiply-adds (8 x 4) go further than 2 for 16; and two blocks per SM, which
// fill one another's waits (P in A's place and no transposed B leave the memory for them).
// Sequences are cut into segments when there are too few heads for the SMs: a first pass
// gives each segment's end state from zero, a chain over the segments their start states,
// and the second pass starts from those. fp32 B=2 N=4000 H=8 Dk=64 Dv=96: 135 us in all
// (64 columns of 4 x 4 per block, with as little shared memory to spare: 171, and 185 with
// one multiply-add per instruction).
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "decay.cuh"
#include "kernels.h"
#include "overlap.h"
#include "scan.cuh"
#include "tc_common.cuh"

namespace la {

using namespace decay;

namespace {

constexpr int kL = 64;              // tokens per chunk
constexpr int kRow = kL + 4;        // floats of a row of tokens in shared memory

// kD: 64-row tiles of the state; kC: columns per block. Tokens and widths past the end are
// zero.
template <int kD, int kC> struct Shared {
    float at[64 * kD * kRow];       // A^T, [d][token]; then P^T, [u][t]
    float sm[64 * kD * (kC + 4)];   // S, [d][column]
};
template <int kD, int kC> struct Common {
    float bn[kL * (64 * kD + 4)];   // B, [token][d] (first pass: w B)
    float cn[kL * (kC + 4)];        // C, [token][column]
    float pw[kL + 4];               // e^{l k}
};

// Four values of a row from value d on; past `width` they are zero.
template <typename T> __device__ __forceinline__ float4 load4(const T* p, int d, int width, bool vec) {
    if (vec) {
        if (d >= width) return make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (sizeof(T) == 4) {
            return __ldg(reinterpret_cast<const float4*>(p + d));
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + d));
            return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                               __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
        }
    }
    return make_float4(d < width ? to_f(p[d]) : 0.f, d + 1 < width ? to_f(p[d + 1]) : 0.f,
                       d + 2 < width ? to_f(p[d + 2]) : 0.f, d + 3 < width ? to_f(p[d + 3]) : 0.f);
}

// Whether every row of x can be read four values at a time.
template <typename T> __device__ __forceinline__ bool whole4(const T* x, const Tensor& t, int width) {
    return ((reinterpret_cast<uintptr_t>(x) | (uintptr_t)(t.ts * (int64_t)sizeof(T))) & (4 * sizeof(T) - 1)) == 0 && width % 4 == 0;
}

// A thread stages values 4 (lane / 8) + 16 i of token 8 warp + lane mod 8: whole 32-byte
// pieces of eight rows at a time, and stores of a transposed tile in two banks' reach.
__device__ __forceinline__ void put_transposed(float* dst, int d, int t, const float4& v) {
    dst[d * kRow + t] = v.x;
    dst[(d + 1) * kRow + t] = v.y;
    dst[(d + 2) * kRow + t] = v.z;
    dst[(d + 3) * kRow + t] = v.w;
}

// r += x y, two columns per instruction.
__device__ __forceinline__ void add_times(float (&r)[4], float x, const float (&y)[4]) {
    asm("{\n.reg .b64 x, y, z, u, v;\nmov.b64 x, {%4, %4};\nmov.b64 y, {%5, %6};\nmov.b64 z, {%7, %8};\n"
        "mov.b64 u, {%0, %1};\nmov.b64 v, {%2, %3};\n"
        "fma.rn.f32x2 u, x, y, u;\nfma.rn.f32x2 v, x, z, v;\n"
        "mov.b64 {%0, %1}, u;\nmov.b64 {%2, %3}, v;\n}"
        : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]) : "f"(x), "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]));
}

// acc += x (w y)^T from row `from` on.
template <int kI>
__device__ __forceinline__ void outer(float (&acc)[kI][4], const float* x, const float* y, float w = 1.f, int from = 0) {
    const float4 v = *reinterpret_cast<const float4*>(y);
    const float b[4] = {w * v.x, w * v.y, w * v.z, w * v.w};
#pragma unroll
    for (int i0 = 0; i0 < kI; i0 += 4) {
        if (i0 + 3 < from) continue;
        const float4 u = *reinterpret_cast<const float4*>(x + i0);
        const float a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i0 + i >= from) add_times(acc[i0 + i], a[i], b);
    }
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Grid: (segments, column blocks, B H). A thread owns kI rows (tokens, or rows of each of
// the state's tiles) by four columns, a warp 4 kI rows by 32 columns. kBlocks: blocks per
// SM that the registers leave room for. kState: only the segment's end state from zero
// (first pass, every segment but the last).
template <typename T, int kD, int kC, bool kState, int kBlocks>
__global__ void __launch_bounds__(256, kBlocks) decay_kernel(const __grid_constant__ Args a) {
    extern __shared__ float smem[];
    Common<kD, kC>& s = *reinterpret_cast<Common<kD, kC>*>(smem);
    Shared<kD, kC>& x = *reinterpret_cast<Shared<kD, kC>*>(smem + sizeof(Common<kD, kC>) / sizeof(float));
    constexpr int kB = 64 * kD + 4, kRowC = kC + 4, kI = kC / 16, kStripes = kC / 32;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tx = 8 * (warp % kStripes) + (lane & 7), ty = 4 * (warp / kStripes) + (lane >> 3);
    const int px = tid & 15, py = tid >> 4;     // the thread's 4 x 4 scores
    const int seg = blockIdx.x, col0 = kC * blockIdx.y;
    const int64_t bh = blockIdx.z, b = bh / a.H, h = bh - b * a.H;
    const int n = tokens_of(a, (int)b);
    const int t0 = min(seg * a.seg_len, n), t1 = min(t0 + a.seg_len, n);
    const int width = min(kC, a.Dc - col0);
    const bool working = 32 * (warp % kStripes) < width;
    const T* A = static_cast<const T*>(a.a.p) + b * a.a.bs + h * a.a.hs;
    const T* Bp = static_cast<const T*>(a.b.p) + b * a.b.bs + h * a.b.hs;
    const T* C = static_cast<const T*>(a.c.p) + b * a.c.bs + h * a.c.hs + col0;
    T* O = static_cast<T*>(const_cast<void*>(a.o.p)) + b * a.o.bs + h * a.o.hs + col0;
    const float l = a.decay[h], l2 = log2_decay(l);
    const int64_t state = (int64_t)a.Da * a.Dc;

    tcc::pdl_launch_dependents();
    tcc::pdl_wait();                    // the second pass follows the chaining kernel
    float st[kD][kI][4];                // rows 64 k + kI ty + i, columns col0 + 4 tx + j
    const float* from = kState ? nullptr : (a.nseg > 1 ? a.seeds + (bh * a.nseg + seg) * state
                                                       : (a.S0 ? a.S0 + bh * state : nullptr));
#pragma unroll
    for (int k = 0; k < kD; ++k)
#pragma unroll
        for (int i = 0; i < kI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 64 * k + kI * ty + i, c = 4 * tx + j;
                st[k][i][j] = from && r < a.Da && c < width ? from[(int64_t)r * a.Dc + col0 + c] : 0.f;
            }
    if (tid <= kL) s.pw[tid] = pow2(tid * l2);
    const int d4 = (a.Da + 3) & ~3;
    const int tok = 8 * (tid >> 5) + (tid & 7), q4 = 4 * ((tid & 31) >> 3);   // staged by this thread
    const bool vec_a = whole4(A, a.a, a.Da), vec_b = whole4(Bp, a.b, a.Da), vec_c = whole4(C, a.c, width);
    __syncthreads();
    for (int c0 = t0; c0 < t1; c0 += kL) {
        const int m = min(kL, t1 - c0);
        // Tokens count from the last one where time is reversed.
        auto token = [&](int i) { return (int64_t)(a.rev ? n - 1 - c0 - i : c0 + i); };
        const int64_t at = token(tok);
        const bool in = tok < m;
        const float weight = in && kState ? s.pw[m - 1 - tok] : 0.f;
        __syncthreads();
#pragma unroll
        for (int d = q4; d < 64 * kD; d += 16) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) v = load4(Bp + at * a.b.ts, d, a.Da, vec_b);
            if constexpr (!kState) {
                float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
                if (in) u = load4(A + at * a.a.ts, d, a.Da, vec_a);
                put_transposed(x.at, d, tok, u);
            }
            if constexpr (kState) v = make_float4(weight * v.x, weight * v.y, weight * v.z, weight * v.w);
            *reinterpret_cast<float4*>(s.bn + tok * kB + d) = v;
        }
#pragma unroll
        for (int d = q4; d < kC; d += 16) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) v = load4(C + at * a.c.ts, d, width, vec_c);
            *reinterpret_cast<float4*>(s.cn + tok * kRowC + d) = v;
        }
        // The next chunk's rows on their way to L2, 128 bytes per thread and tensor (2 to 7 %).
        if (kL + tok < t1 - c0) {
            const int64_t next = token(kL + tok);
            const int d = 8 * q4;
            if (d < a.Da) {
                prefetch_l2(Bp + next * a.b.ts + d);
                if constexpr (!kState) prefetch_l2(A + next * a.a.ts + d);
            }
            if (d < width) prefetch_l2(C + next * a.c.ts + d);
        }
        if constexpr (!kState)
#pragma unroll
            for (int k = 0; k < kD; ++k)
#pragma unroll
                for (int i = 0; i < kI; ++i)
                    *reinterpret_cast<float4*>(x.sm + (64 * k + kI * ty + i) * kRowC + 4 * tx) =
                        make_float4(st[k][i][0], st[k][i][1], st[k][i][2], st[k][i][3]);
        __syncthreads();
        if constexpr (!kState) {
            float o[kI][4] = {}, p[4][4] = {};      // p: tokens u = px + 16 j by t = 4 py + i
            if (working) {
#pragma unroll 4
                for (int d = 0; d < d4; ++d) outer(o, x.at + d * kRow + kI * ty, x.sm + d * kRowC + 4 * tx);
#pragma unroll
                for (int i = 0; i < kI; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= s.pw[kI * ty + i + 1];
            }
            const int last_t = 8 * warp + 7;        // of the warp's scores
            for (int d = 0; d < d4; d += 4) {
                float av[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 v = *reinterpret_cast<const float4*>(x.at + (d + e) * kRow + 4 * py);
                    av[e][0] = v.x, av[e][1] = v.y, av[e][2] = v.z, av[e][3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (16 * j > last_t) break;     // every token is masked
                    const float4 v = *reinterpret_cast<const float4*>(s.bn + (px + 16 * j) * kB + d);
                    add_times(p[j], v.x, av[0]);
                    add_times(p[j], v.y, av[1]);
                    add_times(p[j], v.z, av[2]);
                    add_times(p[j], v.w, av[3]);
                }
            }
            __syncthreads();                        // A has been read
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int u = px + 16 * j;
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int gap = 4 * py + i - u;
                    v[i] = gap >= 0 ? p[j][i] * s.pw[max(gap, 0)] : 0.f;
                }
                if (16 * j <= last_t) *reinterpret_cast<float4*>(x.at + u * kRow + 4 * py) = make_float4(v[0], v[1], v[2], v[3]);
            }
            __syncthreads();
            if (working) {
                // Tokens after a row's own take no part, not even as zeros: an infinity or NaN
                // reaches no earlier token.
#pragma unroll 4
                for (int u = 0; u < kI * ty; ++u) outer(o, x.at + u * kRow + kI * ty, s.cn + u * kRowC + 4 * tx);
#pragma unroll
                for (int u = 0; u < kI; ++u)
                    outer(o, x.at + (kI * ty + u) * kRow + kI * ty, s.cn + (kI * ty + u) * kRowC + 4 * tx, 1.f, u);
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                    T* to = O + token(kI * ty + i) * a.o.ts + 4 * tx;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (kI * ty + i < m && 4 * tx + j < width) to[j] = from_f<T>(a.scale * o[i][j]);
                }
            }
        }
        const Factor f = factor(m * log_decay(l));
#pragma unroll
        for (int k = 0; k < kD; ++k) {
            if (64 * k >= a.Da || !working) break;
            float add[kI][4] = {};
#pragma unroll 4
            for (int u = 0; u < m; ++u) outer(add, s.bn + u * kB + 64 * k + kI * ty, s.cn + u * kRowC + 4 * tx, kState ? 1.f : s.pw[m - 1 - u]);
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) st[k][i][j] = fmaf(f.hi, st[k][i][j], fmaf(f.lo, st[k][i][j], add[i][j]));
        }
    }
    float* to = kState ? a.seeds + (bh * a.nseg + seg) * state
                       : (seg == a.nseg - 1 && a.S_out ? a.S_out + bh * state : nullptr);
    if (to)
#pragma unroll
        for (int k = 0; k < kD; ++k)
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = 64 * k + kI * ty + i, c = 4 * tx + j;
                    if (r < a.Da && c < width) to[(int64_t)r * a.Dc + col0 + c] = st[k][i][j];
                }
}

// In place over a head's segments: the end states (from zero) become the states that the
// segments start from, seed_0 = S0, seed_{i+1} = e^{l tokens_i} seed_i + end_i. A thread
// chains one element, eight segments in flight.
constexpr int kMaxSegments = 64;
__global__ void __launch_bounds__(128)
chain_kernel(const __grid_constant__ Args first, const __grid_constant__ Args second, int chunk) {
    const Args& a = blockIdx.z ? second : first;
    __shared__ Factor f[kMaxSegments];
    __shared__ int empty[kMaxSegments];
    const int64_t bh = blockIdx.y, b = bh / a.H, h = bh - b * a.H;
    tcc::pdl_launch_dependents();
    tcc::pdl_wait();
    if (threadIdx.x < a.nseg) {
        int n = tokens_of(a, (int)b);
        if (a.rev) n = (n + chunk - 1) / chunk * chunk;
        const int m = seg_tokens(a, n, threadIdx.x);
        f[threadIdx.x] = factor(m * log_decay(a.decay[h]));
        empty[threadIdx.x] = m == 0;
    }
    __syncthreads();
    const int e = blockIdx.x * 128 + threadIdx.x, E = a.Da * a.Dc;
    if (e >= E) return;
    float carry = a.S0 ? a.S0[bh * E + e] : 0.f;
    float* p = a.seeds + bh * a.nseg * E + e;
    for (int i0 = 0; i0 < a.nseg; i0 += 8) {
        float end[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i0 + u < a.nseg - 1 && !empty[i0 + u]) end[u] = p[(int64_t)(i0 + u) * E];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int i = i0 + u;
            if (i >= a.nseg) break;
            p[(int64_t)i * E] = carry;
            if (i < a.nseg - 1 && !empty[i]) carry = fmaf(f[i].hi, carry, fmaf(f[i].lo, carry, end[u]));
        }
    }
}

struct StepArgs {
    const void *q, *k, *v;
    void* o;
    int64_t q_bs, q_hs, k_bs, k_hs, v_bs, v_hs, o_bs, o_hs;
    const float* decay;
    float* S;                   // [B, H, Dk, Dv]
    int H, Dk, Dv;
    float scale;
};

// One token per sequence, the state updated in place. It is read and written once (8
// bytes per element against five operations): HBM bandwidth bounds it. A block owns one
// head; a thread owns kV columns of every rows-per-pass-th row and keeps kU rows in flight.
// B=64 H=32 Dk=Dv=128 bf16: 42 us for the state's 268 MB, 0.97 of a copy's rate.
template <typename T, int kV>
__global__ void __launch_bounds__(256) decay_step_kernel(const __grid_constant__ StepArgs a) {
    constexpr int kU = 8;
    __shared__ float ks[kMaxDim], qs[kMaxDim];
    __shared__ float red[256 * kV];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x, b = bh / a.H, h = bh - b * a.H;
    const int lpr = (a.Dv + kV - 1) / kV, rpp = 256 / lpr;   // lanes per row, rows per pass
    const int r0 = tid / lpr, c0 = (tid - r0 * lpr) * kV;
    const bool mine = r0 < rpp;
    float* S = a.S + bh * a.Dk * a.Dv + c0;
    float s[kU][kV];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = base + u * rpp + r0;
            if (!mine || r >= a.Dk) continue;
            if constexpr (kV == 4) {
                const float4 v = *reinterpret_cast<const float4*>(S + (int64_t)r * a.Dv);
                s[u][0] = v.x, s[u][1] = v.y, s[u][2] = v.z, s[u][3] = v.w;
            } else {
                s[u][0] = S[(int64_t)r * a.Dv];
            }
        }
    };
    load(0);
    if (tid < a.Dk) {
        qs[tid] = to_f(static_cast<const T*>(a.q)[b * a.q_bs + h * a.q_hs + tid]);
        ks[tid] = to_f(static_cast<const T*>(a.k)[b * a.k_bs + h * a.k_hs + tid]);
    }
    const T* vp = static_cast<const T*>(a.v) + b * a.v_bs + h * a.v_hs;
    float vv[kV], acc[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) vv[v] = mine ? to_f(vp[c0 + v]) : 0.f, acc[v] = 0.f;
    const Factor f = factor(log_decay(a.decay[h]));   // a state passes it once per token
    __syncthreads();
    for (int base = 0; base < a.Dk; base += kU * rpp) {
        if (base > 0) load(base);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = base + u * rpp + r0;
            if (!mine || r >= a.Dk) continue;
            const float kr = ks[r], qr = qs[r];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                s[u][v] = fmaf(f.hi, s[u][v], fmaf(f.lo, s[u][v], kr * vv[v]));
                acc[v] = fmaf(qr, s[u][v], acc[v]);
            }
            if constexpr (kV == 4)
                *reinterpret_cast<float4*>(S + (int64_t)r * a.Dv) = make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
            else
                S[(int64_t)r * a.Dv] = s[u][0];
        }
    }
    if (mine)
#pragma unroll
        for (int v = 0; v < kV; ++v) red[r0 * a.Dv + c0 + v] = acc[v];
    __syncthreads();
    if (tid < a.Dv) {
        float v = 0.f;
        for (int r = 0; r < rpp; ++r) v += red[r * a.Dv + tid];
        static_cast<T*>(a.o)[b * a.o_bs + h * a.o_hs + tid] = from_f<T>(a.scale * v);
    }
}

template <typename T, int kD, int kC>
cudaError_t run_width(const Args& a, cudaStream_t st) {
    static std::atomic<int> optin[3][tcc::kMaxDevices];
    constexpr int kSums = sizeof(Common<kD, kC>), kMain = kSums + sizeof(Shared<kD, kC>);
    const unsigned BH = (unsigned)(a.B * a.H), blocks = (a.Dc + kC - 1) / kC;
    cudaError_t e;
    if (a.nseg > 1) {
        if ((e = tcc::ensure_smem_optin(decay_kernel<T, kD, kC, true, 2>, kSums, optin[0])) != cudaSuccess) return e;
        decay_kernel<T, kD, kC, true, 2><<<dim3(a.nseg - 1, blocks, BH), 256, kSums, st>>>(a);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        if ((e = launch_chain(&a, 1, 1, st)) != cudaSuccess) return e;
    }
    auto main_pass = [&](auto kernel, std::atomic<int>* in) {
        e = tcc::ensure_smem_optin(kernel, kMain, in);
        return e != cudaSuccess ? e : scan::launch_after(kernel, dim3(a.nseg, blocks, BH), 256, kMain, st, a.nseg > 1, a);
    };
    // Two blocks per SM leave a thread 128 registers: fp32 N=4000 Dk=64 Dv=96, 16 heads 135 us
    // against 193 with one. With no second block to share the SM, more registers hold more
    // loads in flight: two heads 81 us against 105.
    if constexpr (kD == 1) {
        if ((int64_t)a.nseg * blocks * BH > tcc::sm_count()) return main_pass(decay_kernel<T, kD, kC, false, 2>, optin[1]);
    }
    return main_pass(decay_kernel<T, kD, kC, false, 1>, optin[2]);
}

// Columns per block.
int columns(int Dc) { return Dc <= 64 ? 64 : 128; }

template <typename T>
cudaError_t run_simt(const Args& a, cudaStream_t st) {
    if (columns(a.Dc) == 64) return a.Da <= 64 ? run_width<T, 1, 64>(a, st) : run_width<T, 2, 64>(a, st);
    return a.Da <= 64 ? run_width<T, 1, 128>(a, st) : run_width<T, 2, 128>(a, st);
}

// Segments of the CUDA-core path: one while there are blocks for every SM or fewer than four
// chunks.
int simt_segments(int64_t BH, int N, int Da, int Dc) {
    const int64_t blocks = BH * ((Dc + columns(Dc) - 1) / columns(Dc));
    const int64_t slots = (int64_t)tcc::sm_count() * (Da <= 64 ? 2 : 1);
    const int64_t most = (N + kL - 1) / kL / 2;
    int64_t n = blocks > 0 ? slots / blocks : 1;
    n = n < most ? n : most;
    n = n < kMaxSegments ? n : kMaxSegments;
    return n < 2 ? 1 : (int)n;
}

size_t simt_seeds(int64_t BH, int N, int Da, int Dc) {
    const int n = simt_segments(BH, N, Da, Dc);
    return n > 1 ? (size_t)BH * n * Da * Dc : 0;
}

float* seeds_of(void* workspace) { return reinterpret_cast<float*>(static_cast<char*>(workspace) + sizeof(WsHeader)); }

cudaError_t run_cuda_cores(Args a, la_dtype dt, void* workspace, cudaStream_t st) {
    cut(&a, simt_segments((int64_t)a.B * a.H, a.N, a.Da, a.Dc), kL);
    a.seeds = seeds_of(workspace);
    return dt == LA_BF16 ? run_simt<__nv_bfloat16>(a, st) : run_simt<float>(a, st);
}

constexpr int64_t kPromptHeads = 65535, kStepHeads = 2147483647;   // grid axes
la_status check_shape(int B, int H, int N, int Dk, int Dv, la_dtype dt, float scale, int64_t most_heads) {
    if (B < 0 || H < 0 || N < 0 || Dk < 1 || Dv < 1) return LA_ERR_INVALID_ARG;
    if ((dt != LA_F32 && dt != LA_BF16) || !isfinite(scale)) return LA_ERR_INVALID_ARG;
    if (Dk > kMaxDim || Dv > kMaxDim) return LA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > most_heads || N > kScanMaxTokens) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

bool bad(const void* p, la_dtype dt) {
    return !p || (reinterpret_cast<uintptr_t>(p) & (dt == LA_BF16 ? 1 : 3));
}
bool bad4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3; }

// Rows [B, H, N, D], and a whole range, as the overlap checks take them.
Rows3 rows3(const void* p, int64_t B, int64_t H, int64_t N, int64_t D, const int64_t* s, int64_t eb) {
    return {p, D * eb, {B, H, N}, {s[0] * eb, s[1] * eb, s[2] * eb}};
}
Rows3 whole(const void* p, int64_t bytes) { return {p, bytes, {1, 1, 1}, {0, 0, 0}}; }

// Whether an output's rows are disjoint: each axis steps over all that the axes with smaller
// strides cover.
bool disjoint(int64_t B, int64_t H, int64_t N, int64_t D, const int64_t* s) {
    int64_t size[3] = {B, H, N}, stride[3] = {s[0], s[1], s[2]}, reach = D;
    for (int k = 0; k < 3; ++k) {
        int best = -1;
        for (int i = 0; i < 3; ++i)
            if (size[i] > 1 && (best < 0 || stride[i] < stride[best])) best = i;
        if (best < 0) return true;
        if (stride[best] < reach) return false;
        reach += (size[best] - 1) * stride[best];
        size[best] = 1;
    }
    return true;
}

Tensor tensor(const void* p, const int64_t* s) { return {p, s[0], s[1], s[2]}; }

}  // namespace

namespace decay {

cudaError_t launch_chain(const Args* a, int count, int chunk, cudaStream_t st) {
    return scan::launch_after(chain_kernel, dim3((a->Da * a->Dc + 127) / 128, (unsigned)(a->B * a->H), count), 128, 0, st,
                              true, a[0], a[count - 1], chunk);
}

}  // namespace decay

// Enough for either path: rows that are not aligned take the CUDA cores.
size_t decay_workspace(int B, int H, int N, int Dk, int Dv, la_dtype dt, bool backward) {
    const int64_t BH = (int64_t)B * H;
    size_t most = simt_seeds(BH, N, Dk, Dv);
    if (backward) most = std::max(most, simt_seeds(BH, N, Dv, Dk));
    if (dt == LA_BF16 && Dk % 8 == 0 && Dv % 8 == 0) most = std::max(most, tc_seeds(BH, N, Dk, Dv, backward));
    return most * sizeof(float);
}

int decay_launches(int B, int H, int N, int Dk, int Dv, la_dtype dt, bool backward) {
    const int64_t BH = (int64_t)B * H;
    if (dt == LA_BF16 && Dk % 8 == 0 && Dv % 8 == 0) return tc_launches(BH, N, Dk, Dv, backward);
    auto one = [&](int Da, int Dc) { return simt_segments(BH, N, Da, Dc) > 1 ? 3 : 1; };
    return backward ? 2 * one(Dv, Dk) + one(Dk, Dv) : one(Dk, Dv);
}

}  // namespace la

extern "C" {

la_status la_decay_attn_fwd(const void* q, const void* k, const void* v, const float* decay, float scale,
                            const int32_t* lengths, const float* S0, float* S_out, void* o,
                            const int64_t* strides, int B, int H, int N, int Dk, int Dv, la_dtype dt,
                            void* workspace, size_t workspace_bytes, la_stream_t stream) {
    la_status s = la::check_shape(B, H, N, Dk, Dv, dt, scale, la::kPromptHeads);
    if (s != LA_OK) return s;
    const int64_t BH = (int64_t)B * H;
    if (BH == 0) return LA_OK;
    if (!decay || la::bad4(decay) || la::bad4(lengths) || la::bad4(S0) || la::bad4(S_out)) return LA_ERR_INVALID_ARG;
    const size_t state = sizeof(float) * (size_t)BH * Dk * Dv;
    const la::Rows s0 = la::block_of(S0, state), s1 = la::block_of(S_out, state);
    if (S0 != S_out && la::overlap(s0, s1)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0) {
        if (!S_out || S_out == S0) return LA_OK;
        const cudaError_t e = S0 ? cudaMemcpyAsync(S_out, S0, state, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(S_out, 0, state, st);
        return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    if (la::bad(q, dt) || la::bad(k, dt) || la::bad(v, dt) || la::bad(o, dt) || !strides) return LA_ERR_INVALID_ARG;
    if (!la::disjoint(B, H, N, Dv, strides + 9)) return LA_ERR_INVALID_ARG;
    const size_t need = sizeof(la::WsHeader) + la::decay_workspace(B, H, N, Dk, Dv, dt, false);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return LA_ERR_WORKSPACE;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const la::Rows3 qr = la::rows3(q, B, H, N, Dk, strides, eb), kr = la::rows3(k, B, H, N, Dk, strides + 3, eb);
    const la::Rows3 vr = la::rows3(v, B, H, N, Dv, strides + 6, eb), orr = la::rows3(o, B, H, N, Dv, strides + 9, eb);
    const la::Rows3 dr = la::whole(decay, 4 * (int64_t)H), nr = la::whole(lengths, 4 * (int64_t)B);
    const la::Rows3 s0r = la::whole(S0, state), s1r = la::whole(S_out, state), wr = la::whole(workspace, need);
    if (la::overlaps_any(orr, {qr, kr, vr, dr, nr, s0r, s1r, wr}) || la::overlaps_any(s1r, {qr, kr, vr, dr, nr, wr}) ||
        la::overlaps_any(wr, {qr, kr, vr, dr, nr, s0r}))
        return LA_ERR_INVALID_ARG;
    la::decay::Args a = {};
    a.a = la::tensor(q, strides), a.b = la::tensor(k, strides + 3), a.c = la::tensor(v, strides + 6);
    a.o = la::tensor(o, strides + 9);
    a.decay = decay, a.lengths = lengths, a.S0 = S0, a.S_out = S_out;
    a.B = B, a.H = H, a.N = N, a.Da = Dk, a.Dc = Dv, a.scale = scale;
    if (la::tc_supported(a, dt)) {
        a.seeds = la::seeds_of(workspace);
        return la::tc_run(a, workspace, st) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    return la::run_cuda_cores(a, dt, workspace, st) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_decay_attn_bwd(const void* q, const void* k, const void* v, const void* dout, const float* decay,
                            float scale, const int32_t* lengths, void* dq, void* dk, void* dv,
                            const int64_t* strides, int B, int H, int N, int Dk, int Dv, la_dtype dt,
                            void* workspace, size_t workspace_bytes, la_stream_t stream) {
    la_status s = la::check_shape(B, H, N, Dk, Dv, dt, scale, la::kPromptHeads);
    if (s != LA_OK) return s;
    if (B == 0 || H == 0 || N == 0) return LA_OK;
    if (!decay || la::bad4(decay) || la::bad4(lengths) || !strides) return LA_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, dout, (const void*)dq, (const void*)dk, (const void*)dv})
        if (la::bad(p, dt)) return LA_ERR_INVALID_ARG;
    const int64_t *sq = strides, *sk = strides + 3, *sv = strides + 6, *sg = strides + 9;
    const int64_t *tq = strides + 12, *tk = strides + 15, *tv = strides + 18;
    if (!la::disjoint(B, H, N, Dk, tq) || !la::disjoint(B, H, N, Dk, tk) || !la::disjoint(B, H, N, Dv, tv))
        return LA_ERR_INVALID_ARG;
    const size_t need = sizeof(la::WsHeader) + la::decay_workspace(B, H, N, Dk, Dv, dt, true);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need) return LA_ERR_WORKSPACE;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const la::Rows3 qr = la::rows3(q, B, H, N, Dk, sq, eb), kr = la::rows3(k, B, H, N, Dk, sk, eb);
    const la::Rows3 vr = la::rows3(v, B, H, N, Dv, sv, eb), gr = la::rows3(dout, B, H, N, Dv, sg, eb);
    const la::Rows3 dr = la::whole(decay, 4 * (int64_t)H), nr = la::whole(lengths, 4 * (int64_t)B);
    const la::Rows3 wr = la::whole(workspace, need);
    const la::Rows3 oq = la::rows3(dq, B, H, N, Dk, tq, eb), ok = la::rows3(dk, B, H, N, Dk, tk, eb);
    const la::Rows3 ov = la::rows3(dv, B, H, N, Dv, tv, eb);
    for (const la::Rows3* out : {&oq, &ok, &ov, &wr})
        if (la::overlaps_any(*out, {qr, kr, vr, gr, dr, nr})) return LA_ERR_INVALID_ARG;
    if (la::overlap(oq, ok) || la::overlap(oq, ov) || la::overlap(ok, ov) || la::overlaps_any(wr, {oq, ok, ov}))
        return LA_ERR_INVALID_ARG;
    la::decay::Args a = {};
    a.decay = decay, a.lengths = lengths, a.B = B, a.H = H, a.N = N, a.scale = scale;
    const la::decay::Tensor Q = la::tensor(q, sq), K = la::tensor(k, sk), V = la::tensor(v, sv), G = la::tensor(dout, sg);
    la::decay::Args dqs = a, dks = a, dvs = a;
    dqs.a = G, dqs.b = V, dqs.c = K, dqs.o = la::tensor(dq, tq), dqs.Da = Dv, dqs.Dc = Dk;
    dks.a = V, dks.b = G, dks.c = Q, dks.o = la::tensor(dk, tk), dks.Da = Dv, dks.Dc = Dk, dks.rev = 1;
    dvs.a = K, dvs.b = Q, dvs.c = G, dvs.o = la::tensor(dv, tv), dvs.Da = Dk, dvs.Dc = Dv, dvs.rev = 1;
    cudaStream_t st = (cudaStream_t)stream;
    if (la::tc_supported(dqs, dt) && la::tc_supported(dks, dt) && la::tc_supported(dvs, dt)) {
        dqs.seeds = la::seeds_of(workspace);
        return la::tc_backward(dqs, dks, dvs, workspace, st) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    for (const la::decay::Args* sum : {&dqs, &dks, &dvs})
        if (la::run_cuda_cores(*sum, dt, workspace, st) != cudaSuccess) return LA_ERR_CUDA;
    return LA_OK;
}

la_status la_decay_attn_step(const void* q, const void* k, const void* v, const float* decay, float scale,
                             float* S_inout, void* o, const int64_t* strides, int B, int H, int Dk, int Dv,
                             la_dtype dt, la_stream_t stream) {
    la_status s = la::check_shape(B, H, 1, Dk, Dv, dt, scale, la::kStepHeads);
    if (s != LA_OK) return s;
    const int64_t BH = (int64_t)B * H;
    if (BH == 0) return LA_OK;
    if (la::bad(q, dt) || la::bad(k, dt) || la::bad(v, dt) || la::bad(o, dt) || !decay || la::bad4(decay) || !strides ||
        !S_inout || (reinterpret_cast<uintptr_t>(S_inout) & (Dv % 4 ? 3 : 15)))   // 16-byte accesses of four columns
        return LA_ERR_INVALID_ARG;
    const int64_t *sq = strides, *sk = strides + 2, *sv = strides + 4, *so = strides + 6;
    const int64_t no[3] = {so[0], so[1], 0};
    if (!la::disjoint(B, H, 1, Dv, no)) return LA_ERR_INVALID_ARG;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    auto rows = [&](const void* p, int D, const int64_t* t) { return la::Rows{p, B, H, D * eb, t[0] * eb, t[1] * eb}; };
    const la::Rows qr = rows(q, Dk, sq), kr = rows(k, Dk, sk), vr = rows(v, Dv, sv), outr = rows(o, Dv, so);
    const la::Rows dr = la::block_of(decay, 4 * (int64_t)H);
    const la::Rows sr = la::block_of(S_inout, (int64_t)(sizeof(float) * (size_t)BH * Dk * Dv));
    // o may be q, k or v itself (the same rows): a block reads what it replaces.
    for (const la::Rows* r : {&qr, &kr, &vr})
        if (!la::same_rows(*r, outr) && la::overlap(*r, outr)) return LA_ERR_INVALID_ARG;
    if (la::overlap(outr, dr) || la::overlaps_any(sr, {qr, kr, vr, outr, dr})) return LA_ERR_INVALID_ARG;
    const la::StepArgs a = {q, k, v, o, sq[0], sq[1], sk[0], sk[1], sv[0], sv[1], so[0], so[1], decay, S_inout, H, Dk, Dv, scale};
    cudaStream_t st = (cudaStream_t)stream;
    const unsigned blocks = (unsigned)BH;
    if (dt == LA_BF16) {
        if (Dv % 4 == 0) la::decay_step_kernel<__nv_bfloat16, 4><<<blocks, 256, 0, st>>>(a);
        else la::decay_step_kernel<__nv_bfloat16, 1><<<blocks, 256, 0, st>>>(a);
    } else {
        if (Dv % 4 == 0) la::decay_step_kernel<float, 4><<<blocks, 256, 0, st>>>(a);
        else la::decay_step_kernel<float, 1><<<blocks, 256, 0, st>>>(a);
    }
    return cudaPeekAtLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
