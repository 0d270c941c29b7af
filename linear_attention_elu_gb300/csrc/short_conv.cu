// Short causal depthwise convolution over tokens, per channel c:
//   y_t = act(bias_c + sum_{k < W} w[c, k] x[t - W + 1 + k, c]),  act = identity or silu,
// for prompts (x [B, N, C], inputs before the first token from a state of W - 1
// rows) and for single tokens (the state shifted in place).
//
// What bounds it: each value is read once and written once, W multiply-adds and
// one silu each: HBM bandwidth (76 % of the copy rate at B=4 N=4096 C=4352), with the
// issue slots behind it (59 % used, a third of the instructions the silus'; 86 % of the
// copy rate without them). A thread owns one 16-byte
// piece of a row (8 bf16 or 4 fp32 channels) and walks consecutive tokens with the
// last W - 1 rows in registers, so a row is read again only by the neighbouring
// thread of the next token group (W - 1 rows in 64 at best, from L2). Channels that are not
// whole 16-byte pieces, or rows that are not aligned, take one channel per thread.
// Sums are fp32.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"
#include "mixing.cuh"
#include "overlap.h"
#include "tc_common.cuh"

namespace la {

namespace {

constexpr int kThreads = 256;

struct ConvArgs {
    const void* x;
    int64_t x_bs, x_ts;
    const void* w;
    const void* bias;
    const void* s0;          // [B, W - 1, C] or null
    void* s1;                // [B, W - 1, C] or null
    void* y;
    int64_t y_bs, y_ts;
    const int32_t* lengths;  // [B] or null
    int B, N, C, groups, tok, silu;
};

// kV consecutive values at p as floats.
template <typename T, int kV>
__device__ __forceinline__ void load_v(const T* p, float (&f)[kV]) {
    if constexpr (kV == 1) {
        f[0] = to_f(*p);
    } else if constexpr (sizeof(T) == 4) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
}

template <typename T, int kV>
__device__ __forceinline__ void store_v(T* p, const float (&f)[kV]) {
    if constexpr (kV == 1) {
        *p = from_f<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(tcc::pack_bf16(f[0], f[1]), tcc::pack_bf16(f[2], f[3]),
                       tcc::pack_bf16(f[4], f[5]), tcc::pack_bf16(f[6], f[7]));
    }
}

// Weights of kV channels from c0: kV W consecutive values (W 16-byte pieces).
template <typename T, int kV, int kW>
__device__ __forceinline__ void load_weights(const T* w, int c0, float (&f)[kW][kV]) {
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        float v[kV];
        load_v<T, kV>(w + (int64_t)c0 * kW + i * kV, v);
#pragma unroll
        for (int j = 0; j < kV; ++j) f[(i * kV + j) % kW][(i * kV + j) / kW] = v[j];
    }
}

template <typename T, int kV, int kW>
__device__ __forceinline__ void emit(const float (&w)[kW][kV], const float (&bias)[kV],
                                     const float (&win)[kW - 1][kV], const float (&x)[kV], int act,
                                     T* out) {
    float y[kV];
#pragma unroll
    for (int j = 0; j < kV; ++j) {
        float v = bias[j];
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) v = fmaf(w[k][j], win[k][j], v);
        v = fmaf(w[kW - 1][j], x[j], v);
        y[j] = act ? silu(v) : v;
    }
    store_v<T, kV>(out, y);
}

// Input row t of sequence b, or row t + W - 1 of the state before the first token.
template <typename T, int kV, int kW>
__device__ __forceinline__ void input_row(const ConvArgs& a, const T* x, int b, int c0, int t, float (&f)[kV]) {
    if (t >= 0) {
        load_v<T, kV>(x + t * a.x_ts, f);
    } else if (a.s0) {
        load_v<T, kV>(static_cast<const T*>(a.s0) + ((int64_t)b * (kW - 1) + t + kW - 1) * a.C + c0, f);
    } else {
#pragma unroll
        for (int j = 0; j < kV; ++j) f[j] = 0.f;
    }
}

// The last W - 1 of n rows (and of the state before them) to the state after.
template <typename T, int kV, int kW>
__device__ __forceinline__ void write_state(const ConvArgs& a, const T* x, int b, int c0, int n) {
    T* s1 = static_cast<T*>(a.s1) + (int64_t)b * (kW - 1) * a.C + c0;
#pragma unroll
    for (int k = 0; k < kW - 1; ++k) {
        float f[kV];
        input_row<T, kV, kW>(a, x, b, c0, n - (kW - 1) + k, f);
        store_v<T, kV>(s1 + (int64_t)k * a.C, f);
    }
}

// Any channel count and alignment: one channel per thread.
template <typename T, int kW>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const __grid_constant__ ConvArgs a) {
    constexpr int kAhead = 4;                              // rows in flight
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t bg = id / a.C;
    const int c0 = (int)(id - bg * a.C);
    const int b = (int)(bg / a.groups), g = (int)(bg - (int64_t)b * a.groups);
    if (b >= a.B) return;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c0;
    if (g == 0 && a.s1) write_state<T, 1, kW>(a, x, b, c0, n);
    const int t0 = g * a.tok, t1 = min(t0 + a.tok, n);
    if (t0 >= t1) return;
    float w[kW][1], bias[1] = {}, win[kW - 1][1];
    load_weights<T, 1, kW>(static_cast<const T*>(a.w), c0, w);
    if (a.bias) load_v<T, 1>(static_cast<const T*>(a.bias) + c0, bias);
#pragma unroll
    for (int k = 0; k < kW - 1; ++k) input_row<T, 1, kW>(a, x, b, c0, t0 - (kW - 1) + k, win[k]);
    T* y = static_cast<T*>(a.y) + b * a.y_bs + c0;
    for (int t = t0; t < t1; t += kAhead) {
        float v[kAhead][1];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (t + u < t1) load_v<T, 1>(x + (t + u) * a.x_ts, v[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (t + u >= t1) break;
            emit<T, 1, kW>(w, bias, win, v[u], a.silu, y + (t + u) * a.y_ts);
#pragma unroll
            for (int k = 0; k + 1 < kW - 1; ++k) win[k][0] = win[k + 1][0];
            win[kW - 2][0] = v[u][0];
        }
    }
}

// Packed fp32 pairs: one instruction for two channels.
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(uint64_t a, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(a));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Rows of whole 16-byte pieces. The rows ahead are in flight in shared memory: every
// thread copies its own pieces asynchronously into a ring of its own, so that no
// barrier stands between the copies and their use. Two blocks per SM and rings of
// three groups of four rows (B=4 N=4096 C=4352 bf16: 56 us; rows ahead in registers
// instead 72, three groups of two rows 60, four of six 60; three blocks per SM, which
// spill, 92). Two channels per instruction, as packed pairs, took 3 of the 59 us.
constexpr int kRows = 4, kRing = 3;                    // rows per group, groups in the ring
constexpr int kRingBytes = kRows * kRing * kThreads * 16;
static_assert(kRingBytes <= 48 * 1024, "within the shared memory of a launch without an attribute");

template <typename T, int kV, int kW>
__global__ void __launch_bounds__(kThreads, 2) conv_ring_kernel(const __grid_constant__ ConvArgs a) {
    constexpr int kP = kV / 2;
    extern __shared__ uint4 ring[];                        // [kRing kRows][threads]
    const int pieces = a.C / kV;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t bg = id / pieces;
    const int c0 = (int)(id - bg * pieces) * kV;
    const int b = (int)(bg / a.groups), g = (int)(bg - (int64_t)b * a.groups);
    if (b >= a.B) return;
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const T* x = static_cast<const T*>(a.x) + b * a.x_bs + c0;
    if (g == 0 && a.s1) write_state<T, kV, kW>(a, x, b, c0, n);
    const int t0 = g * a.tok, t1 = min(t0 + a.tok, n);
    if (t0 >= t1) return;
    const uint32_t slot = (uint32_t)__cvta_generic_to_shared(ring + threadIdx.x);
    const T* xa = x + (int64_t)t0 * a.x_ts;
    int left = t1 - t0;                                    // rows not yet fetched
    auto fetch = [&](int q) {                              // the next rows into group q
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (u < left) copy16(slot + (q * kRows + u) * kThreads * 16, xa);
            xa += a.x_ts;
        }
        left -= kRows;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int q = 0; q < kRing - 1; ++q) fetch(q);
    uint64_t w[kW][kP], bias[kP], win[kW - 1][kP];
    {
        float f[kW][kV], e[kV] = {};
        load_weights<T, kV, kW>(static_cast<const T*>(a.w), c0, f);
        if (a.bias) load_v<T, kV>(static_cast<const T*>(a.bias) + c0, e);
#pragma unroll
        for (int j = 0; j < kP; ++j) {
            bias[j] = pair_of(e[2 * j], e[2 * j + 1]);
#pragma unroll
            for (int k = 0; k < kW; ++k) w[k][j] = pair_of(f[k][2 * j], f[k][2 * j + 1]);
        }
#pragma unroll
        for (int k = 0; k < kW - 1; ++k) {
            input_row<T, kV, kW>(a, x, b, c0, t0 - (kW - 1) + k, e);
#pragma unroll
            for (int j = 0; j < kP; ++j) win[k][j] = pair_of(e[2 * j], e[2 * j + 1]);
        }
    }
    T* y = static_cast<T*>(a.y) + b * a.y_bs + (int64_t)t0 * a.y_ts + c0;
    int q = 0;
    for (int t = t0; t < t1; t += kRows) {
        fetch(q == 0 ? kRing - 1 : q - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        const uint4* r = ring + q * kRows * kThreads + threadIdx.x;
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
            if (t + u >= t1) break;
            float v[kV];
            load_v<T, kV>(reinterpret_cast<const T*>(r + u * kThreads), v);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const uint64_t in = pair_of(v[2 * j], v[2 * j + 1]);
                uint64_t s = bias[j];
#pragma unroll
                for (int k = 0; k < kW - 1; ++k) s = fma_pair(w[k][j], win[k][j], s);
                s = fma_pair(w[kW - 1][j], in, s);
#pragma unroll
                for (int k = 0; k + 1 < kW - 1; ++k) win[k][j] = win[k + 1][j];
                win[kW - 2][j] = in;
                split(s, &v[2 * j], &v[2 * j + 1]);
            }
            if (a.silu) {
#pragma unroll
                for (int j = 0; j < kV; ++j) v[j] = silu(v[j]);
            }
            store_v<T, kV>(y, v);
            y += a.y_ts;
        }
        q = q + 1 == kRing ? 0 : q + 1;
    }
}

// One token per sequence: x, y [B, C] (row strides x_bs, y_bs); the state s1 is
// shifted by one row in place.
template <typename T, int kV, int kW>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const __grid_constant__ ConvArgs a) {
    const int pieces = a.C / kV;
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t b = id / pieces;
    const int c0 = (int)(id - b * pieces) * kV;
    if (b >= a.B) return;
    T* s = static_cast<T*>(a.s1) + b * (kW - 1) * a.C + c0;
    float win[kW - 1][kV], x[kV], w[kW][kV], bias[kV] = {};
#pragma unroll
    for (int k = 0; k < kW - 1; ++k) load_v<T, kV>(s + (int64_t)k * a.C, win[k]);
    load_v<T, kV>(static_cast<const T*>(a.x) + b * a.x_bs + c0, x);
    load_weights<T, kV, kW>(static_cast<const T*>(a.w), c0, w);
    if (a.bias) load_v<T, kV>(static_cast<const T*>(a.bias) + c0, bias);
#pragma unroll
    for (int k = 0; k + 1 < kW - 1; ++k) store_v<T, kV>(s + (int64_t)k * a.C, win[k + 1]);
    store_v<T, kV>(s + (int64_t)(kW - 2) * a.C, x);
    emit<T, kV, kW>(w, bias, win, x, a.silu, static_cast<T*>(a.y) + b * a.y_bs + c0);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool vector_ok(const ConvArgs& a, int64_t eb) {
    return (a.C * eb) % 16 == 0 && aligned16(a.x) && aligned16(a.w) && aligned16(a.bias) &&
           aligned16(a.s0) && aligned16(a.s1) && aligned16(a.y) && (a.x_bs * eb) % 16 == 0 &&
           (a.x_ts * eb) % 16 == 0 && (a.y_bs * eb) % 16 == 0 && (a.y_ts * eb) % 16 == 0;
}

template <typename T, int kV, int kW>
cudaError_t launch(ConvArgs& a, bool step, cudaStream_t st) {
    const int64_t pieces = a.C / kV;
    if (step) {
        const int64_t blocks = (a.B * pieces + kThreads - 1) / kThreads;
        conv_step_kernel<T, kV, kW><<<(unsigned)blocks, kThreads, 0, st>>>(a);
        return cudaPeekAtLastError();
    }
    // Tokens per thread: 64 (W - 1 rows in 64 are read again, and the weights are loaded
    // once), fewer while that would leave SMs without four blocks each. B=4 N=4096 C=4352
    // bf16 takes 32: 56 us, 16 tokens 68; C=2304 N=3000 29, 96 tokens 33.
    a.tok = 64;
    while (a.tok > 4 && (int64_t)a.B * ((a.N + a.tok - 1) / a.tok) * pieces < 4LL * kThreads * tcc::sm_count())
        a.tok /= 2;
    a.groups = (a.N + a.tok - 1) / a.tok;
    const int64_t blocks = ((int64_t)a.B * a.groups * pieces + kThreads - 1) / kThreads;
    if (blocks > 2147483647LL) return cudaErrorInvalidValue;
    if constexpr (kV > 1) {
        conv_ring_kernel<T, kV, kW><<<(unsigned)blocks, kThreads, kRingBytes, st>>>(a);
    } else {
        conv_fwd_kernel<T, kW><<<(unsigned)blocks, kThreads, 0, st>>>(a);
    }
    return cudaPeekAtLastError();
}

template <typename T, int kV>
cudaError_t by_width(ConvArgs& a, int W, bool step, cudaStream_t st) {
    switch (W) {
        case 2: return launch<T, kV, 2>(a, step, st);
        case 3: return launch<T, kV, 3>(a, step, st);
        default: return launch<T, kV, 4>(a, step, st);
    }
}

cudaError_t run(ConvArgs& a, int W, la_dtype dt, bool step, cudaStream_t st) {
    const bool vec = vector_ok(a, dt == LA_BF16 ? 2 : 4);
    if (dt == LA_BF16)
        return vec ? by_width<__nv_bfloat16, 8>(a, W, step, st) : by_width<__nv_bfloat16, 1>(a, W, step, st);
    return vec ? by_width<float, 4>(a, W, step, st) : by_width<float, 1>(a, W, step, st);
}

la_status check(int B, int N, int C, int W, la_dtype dt) {
    if (B < 0 || N < 0 || C < 1 || W < 1) return LA_ERR_INVALID_ARG;
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (W < 2 || W > 4) return LA_ERR_UNSUPPORTED;
    if ((int64_t)B * N > (int64_t)1 << 30) return LA_ERR_UNSUPPORTED;   // token counts and their roundings fit an int
    return LA_OK;
}

bool bad(const void* p, la_dtype dt) {
    return !p || (reinterpret_cast<uintptr_t>(p) & (dt == LA_BF16 ? 1 : 3));
}

bool bad_or_null(const void* p, la_dtype dt) { return p && bad(p, dt); }

}  // namespace

}  // namespace la

extern "C" {

la_status la_short_conv_fwd(const void* x, int64_t x_batch, int64_t x_token, const void* w,
                            const void* bias, int silu, const int32_t* lengths, const void* state0,
                            void* state_out, void* y, int64_t y_batch, int64_t y_token, int B,
                            int N, int C, int W, la_dtype dt, la_stream_t stream) {
    la_status s = la::check(B, N, C, W, dt);
    if (s != LA_OK) return s;
    if (B == 0) return LA_OK;
    if (la::bad_or_null(bias, dt) || la::bad_or_null(state0, dt) || la::bad_or_null(state_out, dt) ||
        (reinterpret_cast<uintptr_t>(lengths) & 3) || la::bad(w, dt))
        return LA_ERR_INVALID_ARG;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const size_t state = (size_t)B * (W - 1) * C * eb;
    // Threads of other token groups may still read the old state.
    const la::Rows s0 = la::block_of(state0, state), s1 = la::block_of(state_out, state);
    if (la::overlap(s0, s1)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0) {
        if (!state_out) return LA_OK;
        const cudaError_t e = state0 ? cudaMemcpyAsync(state_out, state0, state, cudaMemcpyDeviceToDevice, st)
                                     : cudaMemsetAsync(state_out, 0, state, st);
        return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    if (la::bad(x, dt) || la::bad(y, dt)) return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, N, C, y_batch, y_token)) return LA_ERR_INVALID_ARG;
    const la::Rows xr = la::rows_of(x, B, N, C, x_batch, x_token, eb), yr = la::rows_of(y, B, N, C, y_batch, y_token, eb);
    const la::Rows wr = la::block_of(w, (int64_t)C * W * eb), br = la::block_of(bias, C * eb);
    const la::Rows nr = la::block_of(lengths, 4 * (int64_t)B);
    if (la::overlaps_any(yr, {xr, wr, br, nr, s0, s1}) || la::overlaps_any(s1, {xr, wr, br, nr})) return LA_ERR_INVALID_ARG;
    la::ConvArgs a = {};
    a.x = x, a.x_bs = x_batch, a.x_ts = x_token, a.w = w, a.bias = bias, a.s0 = state0, a.s1 = state_out;
    a.y = y, a.y_bs = y_batch, a.y_ts = y_token, a.lengths = lengths;
    a.B = B, a.N = N, a.C = C, a.silu = silu ? 1 : 0;
    return la::run(a, W, dt, false, st) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_short_conv_step(const void* x, int64_t x_batch, const void* w, const void* bias,
                             int silu, void* state, void* y, int64_t y_batch, int B, int C, int W,
                             la_dtype dt, la_stream_t stream) {
    la_status s = la::check(B, 1, C, W, dt);
    if (s != LA_OK) return s;
    if (B == 0) return LA_OK;
    if (la::bad(x, dt) || la::bad(w, dt) || la::bad(state, dt) || la::bad(y, dt) || la::bad_or_null(bias, dt))
        return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, 1, C, y_batch, 0)) return LA_ERR_INVALID_ARG;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const la::Rows xr = la::rows_of(x, B, 1, C, x_batch, 0, eb), yr = la::rows_of(y, B, 1, C, y_batch, 0, eb);
    const la::Rows wr = la::block_of(w, (int64_t)C * W * eb), br = la::block_of(bias, C * eb);
    const la::Rows sr = la::block_of(state, (int64_t)B * (W - 1) * C * eb);
    // y may be x itself: a thread reads what it replaces.
    if (la::overlaps_any(sr, {xr, wr, br, yr}) || la::overlaps_any(yr, {wr, br}) ||
        (!la::same_rows(xr, yr) && la::overlap(xr, yr)))
        return LA_ERR_INVALID_ARG;
    la::ConvArgs a = {};
    a.x = x, a.x_bs = x_batch, a.w = w, a.bias = bias, a.s1 = state, a.y = y, a.y_bs = y_batch;
    a.B = B, a.N = 1, a.C = C, a.silu = silu ? 1 : 0;
    return la::run(a, W, dt, true, (cudaStream_t)stream) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
