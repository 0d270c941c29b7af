// Group norm over channels-last rows x [B, N, C], with an optional silu and an optional
// gate, and its backward. Per sample b and group g of Cg = C / G neighbouring channels,
// statistics over the group's N Cg values:
//   xh = (x - mean) r,  r = 1 / sqrt(var + eps);  u = w_c xh + b_c;  y = act(u) silu(z)
// With N = 1 a row is a sample of its own: the norm of each head of an attention output
// ([tokens, 1, H D], a group per head), where linear attention has no denominator ("Why
// Replace Attention? The Softmax Bottleneck and the Path to Linear Time", section 6.2,
// gives the denominator whose place it takes). N = height x width is the form of images.
// Backward, from dy with h = dy silu(z) act'(u):
//   db = sum h,  dw = sum h xh,  dz = dy act(u) silu'(z),
//   dx = r (w h - mean(w h) - xh mean(w h xh))   (means over the group)
//
// What bounds it: HBM bandwidth; every value is read once and written once (images twice,
// the second time mostly from L2), two or three dozen operations each. Two forms (times of
// consecutive replays of a captured call; called one by one 33 us for 31, 41 for 38, 25 to 29 for 18):
//  - N = 1: 2^k lanes hold one group of one row in registers; mean and variance in two
//    passes over them; a thread keeps its channels, and their weights, over all its rows.
//    131072 rows of 1024 gated bf16 values: 126 us, 0.97 of a copy's rate; backward of 32765
//    rows of 512: 38 us, 0.67 (instructions, and the sums of the weights in registers).
//  - else: a first kernel leaves each block of rows' mean and sum of squares about it (so
//    that a large mean costs no digits), a second one joins them and writes the outputs.
//    B=16 N=4096 C=320 bf16 silu: 31 us, 0.41 (both passes' instructions, and two launches);
//    backward of B=16 N=1024 C=256 fp32: 18 us, 0.42.
// Sums are fp32 in a fixed order: the same inputs give the same bits.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "mixing.cuh"
#include "overlap.h"
#include "scan.cuh"
#include "tc_common.cuh"

namespace la {

namespace {

struct NormArgs {
    const void *x, *z, *w, *b, *dy;
    void *y, *dz;                                   // y: forward's output, backward's dx
    int64_t x_bs, x_ts, z_bs, z_ts, dy_bs, dy_ts, y_bs, y_ts, dz_bs, dz_ts;
    float *stats, *dw, *db;
    float* partial;                                 // see each kernel
    int B, N, C, G, Cg, silu;
    float eps;
    int lanes, slots;                               // one-token form: lanes per group, per row
    int chunks, per, gb;                            // other form: blocks of rows, their rows, groups per block
    int blocks, over;                               // its backward: blocks of sums, floats before those over a block's parts
};

// V adjacent values as stored.
template <typename T, int V> struct Raw { T v[V]; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 v; };
template <> struct Raw<float, 4> { float4 v; };

template <typename T, int V> __device__ __forceinline__ Raw<T, V> load(const T* p) {
    Raw<T, V> r;
    if constexpr (V == 1) r.v[0] = *p;
    else if constexpr (sizeof(T) == 2) r.v = __ldg(reinterpret_cast<const uint4*>(p));
    else r.v = __ldg(reinterpret_cast<const float4*>(p));
    return r;
}

// V values in fp32, as packed pairs: half the instructions, which bound these kernels next to
// memory.
__device__ __forceinline__ float lo_of(uint64_t v) {
    float a, b;
    unpk2(v, &a, &b);
    return a;
}
__device__ __forceinline__ float hi_of(uint64_t v) {
    float a, b;
    unpk2(v, &a, &b);
    return b;
}
__device__ __forceinline__ uint64_t add1(uint64_t a, uint64_t b) { return add2(a, b); }
__device__ __forceinline__ uint64_t mul1(uint64_t a, uint64_t b) { return mul2(a, b); }
__device__ __forceinline__ uint64_t fma1(uint64_t a, uint64_t b, uint64_t c) { return fma2(a, b, c); }
__device__ __forceinline__ float add1(float a, float b) { return a + b; }
__device__ __forceinline__ float mul1(float a, float b) { return a * b; }
__device__ __forceinline__ float fma1(float a, float b, float c) { return fmaf(a, b, c); }

template <int V> struct Vals {
    static constexpr int n = V / 2;
    uint64_t p[n];
    __device__ __forceinline__ float get(int i) const { return i & 1 ? hi_of(p[i >> 1]) : lo_of(p[i >> 1]); }
    template <typename F> __device__ __forceinline__ void make(F f) {       // value i = f(i)
#pragma unroll
        for (int i = 0; i < n; ++i) p[i] = pk2(f(2 * i), f(2 * i + 1));
    }
};
template <> struct Vals<1> {
    static constexpr int n = 1;
    float p[1];
    __device__ __forceinline__ float get(int) const { return p[0]; }
    template <typename F> __device__ __forceinline__ void make(F f) { p[0] = f(0); }
};
template <int V> __device__ __forceinline__ Vals<V> all(float v) {
    Vals<V> r;
    r.make([=](int) { return v; });
    return r;
}
template <int V> __device__ __forceinline__ Vals<V> operator+(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < r.n; ++i) r.p[i] = add1(a.p[i], b.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Vals<V> operator*(const Vals<V>& a, const Vals<V>& b) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < r.n; ++i) r.p[i] = mul1(a.p[i], b.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ Vals<V> fma(const Vals<V>& a, const Vals<V>& b, const Vals<V>& c) {
    Vals<V> r;
#pragma unroll
    for (int i = 0; i < r.n; ++i) r.p[i] = fma1(a.p[i], b.p[i], c.p[i]);
    return r;
}
template <int V> __device__ __forceinline__ float total(const Vals<V>& a) {
    if constexpr (V == 8) {
        const uint64_t s = add1(add1(a.p[0], a.p[1]), add1(a.p[2], a.p[3]));
        return lo_of(s) + hi_of(s);
    } else if constexpr (V == 4) {
        const uint64_t s = add1(a.p[0], a.p[1]);
        return lo_of(s) + hi_of(s);
    } else {
        return a.p[0];
    }
}
template <typename T, int V> __device__ __forceinline__ Vals<V> floats(const Raw<T, V>& r) {
    Vals<V> f;
    if constexpr (V == 1) {
        f.p[0] = to_f(r.v[0]);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f.p[i] = pk2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
    } else {
        f.p[0] = pk2(r.v.x, r.v.y), f.p[1] = pk2(r.v.z, r.v.w);
    }
    return f;
}
template <typename T, int V> __device__ __forceinline__ void store(T* p, const Vals<V>& f) {
    if constexpr (V == 1) {
        *p = from_f<T>(f.p[0]);
    } else if constexpr (sizeof(T) == 2) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = tcc::pack_bf16(lo_of(f.p[i]), hi_of(f.p[i]));
        *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(lo_of(f.p[0]), hi_of(f.p[0]), lo_of(f.p[1]), hi_of(f.p[1]));
    }
}

// 1 / (1 + e^-v): hardware exponential and reciprocal, a few 2^-23 in all; e^-v overflows to
// infinity below -88.7, and its reciprocal is then 0: the limit.
template <int V> __device__ __forceinline__ Vals<V> sigmoid(const Vals<V>& v) {
    const Vals<V> t = v * all<V>(-1.4426950408889634f);
    Vals<V> e;
    e.make([&](int i) {
        float r;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t.get(i)));
        return r;
    });
    e = e + all<V>(1.f);
    Vals<V> s;
    s.make([&](int i) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e.get(i)));
        return r;
    });
    return s;
}

// y from u.
template <int V> __device__ __forceinline__ Vals<V> forward(Vals<V> u, bool act, bool gate, const Vals<V>& z) {
    if (act) u = u * sigmoid(u);
    if (gate) u = u * (z * sigmoid(z));
    return u;
}

// h = dL/du from u and dy, and dz (in z's place). With s = sigmoid(u), the slope of u s is
// s + u s (1 - s).
template <int V>
__device__ __forceinline__ Vals<V> backward(const Vals<V>& u, const Vals<V>& dy, bool act, bool gate, Vals<V>& z) {
    const Vals<V> one = all<V>(1.f), minus = all<V>(-1.f);
    Vals<V> v = u, h = dy, slope;
    if (act) {
        const Vals<V> s = sigmoid(u);
        v = u * s;
        slope = fma(v, fma(s, minus, one), s);
    }
    if (gate) {
        const Vals<V> s = sigmoid(z), g = z * s;
        z = v * dy * fma(g, fma(s, minus, one), s);
        h = dy * g;
    }
    return act ? h * slope : h;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Neighbouring lanes' sum, kL of them (0: `lanes`, any power of two).
template <int kL> __device__ __forceinline__ float group_sum(float v, int lanes) {
    if constexpr (kL == 0) {
        return lanes_sum(v, lanes);
    } else {
#pragma unroll
        for (int o = kL / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
}

template <typename T, int V> __device__ __forceinline__ Vals<V> weights_of(const void* p, int64_t c, bool in, float other) {
    Vals<V> r;
    r.make([&](int i) { return in && p ? to_f(static_cast<const T*>(p)[c + i]) : other; });
    return r;
}

constexpr int kThreads = 256;

// A thread's own vectors on the way: copied asynchronously to its places in shared memory, some
// steps ahead of their use, so that what is in flight costs no registers. (Loads into registers
// one step ahead left memory idle: 131072 rows of 1024 gated bf16 values 182 us.) Single
// values (V = 1) are loaded when they are used.
template <typename T, int V> struct Ring {
    uint4* own;
    __device__ __forceinline__ explicit Ring(void* smem) : own(static_cast<uint4*>(smem) + threadIdx.x) {}
    __device__ __forceinline__ void fetch(int slot, const T* p) const {
        if constexpr (V > 1)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(own + slot * blockDim.x)), "l"(p) : "memory");
    }
    __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
    template <int kLeft> __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }
    __device__ __forceinline__ Vals<V> get(int slot, const T* p) const {
        Raw<T, V> r;
        if constexpr (V == 1) r = load<T, V>(p);
        else r = *reinterpret_cast<const Raw<T, V>*>(own + slot * blockDim.x);
        return floats<T, V>(r);
    }
};

// One-token form. A row's groups lie side by side over the slots of a block, `lanes` each
// (a power of two), K vectors of V values per lane; rows side by side where several fit. kL:
// the lanes, where the groups fill them and the slots whole blocks, so that every thread has
// values; 0: any number, counted at run time, and a lane past the group's end, or a thread past
// the last whole row, holds nothing.
template <int V, int K, int kL> struct RowPlace {
    int S, R, sub, lanes, g, l, c0, step;
    bool in[K];
    __device__ __forceinline__ explicit RowPlace(const NormArgs& a) {
        const int tid = threadIdx.x;
        S = a.slots;
        R = S <= (int)blockDim.x ? blockDim.x / S : 1;
        sub = S <= (int)blockDim.x ? tid / S : 0;
        const int slot = S <= (int)blockDim.x ? tid - sub * S : blockIdx.y * blockDim.x + tid;
        lanes = kL ? kL : a.lanes;
        g = slot / lanes;
        l = slot - g * lanes;
        c0 = g * a.Cg + l * V;
        step = lanes * V;
#pragma unroll
        for (int k = 0; k < K; ++k) in[k] = kL ? true : sub < R && slot < S && l * V + k * step < a.Cg;
    }
};

template <int K> constexpr int kStages = K == 1 ? 4 : 2;

template <typename T, int V, int K, int kL>
__global__ void __launch_bounds__(kThreads, K == 1 ? 3 : 1) rows_fwd_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][x, z][K][thread]
    constexpr int kS = kStages<K>;
    const RowPlace<V, K, kL> t(a);
    const Ring<T, V> ring(smem);
    const bool act = a.silu != 0, gate = a.z != nullptr;
    Vals<V> w[K], b[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = weights_of<T, V>(a.w, t.c0 + k * t.step, t.in[k], 1.f);
        b[k] = weights_of<T, V>(a.b, t.c0 + k * t.step, t.in[k], 0.f);
    }
    const float inv = 1.f / a.Cg;
    const int stride = gridDim.x * t.R, count = (a.B - (int)blockIdx.x * t.R + stride - 1) / stride;
    int row = blockIdx.x * t.R + t.sub, ahead = row;
    const T* x = static_cast<const T*>(a.x) + t.c0;
    const T* z = static_cast<const T*>(a.z) + (gate ? t.c0 : 0);
    T* y = static_cast<T*>(a.y) + t.c0;
    auto fetch = [&](int i) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t.in[k] && ahead < a.B) {
                ring.fetch(((i % kS) * 2 + 0) * K + k, x + ahead * a.x_bs + k * t.step);
                if (gate) ring.fetch(((i % kS) * 2 + 1) * K + k, z + ahead * a.z_bs + k * t.step);
            }
        ring.commit();
        ahead += stride;                           // at most B + kS strides: B <= 2^30
    };
#pragma unroll
    for (int i = 0; i < kS - 1; ++i) fetch(i);
    for (int i = 0; i < count; ++i, row += stride) {
        ring.template wait<kS - 2>();
        fetch(i + kS - 1);
        const int at = (i % kS) * 2 * K;
        const bool on = row < a.B;
        Vals<V> f[K];
        float sum = 0.f, sq = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && t.in[k]) f[k] = ring.get(at + k, x + row * a.x_bs + k * t.step), sum += total(f[k]);
        const float mean = group_sum<kL>(sum, t.lanes) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && t.in[k]) f[k] = f[k] + all<V>(-mean), sq += total(f[k] * f[k]);
        const float r = rsqrtf(fmaf(group_sum<kL>(sq, t.lanes), inv, a.eps));
        if (a.stats && t.l == 0 && on && t.in[0])
            reinterpret_cast<float2*>(a.stats)[(int64_t)row * a.G + t.g] = make_float2(mean, r);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && t.in[k]) {
                Vals<V> zf = f[k];
                if (gate) zf = ring.get(at + K + k, z + row * a.z_bs + k * t.step);
                store<T, V>(y + row * a.y_bs + k * t.step, forward(fma(f[k] * all<V>(r), w[k], b[k]), act, gate, zf));
            }
    }
}

// partial: [gridDim.x][2][C], the block's sums of h xh and of h.
template <typename T, int V, int K, int kL>
__global__ void __launch_bounds__(kThreads, K > 1 ? 1 : V == 4 && kL ? 3 : 2) rows_bwd_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][x, dy, z][K][thread]; then the rows' sums
    constexpr int kS = kStages<K>;
    const RowPlace<V, K, kL> t(a);
    const Ring<T, V> ring(smem);
    const bool act = a.silu != 0, gate = a.z != nullptr;
    Vals<V> w[K], b[K], dw[K], db[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        w[k] = weights_of<T, V>(a.w, t.c0 + k * t.step, t.in[k], 1.f);
        b[k] = weights_of<T, V>(a.b, t.c0 + k * t.step, t.in[k], 0.f);
        dw[k] = db[k] = all<V>(0.f);
    }
    const float inv = -1.f / a.Cg;
    const int stride = gridDim.x * t.R, count = (a.B - (int)blockIdx.x * t.R + stride - 1) / stride;
    int row = blockIdx.x * t.R + t.sub, ahead = row;
    const T* x = static_cast<const T*>(a.x) + t.c0;
    const T* d = static_cast<const T*>(a.dy) + t.c0;
    const T* z = static_cast<const T*>(a.z) + (gate ? t.c0 : 0);
    T* y = static_cast<T*>(a.y) + t.c0;
    T* dz = static_cast<T*>(a.dz) + (gate ? t.c0 : 0);
    const float2* stats = reinterpret_cast<const float2*>(a.stats) + t.g;
    auto fetch = [&](int i) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (t.in[k] && ahead < a.B) {
                ring.fetch(((i % kS) * 3 + 0) * K + k, x + ahead * a.x_bs + k * t.step);
                ring.fetch(((i % kS) * 3 + 1) * K + k, d + ahead * a.dy_bs + k * t.step);
                if (gate) ring.fetch(((i % kS) * 3 + 2) * K + k, z + ahead * a.z_bs + k * t.step);
            }
        ring.commit();
        ahead += stride;
    };
    auto stats_of = [&](int n) { return n < a.B && t.in[0] ? __ldg(stats + (int64_t)n * a.G) : make_float2(0.f, 0.f); };
#pragma unroll
    for (int i = 0; i < kS - 1; ++i) fetch(i);
    // Two rows ahead: one ahead, the 32765 rows of 512 gated bf16 values took 43 us, not 38.
    float2 st = stats_of(row), st1 = stats_of(row + stride);
    for (int i = 0; i < count; ++i, row += stride) {
        ring.template wait<kS - 2>();
        fetch(i + kS - 1);
        const float2 next = stats_of(row + 2 * stride);
        const int at = (i % kS) * 3 * K;
        const bool on = row < a.B;
        Vals<V> xh[K], gw[K];
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && t.in[k]) {
                xh[k] = (ring.get(at + k, x + row * a.x_bs + k * t.step) + all<V>(-st.x)) * all<V>(st.y);
                Vals<V> zf = xh[k];
                if (gate) zf = ring.get(at + 2 * K + k, z + row * a.z_bs + k * t.step);
                const Vals<V> h = backward(fma(xh[k], w[k], b[k]), ring.get(at + K + k, d + row * a.dy_bs + k * t.step), act, gate, zf);
                if (gate) store<T, V>(dz + row * a.dz_bs + k * t.step, zf);
                dw[k] = fma(h, xh[k], dw[k]);
                db[k] = db[k] + h;
                gw[k] = h * w[k];
                s1 += total(gw[k]);
                s2 += total(gw[k] * xh[k]);
            }
        s1 = group_sum<kL>(s1, t.lanes) * inv;
        s2 = group_sum<kL>(s2, t.lanes) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && t.in[k])
                store<T, V>(y + row * a.y_bs + k * t.step, fma(xh[k], all<V>(s2), gw[k] + all<V>(s1)) * all<V>(st.y));
        st = st1, st1 = next;
    }
    ring.template wait<0>();
    tcc::pdl_launch_dependents();
    // The rows' sums side by side, in order.
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) red[i * kThreads + threadIdx.x] = which ? db[k].get(i) : dw[k].get(i);
            __syncthreads();
            if (t.sub == 0 && t.in[k])
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v = 0.f;
                    for (int j = 0; j < t.R; ++j) v += red[i * kThreads + j * t.S + threadIdx.x];
                    a.partial[((int64_t)blockIdx.x * 2 + which) * a.C + t.c0 + k * t.step + i] = v;
                }
        }
}

// dw (which = 0) or db (1), channels 32 block .. of them: sums over the blocks of partial
// [blocks][2][C], in order within a slice per warp. red: [warps][33].
__device__ __forceinline__ void sum_weights(const float* partial, float* to, int64_t blocks, int C, int block, int which, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, c = block * 32 + lane;
    float v = 0.f;
    if (c < C)
#pragma unroll 8
        for (int64_t i = warp; i < blocks; i += warps) v += partial[(2 * i + which) * C + c];
    red[warp * 33 + lane] = v;
    __syncthreads();
    if (warp == 0 && c < C && to) {
        v = 0.f;
        for (int i = 0; i < warps; ++i) v += red[i * 33 + lane];
        to[c] = v;
    }
}

__global__ void __launch_bounds__(1024) weights_kernel(const float* partial, float* dw, float* db, int64_t blocks, int C) {
    __shared__ float red[32 * 33];
    tcc::pdl_wait();
    sum_weights(partial, blockIdx.y ? db : dw, blocks, C, blockIdx.x, blockIdx.y, red);
}

// The other form's block: rows n0 .. n1 of sample b, the channels of gb groups from c0; a
// thread holds V channels of every subs-th row.
struct Block {
    int b, chunk, n0, n1, g0, ng, c0, cols, sub, subs, c;
    bool on;
};
template <int V> __device__ __forceinline__ Block block_of_rows(const NormArgs& a, int part) {
    Block k;
    k.b = part / a.chunks;
    k.chunk = part - k.b * a.chunks;
    k.n0 = k.chunk * a.per;
    k.n1 = min(k.n0 + a.per, a.N);
    k.g0 = blockIdx.y * a.gb;
    k.ng = min(a.gb, a.G - k.g0);
    k.c0 = k.g0 * a.Cg;
    k.cols = k.ng * a.Cg;
    const int vectors = a.gb * a.Cg / V;
    k.subs = blockDim.x / vectors;
    k.sub = threadIdx.x / vectors;
    k.c = (threadIdx.x - k.sub * vectors) * V;
    k.on = k.sub < k.subs && k.c < k.cols;
    return k;
}

constexpr int kMost = 1024;           // threads, and channels of a group
constexpr int kNarrow = 128;          // channels of a group of single tokens without whole 16-byte pieces
constexpr int kStatsRows = 8;         // rows on the way per thread of the statistics
constexpr int kRows = 4;              // and of the other passes

// The group of each of a thread's V channels from c on.
template <int V> struct Groups {
    int g[V];
    __device__ __forceinline__ Groups(int c, int Cg) {
        g[0] = c / Cg;
        int next = (g[0] + 1) * Cg - c;                // channels until the next group
#pragma unroll
        for (int i = 1; i < V; ++i) {
            g[i] = g[i - 1];
            if (i == next) ++g[i], next += Cg;
        }
    }
};

// partial: [B chunks][G][2], mean of the block's values of a group and sum of squares about it.
template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads, V == 1 ? 1 : 3) stats_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][thread]; then [subs][cols] means, squares
    float* sm = reinterpret_cast<float*>(smem);
    const Block k = block_of_rows<V>(a, blockIdx.x);
    const Ring<T, V> ring(smem);
    // Sums of the differences to the thread's first row, and of their squares. That row c is one
    // of its n values of a channel, so (c - mean)^2 is at most M, the sum of squares about the
    // mean, and what is subtracted from the squares below at most n M: n 2^-24 of M is lost at
    // worst, 2^-23 where c is no outlier.
    Vals<V> first = all<V>(0.f), sum = all<V>(0.f), sq = all<V>(0.f);
    int n = 0;
    if (k.on) {
        const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
        int row = k.n0 + k.sub;
        auto fetch = [&](int i, int r) {
            if (r < k.n1) ring.fetch(i % kStatsRows, x + r * a.x_ts);
            ring.commit();
        };
#pragma unroll
        for (int i = 0; i < kStatsRows - 1; ++i) fetch(i, row + i * k.subs);
        if (row < k.n1) {
            ring.template wait<kStatsRows - 2>();
            first = ring.get(0, x + row * a.x_ts) * all<V>(-1.f);
        }
        for (; row < k.n1; ++n, row += k.subs) {
            ring.template wait<kStatsRows - 2>();
            fetch(n + kStatsRows - 1, row + (kStatsRows - 1) * k.subs);
            const Vals<V> d = ring.get(n % kStatsRows, x + row * a.x_ts) + first;
            sum = sum + d;
            sq = fma(d, d, sq);
        }
        ring.template wait<0>();
    }
    const Vals<V> off = sum * all<V>(n > 0 ? 1.f / n : 0.f), minus = all<V>(-1.f);
    const Vals<V> mean = fma(first, minus, off), m2 = fma(sum * minus, off, sq);
    __syncthreads();
    tcc::pdl_launch_dependents();
    const int rows = k.n1 - k.n0, whole = rows / k.subs, more = rows - whole * k.subs;   // rows of a thread
    float *sm_mean = sm, *sm_sq = sm + k.subs * k.cols;
    if (k.on)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm_mean[k.sub * k.cols + k.c + i] = mean.get(i);
            const float q = m2.get(i);
            sm_sq[k.sub * k.cols + k.c + i] = q < 0.f ? 0.f : q;   // a comparison, so that NaN stays NaN
        }
    __syncthreads();
    const float inv = 1.f / rows;
    for (int c = threadIdx.x; c < k.cols; c += blockDim.x) {
        float m = 0.f, q = 0.f;
        for (int s = 0; s < k.subs; ++s) m = fmaf((float)(whole + (s < more)) * inv, sm_mean[s * k.cols + c], m);
        for (int s = 0; s < k.subs; ++s) {
            const float d = sm_mean[s * k.cols + c] - m;
            q += fmaf((float)(whole + (s < more)) * d, d, sm_sq[s * k.cols + c]);
        }
        sm_mean[c] = m;                            // this thread alone reads and writes column c
        sm_sq[c] = q;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const float each = 1.f / a.Cg;
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        float m = 0.f, q = 0.f;
        for (int c = lane; c < a.Cg; c += 32) m += sm_mean[g * a.Cg + c];
        m = lanes_sum(m, 32) * each;
        for (int c = lane; c < a.Cg; c += 32) {
            const float d = sm_mean[g * a.Cg + c] - m;
            q += fmaf(rows * d, d, sm_sq[g * a.Cg + c]);
        }
        q = lanes_sum(q, 32);
        if (lane == 0)
            *reinterpret_cast<float2*>(a.partial + 2 * ((int64_t)blockIdx.x * a.G + k.g0 + g)) = make_float2(m, q);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads, V == 1 ? 1 : 3) apply_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][x, z][thread]; [groups][2]: -mean, r
    const Block k = block_of_rows<V>(a, blockIdx.x);
    const Ring<T, V> ring(smem);
    float* sm = reinterpret_cast<float*>(smem + (V > 1 ? kRows * 2 * blockDim.x : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
    const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
    T* y = static_cast<T*>(a.y) + k.b * a.y_bs + k.c0 + k.c;
    int row = k.n0 + k.sub;
    auto fetch = [&](int i, int n) {
        if (k.on && n < k.n1) {
            ring.fetch((i % kRows) * 2, x + n * a.x_ts);
            if (gate) ring.fetch((i % kRows) * 2 + 1, z + n * a.z_ts);
        }
        ring.commit();
    };
#pragma unroll
    for (int i = 0; i < kRows - 1; ++i) fetch(i, row + i * k.subs);
    tcc::pdl_wait();
    const float inv = 1.f / a.N, size = (float)a.N * a.Cg;
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        const float2* p = reinterpret_cast<const float2*>(a.partial) + (int64_t)k.b * a.chunks * a.G + k.g0 + g;
        float m = 0.f, q = 0.f;
        for (int i = lane; i < a.chunks; i += 32) m = fmaf((float)min(a.per, a.N - i * a.per) * inv, p[(int64_t)i * a.G].x, m);
        m = lanes_sum(m, 32);
        for (int i = lane; i < a.chunks; i += 32) {
            const float2 v = p[(int64_t)i * a.G];
            q += fmaf((float)min(a.per, a.N - i * a.per) * a.Cg * (v.x - m), v.x - m, v.y);
        }
        const float r = rsqrtf(lanes_sum(q, 32) / size + a.eps);
        if (lane == 0) {
            sm[2 * g] = -m, sm[2 * g + 1] = r;
            if (a.stats && k.chunk == 0)
                *reinterpret_cast<float2*>(a.stats + 2 * ((int64_t)k.b * a.G + k.g0 + g)) = make_float2(m, r);
        }
    }
    __syncthreads();
    if (!k.on) return;
    const Groups<V> gr(k.c, a.Cg);
    Vals<V> mean, scale;
    mean.make([&](int i) { return sm[2 * gr.g[i]]; });
    scale.make([&](int i) { return sm[2 * gr.g[i] + 1]; });
    scale = scale * weights_of<T, V>(a.w, k.c0 + k.c, true, 1.f);
    const Vals<V> bias = weights_of<T, V>(a.b, k.c0 + k.c, true, 0.f);
    for (int i = 0; row < k.n1; ++i, row += k.subs) {
        ring.template wait<kRows - 2>();
        fetch(i + kRows - 1, row + (kRows - 1) * k.subs);
        const Vals<V> f = ring.get((i % kRows) * 2, x + row * a.x_ts) + mean;
        Vals<V> zf = f;
        if (gate) zf = ring.get((i % kRows) * 2 + 1, z + row * a.z_ts);
        store<T, V>(y + row * a.y_ts, forward(fma(f, scale, bias), act, gate, zf));
    }
}

// partial: [blocks][2][C] sums of h xh and of h, then [B chunks][G][2] of w h and of w h xh. kMany:
// more samples than blocks that run at once. A block then takes every blocks-th of them, its channels'
// sums over them in shared memory: what the weights' gradients are summed from stays a few blocks
// per SM however many samples there are. (With a block per sample the backward of B=65536 N=4 C=320
// bf16 took 2357 us, now 1741, and N=16 C=64 1786, now 1128. The loop costs a call without
// it 6 %, B=16 N=1024 C=256 fp32 18.4 us for 17.3: hence two kernels.)
template <typename T, int V, bool kMany>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads, V == 1 ? 1 : V == 8 ? 2 : 3) sums_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][x, dy, z][thread]; then [2][subs][cols]; behind both [2][cols]
    float* sm = reinterpret_cast<float*>(smem);
    const Ring<T, V> ring(smem);
    const bool act = a.silu != 0, gate = a.z != nullptr;
    for (int part = blockIdx.x;; part += gridDim.x) {
        const bool more = kMany && part + (int)gridDim.x < a.B * a.chunks;
        const Block k = block_of_rows<V>(a, part);
        Vals<V> dw = all<V>(0.f), db = all<V>(0.f);
        if (k.on) {
            const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
            const T* d = static_cast<const T*>(a.dy) + k.b * a.dy_bs + k.c0 + k.c;
            const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
            int row = k.n0 + k.sub;
            auto fetch = [&](int i, int n) {
                if (n < k.n1) {
                    ring.fetch((i % kRows) * 3, x + n * a.x_ts);
                    ring.fetch((i % kRows) * 3 + 1, d + n * a.dy_ts);
                    if (gate) ring.fetch((i % kRows) * 3 + 2, z + n * a.z_ts);
                }
                ring.commit();
            };
#pragma unroll
            for (int i = 0; i < kRows - 1; ++i) fetch(i, row + i * k.subs);
            const float2* s = reinterpret_cast<const float2*>(a.stats) + (int64_t)k.b * a.G + k.g0;
            const Groups<V> gr(k.c, a.Cg);
            Vals<V> mean, r;
            mean.make([&](int i) { return -__ldg(s + gr.g[i]).x; });
            r.make([&](int i) { return __ldg(s + gr.g[i]).y; });
            const Vals<V> w = weights_of<T, V>(a.w, k.c0 + k.c, true, 1.f), b = weights_of<T, V>(a.b, k.c0 + k.c, true, 0.f);
            for (int i = 0; row < k.n1; ++i, row += k.subs) {
                ring.template wait<kRows - 2>();
                fetch(i + kRows - 1, row + (kRows - 1) * k.subs);
                const Vals<V> xh = (ring.get((i % kRows) * 3, x + row * a.x_ts) + mean) * r;
                Vals<V> zf = xh;
                if (gate) zf = ring.get((i % kRows) * 3 + 2, z + row * a.z_ts);
                const Vals<V> h = backward(fma(xh, w, b), ring.get((i % kRows) * 3 + 1, d + row * a.dy_ts), act, gate, zf);
                dw = fma(h, xh, dw);
                db = db + h;
            }
            ring.template wait<0>();
        }
        __syncthreads();
        if (!more) tcc::pdl_launch_dependents();
        float *s_w = sm, *s_b = sm + k.subs * k.cols;
        if (k.on)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                s_w[k.sub * k.cols + k.c + i] = dw.get(i);
                s_b[k.sub * k.cols + k.c + i] = db.get(i);
            }
        __syncthreads();
        float* channel = a.partial + (int64_t)blockIdx.x * 2 * a.C + k.c0;
        float* over = sm + a.over;                 // the sums over the block's parts, a thread's own channels
        const bool first = !kMany || part == (int)blockIdx.x;
        for (int c = threadIdx.x; c < k.cols; c += blockDim.x) {
            float u = 0.f, v = 0.f;
            for (int s = 0; s < k.subs; ++s) u += s_w[s * k.cols + c], v += s_b[s * k.cols + c];
            if (first && !more) {
                channel[c] = u;
                channel[a.C + c] = v;
            } else {
                const float du = first ? u : over[c] + u, dv = first ? v : over[k.cols + c] + v;
                (more ? over : channel)[c] = du;
                (more ? over + k.cols : channel + a.C)[c] = dv;
            }
            const float w = a.w ? to_f(static_cast<const T*>(a.w)[k.c0 + c]) : 1.f;
            s_w[c] = w * u;
            s_b[c] = w * v;
        }
        __syncthreads();
        float2* group = reinterpret_cast<float2*>(a.partial + (int64_t)a.blocks * 2 * a.C) + (int64_t)part * a.G + k.g0;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
            float u = 0.f, v = 0.f;
            for (int c = lane; c < a.Cg; c += 32) u += s_b[g * a.Cg + c], v += s_w[g * a.Cg + c];
            u = lanes_sum(u, 32);
            v = lanes_sum(v, 32);
            if (lane == 0) group[g] = make_float2(u, v);
        }
        if (!more) break;
        __syncthreads();                           // the next rows take the place of the sums
    }
}

// The blocks past the rows' sum the weights' gradients meanwhile.
template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads, V == 1 ? 1 : V == 8 ? 2 : 3) apply_bwd_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ uint4 smem[];                // [stage][x, dy, z][thread]; [groups][2]: -means of w h and of w h xh
    const int extra = (int)blockIdx.x - a.B * a.chunks;
    if (extra >= 0) {
        tcc::pdl_wait();
        if (blockIdx.y == 0)
            sum_weights(a.partial, extra & 1 ? a.db : a.dw, a.blocks, a.C, extra >> 1, extra & 1,
                        reinterpret_cast<float*>(smem));
        return;
    }
    const Block k = block_of_rows<V>(a, blockIdx.x);
    const Ring<T, V> ring(smem);
    float* sm = reinterpret_cast<float*>(smem + (V > 1 ? kRows * 3 * blockDim.x : 0));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
    const T* d = static_cast<const T*>(a.dy) + k.b * a.dy_bs + k.c0 + k.c;
    const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
    T* y = static_cast<T*>(a.y) + k.b * a.y_bs + k.c0 + k.c;
    T* dz = static_cast<T*>(a.dz) + (gate ? k.b * a.dz_bs + k.c0 + k.c : 0);
    int row = k.n0 + k.sub;
    auto fetch = [&](int i, int n) {
        if (k.on && n < k.n1) {
            ring.fetch((i % kRows) * 3, x + n * a.x_ts);
            ring.fetch((i % kRows) * 3 + 1, d + n * a.dy_ts);
            if (gate) ring.fetch((i % kRows) * 3 + 2, z + n * a.z_ts);
        }
        ring.commit();
    };
#pragma unroll
    for (int i = 0; i < kRows - 1; ++i) fetch(i, row + i * k.subs);
    tcc::pdl_wait();
    const float2* parts = reinterpret_cast<const float2*>(a.partial + (int64_t)a.blocks * 2 * a.C);
    const float inv = -1.f / ((float)a.N * a.Cg);
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        const float2* p = parts + (int64_t)k.b * a.chunks * a.G + k.g0 + g;
        float u = 0.f, v = 0.f;
        for (int i = lane; i < a.chunks; i += 32) {
            const float2 t = p[(int64_t)i * a.G];
            u += t.x, v += t.y;
        }
        u = lanes_sum(u, 32);
        v = lanes_sum(v, 32);
        if (lane == 0) sm[2 * g] = u * inv, sm[2 * g + 1] = v * inv;
    }
    __syncthreads();
    if (!k.on) return;
    const Groups<V> gr(k.c, a.Cg);
    Vals<V> mean, r, s1, s2;
    const float2* s = reinterpret_cast<const float2*>(a.stats) + (int64_t)k.b * a.G + k.g0;
    mean.make([&](int i) { return -__ldg(s + gr.g[i]).x; });
    r.make([&](int i) { return __ldg(s + gr.g[i]).y; });
    s1.make([&](int i) { return sm[2 * gr.g[i]]; });
    s2.make([&](int i) { return sm[2 * gr.g[i] + 1]; });
    const Vals<V> w = weights_of<T, V>(a.w, k.c0 + k.c, true, 1.f), b = weights_of<T, V>(a.b, k.c0 + k.c, true, 0.f);
    for (int i = 0; row < k.n1; ++i, row += k.subs) {
        ring.template wait<kRows - 2>();
        fetch(i + kRows - 1, row + (kRows - 1) * k.subs);
        const Vals<V> xh = (ring.get((i % kRows) * 3, x + row * a.x_ts) + mean) * r;
        Vals<V> zf = xh;
        if (gate) zf = ring.get((i % kRows) * 3 + 2, z + row * a.z_ts);
        const Vals<V> h = backward(fma(xh, w, b), ring.get((i % kRows) * 3 + 1, d + row * a.dy_ts), act, gate, zf);
        store<T, V>(y + row * a.y_ts, fma(xh, s2, fma(h, w, s1)) * r);
        if (gate) store<T, V>(dz + row * a.dz_ts, zf);
    }
}

// ------------------------------------------------------------------ host side

// Blocks of the one-token backward at most, each of which leaves its sums.
int row_blocks() { return 3 * tcc::sm_count(); }

// Rows of a block of the other form: at least 16, and so many that the blocks run at once, as
// many on an SM as its registers hold (a second wave for a few of them would cost as much
// as the first).
constexpr int kMostPerSm = 3;
void cut_rows(int B, int N, int per_sm, int* per, int* chunks) {
    int64_t want = (int64_t)per_sm * tcc::sm_count() / B;
    want = want < 1 ? 1 : want;
    int64_t p = (N + want - 1) / want;
    p = p < 16 ? 16 : p;
    *per = (int)p;
    *chunks = (int)((N + p - 1) / p);
}

// Blocks of the backward's sums: as many as run at once.
int sum_blocks(int64_t parts, int per_sm) {
    const int64_t most = (int64_t)per_sm * tcc::sm_count();
    return (int)(parts < most ? parts : most);
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Lanes of a group in the one-token form, with K vectors of V values each; 0: does not fit.
int lanes_of(int Cg, int V, int K) {
    if (Cg % V || Cg > 32 * V * K) return 0;
    const int vectors = (Cg / V + K - 1) / K;
    int n = 1;
    while (n < vectors) n *= 2;
    return n;
}

template <typename T, int V, int K, int kL, bool kBackward>
cudaError_t launch_rows(NormArgs a, cudaStream_t st) {
    static std::atomic<int> optin[tcc::kMaxDevices];
    a.lanes = kL ? kL : lanes_of(a.Cg, V, K);
    a.slots = a.G * a.lanes;
    const int R = a.slots <= kThreads ? kThreads / a.slots : 1;
    // Whole rows where every thread has to have values.
    const int threads = kL && a.slots <= kThreads ? R * a.slots : kThreads;
    const int64_t tiles = ((int64_t)a.B + R - 1) / R;
    const unsigned columns = (unsigned)((a.slots + kThreads - 1) / kThreads);
    constexpr int ring = V > 1 ? kStages<K> * (kBackward ? 3 : 2) * K * kThreads * 16 : 0;
    constexpr int sums = kBackward ? kThreads * V * 4 : 0, smem = ring > sums ? ring : sums;
    cudaError_t e;
    if constexpr (!kBackward) {
        if ((e = tcc::ensure_smem_optin(rows_fwd_kernel<T, V, K, kL>, smem, optin)) != cudaSuccess) return e;
        const int64_t most = 3LL * tcc::sm_count();
        rows_fwd_kernel<T, V, K, kL><<<dim3((unsigned)(tiles < most ? tiles : most), columns), threads, smem, st>>>(a);
        return cudaPeekAtLastError();
    } else {
        if ((e = tcc::ensure_smem_optin(rows_bwd_kernel<T, V, K, kL>, smem, optin)) != cudaSuccess) return e;
        const int64_t most = V == 4 && kL ? row_blocks() : row_blocks() / 3 * 2, blocks = tiles < most ? tiles : most;
        rows_bwd_kernel<T, V, K, kL><<<dim3((unsigned)blocks, columns), threads, smem, st>>>(a);
        if ((e = cudaPeekAtLastError()) != cudaSuccess || (!a.dw && !a.db)) return e;
        return scan::launch_after(weights_kernel, dim3((a.C + 31) / 32, 2), 1024, 0, st, true, a.partial, a.dw, a.db, blocks, a.C);
    }
}

// Groups of 4 V, 8 V, 16 V or 32 V channels whose slots fill whole blocks.
template <typename T, int V, bool kBackward>
bool launch_exact(const NormArgs& a, cudaStream_t st, cudaError_t* e) {
    if (a.Cg % V) return false;
    const int lanes = a.Cg / V;
    const int64_t slots = (int64_t)a.G * lanes;
    if (slots > kThreads ? slots % kThreads != 0 : (kThreads / slots) * slots % 32 != 0) return false;
    switch (lanes) {
        case 4: *e = launch_rows<T, V, 1, 4, kBackward>(a, st); return true;
        case 8: *e = launch_rows<T, V, 1, 8, kBackward>(a, st); return true;
        case 16: *e = launch_rows<T, V, 1, 16, kBackward>(a, st); return true;
        case 32: *e = launch_rows<T, V, 1, 32, kBackward>(a, st); return true;
    }
    return false;
}

template <typename T, int V, bool kBackward>
cudaError_t launch_blocks(NormArgs a, cudaStream_t st) {
    const int per_sm = kBackward && V == 8 ? 2 : kMostPerSm;
    cut_rows(a.B, a.N, per_sm, &a.per, &a.chunks);
    // Whole groups per block, whole vectors: as many as its threads hold.
    const int unit = V / gcd(a.Cg, V), hold = (V == 1 ? kMost : kThreads) * V / a.Cg;
    a.gb = hold >= a.G ? a.G : hold / unit * unit;
    const int threads = V == 1 && a.gb * a.Cg > kThreads ? kMost : kThreads;
    const int subs = threads / (a.gb * a.Cg / V);
    const dim3 grid((unsigned)(a.B * a.chunks), (unsigned)((a.G + a.gb - 1) / a.gb));
    const int sums = 2 * (int)sizeof(float) * subs * a.gb * a.Cg, group = 2 * (int)sizeof(float) * a.gb;
    auto ring = [&](int places) { return V > 1 ? places * threads * 16 : 0; };
    auto larger = [](int p, int q) { return p > q ? p : q; };
    static std::atomic<int> optin[3][tcc::kMaxDevices];
    constexpr int kMostRing = V > 1 ? 3 * kRows * kThreads * 16 : 0, kMostSums = 2 * 2 * 4 * kThreads * V * (V == 1 ? 4 : 1);
    cudaError_t e;
    if constexpr (!kBackward) {
        if ((e = tcc::ensure_smem_optin(stats_kernel<T, V>, kMostRing + kMostSums, optin[0])) != cudaSuccess ||
            (e = tcc::ensure_smem_optin(apply_kernel<T, V>, kMostRing + kMostSums, optin[1])) != cudaSuccess)
            return e;
        stats_kernel<T, V><<<grid, threads, larger(ring(kStatsRows), sums), st>>>(a);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        return scan::launch_after(apply_kernel<T, V>, grid, threads, ring(2 * kRows) + group, st, true, a);
    } else {
        if ((e = tcc::ensure_smem_optin(sums_kernel<T, V, false>, kMostRing + kMostSums, optin[0])) != cudaSuccess ||
            (e = tcc::ensure_smem_optin(sums_kernel<T, V, true>, kMostRing + kMostSums, optin[2])) != cudaSuccess ||
            (e = tcc::ensure_smem_optin(apply_bwd_kernel<T, V>, kMostRing + kMostSums, optin[1])) != cudaSuccess)
            return e;
        const int parts = a.B * a.chunks, room = larger(ring(3 * kRows), sums);
        a.blocks = sum_blocks(parts, per_sm);
        a.over = room / (int)sizeof(float);
        const dim3 sum_grid((unsigned)a.blocks, grid.y);
        if (parts > a.blocks) sums_kernel<T, V, true><<<sum_grid, threads, room + 2 * (int)sizeof(float) * a.gb * a.Cg, st>>>(a);
        else sums_kernel<T, V, false><<<sum_grid, threads, room, st>>>(a);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        dim3 more = grid;
        if (a.dw || a.db) more.x += 2 * ((a.C + 31) / 32);
        return scan::launch_after(apply_bwd_kernel<T, V>, more, threads, larger(ring(3 * kRows) + group, 33 * 4 * threads / 32), st,
                                  true, a);
    }
}

// The vector forms need whole 16-byte pieces of every row.
template <typename T, bool kBackward>
cudaError_t launch_norm(const NormArgs& a, bool aligned, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (a.N == 1) {
        cudaError_t e;
        if (aligned && launch_exact<T, V, kBackward>(a, st, &e)) return e;
        if (aligned && lanes_of(a.Cg, V, 1)) return launch_rows<T, V, 1, 0, kBackward>(a, st);
        if (aligned && a.Cg % V == 0) return launch_rows<T, V, kMost / (32 * V), 0, kBackward>(a, st);
        return launch_rows<T, 1, kNarrow / 32, 0, kBackward>(a, st);
    }
    const int unit = V / gcd(a.Cg, V);
    const bool whole = a.G * a.Cg <= kThreads * V || kThreads * V / a.Cg >= unit;
    return aligned && whole ? launch_blocks<T, V, kBackward>(a, st) : launch_blocks<T, 1, kBackward>(a, st);
}

la_status check_norm(int B, int N, int C, int G, la_dtype dt, float eps) {
    if (B < 0 || N < 0 || C < 1 || G < 1 || C % G) return LA_ERR_INVALID_ARG;
    if ((dt != LA_F32 && dt != LA_BF16) || !isfinite(eps) || eps < 0.f) return LA_ERR_INVALID_ARG;
    if (C / G > kMost || C > 65535 * 32 || (int64_t)B * N > (1 << 30)) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

size_t norm_workspace(int B, int N, int C, int G) {
    if (B == 0 || N == 0) return 0;
    int per, chunks;
    cut_rows(B, N, kMostPerSm, &per, &chunks);
    const int64_t parts = (int64_t)B * chunks;
    const size_t blocks = sizeof(float) * 2 * ((size_t)sum_blocks(parts, kMostPerSm) * C + (size_t)parts * G);
    const size_t rows = sizeof(float) * 2 * (size_t)row_blocks() * C;
    return ((N == 1 ? rows : blocks) + 255) & ~(size_t)255;
}

// Whether the one-token form holds these groups.
bool fits(int N, int Cg, int V, bool aligned) { return N > 1 || Cg <= kNarrow || (aligned && Cg % V == 0); }

bool misaligned(const void* p, la_dtype dt) { return reinterpret_cast<uintptr_t>(p) & (dt == LA_BF16 ? 1 : 3); }

}  // namespace

}  // namespace la

extern "C" {

la_status la_group_norm_workspace_size(int B, int N, int C, int G, size_t* bytes) {
    if (!bytes) return LA_ERR_INVALID_ARG;
    const la_status s = la::check_norm(B, N, C, G, LA_F32, 0.f);
    if (s != LA_OK) return s;
    *bytes = la::norm_workspace(B, N, C, G);
    return LA_OK;
}

la_status la_group_norm_fwd(const void* x, int64_t x_batch, int64_t x_token, const void* w, const void* b,
                            const void* z, int64_t z_batch, int64_t z_token, void* y, int64_t y_batch,
                            int64_t y_token, float* stats, int B, int N, int C, int G, la_dtype dt, int silu,
                            float eps, void* workspace, size_t workspace_bytes, la_stream_t stream) {
    const la_status s = la::check_norm(B, N, C, G, dt, eps);
    if (s != LA_OK) return s;
    if (B == 0 || N == 0) return LA_OK;
    for (const void* p : {x, w, b, z, (const void*)y})
        if (la::misaligned(p, dt)) return LA_ERR_INVALID_ARG;
    if (!x || !y || (reinterpret_cast<uintptr_t>(stats) & 7)) return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, N, C, y_batch, y_token)) return LA_ERR_INVALID_ARG;
    const size_t use = N == 1 ? 0 : la::norm_workspace(B, N, C, G);
    if (use && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < use))
        return LA_ERR_WORKSPACE;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const la::Rows xr = la::rows_of(x, B, N, C, x_batch, x_token, eb), zr = la::rows_of(z, B, N, C, z_batch, z_token, eb);
    const la::Rows yr = la::rows_of(y, B, N, C, y_batch, y_token, eb), sr = la::block_of(stats, 8 * (int64_t)B * G);
    const la::Rows wr = la::block_of(w, C * eb), br = la::block_of(b, C * eb), kr = la::block_of(workspace, use);
    if (la::overlaps_any(yr, {xr, zr, wr, br, sr, kr}) || la::overlaps_any(sr, {xr, zr, wr, br, kr}) ||
        la::overlaps_any(kr, {xr, zr, wr, br}))
        return LA_ERR_INVALID_ARG;
    la::NormArgs a = {};
    a.x = x, a.x_bs = x_batch, a.x_ts = x_token, a.w = w, a.b = b, a.z = z, a.z_bs = z_batch, a.z_ts = z_token;
    a.y = y, a.y_bs = y_batch, a.y_ts = y_token, a.stats = stats, a.partial = static_cast<float*>(workspace);
    a.B = B, a.N = N, a.C = C, a.G = G, a.Cg = C / G, a.silu = silu ? 1 : 0, a.eps = eps;
    const int V = 16 / (int)eb;
    auto whole = [&](const void* p, int64_t bs, int64_t ts) {
        return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (B == 1 || bs % V == 0) && (N == 1 || ts % V == 0));
    };
    const bool aligned = C % V == 0 && whole(x, x_batch, x_token) && whole(z, z_batch, z_token) && whole(y, y_batch, y_token);
    if (!la::fits(N, C / G, V, aligned)) return LA_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dt == LA_BF16 ? la::launch_norm<__nv_bfloat16, false>(a, aligned, st)
                                        : la::launch_norm<float, false>(a, aligned, st);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_group_norm_bwd(const void* x, int64_t x_batch, int64_t x_token, const void* w, const void* b,
                            const void* z, int64_t z_batch, int64_t z_token, const void* dy, int64_t dy_batch,
                            int64_t dy_token, const float* stats, void* dx, int64_t dx_batch, int64_t dx_token,
                            void* dz, int64_t dz_batch, int64_t dz_token, float* dw, float* db, int B, int N,
                            int C, int G, la_dtype dt, int silu, void* workspace, size_t workspace_bytes,
                            la_stream_t stream) {
    const la_status s = la::check_norm(B, N, C, G, dt, 0.f);
    if (s != LA_OK) return s;
    cudaStream_t st = (cudaStream_t)stream;
    if (((reinterpret_cast<uintptr_t>(dw) | reinterpret_cast<uintptr_t>(db)) & 3)) return LA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) {                             // sums over nothing
        for (float* p : {dw, db})
            if (p && cudaMemsetAsync(p, 0, sizeof(float) * (size_t)C, st) != cudaSuccess) return LA_ERR_CUDA;
        return LA_OK;
    }
    for (const void* p : {x, w, b, z, dy, (const void*)dx, (const void*)dz})
        if (la::misaligned(p, dt)) return LA_ERR_INVALID_ARG;
    if (!x || !dy || !dx || !stats || (reinterpret_cast<uintptr_t>(stats) & 7) || !z != !dz) return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, N, C, dx_batch, dx_token) || (dz && !la::rows_disjoint(B, N, C, dz_batch, dz_token)))
        return LA_ERR_INVALID_ARG;
    const size_t use = la::norm_workspace(B, N, C, G);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < use) return LA_ERR_WORKSPACE;
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    const la::Rows xr = la::rows_of(x, B, N, C, x_batch, x_token, eb), zr = la::rows_of(z, B, N, C, z_batch, z_token, eb);
    const la::Rows gr = la::rows_of(dy, B, N, C, dy_batch, dy_token, eb);
    const la::Rows xo = la::rows_of(dx, B, N, C, dx_batch, dx_token, eb), zo = la::rows_of(dz, B, N, C, dz_batch, dz_token, eb);
    const la::Rows wr = la::block_of(w, C * eb), br = la::block_of(b, C * eb), sr = la::block_of(stats, 8 * (int64_t)B * G);
    const la::Rows wo = la::block_of(dw, 4 * (int64_t)C), bo = la::block_of(db, 4 * (int64_t)C), kr = la::block_of(workspace, use);
    for (const la::Rows* out : {&xo, &zo, &wo, &bo, &kr})
        if (la::overlaps_any(*out, {xr, zr, gr, wr, br, sr})) return LA_ERR_INVALID_ARG;
    if (la::overlaps_any(xo, {zo, wo, bo, kr}) || la::overlaps_any(zo, {wo, bo, kr}) || la::overlaps_any(wo, {bo, kr}) ||
        la::overlap(bo, kr))
        return LA_ERR_INVALID_ARG;
    la::NormArgs a = {};
    a.x = x, a.x_bs = x_batch, a.x_ts = x_token, a.w = w, a.b = b, a.z = z, a.z_bs = z_batch, a.z_ts = z_token;
    a.dy = dy, a.dy_bs = dy_batch, a.dy_ts = dy_token, a.y = dx, a.y_bs = dx_batch, a.y_ts = dx_token;
    a.dz = dz, a.dz_bs = dz_batch, a.dz_ts = dz_token, a.dw = dw, a.db = db;
    a.stats = const_cast<float*>(stats), a.partial = static_cast<float*>(workspace);
    a.B = B, a.N = N, a.C = C, a.G = G, a.Cg = C / G, a.silu = silu ? 1 : 0;
    const int V = 16 / (int)eb;
    auto whole = [&](const void* p, int64_t bs, int64_t ts) {
        return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (B == 1 || bs % V == 0) && (N == 1 || ts % V == 0));
    };
    const bool aligned = C % V == 0 && whole(x, x_batch, x_token) && whole(z, z_batch, z_token) &&
                         whole(dy, dy_batch, dy_token) && whole(dx, dx_batch, dx_token) && whole(dz, dz_batch, dz_token);
    if (!la::fits(N, C / G, V, aligned)) return LA_ERR_UNSUPPORTED;
    const cudaError_t e = dt == LA_BF16 ? la::launch_norm<__nv_bfloat16, true>(a, aligned, st)
                                        : la::launch_norm<float, true>(a, aligned, st);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
