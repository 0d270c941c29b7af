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
// the second time mostly from L2), two or three dozen operations each. Two forms:
//  - N = 1: 2^k lanes hold one group of one row in registers; mean and variance in two
//    passes over them; a thread keeps its channels, and their weights, over all its rows.
//  - else: a first kernel leaves each block of rows' mean and sum of squares about it (so
//    that a large mean costs no digits), a second one joins them and writes the outputs.
// Sums are fp32 in a fixed order: the same inputs give the same bits.
#include <cuda_bf16.h>
#include <math.h>

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
};

// V adjacent values as stored, and as floats.
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
template <typename T, int V> __device__ __forceinline__ void floats(const Raw<T, V>& r, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = to_f(r.v[0]);
    } else if constexpr (sizeof(T) == 2) {
        const uint32_t u[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
        f[0] = r.v.x, f[1] = r.v.y, f[2] = r.v.z, f[3] = r.v.w;
    }
}
template <typename T, int V> __device__ __forceinline__ void store(T* p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = from_f<T>(f[0]);
    } else if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = make_uint4(tcc::pack_bf16(f[0], f[1]), tcc::pack_bf16(f[2], f[3]),
                                                  tcc::pack_bf16(f[4], f[5]), tcc::pack_bf16(f[6], f[7]));
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
}

__device__ __forceinline__ float sigmoid(float v) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// y of one value from xh.
__device__ __forceinline__ float forward(float u, bool act, bool gate, float z) {
    const float v = act ? silu(u) : u;
    return gate ? v * silu(z) : v;
}

// h = dL/du of one value, and dz.
__device__ __forceinline__ float backward(float u, float dy, bool act, bool gate, float z, float* dz) {
    float v = u, slope = 1.f;
    if (act) {
        const float s = sigmoid(u);
        v = u * s;
        slope = s * fmaf(u, 1.f - s, 1.f);
    }
    float g = dy;
    if (gate) {
        const float s = sigmoid(z);
        *dz = dy * v * (s * fmaf(z, 1.f - s, 1.f));
        g = dy * z * s;
    }
    return g * slope;
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int kThreads = 256;

// One-token form. A row's groups lie side by side over the slots of a block, `lanes` each
// (a power of two; a lane past the group's end holds nothing), K vectors of V values per
// lane; rows side by side where several fit, kU times that many in flight.
template <typename T, int V, int K, int kU>
__global__ void __launch_bounds__(kThreads) rows_fwd_kernel(const __grid_constant__ NormArgs a) {
    const int tid = threadIdx.x, S = a.slots, R = S <= kThreads ? kThreads / S : 1;
    const int sub = S <= kThreads ? tid / S : 0, slot = S <= kThreads ? tid - sub * S : blockIdx.y * kThreads + tid;
    const int g = slot / a.lanes, l = slot - g * a.lanes;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    float w[K][V], b[K][V];
    bool in[K];
    const int c0 = g * a.Cg + l * V, step = a.lanes * V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = sub < R && slot < S && l * V + k * step < a.Cg;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = in[k] && a.w ? to_f(static_cast<const T*>(a.w)[c0 + k * step + i]) : 1.f;
            b[k][i] = in[k] && a.b ? to_f(static_cast<const T*>(a.b)[c0 + k * step + i]) : 0.f;
        }
    }
    const float inv = 1.f / a.Cg;
    for (int64_t base = (int64_t)blockIdx.x * R * kU; base < a.B; base += (int64_t)gridDim.x * R * kU) {
        Raw<T, V> x[kU][K], z[kU][K];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t row = base + u * R + sub;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                x[u][k] = load<T, V>(static_cast<const T*>(a.x) + row * a.x_bs + c0 + k * step);
                if (gate) z[u][k] = load<T, V>(static_cast<const T*>(a.z) + row * a.z_bs + c0 + k * step);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t row = base + u * R + sub;
            float f[K][V], sum = 0.f, sq = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                floats<T, V>(x[u][k], f[k]);
#pragma unroll
                for (int i = 0; i < V; ++i) sum += f[k][i];
            }
            const float mean = lanes_sum(sum, a.lanes) * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    f[k][i] -= mean;
                    sq = fmaf(f[k][i], f[k][i], sq);
                }
            }
            const float r = 1.f / sqrtf(fmaf(lanes_sum(sq, a.lanes), inv, a.eps));
            if (a.stats && l == 0 && in[0] && row < a.B)
                *reinterpret_cast<float2*>(a.stats + 2 * (row * a.G + g)) = make_float2(mean, r);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                float zf[V], y[V];
                if (gate) floats<T, V>(z[u][k], zf);
#pragma unroll
                for (int i = 0; i < V; ++i) y[i] = forward(fmaf(f[k][i] * r, w[k][i], b[k][i]), act, gate, gate ? zf[i] : 0.f);
                store<T, V>(static_cast<T*>(a.y) + row * a.y_bs + c0 + k * step, y);
            }
        }
    }
}

// partial: [gridDim.x][2][C], the block's sums of h xh and of h.
template <typename T, int V, int K, int kU>
__global__ void __launch_bounds__(kThreads) rows_bwd_kernel(const __grid_constant__ NormArgs a) {
    __shared__ float red[kThreads * V];
    const int tid = threadIdx.x, S = a.slots, R = S <= kThreads ? kThreads / S : 1;
    const int sub = S <= kThreads ? tid / S : 0, slot = S <= kThreads ? tid - sub * S : blockIdx.y * kThreads + tid;
    const int g = slot / a.lanes, l = slot - g * a.lanes;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    float w[K][V], b[K][V], dw[K][V], db[K][V];
    bool in[K];
    const int c0 = g * a.Cg + l * V, step = a.lanes * V;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = sub < R && slot < S && l * V + k * step < a.Cg;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            w[k][i] = in[k] && a.w ? to_f(static_cast<const T*>(a.w)[c0 + k * step + i]) : 1.f;
            b[k][i] = in[k] && a.b ? to_f(static_cast<const T*>(a.b)[c0 + k * step + i]) : 0.f;
            dw[k][i] = db[k][i] = 0.f;
        }
    }
    const float inv = 1.f / a.Cg;
    for (int64_t base = (int64_t)blockIdx.x * R * kU; base < a.B; base += (int64_t)gridDim.x * R * kU) {
        Raw<T, V> x[kU][K], d[kU][K], z[kU][K];
        float2 s[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t row = base + u * R + sub;
            s[u] = make_float2(0.f, 0.f);
            if (in[0] && row < a.B) s[u] = __ldg(reinterpret_cast<const float2*>(a.stats + 2 * (row * a.G + g)));
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                x[u][k] = load<T, V>(static_cast<const T*>(a.x) + row * a.x_bs + c0 + k * step);
                d[u][k] = load<T, V>(static_cast<const T*>(a.dy) + row * a.dy_bs + c0 + k * step);
                if (gate) z[u][k] = load<T, V>(static_cast<const T*>(a.z) + row * a.z_bs + c0 + k * step);
            }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t row = base + u * R + sub;
            const float mean = s[u].x, r = s[u].y;
            float xh[K][V], gw[K][V], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                float df[V], zf[V], dz[V];
                floats<T, V>(x[u][k], xh[k]);
                floats<T, V>(d[u][k], df);
                if (gate) floats<T, V>(z[u][k], zf);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[k][i] = (xh[k][i] - mean) * r;
                    const float h = backward(fmaf(xh[k][i], w[k][i], b[k][i]), df[i], act, gate, gate ? zf[i] : 0.f, &dz[i]);
                    dw[k][i] = fmaf(h, xh[k][i], dw[k][i]);
                    db[k][i] += h;
                    gw[k][i] = h * w[k][i];
                    s1 += gw[k][i];
                    s2 = fmaf(gw[k][i], xh[k][i], s2);
                }
                if (gate) store<T, V>(static_cast<T*>(a.dz) + row * a.dz_bs + c0 + k * step, dz);
            }
            s1 = lanes_sum(s1, a.lanes) * inv;
            s2 = lanes_sum(s2, a.lanes) * inv;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (!in[k] || row >= a.B) continue;
                float dx[V];
#pragma unroll
                for (int i = 0; i < V; ++i) dx[i] = r * (gw[k][i] - s1 - xh[k][i] * s2);
                store<T, V>(static_cast<T*>(a.y) + row * a.y_bs + c0 + k * step, dx);
            }
        }
    }
    tcc::pdl_launch_dependents();
    // The rows' sums side by side, in order.
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i) red[i * kThreads + tid] = which ? db[k][i] : dw[k][i];
            __syncthreads();
            if (sub == 0 && in[k])
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float v = 0.f;
                    for (int j = 0; j < R; ++j) v += red[i * kThreads + j * S + tid];
                    a.partial[((int64_t)blockIdx.x * 2 + which) * a.C + c0 + k * step + i] = v;
                }
        }
}

// dw, db = sums over the blocks of partial [blocks][2][C], in order within eight slices.
__global__ void __launch_bounds__(256) weights_kernel(const float* partial, float* dw, float* db, int64_t blocks, int C) {
    __shared__ float red[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    tcc::pdl_wait();
    float v = 0.f;
    if (c < C)
#pragma unroll 8
        for (int64_t i = warp; i < blocks; i += 8) v += partial[(2 * i + blockIdx.y) * C + c];
    red[warp][lane] = v;
    __syncthreads();
    float* to = blockIdx.y ? db : dw;
    if (warp == 0 && c < C && to) {
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v += red[i][lane];
        to[c] = v;
    }
}

// The other form's block: rows n0 .. n1 of sample b, the channels of gb groups from c0; a
// thread holds V channels of every sub-th row.
struct Block {
    int b, chunk, n0, n1, g0, ng, c0, cols, sub, subs, c;
    bool on;
};
template <int V> __device__ __forceinline__ Block block_of_rows(const NormArgs& a) {
    Block k;
    k.b = blockIdx.x / a.chunks;
    k.chunk = blockIdx.x - k.b * a.chunks;
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
constexpr int kTileRows = 8;

// partial: [B chunks][G][2], mean of the block's values of a group and sum of squares about it.
template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads) stats_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];                  // [subs][cols] means, then squares
    const Block k = block_of_rows<V>(a);
    const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
    float mean[V], m2[V];
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mean[i] = m2[i] = 0.f;
    if (k.on)
        for (int r0 = k.n0 + k.sub; r0 < k.n1; r0 += kTileRows * k.subs) {
            Raw<T, V> raw[kTileRows];
            const int m = min((k.n1 - r0 + k.subs - 1) / k.subs, kTileRows);
#pragma unroll
            for (int u = 0; u < kTileRows; ++u)
                if (u < m) raw[u] = load<T, V>(x + (int64_t)(r0 + u * k.subs) * a.x_ts);
            float tm[V], tq[V];
#pragma unroll
            for (int i = 0; i < V; ++i) tm[i] = tq[i] = 0.f;
#pragma unroll
            for (int u = 0; u < kTileRows; ++u)
                if (u < m) {
                    float f[V];
                    floats<T, V>(raw[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) tm[i] += f[i];
                }
            const float each = 1.f / m;
#pragma unroll
            for (int i = 0; i < V; ++i) tm[i] *= each;
#pragma unroll
            for (int u = 0; u < kTileRows; ++u)
                if (u < m) {
                    float f[V];
                    floats<T, V>(raw[u], f);
#pragma unroll
                    for (int i = 0; i < V; ++i) tq[i] = fmaf(f[i] - tm[i], f[i] - tm[i], tq[i]);
                }
            // Joins the tile's mean and squares to those before it.
            const float share = (float)m / (n + m), cross = share * n;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = tm[i] - mean[i];
                mean[i] = fmaf(d, share, mean[i]);
                m2[i] += fmaf(d * d, cross, tq[i]);
            }
            n += m;
        }
    tcc::pdl_launch_dependents();
    const int rows = k.n1 - k.n0;
    float *sm_mean = sm, *sm_sq = sm + k.subs * k.cols;
    if (k.on)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            sm_mean[k.sub * k.cols + k.c + i] = mean[i];
            sm_sq[k.sub * k.cols + k.c + i] = m2[i];
        }
    __syncthreads();
    for (int c = threadIdx.x; c < k.cols; c += blockDim.x) {
        float m = 0.f, q = 0.f;
        const float inv = 1.f / rows;
        for (int s = 0; s < k.subs; ++s) {
            const int cnt = (rows - s + k.subs - 1) / k.subs;
            if (cnt > 0) m = fmaf(cnt * inv, sm_mean[s * k.cols + c], m);
        }
        for (int s = 0; s < k.subs; ++s) {
            const int cnt = (rows - s + k.subs - 1) / k.subs;
            const float d = sm_mean[s * k.cols + c] - m;
            if (cnt > 0) q += fmaf(cnt * d, d, sm_sq[s * k.cols + c]);
        }
        sm_mean[c] = m;
        sm_sq[c] = q;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        float m = 0.f, q = 0.f;
        for (int c = lane; c < a.Cg; c += 32) m += sm_mean[g * a.Cg + c];
        m = lanes_sum(m, 32) / a.Cg;
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
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads) apply_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];                  // [groups][2]: mean, r
    const Block k = block_of_rows<V>(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    tcc::pdl_wait();
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        const float2* p = reinterpret_cast<const float2*>(a.partial) + (int64_t)k.b * a.chunks * a.G + k.g0 + g;
        float m = 0.f, q = 0.f;
        for (int i = lane; i < a.chunks; i += 32) m = fmaf((float)min(a.per, a.N - i * a.per), p[(int64_t)i * a.G].x, m);
        m = lanes_sum(m, 32) / a.N;
        for (int i = lane; i < a.chunks; i += 32) {
            const float2 v = p[(int64_t)i * a.G];
            q += fmaf((float)min(a.per, a.N - i * a.per) * a.Cg * (v.x - m), v.x - m, v.y);
        }
        const float r = 1.f / sqrtf(lanes_sum(q, 32) / ((float)a.N * a.Cg) + a.eps);
        if (lane == 0) {
            sm[2 * g] = m, sm[2 * g + 1] = r;
            if (a.stats && k.chunk == 0)
                *reinterpret_cast<float2*>(a.stats + 2 * ((int64_t)k.b * a.G + k.g0 + g)) = make_float2(m, r);
        }
    }
    __syncthreads();
    if (!k.on) return;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    float mean[V], scale[V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = k.c + i, g = c / a.Cg;
        mean[i] = sm[2 * g];
        scale[i] = sm[2 * g + 1] * (a.w ? to_f(static_cast<const T*>(a.w)[k.c0 + c]) : 1.f);
        bias[i] = a.b ? to_f(static_cast<const T*>(a.b)[k.c0 + c]) : 0.f;
    }
    const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
    const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
    T* y = static_cast<T*>(a.y) + k.b * a.y_bs + k.c0 + k.c;
    constexpr int kU = 4;
    for (int r0 = k.n0 + k.sub; r0 < k.n1; r0 += kU * k.subs) {
        Raw<T, V> rx[kU], rz[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = r0 + u * k.subs;
            if (r >= k.n1) continue;
            rx[u] = load<T, V>(x + (int64_t)r * a.x_ts);
            if (gate) rz[u] = load<T, V>(z + (int64_t)r * a.z_ts);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = r0 + u * k.subs;
            if (r >= k.n1) continue;
            float f[V], zf[V];
            floats<T, V>(rx[u], f);
            if (gate) floats<T, V>(rz[u], zf);
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = forward(fmaf(f[i] - mean[i], scale[i], bias[i]), act, gate, gate ? zf[i] : 0.f);
            store<T, V>(y + (int64_t)r * a.y_ts, f);
        }
    }
}

// partial: [B chunks][2][C] sums of h xh and of h, then [B chunks][G][2] of w h and of w h xh.
template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads) sums_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];                  // [2][subs][cols]
    const Block k = block_of_rows<V>(a);
    const bool act = a.silu != 0, gate = a.z != nullptr;
    float dw[V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dw[i] = db[i] = 0.f;
    if (k.on) {
        float mean[V], r[V], w[V], b[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = k.c0 + k.c + i;
            const float2 s = __ldg(reinterpret_cast<const float2*>(a.stats) + (int64_t)k.b * a.G + c / a.Cg);
            mean[i] = s.x, r[i] = s.y;
            w[i] = a.w ? to_f(static_cast<const T*>(a.w)[c]) : 1.f;
            b[i] = a.b ? to_f(static_cast<const T*>(a.b)[c]) : 0.f;
        }
        const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
        const T* d = static_cast<const T*>(a.dy) + k.b * a.dy_bs + k.c0 + k.c;
        const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
        constexpr int kU = 4;
        for (int r0 = k.n0 + k.sub; r0 < k.n1; r0 += kU * k.subs) {
            Raw<T, V> rx[kU], rd[kU], rz[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                const int n = r0 + u * k.subs;
                if (n >= k.n1) continue;
                rx[u] = load<T, V>(x + (int64_t)n * a.x_ts);
                rd[u] = load<T, V>(d + (int64_t)n * a.dy_ts);
                if (gate) rz[u] = load<T, V>(z + (int64_t)n * a.z_ts);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (r0 + u * k.subs >= k.n1) continue;
                float f[V], df[V], zf[V], dz;
                floats<T, V>(rx[u], f);
                floats<T, V>(rd[u], df);
                if (gate) floats<T, V>(rz[u], zf);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (f[i] - mean[i]) * r[i];
                    const float h = backward(fmaf(xh, w[i], b[i]), df[i], act, gate, gate ? zf[i] : 0.f, &dz);
                    dw[i] = fmaf(h, xh, dw[i]);
                    db[i] += h;
                }
            }
        }
    }
    tcc::pdl_launch_dependents();
    float *s_w = sm, *s_b = sm + k.subs * k.cols;
    if (k.on)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            s_w[k.sub * k.cols + k.c + i] = dw[i];
            s_b[k.sub * k.cols + k.c + i] = db[i];
        }
    __syncthreads();
    float* channel = a.partial + (int64_t)blockIdx.x * 2 * a.C + k.c0;
    for (int c = threadIdx.x; c < k.cols; c += blockDim.x) {
        float u = 0.f, v = 0.f;
        for (int s = 0; s < k.subs; ++s) u += s_w[s * k.cols + c], v += s_b[s * k.cols + c];
        channel[c] = u;
        channel[a.C + c] = v;
        const float w = a.w ? to_f(static_cast<const T*>(a.w)[k.c0 + c]) : 1.f;
        s_w[c] = w * u;
        s_b[c] = w * v;
    }
    __syncthreads();
    float2* group = reinterpret_cast<float2*>(a.partial + (int64_t)a.B * a.chunks * 2 * a.C) + (int64_t)blockIdx.x * a.G + k.g0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        float u = 0.f, v = 0.f;
        for (int c = lane; c < a.Cg; c += 32) u += s_b[g * a.Cg + c], v += s_w[g * a.Cg + c];
        u = lanes_sum(u, 32);
        v = lanes_sum(v, 32);
        if (lane == 0) group[g] = make_float2(u, v);
    }
}

template <typename T, int V>
__global__ void __launch_bounds__(V == 1 ? kMost : kThreads) apply_bwd_kernel(const __grid_constant__ NormArgs a) {
    extern __shared__ float sm[];                  // [groups][2]: means of w h and of w h xh
    const Block k = block_of_rows<V>(a);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    tcc::pdl_launch_dependents();
    tcc::pdl_wait();
    const float2* parts = reinterpret_cast<const float2*>(a.partial + (int64_t)a.B * a.chunks * 2 * a.C);
    for (int g = warp; g < k.ng; g += blockDim.x >> 5) {
        const float2* p = parts + (int64_t)k.b * a.chunks * a.G + k.g0 + g;
        float u = 0.f, v = 0.f;
        for (int i = lane; i < a.chunks; i += 32) u += p[(int64_t)i * a.G].x, v += p[(int64_t)i * a.G].y;
        u = lanes_sum(u, 32);
        v = lanes_sum(v, 32);
        if (lane == 0) sm[2 * g] = u / ((float)a.N * a.Cg), sm[2 * g + 1] = v / ((float)a.N * a.Cg);
    }
    __syncthreads();
    if (!k.on) return;
    const bool act = a.silu != 0, gate = a.z != nullptr;
    float mean[V], r[V], w[V], b[V], s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = k.c + i, g = c / a.Cg;
        const float2 s = __ldg(reinterpret_cast<const float2*>(a.stats) + (int64_t)k.b * a.G + k.g0 + g);
        mean[i] = s.x, r[i] = s.y;
        w[i] = a.w ? to_f(static_cast<const T*>(a.w)[k.c0 + c]) : 1.f;
        b[i] = a.b ? to_f(static_cast<const T*>(a.b)[k.c0 + c]) : 0.f;
        s1[i] = sm[2 * g], s2[i] = sm[2 * g + 1];
    }
    const T* x = static_cast<const T*>(a.x) + k.b * a.x_bs + k.c0 + k.c;
    const T* d = static_cast<const T*>(a.dy) + k.b * a.dy_bs + k.c0 + k.c;
    const T* z = static_cast<const T*>(a.z) + (gate ? k.b * a.z_bs + k.c0 + k.c : 0);
    T* y = static_cast<T*>(a.y) + k.b * a.y_bs + k.c0 + k.c;
    T* dz = static_cast<T*>(a.dz) + (gate ? k.b * a.dz_bs + k.c0 + k.c : 0);
    constexpr int kU = 4;
    for (int r0 = k.n0 + k.sub; r0 < k.n1; r0 += kU * k.subs) {
        Raw<T, V> rx[kU], rd[kU], rz[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int n = r0 + u * k.subs;
            if (n >= k.n1) continue;
            rx[u] = load<T, V>(x + (int64_t)n * a.x_ts);
            rd[u] = load<T, V>(d + (int64_t)n * a.dy_ts);
            if (gate) rz[u] = load<T, V>(z + (int64_t)n * a.z_ts);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int n = r0 + u * k.subs;
            if (n >= k.n1) continue;
            float f[V], df[V], zf[V], dzf[V];
            floats<T, V>(rx[u], f);
            floats<T, V>(rd[u], df);
            if (gate) floats<T, V>(rz[u], zf);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float xh = (f[i] - mean[i]) * r[i];
                const float h = backward(fmaf(xh, w[i], b[i]), df[i], act, gate, gate ? zf[i] : 0.f, &dzf[i]);
                f[i] = r[i] * (h * w[i] - s1[i] - xh * s2[i]);
            }
            store<T, V>(y + (int64_t)n * a.y_ts, f);
            if (gate) store<T, V>(dz + (int64_t)n * a.dz_ts, dzf);
        }
    }
}

// ------------------------------------------------------------------ host side

// Blocks of the one-token backward at most, each of which leaves its sums.
int row_blocks() { return 4 * tcc::sm_count(); }

// Rows of a block of the other form: at least 16, and so many that there are about four
// blocks for every SM.
void cut_rows(int B, int N, int* per, int* chunks) {
    const int64_t want = (4LL * tcc::sm_count() + B - 1) / B;
    int64_t p = (N + want - 1) / want;
    p = p < 16 ? 16 : p;
    *per = (int)p;
    *chunks = (int)((N + p - 1) / p);
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

template <typename T, int V, int K, bool kBackward>
cudaError_t launch_rows(NormArgs a, cudaStream_t st) {
    a.lanes = lanes_of(a.Cg, V, K);
    a.slots = a.G * a.lanes;
    constexpr int kU = kBackward ? (K == 1 ? 2 : 1) : (K == 1 ? 4 : K == 2 ? 2 : 1);
    const int R = a.slots <= kThreads ? kThreads / a.slots : 1;
    const int64_t tiles = ((int64_t)a.B + R * kU - 1) / (R * kU);
    const unsigned columns = (unsigned)((a.slots + kThreads - 1) / kThreads);
    if constexpr (!kBackward) {
        const int64_t most = 8LL * tcc::sm_count();
        rows_fwd_kernel<T, V, K, kU><<<dim3((unsigned)(tiles < most ? tiles : most), columns), kThreads, 0, st>>>(a);
        return cudaPeekAtLastError();
    } else {
        const int64_t most = row_blocks(), blocks = tiles < most ? tiles : most;
        rows_bwd_kernel<T, V, K, kU><<<dim3((unsigned)blocks, columns), kThreads, 0, st>>>(a);
        cudaError_t e = cudaPeekAtLastError();
        if (e != cudaSuccess || (!a.dw && !a.db)) return e;
        return scan::launch_after(weights_kernel, dim3((a.C + 31) / 32, 2), 256, 0, st, true, a.partial, a.dw, a.db, blocks, a.C);
    }
}

template <typename T, int V, bool kBackward>
cudaError_t launch_blocks(NormArgs a, cudaStream_t st) {
    cut_rows(a.B, a.N, &a.per, &a.chunks);
    // Whole groups per block, whole vectors: as many as its threads hold.
    const int unit = V / gcd(a.Cg, V), hold = (V == 1 ? kMost : kThreads) * V / a.Cg;
    a.gb = hold >= a.G ? a.G : hold / unit * unit;
    const int threads = V == 1 && a.gb * a.Cg > kThreads ? kMost : kThreads;
    const int subs = threads / (a.gb * a.Cg / V);
    const dim3 grid((unsigned)(a.B * a.chunks), (unsigned)((a.G + a.gb - 1) / a.gb));
    const size_t sums = 2 * sizeof(float) * (size_t)subs * a.gb * a.Cg, group = 2 * sizeof(float) * (size_t)a.gb;
    if constexpr (!kBackward) {
        stats_kernel<T, V><<<grid, threads, sums, st>>>(a);
        const cudaError_t e = cudaPeekAtLastError();
        return e != cudaSuccess ? e : scan::launch_after(apply_kernel<T, V>, grid, threads, group, st, true, a);
    } else {
        sums_kernel<T, V><<<grid, threads, sums, st>>>(a);
        cudaError_t e = cudaPeekAtLastError();
        if (e != cudaSuccess) return e;
        if ((e = scan::launch_after(apply_bwd_kernel<T, V>, grid, threads, group, st, true, a)) != cudaSuccess ||
            (!a.dw && !a.db))
            return e;
        return scan::launch_after(weights_kernel, dim3((a.C + 31) / 32, 2), 256, 0, st, true, a.partial, a.dw, a.db,
                                  (int64_t)a.B * a.chunks, a.C);
    }
}

// The vector forms need whole 16-byte pieces of every row.
template <typename T, bool kBackward>
cudaError_t launch_norm(const NormArgs& a, bool aligned, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (a.N == 1) {
        if (aligned && lanes_of(a.Cg, V, 1)) return launch_rows<T, V, 1, kBackward>(a, st);
        if (aligned && a.Cg % V == 0) return launch_rows<T, V, kMost / (32 * V), kBackward>(a, st);
        return launch_rows<T, 1, kNarrow / 32, kBackward>(a, st);
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
    cut_rows(B, N, &per, &chunks);
    const size_t blocks = sizeof(float) * (size_t)B * chunks * (2 * (size_t)C + 2 * (size_t)G);
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
