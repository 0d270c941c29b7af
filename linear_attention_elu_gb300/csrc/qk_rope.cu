// Per-head RMS norm of queries and keys and the position rotation, in the pass
// that takes them from the token-major projection [B, N, H, D] to the
// head-major layout [B, H, N, D] of the attention entries; and its backward.
//
// Forward, per row x (one token of one head), with r = 1 / sqrt(mean x^2 + eps):
//   u = r w x (or x without the norm);  a rotated pair (a, b) of u becomes
//   (a cos t - b sin t, b cos t + a sin t),  t = pos[axis_i] f_i.
// Backward, from g_out: g = R^T g_out (the rotation by -t),
//   dw = sum over rows of g xh,   dx = r (w g - xh mean(w g xh)),   xh = r x.
//
// Angles. A pair's table entry holds its frequency as a whole number of 2^-64
// turns, so pos * step modulo 2^64 is the angle's fraction of a turn, exact for
// every position (wrap-around is the reduction modulo 2 pi); its top 32 bits go
// through sincospif. No table over positions, no loss for far tokens.
//
// What bounds it: every value is read once and written once (the backward also
// reads the gradient), two dozen operations each: HBM bandwidth, with 66 to 74 % of the
// issue slots used where there is a norm. A group of D/8
// lanes owns one token and walks its heads, so the angles are computed once per
// token; the stores of neighbouring groups are neighbouring rows of one head. A lane
// holds both values of its pairs: eight neighbours of a row, or, for pairs (i, i + R),
// four and their four partners (with eight neighbours there too, their partners came
// by shuffles: B=16 N=8192 H=8+8 D=128 forward 221 us against 189). The next heads'
// rows are in flight under the current ones. Weights are folded into the cos and sin
// registers. Statistics and sums are fp32.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "overlap.h"
#include "tc_common.cuh"

namespace la {

namespace {

constexpr int kThreads = 256;

// One of q and k: rows at x + b bs + n ts + h D (backward: the gradient dx
// written at the same kind of address), head-major rows at o + ((b H + h) N + n) D.
struct Side {
    const void* x;
    int64_t x_bs, x_ts;
    const void* w;        // [D] or null
    void* y;              // forward: head-major output; backward: dx
    int64_t y_bs, y_ts;   // backward only
    const void* go;       // backward: head-major gradient of the output
    int H;
};

struct Args {
    Side s[2];
    const int32_t* pos;       // [B, N, axes]
    const longlong2* table;   // [R]: (step in 2^-64 turns, axis)
    float* partial;           // backward with the norm: [blocks][2][D]
    int64_t tokens;           // B N
    int axes, R, N, D, norm, heads_per_block;
    float eps, inv_D;
};

template <typename T> struct Raw8;   // eight consecutive values of a row as stored
template <> struct Raw8<__nv_bfloat16> {
    uint4 v;
    template <bool kInter>
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int o0, int o1) {
        if constexpr (kInter) {
            v = __ldg(reinterpret_cast<const uint4*>(p + o0));
        } else {
            const uint2 lo = __ldg(reinterpret_cast<const uint2*>(p + o0)), hi = __ldg(reinterpret_cast<const uint2*>(p + o1));
            v = make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
    }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    }
    template <bool kInter>
    static __device__ __forceinline__ void store(__nv_bfloat16* p, int o0, int o1, const float (&f)[8]) {
        const uint4 u = make_uint4(tcc::pack_bf16(f[0], f[1]), tcc::pack_bf16(f[2], f[3]),
                                   tcc::pack_bf16(f[4], f[5]), tcc::pack_bf16(f[6], f[7]));
        if constexpr (kInter) {
            *reinterpret_cast<uint4*>(p + o0) = u;
        } else {
            *reinterpret_cast<uint2*>(p + o0) = make_uint2(u.x, u.y);
            *reinterpret_cast<uint2*>(p + o1) = make_uint2(u.z, u.w);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    template <bool kInter>
    __device__ __forceinline__ void load(const float* p, int o0, int o1) {
        a = __ldg(reinterpret_cast<const float4*>(p + o0));
        b = __ldg(reinterpret_cast<const float4*>(p + o1));
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    template <bool kInter>
    static __device__ __forceinline__ void store(float* p, int o0, int o1, const float (&f)[8]) {
        *reinterpret_cast<float4*>(p + o0) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(p + o1) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

// Features of lane l: o0 .. o0 + 3 and o1 .. o1 + 3, so that a lane holds both
// values of its pairs. Pairs (2i, 2i + 1), and features past the rotated ones: eight
// neighbours. Pairs (i, i + R): four and their four partners.
template <bool kInter>
__device__ __forceinline__ void lane_features(int R, int l, int* o0, int* o1) {
    const bool halves = !kInter && 8 * l < 2 * R;
    *o0 = halves ? 4 * l : 8 * l;
    *o1 = halves ? R + 4 * l : 8 * l + 4;
}

// cos and sin of pair i at token t. A pair whose axis is past the last given one
// takes the last, so no position is read out of range.
__device__ __forceinline__ void pair_angle(const Args& a, int64_t t, int i, float* c, float* s) {
    const longlong2 e = __ldg(a.table + i);
    const int ax = min(max((int)e.y, 0), a.axes - 1);
    const uint64_t turn = (uint64_t)(int64_t)__ldg(a.pos + t * a.axes + ax) * (uint64_t)e.x;
    sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, s, c);   // 2^-31 half-turns
}

// Rotation of a lane's eight values: out = x c + partner s (s carries the sign).
// Lanes past the rotated features get c = 1, s = 0 and must use a zero partner.
template <bool kInter>
__device__ __forceinline__ void lane_angles(const Args& a, int64_t t, int l, float (&c)[8],
                                            float (&s)[8]) {
    if (8 * l >= 2 * a.R) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
        return;
    }
    if constexpr (kInter) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float cc, ss;
            pair_angle(a, t, 4 * l + j / 2, &cc, &ss);
            c[j] = c[j + 1] = cc;
            s[j] = -ss;
            s[j + 1] = ss;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float cc, ss;
            pair_angle(a, t, 4 * l + j, &cc, &ss);
            c[j] = c[j + 4] = cc;
            s[j] = -ss;
            s[j + 4] = ss;
        }
    }
}

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The partners of a lane's values; zeros past the rotated features.
template <bool kInter>
__device__ __forceinline__ void partner_values(const float (&x)[8], bool rot, float (&p)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = rot ? x[kInter ? j ^ 1 : j ^ 4] : 0.f;
}

// Forward. kLanes: lanes per row (D / 8 rounded up to a power of two; the lanes
// past D / 8 carry zeros). blockIdx.y: a range of the Hq + Hk heads.
// Three blocks of 256 threads per SM for bf16 (B=16 N=8192 H=8+8 D=128: 189 us; four,
// which spill, 210; four with two heads in flight 197), two for fp32, whose rows need
// twice the registers (16 images of 32 x 32: 24.5 us).
template <typename T, int kLanes, bool kInter>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 3 : 2) rope_fwd_kernel(const __grid_constant__ Args a) {
    constexpr int kRows = kThreads / kLanes, kU = 4;   // heads in flight per group
    const int l = threadIdx.x % kLanes;
    const int64_t t_raw = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
    const bool live = t_raw < a.tokens && 8 * l < a.D;
    const int64_t t = min(t_raw, a.tokens - 1);
    const int64_t b = t / a.N, n = t - b * a.N;
    const bool rot = 8 * l < 2 * a.R;
    int o0, o1;
    lane_features<kInter>(a.R, l, &o0, &o1);
    const int h_begin = blockIdx.y * a.heads_per_block;
    const int h_end = min(h_begin + a.heads_per_block, a.s[0].H + a.s[1].H);
    // Heads h .. h + kU - 1 of q and k together, as far as they belong to one side.
    Raw8<T> raw[kU];
    auto fetch = [&](int h) {
        const int side = h >= a.s[0].H;
        const Side& sd = a.s[side];
        const int hs = side ? h - a.s[0].H : h, left = min(h_end - h, sd.H - hs);
        const T* xp = static_cast<const T*>(sd.x) + b * sd.x_bs + n * sd.x_ts + (int64_t)hs * a.D;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            raw[u].zero();
            if (live && u < left) raw[u].template load<kInter>(xp + (int64_t)u * a.D, o0, o1);
        }
    };
    fetch(h_begin);                                    // in flight under the angles
    float c[8], s[8], cw[8], sw[8];
    lane_angles<kInter>(a, t, l, c, s);
    int last = -1;
#pragma unroll 1
    for (int h = h_begin; h < h_end;) {
        const int side = h >= a.s[0].H;
        const Side& sd = a.s[side];
        const int hs = side ? h - a.s[0].H : h, left = min(min(h_end - h, sd.H - hs), kU);
        if (side != last) {
            // Weights folded into the rotation: c w and s w_partner.
            last = side;
            if (sd.w != nullptr) {
                Raw8<T> wr;
                wr.zero();
                if (8 * l < a.D) wr.template load<kInter>(static_cast<const T*>(sd.w), o0, o1);
                float w[8], wp[8];
                wr.get(w);
                partner_values<kInter>(w, rot, wp);
#pragma unroll
                for (int j = 0; j < 8; ++j) cw[j] = c[j] * w[j], sw[j] = s[j] * wp[j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) cw[j] = c[j], sw[j] = s[j];
            }
        }
        Raw8<T> cur[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) cur[u] = raw[u];
        h += left;
        if (h < h_end) fetch(h);                       // in flight under this batch
        T* yp = static_cast<T*>(sd.y) + ((b * sd.H + hs) * a.N + n) * a.D;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            float x[8], p[8], r = 1.f;
            cur[u].get(x);
            partner_values<kInter>(x, rot, p);
            if (a.norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                r = rsqrtf(group_sum<kLanes>(ss) * a.inv_D + a.eps);
            }
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = r * fmaf(x[j], cw[j], p[j] * sw[j]);
            if (live && u < left) Raw8<T>::template store<kInter>(yp + (int64_t)u * a.N * a.D, o0, o1, y);
        }
    }
}

// Adds a block's per-lane dw sums (v[8] for a lane's eight features of every row
// group) in a fixed order and writes D floats at out.
template <int kLanes>
__device__ __forceinline__ void block_dw(float (&v)[8], float (*red)[kMaxDim], int l, int o0,
                                         int o1, int D, float* out) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1) v[j] += __shfl_xor_sync(0xffffffffu, v[j], o);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane < kLanes && 8 * l < D)
#pragma unroll
        for (int j = 0; j < 8; ++j) red[warp][j < 4 ? o0 + j : o1 + j - 4] = v[j];
    __syncthreads();
    if ((int)threadIdx.x < D) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t += red[w][threadIdx.x];
        out[threadIdx.x] = t;
    }
    __syncthreads();
}

// Backward. A block walks token tiles blockIdx.x, + gridDim.x, ..., so that dw
// leaves as one partial row per block.
// With the norm, whose weight sums fill the registers, two blocks per SM and the next
// heads' rows in flight (B=4 N=8191 H=16+4 D=64 bf16 61 us; three blocks without the
// rows ahead 65); without it three blocks, whose warps hide the loads by themselves
// (B=4 N=9216 H=12+12 D=128 78 us; two blocks with the rows ahead 94).
template <typename T, int kLanes, bool kInter, bool kNorm>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 && !kNorm ? 3 : 2) rope_bwd_kernel(const __grid_constant__ Args a) {
    constexpr int kRows = kThreads / kLanes, kU = 2;
    const int l = threadIdx.x % kLanes;
    const bool rot = 8 * l < 2 * a.R;
    int o0, o1;
    lane_features<kInter>(a.R, l, &o0, &o1);
    const int h_begin = blockIdx.y * a.heads_per_block, h_end = h_begin + a.heads_per_block;
    const int64_t tiles = (a.tokens + kRows - 1) / kRows;
    float dw[2][8] = {};
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t t_raw = tile * kRows + threadIdx.x / kLanes;
        const bool live = t_raw < a.tokens && 8 * l < a.D;
        const int64_t t = min(t_raw, a.tokens - 1);
        const int64_t b = t / a.N, n = t - b * a.N;
        // This block's heads of each side, and the rows of the next batch.
        const int h0[2] = {min(h_begin, a.s[0].H), max(h_begin - a.s[0].H, 0)};
        const int h1[2] = {min(h_end, a.s[0].H), min(max(h_end - a.s[0].H, 0), a.s[1].H)};
        Raw8<T> graw[kU], xraw[kU];
        auto fetch = [&](int side, int h) {
            const Side& sd = a.s[side];
            const T* gp = static_cast<const T*>(sd.go) + ((b * sd.H + h) * a.N + n) * a.D;
            const T* xp = kNorm ? static_cast<const T*>(sd.x) + b * sd.x_bs + n * sd.x_ts + (int64_t)h * a.D
                                : nullptr;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                graw[u].zero();
                xraw[u].zero();
                if (live && h + u < h1[side]) {
                    graw[u].template load<kInter>(gp + (int64_t)u * a.N * a.D, o0, o1);
                    if (kNorm) xraw[u].template load<kInter>(xp + (int64_t)u * a.D, o0, o1);
                }
            }
        };
        if constexpr (kNorm) {                         // in flight under the angles
            if (h0[0] < h1[0]) fetch(0, h0[0]);
            else if (h0[1] < h1[1]) fetch(1, h0[1]);
        }
        float c[8], s[8];
        lane_angles<kInter>(a, t, l, c, s);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const Side& sd = a.s[side];
            if (h0[side] >= h1[side]) continue;
            float w[8];
            if (kNorm && sd.w != nullptr && 8 * l < a.D) {
                Raw8<T> wr;
                wr.template load<kInter>(static_cast<const T*>(sd.w), o0, o1);
                wr.get(w);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
            }
            T* yp = static_cast<T*>(sd.y) + b * sd.y_bs + n * sd.y_ts;
            for (int h = h0[side]; h < h1[side]; h += kU) {
                if constexpr (!kNorm) fetch(side, h);
                Raw8<T> gcur[kU], xcur[kU];
#pragma unroll
                for (int u = 0; u < kU; ++u) gcur[u] = graw[u], xcur[u] = xraw[u];
                if constexpr (kNorm) {                 // in flight under this batch
                    if (h + kU < h1[side]) fetch(side, h + kU);
                    else if (side == 0 && h0[1] < h1[1]) fetch(1, h0[1]);
                }
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    float go[8], p[8], g[8], y[8];
                    gcur[u].get(go);
                    partner_values<kInter>(go, rot, p);
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] = fmaf(go[j], c[j], -p[j] * s[j]);
                    if constexpr (kNorm) {
                        float x[8], ss = 0.f, dot = 0.f;
                        xcur[u].get(x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            ss = fmaf(x[j], x[j], ss);
                            dot = fmaf(g[j] * w[j], x[j], dot);
                        }
                        ss = group_sum<kLanes>(ss);
                        dot = group_sum<kLanes>(dot);
                        // A slot that holds no row (past the last token or head) adds nothing to the
                        // weights' sums, without an epsilon either (0 times infinity).
                        const bool row = t_raw < a.tokens && h + u < h1[side];
                        const float r = row ? rsqrtf(ss * a.inv_D + a.eps) : 0.f;
                        // dx = r (w g - xh mean(w g xh)) with xh = r x of order 1: r^3 alone passes
                        // fp32's range for rows below 1e-13.
                        const float k = r * (r * dot * a.inv_D);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float xh = r * x[j];
                            y[j] = fmaf(r * w[j], g[j], -k * xh);
                            dw[side][j] = fmaf(g[j], xh, dw[side][j]);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = g[j];
                    }
                    if (live && h + u < h1[side]) Raw8<T>::template store<kInter>(yp + (int64_t)(h + u) * a.D, o0, o1, y);
                }
            }
        }
    }
    if constexpr (kNorm) {
        __shared__ float red[kThreads / 32][kMaxDim];
        float* out = a.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 * a.D;
        block_dw<kLanes>(dw[0], red, l, o0, o1, a.D, out);
        block_dw<kLanes>(dw[1], red, l, o0, o1, a.D, out + a.D);
    }
}

// Any D, R, stride and alignment: one warp per row, lane i owning features
// i, i + 32, ...; partners through shared memory. Rows are walked token-major
// so that a warp's dw sums stay in registers.
template <typename T, bool kBwd>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ Args a, int inter) {
    constexpr int kWarps = kThreads / 32, kE = kMaxDim / 32;
    __shared__ float buf[kWarps][kMaxDim];
    __shared__ float red[kWarps][kMaxDim];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* row = buf[warp];
    float dw[2][kE] = {};
    for (int side = 0; side < 2; ++side) {
        const Side& sd = a.s[side];
        const int64_t rows = a.tokens * sd.H;
        for (int64_t i = (int64_t)blockIdx.x * kWarps + warp; i < rows; i += (int64_t)gridDim.x * kWarps) {
            const int64_t t = i / sd.H;
            const int h = (int)(i - t * sd.H);
            const int64_t b = t / a.N, n = t - b * a.N;
            const int64_t hm = ((b * sd.H + h) * a.N + n) * a.D;   // head-major row
            const T* xr = static_cast<const T*>(sd.x) + b * sd.x_bs + n * sd.x_ts + (int64_t)h * a.D;
            float x[kE], w[kE], v[kE];
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int e = lane + 32 * j;
                const bool in = e < a.D;
                x[j] = in && (!kBwd || a.norm) ? to_f(xr[e]) : 0.f;
                w[j] = in && sd.w ? to_f(static_cast<const T*>(sd.w)[e]) : 1.f;
                ss = fmaf(x[j], x[j], ss);
                v[j] = kBwd ? (in ? to_f(static_cast<const T*>(sd.go)[hm + e]) : 0.f) : x[j];
            }
            const float r = a.norm ? rsqrtf(group_sum<32>(ss) * a.inv_D + a.eps) : 1.f;
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int e = lane + 32 * j;
                if (!kBwd) v[j] *= r * w[j];
                if (e < a.D) row[e] = v[j];
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int e = lane + 32 * j;
                if (e >= 2 * a.R) continue;
                const bool low = inter ? (e & 1) == 0 : e < a.R;
                const int pr = inter ? e >> 1 : (low ? e : e - a.R);
                const int pe = inter ? e ^ 1 : (low ? e + a.R : e - a.R);
                float c, s;
                pair_angle(a, t, pr, &c, &s);
                if (low != kBwd) s = -s;
                v[j] = fmaf(v[j], c, row[pe] * s);
            }
            __syncwarp();
            if (!kBwd) {
#pragma unroll
                for (int j = 0; j < kE; ++j)
                    if (lane + 32 * j < a.D)
                        static_cast<T*>(sd.y)[hm + lane + 32 * j] = from_f<T>(v[j]);
            } else {
                T* yr = static_cast<T*>(sd.y) + b * sd.y_bs + n * sd.y_ts + (int64_t)h * a.D;
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < kE; ++j) dot = fmaf(v[j] * w[j], x[j], dot);
                const float k = a.norm ? r * (r * group_sum<32>(dot) * a.inv_D) : 0.f;
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    const int e = lane + 32 * j;
                    if (e >= a.D) continue;
                    const float xh = r * x[j];
                    yr[e] = from_f<T>(a.norm ? fmaf(r * w[j], v[j], -k * xh) : v[j]);
                    if (side == 0) dw[0][j] = fmaf(v[j], xh, dw[0][j]);
                    else dw[1][j] = fmaf(v[j], xh, dw[1][j]);
                }
            }
        }
    }
    if (kBwd && a.norm) {
        for (int side = 0; side < 2; ++side) {
#pragma unroll
            for (int j = 0; j < kE; ++j) red[warp][lane + 32 * j] = side ? dw[1][j] : dw[0][j];
            __syncthreads();
            if ((int)threadIdx.x < a.D) {
                float t = 0.f;
                for (int i = 0; i < kWarps; ++i) t += red[i][threadIdx.x];
                a.partial[((int64_t)blockIdx.x * 2 + side) * a.D + threadIdx.x] = t;
            }
            __syncthreads();
        }
    }
}

// dw[side][d] = sum over blocks of partial[block][side][d], in a fixed order.
// A block sums 32 columns: thread (x, y) the rows y, y + 8, ...
__global__ void __launch_bounds__(256) rope_dw_kernel(const float* __restrict__ partial, int blocks,
                                                      int D, float* dwq, float* dwk) {
    tcc::pdl_wait();
    __shared__ float red[8][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + x;   // of 2 D
    float t = 0.f;
    if (col < 2 * D)
        for (int i = y; i < blocks; i += 8) t += partial[(int64_t)i * 2 * D + col];
    red[y][x] = t;
    __syncthreads();
    if (y == 0 && col < 2 * D) {
#pragma unroll
        for (int i = 1; i < 8; ++i) t += red[i][x];
        float* out = col < D ? dwq : dwk;
        if (out) out[col < D ? col : col - D] = t;
    }
}

// Blocks of the backward: four per SM, each walking token tiles; fewer when
// there are fewer tiles. Bounds the partial sums' workspace.
constexpr int kBwdBlocksPerSm = 4;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The vector kernels need whole 16-byte pieces: eight values per lane for bf16
// (two pieces for fp32), and partner groups of four values.
bool vector_ok(const Args& a, size_t eb, bool bwd) {
    if (a.D % 8 || a.R % 4) return false;
    for (const Side& s : a.s) {
        if (s.H == 0) continue;
        if (!aligned16(s.y) || (s.w && !aligned16(s.w))) return false;
        if (s.x && (!aligned16(s.x) || (s.x_bs * (int64_t)eb) % 16 || (s.x_ts * (int64_t)eb) % 16))
            return false;
        if (bwd && (!aligned16(s.go) || (s.y_bs * (int64_t)eb) % 16 || (s.y_ts * (int64_t)eb) % 16))
            return false;
    }
    return true;
}

int lanes_of(int D) { return D <= 32 ? 4 : D <= 64 ? 8 : 16; }

// Heads walked by one block: all of a token's heads share its angles, but with
// few tokens the heads are spread over blocks until the SMs have two each.
int heads_per_block(int64_t tiles, int heads) {
    int per = heads;
    while (per > 1 && tiles * ((heads + per - 1) / per) < 2 * tcc::sm_count()) per = (per + 1) / 2;
    return per;
}

template <typename T, int kLanes>
cudaError_t fwd_vec(Args& a, bool inter, cudaStream_t st) {
    const int64_t tiles = (a.tokens + kThreads / kLanes - 1) / (kThreads / kLanes);
    const int heads = a.s[0].H + a.s[1].H;
    a.heads_per_block = heads_per_block(tiles, heads);
    const dim3 grid((unsigned)tiles, (heads + a.heads_per_block - 1) / a.heads_per_block);
    if (inter) rope_fwd_kernel<T, kLanes, true><<<grid, kThreads, 0, st>>>(a);
    else rope_fwd_kernel<T, kLanes, false><<<grid, kThreads, 0, st>>>(a);
    return cudaPeekAtLastError();
}

template <typename T, int kLanes>
cudaError_t bwd_vec(Args& a, bool inter, int* blocks, cudaStream_t st) {
    const int64_t tiles = (a.tokens + kThreads / kLanes - 1) / (kThreads / kLanes);
    const int heads = a.s[0].H + a.s[1].H;
    const int64_t most = (int64_t)kBwdBlocksPerSm * tcc::sm_count();
    a.heads_per_block = heads_per_block(tiles, heads);
    const int gy = (heads + a.heads_per_block - 1) / a.heads_per_block;
    const int64_t gx = tiles < most / gy ? tiles : (most / gy > 0 ? most / gy : 1);
    const dim3 grid((unsigned)gx, gy);
    *blocks = (int)(gx * gy);
    if (a.norm) {
        if (inter) rope_bwd_kernel<T, kLanes, true, true><<<grid, kThreads, 0, st>>>(a);
        else rope_bwd_kernel<T, kLanes, false, true><<<grid, kThreads, 0, st>>>(a);
    } else {
        if (inter) rope_bwd_kernel<T, kLanes, true, false><<<grid, kThreads, 0, st>>>(a);
        else rope_bwd_kernel<T, kLanes, false, false><<<grid, kThreads, 0, st>>>(a);
    }
    return cudaPeekAtLastError();
}

template <typename T>
cudaError_t run(Args& a, bool bwd, bool inter, int* blocks, cudaStream_t st) {
    if (vector_ok(a, sizeof(T), bwd)) {
        switch (lanes_of(a.D)) {
            case 4: return bwd ? bwd_vec<T, 4>(a, inter, blocks, st) : fwd_vec<T, 4>(a, inter, st);
            case 8: return bwd ? bwd_vec<T, 8>(a, inter, blocks, st) : fwd_vec<T, 8>(a, inter, st);
            default: return bwd ? bwd_vec<T, 16>(a, inter, blocks, st) : fwd_vec<T, 16>(a, inter, st);
        }
    }
    const int64_t rows = a.tokens * (a.s[0].H > a.s[1].H ? a.s[0].H : a.s[1].H);
    const int64_t want = (rows + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t most = (int64_t)kBwdBlocksPerSm * tcc::sm_count();
    const int grid = (int)(want < most ? want : most);
    *blocks = grid;
    if (bwd) rope_any_kernel<T, true><<<grid, kThreads, 0, st>>>(a, inter);
    else rope_any_kernel<T, false><<<grid, kThreads, 0, st>>>(a, inter);
    return cudaPeekAtLastError();
}

// What both directions read, for the checks of overlap.
struct Operands {
    Rows x[2], w[2], pos, table;
};
Operands operands(const Args& a, int B, int N, int D, la_dtype dt, const int32_t* pos, int axes, const int64_t* table,
                  int pairs) {
    const int64_t eb = dt == LA_BF16 ? 2 : 4;
    Operands o;
    for (int i = 0; i < 2; ++i) {
        const Side& sd = a.s[i];
        o.x[i] = rows_of(sd.H ? sd.x : nullptr, B, N, (int64_t)sd.H * D, sd.x_bs, sd.x_ts, eb);
        o.w[i] = block_of(sd.H ? sd.w : nullptr, D * eb);
    }
    o.pos = block_of(pairs > 0 ? pos : nullptr, (int64_t)B * N * axes * 4);
    o.table = block_of(pairs > 0 ? table : nullptr, (int64_t)pairs * 16);
    return o;
}

// v turns modulo one, as a multiple of 2^-64: in two exact steps of 32 bits of the fraction.
uint64_t turn_bits(double v) {
    if (v < 0) return 0 - turn_bits(-v);
    v -= floor(v);
    const double hi = floor(v * 4294967296.0), lo = (v * 4294967296.0 - hi) * 4294967296.0;
    return ((uint64_t)hi << 32) + (uint64_t)llrint(lo);
}

bool elem_aligned(const void* p, la_dtype dt) {
    return (reinterpret_cast<uintptr_t>(p) & (dt == LA_BF16 ? 1 : 3)) == 0;
}

la_status check_shape(int B, int N, int Hq, int Hk, int D, la_dtype dt, const int32_t* pos, int axes,
                      const int64_t* table, int pairs, float eps, int layout) {
    if (B < 0 || N < 0 || Hq < 0 || Hk < 0 || D < 1) return LA_ERR_INVALID_ARG;
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (pairs < 0 || 2 * (int64_t)pairs > D || axes < 1) return LA_ERR_INVALID_ARG;
    if (layout != LA_ROPE_HALVES && layout != LA_ROPE_INTERLEAVED) return LA_ERR_INVALID_ARG;
    if (!isfinite(eps) || eps < 0.f) return LA_ERR_INVALID_ARG;
    if (D > kMaxDim || axes > LA_ROPE_MAX_AXES) return LA_ERR_UNSUPPORTED;
    // A token's heads map to grid.y, and tokens to 31-bit block counts.
    if ((int64_t)Hq + Hk > 65535 || (int64_t)B * N > (int64_t)1 << 31) return LA_ERR_UNSUPPORTED;
    if ((int64_t)B * N == 0 || Hq + Hk == 0) return LA_OK;
    if (pairs > 0) {
        if (!pos || !table || (reinterpret_cast<uintptr_t>(pos) & 3)) return LA_ERR_INVALID_ARG;
        if (!aligned16(table)) return LA_ERR_INVALID_ARG;
    }
    return LA_OK;
}

}  // namespace

}  // namespace la

extern "C" {

la_status la_rope_table(const double* inv_freq, const int32_t* axis, int pairs, int axes,
                        int64_t* table) {
    if (pairs < 0 || axes < 1 || (pairs > 0 && (!inv_freq || !table))) return LA_ERR_INVALID_ARG;
    if (axes > LA_ROPE_MAX_AXES) return LA_ERR_UNSUPPORTED;
    for (int i = 0; i < pairs; ++i) {
        if (!isfinite(inv_freq[i])) return LA_ERR_INVALID_ARG;
        const int ax = axis ? axis[i] : 0;
        if (ax < 0 || ax >= axes) return LA_ERR_INVALID_ARG;
        // Turns per position as the sum of two doubles (1 / (2 pi) is such a sum, the product's
        // rounding is recovered by a fused multiply-add), so that a step is exact to its last
        // unit: far positions multiply its error. Whole turns fall away. (volatile: the rounding
        // is of the product as it stands, whatever the compiler contracts.)
        const volatile double turns = inv_freq[i] * 0.15915494309189535;
        const double rest = fma(inv_freq[i], 0.15915494309189535, -turns) + inv_freq[i] * -9.839338337591243e-18;
        table[2 * i] = (int64_t)(la::turn_bits(turns) + la::turn_bits(rest));
        table[2 * i + 1] = ax;
    }
    return LA_OK;
}

la_status la_qk_norm_rope_fwd(const void* q, int64_t q_batch, int64_t q_token, const void* k,
                              int64_t k_batch, int64_t k_token, const void* wq, const void* wk,
                              const int32_t* pos, int axes, const int64_t* table, int pairs,
                              void* qo, void* ko, int B, int N, int Hq, int Hk, int D, la_dtype dt,
                              int norm, float eps, int layout, la_stream_t stream) {
    la_status s = la::check_shape(B, N, Hq, Hk, D, dt, pos, axes, table, pairs, eps, layout);
    if (s != LA_OK) return s;
    if ((wq || wk) && !norm) return LA_ERR_INVALID_ARG;
    const int64_t tokens = (int64_t)B * N;
    if (tokens == 0 || Hq + Hk == 0) return LA_OK;
    la::Args a = {};
    a.s[0] = {q, q_batch, q_token, wq, qo, 0, 0, nullptr, Hq};
    a.s[1] = {k, k_batch, k_token, wk, ko, 0, 0, nullptr, Hk};
    for (const la::Side& sd : a.s)
        if (sd.H > 0 && (!sd.x || !sd.y || !la::elem_aligned(sd.x, dt) || !la::elem_aligned(sd.y, dt) ||
                         !la::elem_aligned(sd.w, dt)))
            return LA_ERR_INVALID_ARG;
    {
        const la::Operands o = la::operands(a, B, N, D, dt, pos, axes, table, pairs);
        const int64_t eb = dt == LA_BF16 ? 2 : 4;
        const la::Rows yq = la::block_of(Hq ? qo : nullptr, tokens * Hq * D * eb);
        const la::Rows yk = la::block_of(Hk ? ko : nullptr, tokens * Hk * D * eb);
        if (la::overlap(yq, yk) || la::overlaps_any(yq, {o.x[0], o.x[1], o.w[0], o.w[1], o.pos, o.table}) ||
            la::overlaps_any(yk, {o.x[0], o.x[1], o.w[0], o.w[1], o.pos, o.table}))
            return LA_ERR_INVALID_ARG;
    }
    a.pos = pos;
    a.table = reinterpret_cast<const longlong2*>(table);
    a.tokens = tokens;
    a.axes = axes, a.R = pairs, a.N = N, a.D = D, a.norm = norm ? 1 : 0, a.eps = eps, a.inv_D = 1.f / (float)D;
    int blocks = 0;
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dt == LA_BF16
                              ? la::run<__nv_bfloat16>(a, false, layout == LA_ROPE_INTERLEAVED, &blocks, st)
                              : la::run<float>(a, false, layout == LA_ROPE_INTERLEAVED, &blocks, st);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_qk_norm_rope_bwd_workspace_size(int B, int N, int Hq, int Hk, int D, size_t* bytes) {
    if (!bytes || B < 0 || N < 0 || Hq < 0 || Hk < 0 || D < 1) return LA_ERR_INVALID_ARG;
    if (D > la::kMaxDim || (int64_t)Hq + Hk > 65535) return LA_ERR_UNSUPPORTED;
    // One [2, D] row of partial weight gradients per block: at most four blocks
    // per SM, or one per head range when there are more head ranges than that.
    const int64_t most = (int64_t)la::kBwdBlocksPerSm * la::tcc::sm_count();
    const int64_t blocks = most > (int64_t)Hq + Hk ? most : (int64_t)Hq + Hk;
    *bytes = (size_t)(blocks * 2 * D * 4 + 255) / 256 * 256;
    return LA_OK;
}

la_status la_qk_norm_rope_bwd(const void* q, int64_t q_batch, int64_t q_token, const void* k,
                              int64_t k_batch, int64_t k_token, const void* wq, const void* wk,
                              const int32_t* pos, int axes, const int64_t* table, int pairs,
                              const void* dqo, const void* dko, void* dq, int64_t dq_batch,
                              int64_t dq_token, void* dk, int64_t dk_batch, int64_t dk_token,
                              float* dwq, float* dwk, int B, int N, int Hq, int Hk, int D,
                              la_dtype dt, int norm, float eps, int layout, void* workspace,
                              size_t workspace_bytes, la_stream_t stream) {
    la_status s = la::check_shape(B, N, Hq, Hk, D, dt, pos, axes, table, pairs, eps, layout);
    if (s != LA_OK) return s;
    if ((wq || wk || dwq || dwk) && !norm) return LA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(dwq) & 3) || (reinterpret_cast<uintptr_t>(dwk) & 3))
        return LA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const int64_t tokens = (int64_t)B * N;
    if (tokens == 0 || Hq + Hk == 0) {
        // No rows: the weight gradients are zero.
        if (dwq && cudaMemsetAsync(dwq, 0, (size_t)D * 4, st)) return LA_ERR_CUDA;
        if (dwk && cudaMemsetAsync(dwk, 0, (size_t)D * 4, st)) return LA_ERR_CUDA;
        return LA_OK;
    }
    la::Args a = {};
    a.s[0] = {norm ? q : nullptr, q_batch, q_token, wq, dq, dq_batch, dq_token, dqo, Hq};
    a.s[1] = {norm ? k : nullptr, k_batch, k_token, wk, dk, dk_batch, dk_token, dko, Hk};
    for (const la::Side& sd : a.s) {
        if (sd.H == 0) continue;
        if ((norm && !sd.x) || !sd.y || !sd.go || !la::elem_aligned(sd.x, dt) ||
            !la::elem_aligned(sd.y, dt) || !la::elem_aligned(sd.go, dt) || !la::elem_aligned(sd.w, dt))
            return LA_ERR_INVALID_ARG;
        if (!la::rows_disjoint(B, N, (int64_t)sd.H * D, sd.y_bs, sd.y_ts)) return LA_ERR_INVALID_ARG;
    }
    if (norm) {
        size_t need = 0;
        if ((s = la_qk_norm_rope_bwd_workspace_size(B, N, Hq, Hk, D, &need)) != LA_OK) return s;
        if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)
            return LA_ERR_WORKSPACE;
    }
    {
        const la::Operands o = la::operands(a, B, N, D, dt, pos, axes, table, pairs);
        const int64_t eb = dt == LA_BF16 ? 2 : 4;
        la::Rows dx[2], go[2];
        for (int i = 0; i < 2; ++i) {
            const la::Side& sd = a.s[i];
            dx[i] = la::rows_of(sd.H ? sd.y : nullptr, B, N, (int64_t)sd.H * D, sd.y_bs, sd.y_ts, eb);
            go[i] = la::block_of(sd.H ? sd.go : nullptr, tokens * sd.H * D * eb);
        }
        // dx may be its x itself: the lanes that read a row's values replace them.
        for (int i = 0; i < 2; ++i)
            if (la::overlaps_any(dx[i], {dx[1 - i], o.x[1 - i], go[0], go[1], o.w[0], o.w[1], o.pos, o.table}) ||
                (!la::same_rows(dx[i], o.x[i]) && la::overlap(dx[i], o.x[i])))
                return LA_ERR_INVALID_ARG;
    }
    a.pos = pos;
    a.table = reinterpret_cast<const longlong2*>(table);
    a.partial = static_cast<float*>(workspace);
    a.tokens = tokens;
    a.axes = axes, a.R = pairs, a.N = N, a.D = D, a.norm = norm ? 1 : 0, a.eps = eps, a.inv_D = 1.f / (float)D;
    int blocks = 0;
    cudaError_t e = dt == LA_BF16
                        ? la::run<__nv_bfloat16>(a, true, layout == LA_ROPE_INTERLEAVED, &blocks, st)
                        : la::run<float>(a, true, layout == LA_ROPE_INTERLEAVED, &blocks, st);
    if (e != cudaSuccess) return LA_ERR_CUDA;
    if (norm && (dwq || dwk)) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((2 * D + 31) / 32);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, la::rope_dw_kernel, (const float*)workspace, blocks, D, dwq, dwk);
        if (e != cudaSuccess) return LA_ERR_CUDA;
    }
    return LA_OK;
}

}  // extern "C"
