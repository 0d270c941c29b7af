// Selective state space scan, per head (b, h) with its group's B and C:
//   d_t = softplus(step_t + bias_h) (or step_t + bias_h),   a_t = exp(d_t A_h)
//   S_t = a_t S_{t-1} + d_t B_t x_t^T,   y_t = C_t^T S_t + D_h x_t,   y_t *= silu(z_t)
// i.e. causal linear attention ("Why Replace Attention? The Softmax Bottleneck
// and the Path to Linear Time", section 7.2, steps 1-4) with q = C, k = d B,
// v = x, no feature map and no denominator, and a decay of the state per token.
//
// This file: the recurrence on the CUDA cores in fp32 (any type, size, stride),
// the single-token step, the scan over segments, and the entry points. bf16
// with whole 16-byte rows runs on the tensor cores instead (csrc/scan_tc.cu).
//
// The recurrence keeps the state in registers: a warp owns 4 kW columns of one
// head, its 32 lanes 8 row groups x 4 column groups, so a lane holds R = S / 8 rows
// of kW columns, as packed fp32 row pairs. What bounds it are the instructions of the
// eleven or so warps per SM that the registers leave (issue slots 56 % used in the second
// pass, 45 % in the first, B=2 N=4000 H=8 P=S=64), so the decay is taken out of the
// inner loop: within eight tokens the state is kept divided by the decay since their
// start (the update's weight is d_t e^{-l_t}, the read is multiplied by e^{l_t}), two
// operations per element and token instead of three, and multiplied through once at the end. Where eight tokens decay by more
// than e^-40 the plain form runs instead. The eight tokens' reads are summed over
// the row groups by a butterfly that halves the tokens at each step. With too few
// heads for the SMs a sequence is cut into segments: a first pass gives each
// segment's own end state (one operation per element and token: walked backwards,
// the weights reach to the segment's end) and total decay, a scan chains them, and
// the second pass starts each segment from its state.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "mixing.cuh"
#include "overlap.h"
#include "scan.cuh"
#include "tc_common.cuh"

namespace la {

using namespace scan;

namespace {

constexpr int kTok = 32;               // tokens staged per tile

__device__ __forceinline__ uint64_t pk(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float sum2(uint64_t a) {
    float x, y;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a));
    return x + y;
}

// Staged floats per token and operand: 8 row groups of R rows, padded so that
// the groups' vector loads fall into different banks.
template <int R> constexpr int kGroupStride = R == 8 || R == 16 ? R + 4 : R;

// Per-token factors of a tile.
struct Factors {
    float w[kTok];       // weight of the update: d e^{-l} (plain form: d; first pass: d e^{sum to the end})
    float a[kTok];       // e^l, l summed from the start of the token's eight (plain form: e^{d A})
    float plain[kTok / 8];   // != 0: these eight tokens take the plain form
};

// 2 kPairs rows of one lane at p, as packed pairs.
template <int kPairs>
__device__ __forceinline__ void load_pairs(const float* p, uint64_t (&v)[kPairs]) {
    if constexpr (kPairs % 2 == 0) {
#pragma unroll
        for (int i = 0; i < kPairs; i += 2) {
            const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p + 2 * i);
            v[i] = t.x, v[i + 1] = t.y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) v[i] = *reinterpret_cast<const uint64_t*>(p + 2 * i);
    }
}

// kW adjacent values at p (8- or 16-byte aligned).
template <int kW>
__device__ __forceinline__ void load_values(const float* p, float (&v)[kW]) {
    if constexpr (kW == 4) {
        const float4 t = *reinterpret_cast<const float4*>(p);
        v[0] = t.x, v[1] = t.y, v[2] = t.z, v[3] = t.w;
    } else {
        const float2 t = *reinterpret_cast<const float2*>(p);
        v[0] = t.x, v[1] = t.y;
    }
}

// Columns per lane: four share each row's B and C; two for heads of at most 8
// columns, which would leave half of the lanes idle, and for states of more than 64
// rows, whose lanes would hold 48 to 64 values (254 registers with 16 rows).
int lane_columns(int S, int P) { return S > 64 || P <= 8 ? 2 : 4; }

// Grid: (segments, B H). Block: one warp per 4 kW columns of the head.
// kState: only the segment's end state from zero and its decay (first pass).
template <typename T, int R, int kW, bool kState>
__global__ void __launch_bounds__(32 * kMaxDim / (4 * kW)) scan_kernel(const __grid_constant__ ScanArgs a) {
    constexpr int kG = kGroupStride<R>, kRow = 8 * kG, kP = R / 2;
    constexpr int kJ = (8 * R + 31) / 32, kB = R <= 8 ? 8 : 4;
    extern __shared__ float smem[];
    __shared__ Factors fac;
    const int cols = blockDim.x / 8 * kW;               // P rounded up to whole warps
    float* bs = smem;                                   // [kTok][kRow]
    float* xs = bs + kTok * kRow;                       // [kTok][cols]
    float* cs = xs + kTok * cols;                       // [kTok][kRow], second pass
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int rg = lane & 7, col = 4 * kW * warp + kW * (lane >> 3);
    const int seg = blockIdx.x, h = blockIdx.y % a.H;
    const int64_t b = blockIdx.y / a.H, bh = blockIdx.y;
    const int grp = h / (a.H / a.G);
    const int n = a.lengths ? min(max(a.lengths[b], 0), a.N) : a.N;
    const int t0 = min(seg * a.seg_len, n), t1 = min(t0 + a.seg_len, n);
    const T* x = static_cast<const T*>(a.x) + b * a.x_bs + (int64_t)h * a.P;
    const T* z = a.z ? static_cast<const T*>(a.z) + b * a.z_bs + (int64_t)h * a.P : nullptr;
    const T* Bm = static_cast<const T*>(a.Bm) + b * a.b_bs + (int64_t)grp * a.S;
    const T* Cm = static_cast<const T*>(a.Cm) + b * a.c_bs + (int64_t)grp * a.S;
    const T* st = static_cast<const T*>(a.step) + b * a.step_bs + h;
    T* y = static_cast<T*>(a.y) + b * a.y_bs + (int64_t)h * a.P;
    const float A = a.A[h], bias = a.step_bias ? a.step_bias[h] : 0.f, Dh = a.D ? a.D[h] : 0.f;

    // The second pass is a programmatic dependent of the chaining kernel (the wait is a
    // no-op in any other launch).
    tcc::pdl_launch_dependents();
    tcc::pdl_wait();
    // The state: rows rg R .. rg R + R - 1 of columns col .. col + kW - 1.
    uint64_t s[kW][kP];
    const float* from = kState ? nullptr : (a.nseg > 1 ? a.seeds + (bh * a.nseg + seg) * a.S * a.P
                                                       : (a.S0 ? a.S0 + bh * a.S * a.P : nullptr));
#pragma unroll
    for (int c = 0; c < kW; ++c)
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const int r = rg * R + 2 * i;
            float v[2] = {0.f, 0.f};
            if (from && col + c < a.P) {
                if (r < a.S) v[0] = from[(int64_t)r * a.P + col + c];
                if (r + 1 < a.S) v[1] = from[(int64_t)(r + 1) * a.P + col + c];
            }
            s[c][i] = pk(v[0], v[1]);
        }
    float behind = 0.f;                                 // first pass: sum of d A over the tiles behind

    const int tiles = (t1 - t0 + kTok - 1) / kTok;
    for (int k = 0; k < tiles; ++k) {
        const int tile = t0 + (kState ? tiles - 1 - k : k) * kTok, m = min(kTok, t1 - tile);
        __syncthreads();
        // A warp stages every nw-th token, a lane 32 columns apart; kB tokens' loads are
        // all in flight before the first store (one wait on memory per tile and block).
        for (int tb = warp; tb < kTok; tb += kB * nw) {
            float vb[kJ][kB], vc[kJ][kB], vx[4][kB];
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int t = tb + u * nw;
                const bool in = t < m;
                const T* pb = Bm + (int64_t)(tile + t) * a.b_ts;
                const T* pc = Cm + (int64_t)(tile + t) * a.c_ts;
                const T* px = x + (int64_t)(tile + t) * a.x_ts;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int r = lane + 32 * j;
                    vb[j][u] = in && r < a.S ? to_f(pb[r]) : 0.f;
                    if (!kState) vc[j][u] = in && r < a.S ? to_f(pc[r]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int p = lane + 32 * j;
                    vx[j][u] = in && p < a.P ? to_f(px[p]) : 0.f;
                }
            }
#pragma unroll
            for (int u = 0; u < kB; ++u) {
                const int t = tb + u * nw;
                if (t >= kTok) break;
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const int r = lane + 32 * j;
                    if (8 * R < 32 * kJ && r >= 8 * R) continue;
                    const int at = t * kRow + (r / R) * kG + r % R;
                    bs[at] = vb[j][u];
                    if (!kState) cs[at] = vc[j][u];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (lane + 32 * j < cols) xs[t * cols + lane + 32 * j] = vx[j][u];
            }
        }
        if (warp == 0) {
            // One token per lane. A token past the end decays by 1 and adds nothing.
            const float d = lane < m ? step_size(to_f(st[(int64_t)(tile + lane) * a.step_ts]) + bias, a.softplus) : 0.f;
            float l = d * A;
            const float own = l;
            if constexpr (kState) {
                // Sum over the tokens after this one, up to the segment's end.
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const float u = __shfl_down_sync(0xffffffffu, l, o);
                    if (lane + o < 32) l += u;
                }
                const float total = __shfl_sync(0xffffffffu, l, 0);
                float after = __shfl_down_sync(0xffffffffu, l, 1);
                if (lane == 31) after = 0.f;
                fac.w[lane] = d * expf(after + behind);
                behind += total;
            } else {
#pragma unroll
                for (int o = 1; o < 8; o <<= 1) {
                    const float u = __shfl_up_sync(0xffffffffu, l, o, 8);
                    if ((lane & 7) >= o) l += u;
                }
                const float end = __shfl_sync(0xffffffffu, l, 7, 8);
                const bool plain = !(fabsf(end) < 40.f);
                fac.w[lane] = plain ? d : d * expf(-l);
                fac.a[lane] = expf(plain ? own : l);
                if ((lane & 7) == 0) fac.plain[lane >> 3] = plain ? 1.f : 0.f;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int half = 0; half < kTok && half < m; half += 8) {
            if constexpr (kState) {
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int tt = half + t;
                    const float w = fac.w[tt];
                    float xv[kW];
                    load_values<kW>(xs + tt * cols + col, xv);
                    uint64_t bb[kP];
                    load_pairs<kP>(bs + tt * kRow + rg * kG, bb);
#pragma unroll
                    for (int c = 0; c < kW; ++c) {
                        const float v = w * xv[c];
                        const uint64_t x2 = pk(v, v);
#pragma unroll
                        for (int i = 0; i < kP; ++i) s[c][i] = fma2(bb[i], x2, s[c][i]);
                    }
                }
            } else {
                const bool plain = fac.plain[half >> 3] != 0.f;
                float acc[8][kW];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    const int tt = half + t;
                    const float w = fac.w[tt];
                    float xv[kW];
                    load_values<kW>(xs + tt * cols + col, xv);
                    if (plain) {
                        const float at = fac.a[tt];
                        const uint64_t a2 = pk(at, at);
#pragma unroll
                        for (int c = 0; c < kW; ++c)
#pragma unroll
                            for (int i = 0; i < kP; ++i) s[c][i] = mul2(a2, s[c][i]);
                    }
                    uint64_t bb[kP], cc[kP];
                    load_pairs<kP>(bs + tt * kRow + rg * kG, bb);
                    load_pairs<kP>(cs + tt * kRow + rg * kG, cc);
#pragma unroll
                    for (int c = 0; c < kW; ++c) {
                        const float v = w * xv[c];
                        const uint64_t x2 = pk(v, v);
                        uint64_t y2;
#pragma unroll
                        for (int i = 0; i < kP; ++i) {
                            s[c][i] = fma2(bb[i], x2, s[c][i]);
                            y2 = i == 0 ? mul2(cc[0], s[c][0]) : fma2(cc[i], s[c][i], y2);
                        }
                        acc[t][c] = sum2(y2);
                    }
                }
                if (!plain) {
                    const float at = fac.a[half + 7];
                    const uint64_t a2 = pk(at, at);
#pragma unroll
                    for (int c = 0; c < kW; ++c)
#pragma unroll
                        for (int i = 0; i < kP; ++i) s[c][i] = mul2(a2, s[c][i]);
                }
                // Sum over the 8 row groups (lane bits 0-2): each step keeps half of the
                // tokens, so lane rg ends with token rg of the eight.
#pragma unroll
                for (int bit = 2; bit >= 0; --bit) {
                    const int keep = 1 << bit;
                    const bool up = (rg & keep) != 0;
#pragma unroll
                    for (int t = 0; t < keep; ++t)
#pragma unroll
                        for (int c = 0; c < kW; ++c) {
                            const float send = up ? acc[t][c] : acc[t + keep][c];
                            const float mine = up ? acc[t + keep][c] : acc[t][c];
                            acc[t][c] = mine + __shfl_xor_sync(0xffffffffu, send, keep);
                        }
                }
                const int tt = half + rg;
                if (tt < m) {
                    const float at = plain ? 1.f : fac.a[tt];
#pragma unroll
                    for (int c = 0; c < kW; ++c) {
                        if (col + c >= a.P) continue;
                        float v = fmaf(at, acc[0][c], Dh * xs[tt * cols + col + c]);
                        if (z) v *= silu(to_f(z[(int64_t)(tile + tt) * a.z_ts + col + c]));
                        y[(int64_t)(tile + tt) * a.y_ts + col + c] = from_f<T>(v);
                    }
                }
            }
        }
    }
    float* to = kState ? a.seeds + (bh * a.nseg + seg) * a.S * a.P
                       : (seg == a.nseg - 1 && a.S_out ? a.S_out + bh * a.S * a.P : nullptr);
    if (to) {
#pragma unroll
        for (int c = 0; c < kW; ++c) {
            if (col + c >= a.P) continue;
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                const int r = rg * R + 2 * i;
                float lo, hi;
                asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(s[c][i]));
                if (r < a.S) to[(int64_t)r * a.P + col + c] = lo;
                if (r + 1 < a.S) to[(int64_t)(r + 1) * a.P + col + c] = hi;
            }
        }
    }
    if (kState && tid == 0) a.seg_decay[bh * a.nseg + seg] = behind;
}

// In place over a head's segments: the end states (from zero) become the states
// that the segments start from, seed_0 = S0, seed_{i+1} = exp(decay_i) seed_i + end_i; the
// last one's end goes to S_out (which may be S0).
// A thread chains one element (reads and writes of a segment are whole rows of
// threads), sixteen segments in flight; the decays' exponentials are shared.
constexpr int kMaxSegments = 512;
__global__ void __launch_bounds__(128) seed_kernel(const __grid_constant__ ScanArgs a) {
    __shared__ float f[kMaxSegments];
    const int64_t bh = blockIdx.y;
    tcc::pdl_launch_dependents();
    tcc::pdl_wait();
    for (int i = threadIdx.x; i < a.nseg; i += 128) f[i] = expf(a.seg_decay[bh * a.nseg + i]);
    __syncthreads();
    const int e = blockIdx.x * 128 + threadIdx.x, E = a.S * a.P;
    if (e >= E) return;
    float carry = a.S0 ? a.S0[bh * E + e] : 0.f;
    float* p = a.seeds + bh * a.nseg * E + e;
    for (int i0 = 0; i0 < a.nseg; i0 += 16) {
        float end[16];
#pragma unroll
        for (int u = 0; u < 16; ++u)
            if (i0 + u < a.nseg) end[u] = p[(int64_t)(i0 + u) * E];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            if (i0 + u >= a.nseg) break;
            p[(int64_t)(i0 + u) * E] = carry;
            carry = fmaf(f[i0 + u], carry, end[u]);
        }
    }
    if (a.S_out) a.S_out[bh * E + e] = carry;
}

// One token per sequence, the state updated in place. It is read and written
// once (8 bytes per element against a handful of operations): HBM bandwidth
// bounds it. A block owns one head; a thread owns kV columns of every
// rows-per-pass-th row and keeps kU rows in flight.
template <typename T, int kV>
__global__ void __launch_bounds__(256) scan_step_kernel(const __grid_constant__ ScanArgs a) {
    constexpr int kU = 8;
    __shared__ float bs[kMaxDim], cs[kMaxDim], ds[2];
    __shared__ float red[256 * kV];
    const int tid = threadIdx.x;
    const int64_t bh = blockIdx.x, b = bh / a.H;
    const int h = (int)(bh - b * a.H), grp = h / (a.H / a.G);
    const int lpr = (a.P + kV - 1) / kV, rpp = 256 / lpr;   // lanes per row, rows per pass
    const int r0 = tid / lpr, c0 = (tid - r0 * lpr) * kV;
    const bool mine = r0 < rpp;
    float* S = a.S_out + bh * a.S * a.P + c0;
    float s[kU][kV];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = base + u * rpp + r0;
            if (!mine || r >= a.S) continue;
            if constexpr (kV == 4) {
                const float4 v = *reinterpret_cast<const float4*>(S + (int64_t)r * a.P);
                s[u][0] = v.x, s[u][1] = v.y, s[u][2] = v.z, s[u][3] = v.w;
            } else {
                s[u][0] = S[(int64_t)r * a.P];
            }
        }
    };
    load(0);
    const T* xp = static_cast<const T*>(a.x) + b * a.x_bs + (int64_t)h * a.P;
    if (tid < a.S) {
        bs[tid] = to_f(static_cast<const T*>(a.Bm)[b * a.b_bs + (int64_t)grp * a.S + tid]);
        cs[tid] = to_f(static_cast<const T*>(a.Cm)[b * a.c_bs + (int64_t)grp * a.S + tid]);
    }
    if (tid >= 224) {   // one warp: its forty operations in every warp took 3 of 49 us (128 sequences, H=32)
        const float d = step_size(to_f(static_cast<const T*>(a.step)[b * a.step_bs + h]) +
                                      (a.step_bias ? a.step_bias[h] : 0.f), a.softplus);
        const float decay = expf(d * a.A[h]);
        if (tid == 224) ds[0] = d, ds[1] = decay;
    }
    float xd[kV], acc[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) xd[v] = mine ? to_f(xp[c0 + v]) : 0.f, acc[v] = 0.f;
    __syncthreads();
    const float decay = ds[1];
#pragma unroll
    for (int v = 0; v < kV; ++v) xd[v] *= ds[0];
    for (int base = 0; base < a.S; base += kU * rpp) {
        if (base > 0) load(base);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int r = base + u * rpp + r0;
            if (!mine || r >= a.S) continue;
            const float br = bs[r], cr = cs[r];
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                s[u][v] = fmaf(br, xd[v], decay * s[u][v]);
                acc[v] = fmaf(cr, s[u][v], acc[v]);
            }
            if constexpr (kV == 4)
                *reinterpret_cast<float4*>(S + (int64_t)r * a.P) = make_float4(s[u][0], s[u][1], s[u][2], s[u][3]);
            else
                S[(int64_t)r * a.P] = s[u][0];
        }
    }
    if (mine)
#pragma unroll
        for (int v = 0; v < kV; ++v) red[r0 * a.P + c0 + v] = acc[v];
    __syncthreads();
    if (tid < a.P) {
        float v = 0.f;
        for (int r = 0; r < rpp; ++r) v += red[r * a.P + tid];
        v = fmaf(a.D ? a.D[h] : 0.f, to_f(xp[tid]), v);
        if (a.z) v *= silu(to_f(static_cast<const T*>(a.z)[b * a.z_bs + (int64_t)h * a.P + tid]));
        static_cast<T*>(a.y)[b * a.y_bs + (int64_t)h * a.P + tid] = from_f<T>(v);
    }
}

template <typename T, int R, int kW>
cudaError_t recurrence(const ScanArgs& a, int64_t BH, cudaStream_t st) {
    const int warps = (a.P + 4 * kW - 1) / (4 * kW);
    const size_t row = sizeof(float) * kTok * 8 * kGroupStride<R>, x = sizeof(float) * (size_t)kTok * 4 * kW * warps;
    const size_t smem = 2 * row + x;
    static std::atomic<int> optin[tcc::kMaxDevices];
    // The largest head needs more than the 48 KB that need no opting in.
    cudaError_t e = tcc::ensure_smem_optin(scan_kernel<T, R, kW, false>,
                                           (int)(sizeof(float) * kTok * (16 * kGroupStride<R> + kMaxDim)), optin);
    if (e != cudaSuccess) return e;
    const dim3 grid(a.nseg, (unsigned)BH);
    if (a.nseg > 1) {
        scan_kernel<T, R, kW, true><<<grid, 32 * warps, row + x, st>>>(a);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        ScanArgs chain = a;
        chain.S_out = nullptr;                             // the second pass writes it
        if ((e = launch_seeds(chain, BH, st)) != cudaSuccess) return e;
    }
    return launch_after(scan_kernel<T, R, kW, false>, grid, 32 * warps, smem, st, a.nseg > 1, a);
}

template <typename T, int R>
cudaError_t recurrence_by_width(const ScanArgs& a, int64_t BH, cudaStream_t st) {
    if constexpr (R <= 8)
        if (lane_columns(a.S, a.P) == 4) return recurrence<T, R, 4>(a, BH, st);
    return recurrence<T, R, 2>(a, BH, st);
}

template <typename T>
cudaError_t recurrence_by_size(const ScanArgs& a, int64_t BH, cudaStream_t st) {
    if (a.S <= 16) return recurrence_by_width<T, 2>(a, BH, st);
    if (a.S <= 32) return recurrence_by_width<T, 4>(a, BH, st);
    if (a.S <= 64) return recurrence_by_width<T, 8>(a, BH, st);
    if (a.S <= 96) return recurrence_by_width<T, 12>(a, BH, st);
    return recurrence_by_width<T, 16>(a, BH, st);
}

template <typename T>
cudaError_t step(const ScanArgs& a, int64_t BH, cudaStream_t st) {
    if (a.P % 4 == 0) scan_step_kernel<T, 4><<<(unsigned)BH, 256, 0, st>>>(a);
    else scan_step_kernel<T, 1><<<(unsigned)BH, 256, 0, st>>>(a);
    return cudaPeekAtLastError();
}

// most_heads: of all sequences together, the size of the grid's axis that they map to.
constexpr int64_t kPromptHeads = 65535, kStepHeads = 2147483647;
la_status check_shape(int B, int H, int G, int N, int S, int P, la_dtype dt, int64_t most_heads) {
    if (B < 0 || H < 0 || N < 0 || G < 1 || S < 1 || P < 1) return LA_ERR_INVALID_ARG;
    if (dt != LA_F32 && dt != LA_BF16) return LA_ERR_INVALID_ARG;
    if (H % G) return LA_ERR_INVALID_ARG;
    if (S > kMaxDim || P > kMaxDim) return LA_ERR_UNSUPPORTED;
    if ((int64_t)B * H > most_heads) return LA_ERR_UNSUPPORTED;
    if (N > kScanMaxTokens) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

bool bad(const void* p, la_dtype dt) {
    return !p || (reinterpret_cast<uintptr_t>(p) & (dt == LA_BF16 ? 1 : 3));
}

bool bad4(const void* p) { return reinterpret_cast<uintptr_t>(p) & 3; }

}  // namespace

namespace scan {

// Segments of the recurrence: one while there are twelve warps per SM or fewer than
// two stretches of 64 tokens; else as many as give each SM twelve warps in whole
// blocks (B=2 N=4000 H=8 P=64: S=64, three blocks of four warps 78 us, two 98, four
// 93; S=128, two blocks of eight warps 143, three 157). Segments of whole tiles left
// the SMs unevenly loaded (95 us).
int recurrence_segments(int64_t BH, int N, int S, int P) {
    const int columns = 4 * lane_columns(S, P), warps = (P + columns - 1) / columns;
    const int64_t want = (int64_t)((12 + warps - 1) / warps) * tcc::sm_count() / (BH > 0 ? BH : 1);
    const int64_t most = N / 64;
    int64_t n = want < most ? want : most;
    n = n < kMaxSegments ? n : kMaxSegments;
    return n < 2 ? 1 : (int)n;
}

cudaError_t launch_seeds(const ScanArgs& a, int64_t BH, cudaStream_t st) {
    return launch_after(seed_kernel, dim3((a.S * a.P + 127) / 128, (unsigned)BH), 128, 0, st, true, a);
}

}  // namespace scan

namespace {

bool tc_widths(int S, int P, la_dtype dt) { return dt == LA_BF16 && S % 8 == 0 && P % 8 == 0; }

}  // namespace

// Enough for either path (rows that are not aligned take the recurrence) and for
// every number of groups, on which the tensor-core path's segments depend.
size_t scan_workspace(int B, int H, int N, int S, int P, la_dtype dt) {
    const int64_t BH = (int64_t)B * H;
    int n = recurrence_segments(BH, N, S, P);
    if (tc_widths(S, P, dt))
        for (int g = 1; (int64_t)g * g <= H; ++g) {
            if (H % g) continue;
            const int x = tc_segments(B, H, g, N, P), y = tc_segments(B, H, H / g, N, P);
            n = x > n ? x : n;
            n = y > n ? y : n;
        }
    return n > 1 ? (size_t)BH * n * ((size_t)S * P + 1) * sizeof(float) : 0;
}

int scan_launches(int B, int H, int N, int S, int P, la_dtype dt) {
    const int n = tc_widths(S, P, dt) ? tc_segments(B, H, 1, N, P) : recurrence_segments((int64_t)B * H, N, S, P);
    return n > 1 ? 3 : 1;
}

}  // namespace la

extern "C" {

la_status la_selective_scan_fwd(const void* x, int64_t x_batch, int64_t x_token, const void* step,
                                int64_t step_batch, int64_t step_token, const float* A,
                                const void* Bm, int64_t b_batch, int64_t b_token, const void* Cm,
                                int64_t c_batch, int64_t c_token, const float* D, const void* z,
                                int64_t z_batch, int64_t z_token, const float* step_bias,
                                int softplus, const int32_t* lengths, const float* S0,
                                float* S_out, void* y, int64_t y_batch, int64_t y_token, int B,
                                int H, int G, int N, int S, int P, la_dtype dt, void* workspace,
                                size_t workspace_bytes, la_stream_t stream) {
    la_status s = la::check_shape(B, H, G, N, S, P, dt, la::kPromptHeads);   // grid.y
    if (s != LA_OK) return s;
    const int64_t BH = (int64_t)B * H;
    if (BH == 0) return LA_OK;
    if (la::bad4(S0) || la::bad4(S_out) || la::bad4(lengths) || la::bad4(D) || la::bad4(step_bias) ||
        la::bad4(A) || !A)
        return LA_ERR_INVALID_ARG;
    // The final state may replace the initial one, but not overlap it otherwise.
    const size_t state = sizeof(float) * (size_t)BH * S * P;
    const la::Rows s0 = la::block_of(S0, state), s1 = la::block_of(S_out, state);
    if (S0 != S_out && la::overlap(s0, s1)) return LA_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (N == 0) {
        if (!S_out || S_out == S0) return LA_OK;
        const cudaError_t e = S0 ? cudaMemcpyAsync(S_out, S0, state, cudaMemcpyDeviceToDevice, st)
                                 : cudaMemsetAsync(S_out, 0, state, st);
        return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
    }
    if (la::bad(x, dt) || la::bad(step, dt) || la::bad(Bm, dt) || la::bad(Cm, dt) || la::bad(y, dt) ||
        (z && la::bad(z, dt)))
        return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, N, (int64_t)H * P, y_batch, y_token)) return LA_ERR_INVALID_ARG;
    la::scan::ScanArgs a = {};
    a.x = x, a.x_bs = x_batch, a.x_ts = x_token;
    a.step = step, a.step_bs = step_batch, a.step_ts = step_token;
    a.Bm = Bm, a.b_bs = b_batch, a.b_ts = b_token;
    a.Cm = Cm, a.c_bs = c_batch, a.c_ts = c_token;
    a.z = z, a.z_bs = z_batch, a.z_ts = z_token;
    a.y = y, a.y_bs = y_batch, a.y_ts = y_token;
    a.A = A, a.D = D, a.step_bias = step_bias, a.lengths = lengths, a.S0 = S0, a.S_out = S_out;
    a.N = N, a.H = H, a.G = G, a.S = S, a.P = P, a.softplus = softplus ? 1 : 0;
    const bool tc = la::scan::tc_supported(a, B, dt);
    a.nseg = tc ? la::scan::tc_segments(B, H, G, N, P) : la::scan::recurrence_segments(BH, N, S, P);
    a.seg_len = (N + a.nseg - 1) / a.nseg;                 // of the recurrence
    const size_t need = sizeof(la::WsHeader) +
                        (a.nseg > 1 ? (size_t)BH * a.nseg * ((size_t)S * P + 1) * sizeof(float) : 0);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255) || workspace_bytes < need)
        return LA_ERR_WORKSPACE;
    const int64_t eb = dt == LA_BF16 ? 2 : 4, HP = (int64_t)H * P, GS = (int64_t)G * S;
    const la::Rows xr = la::rows_of(x, B, N, HP, x_batch, x_token, eb), zr = la::rows_of(z, B, N, HP, z_batch, z_token, eb);
    const la::Rows dr = la::rows_of(step, B, N, H, step_batch, step_token, eb);
    const la::Rows br = la::rows_of(Bm, B, N, GS, b_batch, b_token, eb), cr = la::rows_of(Cm, B, N, GS, c_batch, c_token, eb);
    const la::Rows yr = la::rows_of(y, B, N, HP, y_batch, y_token, eb);
    const la::Rows Ar = la::block_of(A, 4 * (int64_t)H), Dr = la::block_of(D, 4 * (int64_t)H);
    const la::Rows biasr = la::block_of(step_bias, 4 * (int64_t)H), nr = la::block_of(lengths, 4 * (int64_t)B);
    if (la::overlaps_any(yr, {xr, zr, dr, br, cr, Ar, Dr, biasr, nr, s0, s1}) ||
        la::overlaps_any(s1, {xr, zr, dr, br, cr, Ar, Dr, biasr, nr}))
        return LA_ERR_INVALID_ARG;
    a.seeds = reinterpret_cast<float*>(static_cast<char*>(workspace) + sizeof(la::WsHeader));
    a.seg_decay = a.seeds + (size_t)BH * a.nseg * S * P;
    const cudaError_t e = tc ? la::scan::tc_scan(a, B, workspace, st)
                          : dt == LA_BF16 ? la::recurrence_by_size<__nv_bfloat16>(a, BH, st)
                                          : la::recurrence_by_size<float>(a, BH, st);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

la_status la_selective_scan_step(const void* x, int64_t x_batch, const void* step,
                                 int64_t step_batch, const float* A, const void* Bm,
                                 int64_t b_batch, const void* Cm, int64_t c_batch, const float* D,
                                 const void* z, int64_t z_batch, const float* step_bias,
                                 int softplus, float* S_inout, void* y, int64_t y_batch, int B,
                                 int H, int G, int S, int P, la_dtype dt, la_stream_t stream) {
    la_status s = la::check_shape(B, H, G, 1, S, P, dt, la::kStepHeads);     // grid.x
    if (s != LA_OK) return s;
    const int64_t BH = (int64_t)B * H;
    if (BH == 0) return LA_OK;
    if (la::bad(x, dt) || la::bad(step, dt) || la::bad(Bm, dt) || la::bad(Cm, dt) || la::bad(y, dt) ||
        (z && la::bad(z, dt)) || !A || la::bad4(A) || la::bad4(D) || la::bad4(step_bias) || !S_inout ||
        (reinterpret_cast<uintptr_t>(S_inout) & (P % 4 ? 3 : 15)))   // 16-byte accesses of four columns
        return LA_ERR_INVALID_ARG;
    if (!la::rows_disjoint(B, 1, (int64_t)H * P, y_batch, 0)) return LA_ERR_INVALID_ARG;
    const int64_t eb = dt == LA_BF16 ? 2 : 4, HP = (int64_t)H * P, GS = (int64_t)G * S;
    const la::Rows xr = la::rows_of(x, B, 1, HP, x_batch, 0, eb), zr = la::rows_of(z, B, 1, HP, z_batch, 0, eb);
    const la::Rows dr = la::rows_of(step, B, 1, H, step_batch, 0, eb), yr = la::rows_of(y, B, 1, HP, y_batch, 0, eb);
    const la::Rows br = la::rows_of(Bm, B, 1, GS, b_batch, 0, eb), cr = la::rows_of(Cm, B, 1, GS, c_batch, 0, eb);
    const la::Rows Ar = la::block_of(A, 4 * (int64_t)H), Dr = la::block_of(D, 4 * (int64_t)H);
    const la::Rows biasr = la::block_of(step_bias, 4 * (int64_t)H);
    const la::Rows sr = la::block_of(S_inout, (int64_t)(sizeof(float) * (size_t)BH * S * P));
    // y may be x or z itself: a block reads what it replaces.
    if (la::overlaps_any(sr, {xr, zr, dr, br, cr, Ar, Dr, biasr, yr}) || la::overlaps_any(yr, {dr, br, cr, Ar, Dr, biasr}) ||
        (!la::same_rows(xr, yr) && la::overlap(xr, yr)) || (!la::same_rows(zr, yr) && la::overlap(zr, yr)))
        return LA_ERR_INVALID_ARG;
    la::scan::ScanArgs a = {};
    a.x = x, a.x_bs = x_batch, a.step = step, a.step_bs = step_batch, a.Bm = Bm, a.b_bs = b_batch;
    a.Cm = Cm, a.c_bs = c_batch, a.z = z, a.z_bs = z_batch, a.y = y, a.y_bs = y_batch;
    a.A = A, a.D = D, a.step_bias = step_bias, a.S_out = S_inout;
    a.N = 1, a.H = H, a.G = G, a.S = S, a.P = P, a.softplus = softplus ? 1 : 0;
    const cudaError_t e = dt == LA_BF16 ? la::step<__nv_bfloat16>(a, BH, (cudaStream_t)stream)
                                        : la::step<float>(a, BH, (cudaStream_t)stream);
    return e == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

}  // extern "C"
