// Selective scan on the tensor cores (tcgen05): bf16, S and P multiples of 8,
// 16-byte aligned rows. Definitions in csrc/scan.cu.
//
// Method. For a chunk of 128 tokens of one head with the state S before it, and
// l_t = sum of d A over the chunk's tokens up to t (all exponents below are <= 0):
//   y_i   = e^{l_i} C_i^T S + sum_{j <= i} (C_i . B_j) e^{l_i - l_j} d_j x_j + D x_i
//   S_new = e^{l_end} S + sum_j B_j (d_j e^{l_end - l_j} x_j)^T
// an exact regrouping of the recurrence into products of 128 x 128 tiles:
//   (1) scores C B^T                 M = 128, N = 128, K = S   once per chunk
//   (2) read of the state C S_bf16   M = 128, N = 64,  K = S
//   (3) P x, P = bf16 of the weighted, masked scores     M = 128, N = 64, K = 128
//   (4) S_new: B^T (w x)             M = S,   N = 64,  K = 128, fp32 in TMEM
// A CTA owns two "units" (64 value columns of a head each) of one group and batch,
// so that (1) and the loads of B and C serve both, and walks a range of chunks.
//
// Roundings. x, B, C enter as they are. P and the state of (2) are rounded to bf16
// once each (2^-9 relative, as the output itself). The state is held in fp32 in
// TMEM: it is scaled there per chunk, and (4) adds w x as two bf16 terms (value and
// remainder), which leaves 2^-17 of each term. Decays of P below the diagonal
// 32 x 32 blocks are products of two factors <= 1 around the block row's start,
// e^{l_i - l_m} e^{l_m - l_j}, so only the diagonal blocks take an exponential per
// score; the weights of (4) come from sums taken from the chunk's end, so that a
// small exponent is not a difference of two large ones.
//
// Roles (20 warps, one CTA per SM): TMA; MMA issue; two warps that turn step
// sizes into decays (one per unit); and four warpgroups over the 128 rows: scores
// to P, state, weighted values, output. All hand-offs are mbarriers; every wait is
// bounded. Sequences are cut into segments when there are too few units for the
// SMs: the first pass streams (4) alone, in reverse order of chunks so that the
// weights reach to the segment's end and nothing has to be rescaled; seeds are
// chained by csrc/scan.cu and the second pass starts from them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "scan.cuh"
#include "tc_common.cuh"
#include "tc_util.cuh"

namespace la {

using namespace scan;

namespace {

using namespace tc;
using namespace tcc;

constexpr uint32_t kTile = kTileBytes;             // [128 tokens x 64] bf16
constexpr int kDtRing = 4;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One unit's decays over a chunk, exponents in base 2.
struct Decay {
    float cum[kC];      // l_t: sum up to and including t
    float d[kC];        // step sizes (0 past the sequence's end)
    float w[kC];        // d_t 2^(l_end - l_t)
    float total;        // 2^l_end
    float pad[3];
};

struct Units {
    int pairs, units, blocks;   // CTAs per group, units per group, 64-column blocks per head
    int cps;                    // chunks per segment
    int gate_vec;               // z rows are 16-byte aligned
};

// TMEM columns of the main kernel.
constexpr uint32_t kTmSc = 0, kTmP = 128, kTmY1 = 256, kTmY2 = 320, kTmSt = 384;

struct Misc {
    uint64_t bc_full[2], bc_empty[2], x_full[2], x_empty[2], dt_full[kDtRing], dt_empty[kDtRing];
    uint64_t sc_full, sc_empty, p_full[2], p_empty[2], xw_full, xw_empty, sb_full, sb_empty;
    uint64_t st_full[2], y_full, y_empty, drain;
    uint32_t tmem_slot;
};

// Shared memory of the main kernel, from a 1024-byte boundary.
template <int kT> struct Smem {
    static constexpr uint32_t kStage = 2 * kT * kTile;         // C tiles, then B tiles
    static constexpr uint32_t kX = 2 * kStage;
    static constexpr uint32_t kXw = kX + 2 * kTile;            // value, remainder
    static constexpr uint32_t kSb = kXw + 2 * kTile;           // bf16 state, 64 kT rows
    static constexpr uint32_t kDt = kSb + kT * 64 * 128;
    static constexpr uint32_t kCol = kDt + kDtRing * sizeof(Decay);   // column factors per P warp
    static constexpr uint32_t kMisc = kCol + 4 * 96 * 4;
    static constexpr uint32_t kEnd = kMisc + sizeof(Misc);
    static constexpr size_t kBytes = 1024 + kEnd;
};
static_assert(Smem<2>::kBytes <= 227 * 1024, "main kernel's shared memory");

constexpr int kThreads = 640;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk2(uint64_t v, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(v));
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
__device__ __forceinline__ uint64_t bf2(uint32_t u) {   // two packed bf16 as fp32 pair
    return pk2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
    float a, b;
    unpk2(v, &a, &b);
    return pack_bf16(a, b);
}

// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t limit_us) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_us));
}

// A CTA's place: group, batch, first unit, number of units, chunk range.
struct Place {
    int b, g, unit0, nu, seg, c0, nc, n;
    __device__ int head(const ScanArgs& a, const Units& un, int u) const {
        return g * (a.H / a.G) + (unit0 + u) / un.blocks;
    }
    __device__ int col0(const Units& un, int u) const { return 64 * ((unit0 + u) % un.blocks); }
};

__device__ __forceinline__ Place place(const ScanArgs& a, const Units& un) {
    Place p;
    const int pair = blockIdx.x % un.pairs;
    p.g = blockIdx.x / un.pairs;
    p.seg = blockIdx.y;
    p.b = blockIdx.z;
    p.unit0 = 2 * pair;
    p.nu = min(2, un.units - p.unit0);
    p.n = a.lengths ? min(max(a.lengths[p.b], 0), a.N) : a.N;
    p.c0 = p.seg * un.cps;
    p.nc = min(max((p.n + kC - 1) / kC - p.c0, 0), un.cps);
    return p;
}

// Step sizes of chunk c of head h: lane l holds tokens 4l .. 4l + 3.
__device__ __forceinline__ void load_steps(const ScanArgs& a, const Place& pl, int h, int c,
                                           float (&v)[4]) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.step) + pl.b * a.step_bs + h;
    const int t = c * kC + 4 * (threadIdx.x & 31);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        v[k] = t + k < pl.n ? __bfloat162float(p[(int64_t)(t + k) * a.step_ts]) : 0.f;
}

// Inclusive sums from the chunk's start (cum) and exclusive sums from its end
// (suf) of d A log2 e over the 128 tokens, and the step sizes themselves.
__device__ __forceinline__ void decays(const ScanArgs& a, const Place& pl, int c, float A2, float bias,
                                       const float (&raw)[4], float (&d)[4], float (&cum)[4],
                                       float (&suf)[4], float* total) {
    const int lane = threadIdx.x & 31, t = c * kC + 4 * lane;
    float l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        d[k] = t + k < pl.n ? step_size(raw[k] + bias, a.softplus) : 0.f;
        l[k] = d[k] * A2;
    }
    const float own = (l[0] + l[1]) + (l[2] + l[3]);
    float up = own, down = own;              // inclusive scans over lanes, both directions
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o);
        const float y = __shfl_down_sync(0xffffffffu, down, o);
        if (lane >= o) up += x;
        if (lane + o < 32) down += y;
    }
    *total = __shfl_sync(0xffffffffu, down, 0);
    float before = __shfl_up_sync(0xffffffffu, up, 1), after = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 0) before = 0.f;
    if (lane == 31) after = 0.f;
    cum[0] = before + l[0];
    cum[1] = cum[0] + l[1];
    cum[2] = cum[1] + l[2];
    cum[3] = cum[2] + l[3];
    suf[3] = after;
    suf[2] = suf[3] + l[3];
    suf[1] = suf[2] + l[2];
    suf[0] = suf[1] + l[1];
}

// Row `row` of the weighted values: hi = bf16(w x), lo = bf16(w x - hi).
__device__ __forceinline__ void weigh_row(const uint8_t* x, uint8_t* hi, uint8_t* lo, int row, float w) {
    const uint64_t w2 = pk2(w, w), minus = pk2(-1.f, -1.f);
    const uint32_t base = row * 128;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t off = base + ((j ^ (row & 7)) << 4);
        const uint4 v = *reinterpret_cast<const uint4*>(x + off);
        const uint32_t in[4] = {v.x, v.y, v.z, v.w};
        uint32_t h[4], l[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t p = mul2(bf2(in[k]), w2);
            h[k] = pack2(p);
            l[k] = pack2(fma2(bf2(h[k]), minus, p));
        }
        *reinterpret_cast<uint4*>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

// Rows from `from` on of a [128 x 64] tile set to 0 by its four warps (thread = row).
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(tile + row * 128 + j * 16) = make_uint4(0, 0, 0, 0);
}

// (4): state += B^T (hi + lo), issued by one thread. The second 64-row atom of the
// A operand is the next tile (for kT = 1 whatever tile follows: those lanes are unused).
__device__ __forceinline__ void issue_state(uint32_t dst, uint32_t bt, uint32_t hi, uint32_t lo, bool fresh) {
    const uint32_t id = idesc_bf16_f32(128, 64, true, true);
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)
            mma_bf16(dst, smem_desc(bt + k * 2048, kTile, 1024, kSwizzle128B),
                     smem_desc((part ? lo : hi) + k * 2048, 1024, 1024, kSwizzle128B), id,
                     (fresh && part == 0 && k == 0) ? 0u : 1u);
}

// `pieces` times 8 gate values of a row, zeros past them: 16-byte loads where the
// rows are aligned, else one value at a time.
__device__ __forceinline__ void load_gate(const __nv_bfloat16* p, int pieces, bool vec, uint4 (&z)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        z[j] = make_uint4(0, 0, 0, 0);
        if (j >= pieces) continue;
        if (vec) {
            z[j] = __ldg(reinterpret_cast<const uint4*>(p) + j);
        } else {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned short lo = __ldg(reinterpret_cast<const unsigned short*>(p) + 8 * j + 2 * k);
                const unsigned short hi = __ldg(reinterpret_cast<const unsigned short*>(p) + 8 * j + 2 * k + 1);
                w[k] = (uint32_t)lo | ((uint32_t)hi << 16);
            }
            z[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

template <int kT>
__global__ void __launch_bounds__(kThreads, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap cmap, const __grid_constant__ ScanArgs a,
               const __grid_constant__ Units un, WsHeader* hdr) {
    using L = Smem<kT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    Decay* dts = reinterpret_cast<Decay*>(base + L::kDt);
    uint8_t* sb = base + L::kSb;
    uint8_t *xw_hi = base + L::kXw, *xw_lo = xw_hi + kTile;
    auto ctile = [&](int s) { return base + s * L::kStage; };
    auto btile = [&](int s) { return base + s * L::kStage + kT * kTile; };
    auto xtile = [&](int n) { return base + L::kX + (n & 1) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, un);
    const bool last_seg = pl.seg == a.nseg - 1;
    if (pl.nc == 0 && !(last_seg && a.S_out)) return;
    const int nu = pl.nu, items = pl.nc * nu;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.bc_full[s], 1);
            mbar_init(&m.bc_empty[s], 1);
            mbar_init(&m.x_full[s], 1);
            mbar_init(&m.x_empty[s], 9);      // weights, output (4 warps each), (3)
            mbar_init(&m.p_full[s], 4);
            mbar_init(&m.p_empty[s], 1);
            mbar_init(&m.st_full[s], 1);
        }
        for (int s = 0; s < kDtRing; ++s) {
            mbar_init(&m.dt_full[s], 1);
            mbar_init(&m.dt_empty[s], 12 + 2 * kT);
        }
        mbar_init(&m.sc_full, 1);
        mbar_init(&m.sc_empty, 4);
        mbar_init(&m.xw_full, 4);
        mbar_init(&m.xw_empty, 1);
        mbar_init(&m.sb_full, 2 * kT);
        mbar_init(&m.sb_empty, 1);
        mbar_init(&m.y_full, 1);
        mbar_init(&m.y_empty, 4);
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&m.tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&bmap);
        tma_prefetch_desc(&cmap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;                 // test hook: loads never issued
    const int q = warp & 3, row = 32 * q + lane;           // TMEM lane quarter, tile row
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            int i = 0, n = 0;
            for (; i < pl.nc && ok && !hold; ++i) {
                const int s = i & 1, t = (pl.c0 + i) * kC;
                if (i >= 2 && !(ok = mbar_wait(&m.bc_empty[s], ((i >> 1) - 1) & 1, max_spin))) break;
                mbar_arrive_expect_tx(&m.bc_full[s], 2 * kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k) {
                    tma_load_4d(ctile(s) + k * kTile, &cmap, &m.bc_full[s], 64 * k, pl.g, t, pl.b);
                    tma_load_4d(btile(s) + k * kTile, &bmap, &m.bc_full[s], 64 * k, pl.g, t, pl.b);
                }
                for (int u = 0; u < nu; ++u, ++n) {
                    if (n >= 2 && !(ok = mbar_wait(&m.x_empty[n & 1], ((n >> 1) - 1) & 1, max_spin))) break;
                    mbar_arrive_expect_tx(&m.x_full[n & 1], kTile);
                    tma_load_4d(xtile(n), &xmap, &m.x_full[n & 1], pl.col0(un, u), pl.head(a, un, u), t, pl.b);
                }
            }
            // Every issued load (i chunks, n value tiles) lands before the CTA exits.
            for (int j = max(i - 2, 0); j < i; ++j) mbar_wait(&m.bc_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
            for (int j = max(n - 2, 0); j < n; ++j) mbar_wait(&m.x_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA
        if (lane == 0) {
            const uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
            const uint32_t id_y = idesc_bf16_f32(128, 64, false, true);
            const uint32_t sba = smem_u32(sb), hia = smem_u32(xw_hi), loa = smem_u32(xw_lo);
            auto scores = [&](int i) -> bool {
                if (!mbar_wait(&m.bc_full[i & 1], (i >> 1) & 1, max_spin) ||
                    (i >= 1 && !mbar_wait(&m.sc_empty, (i - 1) & 1, max_spin)))
                    return false;
                tc_fence_after();
                const uint32_t ca = smem_u32(ctile(i & 1)), ba = smem_u32(btile(i & 1));
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k) {
                    const uint32_t off = (k >> 2) * kTile + (k & 3) * 32;
                    mma_bf16(tmem + kTmSc, smem_desc(ca + off, 16, 1024, kSwizzle128B),
                             smem_desc(ba + off, 16, 1024, kSwizzle128B), id_sc, k > 0);
                }
                mma_commit(&m.sc_full);
                return true;
            };
            if (pl.nc > 0) ok = scores(0);
            for (int n = 0, i = 0, u = 0; n < items && ok; ++n) {
                const int s = i & 1;
                const uint32_t ca = smem_u32(ctile(s)), ba = smem_u32(btile(s)), xa = smem_u32(xtile(n));
                // (2)
                if (!(ok = mbar_wait(&m.sb_full, n & 1, max_spin) &&
                           (n < 1 || mbar_wait(&m.y_empty, (n - 1) & 1, max_spin))))
                    break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k)
                    mma_bf16(tmem + kTmY2, smem_desc(ca + (k >> 2) * kTile + (k & 3) * 32, 16, 1024, kSwizzle128B),
                             smem_desc(sba + k * 2048, 1024, 1024, kSwizzle128B), id_y, k > 0);
                mma_commit(&m.sb_empty);
                // (1) of the next chunk as soon as this chunk's scores have been read.
                if (u == nu - 1 && i + 1 < pl.nc && !(ok = scores(i + 1))) break;
                // (3)
                if (!(ok = mbar_wait(&m.p_full[n & 1], (n >> 1) & 1, max_spin) &&
                           mbar_wait(&m.x_full[n & 1], (n >> 1) & 1, max_spin)))
                    break;
                // Rows past a ragged end are cleared by the weights' warps first.
                const bool ragged = a.lengths && (pl.c0 + i + 1) * kC > pl.n;
                if (ragged && !(ok = mbar_wait(&m.xw_full, n & 1, max_spin))) break;
                tc_fence_after();
                const uint32_t pt = tmem + kTmP + 64 * (n & 1);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)
                    mma_bf16_ts(tmem + kTmY1, pt + 8 * k, smem_desc(xa + k * 2048, 1024, 1024, kSwizzle128B),
                                id_y, k > 0);
                mma_commit(&m.p_empty[n & 1]);
                mma_commit(&m.x_empty[n & 1]);
                mma_commit(&m.y_full);
                // (4)
                if (!(ok = mbar_wait(&m.xw_full, n & 1, max_spin))) break;
                tc_fence_after();
                issue_state(tmem + kTmSt + 64 * u, ba, hia, loa, false);
                mma_commit(&m.xw_empty);
                mma_commit(&m.st_full[u]);
                if (++u == nu) {
                    mma_commit(&m.bc_empty[s]);
                    u = 0;
                    ++i;
                }
            }
            mma_commit(&m.drain);              // every issued MMA completes before TMEM is released
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
    } else if (warp < 4) {
        // ------------------------------------------------------------ decays, unit warp - 2
        const int u = warp - 2;
        if (u < nu && pl.nc > 0) {
            const int h = pl.head(a, un, u);
            const float A2 = a.A[h] * kLog2e, bias = a.step_bias ? a.step_bias[h] : 0.f;
            float raw[4];
            load_steps(a, pl, h, pl.c0, raw);
            for (int i = 0; i < pl.nc; ++i) {
                const int n = i * nu + u, slot = n % kDtRing;
                float next[4] = {};
                if (i + 1 < pl.nc) load_steps(a, pl, h, pl.c0 + i + 1, next);
                float d[4], cum[4], suf[4], total;
                decays(a, pl, pl.c0 + i, A2, bias, raw, d, cum, suf, &total);
                if (n >= kDtRing && !(ok = warp_wait(&m.dt_empty[slot], (n / kDtRing - 1) & 1, max_spin))) break;
                Decay& o = dts[slot];
                *reinterpret_cast<float4*>(o.cum + 4 * lane) = make_float4(cum[0], cum[1], cum[2], cum[3]);
                *reinterpret_cast<float4*>(o.d + 4 * lane) = make_float4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<float4*>(o.w + 4 * lane) =
                    make_float4(d[0] * exp2f(suf[0]), d[1] * exp2f(suf[1]), d[2] * exp2f(suf[2]), d[3] * exp2f(suf[3]));
                if (lane == 0) o.total = exp2f(total);
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.dt_full[slot]);
#pragma unroll
                for (int k = 0; k < 4; ++k) raw[k] = next[k];
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------ scores -> P
        float* col = reinterpret_cast<float*>(base + L::kCol) + q * 96;
        // Blocks above the diagonal are zero in both buffers, once.
        {
            const uint32_t z[16] = {};
            for (int b = q + 1; b < 4; ++b) {
                tmem_st16(tmem + lanes + kTmP + 16 * b, z);
                tmem_st16(tmem + lanes + kTmP + 64 + 16 * b, z);
            }
            tmem_st_wait();
        }
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            const int slot = n % kDtRing;
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin))) break;
            const Decay& dc = dts[slot];
            const float ci = dc.cum[row];
            const float cm = q ? dc.cum[32 * q - 1] : 0.f;
            for (int b = 0; b < q; ++b)
                col[32 * b + lane] = ex2(cm - dc.cum[32 * b + lane]) * dc.d[32 * b + lane];
            __syncwarp();
            const float ri = ex2(ci - cm);
            const uint64_t r2 = pk2(ri, ri);
            if (u == 0 && !(ok = warp_wait(&m.sc_full, i & 1, max_spin))) break;
            if (n >= 2 && !(ok = warp_wait(&m.p_empty[n & 1], ((n >> 1) - 1) & 1, max_spin))) break;
            tc_fence_after();
            const uint32_t src = tmem + lanes + kTmSc, dst = tmem + lanes + kTmP + 64 * (n & 1);
            for (int b = 0; b < q; ++b) {
                uint32_t s0[16], s1[16], p[16];
                tmem_ld16(src + 32 * b, s0);
                tmem_ld16(src + 32 * b + 16, s1);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 f = *reinterpret_cast<const float4*>(col + 32 * b + 2 * e);
                    const uint32_t* s = e < 8 ? s0 + 2 * e : s1 + 2 * e - 16;
                    p[e] = pack2(mul2(mul2(pk2(__uint_as_float(s[0]), __uint_as_float(s[1])), pk2(f.x, f.y)), r2));
                    p[e + 1] = pack2(mul2(mul2(pk2(__uint_as_float(s[2]), __uint_as_float(s[3])), pk2(f.z, f.w)), r2));
                }
                tmem_st16(dst + 16 * b, p);
            }
            {
                uint32_t s0[16], s1[16], p[16];
                tmem_ld16(src + 32 * q, s0);
                tmem_ld16(src + 32 * q + 16, s1);
                tmem_ld_wait();
                if (u == nu - 1) {             // the chunk's scores have been read
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.sc_empty);
                }
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    const float4 l = *reinterpret_cast<const float4*>(dc.cum + 32 * q + 2 * e);
                    const float4 d = *reinterpret_cast<const float4*>(dc.d + 32 * q + 2 * e);
                    const uint32_t* s = e < 8 ? s0 + 2 * e : s1 + 2 * e - 16;
                    const float lj[4] = {l.x, l.y, l.z, l.w}, dj[4] = {d.x, d.y, d.z, d.w};
                    float v[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[k] = 2 * e + k <= lane ? __uint_as_float(s[k]) * (ex2(ci - lj[k]) * dj[k]) : 0.f;
                    p[e] = pack_bf16(v[0], v[1]);
                    p[e + 1] = pack_bf16(v[2], v[3]);
                }
                tmem_st16(dst + 16 * q, p);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.p_full[n & 1]);
                mbar_arrive(&m.dt_empty[slot]);
            }
            if (++u == nu) u = 0, ++i;
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------ state
        if (q < 2 * kT) {
            const int64_t head_state = (int64_t)a.S * a.P;
            // The state before the first chunk: row `row` of each unit.
            for (int u = 0; u < nu; ++u) {
                const int64_t bh = (int64_t)pl.b * a.H + pl.head(a, un, u);
                const float* from = a.nseg > 1 ? a.seeds + (bh * a.nseg + pl.seg) * head_state
                                               : (a.S0 ? a.S0 + bh * head_state : nullptr);
                const int p0 = pl.col0(un, u), np = min(64, a.P - p0);
                const float* r = from && row < a.S ? from + (int64_t)row * a.P + p0 : nullptr;
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    uint32_t v[16];
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const uint4 x = r && c + k < np ? *reinterpret_cast<const uint4*>(r + c + k) : make_uint4(0, 0, 0, 0);
                        v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
                    }
                    tmem_st16(tmem + lanes + kTmSt + 64 * u + c, v);
                }
            }
            tmem_st_wait();
            for (int n = 0, i = 0, u = 0; n < items; ++n) {
                const int slot = n % kDtRing;
                if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin) &&
                           (i < 1 || warp_wait(&m.st_full[u], (i - 1) & 1, max_spin)) &&
                           (n < 1 || warp_wait(&m.sb_empty, (n - 1) & 1, max_spin))))
                    break;
                tc_fence_after();
                const float f = dts[slot].total;
                const uint64_t f2 = pk2(f, f);
                const uint32_t st = tmem + lanes + kTmSt + 64 * u;
#pragma unroll
                for (int c = 0; c < 64; c += 32) {
                    uint32_t v[2][16];
                    tmem_ld16(st + c, v[0]);
                    tmem_ld16(st + c + 16, v[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        uint32_t h[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint64_t x = pk2(__uint_as_float(v[k][2 * e]), __uint_as_float(v[k][2 * e + 1]));
                            h[e] = row < a.S ? pack2(x) : 0u;
                            float lo, hi;
                            unpk2(mul2(x, f2), &lo, &hi);
                            v[k][2 * e] = __float_as_uint(lo);
                            v[k][2 * e + 1] = __float_as_uint(hi);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            *reinterpret_cast<uint4*>(sb + sw128_offset(row, c + 16 * k + 8 * e)) =
                                make_uint4(h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]);
                        tmem_st16(st + c + 16 * k, v[k]);
                    }
                }
                tmem_st_wait();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&m.sb_full);
                    mbar_arrive(&m.dt_empty[slot]);
                }
                if (++u == nu) u = 0, ++i;
            }
            // The final state.
            if (ok && last_seg && a.S_out) {
                for (int u = 0; u < nu && ok; ++u) {
                    if (pl.nc > 0 && !(ok = warp_wait(&m.st_full[u], (pl.nc - 1) & 1, max_spin))) break;
                    tc_fence_after();
                    const int64_t bh = (int64_t)pl.b * a.H + pl.head(a, un, u);
                    const int p0 = pl.col0(un, u), np = min(64, a.P - p0);
                    float* r = a.S_out + bh * head_state + (int64_t)row * a.P + p0;
#pragma unroll
                    for (int c = 0; c < 64; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(tmem + lanes + kTmSt + 64 * u + c, v);
                        tmem_ld_wait();
                        if (row >= a.S) continue;
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            if (c + k < np)
                                *reinterpret_cast<uint4*>(r + c + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                    }
                }
            }
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------ weighted values
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            const int slot = n % kDtRing;
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin) &&
                       warp_wait(&m.x_full[n & 1], (n >> 1) & 1, max_spin) &&
                       (n < 1 || warp_wait(&m.xw_empty, (n - 1) & 1, max_spin))))
                break;
            // Rows at or past a ragged end may hold anything: they are cleared in x, and in B
            // for (4). (1) may read such rows of B, whose scores no kept row uses.
            if (a.lengths && (pl.c0 + i + 1) * kC > pl.n) {        // uniform over the block
                if (!(ok = warp_wait(&m.bc_full[i & 1], (i >> 1) & 1, max_spin))) break;
                if ((pl.c0 + i) * kC + row >= pl.n) {
                    zero_row(xtile(n), row);
                    for (int k = 0; k < kT && u == 0; ++k) zero_row(btile(i & 1) + k * kTile, row);
                }
            }
            weigh_row(xtile(n), xw_hi, xw_lo, row, dts[slot].w[row]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.xw_full);
                mbar_arrive(&m.x_empty[n & 1]);
                mbar_arrive(&m.dt_empty[slot]);
            }
            if (++u == nu) u = 0, ++i;
        }
    } else {
        // ------------------------------------------------------------ output
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            const int slot = n % kDtRing;
            const int t = (pl.c0 + i) * kC + row, h = pl.head(a, un, u), p0 = pl.col0(un, u);
            const int pieces = min(64, a.P - p0) >> 3;
            const bool live = t < pl.n;
            const __nv_bfloat16* zr = static_cast<const __nv_bfloat16*>(a.z) + pl.b * a.z_bs +
                                      (int64_t)t * a.z_ts + (int64_t)h * a.P + p0;
            __nv_bfloat16* yr = static_cast<__nv_bfloat16*>(a.y) + pl.b * a.y_bs + (int64_t)t * a.y_ts +
                                (int64_t)h * a.P + p0;
            uint4 z[8];
            if (a.z) load_gate(zr, live ? pieces : 0, un.gate_vec != 0, z);
            const float Dh = a.D ? a.D[h] : 0.f;
            const uint64_t D2 = pk2(Dh, Dh);
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin) &&
                       warp_wait(&m.x_full[n & 1], (n >> 1) & 1, max_spin) &&
                       warp_wait(&m.y_full, n & 1, max_spin)))
                break;
            tc_fence_after();
            const float e = ex2(dts[slot].cum[row]);
            const uint64_t e2 = pk2(e, e);
            const uint8_t* xr = xtile(n) + row * 128;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t y1[16], y2[16];
                tmem_ld16(tmem + lanes + kTmY1 + 16 * c, y1);
                tmem_ld16(tmem + lanes + kTmY2 + 16 * c, y2);
                tmem_ld_wait();
                if (c == 3) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m.y_empty);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int piece = 2 * c + j;
                    const uint4 xv = *reinterpret_cast<const uint4*>(xr + ((piece ^ (row & 7)) << 4));
                    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w};
                    const uint32_t zs[4] = {z[piece].x, z[piece].y, z[piece].z, z[piece].w};
                    uint32_t out[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = 8 * j + 2 * k;
                        uint64_t v = fma2(e2, pk2(__uint_as_float(y2[at]), __uint_as_float(y2[at + 1])),
                                          pk2(__uint_as_float(y1[at]), __uint_as_float(y1[at + 1])));
                        v = fma2(D2, bf2(xs[k]), v);
                        if (a.z) {
                            const float z0 = __uint_as_float(zs[k] << 16), z1 = __uint_as_float(zs[k] & 0xFFFF0000u);
                            v = mul2(v, pk2(silu(z0), silu(z1)));
                        }
                        out[k] = pack2(v);
                    }
                    if (live && piece < pieces)
                        reinterpret_cast<uint4*>(yr)[piece] = make_uint4(out[0], out[1], out[2], out[3]);
                }
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.x_empty[n & 1]);
                mbar_arrive(&m.dt_empty[slot]);
            }
            if (++u == nu) u = 0, ++i;
        }
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// First pass over segments: end state from zero, sum over the segment of
// B_j (d_j e^{l(end) - l_j} x_j)^T, and the segment's total decay. Chunks run from
// the last to the first; the weights carry the sum of the chunks after them.
// Warps: TMA, MMA, decays (two), then two weight groups of four that alternate.
constexpr int kSumThreads = 384;

struct SumMisc {
    uint64_t b_full[2], b_empty[2], x_full[4], x_empty[4], dt_full[kDtRing], dt_empty[kDtRing];
    uint64_t xw_full[2], xw_empty[2], drain;
    uint32_t tmem_slot;
};

template <int kT> struct SumSmem {
    static constexpr uint32_t kX = 2 * kT * kTile;
    static constexpr uint32_t kXw = kX + 4 * kTile;
    static constexpr uint32_t kW = kXw + 4 * kTile;
    static constexpr uint32_t kMisc = kW + kDtRing * kC * 4;
    static constexpr size_t kBytes = 1024 + kMisc + sizeof(SumMisc);
};

template <int kT>
__global__ void __launch_bounds__(kSumThreads, 1)
scan_sums_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap bmap,
                 const __grid_constant__ ScanArgs a, const __grid_constant__ Units un, WsHeader* hdr) {
    using L = SumSmem<kT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    SumMisc& m = *reinterpret_cast<SumMisc*>(base + L::kMisc);
    float* wts = reinterpret_cast<float*>(base + L::kW);
    auto btile = [&](int s) { return base + s * kT * kTile; };
    auto xtile = [&](int n) { return base + L::kX + (n & 3) * kTile; };
    auto xwtile = [&](int n) { return base + L::kXw + (n & 1) * 2 * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, un);
    const int nu = pl.nu, items = pl.nc * nu, c_last = pl.c0 + pl.nc - 1;
    const int64_t head_state = (int64_t)a.S * a.P;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.b_full[s], 1);
            mbar_init(&m.b_empty[s], 1);
            mbar_init(&m.xw_full[s], 4);
            mbar_init(&m.xw_empty[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&m.x_full[s], 1);
            mbar_init(&m.x_empty[s], 4);
            mbar_init(&m.dt_full[s], 1);
            mbar_init(&m.dt_empty[s], 4);
        }
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&m.tmem_slot, 128);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;                 // test hook: loads never issued
    const int q = warp & 3, row = 32 * q + lane;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            int i = 0, n = 0;
            for (; i < pl.nc && ok && !hold; ++i) {
                const int s = i & 1, t = (c_last - i) * kC;
                if (i >= 2 && !(ok = mbar_wait(&m.b_empty[s], ((i >> 1) - 1) & 1, max_spin))) break;
                mbar_arrive_expect_tx(&m.b_full[s], kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    tma_load_4d(btile(s) + k * kTile, &bmap, &m.b_full[s], 64 * k, pl.g, t, pl.b);
                for (int u = 0; u < nu; ++u, ++n) {
                    if (n >= 4 && !(ok = mbar_wait(&m.x_empty[n & 3], ((n >> 2) - 1) & 1, max_spin))) break;
                    mbar_arrive_expect_tx(&m.x_full[n & 3], kTile);
                    tma_load_4d(xtile(n), &xmap, &m.x_full[n & 3], pl.col0(un, u), pl.head(a, un, u), t, pl.b);
                }
            }
            for (int j = max(i - 2, 0); j < i; ++j) mbar_wait(&m.b_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
            for (int j = max(n - 4, 0); j < n; ++j) mbar_wait(&m.x_full[j & 3], (j >> 2) & 1, kDefaultMaxSpin);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            for (int n = 0, i = 0, u = 0; n < items; ++n) {
                if (!(ok = mbar_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin) &&
                           mbar_wait(&m.xw_full[n & 1], (n >> 1) & 1, max_spin)))
                    break;
                tc_fence_after();
                const uint32_t xw = smem_u32(xwtile(n));
                issue_state(tmem + 64 * u, smem_u32(btile(i & 1)), xw, xw + kTile, i == 0);
                mma_commit(&m.xw_empty[n & 1]);
                if (++u == nu) {
                    mma_commit(&m.b_empty[i & 1]);
                    u = 0;
                    ++i;
                }
            }
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
    } else if (warp < 4) {
        const int u = warp - 2;
        if (u < nu) {
            const int h = pl.head(a, un, u);
            const float A2 = a.A[h] * kLog2e, bias = a.step_bias ? a.step_bias[h] : 0.f;
            float raw[4] = {}, after = 0.f;            // after: sum over the chunks behind
            if (pl.nc > 0) load_steps(a, pl, h, c_last, raw);
            for (int i = 0; i < pl.nc; ++i) {
                const int n = i * nu + u, slot = n % kDtRing;
                float next[4] = {};
                if (i + 1 < pl.nc) load_steps(a, pl, h, c_last - i - 1, next);
                float d[4], cum[4], suf[4], total;
                decays(a, pl, c_last - i, A2, bias, raw, d, cum, suf, &total);
                if (n >= kDtRing && !(ok = warp_wait(&m.dt_empty[slot], (n / kDtRing - 1) & 1, max_spin))) break;
                *reinterpret_cast<float4*>(wts + slot * kC + 4 * lane) =
                    make_float4(d[0] * exp2f(suf[0] + after), d[1] * exp2f(suf[1] + after),
                                d[2] * exp2f(suf[2] + after), d[3] * exp2f(suf[3] + after));
                after += total;
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.dt_full[slot]);
#pragma unroll
                for (int k = 0; k < 4; ++k) raw[k] = next[k];
            }
            if (lane == 0 && pl.col0(un, u) == 0)
                a.seg_decay[((int64_t)pl.b * a.H + h) * a.nseg + pl.seg] = after * kLn2;
        }
    } else {
        const int grp = (warp - 4) >> 2;
        for (int n = grp; n < items; n += 2) {
            const int slot = n % kDtRing, i = n / nu, u = n - i * nu;
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin) &&
                       warp_wait(&m.x_full[n & 3], (n >> 2) & 1, max_spin) &&
                       (n < 2 || warp_wait(&m.xw_empty[n & 1], ((n >> 1) - 1) & 1, max_spin))))
                break;
            if (a.lengths && (c_last - i + 1) * kC > pl.n) {
                if (!(ok = warp_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin))) break;
                if ((c_last - i) * kC + row >= pl.n) {
                    zero_row(xtile(n), row);
                    for (int k = 0; k < kT && u == 0; ++k) zero_row(btile(i & 1) + k * kTile, row);
                }
            }
            weigh_row(xtile(n), xwtile(n), xwtile(n) + kTile, row, wts[slot * kC + row]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.xw_full[n & 1]);
                mbar_arrive(&m.x_empty[n & 3]);
                mbar_arrive(&m.dt_empty[slot]);
            }
        }
        if (grp == 0 && ok && (pl.nc == 0 || (ok = warp_wait(&m.drain, 0, max_spin)))) {
            tc_fence_after();
            for (int u = 0; u < nu; ++u) {
                const int64_t bh = (int64_t)pl.b * a.H + pl.head(a, un, u);
                const int p0 = pl.col0(un, u), np = min(64, a.P - p0);
                float* r = a.seeds + (bh * a.nseg + pl.seg) * head_state + (int64_t)row * a.P + p0;
#pragma unroll
                for (int c = 0; c < 64; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tmem + ((uint32_t)(32 * q) << 16) + 64 * u + c, v);
                    tmem_ld_wait();
                    if (row >= a.S) continue;
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (c + k < np)
                            *reinterpret_cast<uint4*>(r + c + k) =
                                pl.nc > 0 ? make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]) : make_uint4(0, 0, 0, 0);
                }
            }
        }
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 128);
}

// Rows [B, N, outer, inner] of bf16 as a 4-D map with boxes of 64 values x 128 tokens;
// values past `inner` and tokens past N read as zero.
bool encode_rows(CUtensorMap* map, const void* p, int inner, int outer, int N, int B, int64_t ts,
                 int64_t bs) {
    EncodeTiled enc = get_encoder();
    if (!enc) return false;
    if (B == 1) bs = ts;                              // any valid stride: never used
    if (N == 1) ts = (int64_t)inner * outer;
    if (B == 1) bs = ts;
    cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)outer, (cuuint64_t)N, (cuuint64_t)B};
    cuuint64_t strides[3] = {(cuuint64_t)inner * 2, (cuuint64_t)ts * 2, (cuuint64_t)bs * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1}, es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

Units units_of(int H, int G, int P) {
    Units un = {};
    un.blocks = (P + 63) / 64;
    un.units = (G > 0 ? H / G : H) * un.blocks;
    un.pairs = (un.units + 1) / 2;
    return un;
}

// CTAs run in waves over the SMs, so the number of segments is the one whose
// waves times chunks is least. In units of one chunk of the main pass: a CTA
// spends about two on starting and ending, the first pass 0.4 per chunk, and
// two further launches about two.
int pick_segments(int64_t ctas, int N) {
    const int nch = (N + kC - 1) / kC, sms = sm_count();
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 64 && n <= nch; ++n) {
        const int cps = (nch + n - 1) / n;
        if ((nch + cps - 1) / cps != n) continue;      // the same split with empty segments
        const double waves = (double)((ctas * n + sms - 1) / sms);
        const double cost = waves * (cps + 2.0) + (n > 1 ? waves * (0.4 * cps + 1.5) + 2.0 : 0.0);
        if (cost < least) least = cost, best = n;
    }
    return best;
}

template <int kT>
cudaError_t launch(const CUtensorMap& xm, const CUtensorMap& bm, const CUtensorMap& cm, const ScanArgs& a,
                   const Units& un, int B, WsHeader* hdr, cudaStream_t st) {
    static std::atomic<int> optin[kMaxDevices], optin_sums[kMaxDevices];
    cudaError_t e = ensure_smem_optin(scan_tc_kernel<kT>, (int)Smem<kT>::kBytes, optin);
    if (e != cudaSuccess) return e;
    const dim3 grid(un.pairs * a.G, a.nseg, B);
    if (a.nseg > 1) {
        e = ensure_smem_optin(scan_sums_kernel<kT>, (int)SumSmem<kT>::kBytes, optin_sums);
        if (e != cudaSuccess) return e;
        scan_sums_kernel<kT><<<grid, kSumThreads, SumSmem<kT>::kBytes, st>>>(xm, bm, a, un, hdr);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        if ((e = launch_seeds(a, (int64_t)B * a.H, st)) != cudaSuccess) return e;
    }
    scan_tc_kernel<kT><<<grid, kThreads, Smem<kT>::kBytes, st>>>(xm, bm, cm, a, un, hdr);
    return cudaPeekAtLastError();
}

}  // namespace

namespace scan {

bool tc_supported(const ScanArgs& a, int B, la_dtype dt) {
    if (dt != LA_BF16 || a.S % 8 || a.P % 8) return false;
    auto rows = [&](const void* p, int64_t ts, int64_t bs) {
        const int64_t most = (int64_t)1 << 38;             // strides stay below 2^40 bytes
        return (reinterpret_cast<uintptr_t>(p) & 15) == 0 &&
               (a.N == 1 || (ts > 0 && ts % 8 == 0 && ts < most)) &&
               (B == 1 || (bs > 0 && bs % 8 == 0 && bs < most));
    };
    if ((reinterpret_cast<uintptr_t>(a.S0) | reinterpret_cast<uintptr_t>(a.S_out)) & 15) return false;
    return rows(a.x, a.x_ts, a.x_bs) && rows(a.Bm, a.b_ts, a.b_bs) && rows(a.Cm, a.c_ts, a.c_bs) &&
           rows(a.y, a.y_ts, a.y_bs);
}

int tc_segments(int64_t B, int H, int G, int N, int P) {
    const Units un = units_of(H, G, P);
    return pick_segments(B * G * un.pairs, N);
}

cudaError_t tc_scan(ScanArgs& a, int B, void* ws_header, cudaStream_t st) {
    Units un = units_of(a.H, a.G, a.P);
    const int nch = (a.N + kC - 1) / kC;
    un.cps = (nch + a.nseg - 1) / a.nseg;
    un.gate_vec = (reinterpret_cast<uintptr_t>(a.z) & 15) == 0 && (a.N == 1 || a.z_ts % 8 == 0) &&
                  (B == 1 || a.z_bs % 8 == 0);
    CUtensorMap xm, bm, cm;
    if (!encode_rows(&xm, a.x, a.P, a.H, a.N, B, a.x_ts, a.x_bs) ||
        !encode_rows(&bm, a.Bm, a.S, a.G, a.N, B, a.b_ts, a.b_bs) ||
        !encode_rows(&cm, a.Cm, a.S, a.G, a.N, B, a.c_ts, a.c_bs))
        return cudaErrorInvalidValue;
    WsHeader* hdr = static_cast<WsHeader*>(ws_header);
    return a.S <= 64 ? launch<1>(xm, bm, cm, a, un, B, hdr, st) : launch<2>(xm, bm, cm, a, un, B, hdr, st);
}

}  // namespace scan

}  // namespace la
