// Decayed linear attention on the tensor cores (tcgen05): bf16, Da and Dc multiples of 8,
// 16-byte aligned rows. Definitions in csrc/decay.cuh and csrc/decay.cu.
//
// Method. For a chunk of 128 tokens of one head with the state S before it, i and j counted
// within the chunk in the order of summation (backwards where time is reversed), f = e^l:
//   o_i   = scale (f^(i+1) A_i^T S + sum_{j <= i} f^(i-j) (A_i . B_j) C_j)
//   S_new = f^m S + sum_j B_j (f^(m-1-j) C_j)^T          (m tokens in the chunk)
// as products of 128-row tiles:
//   (1) scores A B^T                      M = 128, N = 128, K = Da
//   (2) read of the state A S_bf16        M = 128, N = 64,  K = Da
//   (3) P C, P = bf16 of the weighted, masked scores (in TMEM)    K = 128
//   (4) B^T (w C), C weighted             M = Da,  N = 64,  K = 128
// A CTA owns a "unit", 64 columns of C and of the state, and walks the chunks of a segment.
//
// Roundings. A, B, C enter as they are. P and the state of (2) are rounded to bf16 once each
// (half a step, 2^-8, of a term, as the output itself). The state is held in fp32 in
// registers; (4) is summed per chunk from zero and added there, so that the tensor core's
// sums stay short. w C enters it as bf16 terms, each the remainder of those before: two for a
// state that only o reads (2^-16 of w C is left), three for one that the call returns.
// Weights below the diagonal 32 x 32 blocks are products of two factors <= 1, one of the
// row and one of the column; the diagonal blocks take an exponential per score. Every
// factor's exponent is a count of tokens times l, so none is a difference of larger ones.
//
// Schedule. 8 working warps and one that issues loads, products and stores; two CTAs per SM
// (113 KB of shared memory, 256 TMEM columns each), so that one CTA's steps run under the
// other's waits. A working warp owns 32 rows and half of the columns. Hand-offs are
// mbarriers; every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "decay.cuh"
#include "kernels.h"
#include "mixing.cuh"
#include "scan.cuh"
#include "tc_common.cuh"
#include "tc_util.cuh"

namespace la {

using namespace decay;

namespace {

using namespace tc;
using namespace tcc;

constexpr uint32_t kTile = kTileBytes;         // [128 tokens x 64] bf16
constexpr int kWork = 8;                       // working warps
constexpr int kThreads = 32 * (kWork + 1);
constexpr int kNone = 0x7fffffff;

// TMEM columns: scores, whose first half then holds P and whose second half (4), and the two
// parts of the output.
constexpr uint32_t kTmP = 0, kTmSt = 64, kTmO1 = 128, kTmO2 = 192;

struct Misc {
    uint64_t a_full, b_full[2], c_full[2], p_full, o2_full, o_full;
    uint64_t prep, pt, sread, staged, hfree, pair[4], drain;
    uint32_t tmem_slot;
    int any;                    // values of C that are not finite: the first token that has one,
    int first[64];              // and that of each column, counted over the segment
    alignas(16) float tab[32];  // f^(31 - j), by the column's place in its block; read 16 bytes at a time
};
static_assert(sizeof(Misc) <= 1024, "the last kilobyte");

// Shared memory from a 1024-byte boundary. The bf16 state of (2) lies where the second term
// of w C is written once (2) has read it, the output where the first term was.
template <int kT, int kTerms> struct Smem {
    static constexpr int kStages = kT == 1 && kTerms == 2 ? 2 : 1;   // of B and C
    static constexpr uint32_t kA = 0, kB = kT * kTile, kC0 = kB + kStages * kT * kTile;
    static constexpr uint32_t kW = kC0 + kStages * kTile, kS = kW + kTile;
    static constexpr uint32_t kMisc = kW + kTerms * kTile;
    static constexpr int kBytes = kMisc + 1024;
};
static_assert(Smem<1, 2>::kBytes == 113 * 1024 && Smem<2, 2>::kBytes == 113 * 1024, "two CTAs per SM");

// The first pass: B and C, the terms of w C.
template <int kT, int kTerms> struct SumSmem {
    static constexpr int kStages = kT == 1 ? 2 : 1;
    static constexpr uint32_t kB = 0, kC0 = kStages * kT * kTile, kW = kC0 + kStages * kTile;
    static constexpr uint32_t kMisc = kW + kTerms * kTile;
    static constexpr int kBytes = kMisc + 1024;
};

// Coordinate factors of the tensor maps: 0 for an axis of stride 0, whose map has one entry.
struct Geo {
    int cps;                    // chunks per segment
    uint8_t ah, ab, bh, bb, ch, cb;
};

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
__device__ __forceinline__ uint64_t pair2(const uint32_t* v) { return pk2(__uint_as_float(v[0]), __uint_as_float(v[1])); }

// Bounded wait of a whole warp: every lane gets the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t limit_us) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, limit_us));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// Descriptors: steps of 16 rows (or columns) move the start address only.
__device__ __forceinline__ uint64_t step_desc(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }
// Operand with rows of 64 values along M or N (one row per k): steps of 16 rows.
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) { return smem_desc(tile, kTile, 1024, kSwizzle128B); }
// K-major operand (64 k per row of a tile, tiles kTile apart): steps of 16 k.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile) { return smem_desc(tile, 16, 1024, kSwizzle128B); }
__device__ __forceinline__ uint64_t kmajor_step(uint64_t d, int k) {
    return step_desc(d, (k >> 2) * kTile + (k & 3) * 32);
}

// (4), the smallest terms first. The second 64-row atom of the A operand is the tile after
// B's (for kT = 1 whatever tile follows: those lanes are unused).
template <int kTerms>
__device__ __forceinline__ void issue_state(uint32_t dst, uint64_t bt, uint64_t w) {
    constexpr uint32_t id = idesc_bf16_f32(128, 64, true, true);
#pragma unroll
    for (int part = kTerms - 1; part >= 0; --part)
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)
            mma_bf16(dst, step_desc(bt, k * 2048), step_desc(w, part * kTile + k * 2048), id, part < kTerms - 1 || k > 0);
}

// A CTA's place: head, columns, tokens of its sequence, chunks.
struct Place {
    int b, h, col0, seg, n, nch, v0, nc;
    template <bool kRev> __device__ int chunk(int i) const { return kRev ? nch - 1 - v0 - i : v0 + i; }
};
__device__ __forceinline__ Place place(const Args& a, const Geo& geo) {
    Place p;
    p.b = blockIdx.z / a.H;
    p.h = blockIdx.z - p.b * a.H;
    p.col0 = 64 * blockIdx.x;
    p.seg = blockIdx.y;
    p.n = tokens_of(a, p.b);
    p.nch = (p.n + kC - 1) / kC;
    p.v0 = p.seg * geo.cps;
    p.nc = min(max(p.nch - p.v0, 0), geo.cps);
    return p;
}

// Eight weighted values of C: p = w c, its first bf16 term, and the others.
__device__ __forceinline__ void weigh8(uint4 c, uint64_t w2, uint32_t (&hi)[4], uint64_t (&rest)[4]) {
    const uint32_t in[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint64_t p = mul2(bf2(in[k]), w2);
        hi[k] = pack2(p);
        rest[k] = fma2(bf2(hi[k]), pk2(-1.f, -1.f), p);
    }
}
__device__ __forceinline__ void next_term(uint64_t (&rest)[4], uint32_t (&t)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        t[k] = pack2(rest[k]);
        rest[k] = fma2(bf2(t[k]), pk2(-1.f, -1.f), rest[k]);
    }
}

// Columns 32 g .. of row `row` of a C tile: notes the values that are not finite, and clears
// them: (3) would add 0 times them to the tokens before them. (4) has them from the terms.
__device__ __noinline__ void take_out(uint8_t* tile, int row, int g, int token, Misc* m) {
    for (int c = 32 * g; c < 32 * g + 32; ++c) {
        unsigned short* v = reinterpret_cast<unsigned short*>(tile + row * 128 + (((c >> 3) ^ (row & 7)) << 4)) + (c & 7);
        if ((*v & 0x7F80u) != 0x7F80u) continue;
        *v = 0;
        atomicMin(&m->first[c], token);
        atomicMin(&m->any, token);
    }
}

// The outputs that such values reach, set to NaN: columns c .. c + 7 of a row.
__device__ __noinline__ uint4 put_nan(const Misc* m, int c, int token, uint4 o) {
    auto one = [&](uint32_t w, int k) {
        const volatile int* first = m->first + c + k;
        if (first[0] <= token) w = (w & 0xFFFF0000u) | 0x7FFFu;
        if (first[1] <= token) w = (w & 0xFFFFu) | 0x7FFF0000u;
        return w;
    };
    return make_uint4(one(o.x, 0), one(o.y, 2), one(o.z, 4), one(o.w, 6));
}

template <int kT, int kTerms, bool kRev>
__global__ void __launch_bounds__(kThreads, kT == 2 && kTerms == 3 ? 1 : 2)
decay_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap omap,
                const __grid_constant__ Args a, const __grid_constant__ Geo geo, WsHeader* hdr) {
    using L = Smem<kT, kTerms>;
    extern __shared__ __align__(1024) uint8_t base[];
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    auto btile = [&](int i) { return base + L::kB + (i % L::kStages) * kT * kTile; };
    auto ctile = [&](int i) { return base + L::kC0 + (i % L::kStages) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, geo);
    const bool returns = a.S_out && pl.seg == a.nseg - 1;
    if (pl.nc == 0 && !returns) {
        pdl_wait();                            // a dependent launch never ends before what it follows
        return;
    }
    if ((smem_u32(base) & 1023) != 0) {        // the tiles' swizzle needs it; no static shared memory, so it holds
        if (tid == 0) set_status(hdr, LA_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        mbar_init(&m.a_full, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.b_full[s], 1);
            mbar_init(&m.c_full[s], 1);
        }
        for (uint64_t* bar : {&m.p_full, &m.o2_full, &m.o_full, &m.hfree, &m.drain}) mbar_init(bar, 1);
        for (uint64_t* bar : {&m.prep, &m.pt, &m.sread, &m.staged}) mbar_init(bar, kWork);
        for (int s = 0; s < 4; ++s) mbar_init(&m.pair[s], 2);
        fence_mbar_init();
        m.any = kNone;
    }
    if (tid < 64) m.first[tid] = kNone;
    const float l = a.decay[pl.h], l2 = log2_decay(l);
    if (tid < 32) m.tab[tid] = pow2((kRev ? tid : 31 - tid) * l2);
    if (warp == kWork) {
        tmem_alloc(&m.tmem_slot, 256);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();                                // the seeds, where there are segments
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;     // test hook: loads never issued
    bool ok = true;

    if (warp == kWork) {
        if (lane == 0 && pl.nc > 0) {
            const uint32_t base_a = smem_u32(base);
            const uint64_t ak = kmajor_desc(base_a + L::kA), bk = kmajor_desc(base_a + L::kB);
            const uint64_t br = rows_desc(base_a + L::kB), cr = rows_desc(base_a + L::kC0);
            const uint64_t sr = rows_desc(base_a + L::kS), wr = rows_desc(base_a + L::kW);
            constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_o = idesc_bf16_f32(128, 64, false, true);
            int na = 0, nbc = 0;               // chunks of A, of B and C asked for
            auto load_a = [&]() {
                if (hold) return;
                const int t = pl.chunk<kRev>(na) * kC;
                mbar_arrive_expect_tx(&m.a_full, kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    tma_load_4d(base + L::kA + k * kTile, &amap, &m.a_full, 64 * k, geo.ah * pl.h, t, geo.ab * pl.b);
                ++na;
            };
            auto load_bc = [&]() {
                if (hold) return;
                const int t = pl.chunk<kRev>(nbc) * kC, s = nbc % L::kStages;
                mbar_arrive_expect_tx(&m.b_full[s], kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    tma_load_4d(btile(nbc) + k * kTile, &bmap, &m.b_full[s], 64 * k, geo.bh * pl.h, t, geo.bb * pl.b);
                mbar_arrive_expect_tx(&m.c_full[s], kTile);
                tma_load_4d(ctile(nbc), &cmap, &m.c_full[s], pl.col0, geo.ch * pl.h, t, geo.cb * pl.b);
                ++nbc;
            };
            auto scores = [&](int i) -> bool {
                if (!mbar_wait(&m.a_full, i & 1, max_spin) ||
                    !mbar_wait(&m.b_full[i % L::kStages], (i / L::kStages) & 1, max_spin))
                    return false;
                tc_fence_after();
                const uint64_t b = step_desc(bk, (i % L::kStages) * kT * kTile);
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k) mma_bf16(tmem + kTmP, kmajor_step(ak, k), kmajor_step(b, k), id_sc, k > 0);
                mma_commit(&m.p_full);
                return true;
            };
            // The output of chunk i, staged by the working warps; the last, ragged one of a
            // sequence shorter than N was written row by row.
            auto put = [&](int i) -> bool {
                if (!mbar_wait(&m.staged, i & 1, max_spin)) return false;
                const int t = pl.chunk<kRev>(i) * kC;
                if (t + kC <= pl.n || pl.n == a.N) {
                    tma_store_4d(&omap, base + L::kW, pl.col0, pl.h, t, pl.b);
                    tma_store_commit();
                }
                return true;
            };
            load_a();
            for (int s = 0; s < L::kStages && s < pl.nc; ++s) load_bc();
            for (int i = 0; i < pl.nc && ok; ++i) {
                if (i == 0) {
                    ok = scores(0);
                } else if ((ok = put(i - 1))) {
                    tma_store_wait_read<0>();
                    mbar_arrive(&m.hfree);
                }
                if (!ok || !(ok = mbar_wait(&m.prep, i & 1, max_spin))) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k)                                                        // (2)
                    mma_bf16(tmem + kTmO2, kmajor_step(ak, k), step_desc(sr, k * 2048), id_o, k > 0);
                mma_commit(&m.o2_full);
                if (!(ok = mbar_wait(&m.pt, i & 1, max_spin))) break;
                tc_fence_after();
                const int s = i % L::kStages;
                issue_state<kTerms>(tmem + kTmSt, step_desc(br, s * kT * kTile), wr);                   // (4)
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)                                                       // (3)
                    mma_bf16_ts(tmem + kTmO1, tmem + kTmP + 8 * k, step_desc(cr, s * kTile + k * 2048), id_o, k > 0);
                mma_commit(&m.o_full);
                if (!(ok = mbar_wait(&m.o2_full, i & 1, max_spin))) break;
                if (i + 1 < pl.nc) load_a();
                if (!(ok = mbar_wait(&m.o_full, i & 1, max_spin))) break;
                if (i + L::kStages < pl.nc) load_bc();
                if (i + 1 < pl.nc) ok = mbar_wait(&m.sread, i & 1, max_spin) && scores(i + 1);
            }
            if (ok) ok = put(pl.nc - 1);
            tma_store_wait_all<0>();
            // Every load that was asked for lands, and every product completes, before the CTA exits.
            if (na > 0) mbar_wait(&m.a_full, (na - 1) & 1, kDefaultMaxSpin);
            for (int j = max(nbc - L::kStages, 0); j < nbc; ++j) {
                mbar_wait(&m.b_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
                mbar_wait(&m.c_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
            }
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else {
        const int q = warp & 3, g = warp >> 2, row = 32 * q + lane;
        const int qm = kRev ? 3 - q : q, im = kRev ? 127 - lane - 32 * q : row;   // in the order of summation
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        const bool has_state = q < 2 * kT;
        const int64_t state = (int64_t)a.Da * a.Dc, bh = (int64_t)pl.b * a.H + pl.h;
        auto piece = [&](int j) { return (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); };
        // State row `row`, columns col0 + 32 g ..
        float st[32];
        const int c0 = pl.col0 + 32 * g;
        const float* from = a.nseg > 1 ? a.seeds + (bh * a.nseg + pl.seg) * state : (a.S0 ? a.S0 + bh * state : nullptr);
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (has_state && from && row < a.Da && c0 + k < a.Dc) v = *reinterpret_cast<const float4*>(from + (int64_t)row * a.Dc + c0 + k);
            st[k] = v.x, st[k + 1] = v.y, st[k + 2] = v.z, st[k + 3] = v.w;
        }
        const float read = a.scale * pow2((im + 1) * l2);   // weight of the state in this row's output
        for (int i = 0; i < pl.nc; ++i) {
            const int t0 = pl.chunk<kRev>(i) * kC, mt = min(kC, pl.n - t0), s = i % L::kStages, ph = (i / L::kStages) & 1;
            uint8_t *ct = ctile(i), *w0 = base + L::kW;
            // ---------------------------------------------------- state to bf16, first term of w C
            if (has_state)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint4*>(base + L::kS + piece(4 * g + j)) =
                        make_uint4(pack_bf16(st[8 * j], st[8 * j + 1]), pack_bf16(st[8 * j + 2], st[8 * j + 3]),
                                   pack_bf16(st[8 * j + 4], st[8 * j + 5]), pack_bf16(st[8 * j + 6], st[8 * j + 7]));
            if (i > 0 && !(ok = warp_wait(&m.hfree, (i - 1) & 1, max_spin))) break;
            if (!(ok = warp_wait(&m.c_full[s], ph, max_spin))) break;
            // Rows at or past a sequence's end may hold anything: cleared in C, and in B for (4).
            // (Past N the loads filled zeros.)
            const bool ragged = mt < kC && pl.n < a.N;
            if (ragged) {
                if (!(ok = warp_wait(&m.b_full[s], ph, max_spin))) break;
                if (row >= mt)
                    for (int j = 4 * g; j < 4 * g + 4; ++j) {
                        *reinterpret_cast<uint4*>(ct + piece(j)) = make_uint4(0, 0, 0, 0);
                        for (int k = 0; k < kT; ++k)
                            *reinterpret_cast<uint4*>(btile(i) + k * kTile + piece(j)) = make_uint4(0, 0, 0, 0);
                    }
            }
            const float w = pow2((float)(kRev ? row : max(mt - 1 - row, 0)) * l2);
            const uint64_t w2 = pk2(w, w);
            uint64_t bad = 0;
#pragma unroll
            for (int j = 4 * g; j < 4 * g + 4; ++j) {
                const uint4 c = *reinterpret_cast<const uint4*>(ct + piece(j));
                uint32_t hi[4];
                uint64_t rest[4];
                weigh8(c, w2, hi, rest);
                *reinterpret_cast<uint4*>(w0 + piece(j)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                bad = fma2(bf2(c.x), 0, fma2(bf2(c.y), 0, fma2(bf2(c.z), 0, fma2(bf2(c.w), 0, bad))));
            }
            float b0, b1;
            unpk2(bad, &b0, &b1);
            if (!(b0 == 0.f && b1 == 0.f)) take_out(ct, row, g, i * kC + im, &m);
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.prep);
            // ---------------------------------------------------- scores to P
            if (!(ok = warp_wait(&m.p_full, i & 1, max_spin))) break;
            tc_fence_after();
            uint32_t p[2][16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int bm = g + 2 * k, blk = kRev ? 3 - bm : bm;
                if (bm > qm) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) p[k][e] = 0u;
                    continue;
                }
                const float r = pow2((float)(im - 32 * bm - 31) * l2);
                const uint64_t r2 = pk2(r, r);
#pragma unroll
                for (int half = 0; half < 32; half += 16) {
                    uint32_t v[16];
                    tmem_ld16(tmem + lanes + kTmP + 32 * blk + half, v);
                    tmem_ld_wait();
                    if (ragged && kRev && 32 * blk + 32 > mt)   // later tokens that the sequence does not have
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (32 * blk + half + e >= mt) v[e] = 0u;
                    if (bm < qm) {
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(m.tab + half + 2 * e);
                            p[k][half / 2 + e] = pack2(mul2(mul2(pair2(v + 2 * e), f.x), r2));
                            p[k][half / 2 + e + 1] = pack2(mul2(mul2(pair2(v + 2 * e + 2), f.y), r2));
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float x[2];
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int j = half + 2 * e + u, gap = kRev ? j - lane : lane - j;
                                x[u] = gap >= 0 ? __uint_as_float(v[2 * e + u]) * pow2((float)gap * l2) : 0.f;
                            }
                            p[k][half / 2 + e] = pack_bf16(x[0], x[1]);
                        }
                    }
                }
            }
            // Both warps of these rows have read their scores before either writes P over them.
            tc_fence_before();
            warp_arrive(&m.pair[q]);
            if (!(ok = warp_wait(&m.pair[q], i & 1, max_spin))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) tmem_st16(tmem + lanes + kTmP + 16 * (kRev ? 3 - g - 2 * k : g + 2 * k), p[k]);
            // ---------------------------------------------------- the other terms of w C
            if (!(ok = warp_wait(&m.o2_full, i & 1, max_spin))) break;
#pragma unroll
            for (int j = 4 * g; j < 4 * g + 4; ++j) {
                uint32_t t[4];
                uint64_t rest[4];
                weigh8(*reinterpret_cast<const uint4*>(ct + piece(j)), w2, t, rest);
#pragma unroll
                for (int k = 1; k < kTerms; ++k) {
                    next_term(rest, t);
                    *reinterpret_cast<uint4*>(w0 + k * kTile + piece(j)) = make_uint4(t[0], t[1], t[2], t[3]);
                }
            }
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.pt);
            // ---------------------------------------------------- state
            if (!(ok = warp_wait(&m.o_full, i & 1, max_spin))) break;
            tc_fence_after();
            if (has_state) {
                const Factor f = factor((float)(kRev ? kC : mt) * log_decay(l));
                uint32_t v[32];
                tmem_ld16(tmem + lanes + kTmSt + 32 * g, *reinterpret_cast<uint32_t(*)[16]>(v));
                tmem_ld16(tmem + lanes + kTmSt + 32 * g + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) st[k] = fmaf(f.hi, st[k], fmaf(f.lo, st[k], __uint_as_float(v[k])));
            }
            tc_fence_before();
            warp_arrive(&m.sread);
            // ---------------------------------------------------- output
            const bool spoiled = *const_cast<volatile int*>(&m.any) != kNone;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t u[16], v[16], o[8];
                tmem_ld16(tmem + lanes + kTmO1 + 32 * g + 16 * k, u);
                tmem_ld16(tmem + lanes + kTmO2 + 32 * g + 16 * k, v);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = pack2(fma2(pair2(u + 2 * e), pk2(a.scale, a.scale), mul2(pair2(v + 2 * e), pk2(read, read))));
                uint4 x = make_uint4(o[0], o[1], o[2], o[3]), y = make_uint4(o[4], o[5], o[6], o[7]);
                if (spoiled) {
                    x = put_nan(&m, 32 * g + 16 * k, i * kC + im, x);
                    y = put_nan(&m, 32 * g + 16 * k + 8, i * kC + im, y);
                }
                if (!ragged) {
                    *reinterpret_cast<uint4*>(w0 + piece(4 * g + 2 * k)) = x;
                    *reinterpret_cast<uint4*>(w0 + piece(4 * g + 2 * k + 1)) = y;
                } else if (row < mt) {
                    const int c = c0 + 16 * k;
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(const_cast<void*>(a.o.p)) + pl.b * a.o.bs + pl.h * a.o.hs +
                                        (int64_t)(t0 + row) * a.o.ts + c;
                    if (c < a.Dc) *reinterpret_cast<uint4*>(to) = x;
                    if (c + 8 < a.Dc) *reinterpret_cast<uint4*>(to + 8) = y;
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.staged);
        }
        if (ok && returns && has_state && row < a.Da)
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                if (c0 + k < a.Dc)
                    *reinterpret_cast<float4*>(a.S_out + bh * state + (int64_t)row * a.Dc + c0 + k) =
                        make_float4(st[k], st[k + 1], st[k + 2], st[k + 3]);
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWork) tmem_dealloc(tmem, 256);
}

// First pass: a segment's end state from zero (every segment but the last).
template <int kT, int kTerms, bool kRev>
__global__ void __launch_bounds__(kThreads, 2)
decay_sums_kernel(const __grid_constant__ CUtensorMap bmap, const __grid_constant__ CUtensorMap cmap,
                  const __grid_constant__ Args a, const __grid_constant__ Geo geo, WsHeader* hdr) {
    using L = SumSmem<kT, kTerms>;
    extern __shared__ __align__(1024) uint8_t base[];
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    auto btile = [&](int i) { return base + L::kB + (i % L::kStages) * kT * kTile; };
    auto ctile = [&](int i) { return base + L::kC0 + (i % L::kStages) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, geo);
    pdl_launch_dependents();
    if (pl.nc == 0) return;                    // the chaining leaves such segments out
    if ((smem_u32(base) & 1023) != 0) {
        if (tid == 0) set_status(hdr, LA_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.b_full[s], 1);
            mbar_init(&m.c_full[s], 1);
        }
        mbar_init(&m.prep, kWork);
        mbar_init(&m.o_full, 1);
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (warp == kWork) {
        tmem_alloc(&m.tmem_slot, 64);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;
    const float l = a.decay[pl.h], l2 = log2_decay(l);
    bool ok = true;
    if (warp == kWork) {
        if (lane == 0) {
            const uint64_t br = rows_desc(smem_u32(base) + L::kB), wr = rows_desc(smem_u32(base) + L::kW);
            int nbc = 0;
            auto load_bc = [&]() {
                if (hold) return;
                const int t = pl.chunk<kRev>(nbc) * kC, s = nbc % L::kStages;
                mbar_arrive_expect_tx(&m.c_full[s], kTile);
                tma_load_4d(ctile(nbc), &cmap, &m.c_full[s], pl.col0, geo.ch * pl.h, t, geo.cb * pl.b);
                mbar_arrive_expect_tx(&m.b_full[s], kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    tma_load_4d(btile(nbc) + k * kTile, &bmap, &m.b_full[s], 64 * k, geo.bh * pl.h, t, geo.bb * pl.b);
                ++nbc;
            };
            for (int s = 0; s < L::kStages && s < pl.nc; ++s) load_bc();
            for (int i = 0; i < pl.nc; ++i) {
                const int s = i % L::kStages;
                if (!(ok = mbar_wait(&m.b_full[s], (i / L::kStages) & 1, max_spin) && mbar_wait(&m.prep, i & 1, max_spin))) break;
                tc_fence_after();
                issue_state<kTerms>(tmem, step_desc(br, s * kT * kTile), wr);
                mma_commit(&m.o_full);
                if (!(ok = mbar_wait(&m.o_full, i & 1, max_spin))) break;
                if (i + L::kStages < pl.nc) load_bc();
            }
            for (int j = max(nbc - L::kStages, 0); j < nbc; ++j) {
                mbar_wait(&m.b_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
                mbar_wait(&m.c_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
            }
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else {
        const int q = warp & 3, g = warp >> 2, row = 32 * q + lane;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        const bool has_state = q < 2 * kT;
        auto piece = [&](int j) { return (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); };
        float st[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) st[k] = 0.f;
        for (int i = 0; i < pl.nc; ++i) {
            const int t0 = pl.chunk<kRev>(i) * kC, mt = min(kC, pl.n - t0), s = i % L::kStages, ph = (i / L::kStages) & 1;
            uint8_t *ct = ctile(i), *w0 = base + L::kW;
            if (!(ok = warp_wait(&m.c_full[s], ph, max_spin))) break;
            const bool ragged = mt < kC && pl.n < a.N;
            if (ragged && !(ok = warp_wait(&m.b_full[s], ph, max_spin))) break;
            const float w = pow2((float)(kRev ? row : max(mt - 1 - row, 0)) * l2);
            const uint64_t w2 = pk2(w, w);
#pragma unroll
            for (int j = 4 * g; j < 4 * g + 4; ++j) {
                uint4 c = *reinterpret_cast<const uint4*>(ct + piece(j));
                if (ragged && row >= mt) {
                    c = make_uint4(0, 0, 0, 0);
                    for (int k = 0; k < kT; ++k) *reinterpret_cast<uint4*>(btile(i) + k * kTile + piece(j)) = c;
                }
                uint32_t t[4];
                uint64_t rest[4];
                weigh8(c, w2, t, rest);
                *reinterpret_cast<uint4*>(w0 + piece(j)) = make_uint4(t[0], t[1], t[2], t[3]);
#pragma unroll
                for (int k = 1; k < kTerms; ++k) {
                    next_term(rest, t);
                    *reinterpret_cast<uint4*>(w0 + k * kTile + piece(j)) = make_uint4(t[0], t[1], t[2], t[3]);
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.prep);
            if (!(ok = warp_wait(&m.o_full, i & 1, max_spin))) break;
            tc_fence_after();
            if (has_state) {
                const Factor f = factor((float)(kRev ? kC : mt) * log_decay(l));
                uint32_t v[32];
                tmem_ld16(tmem + lanes + 32 * g, *reinterpret_cast<uint32_t(*)[16]>(v));
                tmem_ld16(tmem + lanes + 32 * g + 16, *reinterpret_cast<uint32_t(*)[16]>(v + 16));
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < 32; ++k) st[k] = fmaf(f.hi, st[k], fmaf(f.lo, st[k], __uint_as_float(v[k])));
            }
        }
        const int c0 = pl.col0 + 32 * g;
        float* to = a.seeds + (((int64_t)pl.b * a.H + pl.h) * a.nseg + pl.seg) * a.Da * a.Dc + (int64_t)row * a.Dc + c0;
        if (ok && has_state && row < a.Da)
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                if (c0 + k < a.Dc) *reinterpret_cast<float4*>(to + k) = make_float4(st[k], st[k + 1], st[k + 2], st[k + 3]);
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWork) tmem_dealloc(tmem, 64);
}

// Rows [B, H, N, D] of bf16 as a 4-D map (D, H, N, B) with boxes of 64 values x 128 tokens;
// values past D and tokens past N read as zero. An axis of stride 0 has one entry.
bool encode_rows(CUtensorMap* map, const Tensor& t, int D, int B, int H, int N, uint8_t* hm, uint8_t* bm) {
    EncodeTiled enc = get_encoder();
    if (!enc) return false;
    const bool h1 = H == 1 || t.hs == 0, b1 = B == 1 || t.bs == 0;
    if (hm) *hm = h1 ? 0 : 1;
    if (bm) *bm = b1 ? 0 : 1;
    const cuuint64_t any = 16;                         // a valid stride of an axis with one entry
    cuuint64_t dims[4] = {(cuuint64_t)D, h1 ? 1u : (cuuint64_t)H, (cuuint64_t)N, b1 ? 1u : (cuuint64_t)B};
    cuuint64_t strides[3] = {h1 ? any : (cuuint64_t)t.hs * 2, N == 1 ? any : (cuuint64_t)t.ts * 2,
                             b1 ? any : (cuuint64_t)t.bs * 2};
    cuuint32_t box[4] = {64, 1, (cuuint32_t)kC, 1}, es[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(t.p), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap a, b, c, o;
};

template <int kT, int kTerms, bool kRev>
cudaError_t launch(const Maps& maps, const Args& a, const Geo& geo, WsHeader* hdr, cudaStream_t st) {
    static std::atomic<int> optin[2][kMaxDevices];
    const unsigned units = (a.Dc + 63) / 64, BH = (unsigned)(a.B * a.H);
    cudaError_t e;
    if (a.nseg > 1) {
        constexpr int bytes = SumSmem<kT, kTerms>::kBytes;
        if ((e = ensure_smem_optin(decay_sums_kernel<kT, kTerms, kRev>, bytes, optin[0])) != cudaSuccess) return e;
        decay_sums_kernel<kT, kTerms, kRev><<<dim3(units, a.nseg - 1, BH), kThreads, bytes, st>>>(maps.b, maps.c, a, geo, hdr);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        if ((e = launch_chain(a, kC, st)) != cudaSuccess) return e;
    }
    constexpr int bytes = Smem<kT, kTerms>::kBytes;
    if ((e = ensure_smem_optin(decay_tc_kernel<kT, kTerms, kRev>, bytes, optin[1])) != cudaSuccess) return e;
    return scan::launch_after(decay_tc_kernel<kT, kTerms, kRev>, dim3(units, a.nseg, BH), kThreads, bytes, st, a.nseg > 1,
                              maps.a, maps.b, maps.c, maps.o, a, geo, hdr);
}

template <int kT>
cudaError_t launch_form(const Maps& maps, const Args& a, const Geo& geo, WsHeader* hdr, cudaStream_t st) {
    if (a.rev) return launch<kT, 2, true>(maps, a, geo, hdr, st);
    return a.S_out ? launch<kT, 3, false>(maps, a, geo, hdr, st) : launch<kT, 2, false>(maps, a, geo, hdr, st);
}

}  // namespace

namespace decay {

bool tc_supported(const Args& a, la_dtype dt) {
    if (dt != LA_BF16 || a.Da % 8 || a.Dc % 8) return false;
    if ((reinterpret_cast<uintptr_t>(a.S0) | reinterpret_cast<uintptr_t>(a.S_out)) & 15) return false;
    auto axis = [](int64_t size, int64_t stride, bool shared) {
        return size == 1 || (shared && stride == 0) || (stride > 0 && stride % 8 == 0 && stride < (int64_t)1 << 38);
    };
    auto rows = [&](const Tensor& t, bool in) {
        return (reinterpret_cast<uintptr_t>(t.p) & 15) == 0 && axis(a.B, t.bs, in) && axis(a.H, t.hs, in) &&
               axis(a.N, t.ts, false);
    };
    return rows(a.a, true) && rows(a.b, true) && rows(a.c, true) && rows(a.o, false);
}

int tc_segments(int64_t BH, int N, int Da, int Dc) {
    (void)Da;
    const int64_t ctas = BH * ((Dc + 63) / 64), slots = 2 * (int64_t)sm_count();
    const int64_t most = (N + kC - 1) / kC / 4;
    int64_t n = ctas > 0 ? slots / ctas : 1;
    n = n < most ? n : most;
    n = n < 64 ? n : 64;
    return n < 2 ? 1 : (int)n;
}

cudaError_t tc_run(Args a, void* ws_header, cudaStream_t st) {
    Geo geo = {};
    geo.cps = a.seg_len / kC;
    Maps maps;
    if (!encode_rows(&maps.a, a.a, a.Da, a.B, a.H, a.N, &geo.ah, &geo.ab) ||
        !encode_rows(&maps.b, a.b, a.Da, a.B, a.H, a.N, &geo.bh, &geo.bb) ||
        !encode_rows(&maps.c, a.c, a.Dc, a.B, a.H, a.N, &geo.ch, &geo.cb) ||
        !encode_rows(&maps.o, a.o, a.Dc, a.B, a.H, a.N, nullptr, nullptr))
        return cudaErrorInvalidValue;
    WsHeader* hdr = static_cast<WsHeader*>(ws_header);
    return a.Da <= 64 ? launch_form<1>(maps, a, geo, hdr, st) : launch_form<2>(maps, a, geo, hdr, st);
}

}  // namespace decay

}  // namespace la
