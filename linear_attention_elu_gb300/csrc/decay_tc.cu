// Decayed linear attention on the tensor cores (tcgen05): bf16, Da and Dc multiples of 8,
// 16-byte aligned rows. Definitions in csrc/decay.cuh and csrc/decay.cu.
//
// Method. For a chunk of 128 tokens of one head with the state S before it, i and j counted
// within the chunk in the order of summation (backwards where time is reversed), f = e^l:
//   o_i   = scale (f^(i+1) A_i^T S + sum_{j <= i} f^(i-j) (A_i . B_j) C_j)
//   S_new = f^m S + sum_j B_j (f^(m-1-j) C_j)^T          (m tokens in the chunk)
// as products of 128-row tiles:
//   (1) scores A B^T                      M = 128, N = 128, K = Da
//   (2) read of the state A S             M = 128, N = 64,  K = Da
//   (3) P C, P the weighted, masked scores (in TMEM)              K = 128
//   (4) B^T (w C), C weighted             M = Da,  N = 64,  K = 128
// A CTA walks the chunks of a segment of one head, for one or two "units" of 64 columns of
// C and of the state ((1) and P serve both).
//
// Roundings. A, B, C enter as they are. P and the state of (2) enter as two bf16 terms, the second
// the remainder of the first: 2^-16 of a value is left at most, so that what an output loses beside
// its own rounding depends neither on how many scores make it nor on the call's size. (One term of
// each: 2.3e-3 to 2.4e-3 off in all where the output's rounding is 1.7e-3. What the second terms
// cost, replayed from a graph: B=1 N=65536 H=16 D=64 154 us for 143, B=8 N=4096 H=8 D=64 backward
// 105 for 90.) Where both widths are above 64 the state has one term, see Smem. The state is held
// in fp32 in registers; (4) is summed per chunk from zero and added there, so that the tensor core's
// sums stay short. w C enters it as bf16 terms as well: two for a state that only o reads, three
// for one that the call returns.
// Weights below the diagonal 32 x 32 blocks are products of two factors <= 1, one of the
// row and one of the column; the diagonal blocks take a factor per score. Every
// factor's exponent is a count of tokens times l, so none is a difference of larger ones.
//
// Schedule. Eight working warps per unit, one that issues the products and one for loads and
// stores.
// A working warp owns 32 rows and half of a unit's columns. Within a chunk: (2) and (4) run under
// the step from scores to P; the sums of (4) join the state and (3) takes their TMEM columns; under
// (3) the next w C and the new state go to shared memory; the output is staged where C was. A, B and the
// next scores are on the way from the middle of the chunk on, C from the chunk before. With
// one unit and Da <= 64 two CTAs share an SM, each under the other's waits. Hand-offs are
// mbarriers; every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>
#include <stddef.h>

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
constexpr int kWork = 8;                       // working warps of a unit
constexpr int kNone = 0x7fffffff;

// TMEM columns: scores, P of each 16 of them over their first 8 and its second term over the
// others; per unit (64 columns on) the
// sums of (4), (3)'s part of the output and (2)'s part. With one unit, whose CTA leaves half of
// TMEM to another, (3) takes the columns of (4).
template <int kU> struct Tm {
    static constexpr uint32_t kP = 0, kSt = 128, kO1 = kU == 1 ? 128 : 256, kO2 = kU == 1 ? 192 : 384;
};

struct Misc {
    uint64_t a_full, b_full, c_full[2], p_full[2], s_full, o_full[2];
    uint64_t prep, pt[2], staged, o_free, drain;
    uint32_t tmem_slot;
    int any;                    // values of C that are not finite: the first token that has one,
    int first[128];             // and that of each column, counted over the segment
    alignas(16) float tab[32];  // f^(31 - j), by the column's place in its block; read 16 bytes at a time
    // decay_kv_kernel alone, of a diagonal block:
    alignas(16) float diag[1024];     // its factors, [column / 4][row][4]
    uint32_t mask[512];               // which scores take part, [pair of columns / 2][row][2]
};
constexpr uint32_t misc_bytes(bool table) { return table ? 7 * 1024 : 1024; }
static_assert(sizeof(Misc) <= misc_bytes(true) && offsetof(Misc, diag) <= misc_bytes(false), "barriers and tables");

// Shared memory from a 1024-byte boundary.
template <int kT, int kU, int kTerms> struct Smem {
    static constexpr int kStages = kTerms == 2 ? 2 : 1;               // of C
    static constexpr uint32_t kA = 0, kB = kT * kTile, kC0 = 2 * kT * kTile;
    static constexpr uint32_t kW = kC0 + kStages * kU * kTile;        // [unit][term]
    static constexpr uint32_t kS = kW + kU * kTerms * kTile;          // [unit], 64 kT rows
    // Terms of the state in (2). Where both widths are above 64 a second one would take the place
    // of C's second stage, or of a unit: B=4 N=2047 H=8 D=128 backward 79 us against 60, forward
    // with S_out B=4 N=4096 H=16 187 against 134.
    static constexpr int kReads = kT * kU < 4 ? 2 : 1;
    static constexpr uint32_t kMisc = kS + kReads * kU * kT * kTile / 2;
    static constexpr int kBytes = kMisc + misc_bytes(false);
    static constexpr int kPerSm = kBytes <= 113 * 1024 && kU == 1 ? 2 : 1;
};
static_assert(Smem<1, 1, 2>::kPerSm == 2 && Smem<1, 1, 3>::kPerSm == 2, "two CTAs per SM");
static_assert(Smem<2, 2, 2>::kBytes <= 227 * 1024 && Smem<2, 2, 3>::kBytes <= 227 * 1024, "shared memory");

// The first pass: B and C, the terms of w C.
template <int kT, int kU, int kTerms> struct SumSmem {
    static constexpr int kStages = kT + kU < 4 || kTerms == 2 ? 2 : 1;
    static constexpr uint32_t kB = 0, kC0 = kStages * kT * kTile, kW = kC0 + kStages * kU * kTile;
    static constexpr uint32_t kMisc = kW + kU * kTerms * kTile;
    static constexpr int kBytes = kMisc + misc_bytes(false);
    static constexpr int kPerSm = kBytes <= 113 * 1024 && kU == 1 ? 2 : 1;
};
static_assert(SumSmem<2, 2, 2>::kBytes <= 227 * 1024 && SumSmem<1, 2, 3>::kBytes <= 227 * 1024, "shared memory");

// Coordinate factors of the tensor maps: 0 for an axis of stride 0, whose map has one entry.
struct Geo {
    uint8_t ah, ab, bh, bb, ch, cb;
    uint8_t late;               // the launch before it is not waited for until this one's end: it
                                // started after that launch had seen the chained seeds
};

// What packing left of x, packed.
__device__ __forceinline__ uint32_t remainder2(uint64_t x, uint32_t hi) { return pack2(fma2(bf2(hi), pk2(-1.f, -1.f), x)); }
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

// (4), the smallest terms first, for kU units side by side (a unit's terms follow one another).
// The second 64-row atom of the A operand is the tile after B's (for kT = 1 whatever tile
// follows: those lanes are unused).
template <int kU, int kTerms>
__device__ __forceinline__ void issue_state(uint32_t dst, uint64_t bt, uint32_t w_tile) {
    constexpr uint32_t id = idesc_bf16_f32(128, 64 * kU, true, true);
    const uint64_t w = smem_desc(w_tile, kTerms * kTile, 1024, kSwizzle128B);
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
__device__ __forceinline__ Place place(const Args& a, int units, int bh) {
    Place p;
    p.b = bh / a.H;
    p.h = bh - p.b * a.H;
    p.col0 = 64 * units * blockIdx.x;
    p.seg = blockIdx.y;
    p.n = tokens_of(a, p.b);
    p.nch = (p.n + kC - 1) / kC;
    p.v0 = p.seg * (a.seg_len / kC);
    p.nc = min(max(p.nch - p.v0, 0), a.seg_len / kC);
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

// Columns c0 .. c1 of row `row` of a C tile: notes the values that are not finite, and clears
// them: (3) would add 0 times them to the tokens before them. (4) has them from the terms.
__device__ __noinline__ void take_out(uint8_t* tile, int row, int c0, int c1, int token, int* any, int* first) {
    for (int c = c0; c < c1; ++c) {
        unsigned short* v = reinterpret_cast<unsigned short*>(tile + row * 128 + (((c >> 3) ^ (row & 7)) << 4)) + (c & 7);
        if ((*v & 0x7F80u) != 0x7F80u) continue;
        *v = 0;
        atomicMin(first + c, token);
        atomicMin(any, token);
    }
}

// The outputs that such values reach, set to NaN: eight columns of a row.
__device__ __noinline__ uint4 put_nan(const int* firsts, int token, uint4 o) {
    auto one = [&](uint32_t w, int k) {
        const volatile int* first = firsts + k;
        if (first[0] <= token) w = (w & 0xFFFF0000u) | 0x7FFFu;
        if (first[1] <= token) w = (w & 0xFFFFu) | 0x7FFF0000u;
        return w;
    };
    return make_uint4(one(o.x, 0), one(o.y, 2), one(o.z, 4), one(o.w, 6));
}

// ------------------------------------------------------------ steps of a working warp
// Row `row` = 32 q + lane of the tiles, columns from the 16-byte piece j0 on.

// A state row (fp32 columns) to the bf16 tiles that (2) reads, its terms `term` bytes apart.
template <int kReads, int kCols>
__device__ __forceinline__ void write_state(uint8_t* tile, uint32_t term, const float (&st)[kCols], int row, int j0) {
#pragma unroll
    for (int j = 0; j < kCols / 8; ++j) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint64_t v = pk2(st[8 * j + 2 * k], st[8 * j + 2 * k + 1]);
            hi[k] = pack2(v);
            if (kReads > 1) lo[k] = remainder2(v, hi[k]);
        }
        uint8_t* to = tile + row * 128 + (((j0 + j) ^ (row & 7)) << 4);
        *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if (kReads > 1) *reinterpret_cast<uint4*>(to + term) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// w C of a row: its terms, kTile apart. Returns whether all values are finite.
template <int kTerms, int kPieces = 4>
__device__ __forceinline__ bool write_weighted(const uint8_t* c_tile, uint8_t* terms, float w, int row, int j0) {
    const uint64_t w2 = pk2(w, w);
    uint64_t bad = 0;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const uint32_t at = row * 128 + (((j0 + j) ^ (row & 7)) << 4);
        const uint4 c = *reinterpret_cast<const uint4*>(c_tile + at);
        uint32_t t[4];
        uint64_t rest[4];
        weigh8(c, w2, t, rest);
        *reinterpret_cast<uint4*>(terms + at) = make_uint4(t[0], t[1], t[2], t[3]);
        // The remainder of a value that is not finite is NaN.
        bad = fma2(rest[0], 0, fma2(rest[1], 0, fma2(rest[2], 0, fma2(rest[3], 0, bad))));
#pragma unroll
        for (int k = 1; k < kTerms; ++k) {
            next_term(rest, t);
            *reinterpret_cast<uint4*>(terms + k * kTile + at) = make_uint4(t[0], t[1], t[2], t[3]);
        }
    }
    float b0, b1;
    unpk2(bad, &b0, &b1);
    return b0 == 0.f && b1 == 0.f;
}

// Rows past a sequence's end may hold anything: pieces of one row set to 0.
template <int kPieces = 4> __device__ __forceinline__ void clear_pieces(uint8_t* tile, int row, int j0) {
#pragma unroll
    for (int j = j0; j < j0 + kPieces; ++j)
        *reinterpret_cast<uint4*>(tile + row * 128 + ((j ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
}

// Whether the values of four 16-byte pieces of a row are finite, for the warp as a whole.
__device__ __forceinline__ bool finite_pieces(const uint8_t* tile, int row, int j0) {
    uint32_t bad = 0;
#pragma unroll
    for (int j = j0; j < j0 + 4; ++j) {
        const uint4 x = *reinterpret_cast<const uint4*>(tile + row * 128 + ((j ^ (row & 7)) << 4));
        for (uint32_t v : {x.x, x.y, x.z, x.w}) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(bad) : "r"(v), "r"(0u));
    }
    return __all_sync(0xffffffffu, (bad & 0x7FFF7FFFu) == 0);
}

// kCols columns from c0 of row `row` of a matrix of states [Da, Dc] (transposed: of its transpose).
template <int kCols>
__device__ __forceinline__ void load_state(const Args& a, const float* from, int row, int c0, float (&v)[kCols]) {
#pragma unroll
    for (int k = 0; k < kCols; k += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < a.Da && c0 + k < a.Dc) {
            if (a.seeds_t) {
                const float* t = from + (int64_t)(c0 + k) * a.Da + row;
                x = make_float4(t[0], t[a.Da], t[2 * a.Da], t[3 * a.Da]);
            } else {
                x = *reinterpret_cast<const float4*>(from + (int64_t)row * a.Dc + c0 + k);
            }
        }
        v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
    }
}

// The state before a segment: S0, or what the chaining left, or the ends of the segments before it joined here.
template <int kCols>
__device__ __forceinline__ void start_state(const Args& a, const Place& pl, float l, int row, int c0, float (&st)[kCols]) {
    const int64_t bh = (int64_t)pl.b * a.H + pl.h, state = (int64_t)a.Da * a.Dc;
#pragma unroll
    for (int k = 0; k < kCols; ++k) st[k] = 0.f;
    const bool chained = a.nseg > 1 && !a.fold;
    const float* from = chained ? a.seeds + (bh * a.nseg + pl.seg) * state : (a.S0 ? a.S0 + bh * state : nullptr);
    if (from) load_state(a, from, row, c0, st);
    if (!a.fold) return;
    const int n = a.rev ? pl.nch * kC : pl.n;
#pragma unroll 1
    for (int i = 0; i < pl.seg; ++i) {
        const int m = seg_tokens(a, n, i);
        if (m == 0) break;
        float v[kCols];
        load_state(a, a.seeds + (bh * a.nseg + i) * state, row, c0, v);
        const Factor f = factor((float)m * log_decay(l));
#pragma unroll
        for (int k = 0; k < kCols; ++k) st[k] = fmaf(f.hi, st[k], fmaf(f.lo, st[k], v[k]));
    }
}

// Decay factors of a warp's rows, for every chunk.
struct RowFactors {
    float l2;           // log2 f
    int im;             // the row in the order of summation
};

// 32 lanes x 32 bits, 8 consecutive columns: thread t of the warp writes lane (base + t).
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Four scores of a diagonal block, columns j .. j + 3, to packed P. Scores that take no part are
// cleared as bits: their products may be anything. kTable: factors from the table (one CTA
// per SM; with two the table's reads from shared memory cost more than the exponentials: with P in
// one term, B=1 N=65536 H=16 D=64 forward 151 us against 148, the backward of B=8 N=4096 H=8 D=64
// with one 91 against 92.5).
template <bool kRev, bool kTable>
__device__ __forceinline__ void diagonal4(const uint32_t* v, int j, const RowFactors& rf, float gap, uint32_t keep,
                                          const Misc& m, uint32_t* p, uint32_t* rest) {
    uint64_t f0, f1;
    uint32_t k0, k1;
    if constexpr (kTable) {
        const int lane = threadIdx.x & 31;
        const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(m.diag + 32 * j + 4 * lane);
        const uint2 k = *reinterpret_cast<const uint2*>(m.mask + 16 * j + 2 * lane);
        f0 = f.x, f1 = f.y, k0 = k.x, k1 = k.y;
    } else {
        float x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = pow2((kRev ? gap + (float)u : gap - (float)u) * rf.l2);
        f0 = pk2(x[0], x[1]), f1 = pk2(x[2], x[3]);
        // Bits k and k + 1 of keep to the halves of a word.
        auto halves = [=](int k) { return ((((keep >> k) & 3u) * 0x8001u) & 0x10001u) * 0xFFFFu; };
        k0 = halves(0), k1 = halves(2);
    }
    const uint64_t x0 = mul2(pair2(v), f0), x1 = mul2(pair2(v + 2), f1);
    p[0] = pack2(x0);
    p[1] = pack2(x1);
    rest[0] = remainder2(x0, p[0]) & k0;
    rest[1] = remainder2(x1, p[1]) & k1;
    p[0] &= k0;
    p[1] &= k1;
}

// Scores of block column `blk` (bm in the order of summation) to packed P: 16 of them over the
// first 8 of their columns, what the packing leaves over the other 8. No other warp reads or
// writes those. Loops are kept rolled: what the compiler keeps of unrolled ones from chunk to chunk
// is spilled, and does not fit the little L1 that two CTAs leave (backwards in time the call took
// 1.8 times as long).
template <bool kRev, bool kTable>
__device__ __forceinline__ void scores_to_p(uint32_t tm_p, int blk, int bm, int qm, const RowFactors& rf, const Misc& m, int cut) {
    const int lane = threadIdx.x & 31;
    const float r = pow2((float)(rf.im - 32 * bm - 31) * rf.l2);
    const uint64_t r2 = pk2(r, r);
    const uint32_t at = tm_p + 32 * blk, keep = kRev ? 0xFFFFFFFFu << lane : 0xFFFFFFFFu >> (31 - lane);
#pragma unroll 1
    for (int half = 0; half < 32; half += 16) {
        uint32_t v[16], p[8], rest[8];
        if (bm > qm) {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = rest[e] = 0u;
        } else {
            tmem_ld16(at + half, v);
            tmem_ld_wait();
            if (kRev && 32 * blk + half + 16 > cut)        // later tokens that the sequence does not have
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (32 * blk + half + e >= cut) v[e] = 0u;
            if (bm < qm) {
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(m.tab + half + e);
                    const uint64_t x0 = mul2(mul2(pair2(v + e), f.x), r2), x1 = mul2(mul2(pair2(v + e + 2), f.y), r2);
                    p[e / 2] = pack2(x0);
                    p[e / 2 + 1] = pack2(x1);
                    rest[e / 2] = remainder2(x0, p[e / 2]);
                    rest[e / 2 + 1] = remainder2(x1, p[e / 2 + 1]);
                }
            } else {
                const float gap = (float)(kRev ? half - lane : lane - half);   // a count: times l2 it is rounded once
                const uint32_t bits = keep >> half;
#pragma unroll
                for (int e = 0; e < 16; e += 4)
                    diagonal4<kRev, kTable>(v + e, half + e, rf, kRev ? gap + (float)e : gap - (float)e, bits >> e, m,
                                            p + e / 2, rest + e / 2);
            }
        }
        tmem_st8(at + half, p);
        tmem_st8(at + half + 8, rest);
    }
}

// The chunk's sums join the state: st = f st + sums.
template <int kCols> __device__ __forceinline__ void join_state(uint32_t tm, const Factor& f, float (&st)[kCols]) {
    const uint64_t hi = pk2(f.hi, f.hi), lo = pk2(f.lo, f.lo);
#pragma unroll
    for (int half = 0; half < kCols; half += 16) {
        uint32_t v[16];
        tmem_ld16(tm + half, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            const uint64_t s = pk2(st[half + k], st[half + k + 1]);
            unpk2(fma2(hi, s, fma2(lo, s, pair2(v + k))), &st[half + k], &st[half + k + 1]);
        }
    }
}

// 16 output columns of a row from the two parts.
__device__ __forceinline__ void join_output(uint32_t tm1, uint32_t tm2, float scale, float read, uint4* x, uint4* y) {
    uint32_t u[16], v[16], o[8];
    tmem_ld16(tm1, u);
    tmem_ld16(tm2, v);
    tmem_ld_wait();
    const uint64_t s2 = pk2(scale, scale), r2 = pk2(read, read);
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = pack2(fma2(pair2(u + 2 * e), s2, mul2(pair2(v + 2 * e), r2)));
    *x = make_uint4(o[0], o[1], o[2], o[3]);
    *y = make_uint4(o[4], o[5], o[6], o[7]);
}

// Tables of a head: the columns' factors, and which scores of a diagonal block take part.
template <bool kRev, bool kTable> __device__ __forceinline__ void init_tables(Misc& m, float l2) {
    const int tid = threadIdx.x, lane = tid & 31;
    if (kTable && tid < 256)
        for (int j = 4 * (tid >> 5); j < 4 * (tid >> 5) + 4; ++j) {
            const int gap = kRev ? j - lane : lane - j;
            m.diag[32 * (j & ~3) + 4 * lane + (j & 3)] = gap >= 0 ? pow2((float)gap * l2) : 0.f;
        }
    if (tid < 32) m.tab[tid] = pow2((float)(kRev ? tid : 31 - tid) * l2);
    if (kTable && tid < 256)
        for (int e = 2 * (tid >> 5); e < 2 * (tid >> 5) + 2; ++e) {
            const bool a = kRev ? 2 * e >= lane : 2 * e <= lane, b = kRev ? 2 * e + 1 >= lane : 2 * e + 1 <= lane;
            m.mask[32 * (e & ~1) + 2 * lane + (e & 1)] = (a ? 0xFFFFu : 0u) | (b ? 0xFFFF0000u : 0u);
        }
}

__device__ __forceinline__ RowFactors row_factors(float l2, int im) {
    return {l2, im};
}

template <int kT, int kU, int kTerms, bool kRev>
__global__ void __launch_bounds__(32 * (kU * kWork + 2), Smem<kT, kU, kTerms>::kPerSm)
decay_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
                const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap omap,
                const __grid_constant__ Args a, const __grid_constant__ Geo geo, WsHeader* hdr) {
    using L = Smem<kT, kU, kTerms>;
    using M = Tm<kU>;
    constexpr int kWarps = kU * kWork;
    constexpr uint32_t kCols = kU == 1 ? 256 : 512;
    constexpr int kLow = kRev && kT == 1 ? 64 : 0;     // the state's first lane: where the warps have few scores to convert
    extern __shared__ __align__(1024) uint8_t base[];
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    auto ctile = [&](int i, int u) { return base + L::kC0 + ((i % L::kStages) * kU + u) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, kU, blockIdx.z);
    const bool returns = a.S_out && pl.seg == a.nseg - 1;
    // The seeds, where there are segments. A dependent launch never ends before what it follows.
    if (!geo.late || (pl.nc == 0 && !returns)) pdl_wait();
    pdl_launch_dependents();
    if (pl.nc == 0 && !returns) return;
    if ((smem_u32(base) & 1023) != 0) {        // the tiles' swizzle needs it; no static shared memory, so it holds
        if (tid == 0) set_status(hdr, LA_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        for (uint64_t* bar : {&m.a_full, &m.b_full, &m.c_full[0], &m.c_full[1], &m.p_full[0], &m.s_full, &m.o_full[0], &m.drain})
            mbar_init(bar, 1);
        for (uint64_t* bar : {&m.prep, &m.pt[0], &m.staged}) mbar_init(bar, kWarps);
        fence_mbar_init();
        m.any = kNone;
    }
    if (tid < 128) m.first[tid] = kNone;
    const float l = a.decay[pl.h], l2 = log2_decay(l);
    init_tables<kRev, false>(m, l2);
    if (warp == kWarps) {
        tmem_alloc(&m.tmem_slot, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;     // test hook: loads never issued
    bool ok = true;

    if (warp == kWarps) {
        // ------------------------------------------------------------ products
        if (lane == 0 && pl.nc > 0) {
            const uint32_t base_a = smem_u32(base);
            const uint64_t ak = kmajor_desc(base_a + L::kA), bk = kmajor_desc(base_a + L::kB);
            const uint64_t br = rows_desc(base_a + L::kB), cr = rows_desc(base_a + L::kC0);
            const uint64_t sr = smem_desc(base_a + L::kS, kT * kTile / 2, 1024, kSwizzle128B);   // units side by side
            constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_o = idesc_bf16_f32(128, 64 * kU, false, true);
            auto scores = [&](int i) -> bool {                                                          // (1)
                if (!mbar_wait(&m.a_full, i & 1, max_spin) || !mbar_wait(&m.b_full, i & 1, max_spin)) return false;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k) mma_bf16(tmem + M::kP, kmajor_step(ak, k), kmajor_step(bk, k), id_sc, k > 0);
                mma_commit(&m.p_full[0]);
                return true;
            };
            ok = scores(0);
            for (int i = 0; i < pl.nc && ok; ++i) {
                if (!(ok = mbar_wait(&m.prep, i & 1, max_spin))) break;
                tc_fence_after();
#pragma unroll
                for (int part = L::kReads - 1; part >= 0; --part)                                       // (2)
#pragma unroll
                    for (int k = 0; k < 4 * kT; ++k)
                        mma_bf16(tmem + M::kO2, kmajor_step(ak, k), step_desc(sr, part * kU * kT * kTile / 2 + k * 2048), id_o,
                                 part < L::kReads - 1 || k > 0);
                issue_state<kU, kTerms>(tmem + M::kSt, kLow ? br - (kTile >> 4) : br, base_a + L::kW);  // (4)
                mma_commit(&m.s_full);
                if (!(ok = mbar_wait(&m.pt[0], i & 1, max_spin))) break;
                tc_fence_after();
#pragma unroll
                for (int part = 1; part >= 0; --part)                                                   // (3)
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_bf16_ts(tmem + M::kO1, tmem + M::kP + 16 * k + 8 * part,
                                    step_desc(cr, (i % L::kStages) * kU * kTile + k * 2048), id_o, part < 1 || k > 0);
                mma_commit(&m.o_full[0]);
                if (!(ok = mbar_wait(&m.o_full[0], i & 1, max_spin))) break;
                if (i + 1 < pl.nc) ok = scores(i + 1);
            }
            mma_commit(&m.drain);              // every product completes before the CTA exits
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else if (warp == kWarps + 1) {
        // ------------------------------------------------------------ loads and stores
        if (lane == 0 && pl.nc > 0) {
            int nab = 0, nc = 0;               // chunks of A and B, of C asked for
            auto load_ab = [&]() {
                if (hold) return;
                const int t = pl.chunk<kRev>(nab) * kC;
                mbar_arrive_expect_tx(&m.a_full, kT * kTile);
                mbar_arrive_expect_tx(&m.b_full, kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k) {
                    tma_load_4d(base + L::kA + k * kTile, &amap, &m.a_full, 64 * k, geo.ah * pl.h, t, geo.ab * pl.b);
                    tma_load_4d(base + L::kB + k * kTile, &bmap, &m.b_full, 64 * k, geo.bh * pl.h, t, geo.bb * pl.b);
                }
                if (++nab < pl.nc) {               // the chunk after it comes to L2 ahead of its load
                    const int next = pl.chunk<kRev>(nab) * kC;
#pragma unroll
                    for (int k = 0; k < kT; ++k) {
                        tma_prefetch_4d(&amap, 64 * k, geo.ah * pl.h, next, geo.ab * pl.b);
                        tma_prefetch_4d(&bmap, 64 * k, geo.bh * pl.h, next, geo.bb * pl.b);
                    }
                }
            };
            auto load_c = [&]() {
                if (hold) return;
                const int t = pl.chunk<kRev>(nc) * kC;
                uint64_t* bar = &m.c_full[nc % L::kStages];
                mbar_arrive_expect_tx(bar, kU * kTile);
#pragma unroll
                for (int u = 0; u < kU; ++u) tma_load_4d(ctile(nc, u), &cmap, bar, pl.col0 + 64 * u, geo.ch * pl.h, t, geo.cb * pl.b);
                if (++nc < pl.nc)
#pragma unroll
                    for (int u = 0; u < kU; ++u)
                        tma_prefetch_4d(&cmap, pl.col0 + 64 * u, geo.ch * pl.h, pl.chunk<kRev>(nc) * kC, geo.cb * pl.b);
            };
            load_ab();
            for (int s = 0; s < L::kStages && s < pl.nc; ++s) load_c();
            for (int i = 0; i < pl.nc; ++i) {
                if (!(ok = mbar_wait(&m.s_full, i & 1, max_spin))) break;     // (1), (2) and (4) have read A and B
                if (i + 1 < pl.nc) load_ab();
                // The output, staged by the working warps where C was; the last, ragged one of a
                // sequence shorter than N was written row by row.
                if (!(ok = mbar_wait(&m.staged, i & 1, max_spin))) break;
                const int t = pl.chunk<kRev>(i) * kC;
                if (t + kC <= pl.n || pl.n == a.N) {
#pragma unroll
                    for (int u = 0; u < kU; ++u) tma_store_4d(&omap, ctile(i, u), pl.col0 + 64 * u, pl.h, t, pl.b);
                    tma_store_commit();
                }
                if (i + L::kStages < pl.nc) {      // its place takes C of another chunk
                    tma_store_wait_read<0>();
                    load_c();
                }
            }
            tma_store_wait_all<0>();
            // Every load that was asked for lands before the CTA exits.
            if (nab > 0) {
                mbar_wait(&m.a_full, (nab - 1) & 1, kDefaultMaxSpin);
                mbar_wait(&m.b_full, (nab - 1) & 1, kDefaultMaxSpin);
            }
            for (int j = max(nc - L::kStages, 0); j < nc; ++j)
                mbar_wait(&m.c_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, g4 = warp >> 2, u = g4 >> 1, g = g4 & 1, row = 32 * q + lane;
        const int qm = kRev ? 3 - q : q, im = kRev ? 127 - row : row;
        const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16), tmu = tm + 64 * u + 32 * g;
        const bool has_state = row >= kLow && row < kLow + 64 * kT;
        const int srow = row - kLow;
        const int64_t state = (int64_t)a.Da * a.Dc, bh = (int64_t)pl.b * a.H + pl.h;
        const RowFactors rf = row_factors(l2, im);
        uint8_t *terms = base + L::kW + u * kTerms * kTile, *s_tile = base + L::kS + u * kT * kTile / 2;
        // State row `srow`, columns col0 + 64 u + 32 g ..
        float st[32];
        const int c0 = pl.col0 + 64 * u + 32 * g;
        if (has_state) start_state(a, pl, l, srow, c0, st);
        const float read = a.scale * pow2((float)(im + 1) * l2);   // weight of the state in this row's output
        const Factor whole = factor(kC * log_decay(l));
        // w C of a chunk, once C is there. Rows past the sequence's end are cleared in C, and in B
        // for (4). (Past N the loads filled zeros.) (1) may read such rows of B, whose scores take
        // no part.
        auto weigh = [&](int i) -> bool {
            const int mt = min(kC, pl.n - pl.chunk<kRev>(i) * kC);
            uint8_t* ct = ctile(i, u);
            if (!warp_wait(&m.c_full[i % L::kStages], (i / L::kStages) & 1, max_spin)) return false;
            if (mt < kC && pl.n < a.N) {
                if (!warp_wait(&m.b_full, i & 1, max_spin)) return false;
                if (row >= mt) {
                    clear_pieces(ct, row, 4 * g);
                    for (int k = 0; k < kT; ++k) clear_pieces(base + L::kB + k * kTile, row, 4 * g);
                }
            }
            const float w = pow2((float)(kRev ? row : max(mt - 1 - row, 0)) * l2);
            if (!write_weighted<kTerms>(ct, terms, w, row, 4 * g)) take_out(ct, row, 32 * g, 32 * g + 32, i * kC + im, &m.any, m.first + 64 * u);
            return true;
        };
        auto put_state = [&]() {
            if (has_state) write_state<L::kReads>(s_tile, kU * kT * kTile / 2, st, srow, 4 * g);
        };
        if (pl.nc > 0) ok = weigh(0);              // S0 on its way meanwhile
        put_state();
        for (int i = 0; i < pl.nc && ok; ++i) {
            const int t0 = pl.chunk<kRev>(i) * kC, mt = min(kC, pl.n - t0);
            const bool ragged = mt < kC && pl.n < a.N;
            uint8_t* ct = ctile(i, u);
            // ---------------------------------------------------- the operands of (2) and (4) are there
            if (L::kStages == 1 && i > 0 && !(ok = weigh(i))) break;
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.prep);
            // ---------------------------------------------------- scores to P
            if (!(ok = warp_wait(&m.p_full[0], i & 1, max_spin))) break;
            tc_fence_after();
#pragma unroll 1
            for (int bm = g4; bm < 4; bm += 2 * kU)
                scores_to_p<kRev, false>(tm + M::kP, kRev ? 3 - bm : bm, bm, qm, rf, m, ragged ? mt : kC);
            // ---------------------------------------------------- state
            auto hand_over = [&]() {
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(&m.pt[0]);
            };
            if (kU > 1) hand_over();
            if (!(ok = warp_wait(&m.s_full, i & 1, max_spin))) break;
            tc_fence_after();
            if (has_state) join_state(tmu + M::kSt, kRev || mt == kC ? whole : factor((float)mt * log_decay(l)), st);
            if (kU == 1) hand_over();              // (3) takes the columns of (4)
            // ---------------------------------------------------- the next w C and state, under (3)
            if (L::kStages == 2 && i + 1 < pl.nc && !(ok = weigh(i + 1))) break;
            put_state();
            // ---------------------------------------------------- output
            if (!(ok = warp_wait(&m.o_full[0], i & 1, max_spin))) break;
            tc_fence_after();
            const bool spoiled = *const_cast<volatile int*>(&m.any) != kNone;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint4 x, y;
                join_output(tmu + M::kO1 + 16 * k, tmu + M::kO2 + 16 * k, a.scale, read, &x, &y);
                if (spoiled) {
                    const int* first = m.first + 64 * u + 32 * g + 16 * k;
                    x = put_nan(first, i * kC + im, x);
                    y = put_nan(first + 8, i * kC + im, y);
                }
                if (!ragged) {
                    *reinterpret_cast<uint4*>(ct + row * 128 + (((4 * g + 2 * k) ^ (row & 7)) << 4)) = x;
                    *reinterpret_cast<uint4*>(ct + row * 128 + (((4 * g + 2 * k + 1) ^ (row & 7)) << 4)) = y;
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
        if (ok && returns && has_state && srow < a.Da)
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                if (c0 + k < a.Dc)
                    *reinterpret_cast<float4*>(a.S_out + bh * state + (int64_t)srow * a.Dc + c0 + k) =
                        make_float4(st[k], st[k + 1], st[k + 2], st[k + 3]);
    }
    if (!ok) report_timeout(hdr);
    if (geo.late) pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarps) tmem_dealloc(tmem, kCols);
}

// First pass, of one sum or two: the end state from zero of each segment but the last. Shared
// memory bounds it, the operand reads of (4) before all; so a narrow head's state is summed
// transposed, the first two terms of w C stacked as the 128 rows of one product (8 products of
// 6 KB of operands a chunk for 16), and the terms' sums joined at the end. The third term takes
// columns of its own, with the second in the rows that nobody reads.
template <int kT, int kU, int kTerms>
__global__ void __launch_bounds__(32 * (kU * kWork + 1), SumSmem<kT, kU, kTerms>::kPerSm)
decay_sums_kernel(const __grid_constant__ CUtensorMap bmap0, const __grid_constant__ CUtensorMap cmap0,
                  const __grid_constant__ CUtensorMap bmap1, const __grid_constant__ CUtensorMap cmap1,
                  const __grid_constant__ Args a0, const __grid_constant__ Geo geo0, const __grid_constant__ Args a1,
                  const __grid_constant__ Geo geo1, WsHeader* hdr) {
    const bool second = (int)blockIdx.z >= a0.B * a0.H;
    const Args& a = second ? a1 : a0;
    const Geo& geo = second ? geo1 : geo0;
    const CUtensorMap &bmap = second ? bmap1 : bmap0, &cmap = second ? cmap1 : cmap0;
    using L = SumSmem<kT, kU, kTerms>;
    constexpr int kWarps = kU * kWork;
    constexpr bool kStacked = kT == 1 && kU == 1;
    constexpr uint32_t kCols = kStacked && kTerms == 2 ? 64 : 128;
    extern __shared__ __align__(1024) uint8_t base[];
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    auto btile = [&](int i) { return base + L::kB + (i % L::kStages) * kT * kTile; };
    auto ctile = [&](int i, int u) { return base + L::kC0 + ((i % L::kStages) * kU + u) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, kU, blockIdx.z - (second ? a0.B * a0.H : 0));
    const bool rev = a.rev != 0;
    auto chunk = [&](int i) { return rev ? pl.chunk<true>(i) : pl.chunk<false>(i); };
    pdl_launch_dependents();
    if (pl.nc == 0 || pl.seg >= a.nseg - 1) return;    // segments without tokens are not read
    if ((smem_u32(base) & 1023) != 0) {
        if (tid == 0) set_status(hdr, LA_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        mbar_init(&m.c_full[0], 1);
        mbar_init(&m.c_full[1], 1);
        mbar_init(&m.prep, kWarps);
        mbar_init(&m.s_full, 1);
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (warp == kWarps) {
        tmem_alloc(&m.tmem_slot, kCols);
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
    if (warp == kWarps) {
        if (lane == 0) {
            const uint64_t br = rows_desc(smem_u32(base) + L::kB);
            int n = 0;
            auto load = [&]() {
                if (hold) return;
                const int t = chunk(n) * kC;
                uint64_t* bar = &m.c_full[n % L::kStages];
                mbar_arrive_expect_tx(bar, (kT + kU) * kTile);
#pragma unroll
                for (int u = 0; u < kU; ++u) tma_load_4d(ctile(n, u), &cmap, bar, pl.col0 + 64 * u, geo.ch * pl.h, t, geo.cb * pl.b);
#pragma unroll
                for (int k = 0; k < kT; ++k) tma_load_4d(btile(n) + k * kTile, &bmap, bar, 64 * k, geo.bh * pl.h, t, geo.bb * pl.b);
                if (++n + 1 < pl.nc) {             // the chunk after the next comes to L2 ahead of its load
                    const int later = chunk(n + 1) * kC;
#pragma unroll
                    for (int u = 0; u < kU; ++u) tma_prefetch_4d(&cmap, pl.col0 + 64 * u, geo.ch * pl.h, later, geo.cb * pl.b);
#pragma unroll
                    for (int k = 0; k < kT; ++k) tma_prefetch_4d(&bmap, 64 * k, geo.bh * pl.h, later, geo.bb * pl.b);
                }
            };
            for (int s = 0; s < L::kStages && s < pl.nc; ++s) load();
            for (int i = 0; i < pl.nc; ++i) {
                if (!(ok = mbar_wait(&m.prep, i & 1, max_spin))) break;
                tc_fence_after();
                const uint64_t bt = step_desc(br, (i % L::kStages) * kT * kTile);
                if constexpr (kStacked) {
                    constexpr uint32_t id = idesc_bf16_f32(128, 64, true, true);
                    const uint64_t w = rows_desc(smem_u32(base) + L::kW);
#pragma unroll
                    for (int part = 0; part < kTerms - 1; ++part)
#pragma unroll
                        for (int k = 0; k < kC / 16; ++k)
                            mma_bf16(tmem + 64 * part, step_desc(w, part * kTile + k * 2048), step_desc(bt, k * 2048), id, k > 0);
                } else {
                    issue_state<kU, kTerms>(tmem, bt, smem_u32(base) + L::kW);
                }
                mma_commit(&m.s_full);
                if (!(ok = mbar_wait(&m.s_full, i & 1, max_spin))) break;
                if (i + L::kStages < pl.nc) load();
            }
            for (int j = max(n - L::kStages, 0); j < n; ++j)
                mbar_wait(&m.c_full[j % L::kStages], (j / L::kStages) & 1, kDefaultMaxSpin);
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else {
        const int q = warp & 3, u = warp >> 3, g = (warp >> 2) & 1, row = 32 * q + lane;
        const bool has_state = kStacked || q < 2 * kT;
        const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16) + 64 * u + 32 * g;
        uint8_t* terms = base + L::kW + u * kTerms * kTile;
        const Factor whole = factor(kC * log_decay(l));
        float st[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) st[k] = 0.f;
        for (int i = 0; i < pl.nc; ++i) {
            const int mt = min(kC, pl.n - chunk(i) * kC);
            if (!(ok = warp_wait(&m.c_full[i % L::kStages], (i / L::kStages) & 1, max_spin))) break;
            if (mt < kC && pl.n < a.N && row >= mt) {
                clear_pieces(ctile(i, u), row, 4 * g);
                for (int k = 0; k < kT; ++k) clear_pieces(btile(i) + k * kTile, row, 4 * g);
            }
            write_weighted<kTerms>(ctile(i, u), terms, pow2((float)(rev ? row : max(mt - 1 - row, 0)) * l2), row, 4 * g);
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.prep);
            if (!(ok = warp_wait(&m.s_full, i & 1, max_spin))) break;
            tc_fence_after();
            if (has_state) join_state(tm, rev || mt == kC ? whole : factor((float)mt * log_decay(l)), st);
            if (kStacked && kTerms == 3 && q >= 2) join_state(tm + 64, {1.f, 0.f}, st);
        }
        const int c0 = pl.col0 + 64 * u + 32 * g;
        float* to = a.seeds + (((int64_t)pl.b * a.H + pl.h) * a.nseg + pl.seg) * a.Da * a.Dc;
        if constexpr (kStacked) {
            // Rows 64 .. (terms after the first) to those of the first, column 32 g + k of row `row`.
            float* other = reinterpret_cast<float*>(base + L::kW) + 32 * g * 64 + (row & 63);
            if (q >= 2)
#pragma unroll
                for (int k = 0; k < 32; ++k) other[64 * k] = st[k];
            named_bar(1, 32 * kWarps);             // every working warp comes here, whatever its waits said
            if (ok && q < 2 && row < a.Dc)
#pragma unroll
                for (int k = 0; k < 32; ++k)
                    if (32 * g + k < a.Da) to[(int64_t)(32 * g + k) * a.Dc + row] = st[k] + other[64 * k];
        } else if (ok && has_state && row < a.Da) {
            to += (int64_t)row * a.Dc + c0;
#pragma unroll
            for (int k = 0; k < 32; k += 4)
                if (c0 + k < a.Dc) *reinterpret_cast<float4*>(to + k) = make_float4(st[k], st[k + 1], st[k + 2], st[k + 3]);
        }
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarps) tmem_dealloc(tmem, kCols);
}

// dk and dv of one head in one pass backwards in time (Dk, Dv <= 64). The two sums take the
// same four tiles and the same state R_t = q_t dout_t^T + f R_{t+1}:
//   unit 0, dv: A = K, B = Q, C = dout, state R;   unit 1, dk: A = V, B = dout, C = Q, state R^T
// so (4) and the state are unit 0's alone, and unit 1 reads the same bf16 tile transposed.
// Sixteen working warps, one CTA per SM; every tile double buffered, and the outputs staged in
// tiles of their own, so that a chunk's places take the next but one as soon as its products
// are done. For the steps that the units share a warp owns 16 columns. Backwards in time the rows
// of low lanes have the most scores to convert: the state lies in the high ones, (4) taking the
// tile before Q's for the rows that nobody reads. (1), P, (3) and the output of the units are handed
// on separately, unit 1 ahead, whose (3) waits for no sum of (4): one unit's steps run under the
// other's products. (Handed on together, with the state in the low lanes: B=8 N=4096 H=8 D=64 122 us
// in all, not 105.)
enum { kTileK, kTileV, kTileQ, kTileG };
struct KvSmem {
    static constexpr int kReads = 2;
    static constexpr uint32_t kW = 8 * kTile, kO = kW + 2 * kTile, kS = kO + 2 * kTile, kMisc = kS + kReads * kTile / 2;
    static constexpr int kBytes = kMisc + misc_bytes(true);
};
static_assert(KvSmem::kBytes <= 227 * 1024, "shared memory");
constexpr uint32_t kKvX = 256, kKvO2 = 320;        // TMEM: scores of unit u at 128 u; + 128 u

struct KvMaps {
    CUtensorMap in[4], dk, dv;
};

__global__ void __launch_bounds__(32 * (2 * kWork + 2), 1)
decay_kv_kernel(const __grid_constant__ KvMaps maps, const __grid_constant__ Args a, const __grid_constant__ Tensor dk,
                const __grid_constant__ Geo geo, const __grid_constant__ Geo vgeo, WsHeader* hdr) {
    using L = KvSmem;
    constexpr int kWarps = 2 * kWork;
    extern __shared__ __align__(1024) uint8_t base[];
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    auto tile = [&](int i, int k) { return base + ((i & 1) * 4 + k) * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, 1, blockIdx.z);
    if (pl.nc == 0) {
        pdl_wait();
        return;
    }
    if ((smem_u32(base) & 1023) != 0) {
        if (tid == 0) set_status(hdr, LA_ERR_CUDA);
        return;
    }
    if (tid == 0) {
        for (uint64_t* bar : {&m.c_full[0], &m.c_full[1], &m.p_full[0], &m.p_full[1], &m.s_full, &m.o_full[0],
                              &m.o_full[1], &m.o_free, &m.drain})
            mbar_init(bar, 1);
        for (uint64_t* bar : {&m.prep, &m.pt[0], &m.staged}) mbar_init(bar, kWarps);
        mbar_init(&m.pt[1], kWork);
        fence_mbar_init();
        m.any = kNone;
    }
    if (tid < 128) m.first[tid] = kNone;
    const float l = a.decay[pl.h], l2 = log2_decay(l);
    init_tables<true, true>(m, l2);
    if (warp == kWarps) {
        tmem_alloc(&m.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;
    bool ok = true;

    if (warp == kWarps) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            const uint32_t base_a = smem_u32(base);
            const uint64_t km = kmajor_desc(base_a), rows = rows_desc(base_a);
            const uint64_t sr = rows_desc(base_a + L::kS), sk = kmajor_desc(base_a + L::kS);
            constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
            constexpr uint32_t id_o = idesc_bf16_f32(128, 64, false, true), id_t = idesc_bf16_f32(128, 64, false, false);
            auto at = [&](uint64_t d, int i, int k) { return step_desc(d, ((i & 1) * 4 + k) * kTile); };
            auto scores = [&](int i, int u) {                                                           // (1)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_bf16(tmem + 128 * u, kmajor_step(at(km, i, u), k), kmajor_step(at(km, i, 2 + u), k), id_sc, k > 0);
                mma_commit(&m.p_full[u]);
            };
            auto outputs = [&](int i, int u) {                                                          // (3)
#pragma unroll
                for (int part = 1; part >= 0; --part)
#pragma unroll
                    for (int k = 0; k < kC / 16; ++k)
                        mma_bf16_ts(tmem + kKvX + 128 * u, tmem + 128 * u + 16 * k + 8 * part,
                                    step_desc(at(rows, i, u ? kTileQ : kTileG), k * 2048), id_o, part < 1 || k > 0);
                mma_commit(&m.o_full[u]);
            };
            if ((ok = mbar_wait(&m.c_full[0], 0, max_spin))) {
                tc_fence_after();
                scores(0, 1);
                scores(0, 0);
            }
            for (int i = 0; i < pl.nc && ok; ++i) {
                if (!(ok = mbar_wait(&m.prep, i & 1, max_spin))) break;
                tc_fence_after();
                issue_state<1, 2>(tmem + kKvX, at(rows, i, kTileQ - 1), base_a + L::kW);                // (4)
#pragma unroll
                for (int part = L::kReads - 1; part >= 0; --part)                                       // (2)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t more = part < L::kReads - 1 || k > 0, term = part * kTile / 2;
                        mma_bf16(tmem + kKvO2 + 128, kmajor_step(at(km, i, kTileV), k), step_desc(kmajor_step(sk, k), term), id_t, more);
                        mma_bf16(tmem + kKvO2, kmajor_step(at(km, i, kTileK), k), step_desc(sr, term + k * 2048), id_o, more);
                    }
                mma_commit(&m.s_full);
                if (!(ok = mbar_wait(&m.pt[1], i & 1, max_spin))) break;
                tc_fence_after();
                outputs(i, 1);
                if (!(ok = mbar_wait(&m.pt[0], i & 1, max_spin))) break;
                tc_fence_after();
                outputs(i, 0);
                const bool more = i + 1 < pl.nc;
                if (more && !(ok = mbar_wait(&m.c_full[(i + 1) & 1], ((i + 1) >> 1) & 1, max_spin))) break;
                for (int u = 1; u >= 0; --u) {
                    if (!(ok = mbar_wait(&m.o_full[u], i & 1, max_spin))) break;
                    tc_fence_after();
                    if (more) scores(i + 1, u);
                }
            }
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else if (warp == kWarps + 1) {
        // ------------------------------------------------------------ loads and stores
        if (lane == 0) {
            int n = 0;
            auto load = [&]() {
                if (hold) return;
                const int t = pl.chunk<true>(n) * kC;
                uint64_t* bar = &m.c_full[n & 1];
                mbar_arrive_expect_tx(bar, 4 * kTile);
                tma_load_4d(tile(n, kTileK), &maps.in[kTileK], bar, 0, geo.ah * pl.h, t, geo.ab * pl.b);
                tma_load_4d(tile(n, kTileQ), &maps.in[kTileQ], bar, 0, geo.bh * pl.h, t, geo.bb * pl.b);
                tma_load_4d(tile(n, kTileV), &maps.in[kTileV], bar, 0, vgeo.ah * pl.h, t, vgeo.ab * pl.b);
                tma_load_4d(tile(n, kTileG), &maps.in[kTileG], bar, 0, geo.ch * pl.h, t, geo.cb * pl.b);
                if (++n + 1 < pl.nc) {             // the chunk after the next comes to L2 ahead of its load
                    const int next = pl.chunk<true>(n + 1) * kC;
                    tma_prefetch_4d(&maps.in[kTileK], 0, geo.ah * pl.h, next, geo.ab * pl.b);
                    tma_prefetch_4d(&maps.in[kTileQ], 0, geo.bh * pl.h, next, geo.bb * pl.b);
                    tma_prefetch_4d(&maps.in[kTileV], 0, vgeo.ah * pl.h, next, vgeo.ab * pl.b);
                    tma_prefetch_4d(&maps.in[kTileG], 0, geo.ch * pl.h, next, geo.cb * pl.b);
                }
            };
            load();
            if (pl.nc > 1) load();
            for (int i = 0; i < pl.nc; ++i) {
                // The outputs, staged by the working warps; a ragged chunk's were written row by row. They
                // are there after (3), the last to read a chunk's tiles. (The barrier of (3) itself could
                // complete the next chunk's phase before it is looked at here: the next but one
                // needs these loads, the next does not. This one's next phase needs o_free.)
                if (!(ok = mbar_wait(&m.staged, i & 1, max_spin))) break;
                if (i + 2 < pl.nc) load();
                const int t = pl.chunk<true>(i) * kC;
                if (t + kC <= pl.n || pl.n == a.N) {
                    tma_store_4d(&maps.dv, base + L::kO, 0, pl.h, t, pl.b);
                    tma_store_4d(&maps.dk, base + L::kO + kTile, 0, pl.h, t, pl.b);
                    tma_store_commit();
                    tma_store_wait_read<0>();
                }
                mbar_arrive(&m.o_free);
            }
            tma_store_wait_all<0>();
            for (int j = max(n - 2, 0); j < n; ++j) mbar_wait(&m.c_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, g4 = warp >> 2, u = g4 >> 1, g = g4 & 1, row = 32 * q + lane, im = 127 - row;
        const uint32_t tm = tmem + ((uint32_t)(32 * q) << 16), tmu = tm + kKvX + 128 * u + 32 * g;
        const bool has_state = q >= 2;             // few scores to convert there
        const RowFactors rf = row_factors(l2, im);
        // State row `row - 64`, columns 16 g4 ..
        float st[16];
        if (has_state) start_state(a, pl, l, row - 64, 16 * g4, st);
        const float read = a.scale * pow2((float)(im + 1) * l2), w = pow2((float)row * l2);
        const Factor whole = factor(kC * log_decay(l));
        const Tensor& out = u ? dk : a.o;
        const int width = u ? a.Da : a.Dc;
        // w dout of a chunk, once its tiles are there; whether the values that this unit's (3)
        // reads are finite.
        bool fine = true;
        auto weigh = [&](int i) -> bool {
            const int mt = min(kC, pl.n - pl.chunk<true>(i) * kC);
            uint8_t *gt = tile(i, kTileG), *qt = tile(i, kTileQ);
            if (!warp_wait(&m.c_full[i & 1], (i >> 1) & 1, max_spin)) return false;
            if (mt < kC && pl.n < a.N && row >= mt) {
                clear_pieces<2>(gt, row, 2 * g4);
                clear_pieces<2>(qt, row, 2 * g4);
            }
            write_weighted<2, 2>(gt, base + L::kW, w, row, 2 * g4);
            // (Rows past the sequence's end may not be clear yet: taking values out of them does no harm.)
            fine = finite_pieces(u ? qt : gt, row, 4 * g);
            return true;
        };
        auto put_state = [&]() {
            if (has_state) write_state<L::kReads>(base + L::kS, kTile / 2, st, row - 64, 2 * g4);
        };
        ok = weigh(0);
        put_state();
        for (int i = 0; i < pl.nc && ok; ++i) {
            const int t0 = pl.chunk<true>(i) * kC, mt = min(kC, pl.n - t0);
            const bool ragged = mt < kC && pl.n < a.N;
            uint8_t *gt = tile(i, kTileG), *qt = tile(i, kTileQ), *ct = base + L::kO + u * kTile;
            // ---------------------------------------------------- the operands of (2) and (4) are there
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.prep);
            // ---------------------------------------------------- scores to P
            if (!(ok = warp_wait(&m.p_full[u], i & 1, max_spin))) break;
            tc_fence_after();
#pragma unroll 1
            for (int bm = g; bm < 4; bm += 2) scores_to_p<true, true>(tm + 128 * u, 3 - bm, bm, 3 - q, rf, m, ragged ? mt : kC);
            // ---------------------------------------------------- state
            auto hand_over = [&](uint64_t* to) {
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(to);
            };
            if (u == 1 && fine) hand_over(&m.pt[1]);
            if (!(ok = warp_wait(&m.s_full, i & 1, max_spin))) break;
            tc_fence_after();
            if (has_state) join_state(tm + kKvX + 16 * g4, whole, st);
            // (1) and (4) have read the tiles as they came; (3) must not read values that are not finite.
            if (!fine) {
                take_out(u ? qt : gt, row, 32 * g, 32 * g + 32, i * kC + im, &m.any, m.first + 64 * u);
                fence_proxy_async_smem();
                if (u == 1) hand_over(&m.pt[1]);
            }
            hand_over(&m.pt[0]);                       // its (3) takes the columns of (4)
            // ---------------------------------------------------- the next w dout and state, under (3)
            if (i + 1 < pl.nc && !(ok = weigh(i + 1))) break;
            put_state();
            // ---------------------------------------------------- output
            if (!(ok = warp_wait(&m.o_full[u], i & 1, max_spin))) break;
            tc_fence_after();
            if (i > 0 && !(ok = warp_wait(&m.o_free, (i - 1) & 1, max_spin))) break;
            const bool spoiled = *const_cast<volatile int*>(&m.any) != kNone;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint4 x, y;
                join_output(tmu + 16 * k, tmu + 64 + 16 * k, a.scale, read, &x, &y);
                if (spoiled) {
                    const int* first = m.first + 64 * u + 32 * g + 16 * k;
                    x = put_nan(first, i * kC + im, x);
                    y = put_nan(first + 8, i * kC + im, y);
                }
                if (!ragged) {
                    *reinterpret_cast<uint4*>(ct + row * 128 + (((4 * g + 2 * k) ^ (row & 7)) << 4)) = x;
                    *reinterpret_cast<uint4*>(ct + row * 128 + (((4 * g + 2 * k + 1) ^ (row & 7)) << 4)) = y;
                } else if (row < mt) {
                    const int c = 32 * g + 16 * k;
                    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(const_cast<void*>(out.p)) + pl.b * out.bs + pl.h * out.hs +
                                        (int64_t)(t0 + row) * out.ts + c;
                    if (c < width) *reinterpret_cast<uint4*>(to) = x;
                    if (c + 8 < width) *reinterpret_cast<uint4*>(to + 8) = y;
                }
            }
            fence_proxy_async_smem();
            tc_fence_before();
            warp_arrive(&m.staged);
        }
    }
    if (!ok) report_timeout(hdr);
    pdl_wait();                                // as `late` of decay_tc_kernel
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWarps) tmem_dealloc(tmem, 512);
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

// One sum with its tensor maps.
struct Sum {
    Args a;
    Geo geo;
    CUtensorMap am, bm, cm, om;
    bool encode() {
        geo = {};
        return encode_rows(&am, a.a, a.Da, a.B, a.H, a.N, &geo.ah, &geo.ab) &&
               encode_rows(&bm, a.b, a.Da, a.B, a.H, a.N, &geo.bh, &geo.bb) &&
               encode_rows(&cm, a.c, a.Dc, a.B, a.H, a.N, &geo.ch, &geo.cb) &&
               encode_rows(&om, a.o, a.Dc, a.B, a.H, a.N, nullptr, nullptr);
    }
    unsigned heads() const { return (unsigned)(a.B * a.H); }
};

template <int kT, int kU, int kTerms>
cudaError_t launch_sums(const Sum* s, int count, WsHeader* hdr, cudaStream_t st) {
    static std::atomic<int> optin[kMaxDevices];
    constexpr int bytes = SumSmem<kT, kU, kTerms>::kBytes;
    const cudaError_t e = ensure_smem_optin(decay_sums_kernel<kT, kU, kTerms>, bytes, optin);
    if (e != cudaSuccess) return e;
    const Sum &x = s[0], &y = s[count - 1];
    const dim3 grid((x.a.Dc + 64 * kU - 1) / (64 * kU), x.a.nseg - 1, x.heads() * count);
    decay_sums_kernel<kT, kU, kTerms><<<grid, 32 * (kU * kWork + 1), bytes, st>>>(x.bm, x.cm, y.bm, y.cm, x.a, x.geo, y.a, y.geo, hdr);
    return cudaPeekAtLastError();
}

template <int kT, int kU, int kTerms, bool kRev>
cudaError_t launch_main(const Sum& s, bool dependent, WsHeader* hdr, cudaStream_t st) {
    static std::atomic<int> optin[kMaxDevices];
    constexpr int bytes = Smem<kT, kU, kTerms>::kBytes;
    const cudaError_t e = ensure_smem_optin(decay_tc_kernel<kT, kU, kTerms, kRev>, bytes, optin);
    if (e != cudaSuccess) return e;
    return scan::launch_after(decay_tc_kernel<kT, kU, kTerms, kRev>, dim3((s.a.Dc + 64 * kU - 1) / (64 * kU), s.a.nseg, s.heads()),
                              32 * (kU * kWork + 2), bytes, st, dependent, s.am, s.bm, s.cm, s.om, s.a, s.geo, hdr);
}

// By widths: one or two 64-row tiles of the state, one or two column blocks.
template <int kTerms> cudaError_t sums_of(const Sum* s, int count, WsHeader* hdr, cudaStream_t st) {
    if (s->a.Da <= 64) return s->a.Dc <= 64 ? launch_sums<1, 1, kTerms>(s, count, hdr, st) : launch_sums<1, 2, kTerms>(s, count, hdr, st);
    return s->a.Dc <= 64 ? launch_sums<2, 1, kTerms>(s, count, hdr, st) : launch_sums<2, 2, kTerms>(s, count, hdr, st);
}
template <int kTerms, bool kRev> cudaError_t main_of(const Sum& s, bool dependent, WsHeader* hdr, cudaStream_t st) {
    if (s.a.Da <= 64)
        return s.a.Dc <= 64 ? launch_main<1, 1, kTerms, kRev>(s, dependent, hdr, st)
                            : launch_main<1, 2, kTerms, kRev>(s, dependent, hdr, st);
    return s.a.Dc <= 64 ? launch_main<2, 1, kTerms, kRev>(s, dependent, hdr, st)
                        : launch_main<2, 2, kTerms, kRev>(s, dependent, hdr, st);
}

bool narrow(int Dk, int Dv) { return Dk <= 64 && Dv <= 64; }

// Whether dk and dv come from one pass: narrow heads of more than one chunk. One chunk has no next
// to prepare under its products, and two CTAs per SM do more: the whole backward of N=100 D=64,
// 160 heads 18.1 us against 20.1, 2048 heads 144 against 151 (16 heads of N=64 9.4 against 8.8).
bool together(int N, int Dk, int Dv) { return narrow(Dk, Dv) && N > kC; }

// Segments of the forward pass. CTAs run in waves, so the cut is the one whose waves times
// chunks is least; in chunks: starting and ending a CTA 1, the first pass 0.4 of the main
// pass, and with segments two further launches 2.
int forward_segments(int64_t BH, int N, int Dk, int Dv) {
    const int chunks = (N + kC - 1) / kC;
    const int64_t slots = (narrow(Dk, Dv) ? 2 : 1) * (int64_t)sm_count();
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 64 && n <= chunks; ++n) {
        const int per = (chunks + n - 1) / n;
        if ((chunks + per - 1) / per != n) continue;       // the same split with empty segments
        const double waves = (double)((BH * n + slots - 1) / slots);
        const double cost = waves * (per + 1.0) + (n > 1 ? 0.4 * waves * per + 2.0 : 0.0);
        if (cost < least) least = cost, best = n;
    }
    return best;
}

// Segments of the backward pass, the same for dq and for dk and dv, in chunks of the main
// passes as above. Those run side by side while their CTAs fit the SMs together (two of dq to
// one where heads are narrow), else one after the other. Single calls on a cold L2, B=8 N=4096 H=8
// D=64, 32 chunks, P in one term: not cut 100 us, two segments 120, four 130; B=4 N=2047 H=8
// D=128, 16 chunks: 65, 89, 99.
int backward_segments(int64_t BH, int N, int Dk, int Dv) {
    const int chunks = (N + kC - 1) / kC;
    const double sms = sm_count(), shares[3] = {narrow(Dk, Dv) ? 0.5 : 1.0, 1.0, narrow(Dk, Dv) ? 0.0 : 1.0};
    int best = 1;
    double least = 1e30;
    for (int n = 1; n <= 64 && n <= chunks; ++n) {
        const int per = (chunks + n - 1) / n;
        if ((chunks + per - 1) / per != n || (n > 1 && 2 * BH > 65535)) continue;   // both sums' first passes: grid.z
        double used = 0.0, each = 0.0;
        for (double share : shares) {
            used += share * BH * n;
            if (share > 0.0) each += ceil(share * BH * n / sms) * (per + 1.5);
        }
        const double cost = (used <= sms ? per + 1.5 : each) +
                            (n > 1 ? ceil((shares[0] + shares[2]) * BH * (n - 1) / sms) * (0.4 * per + 1.0) + 1.0 : 0.0);
        if (cost < least) least = cost, best = n;
    }
    return best;
}

// Segments whose end states a CTA of the main pass joins itself; more are chained by a launch
// of their own.
constexpr int kFold = 6;

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

namespace {

void cut_forward(Args* a) {
    cut(a, forward_segments((int64_t)a->B * a->H, a->N, a->Da, a->Dc), kC);
    a->fold = a->nseg - 1 <= kFold;
}
void cut_backward(Args* a) {
    cut(a, backward_segments((int64_t)a->B * a->H, a->N, a->Da, a->Dc), kC);
    a->fold = a->nseg - 1 <= kFold;
}

Args cut_of(int64_t BH, int N, int Dk, int Dv, bool backward) {
    Args a = {};
    a.B = 1, a.H = (int)BH, a.N = N, a.Da = Dk, a.Dc = Dv;
    backward ? cut_backward(&a) : cut_forward(&a);
    return a;
}

}  // namespace

size_t tc_seeds(int64_t BH, int N, int Dk, int Dv, bool backward) {
    const Args a = cut_of(BH, N, Dk, Dv, backward);
    return a.nseg > 1 ? (size_t)BH * a.nseg * Dk * Dv * (backward ? 2 : 1) : 0;
}

int tc_launches(int64_t BH, int N, int Dk, int Dv, bool backward) {
    const Args a = cut_of(BH, N, Dk, Dv, backward);
    const int sums = backward && (Dk <= 64) != (Dv <= 64) ? 2 : 1, main = !backward ? 1 : together(N, Dk, Dv) ? 2 : 3;
    return main + (a.nseg > 1 ? sums + (a.fold ? 0 : 1) : 0);
}

cudaError_t tc_run(Args a, void* ws_header, cudaStream_t st) {
    cut_forward(&a);
    // Where the last segment writes its state over the first one's, only the chaining reads that.
    if (a.S0 && a.S0 == a.S_out) a.fold = a.nseg == 1;
    Sum s = {a};
    if (!s.encode()) return cudaErrorInvalidValue;
    WsHeader* hdr = static_cast<WsHeader*>(ws_header);
    cudaError_t e;
    if (a.nseg > 1) {
        if ((e = a.S_out ? sums_of<3>(&s, 1, hdr, st) : sums_of<2>(&s, 1, hdr, st)) != cudaSuccess) return e;
        if (!a.fold && (e = launch_chain(&a, 1, kC, st)) != cudaSuccess) return e;
    }
    return a.S_out ? main_of<3, false>(s, a.nseg > 1, hdr, st) : main_of<2, false>(s, a.nseg > 1, hdr, st);
}

// With segments the first passes of S (for dq) and of R (for dk and dv) and their chaining; then
// dq and dk and dv, the last two in one pass where it pays.
cudaError_t tc_backward(Args dq, Args dk, Args dv, void* ws_header, cudaStream_t st) {
    cut_backward(&dv);
    const bool cut = dv.nseg > 1;
    for (Args* a : {&dq, &dk}) a->nseg = dv.nseg, a->seg_len = dv.seg_len, a->fold = dv.fold;
    dk.seeds = dv.seeds = dq.seeds + (cut ? (size_t)dq.B * dq.H * dq.nseg * dq.Da * dq.Dc : 0);
    dk.seeds_t = 1;
    Sum s[3] = {{dq}, {dv}, {dk}};
    for (Sum& x : s)
        if (!x.encode()) return cudaErrorInvalidValue;
    WsHeader* hdr = static_cast<WsHeader*>(ws_header);
    cudaError_t e;
    if (cut) {
        const bool alike = (dq.Da <= 64) == (dq.Dc <= 64);   // S and R have the same shape
        if ((e = sums_of<2>(s, alike ? 2 : 1, hdr, st)) != cudaSuccess) return e;
        if (!alike && (e = sums_of<2>(s + 1, 1, hdr, st)) != cudaSuccess) return e;
        const Args chained[2] = {dq, dv};
        if (!dq.fold && (e = launch_chain(chained, 2, kC, st)) != cudaSuccess) return e;
    }
    if ((e = main_of<2, false>(s[0], cut, hdr, st)) != cudaSuccess) return e;
    if (together(dv.N, dv.Da, dv.Dc)) {
        static std::atomic<int> optin[kMaxDevices];
        if ((e = ensure_smem_optin(decay_kv_kernel, KvSmem::kBytes, optin)) != cudaSuccess) return e;
        const KvMaps maps = {{s[1].am, s[2].am, s[1].bm, s[1].cm}, s[2].om, s[1].om};
        return scan::launch_after(decay_kv_kernel, dim3(1, dv.nseg, s[1].heads()), 32 * (2 * kWork + 2), KvSmem::kBytes, st,
                                  true, maps, dv, dk.o, s[1].geo, s[2].geo, hdr);
    }
    s[1].geo.late = s[2].geo.late = 1;
    for (int i = 1; i < 3; ++i)
        if ((e = main_of<2, true>(s[i], true, hdr, st)) != cudaSuccess) return e;
    return cudaSuccess;
}

}  // namespace decay

}  // namespace la
