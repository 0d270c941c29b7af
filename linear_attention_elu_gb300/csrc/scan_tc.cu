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
// once each (at most 2^-8 of a term, as the output itself). The state is held in fp32 in
// TMEM: it is scaled there per chunk, and (4) adds w x as bf16 terms, each the remainder of
// those before. A state that the call returns, and those that segments start from, take
// three (2^-25 of w x is left; states 1e-7 to 7e-7 off in all); a state that is only read
// for y takes two (2^-17), whose tiles leave room for two output slots.
// Decays of P below the diagonal 32 x 32 blocks are products of factors <= 1 (from token j
// to its block's end, over the blocks between, from the block row's start to token i), so
// only the diagonal blocks take an exponential per score. Each factor's exponent is a sum of
// its own tokens; the diagonal blocks' are differences of sums from the block's start, so
// that a small exponent is not a difference of two large ones from further back.
//
// Schedule (20 warps, one CTA per SM). An item is one chunk of one unit. Two groups
// of eight warps alternate items; a warp owns 32 rows and half of the columns. A
// group prepares its item (scores to P, state to bf16 and scaled, weighted values),
// hands it over, and writes its output while the other group prepares the next. One
// thread issues (2), (3), (4) of an item, and (1) of the next chunk, which run under
// the groups' steps. The other warps: TMA loads, step sizes to decays, and the output
// slots (gate in, output in place, TMA store). All hand-offs are mbarriers; every wait
// is bounded. Loops over columns are kept rolled: the steps' code competes for the
// instruction cache (the output step unrolled twice cost 6 % of the call).
// Measured on B=1 N=65536 H=32 P=64 S=128 with a gate, 126 us of HBM time: a form of this
// pass with one warpgroup per step ran 470 us, all sixteen warps on one item 312, two groups
// 290; the call 416.
// A second issuing thread, the products issued by predicate instead of by branch, and
// x kept in registers from the weights to the output all measured slower.
// Sequences are cut into segments when there are too few units for the SMs: the first
// pass streams (4) alone, in reverse order of chunks so that the weights reach to the
// segment's end and nothing has to be rescaled (a quarter of the call); seeds are chained by csrc/scan.cu, which
// writes the final state too, and the second pass starts from them.
// What bounds it: the groups' instructions (about 9,600 of a warp an item of 128 tokens x 64
// values, 44 % of the issue slots, each warp waiting on its own chain of TMEM reads,
// exponentials and hand-offs) next to the products' operand reads from shared memory
// (196 KB an item at 128 bytes a cycle).
#include <cuda.h>
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "mixing.cuh"
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

// One unit's decays over a chunk, exponents in base 2. Sums start at every 32 tokens (the
// blocks of the scores): after a token that decays by a large factor, a sum from the chunk's
// start would leave no digits to the differences between the slow tokens behind it.
struct Decay {
    float loc[kC];      // sum from the token's block's start up to and including t
    float d[kC];        // step sizes, 0 past the sequence's end (not folded into an exponent:
                        // next to a large sum their logarithm would lose its digits)
    float off[192];     // d_t 2^(sum from t to the start of block q): q = 1 32 tokens, then q = 2 64, q = 3 96
    float w[kC];        // d_t 2^(sum over the tokens of the chunk after t), 0 past the end
    float start[kC];    // 2^l_t
    float total;        // 2^l_end
    float pad[3];
};

// A unit's values that are not finite. They would reach the tokens before them too: (3) adds
// 0 x for every later token of the chunk, and 0 times an infinity is NaN. So (3) gets 0 in
// their place, and their columns' outputs are set to NaN from their token on; the state, which
// takes the values as they are, is not finite from there on by itself.
struct Bad {
    int first[64];      // per column, the first such token
    int any;            // the first of all
    int pad[3];
};
constexpr int kNone = 0x7fffffff;

struct Units {
    int ctas, units, blocks;    // CTAs per group, units per group, 64-column blocks per head
    int per;                    // units per CTA, 1 or 2
    int cps;                    // chunks per segment
    int gate_vec;               // z rows are 16-byte aligned
};

// TMEM columns of the main kernel.
constexpr uint32_t kTmSc = 0, kTmP = 128, kTmY1 = 256, kTmY2 = 320, kTmSt = 384;

// Barriers of items are kept per item parity: a group of warps sees every second
// item, and one that skipped phases of a barrier could take an earlier phase's
// parity for its own.
struct Misc {
    uint64_t c_full, c_empty, b_full[2], b_empty[2], x_full[2], x_empty[2], dt_full[kDtRing], dt_empty[kDtRing];
    uint64_t slot_ready[2], y_staged[2], sc_full[2], item_ready, read_done[2], y_full[2], state_done[2], drain;
    uint32_t tmem_slot;
};

// Shared memory of the main kernel, from a 1024-byte boundary. B is double
// buffered; C, which the read of the state frees half an item earlier, is not: its
// 32 KB hold the output slots instead (gate in, output in place, TMA store). With three
// terms of 128 state rows there is room for one slot (B=8 N=333 H=16 S=128: 20.6 us in a
// graph, 18.6 with two terms and two slots).
template <int kT, int kTerms> struct Smem {
    static constexpr int kSlots = kT * kTerms < 6 ? 2 : 1;
    static constexpr uint32_t kC0 = 0, kB0 = kT * kTile;
    static constexpr uint32_t kX = 3 * kT * kTile;
    static constexpr uint32_t kXw = kX + 2 * kTile;            // value, remainder (and its remainder)
    static constexpr uint32_t kOut = kXw + kTerms * kTile;     // gate, then output
    static constexpr uint32_t kSb = kOut + kSlots * kTile;     // bf16 state, 64 kT rows
    static constexpr uint32_t kDt = kSb + kT * 64 * 128;
    static constexpr uint32_t kMask = kDt + (kDtRing * sizeof(Decay) + 127) / 128 * 128;
    static constexpr uint32_t kBad = kMask + 32 * 16 * 4;      // diagonal block: 16 words of pairs per row
    static constexpr uint32_t kMisc = kBad + 2 * sizeof(Bad);
    static constexpr uint32_t kEnd = kMisc + sizeof(Misc);
    static constexpr size_t kBytes = 1024 + kEnd;
};
static_assert(Smem<2, 2>::kBytes <= 227 * 1024 && Smem<2, 3>::kBytes <= 227 * 1024, "main kernel's shared memory");

constexpr int kThreads = 640;
constexpr int kWork = 16;              // warps of the items' steps (two groups); then TMA, MMA, decays, slots
constexpr int kGroup = kWork / 2;
constexpr int kAhead = 3;              // items between a tile's L2 prefetch and its load

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The warp goes on once two loaded values are in every lane's registers. Loads whose values
// are used only later may complete after an arrival that follows them; here the TMA would
// then overwrite what they read.
__device__ __forceinline__ void arrived(uint32_t a, uint32_t b) {
    asm volatile("{\n .reg .pred p, q;\n setp.eq.u32 p, %0, %1;\n vote.sync.any.pred q, p, 0xffffffff;\n}\n" ::"r"(a),
                 "r"(b)
                 : "memory");
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
    const int cta = blockIdx.x % un.ctas;
    p.g = blockIdx.x / un.ctas;
    p.seg = blockIdx.y;
    p.b = blockIdx.z;
    p.unit0 = un.per * cta;
    p.nu = min(un.per, un.units - p.unit0);
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

// Of d A log2 e over the 128 tokens: inclusive sums from the start of each block of 32 (loc),
// exclusive sums from its end (suf) and the blocks' sums; and the step sizes themselves. A
// token's exponent is held within -127, where its factor is 0 in fp32 already, so that sums
// over a block stay below 4096 (digits of 2^-12) and never reach an infinity. A comparison,
// so that NaN stays NaN.
__device__ __forceinline__ void decays(const ScanArgs& a, const Place& pl, int c, float A, float bias,
                                       const float (&raw)[4], float (&d)[4], float (&loc)[4],
                                       float (&suf)[4], float (&blk)[4]) {
    const int lane = threadIdx.x & 31, in = lane & 7, t = c * kC + 4 * lane;
    float l[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        d[k] = t + k < pl.n ? step_size(raw[k] + bias, a.softplus) : 0.f;
        const float e = t + k < pl.n ? d[k] * A * kLog2e : 0.f;
        l[k] = e < -127.f ? -127.f : e;
    }
    const float own = (l[0] + l[1]) + (l[2] + l[3]);
    float up = own, down = own;              // inclusive scans over a block's lanes, both directions
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        const float x = __shfl_up_sync(0xffffffffu, up, o, 8);
        const float y = __shfl_down_sync(0xffffffffu, down, o, 8);
        if (in >= o) up += x;
        if (in + o < 8) down += y;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) blk[k] = __shfl_sync(0xffffffffu, down, 8 * k);
    float before = __shfl_up_sync(0xffffffffu, up, 1, 8), after = __shfl_down_sync(0xffffffffu, down, 1, 8);
    if (in == 0) before = 0.f;
    if (in == 7) after = 0.f;
    loc[0] = before + l[0];
    loc[1] = loc[0] + l[1];
    loc[2] = loc[1] + l[2];
    loc[3] = loc[2] + l[3];
    suf[3] = after;
    suf[2] = suf[3] + l[3];
    suf[1] = suf[2] + l[2];
    suf[0] = suf[1] + l[1];
}

// Sums over the blocks before and after the lane's own.
__device__ __forceinline__ void other_blocks(const float (&blk)[4], float* before, float* after) {
    const int own = (threadIdx.x & 31) >> 3;
    *before = (own > 0 ? blk[0] : 0.f) + (own > 1 ? blk[1] : 0.f) + (own > 2 ? blk[2] : 0.f);
    *after = (own < 1 ? blk[1] : 0.f) + (own < 2 ? blk[2] : 0.f) + (own < 3 ? blk[3] : 0.f);
}

// Sixteen weighted values: hi = bf16(w x), lo = bf16(w x - hi), last = bf16(w x - hi - lo).
__device__ __forceinline__ void weigh16(uint4 a, uint4 b, float w, uint32_t (&hi)[8], uint32_t (&lo)[8],
                                        uint32_t (&last)[8]) {
    const uint64_t w2 = pk2(w, w), minus = pk2(-1.f, -1.f);
    const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint64_t p = mul2(bf2(in[k]), w2);
        hi[k] = pack2(p);
        const uint64_t r = fma2(bf2(hi[k]), minus, p);
        lo[k] = pack2(r);
        last[k] = pack2(fma2(bf2(lo[k]), minus, r));
    }
}

// One row of a [128 x 64] tile set to 0.
__device__ __forceinline__ void zero_row(uint8_t* tile, int row) {
#pragma unroll
    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(tile + row * 128 + j * 16) = make_uint4(0, 0, 0, 0);
}

// Descriptor of the 16-row (or 16-column) step k of an operand whose first one is d:
// only the start address (in 16-byte units) moves.
__device__ __forceinline__ uint64_t step_desc(uint64_t d, uint32_t bytes) { return d + (bytes >> 4); }

// Operand with rows of 64 values along M or N (one row per k): steps of 16 rows.
__device__ __forceinline__ uint64_t rows_desc(uint32_t tile) { return smem_desc(tile, kTile, 1024, kSwizzle128B); }
// K-major operand (64 k per row of a tile, tiles kTile apart): steps of 16 k.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile) { return smem_desc(tile, 16, 1024, kSwizzle128B); }
__device__ __forceinline__ uint64_t kmajor_step(uint64_t d, int k) {
    return step_desc(d, (k >> 2) * kTile + (k & 3) * 32);
}

// (4): state += B^T (sum of the terms), issued by one thread; their tiles follow one another. The second
// 64-row atom of the A operand is the tile after B's (for kT = 1 whatever tile follows:
// those lanes are unused).
template <int kTerms>
__device__ __forceinline__ void issue_state(uint32_t dst, uint64_t bt, uint64_t hi) {
    constexpr uint32_t id = idesc_bf16_f32(128, 64, true, true);
#pragma unroll
    for (int part = 0; part < kTerms; ++part)
#pragma unroll
        for (int k = 0; k < kC / 16; ++k)
            mma_bf16(dst, step_desc(bt, k * 2048), step_desc(hi, part * kTile + k * 2048), id, 1u);
}

// Eight gate values of a row that is not 16-byte aligned.
__device__ __forceinline__ uint4 load_gate(const __nv_bfloat16* p) {
    const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = (uint32_t)__ldg(h + 2 * k) | ((uint32_t)__ldg(h + 2 * k + 1) << 16);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Columns c .. c + 15 of unit u's output row t, to global memory (ragged ends).
__device__ __noinline__ void put_row(const ScanArgs& a, const Place& pl, const Units& un, int u, int t, int c,
                                     uint4 o0, uint4 o1) {
    c += pl.col0(un, u);
    if (t >= pl.n || c >= a.P) return;
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + pl.b * a.y_bs + (int64_t)t * a.y_ts +
                       (int64_t)pl.head(a, un, u) * a.P + c;
    *reinterpret_cast<uint4*>(y) = o0;
    if (c + 8 < a.P) *reinterpret_cast<uint4*>(y + 8) = o1;
}

// The same columns of a gate row that the TMA cannot fetch, to its two pieces of the slot.
__device__ __noinline__ void put_gate(const ScanArgs& a, const Place& pl, const Units& un, int u, int t, int c,
                                      uint8_t* slot, uint32_t pc0, uint32_t pc1) {
    c += pl.col0(un, u);
    const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(a.z) + pl.b * a.z_bs + (int64_t)t * a.z_ts +
                             (int64_t)pl.head(a, un, u) * a.P + c;
    const bool in = t < pl.n;
    *reinterpret_cast<uint4*>(slot + pc0) = in && c < a.P ? load_gate(z) : make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(slot + pc1) = in && c + 8 < a.P ? load_gate(z + 8) : make_uint4(0, 0, 0, 0);
}

// Columns 32 g .. of row `row` of an x tile: notes the values that are not finite, and clears them.
__device__ __noinline__ void take_out(uint8_t* tile, int row, int g, int token, Bad* bad) {
    for (int c = 32 * g; c < 32 * g + 32; ++c) {
        unsigned short* v = reinterpret_cast<unsigned short*>(tile + row * 128 + (((c >> 3) ^ (row & 7)) << 4)) + (c & 7);
        if ((*v & 0x7F80u) != 0x7F80u) continue;
        *v = 0;
        atomicMin(&bad->first[c], token);
        atomicMin(&bad->any, token);
    }
}

// Outputs of the chunk at token t0 that such values reach, set to NaN: in the output slot, or
// (slot null) in the rows that were written one by one. One thread; a column whose first value
// is in an earlier chunk is NaN by its state.
__device__ __noinline__ void put_nan(const ScanArgs& a, const Place& pl, const Units& un, int u, int t0, uint8_t* slot,
                                     const Bad* bad) {
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + pl.b * a.y_bs + (int64_t)pl.head(a, un, u) * a.P + pl.col0(un, u);
    for (int c = 0; c < 64; ++c) {
        const int row0 = *const_cast<const volatile int*>(&bad->first[c]) - t0;
        if (row0 < 0) continue;
        for (int row = row0; row < kC; ++row) {
            if (slot)
                reinterpret_cast<unsigned short*>(slot + row * 128 + (((c >> 3) ^ (row & 7)) << 4))[c & 7] = 0x7FFF;
            else if (t0 + row < pl.n && pl.col0(un, u) + c < a.P)
                y[(t0 + row) * a.y_ts + c] = __ushort_as_bfloat16(0x7FFF);
        }
    }
    fence_proxy_async_smem();
}

// z / (1 + e^-z) of two packed bf16 values. e^-z overflows to infinity and its
// reciprocal is then 0: the limit.
__device__ __forceinline__ uint64_t gate2(uint32_t z) {
    const uint64_t v = bf2(z);
    float t0, t1, r0, r1;
    unpk2(mul2(v, pk2(-kLog2e, -kLog2e)), &t0, &t1);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(1.f + ex2(t0)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(1.f + ex2(t1)));
    return mul2(v, pk2(r0, r1));
}

template <int kT, int kTerms, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
scan_tc_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap cmap, const __grid_constant__ CUtensorMap zmap,
               const __grid_constant__ CUtensorMap ymap, const __grid_constant__ ScanArgs a,
               const __grid_constant__ Units un, WsHeader* hdr) {
    using L = Smem<kT, kTerms>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    Misc& m = *reinterpret_cast<Misc*>(base + L::kMisc);
    Decay* dts = reinterpret_cast<Decay*>(base + L::kDt);
    Bad* bad = reinterpret_cast<Bad*>(base + L::kBad);
    auto btile = [&](int s) { return base + L::kB0 + s * kT * kTile; };
    auto xtile = [&](int n) { return base + L::kX + (n & 1) * kTile; };
    auto oslot = [&](int n) { return base + L::kOut + n % L::kSlots * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, un);
    const bool last_seg = pl.seg == a.nseg - 1;
    if (pl.nc == 0 && !(last_seg && a.S_out)) {
        pdl_wait();                            // a dependent launch never ends before what it follows
        return;
    }
    const int nu = pl.nu, items = pl.nc * nu;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.b_full[s], 1);
            mbar_init(&m.b_empty[s], 1);
            mbar_init(&m.x_full[s], 1);
            mbar_init(&m.x_empty[s], kGroup);
            mbar_init(&m.slot_ready[s], 1);
            mbar_init(&m.y_staged[s], kGroup);
            mbar_init(&m.sc_full[s], 1);
            mbar_init(&m.read_done[s], 1);
            mbar_init(&m.y_full[s], 1);
            mbar_init(&m.state_done[s], 1);
        }
        for (int s = 0; s < kDtRing; ++s) {
            mbar_init(&m.dt_full[s], 1);
            mbar_init(&m.dt_empty[s], kGroup);
        }
        mbar_init(&m.c_full, 1);
        mbar_init(&m.c_empty, 1);
        mbar_init(&m.item_ready, kWork);
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (tid < 2 * (int)(sizeof(Bad) / sizeof(int))) reinterpret_cast<int*>(bad)[tid] = kNone;
    if (warp == kWork + 1) {
        tmem_alloc(&m.tmem_slot, 512);
        tmem_relinquish();
    }
    if (warp == kWork && lane == 0) {
        tma_prefetch_desc(&xmap);
        tma_prefetch_desc(&bmap);
        tma_prefetch_desc(&cmap);
        tma_prefetch_desc(&zmap);
        tma_prefetch_desc(&ymap);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The second pass is a programmatic dependent of the chaining kernel: everything above
    // touches no global memory but the lengths.
    pdl_wait();
    const uint32_t tmem = m.tmem_slot;
    const uint32_t max_spin = hdr->max_spin;
    const bool hold = hdr->hold_item != 0;                 // test hook: loads never issued
    // The last chunk of a ragged sequence is stored row by row: its number, or -1.
    const int by_rows = pl.n < a.N && (pl.c0 + pl.nc) * kC > pl.n ? pl.nc - 1 : -1;
    bool ok = true;

    if (warp == kWork) {
        // ------------------------------------------------------------ TMA loads
        if (lane == 0) {
            int i = 0, n = 0, c = 0;                       // chunks of B, value tiles, chunks of C issued
            auto load_x = [&](int u, int t) -> bool {
                if (n >= 2 && !mbar_wait(&m.x_empty[n & 1], ((n >> 1) - 1) & 1, max_spin)) return false;
                // The value and gate tiles after this one come to L2 ahead of their use.
                const int ia = i + (u + kAhead) / nu, ua = (u + kAhead) % nu;
                if (ia < pl.nc) {
                    const int ta = (pl.c0 + ia) * kC, ha = pl.head(a, un, ua), pa = pl.col0(un, ua);
                    tma_prefetch_4d(&xmap, pa, ha, ta, pl.b);
                    if (un.gate_vec) tma_prefetch_4d(&zmap, pa, ha, ta, pl.b);
                }
                mbar_arrive_expect_tx(&m.x_full[n & 1], kTile);
                tma_load_4d(xtile(n), &xmap, &m.x_full[n & 1], pl.col0(un, u), pl.head(a, un, u), t, pl.b);
                ++n;
                return true;
            };
            while (i < pl.nc && ok && !hold) {
                const int s = i & 1, t = (pl.c0 + i) * kC;
                if (i >= 2 && !(ok = mbar_wait(&m.b_empty[s], ((i >> 1) - 1) & 1, max_spin))) break;
                mbar_arrive_expect_tx(&m.b_full[s], kT * kTile);
#pragma unroll
                for (int k = 0; k < kT; ++k)
                    tma_load_4d(btile(s) + k * kTile, &bmap, &m.b_full[s], 64 * k, pl.g, t, pl.b);
                // C is free once the chunk before has been read from the state for its last unit.
                ok = load_x(0, t) && (i < 1 || mbar_wait(&m.c_empty, (i - 1) & 1, max_spin));
                if (ok) {
                    mbar_arrive_expect_tx(&m.c_full, kT * kTile);
#pragma unroll
                    for (int k = 0; k < kT; ++k)
                        tma_load_4d(base + L::kC0 + k * kTile, &cmap, &m.c_full, 64 * k, pl.g, t, pl.b);
                    ++c;
                    ok = nu < 2 || load_x(1, t);
                }
                ++i;
            }
            // Every issued load lands before the CTA exits.
            for (int j = max(i - 2, 0); j < i; ++j) mbar_wait(&m.b_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
            if (c > 0) mbar_wait(&m.c_full, (c - 1) & 1, kDefaultMaxSpin);
            for (int j = max(n - 2, 0); j < n; ++j) mbar_wait(&m.x_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
        }
    } else if (warp == kWork + 1) {
        // ------------------------------------------------------------ MMA
        // The whole warp walks the loop (its values stay uniform), one lane issues.
        constexpr uint32_t id_sc = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id_y = idesc_bf16_f32(128, 64, false, true);
        const uint32_t base_a = smem_u32(base);
        const uint64_t ca0 = kmajor_desc(base_a + L::kC0), bk0 = kmajor_desc(base_a + L::kB0);
        const uint64_t br0 = rows_desc(base_a + L::kB0), x0 = rows_desc(base_a + L::kX);
        const uint64_t sb0 = rows_desc(base_a + L::kSb), xw0 = rows_desc(base_a + L::kXw);
        const bool leader = lane == 0;
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            if (u == 0) {                      // (1); the items before it have read the old scores
                if (!(ok = warp_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin) && warp_wait(&m.c_full, i & 1, max_spin)))
                    break;
                tc_fence_after();
                if (leader) {
                    const uint64_t ba = step_desc(bk0, (i & 1) * kT * kTile);
#pragma unroll
                    for (int k = 0; k < 4 * kT; ++k)
                        mma_bf16(tmem + kTmSc, kmajor_step(ca0, k), kmajor_step(ba, k), id_sc, k > 0);
                    mma_commit(&m.sc_full[i & 1]);
                }
                __syncwarp();
            }
            if (!(ok = warp_wait(&m.item_ready, n & 1, max_spin))) break;
            tc_fence_after();
            if (leader) {
#pragma unroll
                for (int k = 0; k < 4 * kT; ++k)                                        // (2)
                    mma_bf16(tmem + kTmY2, kmajor_step(ca0, k), step_desc(sb0, k * 2048), id_y, k > 0);
                mma_commit(&m.read_done[n & 1]);
                if (u == nu - 1) mma_commit(&m.c_empty);
                const uint64_t xa = step_desc(x0, (n & 1) * kTile);
                const uint32_t pt = tmem + kTmP + 64 * (n & 1);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)                                       // (3)
                    mma_bf16_ts(tmem + kTmY1, pt + 8 * k, step_desc(xa, k * 2048), id_y, k > 0);
                mma_commit(&m.y_full[n & 1]);
                issue_state<kTerms>(tmem + kTmSt + 64 * u, step_desc(br0, (i & 1) * kT * kTile), xw0);  // (4)
                mma_commit(&m.state_done[n & 1]);
                if (u == nu - 1) mma_commit(&m.b_empty[i & 1]);
            }
            __syncwarp();
            if (++u == nu) u = 0, ++i;
        }
        if (leader) {
            mma_commit(&m.drain);              // every issued MMA completes before TMEM is released
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else if (warp == kWork + 2) {
        // ------------------------------------------------------------ step sizes to decays
        const int h0 = pl.head(a, un, 0), h1 = pl.head(a, un, nu - 1);
        const float A0 = a.A[h0], A1 = a.A[h1];
        const float b0 = a.step_bias ? a.step_bias[h0] : 0.f, b1 = a.step_bias ? a.step_bias[h1] : 0.f;
        float raw[4];
        if (items > 0) load_steps(a, pl, h0, pl.c0, raw);
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            const int slot = n % kDtRing, in = u + 1 == nu ? i + 1 : i, next_u = u + 1 == nu ? 0 : 1;
            float next[4] = {};
            if (n + 1 < items) load_steps(a, pl, next_u ? h1 : h0, pl.c0 + in, next);
            float d[4], loc[4], suf[4], blk[4], before, after;
            decays(a, pl, pl.c0 + i, u ? A1 : A0, u ? b1 : b0, raw, d, loc, suf, blk);
            other_blocks(blk, &before, &after);
            if (n >= kDtRing && !(ok = warp_wait(&m.dt_empty[slot], (n / kDtRing - 1) & 1, max_spin))) break;
            Decay& o = dts[slot];
            *reinterpret_cast<float4*>(o.loc + 4 * lane) = make_float4(loc[0], loc[1], loc[2], loc[3]);
            *reinterpret_cast<float4*>(o.d + 4 * lane) = make_float4(d[0], d[1], d[2], d[3]);
            // To the end of the token's block, over the blocks between, over the blocks after.
            const float out[4] = {d[0] * ex2(suf[0]), d[1] * ex2(suf[1]), d[2] * ex2(suf[2]), d[3] * ex2(suf[3])};
            const int own = lane >> 3;
#pragma unroll
            for (int q = 1; q < 4; ++q) {
                const float f = ex2((own < 1 && q > 1 ? blk[1] : 0.f) + (own < 2 && q > 2 ? blk[2] : 0.f));
                if (own < q)
                    *reinterpret_cast<float4*>(o.off + 16 * q * (q - 1) + 4 * lane) =
                        make_float4(out[0] * f, out[1] * f, out[2] * f, out[3] * f);
            }
            const float rest = ex2(after);
            *reinterpret_cast<float4*>(o.w + 4 * lane) = make_float4(out[0] * rest, out[1] * rest, out[2] * rest, out[3] * rest);
            *reinterpret_cast<float4*>(o.start + 4 * lane) =
                make_float4(ex2(before + loc[0]), ex2(before + loc[1]), ex2(before + loc[2]), ex2(before + loc[3]));
            if (lane == 0) o.total = ex2(blk[0] + blk[1] + blk[2] + blk[3]);
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.dt_full[slot]);
#pragma unroll
            for (int k = 0; k < 4; ++k) raw[k] = next[k];
            i = in, u = next_u;
        }
    } else if (warp == kWork + 3) {
        // ------------------------------------------------------------ output slots
        if (lane == 0) {
            const bool gate = un.gate_vec != 0;
            int opened = 0;
            // Slot of the next item: its gate on the way, or just free.
            auto open_slot = [&](int i, int u) {
                uint64_t* bar = &m.slot_ready[opened & 1];
                if (gate) {
                    mbar_arrive_expect_tx(bar, kTile);
                    tma_load_4d(oslot(opened), &zmap, bar, pl.col0(un, u), pl.head(a, un, u), (pl.c0 + i) * kC, pl.b);
                } else {
                    mbar_arrive(bar);
                }
                ++opened;
            };
            for (int n = 0; n < L::kSlots && n < items && !hold; ++n) open_slot(n / nu, n % nu);
            for (int n = 0, i = 0, u = 0; n < items; ++n) {
                if (!(ok = mbar_wait(&m.y_staged[n & 1], (n >> 1) & 1, max_spin))) break;
                if (*const_cast<volatile int*>(&bad[u].any) != kNone)
                    put_nan(a, pl, un, u, (pl.c0 + i) * kC, i != by_rows ? oslot(n) : nullptr, bad + u);
                if (i != by_rows) {
                    tma_store_4d(&ymap, oslot(n), pl.col0(un, u), pl.head(a, un, u), (pl.c0 + i) * kC, pl.b);
                    tma_store_commit();
                    tma_store_wait_read<0>();
                }
                if (n + L::kSlots < items) open_slot((n + L::kSlots) / nu, (n + L::kSlots) % nu);
                if (++u == nu) u = 0, ++i;
            }
            // Every gate that was asked for lands before the CTA exits.
            for (int j = max(opened - 2, 0); j < opened; ++j)
                mbar_wait(&m.slot_ready[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
        }
    } else {
        // ------------------------------------------------------------ the items' steps
        // Group (item mod 2) of eight warps; a warp's TMEM lane quarter, half of the columns.
        const int grp = warp >> 3, q = warp & 3, g = (warp >> 2) & 1, row = 32 * q + lane;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        const int64_t head_state = (int64_t)a.S * a.P;
        const bool has_state = q < 2 * kT;
        const uint2* mask = reinterpret_cast<const uint2*>(base + L::kMask) + lane;   // [e / 2][lane]
        uint8_t* sb = base + L::kSb;
        const uint32_t ptm = tmem + lanes + kTmP + 64 * grp;
        // Byte offset of this row's 16-byte piece j (columns 8 j ..) in a swizzled tile.
        auto piece = [&](int j) { return (uint32_t)(row * 128 + ((j ^ (row & 7)) << 4)); };
        if (warp < 4)                          // pairs 2e, 2e + 1 up to the row's own token
            for (int e = warp; e < 16; e += 4)
                reinterpret_cast<uint32_t*>(base + L::kMask)[64 * (e >> 1) + 2 * lane + (e & 1)] =
                    2 * e < lane ? 0xFFFFFFFFu : (2 * e == lane ? 0xFFFFu : 0u);
        for (int b = g; b < 4; b += 2)         // blocks above the diagonal stay zero
            if (b > q) {
                const uint32_t z[16] = {};
                tmem_st16(ptm + 16 * b, z);
            }
        float Du[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int h = pl.head(a, un, min(u, nu - 1));
            Du[u] = a.D ? a.D[h] : 0.f;
            // The state before the first chunk (group u writes unit u's).
            if (!has_state || u >= nu || u != grp) continue;
            const int64_t bh = (int64_t)pl.b * a.H + h;
            const float* from = a.nseg > 1 ? a.seeds + (bh * a.nseg + pl.seg) * head_state
                                           : (a.S0 ? a.S0 + bh * head_state : nullptr);
#pragma unroll 1
            for (int c = 0; c < 32; c += 16) {
                const int c0 = pl.col0(un, u) + 32 * g + c;
                uint32_t v[16];
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    const uint4 x = from && row < a.S && c0 + k < a.P
                                        ? *reinterpret_cast<const uint4*>(from + (int64_t)row * a.P + c0 + k)
                                        : make_uint4(0, 0, 0, 0);
                    v[k] = x.x, v[k + 1] = x.y, v[k + 2] = x.z, v[k + 3] = x.w;
                }
                tmem_st16(tmem + lanes + kTmSt + 64 * u + 32 * g + c, v);
            }
        }
        tmem_st_wait();
        named_bar(1, 32 * kWork);              // the mask table
        tc_fence_before();
        // An item is issued when its own group has prepared it and the other group has
        // taken the output of the item before (for the first item there is none).
        if (grp == 1 && lane == 0) mbar_arrive(&m.item_ready);
        for (int n = grp; n < items; n += 2) {
            const int slot = n % kDtRing, i = n / nu, u = n - i * nu, s1 = (n - 1) & 1, ph1 = ((n - 1) >> 1) & 1;
            const Decay& dc = dts[slot];
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kDtRing) & 1, max_spin))) break;
            // Scores to P first, except at a chunk's start, where (1) is still under way.
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                if ((pass == 0) == (u != 0)) {
                    // ------------------------------------------------ scores to P
                    if (!(ok = warp_wait(&m.sc_full[i & 1], (i >> 1) & 1, max_spin))) break;
                    tc_fence_after();
                    const float ci = dc.loc[row];
#pragma unroll 1
                    for (int b = g; b <= q; b += 2) {
                        uint32_t s[2][16], p[16];
                        tmem_ld16(tmem + lanes + kTmSc + 32 * b, s[0]);
                        tmem_ld16(tmem + lanes + kTmSc + 32 * b + 16, s[1]);
                        if (b < q) {
                            const float* col = dc.off + 16 * q * (q - 1) + 32 * b;
                            const float ri = ex2(ci);
                            const uint64_t r2 = pk2(ri, ri);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const ulonglong2 f = *reinterpret_cast<const ulonglong2*>(col + 2 * e);
                                const uint32_t* v = &s[e >> 3][2 * (e & 7)];
                                p[e] = pack2(mul2(mul2(pk2(__uint_as_float(v[0]), __uint_as_float(v[1])), f.x), r2));
                                p[e + 1] = pack2(mul2(mul2(pk2(__uint_as_float(v[2]), __uint_as_float(v[3])), f.y), r2));
                            }
                        } else {
                            // The diagonal block: an exponential per score; pairs past the row's
                            // own token are cleared as bits (their products may be anything).
                            const uint64_t c2 = pk2(ci, ci), minus = pk2(-1.f, -1.f);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(dc.loc + 32 * q + 2 * e);
                                const ulonglong2 d = *reinterpret_cast<const ulonglong2*>(dc.d + 32 * q + 2 * e);
                                const uint2 mk = mask[16 * e];   // 32 (e / 2)
                                const uint32_t* v = &s[e >> 3][2 * (e & 7)];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    float t0, t1;
                                    unpk2(fma2(k ? l.y : l.x, minus, c2), &t0, &t1);
                                    const uint64_t f = mul2(pk2(ex2(t0), ex2(t1)), k ? d.y : d.x);
                                    p[e + k] = pack2(mul2(f, pk2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])))) &
                                               (k ? mk.y : mk.x);
                                }
                            }
                        }
                        tmem_st16(ptm + 16 * b, p);
                    }
                    continue;
                }
                // ---------------------------------------------------- state: bf16 for (2), scaled for (4)
                // (2) of the item before has read the bf16 state; with two units it was issued
                // after (4) of this unit's last item, so that one is done as well.
                if (n > 0 && !(ok = warp_wait(&m.read_done[s1], ph1, max_spin) &&
                                    (nu == 2 || warp_wait(&m.state_done[s1], ph1, max_spin))))
                    break;
                if (has_state) {
                    tc_fence_after();
                    const float f = dc.total;
                    const uint64_t f2 = pk2(f, f);
#pragma unroll 1
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t at = tmem + lanes + kTmSt + 64 * u + 32 * g + 16 * c;
                        uint32_t v[16], h[8];
                        tmem_ld16(at, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint64_t x = pk2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                            h[e] = pack2(x);
                            float lo, hi;
                            unpk2(mul2(x, f2), &lo, &hi);
                            v[2 * e] = __float_as_uint(lo);
                            v[2 * e + 1] = __float_as_uint(hi);
                        }
                        tmem_st16(at, v);
                        if (row >= a.S)                    // padding rows never reach the read
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = 0u;
                        *reinterpret_cast<uint4*>(sb + piece(4 * g + 2 * c)) = make_uint4(h[0], h[1], h[2], h[3]);
                        *reinterpret_cast<uint4*>(sb + piece(4 * g + 2 * c + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
                    }
                }
                // ---------------------------------------------------- weighted values
                if (!(ok = warp_wait(&m.x_full[n & 1], (n >> 1) & 1, max_spin) &&
                           (n == 0 || warp_wait(&m.state_done[s1], ph1, max_spin))))
                    break;
                // Rows at or past a ragged end may hold anything: they are cleared in x, and in
                // B for (4). (1) may read such rows of B, whose scores no kept row uses.
                if (i == by_rows) {
                    if (!(ok = warp_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin))) break;
                    if ((pl.c0 + i) * kC + row >= pl.n)
                        for (int j = 4 * g; j < 4 * g + 4; ++j) {
                            *reinterpret_cast<uint4*>(xtile(n) + piece(j)) = make_uint4(0, 0, 0, 0);
                            for (int k = 0; k < kT; ++k)
                                *reinterpret_cast<uint4*>(btile(i & 1) + k * kTile + piece(j)) = make_uint4(0, 0, 0, 0);
                        }
                }
                const float w = dc.w[row];
                uint32_t bits = 0u;
#pragma unroll 1
                for (int j = 4 * g; j < 4 * g + 4; j += 2) {
                    const uint32_t o0 = piece(j), o1 = piece(j + 1);
                    uint8_t* hi = base + L::kXw;
                    uint32_t wh[8], wl[8], wr[8];
                    weigh16(*reinterpret_cast<const uint4*>(xtile(n) + o0), *reinterpret_cast<const uint4*>(xtile(n) + o1), w,
                            wh, wl, wr);
                    *reinterpret_cast<uint4*>(hi + o0) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
                    *reinterpret_cast<uint4*>(hi + o1) = make_uint4(wh[4], wh[5], wh[6], wh[7]);
                    *reinterpret_cast<uint4*>(hi + kTile + o0) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
                    *reinterpret_cast<uint4*>(hi + kTile + o1) = make_uint4(wl[4], wl[5], wl[6], wl[7]);
                    if constexpr (kTerms == 3) {
                        *reinterpret_cast<uint4*>(hi + 2 * kTile + o0) = make_uint4(wr[0], wr[1], wr[2], wr[3]);
                        *reinterpret_cast<uint4*>(hi + 2 * kTile + o1) = make_uint4(wr[4], wr[5], wr[6], wr[7]);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) bits |= wl[e];
                }
                // A value that is not finite leaves NaN as remainder. Others leave small ones: bits of
                // theirs together make up NaN's exponent only where one is 2 or more.
                if ((bits & 0x7F80u) == 0x7F80u || (bits & 0x7F800000u) == 0x7F800000u)
                    take_out(xtile(n), row, g, (pl.c0 + i) * kC + row, bad + u);
            }
            if (!ok) break;
            // What this warp stored is ready for the tensor cores.
            tmem_st_wait();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.item_ready);
            // -------------------------------------------------------- output
            const float Dh = u ? Du[1] : Du[0], e = dc.start[row];
            const uint64_t D2 = pk2(Dh, Dh), e2 = pk2(e, e);
            if (!(ok = warp_wait(&m.slot_ready[n & 1], (n >> 1) & 1, max_spin) &&
                       warp_wait(&m.y_full[n & 1], (n >> 1) & 1, max_spin)))
                break;
            tc_fence_after();
            if (kGated && un.gate_vec == 0) {
                put_gate(a, pl, un, u, (pl.c0 + i) * kC + row, 32 * g, oslot(n), piece(4 * g), piece(4 * g + 1));
                put_gate(a, pl, un, u, (pl.c0 + i) * kC + row, 32 * g + 16, oslot(n), piece(4 * g + 2), piece(4 * g + 3));
            }
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {                  // 16 columns at a time
                const uint32_t o0 = piece(4 * g + 2 * c), o1 = piece(4 * g + 2 * c + 1);
                const uint32_t ty = tmem + lanes + kTmY1 + 32 * g + 16 * c;
                uint32_t y1[16], y2[16];
                tmem_ld16(ty, y1);
                tmem_ld16(ty + (kTmY2 - kTmY1), y2);
                const uint4 xa = *reinterpret_cast<const uint4*>(xtile(n) + o0), xb = *reinterpret_cast<const uint4*>(xtile(n) + o1);
                const uint32_t xs[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
                uint64_t gt[8];
                if constexpr (kGated) {
                    const uint4 za = *reinterpret_cast<const uint4*>(oslot(n) + o0), zb = *reinterpret_cast<const uint4*>(oslot(n) + o1);
                    const uint32_t zs[8] = {za.x, za.y, za.z, za.w, zb.x, zb.y, zb.z, zb.w};
#pragma unroll
                    for (int f = 0; f < 8; ++f) gt[f] = gate2(zs[f]);
                }
                tmem_ld_wait();
                if (c == 1) {
                    // Y and x are free: the next item may be issued, the tile after it loaded.
                    tc_fence_before();
                    arrived(xa.x, xb.x);
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&m.item_ready);
                        mbar_arrive(&m.x_empty[n & 1]);
                        mbar_arrive(&m.dt_empty[slot]);
                    }
                }
                uint32_t o[8];
#pragma unroll
                for (int f = 0; f < 8; ++f) {
                    uint64_t v = fma2(e2, pk2(__uint_as_float(y2[2 * f]), __uint_as_float(y2[2 * f + 1])),
                                      pk2(__uint_as_float(y1[2 * f]), __uint_as_float(y1[2 * f + 1])));
                    v = fma2(D2, bf2(xs[f]), v);
                    if constexpr (kGated) v = mul2(v, gt[f]);
                    o[f] = pack2(v);
                }
                const uint4 p0 = make_uint4(o[0], o[1], o[2], o[3]), p1 = make_uint4(o[4], o[5], o[6], o[7]);
                if (i != by_rows) {
                    *reinterpret_cast<uint4*>(oslot(n) + o0) = p0;
                    *reinterpret_cast<uint4*>(oslot(n) + o1) = p1;
                } else {
                    put_row(a, pl, un, u, (pl.c0 + i) * kC + row, 32 * g + 16 * c, p0, p1);
                }
            }
            fence_proxy_async_smem();                      // the store reads the slot
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.y_staged[n & 1]);
        }
        // The final state (group u writes unit u's).
        if (ok && last_seg && a.S_out && has_state && grp < nu) {
            if (items == 0 || (ok = warp_wait(&m.state_done[(items - 1) & 1], ((items - 1) >> 1) & 1, max_spin))) {
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                    const int c0 = pl.col0(un, grp) + 32 * g + c;
                    uint32_t v[16];
                    tmem_ld16(tmem + lanes + kTmSt + 64 * grp + 32 * g + c, v);
                    tmem_ld_wait();
                    float* to = a.S_out + ((int64_t)pl.b * a.H + pl.head(a, un, grp)) * head_state + (int64_t)row * a.P + c0;
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (row < a.S && c0 + k < a.P)
                            *reinterpret_cast<uint4*>(to + k) = make_uint4(v[k], v[k + 1], v[k + 2], v[k + 3]);
                }
            }
        }
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWork + 1) tmem_dealloc(tmem, 512);
}

// First pass over segments: end state from zero, sum over the segment of
// B_j (d_j e^{l(end) - l_j} x_j)^T, and the segment's total decay. Chunks run from
// the last to the first; the weights carry the sum of the chunks after them.
// The three terms of w x stand side by side along N, B^T [hi | lo | last], so that an item
// reads B once: 80 KB of operands (the main pass, which has no TMEM left for it, takes the
// terms one after another); D holds S state rows, 64 columns of each term.
// Warps: TMA, MMA, decays (two), then four weight groups of four: two items at a
// time, half of the columns each (one group per item left the pass waiting for
// its weights). Four items' values and two items' terms are in flight.
// What bounds it: shared memory. An item's 16 KB in by TMA (and 16 of B), 16 KB read and 48 KB
// written by the weight groups and 80 KB of operands are 1,400 cycles at 128 bytes each.
constexpr int kSumThreads = 640, kSumRing = 2, kSumX = 4, kSumW = 2, kSumN = 192;

struct SumMisc {
    uint64_t b_full[2], b_empty[2], x_full[kSumX], x_empty[kSumX], w_full[kSumW], w_empty[kSumW];
    uint64_t dt_full[kSumRing], dt_empty[kSumRing], drain;
    uint32_t tmem_slot;
};

template <int kT> struct SumSmem {
    static constexpr uint32_t kX = 2 * kT * kTile;
    static constexpr uint32_t kW = kX + kSumX * kTile;         // three tiles per item
    static constexpr uint32_t kDt = kW + kSumW * 3 * kTile;
    static constexpr uint32_t kMisc = kDt + kSumRing * kC * 4;
    static constexpr size_t kBytes = 1024 + kMisc + sizeof(SumMisc);
};
static_assert(SumSmem<2>::kBytes <= 227 * 1024, "first pass's shared memory");

template <int kT>
__global__ void __launch_bounds__(kSumThreads, 1)
scan_sums_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap bmap,
                 const __grid_constant__ ScanArgs a, const __grid_constant__ Units un, WsHeader* hdr) {
    using L = SumSmem<kT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    SumMisc& m = *reinterpret_cast<SumMisc*>(base + L::kMisc);
    float* wts = reinterpret_cast<float*>(base + L::kDt);
    auto btile = [&](int s) { return base + s * kT * kTile; };
    auto xtile = [&](int n) { return base + L::kX + n % kSumX * kTile; };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place pl = place(a, un);
    const int nu = pl.nu, items = pl.nc * nu, c_last = pl.c0 + pl.nc - 1;
    const int64_t head_state = (int64_t)a.S * a.P;

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(&m.b_full[s], 1);
            mbar_init(&m.b_empty[s], 1);
        }
        for (int s = 0; s < kSumX; ++s) {
            mbar_init(&m.x_full[s], 1);
            mbar_init(&m.x_empty[s], 8);
        }
        for (int s = 0; s < kSumW; ++s) {
            mbar_init(&m.w_full[s], 8);
            mbar_init(&m.w_empty[s], 1);
        }
        for (int s = 0; s < kSumRing; ++s) {
            mbar_init(&m.dt_full[s], 1);
            mbar_init(&m.dt_empty[s], 8);
        }
        mbar_init(&m.drain, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&m.tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
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
                if (i + 2 < pl.nc)                         // to L2 ahead of its load
#pragma unroll
                    for (int k = 0; k < kT; ++k) tma_prefetch_4d(&bmap, 64 * k, pl.g, t - 2 * kC, pl.b);
                for (int u = 0; u < nu; ++u, ++n) {
                    if (i + 3 < pl.nc)
                        tma_prefetch_4d(&xmap, pl.col0(un, u), pl.head(a, un, u), t - 3 * kC, pl.b);
                    uint64_t* full = &m.x_full[n % kSumX];
                    if (n >= kSumX && !(ok = mbar_wait(&m.x_empty[n % kSumX], (n / kSumX - 1) & 1, max_spin))) break;
                    mbar_arrive_expect_tx(full, kTile);
                    tma_load_4d(xtile(n), &xmap, full, pl.col0(un, u), pl.head(a, un, u), t, pl.b);
                }
            }
            for (int j = max(i - 2, 0); j < i; ++j) mbar_wait(&m.b_full[j & 1], (j >> 1) & 1, kDefaultMaxSpin);
            for (int j = max(n - kSumX, 0); j < n; ++j)
                mbar_wait(&m.x_full[j % kSumX], (j / kSumX) & 1, kDefaultMaxSpin);
        }
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16_f32(128, kSumN, true, true);
        const uint32_t base_a = smem_u32(base);
        const uint64_t br0 = rows_desc(base_a), w0 = rows_desc(base_a + L::kW);
        for (int n = 0, i = 0, u = 0; n < items; ++n) {
            if (!(ok = warp_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin) &&
                       warp_wait(&m.w_full[n % kSumW], (n / kSumW) & 1, max_spin)))
                break;
            tc_fence_after();
            if (lane == 0) {
                // (For kT = 1 the second 64-row atom of B^T is whatever tile follows: unused lanes.)
                const uint64_t bt = step_desc(br0, (i & 1) * kT * kTile), w = step_desc(w0, n % kSumW * 3 * kTile);
#pragma unroll
                for (int k = 0; k < kC / 16; ++k)
                    mma_bf16(tmem + kSumN * u, step_desc(bt, k * 2048), step_desc(w, k * 2048), id, i > 0 || k > 0);
                mma_commit(&m.w_empty[n % kSumW]);
                if (u == nu - 1) mma_commit(&m.b_empty[i & 1]);
            }
            __syncwarp();
            if (++u == nu) u = 0, ++i;
        }
        if (lane == 0) {
            mma_commit(&m.drain);
            ok = mbar_wait(&m.drain, 0, kDefaultMaxSpin) && ok;
        }
        __syncwarp();
    } else if (warp < 4) {
        const int u = warp - 2;
        if (u < nu) {
            const int h = pl.head(a, un, u);
            const float A = a.A[h], bias = a.step_bias ? a.step_bias[h] : 0.f;
            float raw[4] = {}, after = 0.f;            // after: sum over the chunks behind
            if (pl.nc > 0) load_steps(a, pl, h, c_last, raw);
            for (int i = 0; i < pl.nc; ++i) {
                const int n = i * nu + u, slot = n % kSumRing;
                float next[4] = {};
                if (i + 1 < pl.nc) load_steps(a, pl, h, c_last - i - 1, next);
                float d[4], loc[4], suf[4], blk[4], before, rest;
                decays(a, pl, c_last - i, A, bias, raw, d, loc, suf, blk);
                other_blocks(blk, &before, &rest);
                if (n >= kSumRing && !(ok = warp_wait(&m.dt_empty[slot], (n / kSumRing - 1) & 1, max_spin))) break;
                rest += after;
                *reinterpret_cast<float4*>(wts + slot * kC + 4 * lane) =
                    make_float4(d[0] * ex2(suf[0] + rest), d[1] * ex2(suf[1] + rest),
                                d[2] * ex2(suf[2] + rest), d[3] * ex2(suf[3] + rest));
                after += blk[0] + blk[1] + blk[2] + blk[3];
                __syncwarp();
                if (lane == 0) mbar_arrive(&m.dt_full[slot]);
#pragma unroll
                for (int k = 0; k < 4; ++k) raw[k] = next[k];
            }
            if (lane == 0 && pl.col0(un, u) == 0)
                a.seg_decay[((int64_t)pl.b * a.H + h) * a.nseg + pl.seg] = after * kLn2;
        }
    } else {
        const int grp = (warp - 4) >> 2, half = grp >> 1;
        for (int n = grp & 1; n < items; n += 2) {
            const int slot = n % kSumRing, i = n / nu, u = n - i * nu;
            if (!(ok = warp_wait(&m.dt_full[slot], (n / kSumRing) & 1, max_spin) &&
                       warp_wait(&m.x_full[n % kSumX], (n / kSumX) & 1, max_spin) &&
                       (n < kSumW || warp_wait(&m.w_empty[n % kSumW], (n / kSumW - 1) & 1, max_spin))))
                break;
            if (a.lengths && (c_last - i + 1) * kC > pl.n) {
                if (!(ok = warp_wait(&m.b_full[i & 1], (i >> 1) & 1, max_spin))) break;
                if ((c_last - i) * kC + row >= pl.n) {     // both halves write the same zeros
                    zero_row(xtile(n), row);
                    for (int k = 0; k < kT && u == 0; ++k) zero_row(btile(i & 1) + k * kTile, row);
                }
            }
            uint8_t* const terms = base + L::kW + n % kSumW * 3 * kTile;
#pragma unroll
            for (int j = 4 * half; j < 4 * half + 4; j += 2) {
                const uint32_t o0 = row * 128 + ((j ^ (row & 7)) << 4), o1 = row * 128 + (((j + 1) ^ (row & 7)) << 4);
                uint32_t t[3][8];
                weigh16(*reinterpret_cast<const uint4*>(xtile(n) + o0), *reinterpret_cast<const uint4*>(xtile(n) + o1),
                        wts[slot * kC + row], t[0], t[1], t[2]);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    *reinterpret_cast<uint4*>(terms + k * kTile + o0) = make_uint4(t[k][0], t[k][1], t[k][2], t[k][3]);
                    *reinterpret_cast<uint4*>(terms + k * kTile + o1) = make_uint4(t[k][4], t[k][5], t[k][6], t[k][7]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&m.w_full[n % kSumW]);
                mbar_arrive(&m.x_empty[n % kSumX]);
                mbar_arrive(&m.dt_empty[slot]);
            }
        }
        // The state of unit u, the sum of the three terms: a thread has a state row, a group
        // sixteen of its columns.
        ok = pl.nc == 0 || (ok && warp_wait(&m.drain, 0, max_spin));
        if (ok) {
            tc_fence_after();
            const uint32_t at = tmem + ((uint32_t)(32 * q) << 16) + 16 * grp;
            for (int u = 0; u < nu && q < 2 * kT; ++u) {
                const int64_t bh = (int64_t)pl.b * a.H + pl.head(a, un, u);
                const int p0 = pl.col0(un, u) + 16 * grp;
                float* to = a.seeds + (bh * a.nseg + pl.seg) * head_state + (int64_t)row * a.P + p0;
                uint32_t v[3][16];
#pragma unroll
                for (int k = 0; k < 3; ++k) tmem_ld16(at + kSumN * u + 64 * k, v[k]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    float f[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        f[k] = pl.nc == 0 ? 0.f
                                          : __uint_as_float(v[0][c + k]) +
                                                (__uint_as_float(v[1][c + k]) + __uint_as_float(v[2][c + k]));
                    if (row < a.S && p0 + c < a.P) *reinterpret_cast<float4*>(to + c) = make_float4(f[0], f[1], f[2], f[3]);
                }
            }
        }
    }
    if (!ok) report_timeout(hdr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
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

Units units_of(int H, int G, int P, int per) {
    Units un = {};
    un.blocks = (P + 63) / 64;
    un.units = (G > 0 ? H / G : H) * un.blocks;
    un.per = per;
    un.ctas = (un.units + per - 1) / per;
    return un;
}

// How the work is cut: two units per CTA share (1) and the loads of B and C, one
// spreads few heads over more SMs; segments spread long sequences. CTAs run in
// waves over the SMs, so the cut is the one whose waves times chunks is least. In
// units of one chunk of two units (about 5 us): a chunk of one unit 0.65, starting
// and ending a CTA 1.3, the first pass 0.35 per chunk, and with segments two
// further launches and the chaining 1 + 0.1 per segment.
struct Cut {
    int per, nseg;
};
Cut pick_cut(int64_t groups, int units, int N) {
    const int nch = (N + kC - 1) / kC, sms = sm_count();
    Cut best = {2, 1};
    double least = 1e30;
    for (int per = 2; per >= 1; --per) {
        const int64_t ctas = groups * ((units + per - 1) / per);
        const double chunk = per == 2 && units > 1 ? 1.0 : 0.65;
        for (int n = 1; n <= 64 && n <= nch; ++n) {
            const int cps = (nch + n - 1) / n;
            if ((nch + cps - 1) / cps != n) continue;      // the same split with empty segments
            const double waves = (double)((ctas * n + sms - 1) / sms);
            const double cost = waves * (cps * chunk + 1.3) +
                                (n > 1 ? waves * (0.35 * cps * chunk + 1.0) + 1.0 + 0.1 * n : 0.0);
            if (cost < least) least = cost, best = {per, n};
        }
    }
    return best;
}

template <int kT, int kTerms, bool kGated>
cudaError_t launch_main(const CUtensorMap& xm, const CUtensorMap& bm, const CUtensorMap& cm, const CUtensorMap& zm,
                        const CUtensorMap& ym, const ScanArgs& a, const Units& un, dim3 grid, WsHeader* hdr,
                        cudaStream_t st) {
    static std::atomic<int> optin[kMaxDevices];
    constexpr size_t bytes = Smem<kT, kTerms>::kBytes;
    const cudaError_t e = ensure_smem_optin(scan_tc_kernel<kT, kTerms, kGated>, (int)bytes, optin);
    if (e != cudaSuccess) return e;
    return launch_after(scan_tc_kernel<kT, kTerms, kGated>, grid, kThreads, bytes, st, a.nseg > 1, xm, bm, cm, zm, ym, a, un,
                        hdr);
}

// The state that a call returns is summed in three terms: by the first pass and the chaining
// where there are segments (the main pass's state serves its outputs alone then), else by the
// main pass.
template <int kT, bool kGated>
cudaError_t launch(const CUtensorMap& xm, const CUtensorMap& bm, const CUtensorMap& cm, const CUtensorMap& zm,
                   const CUtensorMap& ym, ScanArgs a, const Units& un, int B, WsHeader* hdr, cudaStream_t st) {
    const dim3 grid(un.ctas * a.G, a.nseg, B);
    if (a.nseg > 1) {
        static std::atomic<int> optin[kMaxDevices];
        cudaError_t e = ensure_smem_optin(scan_sums_kernel<kT>, (int)SumSmem<kT>::kBytes, optin);
        if (e != cudaSuccess) return e;
        scan_sums_kernel<kT><<<grid, kSumThreads, SumSmem<kT>::kBytes, st>>>(xm, bm, a, un, hdr);
        if ((e = cudaPeekAtLastError()) != cudaSuccess) return e;
        if ((e = launch_seeds(a, (int64_t)B * a.H, st)) != cudaSuccess) return e;
        a.S_out = nullptr;
    }
    return a.S_out ? launch_main<kT, 3, kGated>(xm, bm, cm, zm, ym, a, un, grid, hdr, st)
                   : launch_main<kT, 2, kGated>(xm, bm, cm, zm, ym, a, un, grid, hdr, st);
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
    return pick_cut(B * G, units_of(H, G, P, 1).units, N).nseg;
}

cudaError_t tc_scan(ScanArgs& a, int B, void* ws_header, cudaStream_t st) {
    Units un = units_of(a.H, a.G, a.P, 1);
    un = units_of(a.H, a.G, a.P, pick_cut((int64_t)B * a.G, un.units, a.N).per);
    const int nch = (a.N + kC - 1) / kC;
    un.cps = (nch + a.nseg - 1) / a.nseg;
    un.gate_vec = a.z && (reinterpret_cast<uintptr_t>(a.z) & 15) == 0 &&
                  (a.N == 1 || (a.z_ts > 0 && a.z_ts % 8 == 0)) && (B == 1 || (a.z_bs > 0 && a.z_bs % 8 == 0)) &&
                  a.z_ts < (int64_t)1 << 38 && a.z_bs < (int64_t)1 << 38;
    CUtensorMap xm, bm, cm, zm, ym;
    if (!encode_rows(&xm, a.x, a.P, a.H, a.N, B, a.x_ts, a.x_bs) ||
        !encode_rows(&bm, a.Bm, a.S, a.G, a.N, B, a.b_ts, a.b_bs) ||
        !encode_rows(&cm, a.Cm, a.S, a.G, a.N, B, a.c_ts, a.c_bs) ||
        !encode_rows(&ym, a.y, a.P, a.H, a.N, B, a.y_ts, a.y_bs))
        return cudaErrorInvalidValue;
    zm = xm;                                               // unused without an aligned gate
    if (un.gate_vec && !encode_rows(&zm, a.z, a.P, a.H, a.N, B, a.z_ts, a.z_bs)) return cudaErrorInvalidValue;
    WsHeader* hdr = static_cast<WsHeader*>(ws_header);
    if (a.S <= 64)
        return a.z ? launch<1, true>(xm, bm, cm, zm, ym, a, un, B, hdr, st)
                   : launch<1, false>(xm, bm, cm, zm, ym, a, un, B, hdr, st);
    return a.z ? launch<2, true>(xm, bm, cm, zm, ym, a, un, B, hdr, st)
               : launch<2, false>(xm, bm, cm, zm, ym, a, un, B, hdr, st);
}

}  // namespace scan

}  // namespace la
