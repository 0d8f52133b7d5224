// prefill_scaled.cu -- causal chunked-prefill attention over 8-bit pools with
// a scale for each (block, kv head), on tcgen05 tensor cores.
//
// With K_j = ks_b c_j and V_j = vs_b d_j (codes c, d; b the block of key j),
//     s_j = (scale log2 e ks_b) (q . c_j),  out = sum_j 2^(s_j) vs_b d_j / sum_j 2^(s_j).
// Codes are exact in fp16, so both products take fp16 operands: K and V tiles
// are widened once per CTA, for two q heads of 128 rows each, and the scales
// only touch scores and weights.
//
//  * A CTA owns 128 query rows of the two q heads of a GQA group ("units"; one
//    unit when Hq/Hkv is odd, or for the split tiles of find_prefill_tile).
//    Warp 16 loads Q and the key tiles' codes (128 keys = 8 paged blocks, each
//    one TMA box), warp 17 issues tcgen05.mma, warps 0-7 and 8-15 run the
//    softmax of units 0 and 1, two per quarter of tensor memory's lanes, 16
//    rows each.
//  * Warps 0-15 widen a sixteenth of each K and V tile, from unswizzled codes to
//    the 128-byte swizzled panels the MMAs read, in the time they would wait
//    for scores; the codes' buffers are refilled a tile ahead.  Rows past the
//    last visible key become zero (0 times a NaN code would be NaN).
//  * q goes to fp16 once, each row scaled by a power of two so that its largest
//    value is in [2^14, 2^15); the scores take the factor back.
//  * The running maximum is that of y_j = s_j + log2 vs_b; P = 2^(y_j - m + 12) is
//    the weight with its V scale, in two fp16 terms (the rounded value and what
//    the rounding lost: 2^-22, where one term would be 2^-11), which take exactly
//    the columns of the scores they replace; the row sum adds 2^-9 P / vs_b block
//    by block.  m moves, and O is rescaled, when the maximum grows by more than 2^3:
//    P stays below 2^15, and weights end 2^-36 below the largest.  A key of a
//    small V scale may count for nothing in O and for all in the sum (16 rows of
//    zeros, whose scale is 2^-100, beside one of scale 2^40: v / 17), so from the
//    tile on where the V scales are more than 2^104 apart a pass of its own sums
//    2^(s_j - m + 3), each the square of an exponential of half that, which fp32
//    holds for every scale; sums move to other references in two such halves.
//  * A NaN code in V (the append stores one for a NaN) would reach, as 0 times
//    NaN, the rows of its tile that do not see it.  So in tiles that not all rows
//    see NaN codes are widened to zeros, each dim keeps the first of the CTA's rows
//    that sees one, and from that row on its output is set to NaN after the store.
//  * Measured: 2,048 of 16,384 tokens, 16/8 x 128, 458 us, 563 TFLOP/s (the two
//    terms of P make it 844 of the tensor cores' work); 300 tokens, 32/8 x 64,
//    12.6 us.  A tile of two heads takes some 7,000 cycles, 3,300 of MMAs; issue
//    slots are 48 % busy, the ALU 39 %: what bounds it is each warp's chain
//    through a tile, wait, scores, shuffles, exponentials, stores, with four
//    warps on a scheduler.  Steps of 64 keys with two sets of scores, the MMAs
//    of one beside the softmax of the other, pay that chain's fixed part twice:
//    558 us (300 tokens: 11.2).
//  * Every wait is bounded; copies and MMAs have ended and tensor memory is freed
//    on every exit path.
#include <cfloat>
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "prefill_tile.cuh"
#include "scaled_device.cuh"
#include "tcgen05_rows.cuh"

namespace pkv {
namespace {

constexpr int kTileM = kPrefillRows;
constexpr int kTileN = 128;                          // keys per key tile
constexpr int kUnits = 2;                            // q heads per CTA (max)
constexpr int kBlocksPerTile = kTileN / kBlockSize;  // 8
constexpr int kPanelBytes = 128 * 128;               // 128 rows x 64 fp16, swizzled
constexpr int kTileBytes = 2 * kPanelBytes;
constexpr int kCodeBytes = kTileN * 128;             // a tile's codes at head_dim 128

constexpr int OFF_Q = 0;                             // kUnits Q tiles
constexpr int OFF_K = OFF_Q + kUnits * kTileBytes;   // 2 widened K tiles
constexpr int OFF_V = OFF_K + 2 * kTileBytes;        // 2 widened V tiles
constexpr int OFF_KC = OFF_V + 2 * kTileBytes;       // codes of one K tile
constexpr int OFF_VC = OFF_KC + kCodeBytes;          // codes of one V tile
constexpr int kScaleTiles = 3;                       // tiles whose scales are kept
constexpr int OFF_SCALES = OFF_VC + kCodeBytes;      // [kScaleTiles][8 blocks] TileScales
constexpr int OFF_ROWF = OFF_SCALES + kScaleTiles * kBlocksPerTile * 24;  // [kUnits][128] factor of a row's scores
constexpr int OFF_BAR = OFF_ROWF + kUnits * kTileM * 4;
constexpr int NBAR = 21;
constexpr int OFF_INFO = OFF_BAR + NBAR * 8;
constexpr int OFF_NANS = OFF_INFO + 12 * 4;          // [D] first row that sees a NaN of V, 255: none
constexpr int OFF_TMEM = OFF_NANS + 128;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;     // slack to align the base to 1024 B
static_assert(SMEM_BYTES <= 232448, "shared memory budget (227 KB)");
static_assert(2 * SMEM_BYTES > 228 * 1024, "the 512-column TMEM allocation needs one CTA per SM");

constexpr int kSoftmaxWarps = 8;                     // per unit
constexpr int kLoadWarp = 16, kMmaWarp = 17;
constexpr int kThreads = 32 * 18;
constexpr int kWidenWarps = kSoftmaxWarps * kUnits;  // all of them, whatever the units

constexpr uint32_t kTmemCols = 512;
// Unit u: S and then P (hi, lo) at columns [256u, 256u + 128), O at + 128.
__host__ __device__ constexpr uint32_t col_s(int u) { return static_cast<uint32_t>(u) * 256u; }
__host__ __device__ constexpr uint32_t col_o(int u) { return static_cast<uint32_t>(u) * 256u + 128u; }

// Key tiles that O stays in tensor memory for.  The tensor cores' sums lose half
// a unit in the last place on average at each of a tile's 16 steps, always to
// the same side: 2.5e-6 of the output's norm after 12 tiles, 3.5e-5 after 128.
// Every kKeep tiles O is added, with rounding, to what was moved out before.
constexpr int kKeep = 3;
constexpr float kThreshold = 3.0f, kShift = 12.0f;   // log2 units
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
    const float2* scales;   // [num_blocks][hkv]
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* qsl;
    float* out;
    unsigned long long* err;
    int32_t num_blocks, hkv, hq, num_seqs, num_tokens, max_blocks, ctx_cap, units, split_last;
    int32_t decode_launch;  // the call's decode rows have a launch of their own
    int32_t stall;          // test hook: the MMA warp issues nothing
    float scale_log2;
};

// A block's scales as the softmax takes them, V's twice: operands of packed
// arithmetic.  inv_v: 2^-kSumShift / vs, or zero, and wide not zero, where the V
// scales of the tiles up to this one are more than 2^kWideSpread apart or one is
// 2^(kWideTop + 1) or more: the row sums then come from wide_sums.
struct __align__(8) TileScales {
    float2 log2_v, inv_v;
    float k, wide;
};
// A key whose P = 2^(y - m + 12) is flushed to zero (below 2^-126; m is at most
// the largest s plus the largest log2 vs) weighs less than 2^-(138 - spread) of
// the largest 2^s: 2^-34 here, as little as what two fp16 terms drop.
constexpr int kWideSpread = 104;
// The sums' terms are 2^(s - m + 12 - kSumShift), and m is at least s + log2 vs -
// 3: below 2^107 at the least scale, so that rows of 2^21 keys fit fp32 (without
// the shift 2^13 zero rows would end beyond it).  The largest is at least 2^(2 -
// 122), and inv_v is a normal number.
constexpr int kSumShift = 9, kWideTop = 100;

enum {
    B_QFULL = 0,
    B_QCONV = 1,   // Q in fp16 (8 warps per unit)
    B_KCFULL = 2,  // codes of a K tile and the tile's scales
    B_KCEMPTY = 3, // widened (16 warps)
    B_VCFULL = 4,
    B_VCEMPTY = 5,
    B_KCONV = 6,   // + stage: K tile widened (16 warps)
    B_KEMPTY = 8,  // + stage: read by the MMAs
    B_VCONV = 10,  // + stage
    B_VEMPTY = 12, // + stage
    B_SFULL = 14,  // + unit
    B_PFULL = 16,  // + unit (8 warps)
    B_ODONE = 18,  // + unit
    B_LAST = 20,   // every MMA issued
};

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A pair of weights (below 2^15) as two fp16 pairs: the first 11 bits, and the
// rest rounded, 2^-22 of the weight (2^-25 below 2^-14).
__device__ __forceinline__ void split2(float2 p, uint32_t& hi, uint32_t& lo) {
    const float2 h = make_float2(__uint_as_float(__float_as_uint(p.x) & 0xffffe000u),
                                 __uint_as_float(__float_as_uint(p.y) & 0xffffe000u));
    hi = tc::pack_f16x2(h.x, h.y);
    const float2 r = __ffma2_rn(h, make_float2(-1.f, -1.f), p);
    lo = tc::pack_f16x2(r.x, r.y);
}

// Four codes to two fp16 pairs, exactly.  int8: code + 128 as the low byte of
// 0x6400 is 1024 + 128 + code, less 1152.
template <int KIND>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (KIND == kKindInt8Blocks) {
        w ^= 0x80808080u;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(a) : "r"(__byte_perm(w, 0x64646464u, 0x4140)), "r"(0x64806480u));
        asm("sub.f16x2 %0, %1, %2;" : "=r"(b) : "r"(__byte_perm(w, 0x64646464u, 0x4342)), "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(a), "=r"(b)
            : "r"(w));
    }
}

// Where 16 codes of V have NaNs: zeros in place of their fp16 values, at chunks at0
// and at1 of a panel; first_row[dim], of four dims a word, becomes `row` for those
// dims unless it is smaller.
__device__ __noinline__ void take_nans(uint32_t codes, uint32_t at0, uint32_t at1, uint32_t* first_row, int row) {
    uint32_t x[4], h[4];
    tc::lds128(codes, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t nan = __vcmpeq4(x[i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (i % 2 == 0) tc::lds128(i ? at1 : at0, h);
        h[2 * (i % 2)] &= ~__byte_perm(nan, 0u, 0x1100);
        h[2 * (i % 2) + 1] &= ~__byte_perm(nan, 0u, 0x3322);
        if (i % 2) tc::sts128(i > 1 ? at1 : at0, h[0], h[1], h[2], h[3]);
        if (nan == 0) continue;
        const uint32_t from = (0x01010101u * static_cast<uint32_t>(row)) | ~nan;
        for (uint32_t was = first_row[i], now; (now = __vminu4(was, from)) != was;) {
            const uint32_t found = atomicCAS(first_row + i, was, now);
            if (found == was) break;
            was = found;
        }
    }
}

// NaN over the elements of a row, columns col + 8 i and one on, that see one.
__device__ __noinline__ void store_nans(float* out, const uint8_t* first_row, int row, int col, int dims) {
    for (; col < dims; col += 8)
        for (int i = 0; i < 2; ++i)
            if (row >= first_row[col + i]) out[col + i] = NAN;
}

// A warp's eighth rows of a tile, codes [128][D] to fp16 panels; rows >= nrows
// become zero.  Lane l takes 16 codes of row 8 warp + 2 (l / 8) + (l / 4) % 2:
// at head_dim 128 neighbouring rows take different halves of their chunks, so
// that neither the eight lanes that load nor those that store together meet in
// a bank.  NANS: NaN codes become zero (take_nans), rows of the CTA from r -
// sees_all on see row r of the tile.
template <int D, int KIND, bool NANS>
__device__ __forceinline__ void widen_rows(uint32_t codes, uint32_t tile, int warp, int lane, int nrows,
                                           uint32_t* first_row = nullptr, int sees_all = 0) {
    constexpr int PASSES = D / 64;
    const int rr = (lane >> 2) & 1, row = 8 * warp + 2 * (lane >> 3) + rr;
    uint32_t x[PASSES][4];
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int c = PASSES == 2 ? (lane & 3) + 4 * (rr ^ s) : lane & 3;
        tc::lds128(codes + row * D + c * 16, x[s]);
    }
    uint32_t nan = 0;
#pragma unroll
    for (int s = 0; s < PASSES; ++s) {
        const int c = PASSES == 2 ? (lane & 3) + 4 * (rr ^ s) : lane & 3;
        if (row >= nrows) x[s][0] = x[s][1] = x[s][2] = x[s][3] = 0u;
        if constexpr (NANS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= (x[s][i] & 0x7f7f7f7fu) + 0x01010101u;
        }
        const uint32_t at = tile + (c >> 2) * kPanelBytes + row * 128;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h[4];
            widen4<KIND>(x[s][2 * i], h[0], h[1]);
            widen4<KIND>(x[s][2 * i + 1], h[2], h[3]);
            tc::sts128(at + (((2 * (c & 3) + i) ^ (row & 7)) << 4), h[0], h[1], h[2], h[3]);
        }
    }
    if (NANS && (nan & 0x80808080u)) {
#pragma unroll
        for (int s = 0; s < PASSES; ++s) {
            const int c = PASSES == 2 ? (lane & 3) + 4 * (rr ^ s) : lane & 3;
            const uint32_t at = tile + (c >> 2) * kPanelBytes + row * 128;
            take_nans(codes + row * D + c * 16, at + (((2 * (c & 3)) ^ (row & 7)) << 4),
                      at + (((2 * (c & 3) + 1) ^ (row & 7)) << 4), first_row + 4 * c,
                      max(row - sees_all, 0));
        }
    }
}

// The same for a tile of V that may hold NaN codes and that not all rows see: the
// last one or two of a CTA's, out of line.
template <int D, int KIND>
__device__ __noinline__ void widen_last_v(uint32_t codes, uint32_t tile, int warp, int lane, int nrows,
                                          uint32_t* first_row, int sees_all) {
    widen_rows<D, KIND, true>(codes, tile, warp, lane, nrows, first_row, sees_all);
}

// A block's factor of a row's scores, never so small that it would turn what
// was masked into a NaN.
__device__ __forceinline__ float block_factor(float f, float ks) { return fmaxf(f * ks, FLT_MIN); }

// This thread's part of the sums of 2^(s + sh) over a tile's keys for its rows
// a and b (see the softmax rows), whose scores are at ts.
__device__ __noinline__ float2 wide_sums(uint32_t ts, const TileScales* sct, float fa, float fb, float sha, float shb,
                                         int key0, int pos_a, int pos_b) {
    float la = 0.f, lb = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t s[16];
        tc::tmem_ld16x256b_x4(ts + 32 * c, s);
        tc::tmem_wait_ld(s);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const bool row_b = i & 2;
            const float ks = sct[2 * c + i / 8].k;
            const float y = __uint_as_float(s[i]) * block_factor(row_b ? fb : fa, ks);
            const float t = fast_exp2(0.5f * (y + (row_b ? shb : sha)));
            const bool sees = key0 + 32 * c + 8 * (i / 4) + (i & 1) <= (row_b ? pos_b : pos_a);
            if (row_b) lb = sees ? fmaf(t, t, lb) : lb;
            else la = sees ? fmaf(t, t, la) : la;
        }
    }
    return make_float2(la, lb);
}

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_scaled_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const Params P) {
    constexpr int kPanels = D / 64;  // 64-dim swizzled panels of a tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    PrefillTile* info = reinterpret_cast<PrefillTile*>(smem + OFF_INFO);
    uint8_t* first_row = smem + OFF_NANS;
    constexpr bool kNans = KIND != kKindInt8Blocks;
    static_assert(sizeof(PrefillTile) <= 12 * 4, "info");
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);
    float* rowf = reinterpret_cast<float*>(smem + OFF_ROWF);
    TileScales* scales = reinterpret_cast<TileScales*>(smem + OFF_SCALES);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    const unsigned FULL = 0xffffffffu;

    griddep_launch_dependents();
    if (warp == 0) {
        griddep_wait();
        const PrefillTile t = find_prefill_tile(P.qsl, P.context_lens, P.num_seqs, P.num_tokens, P.ctx_cap, P.units,
                                                P.split_last, blockIdx.x, blockIdx.y, P.err, lane);
        if (lane == 0) *info = t;
        if (kNans) reinterpret_cast<uint32_t*>(first_row)[lane] = 0xffffffffu;
    }
    if (warp == 1 && blockIdx.x == 0 && blockIdx.y == 0) {
        griddep_wait();
        report_unplanned_rows(P.qsl, P.num_seqs, P.split_last, gridDim.x, P.decode_launch, P.err, lane);
    }
    if (threadIdx.x == 32 * kMmaWarp) {
        for (int i = 0; i < NBAR; ++i) {
            const bool widened = i == B_KCEMPTY || i == B_VCEMPTY || (i >= B_KCONV && i < B_KEMPTY) ||
                                 (i >= B_VCONV && i < B_VEMPTY) || i == B_QCONV;
            const bool rows = i >= B_PFULL && i < B_ODONE;
            mbar_init(&bar[i], widened ? kWidenWarps : rows ? kSoftmaxWarps : 1);
        }
        fence_mbar_init();
    }
    if (warp == kLoadWarp) {
        tc::tmem_alloc(tmem_slot, kTmemCols);
        tc::tmem_relinquish();
        if (lane == 0) {
            tc::prefetch_tensormap(&tm_q);
            tc::prefetch_tensormap(&tm_k);
            tc::prefetch_tensormap(&tm_v);
        }
    }
    griddep_wait();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const PrefillTile T = *info;
    const int nt = T.nt, units = T.units;
    const int g = T.h0 / (P.hq / P.hkv);                           // the kv head both units read
    const int nblk = (T.pmax + 1 + kBlockSize - 1) / kBlockSize;   // blocks holding keys 0..pmax
    bool ok = true;

    if (warp == kLoadWarp && nt > 0) {
        // ------------------------------------------------------ TMA producer
        if (lane == 0) {
            mbar_arrive_expect_tx(&bar[B_QFULL], static_cast<uint32_t>(units) * kPanels * kPanelBytes);
            for (int u = 0; u < units; ++u) {
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn)
                    tc::tma_load_3d(smem + OFF_Q + u * kTileBytes + pn * kPanelBytes, &tm_q, 64 * pn, T.h0 + u, T.row0,
                                    &bar[B_QFULL]);
            }
        }
        const int32_t* trow = P.block_tables + static_cast<size_t>(T.s) * P.max_blocks;
        // A tile's table entries and scales are looked up while the tile
        // before it is on its way.
        int slab = 0;
        float ks = 1.f, log2_v = 0.f, inv_v = 1.f;
        int high = -1000, low = 1000;  // exponents of the V scales up to here
        auto look_up = [&](int j) {
            ks = 1.f, log2_v = 0.f, inv_v = 1.f;
            if (lane < min(kBlocksPerTile, nblk - j * kBlocksPerTile)) {
                int e = __ldg(trow + j * kBlocksPerTile + lane);
                bool bad = e < 0 || e >= P.num_blocks;
                if (bad) e = 0;  // never dereference an invalid id
                slab = e * P.hkv + g;
                const float2 s = __ldg(P.scales + slab);
                ks = checked_scale(s.x, bad);
                const float vs = checked_scale(s.y, bad);
                log2_v = log2f(vs);
                inv_v = 1.f / (1 << kSumShift) / vs;
                const int e2 = static_cast<int>(__float_as_uint(vs) >> 23) - 127;
                high = max(high, e2);
                low = min(low, e2);
                if (bad) record_error(P.err, kErrRange, static_cast<uint32_t>(T.s));
            }
        };
        look_up(0);
        int k_tiles = 0, v_tiles = 0;  // asked for
        for (int j = 0; j < nt && ok; ++j) {
            const int nvb = min(kBlocksPerTile, nblk - j * kBlocksPerTile);
            const uint32_t bytes = static_cast<uint32_t>(nvb) * kBlockSize * D;
            const int now = slab;
            if (!mbar_wait_warp(&bar[B_KCEMPTY], (j & 1) ^ 1)) { ok = false; break; }
            high = __reduce_max_sync(FULL, high);
            low = __reduce_min_sync(FULL, low);
            const bool wide = high - low > kWideSpread || high > kWideTop;
            // The tile three before this one has been through its softmax:
            // every warp widened the last K tile after that.
            if (lane < kBlocksPerTile)
                scales[j % kScaleTiles * kBlocksPerTile + lane] = {
                    make_float2(log2_v, log2_v), wide ? make_float2(0.f, 0.f) : make_float2(inv_v, inv_v), ks,
                    wide ? 1.f : 0.f};
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&bar[B_KCFULL], bytes);
            __syncwarp();
            if (lane < nvb)
                tc::tma_load_3d(smem + OFF_KC + lane * kBlockSize * D, &tm_k, 0, 0, now, &bar[B_KCFULL]);
            ++k_tiles;
            if (j + 1 < nt) look_up(j + 1);
            if (!mbar_wait_warp(&bar[B_VCEMPTY], (j & 1) ^ 1)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&bar[B_VCFULL], bytes);
            __syncwarp();
            if (lane < nvb)
                tc::tma_load_3d(smem + OFF_VC + lane * kBlockSize * D, &tm_v, 0, 0, now, &bar[B_VCFULL]);
            ++v_tiles;
            __syncwarp();
        }
        // Never leave with copies in flight, whatever became of the others.
        ok = mbar_wait_warp(&bar[B_QFULL], 0) && ok;
        if (k_tiles > 0) ok = mbar_wait_warp(&bar[B_KCFULL], (k_tiles - 1) & 1) && ok;
        if (v_tiles > 0) ok = mbar_wait_warp(&bar[B_VCFULL], (v_tiles - 1) & 1) && ok;
    } else if (warp == kMmaWarp && nt > 0 && !P.stall) {
        // ------------------------------------------------------ MMA issuer
        constexpr uint32_t kIdescQK = tc::idesc_f16_f32(kTileM, kTileN, 0, 0);
        constexpr uint32_t kIdescPV = tc::idesc_f16_f32(kTileM, D, 0, 1);
        auto qk = [&](int u, int j) {
            const uint32_t sq = smem_addr(smem + OFF_Q + u * kTileBytes);
            const uint32_t sk = smem_addr(smem + OFF_K + (j & 1) * kTileBytes);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t off = (k >> 2) * kPanelBytes + (k & 3) * 32;
                tc::mma_bf16_ss(tmem + col_s(u), tc::smem_desc_sw128(sq + off, 16, 1024),
                                tc::smem_desc_sw128(sk + off, 16, 1024), kIdescQK, k > 0 ? 1u : 0u);
            }
            tc::mma_commit(&bar[B_SFULL + u]);
        };
        // O_u += P_u V: key step k covers keys 16k .. 16k + 15.  The first terms
        // of 32 keys' P take the first 16 of the columns of their scores, the
        // second terms the other 16.
        auto pv = [&](int u, int j) {
            const uint32_t svb = smem_addr(smem + OFF_V + (j & 1) * kTileBytes);
#pragma unroll
            for (int k = 0; k < kTileN / 16; ++k) {
                const uint64_t vdesc = tc::smem_desc_sw128(svb + k * 2048, kPanelBytes, 1024);
                const uint32_t p = tmem + col_s(u) + 32 * (k / 2) + 8 * (k % 2);
                tc::mma_bf16_ts(tmem + col_o(u), p + 16, vdesc, kIdescPV, (j % kKeep > 0 || k > 0) ? 1u : 0u);
                tc::mma_bf16_ts(tmem + col_o(u), p, vdesc, kIdescPV, 1u);
            }
            tc::mma_commit(&bar[B_ODONE + u]);
        };
        ok = mbar_wait_warp(&bar[B_QCONV], 0) && mbar_wait_warp(&bar[B_KCONV], 0);
        if (ok) {
            tc::fence_after_sync();
            if (tc::elect_one()) {
                for (int u = 0; u < units; ++u) qk(u, 0);
                tc::mma_commit(&bar[B_KEMPTY]);
            }
            __syncwarp();
        }
        // Per tile, unit by unit: P_u V, then (once P_u has been read) the
        // next tile's S_u, so that one unit's softmax runs beside the other's
        // MMAs.
        for (int j = 0; j < nt && ok; ++j) {
            if (!mbar_wait_warp(&bar[B_VCONV + (j & 1)], (j >> 1) & 1)) { ok = false; break; }
            const bool next = j + 1 < nt;
            if (next && !mbar_wait_warp(&bar[B_KCONV + ((j + 1) & 1)], ((j + 1) >> 1) & 1)) { ok = false; break; }
            for (int u = 0; u < units && ok; ++u) {
                if (!mbar_wait_warp(&bar[B_PFULL + u], j & 1)) { ok = false; break; }
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    pv(u, j);
                    if (u == units - 1) tc::mma_commit(&bar[B_VEMPTY + (j & 1)]);
                }
                __syncwarp();
                if (next) {
                    if (!mbar_wait_warp(&bar[B_ODONE + u], j & 1)) { ok = false; break; }
                    tc::fence_after_sync();
                    if (tc::elect_one()) qk(u, j + 1);
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (next && tc::elect_one()) tc::mma_commit(&bar[B_KEMPTY + ((j + 1) & 1)]);
            __syncwarp();
        }
        if (tc::elect_one()) tc::mma_commit(&bar[B_LAST]);
        __syncwarp();
        ok = mbar_wait_warp(&bar[B_LAST], 0) && ok;
    } else if (warp < kWidenWarps && nt > 0) {
        // K and V tile j of the sequence to fp16, this warp's rows.
        auto widen_k = [&](int j) -> bool {
            if (!mbar_wait_warp(&bar[B_KCFULL], j & 1) ||
                !mbar_wait_warp(&bar[B_KEMPTY + (j & 1)], ((j >> 1) & 1) ^ 1))
                return false;
            widen_rows<D, KIND, false>(smem_addr(smem + OFF_KC), smem_addr(smem + OFF_K + (j & 1) * kTileBytes), warp,
                                       lane, kTileN);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[B_KCONV + (j & 1)]);
                mbar_arrive(&bar[B_KCEMPTY]);
            }
            return true;
        };
        auto widen_v = [&](int j) -> bool {
            if (!mbar_wait_warp(&bar[B_VCFULL], j & 1) ||
                !mbar_wait_warp(&bar[B_VEMPTY + (j & 1)], ((j >> 1) & 1) ^ 1))
                return false;
            const uint32_t codes = smem_addr(smem + OFF_VC), tile = smem_addr(smem + OFF_V + (j & 1) * kTileBytes);
            const int nrows = j == nt - 1 ? T.klast : kTileN, sees_all = T.pmin - j * kTileN;
            if (kNans && sees_all < kTileN - 1)
                widen_last_v<D, KIND>(codes, tile, warp, lane, nrows, reinterpret_cast<uint32_t*>(first_row), sees_all);
            else
                widen_rows<D, KIND, false>(codes, tile, warp, lane, nrows);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bar[B_VCONV + (j & 1)]);
                mbar_arrive(&bar[B_VCEMPTY]);
            }
            return true;
        };
        // ------------------------------------------------------ Q to fp16
        // Two lanes a row, 64 dims (one panel's 128 bytes) each; the chunks
        // are taken from a place that differs by row, for the banks.
        const int u = warp / kSoftmaxWarps;
        if (u < units) {
            ok = mbar_wait_warp(&bar[B_QFULL], 0);
            if (ok) {
                const int row = 16 * (warp % kSoftmaxWarps) + lane / 2, pn = lane & 1;
                const uint32_t at = smem_addr(smem + OFF_Q + u * kTileBytes) + pn * kPanelBytes + row * 128;
                const bool mine = pn < kPanels;
                float mx = 0.f;
                if (mine) {
#pragma unroll 2
                    for (int c = 0; c < 8; ++c) {
                        uint32_t x[4];
                        tc::lds128(at + (((c + row) & 7) << 4), x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(x[i])), fabsf(bf16hi(x[i]))));
                    }
                }
                mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
                int e = 0;
                if (mx < INFINITY) e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
                // The scale's sign goes with q, so that the scores' factor is
                // not negative, and so does a NaN, which that factor would lose.
                float down = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
                down = isnan(P.scale_log2) ? P.scale_log2 : copysignf(down, P.scale_log2);
                if (mine) {
#pragma unroll 2
                    for (int c = 0; c < 8; ++c) {
                        uint32_t x[4];
                        const uint32_t a = at + (((c + row) & 7) << 4);
                        tc::lds128(a, x);
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = tc::pack_f16x2(bf16lo(x[i]) * down, bf16hi(x[i]) * down);
                        tc::sts128(a, x[0], x[1], x[2], x[3]);
                    }
                }
                if (pn == 0)
                    rowf[u * kTileM + row] =
                        fabsf(P.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
                tc::fence_proxy_async_smem();
            }
        }
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&bar[B_QCONV]);
        ok = ok && widen_k(0);
        if (u >= units) {
            for (int j = 0; j < nt && ok; ++j) ok = widen_v(j) && (j + 1 >= nt || widen_k(j + 1));
        } else {
            // -------------------------------------------------- softmax rows
            // Warps w and w + 4 of a unit share quarter w % 4 of the lanes, 16
            // rows each.  Thread t holds rows t/4 and t/4 + 8 of those and columns
            // 8g + 2(t%4) and + 1 of every group g of 8, so a row's maximum and
            // sum take two shuffles, and its P pairs land in the layout of the
            // 16x128b store.  A block's 16 keys are two groups.
            const int hh = (warp >> 2) & 1;
            const int ma = 32 * (warp & 3) + 16 * hh + lane / 4;  // tile rows ma and ma + 8
            const int mb = ma + 8;
            const int tq = lane & 3;
            const uint32_t tlane = static_cast<uint32_t>(32 * (warp & 3) + 16 * hh) << 16;
            const int pos_a = (ma < T.rows) ? T.pmin + ma : T.pmax;
            const int pos_b = (mb < T.rows) ? T.pmin + mb : T.pmax;
            // Rows of this warp were scaled by its own lanes' neighbours: wait
            // for all of the unit's.
            ok = ok && mbar_wait_warp(&bar[B_QCONV], 0);
            const float fa = rowf[u * kTileM + ma], fb = rowf[u * kTileM + mb];
            // References of P, and of what was moved out of tensor memory.
            float mua = 0.f, mub = 0.f, mfa = 0.f, mfb = 0.f;
            float2 la = make_float2(0.f, 0.f), lb = la;  // row sums, even and odd columns
            // Where rows start in out, worked out when wanted: held over the
            // tiles they would cost the scores their registers.
            const volatile PrefillTile* where = info;
            auto row_at = [&](int m) {
                return P.out + (static_cast<size_t>(where->row0 + m) * P.hq + where->h0 + u) * D;
            };
            // What is moved out waits in the warp's own 16 rows of out, in the
            // order of its registers: D / 8 pieces of 16 bytes a thread, 32 of
            // them together.  (In the rows' own order a request meets eight lines
            // with 32 bytes each: 99 us more over 128 tiles.)  Rows that the warp
            // does not have 16 of are kept in the rows' order.
            const bool whole = 32 * (warp & 3) + 16 * hh + 16 <= T.rows;
            auto pieces = [&]() {
                return reinterpret_cast<float4*>(row_at(32 * (warp & 3) + 16 * hh + (D == 128 ? 0 : lane / 16)) +
                                                 4 * (D == 128 ? lane : lane & 15));
            };
            const int pitch = P.hq * D / 4 * (D == 128 ? 1 : 2);  // of a thread's pieces
            // 32 values of a thread: columns 64 c and on.
            auto load_kept = [&](int c, float (&x)[32]) {
                if (whole) {
                    const float4* src = pieces() + static_cast<size_t>(8 * c) * pitch;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 v = src[static_cast<size_t>(i) * pitch];
                        x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                    }
                } else {
                    const float *oa = row_at(ma) + 2 * tq, *ob = row_at(mb) + 2 * tq;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 va = make_float2(0.f, 0.f), vb = va;
                        if (ma < T.rows) va = *reinterpret_cast<const float2*>(oa + 64 * c + 8 * i);
                        if (mb < T.rows) vb = *reinterpret_cast<const float2*>(ob + 64 * c + 8 * i);
                        x[4 * i] = va.x, x[4 * i + 1] = va.y, x[4 * i + 2] = vb.x, x[4 * i + 3] = vb.y;
                    }
                }
            };
            auto store_rows = [&](int c, const float (&x)[32]) {
                float *oa = row_at(ma) + 2 * tq, *ob = row_at(mb) + 2 * tq;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (ma < T.rows)
                        *reinterpret_cast<float2*>(oa + 64 * c + 8 * i) = make_float2(x[4 * i], x[4 * i + 1]);
                    if (mb < T.rows)
                        *reinterpret_cast<float2*>(ob + 64 * c + 8 * i) = make_float2(x[4 * i + 2], x[4 * i + 3]);
                }
            };
            // x = x fac + (tensor memory's columns 64 c and on) alpha.
            auto join = [&](int c, float (&x)[32], float fac_a, float fac_b, float alpha_a, float alpha_b) {
                uint32_t r[32];
                tc::tmem_ld16x256b_x8(tmem + tlane + col_o(u) + 64 * c, r);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const bool row_b = i & 2;
                    x[i] = fmaf(__uint_as_float(r[i]), row_b ? alpha_b : alpha_a, x[i] * (row_b ? fac_b : fac_a));
                }
            };
            for (int j = 0; j < nt && ok; ++j) {
                if (!widen_v(j) || (j + 1 < nt && !widen_k(j + 1)) || !mbar_wait_warp(&bar[B_SFULL + u], j & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const int kbase = j * kTileN;
                const bool full = kbase + kTileN - 1 <= __shfl_sync(FULL, pos_a, 0);
                const TileScales* sct = scales + j % kScaleTiles * kBlocksPerTile;
                const bool wide = __any_sync(FULL, sct[0].wide != 0.f);
                // The scores are taken from tensor memory twice, 32 keys at a
                // time and the next 32 on their way: held over both passes, 64
                // a thread, they would push other values out of registers.
                const uint32_t ts = tmem + tlane + col_s(u);
                uint32_t sr[2][16];
                // Keys past the row's position (NaN in unused slots included)
                // out of 32 keys' scores.
                auto mask = [&](int c, uint32_t (&s)[16]) {
                    if (full) return;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (kbase + 32 * c + 8 * (i / 4) + 2 * tq + (i & 1) > (i & 2 ? pos_b : pos_a))
                            s[i] = 0xff800000u;
                };
                // Pass 1: each row's largest y = s factor + log2 vs, block by
                // block.
                float xa = -INFINITY, xb = -INFINITY;
                tc::tmem_ld16x256b_x4(ts, sr[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tc::tmem_wait_ld(sr[c & 1]);
                    tc::tmem_ld16x256b_x4(ts + 32 * ((c + 1) & 3), sr[(c + 1) & 1]);  // at last, the first again
                    mask(c, sr[c & 1]);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const uint32_t* s = &sr[c & 1][8 * b];
                        const float ks = sct[2 * c + b].k, lv = sct[2 * c + b].log2_v.x;
                        float va = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
                        float vb = fmaxf(__uint_as_float(s[2]), __uint_as_float(s[3]));
                        va = fmax3(va, __uint_as_float(s[4]), __uint_as_float(s[5]));
                        vb = fmax3(vb, __uint_as_float(s[6]), __uint_as_float(s[7]));
                        xa = fmaxf(xa, fmaf(va, block_factor(fa, ks), lv));
                        xb = fmaxf(xb, fmaf(vb, block_factor(fb, ks), lv));
                    }
                }
                xa = fmaxf(xa, __shfl_xor_sync(FULL, xa, 1));
                xb = fmaxf(xb, __shfl_xor_sync(FULL, xb, 1));
                xa = fmaxf(xa, __shfl_xor_sync(FULL, xa, 2));
                xb = fmaxf(xb, __shfl_xor_sync(FULL, xb, 2));
                // The reference moves in the first tile, and where the largest
                // passed it by more than 2^3.  Rounded down, here and below, P
                // stays below 2^16 however large the scores (past 2^20 or so
                // the sums below are no longer exact).
                float alpha_a = 1.f, alpha_b = 1.f;
                const bool need_a = j == 0 || xa > __fadd_rd(mua, kThreshold);
                const bool need_b = j == 0 || xb > __fadd_rd(mub, kThreshold);
                const bool moves = __any_sync(FULL, need_a || need_b);
                if (moves) {
                    if (need_a) {
                        const float half = fast_exp2(0.5f * (mua - xa));
                        alpha_a = half * half;
                        if (j > 0) la = make_float2(la.x * half * half, la.y * half * half);
                        mua = xa;
                    }
                    if (need_b) {
                        const float half = fast_exp2(0.5f * (mub - xb));
                        alpha_b = half * half;
                        if (j > 0) lb = make_float2(lb.x * half * half, lb.y * half * half);
                        mub = xb;
                    }
                    if (j == 0) {
                        mfa = mua;
                        mfb = mub;
                    }
                }
                // Pass 2: P in two fp16 terms, its first 11 bits and the rest,
                // over the 32 keys' scores; the row sums without the V scales.
                const float sha = __fsub_rd(kShift, mua), shb = __fsub_rd(kShift, mub);
                const float2 ra = make_float2(sha, sha), rb = make_float2(shb, shb);
                if (wide) {
                    tc::tmem_wait_ld(sr[0]);
                    const float2 l = wide_sums(ts, sct, fa, fb, sha - kSumShift, shb - kSumShift, kbase + 2 * tq,
                                               full ? INT32_MAX : pos_a, full ? INT32_MAX : pos_b);
                    la.x += l.x;
                    lb.x += l.y;
                    tc::tmem_ld16x256b_x4(ts, sr[0]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tc::tmem_wait_ld(sr[c & 1]);
                    if (c < 3) tc::tmem_ld16x256b_x4(ts + 32 * (c + 1), sr[(c + 1) & 1]);
                    mask(c, sr[c & 1]);
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const TileScales& sc = sct[2 * c + b];
                        const float ka = block_factor(fa, sc.k), kb = block_factor(fb, sc.k);
                        const float2 pa = make_float2(ka, ka), pb = make_float2(kb, kb);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t* s = &sr[c & 1][4 * (2 * b + h)];
                            const int at = 2 * (2 * b + h);
                            const float2 va = make_float2(__uint_as_float(s[0]), __uint_as_float(s[1]));
                            const float2 vb = make_float2(__uint_as_float(s[2]), __uint_as_float(s[3]));
                            float2 ya = __ffma2_rn(va, pa, sc.log2_v), yb = __ffma2_rn(vb, pb, sc.log2_v);
                            ya = __fadd2_rn(ya, ra);
                            yb = __fadd2_rn(yb, rb);
                            ya = make_float2(fast_exp2(ya.x), fast_exp2(ya.y));
                            yb = make_float2(fast_exp2(yb.x), fast_exp2(yb.y));
                            la = __ffma2_rn(ya, sc.inv_v, la);
                            lb = __ffma2_rn(yb, sc.inv_v, lb);
                            split2(ya, hi[at], lo[at]);
                            split2(yb, hi[at + 1], lo[at + 1]);
                        }
                    }
                    tc::tmem_st16x128b_x4(ts + 32 * c, hi);
                    tc::tmem_st16x128b_x4(ts + 32 * c + 16, lo);
                }
                if (j > 0 && j % kKeep == 0) {
                    // The MMA warp starts O anew with this tile's P V.
                    const float fac_a = fast_exp2(mfa - mua), fac_b = fast_exp2(mfb - mub);
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        float x[32];
                        if (j > kKeep) {
                            load_kept(c, x);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = 0.f;
                        }
                        join(c, x, fac_a, fac_b, alpha_a, alpha_b);
                        if (whole) {
                            float4* dst = pieces() + static_cast<size_t>(8 * c) * pitch;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                dst[static_cast<size_t>(i) * pitch] =
                                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        } else {
                            store_rows(c, x);
                        }
                    }
                    mfa = mua;
                    mfb = mub;
                } else if (moves && j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        uint32_t r[32];
                        const uint32_t at = tmem + tlane + col_o(u) + 64 * c;
                        tc::tmem_ld16x256b_x8(at, r);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            r[4 * i] = __float_as_uint(__uint_as_float(r[4 * i]) * alpha_a);
                            r[4 * i + 1] = __float_as_uint(__uint_as_float(r[4 * i + 1]) * alpha_a);
                            r[4 * i + 2] = __float_as_uint(__uint_as_float(r[4 * i + 2]) * alpha_b);
                            r[4 * i + 3] = __float_as_uint(__uint_as_float(r[4 * i + 3]) * alpha_b);
                        }
                        tc::tmem_st16x256b_x8(at, r);
                    }
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_PFULL + u]);
            }
            if (ok && !mbar_wait_warp(&bar[B_ODONE + u], (nt - 1) & 1)) ok = false;
            if (ok) {
                tc::fence_after_sync();
                float sa = la.x + la.y, sb = lb.x + lb.y;
                sa += __shfl_xor_sync(FULL, sa, 1);
                sb += __shfl_xor_sync(FULL, sb, 1);
                sa += __shfl_xor_sync(FULL, sa, 2);
                sb += __shfl_xor_sync(FULL, sb, 2);
                const float inva = 1.f / (1 << kSumShift) / sa, invb = 1.f / (1 << kSumShift) / sb;
                const float fac_a = fast_exp2(mfa - mua), fac_b = fast_exp2(mfb - mub);
                auto kept_or_zero = [&](int c, float (&x)[32]) {
                    if (nt > kKeep) {
                        load_kept(c, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = 0.f;
                    }
                };
                float x[32], y[D == 128 ? 32 : 1];
                kept_or_zero(0, x);
                join(0, x, fac_a * inva, fac_b * invb, inva, invb);
                if constexpr (D == 128) kept_or_zero(1, y);
                __syncwarp();  // the rows are read before they are written in their own order
                store_rows(0, x);
                if constexpr (D == 128) {
                    join(1, y, fac_a * inva, fac_b * invb, inva, invb);
                    store_rows(1, y);
                }
                if constexpr (kNans) {
                    // Rows from a dim's first_row on see a NaN there.
                    bool any = false;
                    for (int i = lane; i < D / 4; i += 32)
                        any |= reinterpret_cast<const volatile uint32_t*>(first_row)[i] != 0xffffffffu;
                    if (__any_sync(FULL, any)) {
                        if (ma < T.rows) store_nans(row_at(ma), first_row, ma, 2 * tq, D);
                        if (mb < T.rows) store_nans(row_at(mb), first_row, mb, 2 * tq, D);
                    }
                }
            }
        }
    } else if (warp < kWidenWarps && T.bad && T.s >= 0) {
        // Zero rows for a sequence whose arguments are out of range.
        for (int i = threadIdx.x; i < T.rows * units * (D / 4); i += kWidenWarps * 32) {
            const int c = i % (D / 4), h = i / (D / 4) % units, m = i / (D / 4) / units;
            reinterpret_cast<float4*>(P.out + (static_cast<size_t>(T.row0 + m) * P.hq + T.h0 + h) * D)[c] =
                make_float4(0.f, 0.f, 0.f, 0.f);
        }
    }
    if (!ok) record_error(P.err, kErrTimeout, 0x100u + static_cast<uint32_t>(warp));
    // ---------------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kLoadWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D, int KIND>
cudaError_t launch(const Params& P, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, dim3 grid,
                   cudaStream_t stream) {
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(prefill_scaled_kernel<D, KIND>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_overlapped(prefill_scaled_kernel<D, KIND>, grid, dim3(kThreads), SMEM_BYTES, stream, tq, tk, tv, P);
}

}  // namespace

cudaError_t launch_prefill_scaled(const PrefillArgs& a, cudaStream_t stream) {
    if (a.num_tiles == 0) return cudaSuccess;
    const cuuint64_t d = static_cast<cuuint64_t>(a.head_dim);
    CUtensorMap tq, tk, tv;
    {
        const cuuint64_t dims[3] = {d, static_cast<cuuint64_t>(a.num_q_heads), static_cast<cuuint64_t>(a.num_tokens)};
        const cuuint64_t strides[2] = {d * 2, static_cast<cuuint64_t>(a.num_q_heads) * d * 2};
        const cuuint32_t box[3] = {64, 1, kTileM};
        if (!make_bf16_map(&tq, a.q, 3, dims, strides, box)) return cudaErrorInvalidValue;
    }
    {
        // Rows of head_dim codes, 16 a slab, one slab per (block, kv head).
        const cuuint64_t slabs = static_cast<cuuint64_t>(a.num_blocks) * a.num_kv_heads;
        const cuuint64_t dims[3] = {d, kBlockSize, slabs > 0 ? slabs : 1};
        const cuuint64_t strides[2] = {d, d * kBlockSize};
        const cuuint32_t box[3] = {static_cast<cuuint32_t>(a.head_dim), kBlockSize, 1};
        if (!make_tile_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.k_pool, 3, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_NONE) ||
            !make_tile_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.v_pool, 3, dims, strides, box,
                           CU_TENSOR_MAP_SWIZZLE_NONE))
            return cudaErrorInvalidValue;
    }
    Params P;
    P.scales = reinterpret_cast<const float2*>(a.block_scales);
    P.block_tables = a.block_tables;
    P.context_lens = a.context_lens;
    P.qsl = a.query_start_loc;
    P.out = a.out;
    P.err = a.err;
    P.num_blocks = a.num_blocks;
    P.hkv = a.num_kv_heads;
    P.hq = a.num_q_heads;
    P.num_seqs = a.num_seqs;
    P.num_tokens = a.num_tokens;
    P.max_blocks = a.max_blocks_per_seq;
    P.ctx_cap = static_cast<int32_t>(
        std::min<int64_t>(a.max_context_len, static_cast<int64_t>(a.max_blocks_per_seq) * kBlockSize));
    // Two q heads per CTA when a GQA group holds an even number of them.
    P.units = ((a.num_q_heads / a.num_kv_heads) % 2 == 0) ? 2 : 1;
    P.split_last = P.units == 2 ? a.split_last : 0;
    P.decode_launch = a.decode_launch ? 1 : 0;
    P.stall = take_prefill_stall() ? 1 : 0;
    P.scale_log2 = a.scale * kLog2e;
    const dim3 grid(static_cast<unsigned>(a.num_tiles + (P.units == 2 ? a.split_tiles : 0)),
                    static_cast<unsigned>(a.num_q_heads / P.units));
    if (a.head_dim == 128)
        return a.int8_codes ? launch<128, kKindInt8Blocks>(P, tq, tk, tv, grid, stream)
                            : launch<128, kKindE4m3Blocks>(P, tq, tk, tv, grid, stream);
    return a.int8_codes ? launch<64, kKindInt8Blocks>(P, tq, tk, tv, grid, stream)
                        : launch<64, kKindE4m3Blocks>(P, tq, tk, tv, grid, stream);
}

}  // namespace pkv
