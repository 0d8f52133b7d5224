// decode_scaled.cuh -- decode attention over 8-bit pools with a scale for
// each (block, kv head): the consumer warps' block math and the launch.  The
// cut of the work, the producer's walk over the block table, the merge of the
// warps' states and of split contexts are decode_kernel.cuh's.
//
// With K_j = ks_b c_j and V_j = vs_b d_j (codes c, d; b the block of key j),
//     s_j = (scale log2 e ks_b) (q . c_j),  out = sum_j 2^(s_j) vs_b d_j / sum_j 2^(s_j).
// The codes are exact in fp16, so both products run on fp16 operands and the
// scales only touch scores and weights, never the codes.
//
//  * A stage of the ring holds two blocks of one kv head (32 keys), K and V:
//    four swizzled 16-row tiles.  Twice the keys of a stage of the other pools:
//    the maximum's shuffles, the wait and the hand-back are paid once for 32
//    keys, and the two blocks' chains of MMAs run side by side (one block at a
//    time, 68 contexts of 40/40 x 128: 467 us against 422).
//  * The producer warp only leaves orders, slabs and scales of a stage; each
//    consumer warp asks for its own stages as it frees them.  A stage is four
//    tiled copies, which cost one issuing thread about 740 cycles, twice the
//    stage's share of the HBM rate (one producer warp for all: 633 us).
//  * S = K Q^T (m16n8k16): 16 keys by the group's heads (columns that the group
//    lacks are zero).  Lane (g, t) = (lane / 4, lane % 4) gets keys g and g + 8
//    for heads 2t and 2t + 1.  q is scaled per head by a power of two into
//    fp16's upper range; the scores take the factor back.
//  * O^T += V^T P^T, with P in two fp16 terms (rounded, and what the rounding
//    lost: 2^-22, one term would be off by 2^-11), each an 8 x 8 transposition
//    away from S's layout.  O^T's columns are S's heads, so a moved maximum
//    rescales without a shuffle, and a lane holds D / 4 values of O (P V with
//    the heads as rows holds twice that, which leaves room for 8 warps in place
//    of 12: 412 us against 371).
//  * Weights of a block carry its V scale, vs = f 2^e with f in [1, 2): the
//    running maximum is that of s_j + e, u = 2^(s_j + e - m + 11), the weight
//    u f and the term of the sum u 2^-(e + 8), and weights end 2^-36 below the largest
//    (fp16 is exact to 2^-24).  A key of a small V scale may count for nothing in
//    O and for all in the sum (16 rows of zeros, whose scale is 2^-100, beside
//    one of scale 2^40: v / 17), so u is 2^112 larger in blocks whose V scale is
//    more than 2^104 below the item's largest, and sums move to other references
//    by two factors of half the logarithm, since 2^x may be flushed where the sum
//    times 2^x is not.
//  * The order of dims in S and of keys in P V is free: a lane reads whole
//    16-byte pieces of K rows and of V rows (8-byte pieces of V at head_dim
//    64), and rows are dealt to lanes so that the lanes that read together hit
//    different banks of the swizzled tiles (see key_row).
//  * Bound: 68 contexts of 40/40 x 128 run at 0.89 of the measured copy rate.
//    34 contexts of 640 tokens (16/8 x 128) stream their 45 MB in 6.2 us, 7.2
//    TB/s; the other 9 are fixed: 3.3 us from the end of the launch before to
//    the first order (lengths, cut, table, scales), 1.7 to the first stage, and
//    about 3 for the merge.
#pragma once

#include "decode_kernel.cuh"
#include "scaled_device.cuh"
#include "tcgen05_rows.cuh"

namespace pkv {
namespace {

template <int D, int G, int KIND>
struct ScaledCfg {
    static constexpr int HEAD_DIM = D, GROUP = G, ELEM = 1;
    static constexpr bool SCALED = true, MMA = true;
    static constexpr int BPS = 2;
    // Consumer warps: each is bound by the latency of its own chain, so as many
    // as the ring has two stages for (68 contexts of 40/40 x 128: 8 warps
    // 394 us, 11 375, 12 359; 10 that no longer have two stages each, at head
    // groups of 8, 55 against 44 with 8).
    static constexpr int W = G <= 2 ? 12 : 8;
    static constexpr int MERGE_LANES = W <= 8 ? 8 : 16;
    // What a pair costs beyond its blocks, in blocks: its warps' states are
    // handed over and merged, and its last stages leave warps idle.  Without
    // it the CTA that gets the short contexts ends last.  One number for all
    // shapes: over 31 contexts of 300 to 4,011 tokens and 68 of 64 to 32,768,
    // both head_dims, groups of 1, 2, 4 and 8, 0 takes 1.20 of the time with
    // 12, 4 1.14, 8 1.05, 16 1.00 and 24 1.02, and 12 is at most 6 % above the
    // best in any of them; 8 to 64 contexts of 200 to 1,679 tokens: 0 takes 1.05,
    // 8 1.00, 16 1.01, 24 1.00.
    static constexpr int EXTRA_UNITS = 12;
    static constexpr int MERGE_BUFS = 1;
    static constexpr int MERGERS = G == 8 ? 2 : 1;
    static constexpr int PRODUCER_WARP = W, MERGER_WARP = W + 1, THREADS = 32 * (W + 1 + MERGERS);
    static constexpr int ORDERS = 8;  // stages a consumer warp is told of ahead
    static constexpr int SLAB = kBlockSize * D;
    static constexpr int STAGE_BYTES = 4 * SLAB;  // K of two blocks, V of two blocks
    static constexpr int QBYTES = G * D * 2;
    static constexpr int R_ITEMQ = 0;
    static constexpr int R_DESC = R_ITEMQ + kItemRing * QBYTES;
    static constexpr int R_MO = R_DESC + kItemRing * (int)sizeof(ItemDesc);
    static constexpr int R_ML = R_MO + MERGE_BUFS * W * G * D * 4;
    static constexpr int R_WT = R_ML + MERGE_BUFS * W * G * 8;
    static constexpr int R_MSM = align_up(R_WT + G * (W + 1) * 4, 8);
    static constexpr int R_BAR = align_up(R_MSM + G * 8, 8);
    // 226 KB less the regions above, the orders and their barriers, 32 more
    // barriers and the 1,024-byte alignment of the ring; a stage has one barrier.
    static constexpr int STAGES_FIT =
        (226 * 1024 - R_BAR - W * ORDERS * ((int)sizeof(Order) + 16) - 32 * 8 - 32 - 1024) / (STAGE_BYTES + 8);
    static constexpr int SW_FIT = STAGES_FIT / W;
    static constexpr int SW = SW_FIT < 6 ? SW_FIT : 6;
    static constexpr int STAGES = SW * W;
    static constexpr int NBAR = STAGES + 2 * kItemRing + 2 * MERGE_BUFS + 2 * W * ORDERS;
    static constexpr int OFF_REST = STAGES * STAGE_BYTES;
    static constexpr int OFF_ITEMQ = OFF_REST + R_ITEMQ;
    static constexpr int OFF_DESC = OFF_REST + R_DESC;
    static constexpr int OFF_MO = OFF_REST + R_MO;
    static constexpr int OFF_ML = OFF_REST + R_ML;
    static constexpr int OFF_WT = OFF_REST + R_WT;
    static constexpr int OFF_MSM = OFF_REST + R_MSM;
    static constexpr int OFF_BAR = OFF_REST + R_BAR;
    static constexpr int OFF_FLAG = OFF_BAR + NBAR * 8;
    static constexpr int OFF_ORDERS = align_up(OFF_FLAG + 4, 16);
    static constexpr int OFF_NEW = OFF_ORDERS;  // of fused steps only, which there are none of
    static constexpr int SMEM = OFF_ORDERS + W * ORDERS * (int)sizeof(Order) + 1024;
    static_assert(SW >= 1, "ring too shallow");
    static_assert(OFF_ITEMQ % 16 == 0 && OFF_DESC % 16 == 0 && OFF_MO % 16 == 0 && OFF_ML % 8 == 0 &&
                      OFF_BAR % 8 == 0 && STAGE_BYTES % 1024 == 0 && SLAB % 512 == 0,
                  "shared-memory regions aligned for their widest access");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// Stages after which a warp's O and sums join what it has of the item so far, in
// its slot for the merger.  The tensor cores' sums lose half a unit in the last
// place on average at each MMA, always to the same side: a row of 131,072 tokens
// that one CTA reads came out 3e-5 (12 warps) to 8e-5 (8) short of its size, and
// so 7e-7, in the same time (with 8 stages 3e-7; 31 contexts of 64/8 x 128: 37.0
// us, 37.7 with 8).
constexpr int kFoldStages = 16;

// P's exponent against the running maximum: a weight is below 2^(3 + 11 + 1).
constexpr float kScaledThreshold = 3.0f, kScaledShift = 11.0f;

// Byte offset of 16-byte chunk c of row r of a swizzled slab: rows of 128
// bytes with chunks XORed by r mod 8, rows of 64 bytes with chunks XORed by
// (r / 2) mod 4.
template <int D>
__device__ __forceinline__ int slab_at(int r, int c) {
    return D == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Where lane (g, t) reads: K chunk 2t (+ 1) of row key_row(g) (64-byte rows:
// chunk t), its D / 8 dims of V rows key_row(2t) and key_row(2t + 1).  The other half of
// a block is 8 rows on, with the same swizzle.
struct LaneOffsets {
    int k, k1, v0, v1;
};

// Row of a block (within its half) that column n of an S tile stands for.
// Rows of 128 bytes: n itself; reading chunk 2t + c of rows g (K) and chunk g
// of rows 2t (V), eight lanes that read together hit eight 16-byte banks.
// Rows of 64 bytes: K wants neighbouring n on rows of different parity, V wants
// the rows of n = 0, 2, 4, 6 (and 1, 3, 5, 7) to be two of each parity that
// differ in bit 2; n = b2 b1 b0 to row b1, b0, b2 xor b0 does both.
template <int D>
__device__ __forceinline__ int key_row(int n) {
    return D == 128 ? n : ((n & 2) << 1) | ((n & 1) << 1) | ((n >> 2) ^ (n & 1));
}

template <int D>
__device__ __forceinline__ LaneOffsets lane_offsets(int g, int t) {
    LaneOffsets r;
    r.k = slab_at<D>(key_row<D>(g), D == 128 ? 2 * t : t);
    r.k1 = r.k ^ 16;
    const int c = D == 128 ? g : g >> 1, in = D == 128 ? 0 : 8 * (g & 1);
    r.v0 = slab_at<D>(key_row<D>(2 * t), c) + in;
    r.v1 = slab_at<D>(key_row<D>(2 * t + 1), c) + in;
    return r;
}

// Two codes in bytes 0 and 1 (HI: 2 and 3) of w to an fp16 pair, exactly.
// int8: u = code + 128 as the low byte of 0x6400 is 1024 + u, less 1152.
template <int KIND, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t w) {
    if constexpr (KIND == kKindInt8Blocks) {
        const uint32_t biased = __byte_perm(w, 0x64646464u, HI ? 0x4342 : 0x4140);
        uint32_t r;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(r) : "r"(biased), "r"(0x64806480u));
        return r;
    } else {
        return e4m3x2_f16x2(HI ? w >> 16 : w);
    }
}

// int8 codes are loaded with their sign bit turned (code + 128).
template <int KIND>
__device__ __forceinline__ uint32_t turned(uint32_t w) {
    return KIND == kKindInt8Blocks ? w ^ 0x80808080u : w;
}

// Unlike mma_f16 and lds128 free to be moved: the order of a stage's products
// and loads is the compiler's, so that chains run side by side.
__device__ __forceinline__ void mma_free(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of a block, S = K Q^T: lane (g, t) gets those of rows key_row(g) (s[0],
// s[1]) and key_row(g) + 8 (s[2], s[3]) for heads 2t and 2t + 1.
template <int D, int KIND>
__device__ __forceinline__ void scores(const uint8_t* k, const uint32_t (&qb)[D / 8], float (&s)[4],
                                       const LaneOffsets& at) {
    s[0] = s[1] = s[2] = s[3] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        uint32_t w[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint4 u = *reinterpret_cast<const uint4*>(k + (c ? at.k1 : at.k) + x * 8 * D);
            w[x][0] = turned<KIND>(u.x), w[x][1] = turned<KIND>(u.y);
            w[x][2] = turned<KIND>(u.z), w[x][3] = turned<KIND>(u.w);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mma_free(s, widen2<KIND, false>(w[0][i]), widen2<KIND, false>(w[1][i]), widen2<KIND, true>(w[0][i]),
                     widen2<KIND, true>(w[1][i]), qb[2 * (4 * c + i)], qb[2 * (4 * c + i) + 1]);
    }
}

// An 8 x 8 matrix of 16-bit values, lane (g, t) holding row g, columns 2t and
// 2t + 1, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// O^T += V^T P^T over one block: p[0] and p[2] are P (rounded to fp16) of
// the keys of halves 0 and 1, p[1] and p[3] what the rounding lost.  Tile mm's
// rows g and g + 8 are dims (D / 8) g + 2 mm and + 1, its columns the heads.
// Rows past the context are zero where their codes could be NaN.
template <int D, int KIND>
__device__ __forceinline__ void weigh(const uint8_t* v, int valid, const uint32_t (&p)[4], float (&o)[D / 16][4],
                                      const LaneOffsets& at, int t) {
    constexpr int NW = D / 32;  // words of a lane's D / 8 dims
    uint32_t w[4][NW];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint8_t* src = v + (j & 1 ? at.v1 : at.v0) + (j >> 1) * 8 * D;
        if constexpr (D == 128) {
            const uint4 u = *reinterpret_cast<const uint4*>(src);
            w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
        } else {
            const uint2 u = *reinterpret_cast<const uint2*>(src);
            w[j][0] = u.x, w[j][1] = u.y;
        }
        if (KIND != kKindInt8Blocks && valid < kBlockSize) {
            const int row = 8 * (j >> 1) + key_row<D>(2 * t + (j & 1));
#pragma unroll
            for (int i = 0; i < NW; ++i) w[j][i] = row < valid ? w[j][i] : 0u;
        }
#pragma unroll
        for (int i = 0; i < NW; ++i) w[j][i] = turned<KIND>(w[j][i]);
    }
#pragma unroll
    for (int i = 0; i < NW; ++i) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t a = __byte_perm(w[0][i], w[1][i], x ? 0x7362 : 0x5140);
            const uint32_t b = __byte_perm(w[2][i], w[3][i], x ? 0x7362 : 0x5140);
            const uint32_t a0 = widen2<KIND, false>(a), a1 = widen2<KIND, true>(a);
            const uint32_t a2 = widen2<KIND, false>(b), a3 = widen2<KIND, true>(b);
            mma_free(o[2 * i + x], a0, a1, a2, a3, p[0], p[2]);
            mma_free(o[2 * i + x], a0, a1, a2, a3, p[1], p[3]);
        }
    }
}

// Whether the phase with the given parity has completed, for the whole warp.
__device__ __forceinline__ bool mbar_test_warp(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return __all_sync(0xffffffffu, ok);
}

template <class C, int KIND>
__device__ void run_consumer_scaled(const DecodeParams& P, const CUtensorMap* tmk, const CUtensorMap* tmv,
                                    uint8_t* smem, const Bars& B, volatile int* abort_flag,
                                    int warp, int lane) {
    constexpr int D = C::HEAD_DIM, G = C::GROUP;
    constexpr int QW = D / 8;   // q words of a lane: its D / 4 dims
    const unsigned FULL = 0xffffffffu;
    const ItemDesc* descs = reinterpret_cast<const ItemDesc*>(smem + C::OFF_DESC);
    float* mo = reinterpret_cast<float*>(smem + C::OFF_MO);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int g = lane >> 2, t = lane & 3;
    const LaneOffsets at = lane_offsets<D>(g, t);
    const Order* orders = reinterpret_cast<const Order*>(smem + C::OFF_ORDERS) + warp * C::ORDERS;
    uint64_t* ofull = B.ofull + warp * C::ORDERS;
    uint64_t* full = B.full + warp * C::SW;
    uint8_t* ring = smem + warp * C::SW * C::STAGE_BYTES;
    const uint64_t policy = l2_policy_evict_first();
    uint32_t taken = 0, issued = 0, item_seq = 0;  // stages consumed, asked for
    bool ok = true;
    // Asks for the stages that are free and ordered.
    auto issue = [&]() {
        while (issued - taken < C::SW && mbar_test_warp(&ofull[issued % C::ORDERS], (issued / C::ORDERS) & 1)) {
            const Order* o = orders + issued % C::ORDERS;
            const int slab0 = o->slab[0], slab1 = o->slab[1];
            const bool two = o->two != 0;
            if (tc::elect_one()) {
                uint8_t* dst = ring + issued % C::SW * C::STAGE_BYTES;
                uint64_t* bar = &full[issued % C::SW];
                mbar_arrive_expect_tx(bar, (two ? 4 : 2) * C::SLAB);
                tma_slab_g2s(dst, tmk, slab0, bar, policy);
                if (two) tma_slab_g2s(dst + C::SLAB, tmk, slab1, bar, policy);
                tma_slab_g2s(dst + 2 * C::SLAB, tmv, slab0, bar, policy);
                if (two) tma_slab_g2s(dst + 3 * C::SLAB, tmv, slab1, bar, policy);
            }
            __syncwarp();
            ++issued;
        }
    };
    while (ok) {
        const uint32_t slot = item_seq % kItemRing;
        // The item's stages may be ordered before its q has landed.
        issue();
        if (!mbar_test_warp(&B.ifull[slot], (item_seq / kItemRing) & 1)) {
            const uint64_t t0 = global_timer_ns();
            while (ok && !mbar_test_warp(&B.ifull[slot], (item_seq / kItemRing) & 1)) {
                issue();
                ok = !__any_sync(FULL, *abort_flag != 0 || global_timer_ns() - t0 > kWaitLimitNs);
            }
            if (!ok) break;
        }
        const ItemDesc d = descs[slot];
        if (d.s < 0) break;
        // q of head g, dims (D / 4) t and on, as the A operand (zero for g >=
        // G), scaled by a power of two so that the largest is in [2^14, 2^15)
        // of fp16; the scores get the factor back.
        uint32_t qb[QW];
        float f0, f1;
        {
            const uint8_t* qs = smem + C::OFF_ITEMQ + slot * C::QBYTES + (g * D + t * (D / 4)) * 2;
#pragma unroll
            for (int c = 0; c < QW / 4; ++c) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (g < G) u = *reinterpret_cast<const uint4*>(qs + 16 * c);
                qb[4 * c] = u.x, qb[4 * c + 1] = u.y, qb[4 * c + 2] = u.z, qb[4 * c + 3] = u.w;
            }
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < QW; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(qb[i])), fabsf(bf16hi(qb[i]))));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
            int e = 0;
            if (mx < INFINITY) e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
            const float down = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            const float up = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
            for (int i = 0; i < QW; ++i) qb[i] = f16x2_rn(bf16lo(qb[i]) * down, bf16hi(qb[i]) * down);
            f0 = P.scale_log2 * __shfl_sync(FULL, up, 8 * t);
            f1 = P.scale_log2 * __shfl_sync(FULL, up, 8 * t + 4);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.iempty[slot]);
        float m0 = -INFINITY, m1 = -INFINITY, l0, l1;
        float o[D / 16][4];
        const int nst = (d.b1 - d.b0 + 1) / 2;
        const int first = (warp - d.rot + C::W) % C::W;
        const int buf = item_seq % C::MERGE_BUFS;
        int b = first;
        do {
            const bool begun = b != first;
            l0 = l1 = 0.f;
#pragma unroll
            for (int j = 0; j < D / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
            for (const int stop = min(nst, b + kFoldStages * C::W); b < stop; b += C::W) {
                const uint32_t st = taken % C::SW;
                issue();
                if (issued == taken) {  // not even this one is ordered yet
                    if (!mbar_wait_warp(&ofull[taken % C::ORDERS], (taken / C::ORDERS) & 1)) {
                        ok = false;
                        break;
                    }
                    issue();
                }
                if (*abort_flag || !mbar_wait_warp(&full[st], (taken / C::SW) & 1)) {
                    ok = false;
                    break;
                }
                const Order* order = orders + taken % C::ORDERS;
                const int blk = d.b0 + 2 * b;
                const int keys = min(2 * kBlockSize, (min(d.b1 * kBlockSize, d.n) - blk * kBlockSize));
                constexpr int NB = C::BPS;
                const uint8_t* kst = ring + st * C::STAGE_BYTES;
                float u[NB][4];
                BlockScales sc[NB];
                int valid[NB];
                float mb0 = -INFINITY, mb1 = -INFINITY;
#pragma unroll
                for (int i = 0; i < NB; ++i) scores<D, KIND>(kst + i * C::SLAB, qb, u[i], at);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    valid[i] = min(max(keys - i * kBlockSize, 0), kBlockSize);
                    sc[i] = order->scales[i];
                    const float k0 = f0 * sc[i].k, k1 = f1 * sc[i].k;
                    u[i][0] = fmaf(u[i][0], k0, sc[i].e), u[i][1] = fmaf(u[i][1], k1, sc[i].e);
                    u[i][2] = fmaf(u[i][2], k0, sc[i].e), u[i][3] = fmaf(u[i][3], k1, sc[i].e);
                    if (valid[i] < kBlockSize) {
                        if (key_row<D>(g) >= valid[i]) u[i][0] = u[i][1] = -INFINITY;
                        if (key_row<D>(g) + 8 >= valid[i]) u[i][2] = u[i][3] = -INFINITY;
                    }
                    mb0 = fmaxf(mb0, fmaxf(u[i][0], u[i][2]));
                    mb1 = fmaxf(mb1, fmaxf(u[i][1], u[i][3]));
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) {
                    mb0 = fmaxf(mb0, __shfl_xor_sync(FULL, mb0, off));
                    mb1 = fmaxf(mb1, __shfl_xor_sync(FULL, mb1, off));
                }
                // A new reference only where the maximum grew by more than 2^3.
                // Rounded down, here and below, P stays below 2^16 however large the
                // scores (past 2^20 or so these sums are no longer exact).
                const bool moves0 = mb0 > __fadd_rd(m0, kScaledThreshold);
                const bool moves1 = mb1 > __fadd_rd(m1, kScaledThreshold);
                if (__any_sync(FULL, moves0 || moves1)) {
                    const Halves h0(moves0 ? m0 - mb0 : 0.f), h1(moves1 ? m1 - mb1 : 0.f);
                    const float a0 = h0.whole(), a1 = h1.whole();
                    m0 = moves0 ? mb0 : m0;
                    m1 = moves1 ? mb1 : m1;
                    l0 = h0.times(l0);
                    l1 = h1.times(l1);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) o[j][0] *= a0, o[j][1] *= a1, o[j][2] *= a0, o[j][3] *= a1;
                }
                const float add0 = __fsub_rd(kScaledShift, m0), add1 = __fsub_rd(kScaledShift, m1);
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (i > 0 && valid[i] == 0) break;
                    const float up = lifted(sc[i]), up0 = add0 + up, up1 = add1 + up;
                    u[i][0] = fast_exp2(u[i][0] + up0), u[i][1] = fast_exp2(u[i][1] + up1);
                    u[i][2] = fast_exp2(u[i][2] + up0), u[i][3] = fast_exp2(u[i][3] + up1);
                    l0 = fmaf(u[i][0] + u[i][2], sc[i].inv_2e, l0);
                    l1 = fmaf(u[i][1] + u[i][3], sc[i].inv_2e, l1);
                    uint32_t p[4];
                    split_pair_f16(u[i][0] * sc[i].f, u[i][1] * sc[i].f, p[0], p[1]);
                    split_pair_f16(u[i][2] * sc[i].f, u[i][3] * sc[i].f, p[2], p[3]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) p[j] = transposed(p[j]);
                    weigh<D, KIND>(kst + (2 + i) * C::SLAB, valid[i], p, o, at, t);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.oempty[warp * C::ORDERS + taken % C::ORDERS]);
                ++taken;
            }
            if (!ok) break;
            // This warp's state joins its slot for the merger: (m, l) and O of heads
            // 2t and 2t + 1, each lane its D / 8 dims.  The first time the slot is
            // waited for and set, then it is added to (m never falls).
            if (!begun && !mbar_wait_warp(&B.mempty[buf], ((item_seq / C::MERGE_BUFS) & 1) ^ 1)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                l0 += __shfl_xor_sync(FULL, l0, off);
                l1 += __shfl_xor_sync(FULL, l1, off);
            }
            const size_t base = static_cast<size_t>((buf * C::W + warp) * G + 2 * t);
            if (begun) {  // warp-uniform
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (2 * t + e >= G) continue;
                    const float2 was = ml[base + e];
                    const Halves f(was.x - (e ? m1 : m0));
                    const float keep = f.whole();
                    (e ? l1 : l0) += f.times(was.y);
                    const float4* src = reinterpret_cast<const float4*>(mo + (base + e) * D + g * (D / 8));
#pragma unroll
                    for (int j = 0; j < D / 16; j += 2) {
                        const float4 w = src[j / 2];
                        o[j][e] = fmaf(w.x, keep, o[j][e]), o[j][2 + e] = fmaf(w.y, keep, o[j][2 + e]);
                        o[j + 1][e] = fmaf(w.z, keep, o[j + 1][e]), o[j + 1][2 + e] = fmaf(w.w, keep, o[j + 1][2 + e]);
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (2 * t + e < G) {
                    if (g == 0) ml[base + e] = make_float2(e ? m1 : m0, e ? l1 : l0);
                    float* dst = mo + (base + e) * D + g * (D / 8);
#pragma unroll
                    for (int j = 0; j < D / 16; j += 2)
                        *reinterpret_cast<float4*>(dst + 2 * j) =
                            make_float4(o[j][e], o[j][2 + e], o[j + 1][e], o[j + 1][2 + e]);
                }
            }
        } while (b < nst);
        if (!ok) break;
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.mfull[buf]);
        ++item_seq;
    }
    if (!ok) {
        *abort_flag = 1;
        record_error(P.err, kErrTimeout, 2u);
        // Never leave with copies still in flight.
        for (; taken != issued; ++taken) mbar_wait(&full[taken % C::SW], (taken / C::SW) & 1);
    }
}

template <int D, int G, int KIND>
__global__ void __launch_bounds__(ScaledCfg<D, G, KIND>::THREADS, 1)
    decode_scaled_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                         const DecodeParams P) {
    using C = ScaledCfg<D, G, KIND>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    Bars B;
    B.full = bars;
    B.empty = nullptr;  // a consumer warp fills its own stages
    B.ifull = bars + C::STAGES;
    B.iempty = B.ifull + kItemRing;
    B.mfull = B.iempty + kItemRing;
    B.mempty = B.mfull + C::MERGE_BUFS;
    B.ofull = B.mempty + C::MERGE_BUFS;
    B.oempty = B.ofull + C::W * C::ORDERS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    // One arrival completes every barrier but three kinds: consumers and mergers
    // hand a descriptor back, the consumers fill a merge buffer and the mergers
    // empty it.
    for (int i = threadIdx.x; i < C::NBAR; i += C::THREADS) {
        const bool iempty = &bars[i] >= B.iempty && &bars[i] < B.iempty + kItemRing;
        const bool mfull = &bars[i] >= B.mfull && &bars[i] < B.mfull + C::MERGE_BUFS;
        const bool mempty = &bars[i] >= B.mempty && &bars[i] < B.mempty + C::MERGE_BUFS;
        mbar_init(&bars[i], iempty ? C::W + C::MERGERS : mfull ? C::W : mempty ? C::MERGERS : 1);
    }
    if (threadIdx.x == 0) *abort_flag = 0;
    fence_mbar_init();
    griddep_launch_dependents();
    __syncthreads();
    // Until griddep_wait() returns, only L2 prefetches touch global memory.
    if (warp == C::PRODUCER_WARP) {
        griddep_wait();
        if (!P.stall) run_producer<C, false>(P, &tm_k, &tm_v, smem, B, abort_flag, lane);
    } else if (warp >= C::MERGER_WARP) {
        if (warp == C::MERGER_WARP) prefetch_first_blocks<D, G, 1>(P, lane, 2 * C::STAGES);
        griddep_wait();
        run_merger<C>(P, smem, B, abort_flag, lane, warp - C::MERGER_WARP);
    } else {
        prefetch_inputs<D, false>(P, threadIdx.x, C::W * 32);
        griddep_wait();  // consumers read the pools themselves
        run_consumer_scaled<C, KIND>(P, &tm_k, &tm_v, smem, B, abort_flag, warp, lane);
    }
}

template <int D, int G, int KIND>
cudaError_t launch_scaled_one(DecodeParams P, int grid, cudaStream_t stream) {
    using C = ScaledCfg<D, G, KIND>;
    if (P.range_units <= 0) P.extra_units = C::EXTRA_UNITS;
    // Rows of D bytes, 16 a slab, one slab per (block, kv head).
    CUtensorMap tk, tv;
    const cuuint64_t slabs = static_cast<cuuint64_t>(P.num_blocks) * P.hkv;
    const cuuint64_t dims[3] = {D, kBlockSize, slabs > 0 ? slabs : 1};
    const cuuint64_t strides[2] = {D, D * kBlockSize};
    const cuuint32_t box[3] = {D, kBlockSize, 1};
    const CUtensorMapSwizzle swizzle = D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_tile_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, P.k_pool, 3, dims, strides, box, swizzle) ||
        !make_tile_map(&tv, CU_TENSOR_MAP_DATA_TYPE_UINT8, P.v_pool, 3, dims, strides, box, swizzle))
        return cudaErrorInvalidValue;
    static bool configured[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 0 && dev < 64 && !configured[dev]) {
        cudaError_t e = cudaFuncSetAttribute(decode_scaled_kernel<D, G, KIND>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        configured[dev] = true;
    }
    return launch_overlapped(decode_scaled_kernel<D, G, KIND>, dim3(grid), dim3(C::THREADS), C::SMEM, stream, tk, tv,
                             P);
}

template <int D, int KIND>
cudaError_t dispatch_scaled_g(const DecodeParams& P, int G, int grid, cudaStream_t stream) {
    switch (G) {
        case 1: return launch_scaled_one<D, 1, KIND>(P, grid, stream);
        case 2: return launch_scaled_one<D, 2, KIND>(P, grid, stream);
        case 4: return launch_scaled_one<D, 4, KIND>(P, grid, stream);
        case 8: return launch_scaled_one<D, 8, KIND>(P, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int KIND>
cudaError_t launch_decode_scaled_kind(const DecodeArgs& a, bool stall, cudaStream_t stream) {
    const DecodeParams P = decode_params(a, stall);
    const int G = a.num_q_heads / a.num_kv_heads;
    return a.head_dim == 128 ? dispatch_scaled_g<128, KIND>(P, G, a.plan.grid, stream)
                             : dispatch_scaled_g<64, KIND>(P, G, a.plan.grid, stream);
}

}  // namespace
}  // namespace pkv
