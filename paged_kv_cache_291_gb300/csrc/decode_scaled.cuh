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
//    four swizzled 16-row tiles and the two pairs of scales.  Twice the keys
//    of a stage of the other pools: the maximum's shuffles, the wait and the
//    hand-back are paid once for 32 keys, and the two blocks' chains of MMAs
//    run side by side.
//  * S = Q K^T (m16n8k16): rows 0-7 are the group's heads (the rest of the
//    rows, and heads the group lacks, are zero), columns eight keys.  Lane
//    (g, t) = (lane / 4, lane % 4) then holds head g's scores of keys 2t and
//    2t + 1 of each tile: the layout of the A operand of P V, so P moves to no
//    other lane, and a row's maximum takes two shuffles.
//  * O += P V: an fp16 P would be off by 2^-11; the rows that the heads leave
//    free carry the rest instead: rows 0-7 are P rounded to fp16, rows 8-15
//    what the rounding lost, so P goes to 2^-22 in the same MMAs.  The two
//    halves of O are added when the warp hands its state over.
//  * Weights of a block carry its V scale, vs = f 2^e with f in [1, 2): the
//    running maximum is that of s_j + e, u = 2^(s_j + e - m + 11), the weight
//    u f and the term of the sum u 2^-e, so scales far apart lose nothing, and
//    weights end 2^-36 below the largest (fp16 is exact to 2^-24).
//  * The order of dims in S and of keys in P V is free: a lane reads whole
//    16-byte pieces of K rows and of V rows (8-byte pieces of V at head_dim
//    64), and rows are dealt to lanes so that the lanes that read together hit
//    different banks of the swizzled tiles (see key_row).
#pragma once

#include "decode_kernel.cuh"
#include "scaled_device.cuh"

namespace pkv {
namespace {

template <int D, int G, int KIND>
struct ScaledCfg {
    static constexpr int HEAD_DIM = D, GROUP = G, ELEM = 1;
    static constexpr bool SCALED = true, MMA = true;
    static constexpr int BPS = 2;
#ifdef PKV_SCALED_WARPS
    static constexpr int W = PKV_SCALED_WARPS;
#else
    static constexpr int W = 8;  // consumer warps
#endif
    static constexpr int MERGE_LANES = W <= 8 ? 8 : 16;
    static constexpr int MERGE_BUFS = 1;
    static constexpr int PRODUCER_WARP = W, MERGER_WARP = W + 1, THREADS = 32 * (W + 2);
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
    // 226 KB less the regions above, 64 barriers beside the stages' own, the
    // flag and the 1,024-byte alignment of the ring.
    static constexpr int STAGES_FIT = (226 * 1024 - R_BAR - 64 * 8 - 32 - 1024) / (STAGE_BYTES + 16 + 16);
    static constexpr int SW_FIT = STAGES_FIT / W;
    static constexpr int SW = SW_FIT < 6 ? SW_FIT : 6;
    static constexpr int STAGES = SW * W;
    static constexpr int NBAR = 2 * STAGES + 2 * kItemRing + 2 * MERGE_BUFS;
    static constexpr int OFF_REST = STAGES * STAGE_BYTES;
    static constexpr int OFF_ITEMQ = OFF_REST + R_ITEMQ;
    static constexpr int OFF_DESC = OFF_REST + R_DESC;
    static constexpr int OFF_MO = OFF_REST + R_MO;
    static constexpr int OFF_ML = OFF_REST + R_ML;
    static constexpr int OFF_WT = OFF_REST + R_WT;
    static constexpr int OFF_MSM = OFF_REST + R_MSM;
    static constexpr int OFF_BAR = OFF_REST + R_BAR;
    static constexpr int OFF_FLAG = OFF_BAR + NBAR * 8;
    static constexpr int OFF_SCALES = align_up(OFF_FLAG + 4, 16);  // [STAGES] two (K, V) pairs
    static constexpr int OFF_NEW = OFF_SCALES;                     // of fused steps only, which there are none of
    static constexpr int SMEM = OFF_SCALES + STAGES * 16 + 1024;
    static_assert(SW >= 1, "ring too shallow");
    static_assert(OFF_ITEMQ % 16 == 0 && OFF_DESC % 16 == 0 && OFF_MO % 16 == 0 && OFF_ML % 8 == 0 &&
                      OFF_MSM % 8 == 0 && OFF_BAR % 8 == 0 && STAGE_BYTES % 1024 == 0 && SLAB % 512 == 0,
                  "shared-memory regions aligned for their widest access");
    static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// P's exponent against the running maximum: a weight is below 2^(3 + 11 + 1).
constexpr float kScaledThreshold = 3.0f, kScaledShift = 11.0f;

// Byte offset of 16-byte chunk c of row r of a swizzled slab: rows of 128
// bytes with chunks XORed by r mod 8, rows of 64 bytes with chunks XORed by
// (r / 2) mod 4.
template <int D>
__device__ __forceinline__ uint32_t slab_at(int r, int c) {
    return D == 128 ? static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4))
                    : static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

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

// S tile: eight keys (rows key_row(0..7) + 8 half of the slab).
template <int D, int KIND>
__device__ __forceinline__ void scores(const uint8_t* k, int half, const uint32_t (&qa)[D / 8], float (&s)[4], int g,
                                       int t) {
    s[0] = s[1] = s[2] = s[3] = 0.f;
    const int row = 8 * half + key_row<D>(g);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        const uint4 u = lds128(k + slab_at<D>(row, D == 128 ? 2 * t + c : t));
        const uint32_t w[4] = {turned<KIND>(u.x), turned<KIND>(u.y), turned<KIND>(u.z), turned<KIND>(u.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            mma_f16(s, qa[2 * (4 * c + i)], 0u, qa[2 * (4 * c + i) + 1], 0u, widen2<KIND, false>(w[i]),
                    widen2<KIND, true>(w[i]));
    }
}

// O += P V over one block: p[0..1] the hi and lo pair of the keys of half 0,
// p[2..3] of half 1.  Rows past the context are zero where their codes could
// be NaN.
template <int D, int KIND>
__device__ __forceinline__ void weigh(const uint8_t* v, int valid, const uint32_t (&p)[4], float (&o)[D / 8][4], int g,
                                      int t) {
    constexpr int NW = D / 32;  // words of a lane's D / 8 dims
    uint32_t w[4][NW];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int row = 8 * (j >> 1) + key_row<D>(2 * t + (j & 1));
        if constexpr (D == 128) {
            const uint4 u = lds128(v + slab_at<D>(row, g));
            w[j][0] = u.x, w[j][1] = u.y, w[j][2] = u.z, w[j][3] = u.w;
        } else {
            const uint2 u = lds64(v + slab_at<D>(row, g >> 1) + 8 * (g & 1));
            w[j][0] = u.x, w[j][1] = u.y;
        }
        if (KIND != kKindInt8Blocks && valid < kBlockSize) {
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
            mma_f16(o[4 * i + 2 * x], p[0], p[1], p[2], p[3], widen2<KIND, false>(a), widen2<KIND, false>(b));
            mma_f16(o[4 * i + 2 * x + 1], p[0], p[1], p[2], p[3], widen2<KIND, true>(a), widen2<KIND, true>(b));
        }
    }
}

template <class C, int KIND>
__device__ void run_consumer_scaled(const DecodeParams& P, uint8_t* smem, const Bars& B, volatile int* abort_flag,
                                    int warp, int lane) {
    constexpr int D = C::HEAD_DIM, G = C::GROUP;
    constexpr int QW = D / 8;   // q words of a lane: its D / 4 dims
    const unsigned FULL = 0xffffffffu;
    const ItemDesc* descs = reinterpret_cast<const ItemDesc*>(smem + C::OFF_DESC);
    float* mo = reinterpret_cast<float*>(smem + C::OFF_MO);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int g = lane >> 2, t = lane & 3;
    uint32_t taken = 0, item_seq = 0;
    bool ok = true;
    while (ok) {
        const uint32_t slot = item_seq % kItemRing;
        if (*abort_flag || !mbar_wait_warp(&B.ifull[slot], (item_seq / kItemRing) & 1)) {
            ok = false;
            break;
        }
        const ItemDesc d = descs[slot];
        if (d.s < 0) break;
        // q of head g, dims (D / 4) t and on, as the A operand (zero for g >=
        // G), scaled by a power of two so that the largest is in [2^14, 2^15)
        // of fp16; the scores get the factor back.
        uint32_t qa[QW];
        float f;
        {
            const uint8_t* qs = smem + C::OFF_ITEMQ + slot * C::QBYTES + (g * D + t * (D / 4)) * 2;
#pragma unroll
            for (int c = 0; c < QW / 4; ++c) {
                uint4 u = make_uint4(0u, 0u, 0u, 0u);
                if (g < G) u = lds128(qs + 16 * c);
                qa[4 * c] = u.x, qa[4 * c + 1] = u.y, qa[4 * c + 2] = u.z, qa[4 * c + 3] = u.w;
            }
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < QW; ++i) mx = fmaxf(mx, fmaxf(fabsf(bf16lo(qa[i])), fabsf(bf16hi(qa[i]))));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
            int e = 0;
            if (mx < INFINITY) e = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
            const float down = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
            const float up = __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
            for (int i = 0; i < QW; ++i) qa[i] = f16x2_rn(bf16lo(qa[i]) * down, bf16hi(qa[i]) * down);
            f = P.scale_log2 * up;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.iempty[slot]);
        float m = -INFINITY, l = 0.f;
        float o[D / 8][4];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
        const int nst = (d.b1 - d.b0 + 1) / 2;
        const int first = (warp - d.rot + C::W) % C::W;
        for (int b = first; b < nst; b += C::W) {
            const uint32_t st = static_cast<uint32_t>(warp * C::SW) + taken % C::SW;
            if (*abort_flag || !mbar_wait_warp(&B.full[st], (taken / C::SW) & 1)) {
                ok = false;
                break;
            }
            const int blk = d.b0 + 2 * b;
            const int keys = min(2 * kBlockSize, (min(d.b1 * kBlockSize, d.n) - blk * kBlockSize));
            const int valid[2] = {min(keys, kBlockSize), max(keys - kBlockSize, 0)};
            const uint8_t* kst = smem + st * C::STAGE_BYTES;
            float4 sc = *reinterpret_cast<const float4*>(smem + C::OFF_SCALES + st * 16);
            if (valid[1] == 0) sc.z = sc.w = 1.f;
            bool bad = false;
            const float ks[2] = {checked_scale(sc.x, bad), checked_scale(sc.z, bad)};
            const float vs[2] = {checked_scale(sc.y, bad), checked_scale(sc.w, bad)};
            if (bad && lane == 0) record_error(P.err, kErrRange, static_cast<uint32_t>(d.s));
            // Scores of keys 8 half + key_row(2t), key_row(2t + 1) of each block.
            float x[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float s[4];
                    scores<D, KIND>(kst + i * C::SLAB, half, qa, s, g, t);
                    x[i][2 * half] = s[0], x[i][2 * half + 1] = s[1];
                }
            }
            float mb = -INFINITY, ve[2], vf[2], back[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t bits = __float_as_uint(vs[i]);
                const int e = static_cast<int>(bits >> 23) - 127;
                ve[i] = static_cast<float>(e);
                vf[i] = __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
                back[i] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                const float kf = f * ks[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[i][j] *= kf;
                    if (valid[i] < kBlockSize && 8 * (j >> 1) + key_row<D>(2 * t + (j & 1)) >= valid[i])
                        x[i][j] = -INFINITY;
                }
                mb = fmaxf(mb, fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])) + ve[i]);
            }
            mb = fmaxf(mb, __shfl_xor_sync(FULL, mb, 1));
            mb = fmaxf(mb, __shfl_xor_sync(FULL, mb, 2));
            const bool moves = mb > m + kScaledThreshold;
            if (__any_sync(FULL, moves)) {
                const float a = moves ? fast_exp2(m - mb) : 1.f;
                m = moves ? mb : m;
                l *= a;
#pragma unroll
                for (int j = 0; j < D / 8; ++j) o[j][0] *= a, o[j][1] *= a, o[j][2] *= a, o[j][3] *= a;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i == 1 && valid[1] == 0) break;
                const float add = ve[i] + kScaledShift - m;
                float u[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) u[j] = fast_exp2(x[i][j] + add);
                l = fmaf((u[0] + u[1]) + (u[2] + u[3]), back[i], l);
                uint32_t p[4];
                split_pair_f16(u[0] * vf[i], u[1] * vf[i], p[0], p[1]);
                split_pair_f16(u[2] * vf[i], u[3] * vf[i], p[2], p[3]);
                weigh<D, KIND>(kst + (2 + i) * C::SLAB, valid[i], p, o, g, t);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.empty[st]);
            ++taken;
        }
        if (!ok) break;
        // This warp's state for the merger: lane (g, t) has dims (D / 4) t
        // and on of head g, D / 8 of them in the first accumulator of each
        // pair and D / 8 in the second.
        const int buf = item_seq % C::MERGE_BUFS;
        if (!mbar_wait_warp(&B.mempty[buf], ((item_seq / C::MERGE_BUFS) & 1) ^ 1)) {
            ok = false;
            break;
        }
        l += __shfl_xor_sync(FULL, l, 1);
        l += __shfl_xor_sync(FULL, l, 2);
        if (g < G) {
            const size_t base = static_cast<size_t>((buf * C::W + warp) * G + g);
            if (t == 0) ml[base] = make_float2(m, l);
            float* dst = mo + base * D + t * (D / 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int j = 0; j < D / 8; j += 4)
                    *reinterpret_cast<float4*>(dst + e * (D / 8) + j) =
                        make_float4(o[j][e] + o[j][2 + e], o[j + 1][e] + o[j + 1][2 + e],
                                    o[j + 2][e] + o[j + 2][2 + e], o[j + 3][e] + o[j + 3][2 + e]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.mfull[buf]);
        ++item_seq;
    }
    if (!ok) {
        *abort_flag = 1;
        record_error(P.err, kErrTimeout, 2u);
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
    B.empty = bars + C::STAGES;
    B.ifull = bars + 2 * C::STAGES;
    B.iempty = B.ifull + kItemRing;
    B.mfull = B.iempty + kItemRing;
    B.mempty = B.mfull + C::MERGE_BUFS;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_FLAG);
    const int warp = threadIdx.x / 32;
    const int lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&B.full[i], 2);  // the tiles' bytes, the scales
            mbar_init(&B.empty[i], 1);
        }
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(&B.ifull[i], 1);
            mbar_init(&B.iempty[i], C::W + 1);
        }
        for (int i = 0; i < C::MERGE_BUFS; ++i) {
            mbar_init(&B.mfull[i], C::W);
            mbar_init(&B.mempty[i], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    griddep_launch_dependents();
    __syncthreads();
    // Until griddep_wait() returns, only L2 prefetches touch global memory.
    if (warp == C::PRODUCER_WARP) {
        griddep_wait();
        if (!P.stall) run_producer<C, false>(P, &tm_k, &tm_v, smem, B, abort_flag, lane);
    } else if (warp == C::MERGER_WARP) {
        prefetch_first_blocks<D, G, 1>(P, lane, 2 * C::STAGES);
        griddep_wait();
        run_merger<C>(P, smem, B, abort_flag, lane);
    } else {
        prefetch_inputs<D, false>(P, threadIdx.x, C::W * 32);
        run_consumer_scaled<C, KIND>(P, smem, B, abort_flag, warp, lane);
    }
}

template <int D, int G, int KIND>
cudaError_t launch_scaled_one(const DecodeParams& P, int grid, cudaStream_t stream) {
    using C = ScaledCfg<D, G, KIND>;
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
