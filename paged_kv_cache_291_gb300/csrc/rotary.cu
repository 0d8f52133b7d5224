// rotary.cu -- rotary positions with one to four axes, and the same fused
// with the store of the step's K and V rows in the paged pool.
//
// Mathematics.  Pair i of a row is turned by the angle
//     a(t, i) = positions[axis(i)][t] * inv_freq[i],
//     (x, y) -> (x cos a - y sin a, x sin a + y cos a).
// The fp32 product position * inv_freq is off by up to 2^-24 of the angle,
// which at position 10^6 is 0.06 radian, so the angle is formed in turns in
// 64-bit fixed point instead: F = frac(inv_freq / 2 pi) * 2^64, and
// position * F modulo 2^64 is the fraction of a turn, with no reduction step
// (the wrap of the integer product is the reduction).  inv_freq / 2 pi is an
// fp32 pair product (2^-48 relative), so the angle is off by at most
// 2^-48 |position * inv_freq|: 2^-28 radian at position 2^20, frequency 1.
// cos and sin of the top 32 bits come from sincospif.  The rotation is fp32
// and rounds once, to bf16 or (e4m3 pools) straight to the 8-bit code.
//
// Layout.  A warp takes one token and a run of its rows (q heads, then k
// heads, then v heads for the cache write).  A lane owns 16 elements of a
// row, loaded as two 16-byte vectors that hold 8 pairs (dims 8j and p + 8j
// of the halves, or 16j and 16j + 8 when pairs are adjacent), so d/16 lanes
// share a row and 512/d rows go side by side.  The lanes that hold the same
// pairs of different rows split their sines and cosines and trade them by
// shuffles; the values stay in registers for all the warp's rows.
//
// Bound: HBM (each row is read and written once; ~1 flop per byte).  16,381
// tokens of 80 rows of 128: 671 MB in 98.5 us, 6.8 TB/s, the rate of a copy;
// 2,048 tokens of 16/8 heads into the cache 6.1 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kWarps = 4;    // warps per CTA, each with its own (token, run of rows)
constexpr int kRowsAhead = 2;  // row groups whose loads are in flight together

// cos and sin of 2 pi * frac(pos * inv_freq / 2 pi).
__device__ __forceinline__ void turn_of(float f, int32_t pos, float& c, float& s) {
    constexpr double kInvTwoPi = 0.15915494309189533576888;
    constexpr float kHi = static_cast<float>(kInvTwoPi);
    constexpr float kLo = static_cast<float>(kInvTwoPi - static_cast<double>(kHi));
    float hi = f * kHi;
    float lo = fmaf(f, kLo, fmaf(f, kHi, -hi));
    hi -= rintf(hi);  // exact; whole turns do not matter
    lo -= rintf(lo);  // above 2^23 turns a step this part has some too
    const long long step = __float2ll_rn(hi * 0x1p64f) + __float2ll_rn(lo * 0x1p64f);
    const unsigned long long turns =
        static_cast<unsigned long long>(step) * static_cast<unsigned long long>(static_cast<long long>(pos));
    const float half_turns = static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
    sincospif(half_turns, &s, &c);
    if (!(fabsf(f) <= 3.402823466e38f)) c = s = __int_as_float(0x7fffffff);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16lo(w[i]);
        x[2 * i + 1] = bf16hi(w[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv));
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Mode: 0 rotate q and k into q_out and k_out; 1 k and v to a bf16 pool;
// 2 k and v to an e4m3 pool.
template <int D, int MODE>
__global__ void __launch_bounds__(32 * kWarps) rotary_kernel(const RotaryArgs A) {
    constexpr int LPR = D / 16;     // lanes per row
    constexpr int ROWS = 32 / LPR;  // rows side by side
    constexpr int OWN = 8 / ROWS;   // pairs whose sine and cosine a lane computes
    griddep_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int j = lane % LPR, rep = lane / LPR;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    griddep_wait();
    const int64_t t = item / A.runs;
    if (t >= A.num_tokens) return;
    const int run = static_cast<int>(item - t * A.runs);
    const int rows = A.num_q_heads + (MODE == 0 ? 1 : 2) * A.num_kv_heads;
    const int row0 = run * A.rows_per_run;
    const int row1 = min(rows, row0 + A.rows_per_run);

    // Where the lane's two vectors sit in a row, and whether they turn.
    const int p = A.rot_dim / 2;
    const bool turns = A.adjacent ? 16 * j < A.rot_dim : 8 * j < p;
    const int e0 = turns && !A.adjacent ? 8 * j : 16 * j;
    const int e1 = turns && !A.adjacent ? p + 8 * j : 16 * j + 8;
    int64_t slot = 0;
    if (MODE != 0) {
        slot = __ldg(A.slot_mapping + t);
        if (slot >= A.num_slots) {
            if (run == 0 && lane == 0) record_error(A.err, kErrRange, static_cast<uint32_t>(t));
            slot = -1;
        }
    }
    const uint16_t* qt = A.q + t * A.q_stride;
    const uint16_t* kt = A.k + t * A.k_stride;
    const uint16_t* vt = MODE != 0 ? A.v + t * A.v_stride : nullptr;

    auto source = [&](int row) -> const uint16_t* {
        if (row < A.num_q_heads) return qt + static_cast<int64_t>(row) * D;
        row -= A.num_q_heads;
        if (MODE == 0 || row < A.num_kv_heads) return kt + static_cast<int64_t>(row) * D;
        return vt + static_cast<int64_t>(row - A.num_kv_heads) * D;
    };
    auto load = [&](int row, uint4& a, uint4& b) {
        if (row < row1) {
            const uint16_t* r = source(row);
            a = *reinterpret_cast<const uint4*>(r + e0);
            b = *reinterpret_cast<const uint4*>(r + e1);
        }
    };
    uint4 a[kRowsAhead], b[kRowsAhead];
#pragma unroll
    for (int n = 0; n < kRowsAhead; ++n) load(row0 + n * ROWS + rep, a[n], b[n]);

    // Sines and cosines of pairs 8j .. 8j+7, OWN of them computed here.
    float c[8], s[8];
    {
        float oc[OWN], os[OWN];
#pragma unroll
        for (int e = 0; e < OWN; ++e) {
            const int i = 8 * j + rep * OWN + e;
            oc[e] = 1.f;
            os[e] = 0.f;
            if (i < p) {
                const int axis = static_cast<int>(A.axis_of_pair[i >> 5] >> (2 * (i & 31))) & 3;
                turn_of(__ldg(A.inv_freq + i), __ldg(A.positions + axis * static_cast<int64_t>(A.num_tokens) + t),
                        oc[e], os[e]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c[i] = __shfl_sync(0xffffffffu, oc[i % OWN], (i / OWN) * LPR + j);
            s[i] = __shfl_sync(0xffffffffu, os[i % OWN], (i / OWN) * LPR + j);
        }
    }

    auto finish = [&](int row, uint4 ua, uint4 ub) {
        const int kv = row - A.num_q_heads;
        const bool is_v = MODE != 0 && kv >= A.num_kv_heads;
        float x[8], y[8];
        unpack8(ua, x);
        unpack8(ub, y);
        if (turns && !is_v) {
            if (A.adjacent) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = x[2 * i], p1 = x[2 * i + 1], r0 = y[2 * i], r1 = y[2 * i + 1];
                    x[2 * i] = fmaf(p0, c[i], -(p1 * s[i]));
                    x[2 * i + 1] = fmaf(p0, s[i], p1 * c[i]);
                    y[2 * i] = fmaf(r0, c[4 + i], -(r1 * s[4 + i]));
                    y[2 * i + 1] = fmaf(r0, s[4 + i], r1 * c[4 + i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = x[i], w = y[i];
                    x[i] = fmaf(u, c[i], -(w * s[i]));
                    y[i] = fmaf(u, s[i], w * c[i]);
                }
            }
            if (MODE != 2 || kv < 0) {
                ua = pack8(x);
                ub = pack8(y);
            }
        }
        if (kv < 0 || MODE == 0) {
            uint16_t* o = kv < 0 ? A.q_out + (t * A.num_q_heads + row) * D : A.k_out + (t * A.num_kv_heads + kv) * D;
            *reinterpret_cast<uint4*>(o + e0) = ua;
            *reinterpret_cast<uint4*>(o + e1) = ub;
            return;
        }
        if (slot < 0) return;
        const int h = is_v ? kv - A.num_kv_heads : kv;
        const int64_t at = (((slot / kBlockSize) * A.num_kv_heads + h) * kBlockSize + slot % kBlockSize) * D;
        if (MODE == 1) {
            uint16_t* o = static_cast<uint16_t*>(is_v ? A.v_pool : A.k_pool) + at;
            *reinterpret_cast<uint4*>(o + e0) = ua;
            *reinterpret_cast<uint4*>(o + e1) = ub;
        } else {
            uint8_t* o = static_cast<uint8_t*>(is_v ? A.v_pool : A.k_pool) + at;
            const float inv = is_v ? A.v_inv : A.k_inv;
            *reinterpret_cast<uint2*>(o + e0) = codes8(x, inv);
            *reinterpret_cast<uint2*>(o + e1) = codes8(y, inv);
        }
    };
    for (int row = row0 + rep; row < row1; row += kRowsAhead * ROWS) {
#pragma unroll
        for (int n = 0; n < kRowsAhead; ++n) {
            const uint4 ua = a[n], ub = b[n];
            load(row + (n + kRowsAhead) * ROWS, a[n], b[n]);
            if (row + n * ROWS < row1) finish(row + n * ROWS, ua, ub);
        }
    }
}

template <int D, int MODE>
cudaError_t launch(const RotaryArgs& a, cudaStream_t stream) {
    const int64_t items = static_cast<int64_t>(a.num_tokens) * a.runs;
    return launch_overlapped(rotary_kernel<D, MODE>, dim3(static_cast<unsigned>((items + kWarps - 1) / kWarps)),
                             dim3(32 * kWarps), 0, stream, a);
}

}  // namespace

cudaError_t launch_rotary(RotaryArgs a, int num_sms, cudaStream_t stream) {
    const int mode = a.k_pool == nullptr ? 0 : a.kv_e4m3 ? 2 : 1;
    const int rows = a.num_q_heads + (mode == 0 ? 1 : 2) * a.num_kv_heads;
    const int side = 512 / a.head_dim;  // rows a warp holds side by side
    const int groups = (rows + side - 1) / side;
    // A warp's sines and cosines serve all its rows, so a token goes to one
    // warp where there are tokens enough for 16 warps an SM, and to more where
    // not; a warp that takes more than 7 row groups ends too long after the
    // others.
    const int64_t want = static_cast<int64_t>(num_sms) * 16;
    int64_t runs = (want + a.num_tokens - 1) / a.num_tokens;
    runs = runs > (groups + 6) / 7 ? runs : (groups + 6) / 7;
    if (runs > groups) runs = groups;
    a.rows_per_run = static_cast<int32_t>((groups + runs - 1) / runs) * side;
    a.runs = (rows + a.rows_per_run - 1) / a.rows_per_run;
    if (a.head_dim == 64)
        return mode == 0 ? launch<64, 0>(a, stream) : mode == 1 ? launch<64, 1>(a, stream) : launch<64, 2>(a, stream);
    return mode == 0 ? launch<128, 0>(a, stream) : mode == 1 ? launch<128, 1>(a, stream) : launch<128, 2>(a, stream);
}

}  // namespace pkv
