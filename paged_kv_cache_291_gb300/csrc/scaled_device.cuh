// scaled_device.cuh -- 8-bit pools with a scale for each (block, kv head):
// codes to and from fp32, the scale's rule, and the search for the sequence a
// block belongs to.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pkv_device.cuh"

namespace pkv {

// Element kinds, as the kernels are instantiated (pkv_cache_t.kv_dtype).
constexpr int kKindBf16 = 0, kKindE4m3 = 1, kKindE4m3Blocks = 2, kKindInt8Blocks = 3;

constexpr float kLeastScale = 0x1p-100f, kMostScale = 0x1p122f;

// The largest code of a kind, and its reciprocal rounded to fp32.
template <int KIND>
constexpr float code_max() { return KIND == kKindInt8Blocks ? 127.f : 448.f; }
template <int KIND>
constexpr float inv_code_max() { return 1.f / code_max<KIND>(); }

// A stored scale as the calls use it: 2^-100 to 2^122 (the append's are in
// there for every bf16 value); anything else (`bad` is then set) counts as
// 2^-100.
__device__ __forceinline__ float checked_scale(float s, bool& bad) {
    const bool ok = s >= kLeastScale && s <= kMostScale;
    bad |= !ok;
    return ok ? s : kLeastScale;
}

// Four codes (bytes of w, lowest first) to fp32, exactly.
template <int KIND>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
    if constexpr (KIND == kKindInt8Blocks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
    } else {
        uint32_t h[2];
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h[0]), "=r"(h[1])
            : "r"(w));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
                : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
                : "r"(h[i]));
    }
}

// Four fp32 to the nearest codes, ties to even, saturating; a NaN gives the
// NaN code of e4m3 (int8 has none: callers hand it no NaN).
template <int KIND>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
    if constexpr (KIND == kKindInt8Blocks) {
        const float x[4] = {a, b, c, d};
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(x[i], -127.f), 127.f)));
        return __byte_perm(__byte_perm(r[0], r[1], 0x0040), __byte_perm(r[2], r[3], 0x0040), 0x5410);
    } else {
        return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
    }
}

// The sequence that owns unit u of a batch's block units, for a whole warp:
// sequence s owns units start[s] / 16 + 2 s and on, one for each block its
// new rows touch (rows + 14 more can touch (rows + 30) / 16 blocks, and the
// next sequence's units start at least rows / 16 + 2 later).  Returns the
// last sequence whose first unit is not above u.
__device__ __forceinline__ int sequence_of_unit(const int32_t* start, int num_seqs, int u, int lane) {
    int lo = 0, hi = num_seqs;  // the answer is in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int s = lo + lane * step;
        const bool below = s < hi && static_cast<long long>(__ldg(start + s)) / kBlockSize + 2ll * s <= u;
        const unsigned votes = __ballot_sync(0xffffffffu, below);
        const int last = votes ? 31 - __clz(votes) : 0;
        lo = lo + last * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

}  // namespace pkv
