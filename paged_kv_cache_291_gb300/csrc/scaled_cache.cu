// scaled_cache.cu -- the write into 8-bit pools with a scale for each (block,
// kv head), and the read of rows from a pool of any kind.
//
// cache_append: per (block, kv head) that the step's new rows touch, K and V
// apart,
//     scale = max(old, amax / L, 2^-100),  code(x) = nearest(x / scale)
// (L the largest code), and where the scale has grown over that of the rows
// already in the block, code' = nearest(value(code) old / scale) for those.
// cache_read: value(code) * scale, rounded to bf16.
//
// Both move bytes: 2 read and 1 written per element and the other way round,
// so HBM bounds them once there are a few thousand rows, and the chain start
// -> length -> table -> scale -> rows below that.  A warp takes the 16 rows of
// one (block, kv head), K or V: the rows of a block are what shares a scale,
// so the largest value, the codes and the scale need no other warp, and the
// codes are one contiguous run of the pool.  All rows of the warp are loaded
// before the first is used (8 loads of 16 bytes a lane at head_dim 128).
// Measured: append of 16,381 rows of 40 heads x 128 (503 MB) 77.3 us, 0.96 of
// the copy rate; read of 30,000 such rows (921 MB) 137 to 141 us, 0.97 to 1.00.
// No gain from persistent CTAs, several jobs a warp in turn, or earlier rows'
// codes loaded together with the new rows (79.2 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "scaled_device.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;

struct RowsParams {
    uint8_t* k_pool;
    uint8_t* v_pool;
    float* scales;             // [num_blocks][hkv][2]
    const uint16_t* k_new;     // append
    const uint16_t* v_new;
    uint16_t* k_out;           // read
    uint16_t* v_out;
    int64_t k_stride, v_stride;
    const int32_t* start;      // [num_seqs + 1]
    const int32_t* context_lens;
    const int32_t* block_tables;
    unsigned long long* err;
    int32_t num_tokens, num_seqs, max_blocks, num_blocks, hkv;
    float k_scale, v_scale;    // pools with one scale
};

// The rows of one block of a sequence that a call stores or reads.
struct UnitRows {
    int s;
    int first, last;  // rows of the block, [first, last)
    int token;        // of row `first`
    int phys;         // -1: block id out of range
    bool valid;       // the sequence's arguments are in range (else: no block, rows of `token` on)
};

// Whether sequence s's rows and context are in range.
__device__ __forceinline__ bool sequence_fits(const RowsParams& P, int a, int b, int n) {
    return a >= 0 && b >= a && b <= P.num_tokens &&
           (b == a || (n >= b - a && n <= static_cast<long long>(P.max_blocks) * kBlockSize));
}

// Unit u of the batch; false if it has no rows.
__device__ __forceinline__ bool find_rows(const RowsParams& P, int u, int lane, UnitRows& r) {
    const int s = sequence_of_unit(P.start, P.num_seqs, u, lane);
    const int a = __ldg(P.start + s), b = __ldg(P.start + s + 1), n = __ldg(P.context_lens + s);
    const long long j = u - (static_cast<long long>(a) / kBlockSize + 2ll * s);
    if (j < 0 || b <= a) return false;
    r.s = s;
    r.valid = sequence_fits(P, a, b, n);
    if (!r.valid) {
        // For the read: rows 16 j .. of the sequence's own, where they are
        // rows of the call.
        if (a < 0 || b > P.num_tokens) return false;
        const long long at = a + j * kBlockSize;
        if (at >= b) return false;
        r.token = static_cast<int>(at);
        r.first = 0;
        r.last = static_cast<int>(min(static_cast<long long>(kBlockSize), b - at));
        r.phys = -1;
        return true;
    }
    const int at = n - (b - a);  // position of the sequence's first row
    const int blk = at / kBlockSize + static_cast<int>(j);
    if (blk * static_cast<long long>(kBlockSize) >= n) return false;
    r.first = max(at - blk * kBlockSize, 0);
    r.last = min(n - blk * kBlockSize, kBlockSize);
    r.token = a + blk * kBlockSize + r.first - at;
    r.phys = __ldg(P.block_tables + static_cast<size_t>(s) * P.max_blocks + blk);
    if (r.phys < 0 || r.phys >= P.num_blocks) {
        if (lane == 0 && blockIdx.y == 0) record_error(P.err, kErrRange, static_cast<uint32_t>(s));
        r.phys = -1;
    }
    return true;
}

// The first CTA looks at every sequence's arguments; the others skip what is
// out of range.
__device__ __forceinline__ void check_sequences(const RowsParams& P) {
    for (int s = threadIdx.x; s < P.num_seqs; s += kWarps * 32) {
        const int a = __ldg(P.start + s), b = __ldg(P.start + s + 1);
        if (!sequence_fits(P, a, b, __ldg(P.context_lens + s)) || (s == 0 && a != 0))
            record_error(P.err, kErrRange, static_cast<uint32_t>(s));
    }
}

// Largest magnitudes of the halves of m and of 8 bf16, a NaN above all; the
// signs of the result mean nothing.
__device__ __forceinline__ uint32_t max_bf16_sizes(uint4 x, uint32_t m) {
    auto larger = [](uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    };
    return larger(larger(larger(larger(m, x.x), x.y), x.z), x.w);
}

__device__ __forceinline__ uint32_t warp_max_size(uint32_t m) {
    return __reduce_max_sync(0xffffffffu, max(m & 0x7fffu, (m >> 16) & 0x7fffu));
}

// A bf16 pair without its NaNs, and without its infinities too where FINITE.
template <bool FINITE>
__device__ __forceinline__ uint32_t tame(uint32_t x) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t v = (x >> (16 * i)) & 0xffffu, size = v & 0x7fffu;
        if (FINITE ? size < 0x7f80u : size <= 0x7f80u) r |= v << (16 * i);
    }
    return r;
}

template <bool FINITE>
__device__ __forceinline__ uint4 tame8(uint4 x) {
    return make_uint4(tame<FINITE>(x.x), tame<FINITE>(x.y), tame<FINITE>(x.z), tame<FINITE>(x.w));
}

// Eight values to codes under the scale 1 / inv.  WITHIN: none is above the
// largest code but for rounding, as where the scale comes from their own
// largest; int8 then needs no clamp, and the sum with 1.5 2^23 rounds to
// nearest even into its last byte (16,381 rows of 40 heads x 128: 94 us clamped
// and converted, the ALU 62 % busy, against 85.7).
template <int KIND, bool WITHIN>
__device__ __forceinline__ uint2 encode8(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float f[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            f[n] = __fmul_rn(n & 1 ? bf16hi(w[2 * i + n / 2]) : bf16lo(w[2 * i + n / 2]), inv);
        if constexpr (KIND == kKindInt8Blocks && WITHIN) {
            // Not in pairs: __fmul2_rn and __fadd2_rn came out fused, and a
            // product next to a tie then goes the other way.
            uint32_t u[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) u[n] = __float_as_uint(__fadd_rn(f[n], 0x1.8p23f));
            r[i] = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
        } else {
            r[i] = encode4<KIND>(f[0], f[1], f[2], f[3]);
        }
    }
    return make_uint2(r[0], r[1]);
}

// Codes encoded again under a scale 1 / ratio times theirs.
template <int KIND>
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
    float x[4];
    decode4<KIND>(w, x);
    return encode4<KIND>(__fmul_rn(x[0], ratio), __fmul_rn(x[1], ratio), __fmul_rn(x[2], ratio),
                         __fmul_rn(x[3], ratio));
}

// Grid: x = block units (num_tokens / 16 + 2 num_seqs), y = groups of 8 of the
// 2 num_kv_heads (head, K or V) jobs, one a warp.
template <int D, int KIND, int CTAS>
__global__ void __launch_bounds__(kWarps * 32, CTAS) cache_append_kernel(const RowsParams P) {
    constexpr int LPR = D / 8;                // lanes a row, 8 elements each
    constexpr int RPP = 32 / LPR;             // rows a pass
    constexpr int NP = kBlockSize / RPP;      // passes
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(P);
    const int job = blockIdx.y * kWarps + warp;
    if (job >= 2 * P.hkv) return;
    const int h = job >> 1, which = job & 1;
    UnitRows r;
    if (!find_rows(P, blockIdx.x, lane, r) || !r.valid || r.phys < 0) return;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    const uint16_t* src = (which ? P.v_new : P.k_new) + h * D + col;
    const int64_t stride = which ? P.v_stride : P.k_stride;
    const size_t slab = static_cast<size_t>(r.phys) * P.hkv + h;
    uint8_t* dst = (which ? P.v_pool : P.k_pool) + slab * (kBlockSize * D) + col;
    float* scale_at = P.scales + 2 * slab + which;
    float old = 0.f;
    bool bad = false;
    if (r.first > 0) old = checked_scale(*scale_at, bad);
    uint4 x[NP];
    uint32_t most2 = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + sub;
        x[p] = make_uint4(0u, 0u, 0u, 0u);
        if (row >= r.first && row < r.last)
            x[p] = __ldg(reinterpret_cast<const uint4*>(src + (r.token + row - r.first) * stride));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) most2 = max_bf16_sizes(x[p], most2);
    uint32_t most = warp_max_size(most2);
    const bool wild = most >= 0x7f80u;  // a value that is not finite, for the whole warp
    if (wild) {
        bad = true;
        most2 = 0;
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            most2 = max_bf16_sizes(tame8<true>(x[p]), most2);
            if (KIND == kKindInt8Blocks) x[p] = tame8<false>(x[p]);  // has no code for a NaN
        }
        most = warp_max_size(most2);
    }
    const float scale =
        fmaxf(fmaxf(old, __fmul_rn(__uint_as_float(most << 16), inv_code_max<KIND>())), kLeastScale);
    const float inv = __frcp_rn(scale);
    if (scale > old && r.first > 0) {
        const float ratio = __fmul_rn(old, inv);
        constexpr int C = CTAS > 3 ? 4 : NP;  // rows a lane at a time: what fits beside x
#pragma unroll 1
        for (int row = sub; row < r.first; row += C * RPP) {
            uint2 c[C];
#pragma unroll
            for (int p = 0; p < C; ++p)
                if (row + p * RPP < r.first) c[p] = *reinterpret_cast<const uint2*>(dst + (row + p * RPP) * D);
#pragma unroll
            for (int p = 0; p < C; ++p)
                if (row + p * RPP < r.first)
                    *reinterpret_cast<uint2*>(dst + (row + p * RPP) * D) =
                        make_uint2(recode4<KIND>(c[p].x, ratio), recode4<KIND>(c[p].y, ratio));
        }
    }
    if (lane == 0) {
        if (scale > old || r.first == 0 || bad) *scale_at = scale;
        if (bad) record_error(P.err, kErrRange, static_cast<uint32_t>(r.s));
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + sub;
        if (row >= r.first && row < r.last)
            *reinterpret_cast<uint2*>(dst + row * D) =
                wild ? encode8<KIND, false>(x[p], inv) : encode8<KIND, true>(x[p], inv);
    }
}

// The same grid; a lane's 8 elements of a row are one 16-byte store.
template <int D, int KIND>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(const RowsParams P) {
    constexpr int LPR = D / 8, RPP = 32 / LPR, NP = kBlockSize / RPP;
    constexpr int EB = KIND == kKindBf16 ? 2 : 1;
    griddep_launch_dependents();
    griddep_wait();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x == 0 && blockIdx.y == 0) check_sequences(P);
    const int job = blockIdx.y * kWarps + warp;
    if (job >= 2 * P.hkv) return;
    const int h = job >> 1, which = job & 1;
    UnitRows r;
    if (!find_rows(P, blockIdx.x, lane, r)) return;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    uint16_t* dst = (which ? P.v_out : P.k_out) + h * D + col;
    const size_t slab = static_cast<size_t>(max(r.phys, 0)) * P.hkv + h;
    const uint8_t* src = (which ? P.v_pool : P.k_pool) + (slab * (kBlockSize * D) + col) * EB;
    float scale = which ? P.v_scale : P.k_scale;
    bool bad = false;
    if (KIND >= kKindE4m3Blocks && r.phys >= 0) scale = checked_scale(__ldg(P.scales + 2 * slab + which), bad);
    uint4 x[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + sub;
        x[p] = make_uint4(0u, 0u, 0u, 0u);
        if (r.phys >= 0 && row >= r.first && row < r.last) {
            if constexpr (EB == 2) {
                x[p] = __ldg(reinterpret_cast<const uint4*>(src + row * D * EB));
            } else {
                const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + row * D));
                x[p].x = c.x, x[p].y = c.y;
            }
        }
    }
    if (bad && lane == 0) record_error(P.err, kErrRange, static_cast<uint32_t>(r.s));
#pragma unroll
    for (int p = 0; p < NP; ++p) {
        const int row = p * RPP + sub;
        if constexpr (EB == 1) {
            float f[8];
            decode4<KIND>(x[p].x, *reinterpret_cast<float(*)[4]>(&f[0]));
            decode4<KIND>(x[p].y, *reinterpret_cast<float(*)[4]>(&f[4]));
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b =
                    __floats2bfloat162_rn(__fmul_rn(f[2 * i], scale), __fmul_rn(f[2 * i + 1], scale));
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            x[p] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (row >= r.first && row < r.last)
            *reinterpret_cast<uint4*>(dst + static_cast<size_t>(r.token + row - r.first) * P.hkv * D) = x[p];
    }
}

RowsParams params_of(const CacheRowsArgs& a) {
    RowsParams P = {};
    P.k_pool = static_cast<uint8_t*>(a.k_pool);
    P.v_pool = static_cast<uint8_t*>(a.v_pool);
    P.scales = a.block_scales;
    P.k_new = static_cast<const uint16_t*>(a.k_new);
    P.v_new = static_cast<const uint16_t*>(a.v_new);
    P.k_out = static_cast<uint16_t*>(a.k_out);
    P.v_out = static_cast<uint16_t*>(a.v_out);
    P.k_stride = a.k_stride;
    P.v_stride = a.v_stride;
    P.start = a.query_start_loc;
    P.context_lens = a.context_lens;
    P.block_tables = a.block_tables;
    P.err = a.err;
    P.num_tokens = a.num_tokens;
    P.num_seqs = a.num_seqs;
    P.max_blocks = a.max_blocks_per_seq;
    P.num_blocks = a.num_blocks;
    P.hkv = a.num_kv_heads;
    P.k_scale = a.k_scale;
    P.v_scale = a.v_scale;
    return P;
}

dim3 rows_grid(const CacheRowsArgs& a) {
    return dim3(static_cast<unsigned>(a.num_tokens / kBlockSize + 2ll * a.num_seqs),
                static_cast<unsigned>((2 * a.num_kv_heads + kWarps - 1) / kWarps));
}

cudaError_t launch_rows(void (*kernel)(RowsParams), const CacheRowsArgs& a, cudaStream_t stream) {
    return launch_overlapped(kernel, rows_grid(a), dim3(kWarps * 32), 0, stream, params_of(a));
}

// With registers for 4 CTAs per SM, or for 3 where all CTAs are there at once:
// 16,381 rows of 40 heads x 128 take 77.3 and 85.7 us, 1,568 rows of 8 heads x
// 128 (336 CTAs) 4.8 and 4.1.
template <int KIND>
cudaError_t launch_append_kind(const CacheRowsArgs& a, int num_sms, cudaStream_t stream) {
    const dim3 grid = rows_grid(a);
    const bool at_once = static_cast<long long>(grid.x) * grid.y <= 3ll * num_sms;
    if (a.head_dim == 128)
        return launch_rows(at_once ? cache_append_kernel<128, KIND, 3> : cache_append_kernel<128, KIND, 4>, a, stream);
    return launch_rows(at_once ? cache_append_kernel<64, KIND, 3> : cache_append_kernel<64, KIND, 4>, a, stream);
}

template <int KIND>
cudaError_t launch_read_kind(const CacheRowsArgs& a, cudaStream_t stream) {
    return launch_rows(a.head_dim == 128 ? cache_read_kernel<128, KIND> : cache_read_kernel<64, KIND>, a, stream);
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsArgs& a, int num_sms, cudaStream_t stream) {
    return a.kv_dtype == kKindInt8Blocks ? launch_append_kind<kKindInt8Blocks>(a, num_sms, stream)
                                         : launch_append_kind<kKindE4m3Blocks>(a, num_sms, stream);
}

cudaError_t launch_cache_read(const CacheRowsArgs& a, cudaStream_t stream) {
    switch (a.kv_dtype) {
        case kKindBf16: return launch_read_kind<kKindBf16>(a, stream);
        case kKindE4m3: return launch_read_kind<kKindE4m3>(a, stream);
        case kKindE4m3Blocks: return launch_read_kind<kKindE4m3Blocks>(a, stream);
        default: return launch_read_kind<kKindInt8Blocks>(a, stream);
    }
}

}  // namespace pkv
