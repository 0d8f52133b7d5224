// scaled_attention.cu -- attention over 8-bit pools with a scale for each
// (block, kv head): out = softmax_j(scale q . K_j) V_j with K_j, V_j code
// values times their block's scales.  A warp takes one query row of one q
// head and goes over its keys in order with a running maximum and sum; a lane
// owns D / 32 consecutive dims.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "scaled_device.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 8;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int KIND>
__global__ void __launch_bounds__(kWarps * 32) scaled_attention_kernel(const ScaledArgs P) {
    constexpr int DPL = D / 32;
    griddep_launch_dependents();
    griddep_wait();
    const int lane = threadIdx.x % 32;
    const int h = blockIdx.y;
    const int t = blockIdx.x * kWarps + threadIdx.x / 32;
    if (t >= P.num_tokens) return;
    int s = t, n, pos;
    if (P.query_start_loc != nullptr) {
        int lo = 0, hi = P.num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (__ldg(P.query_start_loc + mid) <= t) lo = mid; else hi = mid;
        }
        s = lo;
    }
    n = __ldg(P.context_lens + s);
    const int cap = static_cast<int>(min(static_cast<long long>(P.max_context_len),
                                         static_cast<long long>(P.max_blocks_per_seq) * kBlockSize));
    const int ql = P.query_start_loc == nullptr ? 1 : __ldg(P.query_start_loc + s + 1) - __ldg(P.query_start_loc + s);
    bool zero = false;
    if (n < 0 || n > cap || (ql > 1 && ql > n)) {
        if (lane == 0) record_error(P.err, kErrRange, static_cast<uint32_t>(s));
        zero = ql > 1;
        n = n < 0 ? 0 : min(n, cap);
    }
    pos = P.query_start_loc == nullptr ? n - 1 : n - ql + t - __ldg(P.query_start_loc + s);
    float* out = P.out + (static_cast<size_t>(t) * P.num_q_heads + h) * D + lane * DPL;
    float q[DPL], o[DPL];
    const uint16_t* qrow =
        static_cast<const uint16_t*>(P.q) + (static_cast<size_t>(t) * P.num_q_heads + h) * D + lane * DPL;
#pragma unroll
    for (int i = 0; i < DPL; ++i) {
        q[i] = __uint_as_float(static_cast<uint32_t>(qrow[i]) << 16) * (P.scale * kLog2e);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int g = h / (P.num_q_heads / P.num_kv_heads);
    const int last = zero ? -1 : pos;
    bool bad = false;
    for (int b = 0; b * kBlockSize <= last; ++b) {
        int phys = __ldg(P.block_tables + static_cast<size_t>(s) * P.max_blocks_per_seq + b);
        if (phys < 0 || phys >= P.num_blocks) {
            bad = true;
            phys = 0;
        }
        const size_t slab = static_cast<size_t>(phys) * P.num_kv_heads + g;
        const float ks = checked_scale(__ldg(P.block_scales + 2 * slab), bad);
        const float vs = checked_scale(__ldg(P.block_scales + 2 * slab + 1), bad);
        const uint8_t* k = static_cast<const uint8_t*>(P.k_pool) + slab * (kBlockSize * D) + lane * DPL;
        const uint8_t* v = static_cast<const uint8_t*>(P.v_pool) + slab * (kBlockSize * D) + lane * DPL;
        const int cnt = min(kBlockSize, last + 1 - b * kBlockSize);
        for (int r = 0; r < cnt; ++r) {
            float x[4], y[4];
            uint32_t wk, wv;
            if (DPL == 4) {
                wk = __ldg(reinterpret_cast<const uint32_t*>(k + r * D));
                wv = __ldg(reinterpret_cast<const uint32_t*>(v + r * D));
            } else {
                wk = __ldg(reinterpret_cast<const uint16_t*>(k + r * D));
                wv = __ldg(reinterpret_cast<const uint16_t*>(v + r * D));
            }
            decode4<KIND>(wk, x);
            decode4<KIND>(wv, y);
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < DPL; ++i) part = fmaf(q[i], x[i], part);
            const float sc = warp_sum(part) * ks;
            const float mn = fmaxf(m, sc);
            const float alpha = exp2f(m - mn), p = exp2f(sc - mn);
            m = mn;
            l = l * alpha + p;
#pragma unroll
            for (int i = 0; i < DPL; ++i) o[i] = fmaf(p, y[i] * vs, o[i] * alpha);
        }
    }
    if (bad && lane == 0) record_error(P.err, kErrRange, static_cast<uint32_t>(s));
#pragma unroll
    for (int i = 0; i < DPL; ++i) out[i] = l == 0.f ? 0.f : o[i] / l;  // 0: no keys
}

}  // namespace

cudaError_t launch_scaled_attention(const ScaledArgs& a, cudaStream_t stream) {
    if (a.num_tokens == 0) return cudaSuccess;
    const dim3 grid((a.num_tokens + kWarps - 1) / kWarps, a.num_q_heads);
    const bool i8 = a.kv_dtype == kKindInt8Blocks;
    auto kernel = a.head_dim == 128
                      ? (i8 ? scaled_attention_kernel<128, kKindInt8Blocks> : scaled_attention_kernel<128, kKindE4m3Blocks>)
                      : (i8 ? scaled_attention_kernel<64, kKindInt8Blocks> : scaled_attention_kernel<64, kKindE4m3Blocks>);
    return launch_overlapped(kernel, grid, dim3(kWarps * 32), 0, stream, a);
}

}  // namespace pkv
