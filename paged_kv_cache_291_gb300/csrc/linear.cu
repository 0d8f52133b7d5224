// linear.cu -- linear attention with a decay for each head, recurrent form:
// one new token per sequence (or a few), over its fp32 state.
//
// Mathematics.  Per sequence and kv head a state S [d][d] (k index, v index):
//     S <- exp(log_decay) S + k v^T,      out_h = scale * q_h^T S
// for the q heads h of the group.  Everything is fp32; the decay is applied
// as an fp32 pair (linear_device.cuh), one fused rounding per element.
//
// Split.  The columns of S (v index) do not mix, so a CTA takes 32 of them:
// 128-byte row segments, [d][32] floats in registers (thread = one float4
// of columns, every 16th row), nothing joined across CTAs.  The sum over
// rows that gives out is a shuffle over the lanes with the same columns and
// one pass through shared memory.
//
// Bound: HBM, 8 d^2 bytes of state per (sequence, kv head) against 2 d^2
// (1 + group) flops.  128 sequences of 40 heads of 128: 678 MB in 99.3 us,
// 6.8 TB/s, the rate of a copy; one sequence of 16 heads 2.8 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "linear_device.cuh"

namespace pkv {
namespace {

constexpr int kThreads = kScanThreads;
constexpr int kCols = 32;                       // columns of S per CTA
constexpr int kRowLanes = kThreads / (kCols / 4);  // 16 threads share a column quad
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float bf16_to_f32(uint16_t u) { return __uint_as_float(static_cast<uint32_t>(u) << 16); }

// TT: tokens staged at a time.  SCAN: the first scan.blocks CTAs join the
// chunked form's ranges; the decode call's kernel does without, whose
// registers it would take.
template <int D, int G, int TT, bool SCAN>
__global__ void __launch_bounds__(kThreads) linear_recurrent_kernel(const LinearArgs A, const LinearScan scan) {
    constexpr int RPT = D / kRowLanes;          // rows of S per thread
    constexpr int SLICES = D / kCols;
    // sv and red are read and written as float4
    __shared__ __align__(16) float sk[TT][D], sv[TT][kCols], sq[TT][G][D];
    __shared__ __align__(16) float red[TT][kWarps][G][kCols];
    __shared__ float2 lam_s;
    griddep_launch_dependents();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    int unit = blockIdx.x;
    if constexpr (SCAN) {
        if (unit < scan.blocks) {
            griddep_wait();
            scan_ranges(A, scan, unit);
            return;
        }
        unit -= scan.blocks;
    }
    const int slice = unit % SLICES;
    const int h = unit / SLICES % A.num_kv_heads;
    const int s = unit / SLICES / A.num_kv_heads;
    const int col = (tid % 8) * 4;              // within the slice
    const int r0 = tid / 8;
    griddep_wait();
    const bool first = h == 0 && slice == 0;
    const LinearSeq q = linear_seq(A, s, first && tid == 0);
    if (q.rows == 0 || q.rows > A.max_recurrent) {
        // rows that the host left to no kernel
        if (q.rows > 0 && !A.chunk_rows && first && tid == 0) record_error(A.err, kErrRange, static_cast<uint32_t>(s));
        return;
    }
    if (q.bad) {
        for (int i = tid; i < q.rows * G * kCols; i += kThreads) {
            const int t = i / (G * kCols), g = i / kCols % G;
            A.out[(static_cast<int64_t>(q.row0 + t) * A.num_q_heads + h * G + g) * D + slice * kCols + i % kCols] = 0.f;
        }
        return;
    }
    const int64_t head = static_cast<int64_t>(D) * D;
    float4 S[RPT];
    if (q.load >= 0) {
        const float* p = A.states + (static_cast<int64_t>(q.load) * A.num_kv_heads + h) * head + slice * kCols + col;
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = *reinterpret_cast<const float4*>(p + (r0 + i * kRowLanes) * D);
    } else {
#pragma unroll
        for (int i = 0; i < RPT; ++i) S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (tid == 0) lam_s = decay_pair(clean_log_decay(A, h, true), 1);
    if (first && q.store >= 0) {
        // A slot that two sequences store to, or that one stores to and
        // another reads, has no defined content: reported.
        for (int o = tid; o < A.num_seqs; o += kThreads)
            if (o != s && linear_shares(A, o, q.store)) record_error(A.err, kErrAlias, static_cast<uint32_t>(s));
    }
    for (int t0 = 0; t0 < q.rows; t0 += TT) {
        const int tt = min(TT, q.rows - t0);
        for (int i = tid; i < tt * D; i += kThreads) {
            const int t = i / D, e = i % D;
            sk[t][e] = bf16_to_f32(A.k[(q.row0 + t0 + t) * A.k_stride + static_cast<int64_t>(h) * D + e]);
        }
        for (int i = tid; i < tt * kCols; i += kThreads) {
            const int t = i / kCols, e = i % kCols;
            sv[t][e] =
                bf16_to_f32(A.v[(q.row0 + t0 + t) * A.v_stride + static_cast<int64_t>(h) * D + slice * kCols + e]);
        }
        for (int i = tid; i < tt * G * D; i += kThreads) {
            const int t = i / (G * D), e = i % (G * D);
            sq[t][e / D][e % D] =
                bf16_to_f32(A.q[(q.row0 + t0 + t) * A.q_stride + static_cast<int64_t>(h) * G * D + e]);
        }
        __syncthreads();
        const float2 lam = lam_s;
#pragma unroll 1
        for (int t = 0; t < tt; ++t) {
            const float4 v = *reinterpret_cast<const float4*>(&sv[t][col]);
            float4 o[G];
#pragma unroll
            for (int g = 0; g < G; ++g) o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = r0 + i * kRowLanes;
                const float k = sk[t][r];
                S[i].x = fmaf(S[i].x, lam.x, fmaf(S[i].x, lam.y, k * v.x));
                S[i].y = fmaf(S[i].y, lam.x, fmaf(S[i].y, lam.y, k * v.y));
                S[i].z = fmaf(S[i].z, lam.x, fmaf(S[i].z, lam.y, k * v.z));
                S[i].w = fmaf(S[i].w, lam.x, fmaf(S[i].w, lam.y, k * v.w));
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const float x = sq[t][g][r];
                    o[g].x = fmaf(x, S[i].x, o[g].x);
                    o[g].y = fmaf(x, S[i].y, o[g].y);
                    o[g].z = fmaf(x, S[i].z, o[g].z);
                    o[g].w = fmaf(x, S[i].w, o[g].w);
                }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
#pragma unroll
                for (int m = 8; m < 32; m *= 2) {
                    o[g].x += __shfl_xor_sync(0xffffffffu, o[g].x, m);
                    o[g].y += __shfl_xor_sync(0xffffffffu, o[g].y, m);
                    o[g].z += __shfl_xor_sync(0xffffffffu, o[g].z, m);
                    o[g].w += __shfl_xor_sync(0xffffffffu, o[g].w, m);
                }
                if (lane < 8) *reinterpret_cast<float4*>(&red[t][warp][g][col]) = o[g];
            }
        }
        __syncthreads();
        for (int i = tid; i < tt * G * kCols; i += kThreads) {
            const int t = i / (G * kCols), g = i / kCols % G, e = i % kCols;
            float x = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) x += red[t][w][g][e];
            A.out[(static_cast<int64_t>(q.row0 + t0 + t) * A.num_q_heads + h * G + g) * D + slice * kCols + e] =
                A.scale * x;
        }
    }
    if (q.store >= 0) {
        float* p = A.states + (static_cast<int64_t>(q.store) * A.num_kv_heads + h) * head + slice * kCols + col;
#pragma unroll
        for (int i = 0; i < RPT; ++i) *reinterpret_cast<float4*>(p + (r0 + i * kRowLanes) * D) = S[i];
    }
}

template <int D, int G>
cudaError_t launch(const LinearArgs& a, int32_t longest, const LinearScan& scan, cudaStream_t stream) {
    const int64_t grid = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads * (D / kCols) + scan.blocks;
    if (grid > 0x7fffffff) return cudaErrorInvalidValue;
    auto kernel = scan.blocks == 0 ? (longest <= 1 ? linear_recurrent_kernel<D, G, 1, false>
                                                   : linear_recurrent_kernel<D, G, 4, false>)
                                   : (longest <= 1 ? linear_recurrent_kernel<D, G, 1, true>
                                                   : linear_recurrent_kernel<D, G, 4, true>);
    return launch_overlapped(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, stream, a, scan);
}

template <int D>
cudaError_t launch_groups(const LinearArgs& a, int32_t longest, const LinearScan& scan, cudaStream_t stream) {
    switch (a.num_q_heads / a.num_kv_heads) {
        case 1: return launch<D, 1>(a, longest, scan, stream);
        case 2: return launch<D, 2>(a, longest, scan, stream);
        case 4: return launch<D, 4>(a, longest, scan, stream);
        default: return launch<D, 8>(a, longest, scan, stream);
    }
}

}  // namespace

cudaError_t launch_linear_recurrent(const LinearArgs& a, int32_t longest, const LinearScan& scan, cudaStream_t stream) {
    return a.head_dim == 64 ? launch_groups<64>(a, longest, scan, stream) : launch_groups<128>(a, longest, scan, stream);
}

}  // namespace pkv
