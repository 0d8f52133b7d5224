// linear_device.cuh -- what the two forms of linear attention share: which
// rows and states a sequence has, and the decay in extended precision.
#pragma once

#include <cstdint>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// One sequence of a linear-attention call.
struct LinearSeq {
    int32_t row0;    // first row
    int32_t rows;    // new tokens (0: nothing to do)
    int32_t load;    // slot its state is read from, -1: it starts from zero
    int32_t store;   // slot its state goes to, -1: nowhere
    int32_t bad;     // rows get zeros and no state is stored
};

// `report`: whether this thread records what is out of range.
__device__ __forceinline__ LinearSeq linear_seq(const LinearArgs& A, int s, bool report) {
    LinearSeq q;
    // loads that hang on nothing, together
    const int n = __ldg(A.context_lens + s), from = __ldg(A.state_slots + s), to = __ldg(A.new_slots + s);
    if (A.query_start_loc != nullptr) {
        q.row0 = __ldg(A.query_start_loc + s);
        const int end = __ldg(A.query_start_loc + s + 1);
        q.rows = end - q.row0;
        if (q.row0 < 0 || end < q.row0 || end > A.num_tokens) {
            if (report) record_error(A.err, kErrRange, static_cast<uint32_t>(s));
            q.row0 = q.rows = 0;
        }
    } else {
        q.row0 = s;
        q.rows = 1;
    }
    q.load = q.store = -1;
    q.bad = 0;
    if (q.rows == 0) return q;
    if (n < q.rows) {
        // A single-token row without a context is padding; anything else
        // contradicts itself.
        q.bad = 1;
        if (report && !(n == 0 && A.query_start_loc == nullptr))
            record_error(A.err, kErrRange, static_cast<uint32_t>(s));
        return q;
    }
    if ((n > q.rows && from >= A.num_slots) || to >= A.num_slots) {
        if (report) record_error(A.err, kErrRange, static_cast<uint32_t>(s));
        q.bad = 1;
        return q;
    }
    if (n > q.rows && from < 0) {
        q.bad = 1;  // no state to go on from: a skipped sequence
        return q;
    }
    q.load = n > q.rows ? from : -1;
    q.store = to;
    return q;
}

// Whether a sequence reads or stores that slot (for the check of shared
// slots): as linear_seq has it, where one that is skipped or refused does
// neither.  (With the slots read before the lengths a decode call of 128 x 40
// states took 106 us in place of 99.)
__device__ __forceinline__ bool linear_shares(const LinearArgs& A, int other, int store) {
    const int n = __ldg(A.context_lens + other);
    int rows = 1;
    if (A.query_start_loc != nullptr) {
        const int row0 = __ldg(A.query_start_loc + other), end = __ldg(A.query_start_loc + other + 1);
        rows = row0 < 0 || end > A.num_tokens ? 0 : end - row0;
    }
    if (rows <= 0 || n < rows) return false;
    const int to = __ldg(A.new_slots + other);
    if (n == rows) return to == store;
    const int from = __ldg(A.state_slots + other);
    return (to == store || from == store) && to < A.num_slots && from >= 0 && from < A.num_slots;
}

// A log decay above 0 or NaN counts as 0 and is reported; -inf keeps nothing.
__device__ __forceinline__ float clean_log_decay(const LinearArgs& A, int h, bool report) {
    float g = __ldg(A.log_decay + h);
    if (!(g <= 0.f)) {
        if (report) record_error(A.err, kErrRange, static_cast<uint32_t>(h));
        g = 0.f;
    }
    return fmaxf(g, -1e30f);
}

// exp(g * tokens) as hi + lo, g <= 0.  A state is multiplied by it once per
// token or chunk, so the 2^-25 of one fp32 factor would grow with the length
// of the context.  x = g * tokens as an fp32 pair; n = the nearest whole
// multiple of ln 2, r = x - n ln 2 (Cody and Waite's reduction: ln 2 in two
// parts, the first short enough that n times it is exact), |r| <= 0.35; exp(r) = 1 + r + r^2 (1/2 + r/6 +
// ...), the Taylor terms from r^2 on in fp32: off by 2^-24 of r^2 / 2, which
// for the slow decays, where it counts, is far below 2^-40.
__device__ __forceinline__ float2 decay_pair(float g, int tokens) {
    const float t = static_cast<float>(tokens);
    const float x = g * t;
    if (x < -100.f) return make_float2(0.f, 0.f);
    const float xl = fmaf(g, t, -x);
    const float n = rintf(x * 1.44269504f);
    constexpr float kLn2Hi = 0.693145752f;       // 15 bits
    constexpr float kLn2Lo = 1.42860677e-6f;     // ln 2 - kLn2Hi
    const float rh = fmaf(n, -kLn2Hi, x);
    const float rl = fmaf(n, -kLn2Lo, xl);
    const float r = rh + rl;
    float p = 1.f / 362880.f;
    p = fmaf(p, r, 1.f / 40320.f);
    p = fmaf(p, r, 1.f / 5040.f);
    p = fmaf(p, r, 1.f / 720.f);
    p = fmaf(p, r, 1.f / 120.f);
    p = fmaf(p, r, 1.f / 24.f);
    p = fmaf(p, r, 1.f / 6.f);
    p = fmaf(p, r, 0.5f);
    const float tail = fmaf(p * r, r, rl);       // what 1 + rh lacks
    const float one = 1.f + rh;
    const float rest = (rh - (one - 1.f)) + tail;
    const float hi = one + rest;
    const float lo = rest - (hi - one);
    const float scale = exp2f(n);
    return make_float2(hi * scale, lo * scale);
}

constexpr int kScanThreads = 128;
constexpr int kLinearChunk = 64;  // tokens of a chunk

// The states at the ends of the ranges, from the ranges' own: bounds[x] <-
// lam^(tokens of the segment) (state before it) + bounds[x], in order, the
// state before being the sequence's where the segment begins it and
// bounds[x - 1] otherwise.  Block `block` of S.blocks; a thread carries two
// elements.
__device__ __forceinline__ void scan_ranges(const LinearArgs& A, const LinearScan& S, int block) {
    __shared__ float2 lam_s;
    __shared__ __align__(16) int4 tails[kScanThreads];
    const int slices = A.head_dim * A.head_dim / (2 * kScanThreads);
    const int h = block / slices, tid = threadIdx.x;
    const float g = clean_log_decay(A, h, false);
    const int64_t head = static_cast<int64_t>(A.head_dim) * A.head_dim;
    const int64_t e = (static_cast<int64_t>(block % slices) * kScanThreads + tid) * 2;
    float* p = S.bounds + h * head + e;
    const int64_t step = static_cast<int64_t>(A.num_kv_heads) * head;
    float2 x = make_float2(0.f, 0.f);
    // Loads of several ranges together: they hang on nothing but the list,
    // and the first ones not even on that.
    constexpr int kBatch = 8;
    for (int r0 = 0; r0 < S.ranges - 1; r0 += kBatch) {
        const int n = min(kBatch, S.ranges - 1 - r0);
        const bool list = r0 % kScanThreads == 0;
        if (list) {
            if (r0 > 0) __syncthreads();
            if (r0 + tid < S.ranges - 1) tails[tid] = S.tails[r0 + tid];
            if (r0 == 0 && tid == kScanThreads - 1) lam_s = decay_pair(g, S.tokens);
        }
        float2 y[kBatch], before[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (j < n) y[j] = *reinterpret_cast<const float2*>(p + (r0 + j) * step);
        if (list) __syncthreads();
        const int4* tail = tails + r0 % kScanThreads;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            before[j] = make_float2(0.f, 0.f);
            if (j < n && tail[j].x > 0 && tail[j].y && tail[j].w >= 0)
                before[j] = *reinterpret_cast<const float2*>(
                    A.states + (static_cast<int64_t>(tail[j].w) * A.num_kv_heads + h) * head + e);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
            if (j >= n || tail[j].x <= 0) continue;
            float2 f = lam_s;
            if (tail[j].y) {
                // a sequence's first segment: its length is its own, its factor applied once
                f = make_float2(expf(g * static_cast<float>(tail[j].x * kLinearChunk)), 0.f);
                x = before[j];
            }
            x.x = fmaf(x.x, f.x, fmaf(x.x, f.y, y[j].x));
            x.y = fmaf(x.y, f.x, fmaf(x.y, f.y, y[j].y));
            *reinterpret_cast<float2*>(p + (r0 + j) * step) = x;
        }
    }
}

}  // namespace pkv
