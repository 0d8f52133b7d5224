// linear_chunk.cu -- linear attention with a decay for each head, chunked
// form on tcgen05 tensor cores.
//
// Mathematics.  The recurrence S <- lam S + k v^T, o = scale q^T S over a
// chunk of C = 64 tokens (t, s count inside it, S is the state before it):
//     P[s][t]  = scale lam^(t-s) (k_s . q_t)   for s <= t, else 0
//     O^T      = scale lam^(t+1) (S^T Q^T)[.][t] + V^T P
//     S^T     <- lam^C S^T + (V~)^T K,         V~_s = lam^(C-1-s) v_s
// Four products of bf16 inputs with fp32 sums, held transposed so that every
// one has the v index (or s) in the 128 tensor-memory lanes, S^T can stay in
// tensor memory as an accumulator and be read from there as an operand, and
// an output column is a coalesced row segment.
//
// Precision.  q, k and v are exact in bf16; S, P and V~ are fp32 values.  Each
// is split into three bf16 terms (8 + 8 + 8 bits, exact), and
// its product is taken three times, so that operands of 24 bits go in whole;
// two terms would be off by up to 2^-19 of a value's binade.  The products'
// fp32 sums truncate, where an fp32 add rounds: 300 tokens are off by 2.3e-7
// of the norm, 16,384 by 5.9e-7 to 6.6e-7, plain fp32 sums by 2.1e-7 and
// 2.3e-7.  The state's decay factor is an fp32 pair.
//
// Split.  A CTA takes one kv head of a range of chunks and walks them; all q
// heads of the group share the state's work.  Its warps have
// one part each: loads (TMA, 128-byte swizzle), MMA issue, P, V~, S (read,
// split, decay) and the output; barriers order them, so the tensor cores work
// on one chunk while the others prepare the next.
// The chunks of all sequences are cut into equal ranges, one CTA each per kv
// head, whatever the lengths of the sequences.  Where a border lies inside a
// sequence, linear_state_kernel sums the part's own state first and
// linear_scan_kernel carries the states over the borders.  The CTAs of one
// launch come in no order, so a slot that a sequence reads in its first range
// and replaces in its last is copied by linear_state_kernel for the first.
// Where a group's q heads are dealt to several CTAs, all of them read the slot
// and reach the same new state; the last to reach it stores it.
//
// Bound.  A chunk's chain: the state is split (1,500 to 2,000 cycles), read by
// the outputs' product (900), updated (900).  At head_dim 128 and one q head a
// chunk takes 5,000 cycles against 3,500 of its bytes at HBM's rate; the
// tensor pipe is 38% active and nothing is full.  16,384 tokens of 16 heads of
// 128: 119 us (states of the ranges 24, scan 5, main 85); 12 prompts, 6,171
// tokens, 32/8 heads of 64: 53 us.
//
// Every wait is bounded; TMEM is freed on every exit path.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <memory>
#include <new>

#include "linear_device.cuh"
#include "tcgen05_rows.cuh"

namespace pkv {
namespace {

constexpr int C = kLinearChunk;          // tokens per chunk
constexpr int kPanel = C * 128;          // [64 tokens][64 dims] bf16, 128-byte swizzle
constexpr int kPTile = C * 128;          // one term of P, [64 s][64 t] bf16

// Ring depths and the shared-memory map of the main kernel.
template <int D>
struct Layout {
    static constexpr int kTile = D / 64 * kPanel;     // a K, V or Q tile, or one term of V~
    static constexpr int kKv = D == 64 ? 4 : 3;       // K and V stages
    static constexpr int kQ = D == 64 ? 4 : 2;        // Q stages
    static constexpr int OFF_K = 0;
    static constexpr int OFF_V = OFF_K + kKv * kTile;
    static constexpr int OFF_Q = OFF_V + kKv * kTile;
    static constexpr int OFF_VT = OFF_Q + kQ * kTile;
    static constexpr int OFF_P = OFF_VT + 3 * kTile;  // two buffers of three terms
    static constexpr int OFF_REST = OFF_P + 2 * 3 * kPTile;
    // TMEM columns: scores, S, its three terms, the two parts of the outputs.
    // V P takes P's terms one after the other into one sum at head_dim 128; at
    // 64 there are columns for three sums, so they go side by side in one MMA
    // of N = 192, which reads V once (a ragged batch of 12 prompts, 32/8
    // heads: 49.5 to 39 us).
    static constexpr int kSums = D == 64 ? 3 : 1;
    static constexpr uint32_t COL_SCORES = 0, COL_S = C, COL_SB = COL_S + D, COL_OS = COL_SB + 3 * D / 2,
                              COL_OP = COL_OS + C;
    static_assert(COL_OP + kSums * C <= 512, "TMEM columns");
};
constexpr int TAB_P = 0;                              // float[128]: scale lam^(t-s) at 63 + t - s
constexpr int TAB_O = 128;                            // float[64]: scale lam^(t+1)
constexpr int TAB_V = 192;                            // float[64]: lam^j
constexpr int TAB_LAM = 256;                          // float2: lam^64
constexpr int kBadBuffers = 3;

enum {
    B_KVFULL = 0,               // + stage (room for 4)
    B_KVEMPTY = B_KVFULL + 4,
    B_QFULL = B_KVEMPTY + 4,
    B_QEMPTY = B_QFULL + 4,
    B_SCORES = B_QEMPTY + 4,    // scores in TMEM
    B_SCFREE,                   // and read (3 arrivals)
    B_P,                        // + buffer: P in shared memory (3 arrivals)
    B_PFREE = B_P + 2,          // + buffer: P read
    B_S = B_PFREE + 2,          // S split and decayed (8 arrivals)
    B_SFREE,                    // the split S read by every q head of the chunk
    B_VT,                       // V~ in shared memory (4 arrivals)
    B_VTFREE,                   // V~ read, S holds the chunk
    B_OS,                       // the state's part of the outputs in TMEM
    B_OSFREE,                   // and read (8 arrivals)
    B_OP,                       // the scores' part
    B_OPFREE,
    NBAR
};
enum { I_SEGS = 0, I_CHUNKS, I_BAD, I_COUNT };

constexpr int kMaxSegments = 128;  // of one range: ranges are at most this long when there are more sequences
constexpr int kFromBounds = -2, kFromStarts = -3;

// K and V are read twice in the same order, by the state kernel and by the
// main one.  When they are more than the L2 keeps beside the rest, the oldest
// lines, which are wanted first, would go first: the state kernel then loads
// with evict_first, so that its later tiles replace each other.  16 heads of
// 128, calls on the same inputs in a graph: 134 MB of K and V 121.7 to 117.3
// us, 67 MB 70.2 to 68.5, 50 MB 54.9 and 55.0, 34 MB 41.8 both ways.
constexpr int64_t kOverflowBytes = 40 << 20;

struct Segment {
    int row0, rows;   // rows <= 0: -rows rows get zeros and nothing else happens
    int load, store;  // slots, -1: none; load kFromBounds: the state at the end of the range before;
                      // kFromStarts: this range's copy of a slot that a later range's CTA stores to;
                      // store -2 - slot: other CTAs read this slot too, the last of them stores
    int seq, first;   // first: holds the sequence's first row
    int pad[2];
};

// The list's first segments are in shared memory: most lists have no more,
// and every warp starts with a look at them.
constexpr int kNearSegments = 4;
struct Segments {
    Segment *near, *far;
    __device__ __forceinline__ Segment& operator[](int k) const { return k < kNearSegments ? near[k] : far[k]; }
};

// Warps, spread so that the four SM sub-partitions (warp % 4, which is also
// the TMEM lane quarter a warp can reach) carry about the same work.
constexpr int kThreads = 768;
constexpr int kLoadWarp = 2, kMmaWarp = 3;
// P: warps 0 (s 0-31, t 0-31), 4 (s 0-31, t 32-63) and 1 (s 32-63, t 32-63)
// V~: warps 2 (which also loads), 5, 6 and 7
constexpr int kVWarps = 4, kSWarp = 8, kSWarps = 8, kOWarp = 16, kOWarps = 8;

// What follows the tiles.
struct Rest {
    alignas(16) float tab[260];
    int bad_rows[kBadBuffers][128];  // see where V~ is made
    Segment near[kNearSegments];
    uint64_t bar[NBAR];
    int info[I_COUNT];
    int stores[kSWarps];             // whether the warp's CTA is the one that stores a shared segment
    uint32_t tmem;
};
template <int D>
constexpr int smem_bytes() {
    return Layout<D>::OFF_REST + static_cast<int>(sizeof(Rest));
}
static_assert(smem_bytes<128>() <= 232448, "shared memory budget (227 KB)");
static_assert(2 * smem_bytes<64>() > 228 * 1024, "the 512-column TMEM allocation needs one CTA per SM");

constexpr uint32_t kTmemCols = 512;

// Work: the chunks of the sequences in order (those of more than
// max_recurrent rows), cut into ranges of equal counts; a CTA takes one range
// of one kv head.  A range is a list of segments, each a run of one
// sequence's chunks; only the first can continue a sequence that began in an
// earlier range, and only the last can be continued.
struct ChunkParams {
    LinearArgs A;
    float* bounds;          // fp32 [ranges - 1][Hkv][d][d]: the state at the end of each range
    float* starts;          // the same: where a range's last segment begins a sequence that goes on in place, its state
    int4* tails;            // [ranges - 1]: what the scan needs of a range's last segment
    uint32_t* claims;       // [num_seqs][Hkv], cleared by an earlier launch: CTAs of a shared segment that have
                            // read its slot, 4 bits for each of the warps that hold a part of the state
    Segment* segments;      // [ranges][CTAs of a range][kMaxSegments]
    int32_t ranges, range;  // ranges, and chunks of each
    int32_t units;          // chunks the host counted
    int32_t subs;           // CTAs a kv head's group of q heads is dealt to
    int32_t overflow;       // K and V, which are read twice, are more than the L2 keeps
    int32_t cut;            // the ranges' own states are there and joined
};

// One warp: calls f(sequence s, what it is, its first unit, the unit behind
// its last, whether it has units in [u0, u1), the lanes' ballot of that) in
// every lane; returns the units seen (all of them when `count`).  A sequence
// is read as a whole before its units are known: one round trip, not two.
template <typename F>
__device__ __forceinline__ int scan_units(const ChunkParams& P, int u0, int u1, bool count, F f) {
    const unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x % 32;
    int base = 0;
    for (int s0 = 0; s0 < P.A.num_seqs && (base < u1 || count); s0 += 32) {
        LinearSeq q = {};
        if (s0 + lane < P.A.num_seqs) q = linear_seq(P.A, s0 + lane, false);
        const int nc = q.rows > P.A.max_recurrent ? (q.rows + C - 1) / C : 0;
        int incl = nc;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += t;
        }
        const int first = base + incl - nc, end = base + incl;
        const bool in = nc > 0 && first < u1 && end > u0;
        f(s0 + lane, q, first, end, in, __ballot_sync(FULL, in));
        base += __shfl_sync(FULL, incl, 31);
    }
    return base;
}

// Walks the chunks of a range in order.
struct Cursor {
    Segments seg;
    int k, n;
    int row, left;  // the chunk's first row, and rows left in its segment

    __device__ __forceinline__ Cursor(Segments s, int count) : seg(s), k(-1), n(count), row(0), left(0) { open(); }
    __device__ __forceinline__ void open() {
        left = 0;
        while (left <= 0 && ++k < n) {
            row = seg[k].row0;
            left = seg[k].rows;
        }
    }
    __device__ __forceinline__ void next() {
        row += C;
        left -= C;
        if (left <= 0) open();
    }
};

__device__ __forceinline__ uint32_t pack_bf16(float2 x) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(x.y), "f"(x.x));
    return r;
}

__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
    uint32_t lo;
    asm("mul.lo.u32 %0, %1, 65536;" : "=r"(lo) : "r"(u));
    return make_float2(__uint_as_float(lo), __uint_as_float(u & 0xffff0000u));
}

// x - h for the two bf16 of h, exactly: one mixed-precision fma each, which
// takes a half of the pair as it is.  Shifts, masks and packs share a pipe of
// half the rate, and these conversions fill it.
__device__ __forceinline__ float2 less_bf16(float2 x, uint32_t h) {
    float2 r;
    asm("{\n\t.reg .b16 lo, hi, m;\n\t"
        "mov.b32 {lo, hi}, %2;\n\t"
        "mov.b16 m, 0xBF80;\n\t"  // -1
        "fma.rn.f32.bf16 %0, lo, m, %3;\n\t"
        "fma.rn.f32.bf16 %1, hi, m, %4;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "r"(h), "f"(x.x), "f"(x.y));
    return r;
}

// Two fp32 values as three packed bf16 pairs that sum to them exactly: each
// term is what is left, rounded to nearest.
__device__ __forceinline__ void split3(float2 x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = pack_bf16(x);
    x = less_bf16(x, hi);
    mid = pack_bf16(x);
    lo = pack_bf16(less_bf16(x, mid));
}

// The next row's address, computed where it is used (32 hoisted ones would
// not fit the registers).
__device__ __forceinline__ float* walk(float* p, int64_t bytes) {
    asm volatile("add.s64 %0, %0, %1;" : "+l"(p) : "l"(bytes));
    return p;
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) { return mbar_wait_warp(bar, parity); }

// V~ of one chunk, elementwise over the swizzled V tile: factor[rows - 1 - s]
// * v_s in three terms.  Rows past the piece become zero, there and in
// K and V: they are other sequences' tokens, and a zero factor times a NaN
// would poison the products.  Returns 0, or NaN if a value was not finite.
template <int D, int TERM, int THREADS, int UNROLL>
__device__ __forceinline__ float convert_v(uint32_t sk, uint32_t sv, uint32_t svt, const float* factor, int rows,
                                           int tid) {
    constexpr int kChunks = C * D * 2 / 16;  // 16-byte vectors of the tile
    float2 acc = make_float2(0.f, 0.f);
    const float2 zero = make_float2(0.f, 0.f);
#pragma unroll UNROLL
    for (int i = tid; i < kChunks; i += THREADS) {
        const int row = (i >> 3) & (C - 1);
        const uint32_t at = static_cast<uint32_t>(i) * 16u;
        if (row < rows) {
            uint32_t x[4], hi[4], mid[4], lo[4];
            tc::lds128(sv + at, x);
            const float f = factor[rows - 1 - row];
            const float2 ff = make_float2(f, f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 v = unpack_bf16(x[j]);
                acc = __ffma2_rn(v, zero, acc);
                split3(__fmul2_rn(v, ff), hi[j], mid[j], lo[j]);
            }
            tc::sts128(svt + at, hi[0], hi[1], hi[2], hi[3]);
            tc::sts128(svt + TERM + at, mid[0], mid[1], mid[2], mid[3]);
            tc::sts128(svt + 2 * TERM + at, lo[0], lo[1], lo[2], lo[3]);
        } else {
            tc::sts128(svt + at, 0u, 0u, 0u, 0u);
            tc::sts128(svt + TERM + at, 0u, 0u, 0u, 0u);
            tc::sts128(svt + 2 * TERM + at, 0u, 0u, 0u, 0u);
            tc::sts128(sv + at, 0u, 0u, 0u, 0u);
            tc::sts128(sk + at, 0u, 0u, 0u, 0u);
        }
    }
    return acc.x + acc.y;
}

// S^T += (V~)^T K for one chunk, V~ in three terms: A is V~ stored [s][v]
// (v contiguous), B is K stored [s][k] (k contiguous).
template <int D, int TERM>
__device__ __forceinline__ void mma_state(uint32_t col_s, uint32_t svt, uint32_t sk, bool accumulate) {
    constexpr uint32_t kIdesc = tc::idesc_bf16_f32(128, D, 1, 1);
    const uint64_t b = tc::smem_desc_sw128(sk, kPanel, 1024);
#pragma unroll 1
    for (int part = 2; part >= 0; --part) {  // smallest first: the sums truncate
        const uint64_t a = tc::smem_desc_sw128(svt + part * TERM, kPanel, 1024);
#pragma unroll
        for (int k = 0; k < C / 16; ++k)
            tc::mma_bf16_ss(col_s, a + k * (2048 >> 4), b + k * (2048 >> 4), kIdesc,
                            accumulate || part < 2 || k > 0 ? 1u : 0u);
    }
}

// G: q heads per CTA.  DEALT: the group's q heads are dealt to P.subs CTAs,
// otherwise one (a kernel starts with cold instructions: without the counting
// 30 ranges of two chunks, 3 heads of 64, take 21.1 us and with it 22.1).
template <int D, int G, bool DEALT>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v, const ChunkParams P) {
    using L = Layout<D>;
    constexpr int kPanels = D / 64;
    constexpr int kTile = L::kTile, kKv = L::kKv, kQ = L::kQ;
    extern __shared__ __align__(1024) uint8_t smem[];
    Rest& rest = *reinterpret_cast<Rest*>(smem + L::OFF_REST);
    uint64_t* bar = rest.bar;
    int* info = rest.info;
    float* tab = rest.tab;
    uint32_t* tmem_slot = &rest.tmem;
    const LinearArgs& A = P.A;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int subs = DEALT ? P.subs : 1;
    const int h = blockIdx.y / subs, sub = blockIdx.y % subs;
    const int hq0 = (h * subs + sub) * G;  // first of this CTA's q heads
    const bool reports = blockIdx.y == 0;

    // ---------------------------------------------------------- setup
    griddep_launch_dependents();
    if ((smem_addr(smem) & 1023) != 0) {  // the swizzled tiles need it; dynamic shared memory starts there
        griddep_wait();
        if (threadIdx.x == 0) record_error(A.err, kErrRange, 0xffffffffu);
        return;
    }
    if (threadIdx.x == 32 * kMmaWarp) {
        for (int i = 0; i < NBAR; ++i)
            mbar_init(&bar[i], i == B_SCFREE || i == B_P || i == B_P + 1 ? 3u
                                : i == B_S                                ? static_cast<uint32_t>(kSWarps)
                                : i == B_VT                               ? static_cast<uint32_t>(kVWarps)
                                : i == B_OSFREE || i == B_OPFREE          ? static_cast<uint32_t>(kOWarps)
                                                                          : 1u);
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
    for (int i = threadIdx.x; i < kBadBuffers * 128; i += kThreads) rest.bad_rows[0][i] = 0;
    for (int i = threadIdx.x; i < 2 * 3 * kPTile / 16; i += kThreads)
        tc::sts128(smem_addr(smem + L::OFF_P) + i * 16, 0u, 0u, 0u, 0u);
    tc::fence_proxy_async_smem();
    griddep_wait();
    const Segments segs = {
        rest.near, P.segments + (static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y) * kMaxSegments};
    if (warp == 0) {
        const bool last = blockIdx.x == gridDim.x - 1 && reports;
        const int u0 = blockIdx.x * P.range, u1 = u0 + P.range;
        int nseg = 0, chunks = 0, any_bad = 0;
        const int seen = scan_units(P, u0, u1, last, [&](int s, const LinearSeq& q, int first, int end, bool in,
                                                          unsigned lanes) {
            const int k = nseg + __popc(lanes & ((1u << lane) - 1));
            int n = 0, bad = 0;
            if (in && k < kMaxSegments) {
                if (q.bad && reports && first >= u0) linear_seq(A, s, true);
                const int c0 = max(u0, first) - first, c1 = min(u1, end) - first;
                Segment g;
                g.row0 = q.row0 + c0 * C;
                g.rows = min(q.rows, c1 * C) - c0 * C;
                // In place, the CTA of the sequence's last range may store
                // before this one reads: the state has been copied.  Of the
                // CTAs that share a kv head's q heads, one stores.
                const bool place = c0 == 0 && q.load >= 0 && q.load == q.store;
                g.load = c0 > 0 ? kFromBounds : place && end > u1 ? kFromStarts : q.load;
                if (end > u1) g.store = -1;
                else if (DEALT && place) g.store = -2 - q.store;
                else g.store = sub == 0 ? q.store : -1;
                g.seq = s;
                g.first = c0 == 0;
                bad = q.bad;
                // Device lengths that are not the host's: the plan cuts no
                // sequence, or ends before this one does, so its states are
                // not carried over the border.
                if (!P.cut ? c0 > 0 || end > u1 : end > u1 && blockIdx.x == gridDim.x - 1) {
                    if (reports) record_error(A.err, kErrRange, static_cast<uint32_t>(s));
                    bad = 1;
                }
                n = bad ? 0 : c1 - c0;
                if (bad) g.rows = -g.rows;
                segs[k] = g;
            }
            nseg += __popc(lanes);
            chunks += __reduce_add_sync(0xffffffffu, n);
            any_bad |= __any_sync(0xffffffffu, bad);
        });
        if (last && seen != P.units && lane == 0) record_error(A.err, kErrRange, static_cast<uint32_t>(A.num_seqs));
        if (last && !A.recurrent_rows) {
            // rows that the host left to no kernel
            for (int s = lane; s < A.num_seqs; s += 32) {
                const LinearSeq q = linear_seq(A, s, true);
                if (q.rows > 0 && q.rows <= A.max_recurrent) record_error(A.err, kErrRange, static_cast<uint32_t>(s));
            }
        }
        if (nseg > kMaxSegments) {
            // device lengths that are not the host's: the rest is dropped
            if (lane == 0) record_error(A.err, kErrRange, static_cast<uint32_t>(A.num_seqs));
            nseg = kMaxSegments;
        }
        if (lane == 0) {
            info[I_SEGS] = nseg;
            info[I_CHUNKS] = chunks;
            info[I_BAD] = any_bad;
        }
    } else if (warp == kSWarp) {
        if (lane == 0) {
            const float2 x = decay_pair(clean_log_decay(A, h, true), C);
            tab[TAB_LAM] = x.x;
            tab[TAB_LAM + 1] = x.y;
        }
    } else if (warp == kSWarp + 1 || warp == kSWarp + 2) {
        const float g = clean_log_decay(A, h, false);
        const int j = 32 * (warp - kSWarp - 1) + lane;
        const float x = expf(g * static_cast<float>(j));
        tab[TAB_V + j] = x;
        tab[TAB_P + 63 + j] = A.scale * x;
        if (j < 63) tab[TAB_P + j] = 0.f;
        tab[TAB_O + j] = A.scale * expf(g * static_cast<float>(j + 1));
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int nseg = info[I_SEGS], nch = info[I_CHUNKS];
    const int nitems = nch * G;
    bool ok = true;

    if (warp == kMmaWarp) {
        // ------------------------------------------------------ MMA issuer
        // Order of the products: the state's outputs first, which frees the
        // terms of S, then the state's update, so that the S warps work while
        // the scores of the next item and P V run.
        constexpr uint32_t kIdescScores = tc::idesc_bf16_f32(128, C, 0, 0);
        constexpr uint32_t kIdescOS = tc::idesc_bf16_f32(128, C, 0, 0);
        constexpr uint32_t kIdescOP = tc::idesc_bf16_f32(128, L::kSums * C, 1, 1);
        const uint32_t sk0 = smem_addr(smem + L::OFF_K), sv0 = smem_addr(smem + L::OFF_V), sq0 = smem_addr(smem + L::OFF_Q);
        const uint32_t svt = smem_addr(smem + L::OFF_VT), sp = smem_addr(smem + L::OFF_P);
        // scores[s][t] = k_s . q_t (lanes past 63 take the rows that follow K in
        // shared memory: never read)
        // Descriptors of consecutive K steps differ by their address field.
        auto scores = [&](int n) {
            const uint64_t a = tc::smem_desc_sw128(sk0 + (n / G % kKv) * kTile, 16, 1024);
            const uint64_t b = tc::smem_desc_sw128(sq0 + (n % kQ) * kTile, 16, 1024);
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                const uint32_t step = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
                tc::mma_bf16_ss(tmem + L::COL_SCORES, a + step, b + step, kIdescScores, k > 0 ? 1u : 0u);
            }
            tc::mma_commit(&bar[B_SCORES]);
        };
        // O_S^T[v][t] = sum_k S^T[v][k] q_t[k], S^T in three terms from TMEM
        auto out_state = [&](int n) {
            const uint64_t b = tc::smem_desc_sw128(sq0 + (n % kQ) * kTile, 16, 1024);
#pragma unroll 1
            for (int part = 2; part >= 0; --part) {
                const uint32_t a = tmem + L::COL_SB + part * (D / 2);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc::mma_bf16_ts(tmem + L::COL_OS, a + 8 * k, b + (((k >> 2) * kPanel + (k & 3) * 32) >> 4), kIdescOS,
                                    part < 2 || k > 0 ? 1u : 0u);
            }
            tc::mma_commit(&bar[B_QEMPTY + n % kQ]);
            tc::mma_commit(&bar[B_OS]);
        };
        // O_P^T[v][t] = sum_s V[s][v] P[s][t], P in three terms
        auto out_scores = [&](int n) {
            const uint64_t a = tc::smem_desc_sw128(sv0 + (n / G % kKv) * kTile, kPanel, 1024);
#pragma unroll 1
            for (int part = 3 - L::kSums; part >= 0; --part) {
                const uint64_t b = tc::smem_desc_sw128(sp + ((n & 1) * 3 + part) * kPTile, kPTile, 1024);
#pragma unroll
                for (int k = 0; k < C / 16; ++k)
                    tc::mma_bf16_ss(tmem + L::COL_OP, a + k * (2048 >> 4), b + k * (2048 >> 4), kIdescOP,
                                    part < 3 - L::kSums || k > 0 ? 1u : 0u);
            }
            if (n % G == G - 1) tc::mma_commit(&bar[B_KVEMPTY + n / G % kKv]);
            tc::mma_commit(&bar[B_PFREE + (n & 1)]);
            tc::mma_commit(&bar[B_OP]);  // last: once it is seen, nothing of this thread is in flight
        };
        if (nitems > 0) {
            ok = warp_wait(&bar[B_KVFULL], 0) && warp_wait(&bar[B_QFULL], 0);
            if (ok && tc::elect_one()) scores(0);
            __syncwarp();
        }
        for (int n = 0; n < nitems && ok; ++n) {
            const int i = n / G, g = n % G;
            if (g == 0 && !warp_wait(&bar[B_S], i & 1)) { ok = false; break; }
            if (n > 0 && !warp_wait(&bar[B_OSFREE], (n - 1) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (tc::elect_one()) {
                out_state(n);
                if (g == G - 1) tc::mma_commit(&bar[B_SFREE]);
            }
            __syncwarp();
            if (g == 0) {
                if (!warp_wait(&bar[B_VT], i & 1)) { ok = false; break; }
                if (tc::elect_one()) {
                    mma_state<D, kTile>(tmem + L::COL_S, svt, sk0 + (i % kKv) * kTile, true);
                    tc::mma_commit(&bar[B_VTFREE]);
                }
                __syncwarp();
            }
            if (n + 1 < nitems) {
                const int i1 = (n + 1) / G;
                if (!warp_wait(&bar[B_SCFREE], n & 1) ||
                    (i1 != i && !warp_wait(&bar[B_KVFULL + i1 % kKv], (i1 / kKv) & 1)) ||
                    !warp_wait(&bar[B_QFULL + (n + 1) % kQ], ((n + 1) / kQ) & 1)) {
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                if (tc::elect_one()) scores(n + 1);
                __syncwarp();
            }
            if (!warp_wait(&bar[B_P + (n & 1)], (n >> 1) & 1)) { ok = false; break; }
            if (n > 0 && !warp_wait(&bar[B_OPFREE], (n - 1) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (tc::elect_one()) out_scores(n);
            __syncwarp();
        }
    } else if (warp == 0 || warp == 1 || warp == 4) {
        // ------------------------------------------------------ P
        const int s = 32 * (warp & 1) + lane, begin = warp == 0 ? 0 : 32;
        const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * (warp & 1)) << 16) + L::COL_SCORES + begin;
        const uint32_t prow = smem_addr(smem + L::OFF_P) + s * 128;
        const float* f = tab + TAB_P + 63 - s + begin;
        // Rows 32-63 keep the zeros of tokens 0-31 that the set-up wrote.
        auto convert = [&](uint32_t (&x)[32], uint32_t at, int first) {
            // factors first: they cannot be loaded past the stores
#pragma unroll
            for (int t = 0; t < 32; t += 2) {
                float2 y = __fmul2_rn(make_float2(__uint_as_float(x[t]), __uint_as_float(x[t + 1])),
                                      make_float2(f[t], f[t + 1]));
                // a masked score may be NaN (another sequence's key): selected away, not multiplied by 0
                if (t < first) y.x = 0.f;
                if (t + 1 < first) y.y = 0.f;
                x[t] = __float_as_uint(y.x);
                x[t + 1] = __float_as_uint(y.y);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int t = 8 * c + 2 * j;
                    split3(make_float2(__uint_as_float(x[t]), __uint_as_float(x[t + 1])), hi[j], mid[j], lo[j]);
                }
                const uint32_t a = at + (((begin / 8 + c) ^ (s & 7)) << 4);
                tc::sts128(a, hi[0], hi[1], hi[2], hi[3]);
                tc::sts128(a + kPTile, mid[0], mid[1], mid[2], mid[3]);
                tc::sts128(a + 2 * kPTile, lo[0], lo[1], lo[2], lo[3]);
            }
        };
        for (int n = 0; n < nitems && ok; ++n) {
            if (!warp_wait(&bar[B_SCORES], n & 1)) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t x[32];
            tc::tmem_ld32x32b_x32(taddr, x);
            tc::tmem_wait_ld();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_SCFREE]);
            if (!warp_wait(&bar[B_PFREE + (n & 1)], ((n >> 1) & 1) ^ 1)) { ok = false; break; }
            const uint32_t at = prow + (n & 1) * 3 * kPTile;
            convert(x, at, warp == 4 ? 0 : lane);
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_P + (n & 1)]);
        }
    } else if (warp >= kSWarp && warp < kSWarp + kSWarps) {
        // ------------------------------------------------------ S
        // Lane = v index; the second four warps take the second half of the
        // columns.  Per chunk: the three terms of S for the outputs and
        // lam^rows S back into the accumulator for the update.
        constexpr int kCols = D / 2, kBatches = kCols / 16;
        const int w = warp & 3, dv = 32 * w + lane, c0 = warp - kSWarp < 4 ? 0 : kCols;
        const bool live = 32 * w < D;
        const uint32_t ts = tmem + (static_cast<uint32_t>(32 * w) << 16) + L::COL_S + c0;
        const uint32_t tb = tmem + (static_cast<uint32_t>(32 * w) << 16) + L::COL_SB + c0 / 2;
        const int64_t head = static_cast<int64_t>(D) * D;
        auto state_at = [&](int load) -> const float* {
            if (load == kFromBounds)
                return P.bounds + (static_cast<int64_t>(blockIdx.x - 1) * A.num_kv_heads + h) * head;
            if (load == kFromStarts) return P.starts + (static_cast<int64_t>(blockIdx.x) * A.num_kv_heads + h) * head;
            return load >= 0 ? A.states + (static_cast<int64_t>(load) * A.num_kv_heads + h) * head : nullptr;
        };
        auto split = [&](uint32_t (&x)[16], int b, float2 lam) {
            uint32_t hi[8], mid[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float2 y = make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                split3(y, hi[j], mid[j], lo[j]);
                y = __ffma2_rn(y, make_float2(lam.x, lam.x), __fmul2_rn(y, make_float2(lam.y, lam.y)));
                x[2 * j] = __float_as_uint(y.x);
                x[2 * j + 1] = __float_as_uint(y.y);
            }
            tc::tmem_st32x32b_x8(tb + 8 * b, hi);
            tc::tmem_st32x32b_x8(tb + D / 2 + 8 * b, mid);
            tc::tmem_st32x32b_x8(tb + D + 8 * b, lo);
            tc::tmem_st32x32b_x16(ts + 16 * b, x);
        };
        int i = 0;  // chunk of the range
        for (int k = 0; k < nseg && ok; ++k) {
            const int rows = segs[k].rows, store = segs[k].store;
            if (rows <= 0) continue;
            // The last segment's update has to be in before S is replaced.
            if (i > 0 && !warp_wait(&bar[B_VTFREE], (i - 1) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            const float* from = state_at(segs[k].load);
            if (live) {
#pragma unroll 1
                for (int b = 0; b < kCols / 32; ++b) {
                    uint32_t x[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        x[j] = from != nullptr ? __float_as_uint(from[(c0 + 32 * b + j) * D + dv]) : 0u;
                    tc::tmem_st32x32b_x32(ts + 32 * b, x);
                }
                tc::tmem_wait_st();
            }
            if (k + 1 < nseg && segs[k + 1].rows > 0 && segs[k + 1].load >= 0) {
                const float* next = state_at(segs[k + 1].load);
                for (int j = threadIdx.x - 32 * kSWarp; j < D * D / 32; j += 32 * kSWarps) prefetch_l2(next + 32 * j);
            }
            for (int left = rows; left > 0; left -= C, ++i) {
                // S may be read when the last chunk's update is in it, its
                // terms replaced when the last outputs have read them.
                if (i > 0 && !warp_wait(&bar[B_VTFREE], (i - 1) & 1)) { ok = false; break; }
                tc::fence_after_sync();
                uint32_t xa[16], xb[16];
                if (live) tc::tmem_ld32x32b_x16(ts, xa);
                if (i > 0 && !warp_wait(&bar[B_SFREE], (i - 1) & 1)) { ok = false; break; }
                tc::fence_after_sync();
                // a tail's factor is applied once: fp32 is enough
                const float2 lam = left >= C ? make_float2(tab[TAB_LAM], tab[TAB_LAM + 1]) : make_float2(tab[TAB_V + left], 0.f);
                if (live) {
#pragma unroll 1
                    for (int b = 0; b < kBatches; b += 2) {
                        tc::tmem_wait_ld();
                        tc::tmem_ld32x32b_x16(ts + 16 * b + 16, xb);
                        split(xa, b, lam);
                        tc::tmem_wait_ld();
                        if (b + 2 < kBatches) tc::tmem_ld32x32b_x16(ts + 16 * b + 32, xa);
                        split(xb, b + 1, lam);
                    }
                    tc::tmem_wait_st();
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar[B_S]);
                if (DEALT && store < -1 && left == rows && lane == 0) {
                    // The same warp of every CTA that reads the slot holds the
                    // same part of the state.  Whoever comes last here
                    // knows that the others have read it, and stores it at
                    // the end.  Here, because this warp waits for the update
                    // next (at the end it would be 1 us a segment).
                    const int at = 4 * (warp - kSWarp);
                    __threadfence();
                    const uint32_t before =
                        atomicAdd(P.claims + static_cast<int64_t>(segs[k].seq) * A.num_kv_heads + h, 1u << at);
                    __threadfence();
                    rest.stores[warp - kSWarp] = ((before >> at) & 15u) == static_cast<uint32_t>(P.subs - 1);
                }
            }
            if (!ok || store == -1) continue;
            int slot = store;
            if constexpr (DEALT) {
                __syncwarp();
                if (store < -1) {
                    if (!rest.stores[warp - kSWarp]) continue;
                    slot = -2 - store;
                }
            }
            if (!warp_wait(&bar[B_VTFREE], (i - 1) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (live) {
                float* to = A.states + (static_cast<int64_t>(slot) * A.num_kv_heads + h) * head + dv;
#pragma unroll 1
                for (int b = 0; b < kCols / 32; ++b) {
                    uint32_t x[32];
                    tc::tmem_ld32x32b_x32(ts + 32 * b, x);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) to[(c0 + 32 * b + j) * D] = __uint_as_float(x[j]);
                }
            }
        }
    } else if (warp == kLoadWarp || (warp >= 5 && warp < 8)) {
        // ------------------------------------------------------ loads and V~
        // The load warp converts its share too.  The loads that follow chunk
        // i's conversion wait for items that end before the next conversion
        // could start, so neither holds the other up.
        Cursor kv_at(segs, nseg), q_at(segs, nseg), at(segs, nseg);
        int kv_next = 0, q_next = 0;
        auto load_kv = [&]() -> bool {
            if (kv_next >= nch) return true;
            const int st = kv_next % kKv;
            if (!warp_wait(&bar[B_KVEMPTY + st], ((kv_next / kKv) & 1) ^ 1)) return false;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx(&bar[B_KVFULL + st], 2u * kPanels * kPanel);
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) {
                    tc::tma_load_3d(smem + L::OFF_K + st * kTile + pn * kPanel, &tm_k, 64 * pn, h, kv_at.row,
                                    &bar[B_KVFULL + st]);
                    tc::tma_load_3d(smem + L::OFF_V + st * kTile + pn * kPanel, &tm_v, 64 * pn, h, kv_at.row,
                                    &bar[B_KVFULL + st]);
                }
            }
            __syncwarp();
            ++kv_next;
            kv_at.next();
            return true;
        };
        auto load_q = [&]() -> bool {
            if (q_next >= nitems) return true;
            const int st = q_next % kQ;
            if (!warp_wait(&bar[B_QEMPTY + st], ((q_next / kQ) & 1) ^ 1)) return false;
            if (tc::elect_one()) {
                mbar_arrive_expect_tx(&bar[B_QFULL + st], static_cast<uint32_t>(kPanels) * kPanel);
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn)
                    tc::tma_load_3d(smem + L::OFF_Q + st * kTile + pn * kPanel, &tm_q, 64 * pn, hq0 + q_next % G,
                                    q_at.row, &bar[B_QFULL + st]);
            }
            __syncwarp();
            ++q_next;
            if (q_next % G == 0) q_at.next();
            return true;
        };
        if (warp == kLoadWarp) {
            ok = load_kv();
            for (int n = 0; n < kQ && ok; ++n) ok = load_q();
            for (int i = 1; i < kKv - 1 && ok; ++i) ok = load_kv();
        }
        const int tid = 32 * (warp == kLoadWarp ? 0 : warp - 4) + lane;
        for (int i = 0; i < nch && ok; ++i) {
            const int st = i % kKv;
            if (!warp_wait(&bar[B_KVFULL + st], (i / kKv) & 1)) { ok = false; break; }
            if (!warp_wait(&bar[B_VTFREE], (i & 1) ^ 1)) { ok = false; break; }
            const int nrows = min(C, at.left);
            at.next();
            // Chunk i - 1's update has read its first item's q by now.
            if (warp == kLoadWarp && i > 0)
                while (q_next <= (i - 1) * G + kQ && q_next < nitems && ok) ok = load_q();
            const uint32_t sk = smem_addr(smem + L::OFF_K + st * kTile), sv = smem_addr(smem + L::OFF_V + st * kTile);
            const float acc = convert_v<D, kTile, 32 * kVWarps, 4>(sk, sv, smem_addr(smem + L::OFF_VT), tab + TAB_V,
                                                                     nrows, tid);
            if (acc != 0.f) {
                // A value that is not finite reaches the outputs of its column
                // from its row on, and no earlier row: it leaves V for P V
                // (V~ carries it into the state), and its row is noted.
                for (int c = tid; c < C * D * 2 / 16; c += 32 * kVWarps) {
                    const int row = (c >> 3) & (C - 1);
                    if (row >= nrows) continue;
                    uint32_t x[4];
                    tc::lds128(sv + c * 16, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t u = (x[e / 2] >> (16 * (e % 2))) & 0xffffu;
                        if ((u & 0x7f80u) == 0x7f80u) {
                            x[e / 2] &= e % 2 ? 0x0000ffffu : 0xffff0000u;
                            const int col = (c >> 9) * 64 + (((c & 7) ^ (row & 7)) << 3) + e;
                            atomicMax(&rest.bad_rows[i % kBadBuffers][col], ((i + 1) << 6) | (C - 1 - row));
                        }
                    }
                    tc::sts128(sv + c * 16, x[0], x[1], x[2], x[3]);
                }
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_VT]);
            if (warp == kLoadWarp) {
                while (q_next < i * G + kQ && q_next < nitems && ok) ok = load_q();
                ok = ok && load_kv();
            }
        }
        if (warp == kLoadWarp)
            while (q_next < nitems && ok) ok = load_q();
    } else {
        // ------------------------------------------------------ outputs
        // Lane = v index, column = token: a warp stores 32 consecutive floats
        // of a row; the second four warps take tokens 32-63.  The state's part
        // is taken into registers as soon as it is there, so that the next
        // item's can be computed.
        const int w = warp & 3, dv = 32 * w + lane, t0 = warp - kOWarp < 4 ? 0 : 32;
        const bool live = 32 * w < D;
        const uint32_t tl = tmem + (static_cast<uint32_t>(32 * w) << 16) + t0;
        const int64_t row_step = static_cast<int64_t>(A.num_q_heads) * D;
        const float* f = tab + TAB_O + t0;
        const int64_t row_bytes = row_step * 4;
        Cursor at(segs, nseg);
        for (int n = 0; n < nitems && ok; ++n) {
            const int i = n / G, g = n % G;
            if (!warp_wait(&bar[B_OS], n & 1)) { ok = false; break; }
            tc::fence_after_sync();
            uint32_t xs[32];
            if (live) {
                tc::tmem_ld32x32b_x32(tl + L::COL_OS, xs);
                tc::tmem_wait_ld();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_OSFREE]);
            // the factors here, not among the stores, which they could not be loaded past
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                const float4 ff = *reinterpret_cast<const float4*>(f + j);
                xs[j] = __float_as_uint(ff.x * __uint_as_float(xs[j]));
                xs[j + 1] = __float_as_uint(ff.y * __uint_as_float(xs[j + 1]));
                xs[j + 2] = __float_as_uint(ff.z * __uint_as_float(xs[j + 2]));
                xs[j + 3] = __float_as_uint(ff.w * __uint_as_float(xs[j + 3]));
            }
            if (!warp_wait(&bar[B_OP], n & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (live) {
#pragma unroll
                for (int part = L::kSums - 1; part >= 0; --part) {
                    uint32_t xp[32];
                    tc::tmem_ld32x32b_x32(tl + L::COL_OP + part * C, xp);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        xs[j] = __float_as_uint(__uint_as_float(xs[j]) + __uint_as_float(xp[j]));
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[B_OPFREE]);
            if (live) {
                const int nrows = min(C, at.left) - t0;
                const int mark = rest.bad_rows[i % kBadBuffers][dv];
                const int nan_from = max(((mark >> 6) == i + 1 ? C - 1 - (mark & (C - 1)) : C) - t0, 0);
                float* o = A.out + (static_cast<int64_t>(at.row) + t0) * row_step + (hq0 + g) * D + dv;
                const int plain = min(nrows, nan_from);
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    if (j < plain) *o = __uint_as_float(xs[j]);
                    o = walk(o, row_bytes);
                }
                for (int j = plain; j < min(nrows, 32); ++j)  // behind a value that is not finite
                    o[(j - 32) * row_step] = __int_as_float(0x7fffffff);
            }
            if (g == G - 1) at.next();
        }
    }
    if (info[I_BAD]) {
        for (int k = 0; k < nseg; ++k) {
            const int64_t n = -static_cast<int64_t>(segs[k].rows) * G * D;  // negative for the others
            for (int64_t i = threadIdx.x; i < n; i += kThreads)
                A.out[(segs[k].row0 + i / (G * D)) * static_cast<int64_t>(A.num_q_heads) * D + hq0 * D +
                      i % (G * D)] = 0.f;
        }
    }
    if (reports) {
        // A slot that two sequences store to, or that one stores to and
        // another reads, has no defined content: reported.
        for (int k = 0; k < nseg; ++k) {
            if (segs[k].rows <= 0 || !segs[k].first) continue;
            const int to = __ldg(A.new_slots + segs[k].seq);
            if (to < 0) continue;
            for (int o = threadIdx.x; o < A.num_seqs; o += kThreads)
                if (o != segs[k].seq && linear_shares(A, o, to))
                    record_error(A.err, kErrAlias, static_cast<uint32_t>(segs[k].seq));
        }
    }
    if (!ok) record_error(A.err, kErrTimeout, 0x200u + static_cast<uint32_t>(warp));
    // ---------------------------------------------------------- teardown
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == kLoadWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- ranges' own states
// The own state, from zero, of a range's last segment, where its sequence
// goes on in the next range: sum_s lam^(end-1-s) k_s v_s^T over the segment's
// tokens, one accumulation with no rescaling (the factor of a chunk's end is
// part of V~).  Warps 0-7 make V~, 8 loads, 9 issues the MMAs; warps 0-3
// store the sum.  Warps 10 and 11 copy the state that the call replaces in place,
// if it does: beside the others (after them it was 1.3 us of a prompt of 300
// tokens).  There is room in tensor memory here, so V~ goes there: it
// is read from the V tile by transposing 8x8 loads, whose fragments are what
// a 16-lane store takes, and the product needs shared memory for K alone.
// (With V~ in shared memory the kernel was bound by it: 31 us for 8 ranges of
// 29 chunks and 16 heads of 128.)
constexpr int kStateThreads = 384;
constexpr int kStateStages = 5;
constexpr int kTile = 2 * kPanel;        // room for head_dim 128
constexpr int SOFF_K = 0;
constexpr int SOFF_V = SOFF_K + kStateStages * kTile;
constexpr int SOFF_BAR = SOFF_V + kStateStages * kTile;
enum { SB_FULL = 0, SB_EMPTY = kStateStages, SB_VT = 2 * kStateStages, SB_VTFREE = SB_VT + 2, SB_DONE = SB_VTFREE + 2, SNBAR };
constexpr int SOFF_INFO = SOFF_BAR + SNBAR * 8;
constexpr int SOFF_TMEM = SOFF_INFO + 8 * 4;
constexpr int STATE_SMEM = SOFF_TMEM + 16 + 1024;
static_assert(STATE_SMEM <= 232448, "shared memory budget (227 KB)");
static_assert(2 * STATE_SMEM > 228 * 1024, "the 512-column TMEM allocation needs one CTA per SM");
constexpr uint32_t SCOL_VT = 128;        // V~: two buffers of three terms of 32 columns

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t saddr, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                 : "r"(saddr)
                 : "memory");
}

template <int D>
__global__ void __launch_bounds__(kStateThreads, 1)
    linear_state_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const ChunkParams P) {
    constexpr int kPanels = D / 64;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + SOFF_BAR);
    int* info = reinterpret_cast<int*>(smem + SOFF_INFO);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + SOFF_TMEM);
    const LinearArgs& A = P.A;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int h = blockIdx.y;
    griddep_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < SNBAR; ++i) mbar_init(&bar[i], i == SB_VT || i == SB_VT + 1 ? 8u : 1u);
        fence_mbar_init();
    }
    if (warp == 8) {
        tc::tmem_alloc(tmem_slot, kTmemCols);
        tc::tmem_relinquish();
        if (lane == 0) {
            tc::prefetch_tensormap(&tm_k);
            tc::prefetch_tensormap(&tm_v);
        }
    }
    griddep_wait();
    if (warp == 0) {
        const int u0 = blockIdx.x * P.range, u1 = u0 + P.range;
        if (lane == 0) {
            info[0] = info[1] = 0;
            info[2] = -1;
            if (h == 0) P.tails[blockIdx.x] = make_int4(0, 0, 0, -1);
        }
        __syncwarp();
        scan_units(P, u1 - 1, u1, false, [&](int, const LinearSeq& q, int first, int end, bool in, unsigned) {
            if (!in || end <= u1 || q.bad) return;
            const int c0 = max(u0, first) - first, c1 = u1 - first;
            info[0] = q.row0 + c0 * C;
            info[1] = c1 - c0;
            if (c0 == 0 && q.load == q.store) info[2] = q.load;
            // chunks, whether it holds the sequence's first row, and the state that goes before it
            if (h == 0) P.tails[blockIdx.x] = make_int4(c1 - c0, c0 == 0, 0, q.load);
        });
    } else if (warp == 10 && P.subs > 1) {
        const int64_t n = static_cast<int64_t>(A.num_seqs) * A.num_kv_heads;
        for (int64_t i = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 32 + lane; i < n;
             i += static_cast<int64_t>(gridDim.x) * gridDim.y * 32)
            P.claims[i] = 0;
    }
    const float g = clean_log_decay(A, h, false);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int row0 = info[0], nch = info[1];
    bool ok = true;
    if (warp == 8) {
        const uint64_t policy = P.overflow ? l2_policy_evict_first() : tc::l2_policy_evict_normal();
        for (int i = 0; i < nch && ok; ++i) {
            const int st = i % kStateStages;
            if (!warp_wait(&bar[SB_EMPTY + st], ((i / kStateStages) & 1) ^ 1)) { ok = false; break; }
            if (tc::elect_one()) {
                mbar_arrive_expect_tx(&bar[SB_FULL + st], 2u * kPanels * kPanel);
#pragma unroll
                for (int pn = 0; pn < kPanels; ++pn) {
                    tc::tma_load_3d(smem + SOFF_V + st * kTile + pn * kPanel, &tm_v, 64 * pn, h, row0 + i * C,
                                    &bar[SB_FULL + st], policy);
                    tc::tma_load_3d(smem + SOFF_K + st * kTile + pn * kPanel, &tm_k, 64 * pn, h, row0 + i * C,
                                    &bar[SB_FULL + st], policy);
                }
            }
            __syncwarp();
        }
    } else if (warp == 9) {
        for (int i = 0; i < nch && ok; ++i) {
            const int st = i % kStateStages, vb = i & 1;
            if (!warp_wait(&bar[SB_VT + vb], (i >> 1) & 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (tc::elect_one()) {
                constexpr uint32_t kIdesc = tc::idesc_bf16_f32(128, D, 0, 1);
                const uint64_t b = tc::smem_desc_sw128(smem_addr(smem + SOFF_K + st * kTile), kPanel, 1024);
#pragma unroll 1
                for (int part = 2; part >= 0; --part) {  // smallest first: the sums truncate
                    const uint32_t a = tmem + SCOL_VT + (vb * 3 + part) * (C / 2);
#pragma unroll
                    for (int k = 0; k < C / 16; ++k)
                        tc::mma_bf16_ts(tmem, a + 8 * k, b + k * (2048 >> 4), kIdesc,
                                        i > 0 || part < 2 || k > 0 ? 1u : 0u);
                }
                tc::mma_commit(&bar[SB_EMPTY + st]);
                tc::mma_commit(&bar[SB_VTFREE + vb]);
                if (i == nch - 1) tc::mma_commit(&bar[SB_DONE]);
            }
            __syncwarp();
        }
    } else if (warp >= 10) {
        if (info[2] >= 0) {
            const float4* src = reinterpret_cast<const float4*>(
                A.states + (static_cast<int64_t>(info[2]) * A.num_kv_heads + h) * D * D);
            float4* dst = reinterpret_cast<float4*>(
                P.starts + (static_cast<int64_t>(blockIdx.x) * A.num_kv_heads + h) * D * D);
            constexpr int kCopiers = kStateThreads - 320, kAhead = 16;
#pragma unroll 1
            for (int at = threadIdx.x - 320; at < D * D / 4; at += kCopiers * kAhead) {
                float4 x[kAhead];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) x[j] = src[at + kCopiers * j];
#pragma unroll
                for (int j = 0; j < kAhead; ++j) dst[at + kCopiers * j] = x[j];
            }
        }
    } else {
        // Warp w: 16 lanes (v indices) from 32 (w % 4) + 16 (w / 4).  Thread t
        // holds lanes t/4 and t/4 + 8 of them, tokens 8 g + 2 (t % 4) and + 1.
        const int dv0 = 32 * (warp & 3) + 16 * (warp >> 2);
        const bool live = dv0 < D;
        const int m = lane >> 3;  // the matrix whose row address this lane gives
        const uint32_t row = 8 * (m >> 1) + (lane & 7);
        const uint32_t from = (dv0 / 64) * kPanel + row * 128 + ((((dv0 % 64) / 8 + (m & 1)) ^ (lane & 7)) << 4);
        const uint32_t to = tmem + (static_cast<uint32_t>(dv0) << 16) + SCOL_VT;
        float2 f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int s = 8 * j + 2 * (lane & 3);
            f[j] = make_float2(expf(g * static_cast<float>(C - 1 - s)), expf(g * static_cast<float>(C - 2 - s)));
        }
        for (int i = 0; i < nch && ok; ++i) {
            const int st = i % kStateStages, vb = i & 1;
            const float x = expf(g * static_cast<float>((nch - 1 - i) * C));
            const float2 end = make_float2(x, x);
            if (!warp_wait(&bar[SB_FULL + st], (i / kStateStages) & 1)) { ok = false; break; }
            if (!warp_wait(&bar[SB_VTFREE + vb], ((i >> 1) & 1) ^ 1)) { ok = false; break; }
            tc::fence_after_sync();
            if (live) {
                const uint32_t tile = smem_addr(smem + SOFF_V + st * kTile) + from;
                uint32_t v[16], hi[16], mid[16], lo[16];
#pragma unroll
                for (int j = 0; j < 4; ++j)  // 16 tokens each
                    ldmatrix_x4_trans(tile + j * 2048, v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    split3(__fmul2_rn(unpack_bf16(v[j]), __fmul2_rn(f[j / 2], end)), hi[j], mid[j], lo[j]);
                tc::tmem_st16x128b_x8(to + (vb * 3) * (C / 2), hi);
                tc::tmem_st16x128b_x8(to + (vb * 3 + 1) * (C / 2), mid);
                tc::tmem_st16x128b_x8(to + (vb * 3 + 2) * (C / 2), lo);
                tc::tmem_wait_st();
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar[SB_VT + vb]);
        }
        if (ok && nch > 0 && 32 * warp < D) {
            if (!warp_wait(&bar[SB_DONE], 0)) {
                ok = false;
            } else {
                tc::fence_after_sync();
                float* to = P.bounds + (static_cast<int64_t>(blockIdx.x) * A.num_kv_heads + h) * D * D + 32 * warp + lane;
#pragma unroll
                for (int b = 0; b < D / 32; ++b) {
                    uint32_t x[32];
                    tc::tmem_ld32x32b_x32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + 32 * b, x);
                    tc::tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) to[(32 * b + j) * D] = __uint_as_float(x[j]);
                }
            }
        }
    }
    if (!ok) record_error(A.err, kErrTimeout, 0x300u + static_cast<uint32_t>(warp));
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tmem, kTmemCols);
}

__global__ void __launch_bounds__(kScanThreads) linear_scan_kernel(const LinearArgs A, const LinearScan S) {
    griddep_launch_dependents();
    griddep_wait();
    scan_ranges(A, S, blockIdx.x);
}

// The counters of dealt q heads, where linear_state_kernel does not clear them.
__global__ void __launch_bounds__(kScanThreads) linear_clear_kernel(uint32_t* claims, int64_t n) {
    griddep_launch_dependents();
    griddep_wait();
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kScanThreads + threadIdx.x; i < n;
         i += static_cast<int64_t>(gridDim.x) * kScanThreads)
        claims[i] = 0;
}

bool rows_map(CUtensorMap* map, const void* base, int64_t stride, int32_t heads, int32_t d, int32_t tokens) {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {64, 1, C};
    return make_bf16_map(map, base, 3, dims, strides, box);
}

template <typename K>
cudaError_t configure(K kernel, int smem, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess || (dev < 64 && done[dev])) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

template <int D, int G, bool DEALT>
cudaError_t launch_main(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& P,
                        cudaStream_t stream) {
    static bool done[64] = {};
    cudaError_t e = configure(linear_chunk_kernel<D, G, DEALT>, smem_bytes<D>(), done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(linear_chunk_kernel<D, G, DEALT>, dim3(P.ranges, P.A.num_kv_heads * P.subs), dim3(kThreads),
                             smem_bytes<D>(), stream, tq, tk, tv, P);
}

template <int D>
cudaError_t launch_state(const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& P, cudaStream_t stream) {
    static bool done[64] = {};
    cudaError_t e = configure(linear_state_kernel<D>, STATE_SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_overlapped(linear_state_kernel<D>, dim3(P.ranges - 1, P.A.num_kv_heads), dim3(kStateThreads),
                             STATE_SMEM, stream, tk, tv, P);
}

template <int D, bool DEALT>
cudaError_t launch_groups(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& P,
                          cudaStream_t stream) {
    switch (P.A.num_q_heads / P.A.num_kv_heads / P.subs) {
        case 1: return launch_main<D, 1, DEALT>(tq, tk, tv, P, stream);
        case 2: return launch_main<D, 2, DEALT>(tq, tk, tv, P, stream);
        case 4: return launch_main<D, 4, DEALT>(tq, tk, tv, P, stream);
        default: return launch_main<D, DEALT ? 4 : 8, DEALT>(tq, tk, tv, P, stream);  // 8 are never dealt
    }
}

}  // namespace

// Ranges a plan may have: two waves of CTAs, or what keeps every range within
// the segments a CTA lists.
static int64_t max_ranges(int32_t num_seqs, int32_t num_tokens, int32_t num_kv_heads, int num_sms) {
    const int64_t waves = (2 * static_cast<int64_t>(num_sms) + num_kv_heads - 1) / num_kv_heads;
    const int64_t units = num_tokens / C + num_seqs;
    const int64_t lists = num_seqs > kMaxSegments ? (units + kMaxSegments - 1) / kMaxSegments : 0;
    return waves > lists ? waves : lists;
}

static size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t linear_workspace_bytes(int32_t num_seqs, int32_t num_tokens, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int num_sms) {
    const size_t n = static_cast<size_t>(max_ranges(num_seqs, num_tokens, num_kv_heads, num_sms));
    return round256(n * sizeof(int4)) + 2 * n * num_kv_heads * head_dim * head_dim * sizeof(float) +
           n * num_q_heads * kMaxSegments * sizeof(Segment) +
           static_cast<size_t>(num_seqs) * num_kv_heads * sizeof(uint32_t);
}

LinearPlan plan_linear(const int32_t* qsl, int32_t num_seqs, int32_t num_tokens, int32_t num_kv_heads, int32_t group,
                       int32_t head_dim, int num_sms, int32_t max_recurrent) {
    LinearPlan best = {0, 0, 0, 0, 1, false};
    int64_t units = 0;
    for (int32_t s = 0; s < num_seqs; ++s) {
        const int32_t rows = qsl[s + 1] - qsl[s];
        if (rows <= max_recurrent) best.recurrent = rows > best.recurrent ? rows : best.recurrent;
        else units += (rows + C - 1) / C;
    }
    if (units == 0) return best;
    best.units = static_cast<int32_t>(units);
    const int64_t most = max_ranges(num_seqs, num_tokens, num_kv_heads, num_sms);
    // Whether a range may end at a unit without cutting a sequence (without
    // the room to say so, none may: the join is then launched needlessly).
    std::unique_ptr<uint8_t[]> begins(new (std::nothrow) uint8_t[static_cast<size_t>(units)]());
    for (int32_t s = 0, at = 0; s < num_seqs && begins; ++s) {
        const int32_t rows = qsl[s + 1] - qsl[s];
        if (rows <= max_recurrent) continue;
        begins[at] = 1;
        at += (rows + C - 1) / C;
    }
    // Microseconds of a chunk in the main kernel (what a chunk costs, and each
    // of its q heads) and in the state kernel, of a kernel's start and end,
    // and of the two more kernels that join ranges.  More ranges fill more
    // SMs; where they cut sequences, the state kernel reads K and V of all but
    // the last range once more, and the states are carried over.  Dealing a
    // group's q heads to several CTAs fills SMs too, repeats the state's work
    // in each, and takes a launch that clears their counters where the state
    // kernel is not there to do it.  The constants are fitted to the times of
    // forced plans over nine batches (128 to 16,384 tokens, both widths, one
    // sequence and many), of which the plans taken were within 4 % of the best.
    const bool narrow = head_dim == 64;
    const double fixed = narrow ? 0.45 : 1.3, item = narrow ? 1.25 : 1.3, state = narrow ? 0.5 : 1.0, start = 5.5,
                 clear = 0.9;
    const int64_t least = num_seqs > kMaxSegments ? (units + kMaxSegments - 1) / kMaxSegments : 1;
    const int64_t last = most < units ? most : units;
    double best_us = 1e30;
    for (int32_t subs = 1; subs <= group; subs *= 2) {
        const int64_t heads = static_cast<int64_t>(num_kv_heads) * subs;
        const double chunk = fixed + item * (group / subs);
        auto consider = [&](int64_t count) {
            if (count < least || count > last) return;
            const int64_t range = (units + count - 1) / count, ranges = (units + range - 1) / range;  // count or fewer
            double us = (ranges * heads + num_sms - 1) / num_sms * (start + range * chunk);
            if (us >= best_us) return;
            bool cut = false;  // whether a border lies inside a sequence
            for (int64_t u = range; u < units && !cut; u += range) cut = !begins || begins[u] == 0;
            if (cut) us += 7.0 + 0.15 * ranges + ((ranges - 1) * num_kv_heads + num_sms - 1) / num_sms * range * state;
            if (subs > 1 && !cut) us += clear;
            if (us >= best_us) return;
            best_us = us;
            best.ranges = static_cast<int32_t>(ranges);
            best.range = static_cast<int32_t>(range);
            best.subs = subs;
            best.cut = cut;
        };
        // What fits one and two waves of CTAs, then a spread of counts.
        consider(num_sms / heads);
        consider(2 * num_sms / heads);
        for (int64_t n = least; n <= last; n += 1 + n / 16) consider(n);
    }
    return best;
}

cudaError_t launch_linear_prefill(const LinearArgs& a, const LinearPlan& plan, void* workspace, int num_sms,
                                  cudaStream_t stream) {
    if (plan.units == 0)
        return plan.recurrent > 0 ? launch_linear_recurrent(a, plan.recurrent, LinearScan{}, stream) : cudaSuccess;
    CUtensorMap tq, tk, tv;
    if (!rows_map(&tq, a.q, a.q_stride, a.num_q_heads, a.head_dim, a.num_tokens) ||
        !rows_map(&tk, a.k, a.k_stride, a.num_kv_heads, a.head_dim, a.num_tokens) ||
        !rows_map(&tv, a.v, a.v_stride, a.num_kv_heads, a.head_dim, a.num_tokens))
        return cudaErrorInvalidValue;
    const size_t n = static_cast<size_t>(max_ranges(a.num_seqs, a.num_tokens, a.num_kv_heads, num_sms));
    ChunkParams P;
    P.A = a;
    uint8_t* at = static_cast<uint8_t*>(workspace);
    P.tails = reinterpret_cast<int4*>(at);
    at += round256(n * sizeof(int4));
    P.bounds = reinterpret_cast<float*>(at);
    const size_t states = n * a.num_kv_heads * static_cast<size_t>(a.head_dim) * a.head_dim;
    at += states * sizeof(float);
    P.starts = P.bounds + states;
    at += states * sizeof(float);
    P.segments = reinterpret_cast<Segment*>(at);
    at += n * a.num_q_heads * kMaxSegments * sizeof(Segment);
    P.claims = reinterpret_cast<uint32_t*>(at);
    P.ranges = plan.ranges;
    P.range = plan.range;
    P.units = plan.units;
    P.subs = plan.subs;
    P.cut = plan.cut;
    P.overflow = static_cast<int64_t>(plan.units) * C * a.num_kv_heads * a.head_dim * 4 > kOverflowBytes;
    LinearScan scan = {};
    cudaError_t e = cudaSuccess;
    if (plan.cut) {
        e = a.head_dim == 64 ? launch_state<64>(tk, tv, P, stream) : launch_state<128>(tk, tv, P, stream);
        if (e != cudaSuccess) return e;
        scan.bounds = P.bounds;
        scan.tails = P.tails;
        scan.ranges = P.ranges;
        scan.tokens = P.range * C;
        scan.blocks = a.num_kv_heads * (a.head_dim * a.head_dim / (2 * kScanThreads));
    }
    // The scan rides in the recurrent form's grid where there is one.
    if (plan.recurrent > 0)
        e = launch_linear_recurrent(a, plan.recurrent, scan, stream);
    else if (plan.cut)
        e = launch_overlapped(linear_scan_kernel, dim3(scan.blocks), dim3(kScanThreads), 0, stream, a, scan);
    if (e != cudaSuccess) return e;
    if (plan.subs > 1 && !plan.cut) {
        const int64_t n = static_cast<int64_t>(a.num_seqs) * a.num_kv_heads;
        const int64_t blocks = (n + 8 * kScanThreads - 1) / (8 * kScanThreads);
        e = launch_overlapped(linear_clear_kernel, dim3(static_cast<unsigned>(blocks < num_sms ? blocks : num_sms)),
                              dim3(kScanThreads), 0, stream, P.claims, n);
        if (e != cudaSuccess) return e;
    }
    if (P.subs > 1)
        return a.head_dim == 64 ? launch_groups<64, true>(tq, tk, tv, P, stream)
                                : launch_groups<128, true>(tq, tk, tv, P, stream);
    return a.head_dim == 64 ? launch_groups<64, false>(tq, tk, tv, P, stream)
                            : launch_groups<128, false>(tq, tk, tv, P, stream);
}

}  // namespace pkv
