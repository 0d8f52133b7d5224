// prefill_tile.cuh -- which query rows a CTA of the prefill kernels takes.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "pkv_device.cuh"

namespace pkv {

constexpr int kPrefillRows = 128;  // query rows of a CTA and q head

// A CTA's share of a mixed batch: rows row0 .. row0 + rows - 1 of sequence s,
// at positions pmin .. pmax, for `units` q heads from h0 on; nt key tiles of
// 128, the last with klast visible keys.  bad: the sequence's context is out
// of range (its rows are zero), or the call has no such tile or rows (s < 0).
struct PrefillTile {
    int s, row0, rows, pmin, pmax, nt, klast, bad, units, h0;
};

// For a whole warp, the result on every lane.  Entries are numbered over the
// prefill sequences (query_len > 1) in order, one per row tile of 128 rows
// (ceil(qlen/128) tiles), and two for each of the last split_last tiles (one
// per q head).
__device__ __forceinline__ PrefillTile find_prefill_tile(const int32_t* qsl, const int32_t* context_lens,
                                                         int num_seqs, int num_tokens, int ctx_cap,
                                                         int cta_units, int split_last, int tile, int pair,
                                                         unsigned long long* err, int lane) {
    const unsigned FULL = 0xffffffffu;
    const int split = cta_units == 2 ? split_last : 0;
    int base = 0, found = -1, e = 0, nt_s = 0;
    for (int s0 = 0; s0 < num_seqs && found < 0; s0 += 32) {
        const int s = s0 + lane;
        int nt = 0;
        if (s < num_seqs) {
            const int ql = __ldg(qsl + s + 1) - __ldg(qsl + s);
            nt = ql > 1 ? (ql + kPrefillRows - 1) / kPrefillRows : 0;
        }
        const int ne = nt + min(split, nt);
        int incl = ne;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(FULL, base + incl > tile);
        if (hit) {
            const int j = __ffs(hit) - 1;
            found = s0 + j;
            e = tile - (base + __shfl_sync(FULL, incl - ne, j));
            nt_s = __shfl_sync(FULL, nt, j);
        } else {
            base += __shfl_sync(FULL, incl, 31);
        }
    }
    // Entry e of the sequence: row tile e while e < nt - sl (both heads), then
    // tile nt - sl + (e - (nt - sl)) / 2, one head each.
    const int sl = min(split, nt_s);
    PrefillTile r = {};
    r.s = found;
    r.units = cta_units;
    r.h0 = pair * cta_units;
    int tloc = e;
    if (sl > 0 && e >= nt_s - sl) {
        const int k = e - (nt_s - sl);
        tloc = nt_s - sl + k / 2;
        r.units = 1;
        r.h0 += k % 2;
    }
    if (found < 0) {
        r.bad = 1;
        return r;
    }
    const int q0 = __ldg(qsl + found);
    const int ql = __ldg(qsl + found + 1) - q0;
    if (q0 < 0 || q0 > num_tokens - ql) {  // rows the call does not have
        if (lane == 0) record_error(err, kErrRange, static_cast<uint32_t>(found));
        r.s = -1;
        r.bad = 1;
        return r;
    }
    const int ctx = __ldg(context_lens + found);
    if (ctx > ctx_cap || ql > ctx) {
        if (lane == 0) record_error(err, kErrRange, static_cast<uint32_t>(found));
        r.bad = 1;
    }
    r.row0 = q0 + tloc * kPrefillRows;
    r.rows = min(kPrefillRows, ql - tloc * kPrefillRows);
    r.pmin = ctx - ql + tloc * kPrefillRows;
    r.pmax = r.pmin + r.rows - 1;
    r.nt = r.bad ? 0 : r.pmax / 128 + 1;
    r.klast = r.pmax + 1 - (r.pmax / 128) * 128;
    return r;
}

// Reports a sequence that the device's starts give rows for which the plan from
// the host's has nothing: the last prefill sequence where they need more entries
// than the grid's `entries`, a decode row in a call without a decode launch; or a
// start below the one before.  For a whole warp of the CTA with the fewest keys,
// beside the search for its tile (2,048 of 16,384 tokens, 8-bit pools: 458 us, 455
// without; two prompts of 300 beside 4,096 decode rows: 274 and 269).
static __device__ __noinline__ void report_unplanned_rows(const int32_t* qsl, int num_seqs, int split, int entries,
                                                          int decode_launch, unsigned long long* err, int lane) {
    const unsigned FULL = 0xffffffffu;
    int count = 0, last = -1, wrong = INT32_MAX;
#pragma unroll 4
    for (int s = lane; s < num_seqs; s += 32) {
        const int ql = __ldg(qsl + s + 1) - __ldg(qsl + s);
        const int nt = ql > 1 ? (ql + kPrefillRows - 1) / kPrefillRows : 0;
        count += nt + min(split, nt);
        if (nt > 0) last = s;
        if (ql < 0 || (ql == 1 && !decode_launch)) wrong = min(wrong, s);
    }
    wrong = __reduce_min_sync(FULL, wrong);
    if (__reduce_add_sync(FULL, count) > entries) wrong = min(wrong, __reduce_max_sync(FULL, last));
    if (wrong < INT32_MAX && lane == 0) record_error(err, kErrRange, static_cast<uint32_t>(wrong));
}

}  // namespace pkv
