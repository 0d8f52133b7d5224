#include <cstdint>
#include <memory>
#include <new>
#include <cstdio>
#include <cstdlib>
struct LinearPlan { int32_t recurrent, units, ranges, range, subs; bool cut; };
constexpr int C=64, kMaxSegments=128;
static int64_t max_ranges(int32_t num_seqs, int32_t num_tokens, int32_t num_kv_heads, int num_sms) {
    const int64_t waves = (2 * static_cast<int64_t>(num_sms) + num_kv_heads - 1) / num_kv_heads;
    const int64_t units = num_tokens / C + num_seqs;
    const int64_t lists = num_seqs > kMaxSegments ? (units + kMaxSegments - 1) / kMaxSegments : 0;
    return waves > lists ? waves : lists;
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
    // in each, and takes a launch that clears their counters where there is
    // none before the main kernel anyway.  The constants are fitted to the times of forced plans
    // over nine batches (128 to 16,384 tokens, both widths, one sequence and
    // many); the plans taken are within 4 % of the best forced one.
    const bool narrow = head_dim == 64;
    const double fixed = narrow ? 0.45 : 1.3, item = narrow ? 1.25 : 1.3, state = narrow ? 0.5 : 1.0, start = 5.5,
                 clear = 1.5;
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
            if (subs > 1 && !cut && best.recurrent == 0) us += clear;
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


extern "C" void plan(const int32_t*q,int s,int t,int h,int g,int d,int sms,int mr,int32_t*o){auto p=plan_linear(q,s,t,h,g,d,sms,mr);o[0]=p.recurrent;o[1]=p.units;o[2]=p.ranges;o[3]=p.range;o[4]=p.subs;o[5]=p.cut;}
