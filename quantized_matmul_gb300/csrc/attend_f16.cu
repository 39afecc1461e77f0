// Attention of one new token over an f16 cache (attend.cuh), and how the
// sequences are split over CTAs.
#include "attend.cuh"

namespace qmm {

namespace {

// Splits are cut in units of this many tokens.
constexpr int64_t kSpanUnit = 128;
// Up to this many tokens a cluster of 8 CTAs a head finishes before as many
// splits as there is room for and their join do (32 query and 8 key heads of
// 128, f16, 577 tokens: 4.2 us; 1024 tokens: 4.3 against 7 us).  A cluster's
// CTAs need their SMs at once, so large batches are split.
constexpr int64_t kShort = 1024;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Plan {
    int64_t splits, span;
    bool cluster;
};

// `wave`: the CTAs that are resident at once; `ctas`: (sequence, key head,
// head tile) triples; `tokens`: the most that one attends to.
Plan plan(int64_t wave, int64_t batch, int64_t ctas, int64_t tokens) {
    tokens = tokens > 1 ? tokens : 1;
    int64_t splits = wave / ctas;
    const bool cluster = splits >= 8 && tokens <= kShort;
    if (cluster) {
        splits = 8;
    } else if (batch > 1) {
        // Lengths differ: a few waves of splits of about 1024 tokens keep the
        // SMs busy to the end (32 sequences of up to 4096 tokens, f16: two
        // waves 56 us, four 52, eight of shorter splits 54; splits of 4096
        // tokens 63).
        const int64_t fine = 4 * wave / ctas, cap = ceil_div(tokens, 8 * kSpanUnit);
        const int64_t some = fine < cap ? fine : cap;
        splits = some > splits ? some : splits;
    }
    const int64_t units = ceil_div(tokens, kSpanUnit);
    splits = splits < units ? splits : units;
    splits = splits < 1 ? 1 : splits;
    const int64_t per = ceil_div(units, splits);
    return {ceil_div(units, per), per * kSpanUnit, cluster};
}

AttendShape shape_of(bool q8, int64_t d, int64_t group) {
    return q8 ? attend_q8_0_shape((int)d, (int)group) : attend_f16_shape((int)d, (int)group);
}

}  // namespace

void attend_plan(AttendArgs &a) {
    a.group = a.heads / a.kv_heads;
    const AttendShape shape = shape_of(a.kd != nullptr, a.d, a.group);
    a.head_tiles = (int)ceil_div(a.group, shape.heads);
    const int64_t seen = a.window > 0 && a.window < a.max_tokens ? a.window : a.max_tokens;
    const Plan p = plan((int64_t)shape.ctas * device_sm_count(), a.batch,
                        (int64_t)a.batch * a.kv_heads * a.head_tiles, seen);
    a.splits = (int)p.splits;
    a.span = (int)p.span;
    a.cluster = p.cluster && p.splits > 1;
    // 2^(31 + s) / page_size rounded up, s = ceil(log2(page_size)): its error
    // times a token below 2^31 stays below 1 / page_size of a whole quotient
    int s = 0;
    while (((int64_t)1 << s) < a.page_size) ++s;
    a.page_shift = 31 + s;
    a.page_mul = (uint32_t)(((uint64_t)1 << (31 + s)) / (uint64_t)a.page_size + 1);
}

// For either type and any window.  A window may turn a plan for more tokens
// into any with at most as many splits as its first bound allows, so that
// bound counts, and not what is left of it.
size_t attend_workspace_bytes(int64_t batch, int64_t heads, int64_t kv_heads, int64_t d,
                              int64_t max_tokens) {
    int64_t most = 1;
    for (const bool q8 : {false, true}) {
        const AttendShape shape = shape_of(q8, d, heads / kv_heads);
        const int64_t wave = (int64_t)shape.ctas * device_sm_count();
        const int64_t ctas = batch * kv_heads * ceil_div(heads / kv_heads, shape.heads);
        const Plan p = plan(wave, batch, ctas, max_tokens);
        if (p.cluster) continue;  // fewer tokens are a cluster's as well
        int64_t splits = wave / ctas;
        if (batch > 1) {
            const int64_t fine = 4 * wave / ctas, cap = ceil_div(max_tokens, 8 * kSpanUnit);
            const int64_t some = fine < cap ? fine : cap;
            splits = some > splits ? some : splits;
        }
        const int64_t units = ceil_div(max_tokens, kSpanUnit);
        splits = splits < units ? splits : units;
        most = splits > most ? splits : most;
    }
    return most <= 1 ? 0 : (size_t)(batch * heads * most * (d + 2) * 4);
}

AttendShape attend_f16_shape(int d, int group) { return attend_shape<false>(d, group); }

cudaError_t launch_attend_f16(const AttendArgs &a, cudaStream_t s) { return launch_attend<false>(a, s); }

cudaError_t attend_f16_read_and_clear_error(unsigned int *word, cudaStream_t s) {
    return exchange_read_and_clear_error(word, s);
}

}  // namespace qmm
