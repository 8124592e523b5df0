// Index arithmetic of a step's sequences and their pages, shared by the kernels
// and (compiled for the host alone) by the tests: nothing read from the device
// tables is used before it has been clamped here.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define TQ2_HD __host__ __device__ __forceinline__
#else
#define TQ2_HD inline
#endif

namespace tq2 {

// Device view of a step's sequences (tq2_batch) with the cache's paging.
struct BatchView {
    const int *q_start;
    const int *kv_len;
    const int *page_table;
    int64_t tokens;
    int64_t table_stride;
    int64_t pages;
    int seqs;
    int max_q;
    int max_kv;
    int page_size;
};

// New tokens [q0, q0 + n) and keys [0, kv) of a sequence.
struct SeqSpan {
    int q0, n, kv;
};

// Sequence b's span, clamped to the step's tokens, max_q, max_kv and the table's
// width; `bad` becomes true if a clamp changed anything.
TQ2_HD SeqSpan seq_span(const BatchView &bt, int b, bool &bad) {
    const int64_t lo = bt.q_start[b], hi = bt.q_start[b + 1], len = bt.kv_len[b];
    const int64_t q0 = lo < 0 ? 0 : (lo > bt.tokens ? bt.tokens : lo);
    int64_t q1 = hi < q0 ? q0 : (hi > bt.tokens ? bt.tokens : hi);
    if (q1 - q0 > bt.max_q) q1 = q0 + bt.max_q;
    const int64_t cap = bt.table_stride * int64_t(bt.page_size);
    const int64_t top = cap < bt.max_kv ? cap : int64_t(bt.max_kv);
    const int64_t kv = len < 0 ? 0 : (len > top ? top : len);
    if (q0 != lo || q1 != hi || kv != len) bad = true;
    return SeqSpan{int(q0), int(q1 - q0), int(kv)};
}

// The page in entry `entry` of sequence b's table; -1 (and `bad`) if the cache
// has no such page.
TQ2_HD int64_t page_of(const BatchView &bt, int b, int entry, bool &bad) {
    const int p = bt.page_table[int64_t(b) * bt.table_stride + entry];
    if (p >= 0 && int64_t(p) < bt.pages) return p;
    bad = true;
    return -1;
}

// The sequence whose new tokens include t (q_start[b] <= t < q_start[b + 1]), or
// -1: a guess that is right when every sequence has max_q new tokens (decoding,
// drafts, one prompt), then a binary search.
TQ2_HD int seq_of(const BatchView &bt, int64_t t) {
    const int64_t g = t / bt.max_q;
    if (g < bt.seqs && bt.q_start[g] <= t && t < bt.q_start[g + 1]) return int(g);
    int lo = 0, hi = bt.seqs;
    if (t < bt.q_start[0] || t >= bt.q_start[hi]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (bt.q_start[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Keys [lo, hi) that new token i of a span sees.
struct KeyRange {
    int lo, hi;
};
TQ2_HD KeyRange keys_of(const SeqSpan &sp, int i, int64_t window, bool causal) {
    const int64_t pos = int64_t(sp.kv) - sp.n + i;  // below kv
    int64_t hi = causal ? pos + 1 : int64_t(sp.kv), lo = window && window <= pos ? pos + 1 - window : 0;  // (any window)
    if (hi < lo) hi = lo;
    return KeyRange{int(lo), int(hi)};
}

// What new tokens i0 .. i1 of a span see together: some of them sees a key only in
// [lo, hi), every one of them sees all of [lo_all, hi_all) (which may be empty).
struct RowSpan {
    int lo, hi, lo_all, hi_all;
};
TQ2_HD RowSpan rows_see(const SeqSpan &sp, int i0, int i1, int64_t window, bool causal) {
    const KeyRange first = keys_of(sp, i0, window, causal), last = keys_of(sp, i1, window, causal);
    return RowSpan{first.lo, last.hi, last.lo, first.hi};
}

// Boxes (rows inside one page) of a tile of keys [from, from + keys) that hold a key
// of [first, last): box i is keys from + i * rows on, i in [lo, hi).
struct BoxRange {
    int lo, hi;
};
TQ2_HD BoxRange boxes_of(int from, int keys, int rows, int first, int last) {
    const int per = keys / rows;
    int lo = first > from ? (first - from) / rows : 0, hi = last - from < keys ? (last - from + rows - 1) / rows : per;
    if (lo > per) lo = per;
    if (hi < lo || last <= first) hi = lo;
    return BoxRange{lo, hi};
}

// An item: rows [row0, row0 + rows) of a span (row = token * group + head, at most `most`),
// what they see, and the blocks of `keys` keys that hold it (0: no key).
struct ItemSpan {
    RowSpan see;
    int rows, block0, blocks;
};
TQ2_HD ItemSpan item_span(const SeqSpan &sp, int group, int row0, int most, int64_t window, bool causal, int keys) {
    const int64_t left = int64_t(sp.n) * group - row0;
    ItemSpan it{};
    it.rows = int(left < most ? left : most);
    it.see = rows_see(sp, row0 / group, (row0 + it.rows - 1) / group, window, causal);
    if (it.see.hi <= it.see.lo) return it;
    it.block0 = it.see.lo / keys;
    it.blocks = (it.see.hi + keys - 1) / keys - it.block0;
    return it;
}

// The tiles of `keys` keys that hold a key some token of a span sees, and the units of
// work that the span's (sequence, key head) pairs are shared out in: tiles if they
// may be split among CTAs, else whole pairs.
struct TileSpan {
    int tile0, tiles, units;
};
TQ2_HD TileSpan tiles_of(const SeqSpan &sp, int64_t window, bool causal, int keys, bool split) {
    if (sp.n == 0) return TileSpan{0, 0, 0};
    const RowSpan r = rows_see(sp, 0, sp.n - 1, window, causal);
    const int tile0 = r.lo / keys, tiles = r.hi > r.lo ? (r.hi + keys - 1) / keys - tile0 : 0;
    return TileSpan{tile0, tiles, split && tiles > 1 ? tiles : 1};
}

}  // namespace tq2
