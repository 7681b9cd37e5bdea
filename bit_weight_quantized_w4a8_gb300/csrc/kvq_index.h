// kvq_index.h -- where a token's key and value lie in the paged cache: the
// look-ups of kvq_batch_t and their range checks, for the kernels and for
// host tests.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KVQ_HD __host__ __device__ __forceinline__
#else
#define KVQ_HD inline
#endif

namespace w4a8 {

// CTAs of `per` tokens each for `tokens` of them, up to 2^31 - 1.
KVQ_HD int kvq_ctas(int tokens, int per) { return tokens / per + (tokens % per != 0); }

// Sequence of token i: the b with cu[b] <= i < cu[b + 1], or -1 when the
// offsets hold none (they do not cover i, are negative or not in order).
KVQ_HD int kvq_find_seq(const int32_t* cu, int seqs, int i) {
    int lo = 0, hi = seqs;  // cu[lo] <= i would hold, cu[hi] > i
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (cu[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    return cu[lo] >= 0 && cu[lo] <= i && i < cu[lo + 1] ? lo : -1;
}

// Whether token i lies behind the last sequence: a step planned for more tokens than went in.
KVQ_HD bool kvq_behind(const int32_t* cu, int seqs, int i) { return cu[seqs] >= 0 && i >= cu[seqs]; }

// Slot of token i of the sequence b that kvq_find_seq gives, or -1 where its start is negative.
KVQ_HD int64_t kvq_token_slot(const int32_t* cu, const int32_t* start, int b, int i) {
    const int64_t s = start[b];
    return s < 0 ? -1 : s + (i - cu[b]);
}

// Row of the pool (page * page_size + offset) of slot s of sequence b, or -1
// when the slot lies past the table or its page outside the pool.  page_size
// = 1 << shift.
KVQ_HD int64_t kvq_slot_row(const int32_t* table, int64_t max_pages, int64_t pages, int shift, int b,
                            int64_t s) {
    if (s < 0 || (s >> shift) >= max_pages) return -1;
    const int64_t p = table[b * max_pages + (s >> shift)];
    if (p < 0 || p >= pages) return -1;
    return (p << shift) + (s & ((1 << shift) - 1));
}

// Sequence b's tokens [first, first + count) and start, from arrays that may
// hold anything: count and start are 0 unless 0 <= cu[b] <= cu[b + 1] <= tokens
// and 0 <= start.  end, the slots in use, is cut to what the table holds (and to
// kKvqMaxSlots, so that slots and the blocks past them are 32-bit numbers); ok
// tells whether all was in range.
constexpr int kKvqMaxSlots = 0x7FFFF000;
struct KvqSeq {
    int first, count, start, end;
    bool ok;
};
KVQ_HD KvqSeq kvq_seq(const int32_t* cu, const int32_t* start, int b, int64_t tokens, int64_t max_pages,
                      int shift) {
    KvqSeq q;
    const int64_t lo = cu[b], hi = cu[b + 1], s = start[b];
    const int64_t room = max_pages << shift, slots = room < kKvqMaxSlots ? room : kKvqMaxSlots;
    const bool sound = lo >= 0 && lo <= hi && hi <= tokens && s >= 0;
    q.first = (int)lo;
    q.count = sound ? (int)(hi - lo) : 0;
    q.start = sound ? (int)s : 0;
    const int64_t e = (int64_t)q.start + q.count;
    q.end = (int)(e < slots ? e : slots);
    q.ok = sound && s + (hi - lo) <= slots;
    return q;
}

}  // namespace w4a8
