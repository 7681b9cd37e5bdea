// kvq_attn.cuh -- what the two attention kernels share: their arguments, the
// cutting of a batch's work into equal runs for the CTAs, and small pieces.
//
// The rows of a (sequence, cache head), tokens x group of them, are taken in
// tiles of R rows and row blocks of up to P tiles; a row block walks the
// sequence's keys in units, each of which counts what it costs (for P = 2: 5 with
// two tiles, 3 with one, as measured: the keys cost the same, the rows less).
// Every row block has the units of its sequence's whole length: without a mask, an early
// block's last ones, which none of its rows sees, are counted too (and the tile kernel computes
// them), nothing up to 64 tokens, half of the work for a long prompt from an empty cache.
// The batch's work, ordered by sequence, head, row block and key, is cut into
// one run per CTA on the device, from the lengths found there: long and
// short sequences fill the GPU alike, a captured graph follows its lengths,
// and which CTA does what depends on nothing else.
#pragma once

#include "layer.cuh"

namespace w4a8 {

struct AttnArgs {
    KvqCacheArg c;
    KvqBatchArg b;
    const __half* Q;
    const uint64_t* mask;
    __half* out;
    int heads_q, group;  // query heads of a cache head
    float scale_log2;    // scale * log2(e)
    unsigned* tickets;   // arrival counters, one per CTA
    float* parts;        // the CTAs' pieces of tiles that they share
};
static __device__ unsigned g_attn_error;  // each kernel's file has its own

constexpr int kAttnTicketBytes = 4096;
constexpr int kAttnMaxCtas = kAttnTicketBytes / 4;

__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22 relative
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// A row's reference M: its weights are 2^(t - M) vs.  A bound of log2 of the largest one is
// kTop when M is set and may grow by kSlack before M is raised and the sums rescaled;
// weights down to 2^-23 of the largest 2^(t - M) times the largest vs keep 11 bits.
constexpr float kTop = 10.f, kSlack = 4.f;
// e with v < 2^e for the finite value scale v >= 0 whose bits are given, kLeastValue at least:
// smaller values (zeros above all) give outputs of at most 2^-17, and a reference taken
// that low would make the sum of 2^(t - reference) overflow: at -100, 2^18
// keys of zero values did (outputs of 0).
constexpr float kLeastValue = -24.f;
__device__ __forceinline__ float log2_bound(uint32_t bits) {
    return fmaxf((float)((int)(bits >> 23) - 126), kLeastValue);
}
__device__ __forceinline__ uint32_t hsub2_u(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t hfma2_u(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// 8-bit codes: bytes u = code + 128 (an xor) under the exponent byte 0x64 read
// as 1024 + u, so subtracting 1152 leaves the code exactly.
__device__ __forceinline__ void widen8(uint32_t w, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2_u(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2_u(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
}
// 4-bit codes, nibbles i and i + 4 of a word: 1032 + code and 1024 + 16 (code +
// 8) in the low and high nibble of a byte, then - 1032, or / 16 - 72.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& n0, uint32_t& n1) {
    n0 = hsub2_u((w & 0x000F000Fu) ^ 0x64086408u, 0x64086408u);
    n1 = hfma2_u((w & 0x00F000F0u) ^ 0x64806480u, 0x2C002C00u, 0xD480D480u);
}

// A row block's part that falls to this CTA.
struct AttnTile {
    KvqSeq s;
    int b, h;
    int row0, rows;    // its rows, row = token * group + head within the group
    int tiles;         // of R rows
    int units, u0, u1; // key units of the row block, and of this CTA
    int key_end;       // slots that some of its rows may see end here
    int64_t first;     // place of its first unit in the batch's work
};

template <int THREADS, int R, int P, int UNIT>
struct AttnWalk {
    int64_t per, at, end, seq_first;
    int b;

    struct Shared {
        int64_t units[THREADS / 32], find[2];
    };
    static constexpr int kCost1 = P == 1 ? 1 : 3, kCostP = P == 1 ? 1 : 5;  // of a unit: 92 to 157 ps a key measured
    static_assert(P <= 2, "a row block has one tile or P");
    struct Work {
        int64_t tiles, units, per_head;
    };
    static __device__ __forceinline__ Work work(const AttnArgs& a, const KvqSeq& s) {
        Work w;
        w.tiles = ((int64_t)s.count * a.group + R - 1) / R;
        const int e = keys(a, s);
        w.units = e > 0 ? (e + UNIT - 1) / UNIT : 1;  // one at least: it writes the zeros
        w.per_head = w.units * (w.tiles / P * kCostP + (w.tiles % P ? kCost1 : 0));
        return w;
    }
    static __device__ __forceinline__ bool too_wide(const AttnArgs& a, const KvqSeq& s) {
        return a.mask != nullptr && s.count > KVQ_MAX_TREE;
    }
    static __device__ __forceinline__ int keys(const AttnArgs& a, const KvqSeq& s) {
        return too_wide(a, s) ? 0 : s.end;
    }
    static __device__ __forceinline__ KvqSeq seq(const AttnArgs& a, int i) {
        return kvq_seq(a.b.cu, a.b.start, i, a.b.tokens, a.b.max_pages, a.c.shift);
    }

    // The run of this CTA; false when it has none.  Every thread calls it.
    __device__ bool init(const AttnArgs& a, Shared& sh) {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        int64_t total = 0;
        for (int i = tid; i < a.b.seqs; i += THREADS) {
            const KvqSeq s = seq(a, i);
            if (!s.ok || too_wide(a, s)) atomicOr(&g_attn_error, kErrCacheRange);
            const Work w = work(a, s);
            total += w.per_head * a.c.heads;
        }
        #pragma unroll
        for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
        if (lane == 0) sh.units[warp] = total;
        __syncthreads();
        total = 0;
        for (int w = 0; w < THREADS / 32; ++w) total += sh.units[w];
        // no less than a unit, so that every CTA from the first to the
        // last with a part of a row block has one
        per = max((int64_t)kCostP, (total + gridDim.x - 1) / gridDim.x);
        at = per * blockIdx.x;
        end = min(at + per, total);
        if (at >= end) return false;
        if (warp == 0) {  // the sequence that holds unit `at`, 32 sequences a time
            int64_t before = 0;
            for (int b0 = 0; b0 < a.b.seqs; b0 += 32) {
                int64_t n = 0;
                if (b0 + lane < a.b.seqs) {
                    const Work w = work(a, seq(a, b0 + lane));
                    n = w.per_head * a.c.heads;
                }
                int64_t sum = n;
                #pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t x = __shfl_up_sync(0xFFFFFFFFu, sum, o);
                    if (lane >= o) sum += x;
                }
                const unsigned past = __ballot_sync(0xFFFFFFFFu, before + sum > at);
                if (past) {
                    if (lane == __ffs(past) - 1) {
                        sh.find[0] = b0 + lane;
                        sh.find[1] = before + sum - n;
                    }
                    break;
                }
                before += __shfl_sync(0xFFFFFFFFu, sum, 31);
            }
        }
        __syncthreads();
        b = (int)sh.find[0];
        seq_first = sh.find[1];
        return true;
    }

    // The next row block that this CTA has a part of; false at the run's end.
    __device__ bool next(const AttnArgs& a, AttnTile& t) {
        while (at < end) {
            t.s = seq(a, b);
            const Work w = work(a, t.s);
            const int64_t per_head = w.per_head;
            if (at >= seq_first + per_head * a.c.heads) {
                seq_first += per_head * a.c.heads;
                ++b;
                continue;
            }
            t.b = b;
            t.h = (int)((at - seq_first) / per_head);
            const int64_t in_head = at - seq_first - t.h * per_head;
            const int64_t rb = in_head / (kCostP * w.units);
            t.tiles = (int)min((int64_t)P, w.tiles - rb * P);
            t.first = seq_first + t.h * per_head + rb * kCostP * w.units;
            const int cost = t.tiles == P ? kCostP : kCost1;
            t.row0 = (int)(rb * P * R);
            t.rows = (int)min((int64_t)P * R, (int64_t)t.s.count * a.group - t.row0);
            t.units = (int)w.units;
            // a unit belongs to the run in which it begins
            t.u0 = (int)((at - t.first + cost - 1) / cost);
            t.u1 = (int)min(w.units, (end - t.first + cost - 1) / cost);
            at = min(end, t.first + w.units * cost);
            t.key_end = keys(a, t.s);
            if (a.mask == nullptr) {
                const int64_t last = (int64_t)t.s.start + (t.row0 + t.rows - 1) / a.group + 1;
                if (last < t.key_end) t.key_end = (int)last;
            }
            if (t.u0 < t.u1) return true;
        }
        return false;
    }
    // The first and last CTA with a part of the row block.
    __device__ __forceinline__ int64_t first_cta(const AttnTile& t) const { return t.first / per; }
    __device__ __forceinline__ int64_t last_cta(const AttnTile& t) const {
        return (t.first + (int64_t)(t.units - 1) * (t.tiles == P ? kCostP : kCost1)) / per;
    }
};

}  // namespace w4a8
