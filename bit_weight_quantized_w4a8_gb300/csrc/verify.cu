// verify.cu -- which of a step's drafted tokens stay: the drafts tested against
// the target's logits one after the other, and the next token drawn.
//
// With w_j = exp(l_j / T) over the vocabulary and Z its sum, a child x of node i
// is taken when u q(x) Z < w(x) (q = 1 for drafts without probabilities).
// After a refusal the weights are
//   drafts without probabilities:  w with the refused tokens at 0,
//   with them:  max(w - q A, 0), A = Z before the first refusal, and each later
//   one adds what the weights then summed to: max(max(w - q Z, 0) - q R, 0) =
//   max(w - q (Z + R), 0), so one number stands for all refusals at a node.
// The token after the last one taken is the first whose cumulative weight passes
// u times the sum.
//
// Two launches.  The first reads every row once (what bounds the call): maximum,
// its first place and the fp32 sum of weights, a row cut into slices for enough CTAs.
// The second has a cluster of CTAs a sequence, which all walk the drafts on the
// same numbers, and go over the last row once more for the draw.
//
// The draw compares a random number with sums over 10^5 weights: in fp32 their
// roundings would decide between neighbours now and then.  So the fp32 sums only
// decide where the number lies further from the token's two edges than they can be off: by
// at most kOff Z, counted at its definition.  Otherwise the row's weights are taken as integers:
// w in units of 2^-40 of the largest, each within 3 units of the exact value (the
// exponent's argument in two floats, a table of 2^(i/128), a polynomial of four terms), so
// that sums are exact, in any order and split.  That is 40 instructions a weight: a CTA's
// 19008 weights of a row of 152064 take 8.4 us, 14.5 with the draft's probabilities, in fp32 2.7.
//
// With 152064 tokens, in a graph: one greedy chain of 5 6.2 us; 24 trees of up to 12 52 to 55 (bytes at
// the copy rate: 23), of which the first launch takes 30 (5.1 TB/s: its start and end are as long as a
// third of it) and the second 33, some sequence always being left open by the fp32 sums; 61
// chains with probabilities 88 to 111 (36), by how many of them are left open on the same SMs: 39 and 60 to 75.
// The second launch is held to 64 registers (two CTAs of 512 threads an SM).  Drafts with and without
// probabilities have variants of their own: in one, which spilled 76 to 96 bytes, 24 trees took 57.5 us and 61 chains
// 2 more; with probabilities 28 to 40 bytes are left.
#include <cooperative_groups.h>

#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_verify_error;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kDrawThreads = 512;  // of the second launch, at most
constexpr int kDrawWarps = kDrawThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr int kTile = 128;        // weights of a warp's load, 4 a lane
constexpr int kSeg = 512;         // of a segment, 16 a lane
constexpr int kMaxDrafts = KVQ_MAX_TREE;
constexpr int kMaxSlices = 32;    // of a row, in the first launch
constexpr float kGreedyBelow = 0x1p-20f;

// How far an fp32 sum over weights of a row may be off, relative to the row's whole sum Z, in units of
// 2^-24: a weight exp2(t), t = (l - max) c with two roundings and 1.2 in c (a rounded quotient of a rounded
// constant), is within 3.2 |t| ln 2 + 4 (ex2.approx), and the mean of |t| over the distribution is at most
// log2(vocab) <= 22: 53; the factors that bring sums of the first launch to one maximum the same: 53; additions of
// 16 weights, over a warp, 8 warps and 32 slices, the others in 64 bits: 21 (the first launch's sum
// Z: 127); refused tokens' weights taken off: 53.  180 in all, below 2^-16.
constexpr float kOff = 0x1p-16f;

struct RowPart {
    float top, sum;  // maximum; sum of exp2((l - top) c), NaN where a value is NaN or +infinity
    int at;          // first place of the maximum
    int pad;
};

struct VerifyArgs {
    const void *L, *Q;
    int64_t ld_l, ld_q;
    int q_f16, vocab, tokens, seqs;
    const int32_t *cu, *ids;
    const uint64_t* mask;
    const float *temp, *u;
    int32_t *keep, *out, *count;
    RowPart* parts;  // [tokens][slices]
    int slices, seg_count;
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __half* p) { return __half2float(*p); }

// Four values from j on; past the end (of n) `past`.  wide: rows on 16 (8) bytes.
template <typename T>
__device__ __forceinline__ void load_run(const T* row, int j, int n, bool wide, float past, float* v) {
    if (wide && j + 4 <= n) {
        const float4 x = load4(row + j);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = j + k < n ? load1(row + j + k) : past;
    }
}
template <typename T>
__device__ __forceinline__ bool row_wide(const T* row) {
    return (reinterpret_cast<uintptr_t>(row) % (4 * sizeof(T))) == 0;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2(e) / T in two floats; greedy where T is below kGreedyBelow (or no number):
// the sum then only tells NaN and infinity.
struct Scale {
    float hi, lo;
    bool greedy;
};
__device__ __forceinline__ Scale scale_of(const float* temp, int b) {
    constexpr float kLog2E = 1.44269502162933349609375f, kLog2ELo = 1.9259629911266175e-8f;
    float t = temp != nullptr ? temp[b] : 1.f;
    Scale s;
    s.greedy = !(t >= kGreedyBelow);
    t = s.greedy ? 1.f : fminf(t, 0x1p60f);
    s.hi = __fdiv_rn(kLog2E, t);
    s.lo = __fdiv_rn(fmaf(-s.hi, t, kLog2E) + kLog2ELo, t);  // the remainder is exact
    return s;
}

// ---------------------------------------------------------------------------
// first launch: maxima and sums
// ---------------------------------------------------------------------------

__device__ __forceinline__ void join(RowPart& a, const RowPart& b, float c) {
    const float top = fmaxf(a.top, b.top);
    // (nothing but -infinity so far: its sum is 0 and stays)
    const float fa = a.top == top ? 1.f : ex2((a.top - top) * c), fb = b.top == top ? 1.f : ex2((b.top - top) * c);
    a.at = a.top > b.top ? a.at : b.top > a.top ? b.at : min(a.at, b.at);
    a.sum = a.sum * fa + b.sum * fb;
    a.top = top;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_rows_kernel(const VerifyArgs a) {
    constexpr int U = 4;  // runs of 4 under way
    __shared__ RowPart part[kVerifyWarps];
    // in this order: when the second launch starts, what the caller's kernels wrote is there
    griddep_wait();
    griddep_launch_dependents();
    const int t = blockIdx.x;
    const T* row = static_cast<const T*>(a.L) + t * a.ld_l;
    const bool wide = row_wide(row);
    const int runs = (a.vocab + 3) / 4, per = (runs + a.slices - 1) / a.slices;
    const int lo = blockIdx.y * per, hi = min(lo + per, runs);
    float v[U][4];
    auto load = [&](int r) {
        #pragma unroll
        for (int k = 0; k < U; ++k) {
            const int q = r + k * kVerifyThreads;
            load_run(row, 4 * q, q < hi ? a.vocab : 0, wide, -INFINITY, v[k]);
        }
    };
    if (lo + (int)threadIdx.x < hi) load(lo + threadIdx.x);  // before the sequence is known
    const int b = kvq_find_seq(a.cu, a.seqs, t);
    if (b < 0) return;
    const float c = scale_of(a.temp, b).hi;
    RowPart p = {-INFINITY, 0.f, 0x7FFFFFFF, 0};
    double all = 0.0;  // (a thread adds up to 2^22 / 4096 times)
    for (int r = lo + threadIdx.x; r < hi; r += U * kVerifyThreads) {
        float m = p.top;
        #pragma unroll
        for (int k = 0; k < U; ++k) m = fmaxf(m, fmaxf(fmaxf(v[k][0], v[k][1]), fmaxf(v[k][2], v[k][3])));
        if (m > p.top) {
            all *= ex2((p.top - m) * c);  // (0 while there was none)
            p.top = m;
            #pragma unroll
            for (int k = U * 4 - 1; k >= 0; --k)
                if (v[k / 4][k % 4] == m) p.at = 4 * (r + k / 4 * kVerifyThreads) + k % 4;
        }
        if (m > -INFINITY) {
            float sum = 0.f;
            #pragma unroll
            for (int k = 0; k < U; ++k)
                sum += (ex2((v[k][0] - m) * c) + ex2((v[k][1] - m) * c)) + (ex2((v[k][2] - m) * c) + ex2((v[k][3] - m) * c));
            all += sum;
        } else {  // all -infinity, or NaN
            #pragma unroll
            for (int k = 0; k < U * 4; ++k)
                if (v[k / 4][k % 4] != v[k / 4][k % 4]) all = NAN;
        }
        if (r + U * kVerifyThreads < hi) load(r + U * kVerifyThreads);
    }
    p.sum = (float)all;
    #pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
        const RowPart q = {__shfl_xor_sync(0xFFFFFFFFu, p.top, o), __shfl_xor_sync(0xFFFFFFFFu, p.sum, o),
                           __shfl_xor_sync(0xFFFFFFFFu, p.at, o), 0};
        join(p, q, c);
    }
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = p;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kVerifyWarps; ++w) join(p, part[w], c);
        a.parts[(int64_t)t * a.slices + blockIdx.y] = p;
    }
}

// ---------------------------------------------------------------------------
// weights as integers
// ---------------------------------------------------------------------------

// 2^(i / 128) in units of 2^-40, by the exponential's series.
struct Pow2Table {
    uint64_t v[128];
    constexpr Pow2Table() : v() {
        for (int i = 0; i < 128; ++i) {
            const double x = 0.69314718055994530942 * i / 128;
            double term = 1.0, sum = 0.0;
            for (int k = 1; k < 24; ++k) {
                sum += term;
                term *= x / k;
            }
            v[i] = (uint64_t)(sum * 1099511627776.0 + 0.5);
        }
    }
};
__device__ const Pow2Table kPow2{};  // (in constant memory its divergent reads came one by one)

struct Unit {
    float hi, lo, top;  // log2(e) / T, the row's maximum
};

// exp((l - top) / T) in units of 2^-40, 0 below half a unit.  With y = yh + yl what is left of the exponent
// after the table's 2^(k/128), |y| <= 2^-8.5: exp(y) - 1 = yh + (yl + yh yl + yh^2 (1/2 + yh/6 + yh^2/24)), of which
// the term yh yl (yl holds the rounding of the scaled difference) makes up to 150 units and yh^5 / 120 less
// than 1/100.  Worst of 10^8 logits at temperatures from 0.1 to 7: 2.6 units.
__device__ __forceinline__ uint64_t weight(float l, const Unit& s, const uint64_t* pow2) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
    // the difference in two floats, before it is scaled: logits near the type's ends must not overflow
    const float dh = l - s.top, b = dh - l, dl = (l - (dh - b)) - (s.top + b);
    const float d = dh * s.hi;
    if (!(d > -41.f)) return 0;
    const float e = fmaf(dl, s.hi, fmaf(dh, s.lo, fmaf(dh, s.hi, -d)));
    const float t = fmaf(d, 128.f, kMagic);
    const int k = __float_as_int(t) - __float_as_int(kMagic);  // nearest 1/128
    const float r = fmaf(t - kMagic, -1.f / 128.f, d);         // exact, |r| <= 1/256
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.90465429995776e-9f;
    const float yh = r * kLn2;
    const float yl = fmaf(r, kLn2, -yh) + fmaf(r, kLn2Lo, e * kLn2);
    const float q = fmaf(yh, fmaf(yh, fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f), yl), yl);
    const int z = __float2int_rn(yh * 0x1p39f) + __float2int_rn(q * 0x1p39f);  // exp(y) - 1
    const uint64_t w = pow2[k & 127];
    const int64_t v = (int64_t)w + ((int64_t)(uint32_t)(w >> 9) * z >> 30);
    const int n = -(k >> 7);  // 0 .. 41
    return ((uint64_t)v + ((uint64_t)1 << n >> 1)) >> n;
}

// f = m 2^-sh for f in (0, 1]; sh 23 .. 149.
__device__ __forceinline__ int split(float f, uint32_t& m) {
    const uint32_t bits = __float_as_uint(f);
    const int ex = bits >> 23;
    m = (bits & 0x7FFFFFu) | (ex != 0 ? 0x800000u : 0u);
    return 150 - (ex != 0 ? ex : 1);
}
// floor(u a), u in [0, 1).
__device__ __forceinline__ uint64_t target_of(float u, uint64_t a) {
    uint32_t m;
    const int sh = split(u, m);
    const uint64_t hi = __umul64hi(a, m), lo = a * m;
    return sh < 64 ? hi << (64 - sh) | lo >> sh : sh < 128 ? hi >> (sh - 64) : 0;
}
// What refusals take off in all, A = m 2^sh: sh is 0 until the sum passes 64 bits (2^22 weights, 63 times, reach
// 2^68), then each step cuts off less than 2^-63 of it.
struct Cut {
    uint64_t m;
    int sh;
    __device__ __forceinline__ void add(uint64_t x) {
        m += x >>= sh;
        if (m < x) m = m >> 1 | (uint64_t)1 << 63, ++sh;
    }
};
// q A to nearest (cut off instead, 10^5 weights less q A would all lean to one side, and their
// sum by as many halves of a unit), above 64 bits their largest number.  q outside [0, 1]: the
// nearest inside; NaN: 0.
__device__ __forceinline__ uint64_t part_of(float q, const Cut& a) {
    if (!(q > 0.f)) return 0;
    uint32_t f;
    const int sh = split(fminf(q, 1.f), f) - a.sh;  // q A = f m 2^-sh, sh 19 .. 149
    const uint64_t hi = (uint64_t)(uint32_t)(a.m >> 32) * f, lo = (uint64_t)(uint32_t)a.m * f;  // each below 2^56
    if (sh <= 32) {
        const uint64_t x = hi << (32 - sh), y = x + ((lo + (1u << (sh - 1))) >> sh);
        return hi >> 32 >> sh != 0 || y < x ? ~(uint64_t)0 : y;
    }
    return sh < 92 ? (hi + (lo >> 32) + ((uint64_t)1 << (sh - 33))) >> (sh - 32) : 0;
}

// ---------------------------------------------------------------------------
// second launch: the walk and the draw
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
    #pragma unroll
    for (int o = 16; o >= 1; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum(float v) {
    #pragma unroll
    for (int o = 16; o >= 1; o /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// Inclusive prefix over the warp.
__device__ __forceinline__ uint64_t warp_prefix(uint64_t v) {
    const int lane = threadIdx.x % 32;
    #pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += y;
    }
    return v;
}
// fp32 weights in the draw's units (64-bit floating point is slow here).
__device__ __forceinline__ uint64_t to_units(float w) { return __float2ull_rn(w * 0x1p40f); }

struct DrawShared {
    uint64_t pow2[128];
    RowPart row[kMaxDrafts];
    float u[kMaxDrafts], w[kMaxDrafts], q[kMaxDrafts];  // of each draft at its parent
    int id[kMaxDrafts], parent[kMaxDrafts], taken[kMaxDrafts], refused[kMaxDrafts];
    uint64_t cta_sum[2];
    float q_warp[kDrawWarps], q_sum[2];
    int verdict;  // the token that the fp32 sums give, -1 where they leave it open
};

// Sums over a row by the cluster, and the token where they pass a number.  Each CTA has
// a run of segments and the sums of each in shared memory, in the draw's units.  Q: drafts with probabilities.
template <typename T, bool Q>
struct Draw {
    const VerifyArgs& a;
    DrawShared& s;
    uint64_t* sums;
    const Scale c;
    int rank, s0, s1, passes;
    bool open;               // another CTA may still read this one's sums
    uint64_t before, total;  // of the CTAs ahead; of all
    float q_total;

    // A lane's 16 of a segment, 4 runs of 4, 128 apart; past the end -infinity and 0.
    template <typename X>
    __device__ __forceinline__ void load_seg(const X* row, int seg, float past, float (&v)[16]) const {
        const int j = seg * kSeg + 4 * (int)(threadIdx.x % 32);
        if (row_wide(row) && (seg + 1) * kSeg <= a.vocab) {
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 x = load4(row + j + k * kTile);
                v[4 * k] = x.x, v[4 * k + 1] = x.y, v[4 * k + 2] = x.z, v[4 * k + 3] = x.w;
            }
        } else {
            #pragma unroll
            for (int k = 0; k < 16; ++k) v[k] = j + k / 4 * kTile + k % 4 < a.vocab ? load1(row + j + k / 4 * kTile + k % 4) : past;
        }
    }
    __device__ __forceinline__ const T* row(int64_t t) const { return static_cast<const T*>(a.L) + t * a.ld_l; }
    __device__ __forceinline__ void load_q(int64_t t, int seg, float (&v)[16]) const {
        if (a.q_f16)
            load_seg(static_cast<const __half*>(a.Q) + t * a.ld_q, seg, 0.f, v);
        else
            load_seg(static_cast<const float*>(a.Q) + t * a.ld_q, seg, 0.f, v);
    }

    // What is left of a weight: of logit l with draft probability q, in fp32 (relative to
    // exp of the row's maximum, Z the row's sum; with_q: less q Z) ...
    struct Fast {
        float top, c, z;
        bool with_q;
        __device__ __forceinline__ float value(float l, float q) const {
            const float w = l > -INFINITY ? ex2((l - top) * c) : 0.f;
            return Q && with_q ? fmaxf(w - (q > 0.f ? fminf(q, 1.f) : 0.f) * z, 0.f) : w;
        }
        __device__ __forceinline__ uint64_t units(float l, float q) const { return to_units(value(l, q)); }
        __device__ __forceinline__ uint64_t lanes(const float (&l)[16], const float (&q)[16]) const {
            float sum = 0.f;
            #pragma unroll
            for (int k = 0; k < 16; ++k) sum += value(l[k], q[k]);
            return to_units(warp_sum(sum));
        }
    };
    // ... and as integers, exact sums (cut: A).
    struct Exact {
        Unit unit;
        Cut cut;
        const uint64_t* pow2;
        bool with_q;
        __device__ __forceinline__ uint64_t units(float l, float q) const {
            const uint64_t w = weight(l, unit, pow2), x = Q && with_q ? part_of(q, cut) : 0;
            return w > x ? w - x : 0;
        }
        __device__ __forceinline__ uint64_t lanes(const float (&l)[16], const float (&q)[16]) const {
            // four at a time, the others waiting in line: 16 copies of the code took longer to
            // fetch than to run
            uint64_t sum = 0;
            float x[16], y[16];
            #pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = l[k], y[k] = q[k];
            #pragma unroll 1
            for (int g = 0; g < 4; ++g) {
                #pragma unroll
                for (int k = 0; k < 4; ++k) sum += units(x[k], y[k]);
                #pragma unroll
                for (int k = 0; k < 12; ++k) x[k] = x[k + 4], y[k] = y[k + 4];
            }
            return warp_sum(sum);
        }
    };

    // The sums of row t, of the tokens in s.refused 0.
    template <typename W>
    __device__ void pass(int64_t t, const W& w, int refused) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        float q_mine = 0.f;
        const int warps = blockDim.x / 32;
        for (int seg = s0 + warp; seg < s1; seg += warps) {
            float l[16], q[16];
            load_seg(row(t), seg, -INFINITY, l);
            if (Q && w.with_q) {
                load_q(t, seg, q);
                #pragma unroll
                for (int k = 0; k < 16; ++k) q_mine += fminf(fabsf(q[k]), 1.f);
            } else {
                #pragma unroll
                for (int k = 0; k < 16; ++k) q[k] = 0.f;
            }
            const uint64_t sum = w.lanes(l, q);
            if (lane == 0) sums[seg - s0] = sum;
        }
        q_mine = warp_sum(q_mine);
        if (lane == 0) s.q_warp[warp] = q_mine;
        __syncthreads();
        const int slot = passes++ & 1;  // one barrier a pass: the next but one writes here again
        if (warp == 0) {
            for (int i = 0; i < refused; ++i) {
                const int seg = s.refused[i] / kSeg;
                if (lane == 0 && seg >= s0 && seg < s1) {
                    const uint64_t x = w.units(load1(row(t) + s.refused[i]), 0.f);
                    sums[seg - s0] -= x < sums[seg - s0] ? x : sums[seg - s0];
                }
            }
            __syncwarp();
            uint64_t v = 0;
            for (int x = lane; x < s1 - s0; x += 32) v += sums[x];
            v = warp_sum(v);
            if (lane == 0) {
                s.cta_sum[slot] = v;
                float x = 0.f;
                for (int i = 0; i < warps; ++i) x += s.q_warp[i];
                s.q_sum[slot] = x;
            }
        }
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        before = total = 0;
        q_total = 0.f;
        #pragma unroll
        for (int r = 0; r < kVerifyCluster; ++r) {
            const uint64_t x = *cl.map_shared_rank(&s.cta_sum[slot], r);
            q_total += *cl.map_shared_rank(&s.q_sum[slot], r);
            if (r < rank) before += x;
            total += x;
        }
        open = true;
    }

    // The first token whose cumulative sum passes `target` by more than `off`, the token before
    // it staying behind by more than `off`, in one lane of the CTA and the warp that hold it;
    // -1 elsewhere, and where it is closer.
    template <typename W>
    __device__ int find(int64_t t, const W& w, int refused, uint64_t target, uint64_t off) const {
        if (threadIdx.x >= 32 || target < before) return -1;
        const int lane = threadIdx.x;
        uint64_t run = before;
        for (int x = 0; x < s1 - s0; x += 32) {
            const uint64_t v = x + lane < s1 - s0 ? sums[x + lane] : 0, up = run + warp_prefix(v);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, up > target);
            if (hit == 0) {
                run = __shfl_sync(0xFFFFFFFFu, up, 31);
                continue;
            }
            const int first = __ffs(hit) - 1, seg = s0 + x + first;
            run = __shfl_sync(0xFFFFFFFFu, up - v, first);
            float l[16], q[16];
            load_seg(row(t), seg, -INFINITY, l);
            if (Q && w.with_q) {
                load_q(t, seg, q);
            } else {
                #pragma unroll
                for (int k = 0; k < 16; ++k) q[k] = 0.f;
            }
            #pragma unroll 1
            for (int k = 0; k < 4; ++k) {
                uint64_t y[4], sum = 0;
                #pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = w.units(l[i], q[i]);
                #pragma unroll
                for (int i = 0; i < 12; ++i) l[i] = l[i + 4], q[i] = q[i + 4];
                for (int r = 0; r < refused; ++r) {
                    const int off_lane = s.refused[r] - (seg * kSeg + k * kTile + 4 * lane);
                    #pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (off_lane == i) y[i] = 0;
                }
                #pragma unroll
                for (int i = 0; i < 4; ++i) sum += y[i];
                const uint64_t end = run + warp_prefix(sum);
                const unsigned in = __ballot_sync(0xFFFFFFFFu, end > target);
                if (in != 0) {
                    if (lane != __ffs(in) - 1) return -1;
                    uint64_t at = end - sum;
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t lo = at;
                        at += y[i];
                        if (at > target)
                            return (off == 0 || (lo + off < target && target + off < at))
                                       ? seg * kSeg + k * kTile + 4 * lane + i
                                       : -1;
                    }
                }
                run = __shfl_sync(0xFFFFFFFFu, end, 31);
            }
            return -1;
        }
        return -1;
    }
};

template <typename T, bool Q>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw_kernel(const VerifyArgs a) {
    extern __shared__ uint64_t seg_sums[];
    __shared__ DrawShared s;
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, rank = (int)cl.block_rank();
    // All that does not come from the first launch is fetched while that one runs: offsets, drafts
    // and their logits at their parents.
    if (tid < 128) s.pow2[tid] = kPow2.v[tid];
    if (tid == 0) s.verdict = -1;
    const int b = blockIdx.x / kVerifyCluster;
    const int first = a.cu[b], end = a.cu[b + 1], n = end - first;
    const bool sound = first >= 0 && n >= 0 && end <= a.tokens;
    if (!sound || n == 0 || n > kMaxDrafts) {  // the whole cluster
        griddep_wait();  // (the next kernel must not overtake the first launch)
        if (rank == 0) {
            if (tid == 0) {
                a.count[b] = 0;
                if (n != 0 || !sound) atomicOr(&g_verify_error, kErrCacheRange);
            }
            if (sound)
                for (int i = tid; i < n; i += blockDim.x) a.keep[first + i] = a.out[first + i] = -1;
        }
        return;
    }
    const Scale c = scale_of(a.temp, b);
    int up = tid - 1, id = -1;
    float l = -INFINITY, q = 0.f;
    if (tid < n) {
        const int64_t t = first + tid;
        id = a.ids[t];
        s.u[tid] = fminf(fmaxf(a.u[t], 0.f), 0x1.fffffep-1f);  // (NaN: 0)
        s.id[tid] = id;
        if (a.mask != nullptr) {  // the ancestor drafted last
            const uint64_t below = a.mask[t] & (((uint64_t)1 << tid) - 1);
            up = 63 - __clzll((long long)below);  // -1: none
        }
        s.parent[tid] = up;
        if (tid == 0 || up < 0 || id < 0 || id >= a.vocab) id = -1;
        if (id >= 0) {
            l = load1(static_cast<const T*>(a.L) + (first + up) * a.ld_l + id);
            if (Q) {
                const int64_t i = (first + up) * a.ld_q + id;
                q = a.q_f16 ? __half2float(static_cast<const __half*>(a.Q)[i]) : static_cast<const float*>(a.Q)[i];
                q = fminf(fmaxf(q, 0.f), 1.f);
            }
        }
    }
    griddep_launch_dependents();
    griddep_wait();
    #pragma unroll 1
    for (int r = warp; r < n; r += blockDim.x / 32) {  // a row's slices, one a lane
        RowPart p = {-INFINITY, 0.f, 0x7FFFFFFF, 0};
        if (lane < a.slices) p = a.parts[(int64_t)(first + r) * a.slices + lane];
        #pragma unroll 1
        for (int o = 16; o >= 1; o /= 2) {
            const RowPart x = {__shfl_xor_sync(0xFFFFFFFFu, p.top, o), __shfl_xor_sync(0xFFFFFFFFu, p.sum, o),
                               __shfl_xor_sync(0xFFFFFFFFu, p.at, o), 0};
            join(p, x, c.hi);
        }
        if (lane == 0) {
            if (!(p.top > -INFINITY)) p.sum = NAN;
            s.row[r] = p;
        }
    }
    __syncthreads();
    if (tid > 0 && tid < n) {
        float w = 0.f;
        if (id >= 0) {
            const float d = l - s.row[up].top;
            const float x = d * c.hi, e = fmaf(d, c.lo, fmaf(d, c.hi, -x));
            w = exp2f(x) * fmaf(e, 0.693147182f, 1.f);  // (NaN for a row of no use: every test fails)
            if (!(d > -INFINITY)) w = 0.f;
        }
        s.w[tid] = w;
        s.q[tid] = q;
    }
    __syncthreads();

    const int seg_per = (a.seg_count + kVerifyCluster - 1) / kVerifyCluster;
    Draw<T, Q> dr{a, s, seg_sums, c};
    dr.rank = rank;
    dr.s0 = min(rank * seg_per, a.seg_count);
    dr.s1 = min(dr.s0 + seg_per, a.seg_count);
    dr.passes = 0;
    dr.open = false;
    dr.total = 0;

    // Every thread of the cluster takes the same way through this: it depends on
    // shared values that all CTAs computed alike, and on the passes' totals.
    int node = 0, taken = 1, refused = 0, cuts = 0, todo = 0;  // cuts of todo made
    float gone = 0.f;                                          // weights of the refused
    Cut cut = {0, 0};
    auto exact = [&](bool less) {
        return typename Draw<T, Q>::Exact{{c.hi, c.lo, s.row[node].top}, cut, s.pow2, less};
    };
    // The sums of what is left at the node, by the integers.
    auto exact_sums = [&]() {
        if (cuts == 0) dr.pass(first + node, exact(false), refused);
        for (; cuts < todo && dr.total != 0; ++cuts) {  // (0: nothing more is taken off)
            cut.add(dr.total);
            dr.pass(first + node, exact(true), 0);
        }
        cuts = todo;
    };
    #pragma unroll 1
    for (int i = 1; i < n; ++i) {
        if (s.parent[i] != node) continue;
        const RowPart& p = s.row[node];
        if (p.sum != p.sum) continue;  // no distribution: no child is taken, and no pass made for one
        const int id = s.id[i];
        const float w = s.w[i];  // (0 for tokens outside the vocabulary)
        bool yes;
        if (c.greedy) {
            yes = id == p.at;
        } else {
            float u = s.u[i];
            bool weighs = w > 0.f, open;
            if (!Q) {
                #pragma unroll 1
                for (int k = 0; k < refused; ++k) weighs &= s.refused[k] != id;
                // The fp32 sum of what is left is off by up to kOff Z, whatever is left: near enough to the
                // border (2^-20 of w: its own roundings) the integers decide.
                const float side = u * (p.sum - gone) - w;
                yes = weighs && side < 0.f;
                open = weighs && refused > 0 && !(fabsf(side) > u * kOff * p.sum + 0x1p-20f * w);
            } else {
                u *= s.q[i];
                yes = todo == 0 && u * p.sum < w;
                open = todo > 0 && weighs;
            }
            if (open) {
                exact_sums();
                yes = target_of(u, dr.total) < exact(todo > 0).units(load1(dr.row(first + node) + id), s.q[i]);
            }
            if (!yes && Q) {
                ++todo;
            } else if (!yes && weighs) {
                gone += w;
                __syncthreads();
                if (tid == 0) s.refused[refused] = id;
                __syncthreads();
                ++refused;
            }
        }
        if (yes) {
            if (tid == 0) s.taken[taken] = i;
            ++taken;
            node = i;
            refused = cuts = todo = 0;
            gone = 0.f;
            cut = {0, 0};
        }
    }
    // the token after the last one taken
    const RowPart p = s.row[node];
    const int64_t t = first + node;
    const float u = s.u[0];
    int next = -1;
    bool mine = rank == 0 && tid == 0;
    if (p.sum == p.sum && c.greedy) {
        next = p.at;
    } else if (p.sum == p.sum) {
        if (todo == 0 || (todo == 1 && cuts == 0)) {
            // in fp32, after a refusal less q Z
            const typename Draw<T, Q>::Fast w = {p.top, c.hi, p.sum, todo == 1};
            dr.pass(t, w, refused);
            // (probabilities may sum to the vocabulary's size: at most 2^21 weights, half of the largest sum)
            const uint64_t off = to_units(fminf(2.f * kOff * p.sum * (1.f + dr.q_total), 0x1p21f)) + 2;
            const int x = dr.find(t, w, refused, target_of(u, dr.total), off);
            if (x >= 0)
                for (int r = 0; r < kVerifyCluster; ++r) *cl.map_shared_rank(&s.verdict, r) = x;
            cl.sync();
            dr.open = false;
            next = s.verdict;
        }
        if (next < 0) {
            for (;;) {
                exact_sums();
                if (dr.total != 0 || (todo == 0 && refused == 0)) break;
                todo = cuts = refused = 0;  // nothing left but roundings: the whole row
            }
            next = dr.find(t, exact(todo > 0), refused, target_of(u, dr.total), 0);
            mine = next >= 0 || (dr.total == 0 && mine);
        }
    }
    __syncthreads();  // s.taken
    if (mine) a.out[first + taken - 1] = next;
    if (rank == 0) {
        if (tid == 0) a.count[b] = taken;
        if (tid < n) {
            a.keep[first + tid] = tid == 0 ? 0 : tid < taken ? s.taken[tid] : -1;
            if (tid != taken - 1) a.out[first + tid] = tid < taken - 1 ? s.id[s.taken[tid + 1]] : -1;
        }
    }
    if (dr.open) cl.sync();  // no CTA leaves while its sums may be read
}

int verify_slices(int64_t tokens, int64_t vocab, int sms) {
    // about four CTAs an SM, slices of at least 4096 logits
    int64_t s = (4 * sms + tokens - 1) / tokens;
    const int64_t most = (vocab + 4095) / 4096;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > kMaxSlices ? kMaxSlices : s);
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs& a, int sms, unsigned flags, cudaStream_t stream) {
    cudaError_t e = layer_launch(verify_rows_kernel<T>, dim3((unsigned)a.tokens, (unsigned)a.slices), kVerifyThreads, 0, flags,
                                 stream, a);
    if (e != cudaSuccess) return e;
    const int per = (a.seg_count + kVerifyCluster - 1) / kVerifyCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.seqs * kVerifyCluster));
    // (64 registers a thread: 2 CTAs of 512 or 4 of 256 threads an SM; all clusters resident
    // comes first, then more warps for the passes)
    cfg.blockDim = dim3((unsigned)(a.seqs * kVerifyCluster <= 2 * sms ? kDrawThreads : kDrawThreads / 2));
    cfg.dynamicSmemBytes = (size_t)per * sizeof(uint64_t);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kVerifyCluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return a.Q != nullptr ? cudaLaunchKernelEx(&cfg, verify_draw_kernel<T, true>, a)
                          : cudaLaunchKernelEx(&cfg, verify_draw_kernel<T, false>, a);
}

}  // namespace

size_t draft_verify_workspace(int64_t tokens, int64_t vocab, int sms) {
    return (size_t)tokens * verify_slices(tokens, vocab, sms) * sizeof(RowPart);
}

cudaError_t launch_draft_verify(const void* L, int l_f16, int64_t ld_l, int64_t vocab, const int32_t* cu, int64_t seqs,
                                int64_t tokens, const int32_t* ids, const uint64_t* mask, const void* Q, int q_f16,
                                int64_t ld_q, const float* temp, const float* u, int32_t* keep, int32_t* out,
                                int32_t* count, void* ws, int sms, unsigned flags, cudaStream_t stream) {
    const int slices = verify_slices(tokens, vocab, sms), segs = (int)((vocab + kSeg - 1) / kSeg);
    const VerifyArgs a = {L, Q, ld_l, ld_q, q_f16, (int)vocab, (int)tokens, (int)seqs, cu, ids, mask, temp, u, keep, out,
                          count, static_cast<RowPart*>(ws), slices, segs};
    return l_f16 ? launch_verify<__half>(a, sms, flags, stream) : launch_verify<float>(a, sms, flags, stream);
}

cudaError_t read_and_clear_verify_error(unsigned* flags, cudaStream_t stream) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_verify_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_verify_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *flags |= v;
    return e;
}

}  // namespace w4a8
