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
// same numbers, and go over one row for the draw (over as many more as
// there are refusals at the node with draft probabilities).
//
// The draw compares a random number with sums over 10^5 weights: in fp32 their
// roundings would decide between neighbours now and then.  The weights of the
// draw are integers instead: w / 2^ceil(max) in units of 2^-40, each within a
// few units of the exact value (the exponent's argument in two floats, a table of 2^(i/128), a
// polynomial of four terms), so sums are exact, in any order and split.
#include <cooperative_groups.h>

#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_verify_error;

constexpr int kVerifyThreads = 256;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyCluster = 8;
constexpr int kTile = 128;        // weights of a tile, 4 a lane
constexpr int kMaxDrafts = KVQ_MAX_TREE;
constexpr int kMaxSlices = 32;    // of a row, in the first launch
constexpr float kGreedyBelow = 0x1p-20f;

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
    int slices;
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
    const float t = temp != nullptr ? temp[b] : 1.f;
    Scale s;
    s.greedy = !(t >= kGreedyBelow);
    const double c = 1.4426950408889634074 / (s.greedy ? 1.0 : (double)fminf(t, 0x1p60f));
    s.hi = (float)c;
    s.lo = (float)(c - (double)s.hi);
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
    griddep_launch_dependents();
    griddep_wait();
    const int t = blockIdx.x;
    const int b = kvq_find_seq(a.cu, a.seqs, t);
    if (b < 0) return;
    const float c = scale_of(a.temp, b).hi;
    const T* row = static_cast<const T*>(a.L) + t * a.ld_l;
    const bool wide = row_wide(row);
    const int runs = (a.vocab + 3) / 4, per = (runs + a.slices - 1) / a.slices;
    const int lo = blockIdx.y * per, hi = min(lo + per, runs);
    RowPart p = {-INFINITY, 0.f, 0x7FFFFFFF, 0};
    for (int r = lo + threadIdx.x; r < hi; r += U * kVerifyThreads) {
        float v[U][4];
        #pragma unroll
        for (int k = 0; k < U; ++k) {
            const int q = r + k * kVerifyThreads;
            load_run(row, 4 * q, q < hi ? a.vocab : 0, wide, -INFINITY, v[k]);
        }
        float m = p.top;
        #pragma unroll
        for (int k = 0; k < U; ++k) m = fmaxf(m, fmaxf(fmaxf(v[k][0], v[k][1]), fmaxf(v[k][2], v[k][3])));
        if (m > p.top) {
            p.sum *= ex2((p.top - m) * c);  // (0 while there was none)
            p.top = m;
            #pragma unroll
            for (int k = U * 4 - 1; k >= 0; --k)
                if (v[k / 4][k % 4] == m) p.at = 4 * (r + k / 4 * kVerifyThreads) + k % 4;
        }
        if (m > -INFINITY) {
            #pragma unroll
            for (int k = 0; k < U; ++k)
                p.sum += (ex2((v[k][0] - m) * c) + ex2((v[k][1] - m) * c)) + (ex2((v[k][2] - m) * c) + ex2((v[k][3] - m) * c));
        } else {  // all -infinity, or NaN
            #pragma unroll
            for (int k = 0; k < U * 4; ++k)
                if (v[k / 4][k % 4] != v[k / 4][k % 4]) p.sum = NAN;
        }
    }
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
__constant__ constexpr Pow2Table kPow2{};

struct Unit {
    float hi, lo, ref;  // log2(e) / T, the whole power of two above the largest weight
};

// exp2(l c - ref) in units of 2^-40, 0 below half a unit.
__device__ __forceinline__ uint64_t weight(float l, const Unit& s, const uint64_t* pow2) {
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
    const float p = l * s.hi;
    const float e = fmaf(l, s.lo, fmaf(l, s.hi, -p));
    const float d = p - s.ref;  // exact where it is above -41
    if (!(d > -41.f)) return 0;
    const float t = fmaf(d, 128.f, kMagic);
    const int k = __float_as_int(t) - __float_as_int(kMagic);  // nearest 1/128
    const float r = fmaf(t - kMagic, -1.f / 128.f, d);         // exact, |r| <= 1/256
    constexpr float kLn2 = 0.693147182464599609375f, kLn2Lo = -1.90465429995776e-9f;
    const float yh = r * kLn2;
    const float yl = fmaf(r, kLn2, -yh) + fmaf(r, kLn2Lo, e * kLn2);
    const float q = yh * yh * fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f);
    const int z = __float2int_rn(yh * 0x1p39f) + __float2int_rn((yl + q) * 0x1p39f);  // exp(y) - 1
    const uint64_t w = pow2[k & 127];
    const int64_t v = (int64_t)w + ((int64_t)(uint32_t)(w >> 9) * z >> 30);
    const int n = -(k >> 7);  // 0 .. 41
    return ((uint64_t)v + ((uint64_t)1 << n >> 1)) >> n;
}

// floor(f a) for f in [0, 1]; 0 for a negative f or NaN.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t a) {
    if (!(f > 0.f)) return 0;
    if (f >= 1.f) return a;
    const uint32_t bits = __float_as_uint(f);
    const int ex = bits >> 23;  // f = m 2^-sh
    const uint64_t m = (bits & 0x7FFFFFu) | (ex != 0 ? 0x800000u : 0u);
    const int sh = 150 - (ex != 0 ? ex : 1);  // 24 .. 149
    const uint64_t hi = __umul64hi(a, m), lo = a * m;
    return sh < 64 ? hi << (64 - sh) | lo >> sh : sh < 128 ? hi >> (sh - 64) : 0;
}

// ---------------------------------------------------------------------------
// second launch: the walk and the draw
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
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

struct DrawShared {
    uint64_t pow2[128];
    RowPart row[kMaxDrafts];
    float u[kMaxDrafts], w[kMaxDrafts], q[kMaxDrafts];  // of each draft at its parent
    int id[kMaxDrafts], parent[kMaxDrafts], taken[kMaxDrafts], refused[kMaxDrafts];
    uint64_t cta_sum[2], warp[kVerifyWarps];
};

template <typename T>
struct Draw {
    const VerifyArgs& a;
    DrawShared& s;
    uint64_t* tile_sum;  // of this CTA's tiles
    int tiles, per, t0, t1, rank, ctas, passes;
    uint64_t before, total;  // of the CTAs ahead; of all

    // The weights that a pass sums: of row t in unit `unit`, less q times `cut`
    // (0: the weights themselves).
    __device__ __forceinline__ float q_at(int64_t t, int j) const {
        const int64_t i = t * a.ld_q + j;
        return a.q_f16 ? __half2float(static_cast<const __half*>(a.Q)[i]) : static_cast<const float*>(a.Q)[i];
    }
    __device__ __forceinline__ uint64_t left(float l, float q, const Unit& unit, uint64_t cut) const {
        const uint64_t w = weight(l, unit, s.pow2), c = cut != 0 ? part_of(q, cut) : 0;
        return w > c ? w - c : 0;
    }
    __device__ __forceinline__ void load_tile(int64_t t, int tile, bool with_q, float* l, float* q) const {
        const int j = tile * kTile + 4 * (threadIdx.x % 32);
        const T* row = static_cast<const T*>(a.L) + t * a.ld_l;
        load_run(row, j, a.vocab, row_wide(row), -INFINITY, l);
        if (!with_q) return;
        if (a.q_f16) {
            const __half* r = static_cast<const __half*>(a.Q) + t * a.ld_q;
            load_run(r, j, a.vocab, row_wide(r), 0.f, q);
        } else {
            const float* r = static_cast<const float*>(a.Q) + t * a.ld_q;
            load_run(r, j, a.vocab, row_wide(r), 0.f, q);
        }
    }

    // Sums of this CTA's tiles, of the CTAs before it and of all; the tokens in
    // s.refused count 0.
    __device__ void pass(int64_t t, const Unit& unit, uint64_t cut, int refused) {
        const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
        constexpr int U = 2;
        for (int x = t0 + warp; x < t1; x += U * kVerifyWarps) {
            float l[U][4], q[U][4];
            #pragma unroll
            for (int k = 0; k < U; ++k)
                if (x + k * kVerifyWarps < t1) load_tile(t, x + k * kVerifyWarps, cut != 0, l[k], q[k]);
            #pragma unroll
            for (int k = 0; k < U; ++k) {
                if (x + k * kVerifyWarps >= t1) break;
                uint64_t v = 0;
                #pragma unroll
                for (int i = 0; i < 4; ++i) v += left(l[k][i], cut != 0 ? q[k][i] : 0.f, unit, cut);
                v = warp_sum(v);
                if (lane == 0) tile_sum[x + k * kVerifyWarps - t0] = v;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0)
            for (int i = 0; i < refused; ++i) {
                const int x = s.refused[i] / kTile;
                if (x >= t0 && x < t1)
                    tile_sum[x - t0] -= weight(load1(static_cast<const T*>(a.L) + t * a.ld_l + s.refused[i]), unit, s.pow2);
            }
        __syncthreads();
        uint64_t v = 0;
        for (int x = threadIdx.x; x < t1 - t0; x += kVerifyThreads) v += tile_sum[x];
        v = warp_sum(v);
        if (lane == 0) s.warp[warp] = v;
        __syncthreads();
        const int slot = passes++ & 1;  // one barrier a pass: the next but one writes here again
        if (threadIdx.x == 0) {
            v = 0;
            for (int i = 0; i < kVerifyWarps; ++i) v += s.warp[i];
            s.cta_sum[slot] = v;
        }
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        before = total = 0;
        for (int r = 0; r < ctas; ++r) {
            const uint64_t c = *cl.map_shared_rank(&s.cta_sum[slot], r);
            if (r < rank) before += c;
            total += c;
        }
    }

    // The first token whose cumulative weight passes `target`, in the CTA and the
    // warp that hold it; -1 elsewhere.
    __device__ int find(int64_t t, const Unit& unit, uint64_t cut, int refused, uint64_t target) const {
        if (threadIdx.x >= 32 || target < before) return -1;
        const int lane = threadIdx.x;
        uint64_t run = before;
        for (int x = t0; x < t1; x += 32) {
            const uint64_t v = x + lane < t1 ? tile_sum[x - t0 + lane] : 0, up = run + warp_prefix(v);
            const unsigned hit = __ballot_sync(0xFFFFFFFFu, up > target);
            if (hit == 0) {
                run = __shfl_sync(0xFFFFFFFFu, up, 31);
                continue;
            }
            const int first = __ffs(hit) - 1;
            run = __shfl_sync(0xFFFFFFFFu, up - v, first);
            float l[4], q[4];
            load_tile(t, x + first, cut != 0, l, q);
            uint64_t w[4], sum = 0;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = left(l[i], cut != 0 ? q[i] : 0.f, unit, cut);
                for (int k = 0; k < refused; ++k)
                    if (s.refused[k] == (x + first) * kTile + 4 * lane + i) w[i] = 0;
                sum += w[i];
            }
            const uint64_t end = run + warp_prefix(sum);
            const unsigned in = __ballot_sync(0xFFFFFFFFu, end > target);
            if (in == 0 || lane != __ffs(in) - 1) return -1;
            uint64_t c = end - sum;
            #pragma unroll
            for (int i = 0; i < 4; ++i) {
                c += w[i];
                if (c > target) return (x + first) * kTile + 4 * lane + i;
            }
        }
        return -1;
    }
};

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_draw_kernel(const VerifyArgs a) {
    extern __shared__ uint64_t tile_sum[];
    __shared__ DrawShared s;
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x < 128) s.pow2[threadIdx.x] = kPow2.v[threadIdx.x];
    griddep_launch_dependents();
    griddep_wait();
    const int b = blockIdx.x / kVerifyCluster;
    const int first = a.cu[b], end = a.cu[b + 1], n = end - first;
    const bool sound = first >= 0 && n >= 0 && end <= a.tokens;
    if (!sound || n == 0 || n > kMaxDrafts) {  // the whole cluster
        if (cl.block_rank() == 0) {
            if (threadIdx.x == 0) {
                a.count[b] = 0;
                if (n != 0 || !sound) atomicOr(&g_verify_error, kErrCacheRange);
            }
            if (sound)
                for (int i = threadIdx.x; i < n; i += kVerifyThreads) a.keep[first + i] = a.out[first + i] = -1;
        }
        return;
    }
    const Scale c = scale_of(a.temp, b);
    const int tid = threadIdx.x;
    if (tid < n) {
        const int64_t t = first + tid;
        RowPart p = a.parts[t * a.slices];
        for (int i = 1; i < a.slices; ++i) join(p, a.parts[t * a.slices + i], c.hi);
        if (!(p.top > -INFINITY)) p.sum = NAN;
        s.row[tid] = p;
        s.u[tid] = a.u[t];
        s.id[tid] = a.ids[t];
        int up = tid - 1;
        if (a.mask != nullptr) {  // the ancestor drafted last
            const uint64_t below = a.mask[t] & (((uint64_t)1 << tid) - 1);
            up = 63 - __clzll((long long)below);  // -1: none
        }
        s.parent[tid] = up;
    }
    __syncthreads();
    if (tid > 0 && tid < n) {
        const int up = s.parent[tid], id = s.id[tid];
        float w = 0.f, q = 0.f;
        if (up >= 0 && id >= 0 && id < a.vocab) {
            const float d = load1(static_cast<const T*>(a.L) + (first + up) * a.ld_l + id) - s.row[up].top;
            const float x = d * c.hi, e = fmaf(d, c.lo, fmaf(d, c.hi, -x));
            w = exp2f(x) * fmaf(e, 0.693147182f, 1.f);  // (NaN for a row of no use: every test fails)
            if (!(d > -INFINITY)) w = 0.f;
            if (a.Q != nullptr) {
                const int64_t i = (first + up) * a.ld_q + id;
                q = a.q_f16 ? __half2float(static_cast<const __half*>(a.Q)[i]) : static_cast<const float*>(a.Q)[i];
            }
        }
        s.w[tid] = w;
        s.q[tid] = q;
    }
    __syncthreads();

    Draw<T> dr{a, s, tile_sum};
    dr.tiles = (a.vocab + kTile - 1) / kTile;
    dr.per = (dr.tiles + kVerifyCluster - 1) / kVerifyCluster;
    dr.rank = (int)cl.block_rank();
    dr.ctas = kVerifyCluster;
    dr.t0 = min(dr.rank * dr.per, dr.tiles);
    dr.t1 = min(dr.t0 + dr.per, dr.tiles);
    dr.passes = 0;

    // Every thread of the cluster takes the same way through this: it depends on
    // shared values that all CTAs computed alike, and on the passes' totals.
    int node = 0, taken = 1, refused = 0, cuts = 0, todo = 0;  // cuts of todo made
    float gone = 0.f;                                          // weights of the refused
    uint64_t cut = 0;
    auto unit_of = [&](int i) { return Unit{c.hi, c.lo, ceilf(s.row[i].top * c.hi)}; };
    auto make_cuts = [&]() {
        const Unit unit = unit_of(node);
        while (cuts < todo) {
            if (cuts == 0) {
                dr.pass(first + node, unit, 0, 0);
                cut = dr.total;
            } else {
                cut += dr.total;
            }
            if (cut == 0) break;
            dr.pass(first + node, unit, cut, 0);
            ++cuts;
        }
        cuts = todo;
    };
    for (int i = 1; i < n; ++i) {
        if (s.parent[i] != node) continue;
        const RowPart& p = s.row[node];
        const int id = s.id[i];
        bool yes;
        if (c.greedy) {
            yes = id == p.at && p.sum == p.sum;
        } else if (a.Q == nullptr) {
            bool again = false;
            for (int k = 0; k < refused; ++k) again |= s.refused[k] == id;
            yes = !again && s.u[i] * (p.sum - gone) < s.w[i];
            if (!yes && !again && id >= 0 && id < a.vocab && s.w[i] > 0.f) {
                gone += s.w[i];
                __syncthreads();
                if (tid == 0) s.refused[refused] = id;
                __syncthreads();
                ++refused;
            }
        } else if (todo == 0) {
            yes = s.u[i] * s.q[i] * p.sum < s.w[i];
            todo += !yes;
        } else {
            make_cuts();
            uint64_t w = 0;
            if (id >= 0 && id < a.vocab)
                w = dr.left(load1(static_cast<const T*>(a.L) + (first + node) * a.ld_l + id), s.q[i], unit_of(node), cut);
            yes = (double)s.u[i] * s.q[i] * (double)dr.total < (double)w;
            todo += !yes;
        }
        if (yes) {
            if (tid == 0) s.taken[taken] = i;
            ++taken;
            node = i;
            refused = cuts = todo = 0;
            gone = 0.f;
            cut = 0;
        }
    }
    // the token after the last one taken
    const RowPart p = s.row[node];
    int next = -1;
    bool mine = false;
    if (p.sum != p.sum) {  // no distribution
        mine = dr.rank == 0 && tid == 0;
    } else if (c.greedy) {
        next = p.at;
        mine = dr.rank == 0 && tid == 0;
    } else {
        const Unit unit = unit_of(node);
        make_cuts();
        if (todo == 0) dr.pass(first + node, unit, 0, refused);
        if (dr.total == 0 && (todo != 0 || refused != 0)) {  // nothing left but roundings: the whole row
            cut = 0;
            refused = 0;
            dr.pass(first + node, unit, 0, 0);
        }
        const float u = s.u[0];
        const uint64_t target = part_of(u < 1.f ? u : 0x1.fffffep-1f, dr.total);
        next = dr.find(first + node, unit, cut, refused, target);
        mine = next >= 0;
        if (dr.total == 0) mine = dr.rank == 0 && tid == 0;
    }
    __syncthreads();
    if (mine) a.out[first + taken - 1] = next;
    if (dr.rank == 0) {
        if (tid == 0) a.count[b] = taken;
        if (tid < n) {
            a.keep[first + tid] = tid == 0 ? 0 : tid < taken ? s.taken[tid] : -1;
            if (tid != taken - 1) a.out[first + tid] = tid < taken - 1 ? s.id[s.taken[tid + 1]] : -1;
        }
    }
    cl.sync();  // no CTA leaves while its sums may be read
}

int verify_slices(int64_t tokens, int64_t vocab, int sms) {
    // about four CTAs an SM, slices of at least 4096 logits
    int64_t s = (4 * sms + tokens - 1) / tokens;
    const int64_t most = (vocab + 4095) / 4096;
    s = s < most ? s : most;
    return (int)(s < 1 ? 1 : s > kMaxSlices ? kMaxSlices : s);
}

template <typename T>
cudaError_t launch_verify(const VerifyArgs& a, unsigned flags, cudaStream_t stream) {
    cudaError_t e = layer_launch(verify_rows_kernel<T>, dim3((unsigned)a.tokens, (unsigned)a.slices), kVerifyThreads, 0, flags,
                                 stream, a);
    if (e != cudaSuccess) return e;
    const int tiles = (a.vocab + kTile - 1) / kTile, per = (tiles + kVerifyCluster - 1) / kVerifyCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.seqs * kVerifyCluster));
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.dynamicSmemBytes = (size_t)per * sizeof(uint64_t);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kVerifyCluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_draw_kernel<T>, a);
}

}  // namespace

size_t draft_verify_workspace(int64_t tokens, int64_t vocab, int sms) {
    return (size_t)tokens * verify_slices(tokens, vocab, sms) * sizeof(RowPart);
}

cudaError_t launch_draft_verify(const void* L, int l_f16, int64_t ld_l, int64_t vocab, const int32_t* cu, int64_t seqs,
                                int64_t tokens, const int32_t* ids, const uint64_t* mask, const void* Q, int q_f16,
                                int64_t ld_q, const float* temp, const float* u, int32_t* keep, int32_t* out,
                                int32_t* count, void* ws, int sms, unsigned flags, cudaStream_t stream) {
    const VerifyArgs a = {L, Q, ld_l, ld_q, q_f16, (int)vocab, (int)tokens, (int)seqs, cu, ids, mask, temp, u, keep, out,
                          count, static_cast<RowPart*>(ws), verify_slices(tokens, vocab, sms)};
    return l_f16 ? launch_verify<__half>(a, flags, stream) : launch_verify<float>(a, flags, stream);
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
