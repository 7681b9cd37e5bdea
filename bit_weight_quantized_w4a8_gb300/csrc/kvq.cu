// kvq.cu -- rotary positions and the quantized paged key/value cache: the
// write (rotation, quantization and placement in one pass), the read back,
// and the move of a tree's accepted tokens.
//
// All three are bound by memory: every value is read once and written once.
// The angle: with f = freq / (2 pi) as the 64-bit fraction of a turn F = f 2^64
// (mod 2^64), the turns of position p are p F mod 2^64, exact in integers
// whatever p; its top 32 bits, read as a signed number of 2^-32 turns, go
// through one rounding to fp32 into sincospi.
//
// Measured in graphs: 8191 x 32 x 128 fp32 rotated into binary16 31.1 us, 95% of the copy
// rate (cos and sin once per token for all heads; the first loads issued before them, 33.6
// without); 8190 tokens written with 32 query heads 36.4 us (41.3 with the
// queries in the keys' loop and a division per code); 200000 x 4 x 128 4-bit codes
// read back in 83 us, 92% (8 values a thread, whole-line stores; 104 with 16 in two
// stores); one row 1.9, 7 tokens written 3.1.
#include <type_traits>

#include "actq.cuh"
#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

__device__ unsigned g_kvq_error;

constexpr int kLayerThreads = 256;

__device__ __forceinline__ uint64_t turn_fraction(double freq) {
    const double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
    return (uint64_t)__double2ull_rz((t - floor(t)) * 18446744073709551616.0);
}
__device__ __forceinline__ float2 turn_cos_sin(uint64_t f, int pos, float mscale) {
    const int32_t top = (int32_t)(uint32_t)((f * (uint64_t)(int64_t)pos) >> 32);
    float s, c;
    sincospif((float)top * 0x1p-31f, &s, &c);  // 2^-32 turns = 2^-31 half turns
    return make_float2(c * mscale, s * mscale);
}

struct RopeArg {
    const int32_t* pos;   // [axes][tokens]
    const double* freqs;  // NULL: no rotation
    int rot, inter;
    float mscale;
    int64_t ld_pos;
    int axes;          // that the pairs use
    uint32_t axis[8];  // of each pair, two bits, in the launch's constants
};

struct WriteArgs {
    KvqCacheArg c;
    KvqBatchArg b;
    RopeArg rope;
    const void *Q, *K, *V;
    int64_t ld_q, ld_k, ld_v;
    int heads_q, tokens_per_cta;
    void* Y;  // rotated queries
    int64_t ld_y;
    int y_wide;  // binary16 rows on 16 bytes: runs of 8 go out in one store
};

// A head's vector is spread over DIM / 8 lanes of 8 values in two runs of 4
// (at oa and ob), so that a lane holds whole pairs: in the half layout lane
// l < rot / 8 has 4l.. and rot / 2 + 4l.., otherwise 8l.. and 8l + 4...
// cs: cos and sin of pairs 4l..4l+3.
__device__ __forceinline__ void rotate8(float4& a, float4& b, const float2* cs, int inter) {
    const float2 c0 = cs[0], c1 = cs[1], c2 = cs[2], c3 = cs[3];
    auto turn = [](float& x, float& y, float2 c) {
        const float t = fmaf(x, c.x, -(y * c.y));
        y = fmaf(y, c.x, x * c.y);
        x = t;
    };
    if (inter) {
        turn(a.x, a.y, c0);
        turn(a.z, a.w, c1);
        turn(b.x, b.y, c2);
        turn(b.z, b.w, c3);
    } else {
        turn(a.x, b.x, c0);
        turn(a.y, b.y, c1);
        turn(a.z, b.z, c2);
        turn(a.w, b.w, c3);
    }
}

// Codes of four values, a byte each: clamp(round_half_away(x / s), +-top), or 0
// where s is 0, infinite or NaN (the scale then tells what the vector holds).
// Exact form: an IEEE division and roundf per value.
__device__ __noinline__ uint32_t codes4_exact(float4 v, float s, float top) {
    if (!(s < INFINITY)) return 0u;
    return (uint32_t)(layer_code(v.x, s, top) & 0xFF) | (uint32_t)(layer_code(v.y, s, top) & 0xFF) << 8 |
           (uint32_t)(layer_code(v.z, s, top) & 0xFF) << 16 | (uint32_t)(layer_code(v.w, s, top) & 0xFF) << 24;
}
// Fast form, with 1 / s bracketed by lo and hi (quant_bracket): the IEEE quotient
// lies strictly between x lo and x hi, so where both round to one integer that is
// the code, no tie is involved, and |x| <= top s up to two roundings of s needs
// no clamp; the few others take the exact form.  All of this needs a normal, finite s: below
// 2^-126 its own rounding is no longer relative (the largest code may need the clamp),
// below 2^-128 the bracket is infinite; such vectors take the exact form too.
__device__ __forceinline__ uint32_t codes4(float4 v, float s, float top, float lo, float hi) {
    if (!(s >= 0x1p-126f && s < INFINITY)) return codes4_exact(v, s, top);
    constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: the sum's low bits hold the rounded product
    const float x[4] = {v.x, v.y, v.z, v.w};
    uint32_t y[4], diff = 0u;
    #pragma unroll
    for (int k = 0; k < 4; ++k) {
        y[k] = __float_as_uint(__fmaf_rn(x[k], lo, kMagic));
        diff |= y[k] ^ __float_as_uint(__fmaf_rn(x[k], hi, kMagic));
    }
    if (diff != 0u) return codes4_exact(v, s, top);
    return __byte_perm(__byte_perm(y[0], y[1], 0x0040), __byte_perm(y[2], y[3], 0x0040), 0x5410);
}

// Walks the (token, vector) pairs of a CTA, one per group of LPV lanes and two
// at a time, without a division: `vecs` vectors of each token, `part` of `parts`
// CTAs that share them.  Whole warps iterate together.
template <int LPV>
struct PairWalk {
    int t, v, vecs, step_t, step_v, left, stride;
    __device__ __forceinline__ PairWalk(int nt, int vecs_, int part, int parts) : vecs(vecs_) {
        constexpr int GROUPS = kLayerThreads / LPV;
        const int e = part * GROUPS + threadIdx.x / LPV;
        t = e / vecs;
        v = e - t * vecs;
        stride = parts * GROUPS;
        step_t = stride / vecs;
        step_v = stride % vecs;
        left = nt * vecs - part * GROUPS;  // pairs from the CTA's first group on
    }
    __device__ __forceinline__ void next() {
        t += step_t;
        v += step_v;
        if (v >= vecs) v -= vecs, ++t;
    }
};

// Queries [0, heads_q) rotated to Y, then keys and values quantized into the cache
// (HAS_KV).  A CTA takes tokens_per_cta tokens (gridDim.y CTAs share their
// vectors) and computes their cos and sin once for all heads, with the first
// queries under way.  Queries come first, on their own: with the keys' slots, a chain of
// loads, in front of every load and both kinds in one loop, 8190 tokens of 32 +
// 2 heads took 44 us instead of 36.5 (a floor of 33).
// AXES: positions of more than one axis, in a variant of its own (the look-up of a pair's axis costs the
// calls without one 6%: 8191 x 32 x 128 34.9 us a call instead of 32.8), held to the 48 registers of
// the other: with 56, hence four CTAs an SM, 33.2 us in a graph instead of 31.9, as with one axis.  All
// axes' positions loaded side by side with the look-up: 34.
template <typename TX, typename TYO, int DIM, int BITS, bool HAS_KV, bool AXES>
__global__ void __launch_bounds__(kLayerThreads, AXES ? 5 : 0) rope_write_kernel(const WriteArgs a) {
    constexpr int LPV = DIM / 8;
    extern __shared__ float2 cs[];  // [tokens_per_cta][rot / 2]
    __shared__ int64_t slot_row[16];
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * a.tokens_per_cta;
    const int nt = min(a.tokens_per_cta, a.b.tokens - t0);
    const int pairs = a.rope.freqs != nullptr ? a.rope.rot / 2 : 0;
    const int l = threadIdx.x % LPV;
    const bool half = !a.rope.inter && 8 * l < 2 * pairs;
    // a lane's two runs of a turned vector, and of one that stays in order
    const int oa = half ? 4 * l : 8 * l, ob = half ? pairs + 4 * l : 8 * l + 4;

    float4 va[2], vb[2];
    int vt[2], vv[2];
    bool live[2];
    auto load_q = [&](PairWalk<LPV>& w) {
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
            vt[i] = w.t;
            vv[i] = w.v;
            live[i] = w.t < nt;
            if (live[i]) {
                const TX* x = static_cast<const TX*>(a.Q) + (int64_t)(t0 + w.t) * a.ld_q + (int64_t)w.v * DIM;
                va[i] = load4(x + oa);
                vb[i] = load4(x + ob);
            }
            w.next();
        }
    };
    PairWalk<LPV> wq(nt, max(a.heads_q, 1), blockIdx.y, gridDim.y);
    if (a.heads_q > 0) load_q(wq);
    int64_t row = -1;
    if constexpr (HAS_KV) {
        if ((int)threadIdx.x < nt) {
            const int i = t0 + threadIdx.x;
            const int b = kvq_find_seq(a.b.cu, a.b.seqs, i);
            if (b >= 0) {
                const int64_t slot = kvq_token_slot(a.b.cu, a.b.start, b, i);
                if (slot >= 0) row = kvq_slot_row(a.b.table, a.b.max_pages, a.c.pages, a.c.shift, b, slot);
            }
            if (row < 0 && (b >= 0 || !kvq_behind(a.b.cu, a.b.seqs, i))) atomicOr(&g_kvq_error, kErrCacheRange);
            slot_row[threadIdx.x] = row;
        }
    }
    // the last threads, whose warps have no look-up to make, first
    for (int e = kLayerThreads - 1 - (int)threadIdx.x; e < nt * pairs; e += kLayerThreads) {
        const int t = e / pairs, i = e - t * pairs;
        if constexpr (AXES) {
            const int64_t axis = a.rope.axis[i >> 4] >> (2 * (i & 15)) & 3;
            cs[e] = turn_cos_sin(turn_fraction(a.rope.freqs[i]), a.rope.pos[axis * a.rope.ld_pos + t0 + t], a.rope.mscale);
        } else {
            cs[e] = turn_cos_sin(turn_fraction(a.rope.freqs[i]), a.rope.pos[t0 + t], a.rope.mscale);
        }
    }
    __syncthreads();
    if (a.heads_q > 0) {
        for (;;) {
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!live[i]) continue;
                if (8 * l < 2 * pairs) rotate8(va[i], vb[i], cs + vt[i] * pairs + 4 * l, a.rope.inter);
                TYO* y = static_cast<TYO*>(a.Y) + (int64_t)(t0 + vt[i]) * a.ld_y + (int64_t)vv[i] * DIM;
                if (sizeof(TYO) == 2 && ob == oa + 4 && a.y_wide) {
                    *reinterpret_cast<uint4*>(y + oa) = make_uint4(pack_half2(va[i].x, va[i].y), pack_half2(va[i].z, va[i].w),
                                                                   pack_half2(vb[i].x, vb[i].y), pack_half2(vb[i].z, vb[i].w));
                } else {
                    store4(y + oa, va[i]);
                    store4(y + ob, vb[i]);
                }
            }
            wq.left -= 2 * wq.stride;
            if (wq.left <= 0) break;
            load_q(wq);
        }
    }
    if constexpr (HAS_KV) {
        const int kv_heads = a.c.heads;
        // the CTAs with the fewest queries first
        PairWalk<LPV> w(nt, 2 * kv_heads, gridDim.y - 1 - blockIdx.y, gridDim.y);
        for (; w.left > 0; w.left -= 2 * w.stride) {
            int pa[2], pb[2];
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                vt[i] = w.t;
                vv[i] = w.v;
                live[i] = w.t < nt;
                const bool turned = w.v < kv_heads && 8 * l < 2 * pairs;  // a value has no pairs
                pa[i] = turned ? oa : 8 * l;
                pb[i] = turned ? ob : 8 * l + 4;
                va[i] = vb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (live[i]) {
                    const int64_t tok = t0 + w.t;
                    const TX* x = w.v < kv_heads ? static_cast<const TX*>(a.K) + tok * a.ld_k + (int64_t)w.v * DIM
                                                 : static_cast<const TX*>(a.V) + tok * a.ld_v + (int64_t)(w.v - kv_heads) * DIM;
                    va[i] = load4(x + pa[i]);
                    vb[i] = load4(x + pb[i]);
                }
                w.next();
            }
            #pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int kv = vv[i] >= kv_heads;  // 0 key, 1 value
                if (live[i] && !kv && 8 * l < 2 * pairs) rotate8(va[i], vb[i], cs + vt[i] * pairs + 4 * l, a.rope.inter);
                float m = max_nan(absmax4_nan(va[i]), absmax4_nan(vb[i]));
                #pragma unroll
                for (int o = LPV / 2; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
                if (live[i] && slot_row[vt[i]] >= 0) {
                    constexpr float top = BITS == 8 ? 127.f : 7.f;
                    const float s = __fmul_rn(m, 1.f / top);
                    float lo, hi;
                    quant_bracket(s, &lo, &hi);
                    const int64_t vec = kvq_vec(a.c, slot_row[vt[i]], vv[i] - kv * kv_heads);
                    const uint32_t qa = codes4(va[i], s, top, lo, hi), qb = codes4(vb[i], s, top, lo, hi);
                    uint8_t* codes = (kv ? a.c.v : a.c.k) + vec * (DIM * BITS / 8);
                    if constexpr (BITS == 8) {
                        *reinterpret_cast<uint32_t*>(codes + pa[i]) = qa;
                        *reinterpret_cast<uint32_t*>(codes + pb[i]) = qb;
                    } else {
                        auto pack = [](uint32_t q) {  // low nibbles of 4 bytes -> 16 bits
                            q &= 0x0F0F0F0Fu;
                            q |= q >> 4;
                            return (uint16_t)((q & 0xFFu) | ((q >> 8) & 0xFF00u));
                        };
                        *reinterpret_cast<uint16_t*>(codes + pa[i] / 2) = pack(qa);
                        *reinterpret_cast<uint16_t*>(codes + pb[i] / 2) = pack(qb);
                    }
                    if (l == 0) (kv ? a.c.vs : a.c.ks)[vec] = s;
                }
            }
        }
    }
}

// axis: host array of rot / 2 entries below 4, or NULL (one axis).
RopeArg rope_arg(const int32_t* pos, int64_t tokens, const uint8_t* axis, const double* freqs, int rot, int inter,
                 float mscale) {
    RopeArg r = {pos, freqs, rot, inter, mscale, tokens, 1, {}};
    for (int i = 0; axis != nullptr && i < rot / 2; ++i) {
        r.axes = r.axes > axis[i] ? r.axes : axis[i] + 1;
        r.axis[i / 16] |= (uint32_t)axis[i] << (2 * (i % 16));
    }
    return r;
}

template <typename TX, typename TYO, int BITS, bool HAS_KV>
cudaError_t launch_write(const WriteArgs& a0, int dim, int sms, unsigned flags, cudaStream_t stream) {
    WriteArgs a = a0;
    a.y_wide = reinterpret_cast<uintptr_t>(a.Y) % 16 == 0 && a.ld_y % 8 == 0;
    const int vecs = a.heads_q + (HAS_KV ? 2 * a.c.heads : 0);
    a.tokens_per_cta = a.b.tokens >= 8 * sms ? 4 : 1;
    const int ctas = kvq_ctas(a.b.tokens, a.tokens_per_cta);
    const int groups = kLayerThreads / (dim / 8);
    int gy = 1;
    while (ctas * gy < 2 * sms && gy * groups < vecs * a.tokens_per_cta) gy *= 2;
    const dim3 grid((unsigned)ctas, (unsigned)gy);
    const int smem = a.tokens_per_cta * (a.rope.rot / 2) * (int)sizeof(float2);
    auto go = [&](auto* one, auto* several) {
        return layer_launch(a.rope.axes > 1 ? several : one, grid, kLayerThreads, smem, flags, stream, a);
    };
    switch (dim) {
        case 64: return go(rope_write_kernel<TX, TYO, 64, BITS, HAS_KV, false>, rope_write_kernel<TX, TYO, 64, BITS, HAS_KV, true>);
        case 128: return go(rope_write_kernel<TX, TYO, 128, BITS, HAS_KV, false>, rope_write_kernel<TX, TYO, 128, BITS, HAS_KV, true>);
        case 256: return go(rope_write_kernel<TX, TYO, 256, BITS, HAS_KV, false>, rope_write_kernel<TX, TYO, 256, BITS, HAS_KV, true>);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// read back
// ---------------------------------------------------------------------------

// A CTA reads per_cta tokens; a thread takes 8 values of a key and of the value,
// so that a warp's stores are whole lines (16 values in two stores each took
// 104 us instead of 84 at 200,000 tokens of 4 heads and 4 bits, a floor of 76), of
// two vectors at a time, and steps through (token, head) without a division.
constexpr int kReadTokens = 32;
template <typename TO, int DIM, int BITS>
__global__ void __launch_bounds__(kLayerThreads) kvq_read_kernel(const KvqCacheArg c, const KvqBatchArg b, int per_cta,
                                                                 TO* K, TO* V) {
    constexpr int UPV = DIM / 8;                   // units of 8 values per vector
    constexpr int STEP = kLayerThreads / UPV;      // vectors that a pass of the CTA takes
    constexpr int U = 2;
    __shared__ int64_t slot_row[kReadTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * per_cta;
    const int nt = min(per_cta, b.tokens - t0);
    if ((int)threadIdx.x < nt) {
        const int i = t0 + threadIdx.x;
        int64_t row = -1;
        const int s = kvq_find_seq(b.cu, b.seqs, i);
        if (s >= 0) row = kvq_slot_row(b.table, b.max_pages, c.pages, c.shift, s, kvq_token_slot(b.cu, b.start, s, i));
        if (row < 0 && (s >= 0 || !kvq_behind(b.cu, b.seqs, i))) atomicOr(&g_kvq_error, kErrCacheRange);
        slot_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int u = threadIdx.x % UPV;
    const int step_t = STEP / c.heads, step_h = STEP % c.heads;
    int t = threadIdx.x / UPV / c.heads, h = threadIdx.x / UPV % c.heads;
    while (t < nt) {
        uint32_t w[U][2][BITS / 4];  // [vector][key, value]
        float s[U][2];
        int at[U];  // vector of the CTA's, -1: none
        #pragma unroll
        for (int x = 0; x < U; ++x) {
            const int64_t row = t < nt ? slot_row[t] : -1;
            at[x] = row >= 0 ? t * c.heads + h : -1;
            const int64_t vec = row >= 0 ? kvq_vec(c, row, h) : 0;
            #pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const uint8_t* p = (kv ? c.v : c.k) + vec * (DIM * BITS / 8) + u * BITS;
                if constexpr (BITS == 8) {
                    const uint2 q = *reinterpret_cast<const uint2*>(p);
                    w[x][kv][0] = q.x, w[x][kv][1] = q.y;
                } else {
                    w[x][kv][0] = *reinterpret_cast<const uint32_t*>(p);
                }
                s[x][kv] = (kv ? c.vs : c.ks)[vec];
            }
            t += step_t;
            h += step_h;
            if (h >= c.heads) h -= c.heads, ++t;
        }
        #pragma unroll
        for (int x = 0; x < U; ++x)
            #pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                if (at[x] < 0) continue;
                float v[8];
                #pragma unroll
                for (int k = 0; k < 8; ++k) {
                    constexpr int PER = 32 / BITS;  // codes of a word
                    v[k] = (float)((int32_t)(w[x][kv][k / PER] << (32 - BITS - BITS * (k % PER))) >> (32 - BITS)) * s[x][kv];
                }
                TO* o = (kv ? V : K) + ((int64_t)t0 * c.heads + at[x]) * DIM + 8 * u;
                if constexpr (sizeof(TO) == 2) {
                    *reinterpret_cast<uint4*>(o) = make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]),
                                                              pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
                } else {
                    store4(o, make_float4(v[0], v[1], v[2], v[3]));
                    store4(o + 4, make_float4(v[4], v[5], v[6], v[7]));
                }
            }
    }
}

// ---------------------------------------------------------------------------
// move of the accepted tokens
// ---------------------------------------------------------------------------

// One CTA per (sequence, head): the kept vectors go through shared memory,
// so that an entry may name any slot of the tree.
__global__ void __launch_bounds__(kLayerThreads) kvq_keep_kernel(const KvqCacheArg c, const KvqBatchArg b,
                                                            const int32_t* __restrict__ keep, int vec_bytes,
                                                            int max_tree) {
    extern __shared__ __align__(16) uint8_t buf[];  // [2][max_tree][vec_bytes]
    __shared__ float scale[2][64];
    __shared__ int64_t from[64], to[64];
    __shared__ int n_keep, bad;
    griddep_launch_dependents();
    griddep_wait();
    const int sq = blockIdx.x, h = blockIdx.y;
    if (threadIdx.x == 0) {
        const KvqSeq q = kvq_seq(b.cu, b.start, sq, b.tokens, b.max_pages, c.shift);
        int n = 0, wrong = !q.ok || q.count > max_tree;
        while (!wrong && n < q.count && keep[q.first + n] >= 0) {
            const int k = keep[q.first + n];
            if (k >= q.count) {
                wrong = 1;
                break;
            }
            from[n] = kvq_slot_row(b.table, b.max_pages, c.pages, c.shift, sq, q.start + k);
            to[n] = kvq_slot_row(b.table, b.max_pages, c.pages, c.shift, sq, q.start + n);
            wrong |= from[n] < 0 || to[n] < 0;
            ++n;
        }
        n_keep = n;
        bad = wrong;
        if (wrong) atomicOr(&g_kvq_error, kErrCacheRange);
    }
    __syncthreads();
    if (bad || n_keep == 0) return;
    const int words = vec_bytes / 16, n = n_keep;
    for (int e = threadIdx.x; e < 2 * n * words; e += kLayerThreads) {
        const int kv = e >= n * words, r = e - kv * n * words, i = r / words, w = r - i * words;
        const int64_t vec = kvq_vec(c, from[i], h);
        reinterpret_cast<uint4*>(buf)[e] = reinterpret_cast<const uint4*>((kv ? c.v : c.k) + vec * vec_bytes)[w];
        if (w == 0) scale[kv][i] = (kv ? c.vs : c.ks)[vec];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * n * words; e += kLayerThreads) {
        const int kv = e >= n * words, r = e - kv * n * words, i = r / words, w = r - i * words;
        const int64_t vec = kvq_vec(c, to[i], h);
        reinterpret_cast<uint4*>((kv ? c.v : c.k) + vec * vec_bytes)[w] = reinterpret_cast<const uint4*>(buf)[e];
        if (w == 0) (kv ? c.vs : c.ks)[vec] = scale[kv][i];
    }
}

}  // namespace

cudaError_t launch_rope_rotate(const void* X, int x_f16, int64_t ld_x, int64_t tokens, int heads, int dim,
                               const int32_t* pos, const uint8_t* axis, const double* freqs, int rot, int inter,
                               float mscale, void* Y, int y_f16, int64_t ld_y, int sms, unsigned flags, cudaStream_t stream) {
    WriteArgs a = {};
    a.b.tokens = (int)tokens;
    a.rope = rope_arg(pos, tokens, axis, freqs, rot, inter, mscale);
    a.Q = X;
    a.ld_q = ld_x;
    a.heads_q = heads;
    a.Y = Y;
    a.ld_y = ld_y;
    if (x_f16)
        return y_f16 ? launch_write<__half, __half, 8, false>(a, dim, sms, flags, stream)
                     : launch_write<__half, float, 8, false>(a, dim, sms, flags, stream);
    return y_f16 ? launch_write<float, __half, 8, false>(a, dim, sms, flags, stream)
                 : launch_write<float, float, 8, false>(a, dim, sms, flags, stream);
}

cudaError_t launch_kvq_write(const kvq_cache_t& c, const kvq_batch_t& b, const void* K, int64_t ld_k, const void* V,
                             int64_t ld_v, const void* Q, int64_t ld_q, int heads_q, int x_f16, const int32_t* pos,
                             const uint8_t* axis, const double* freqs, int rot, int inter, float mscale,
                             uint16_t* Q_out, int sms, unsigned flags, cudaStream_t stream) {
    WriteArgs a = {};
    a.c = cache_arg(c);
    a.b = batch_arg(b);
    a.rope = rope_arg(pos, b.tokens, axis, freqs, freqs ? rot : 0, inter, mscale);
    a.Q = Q;
    a.K = K;
    a.V = V;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.heads_q = Q ? heads_q : 0;
    a.Y = Q_out;
    a.ld_y = (int64_t)heads_q * c.dim;
    if (x_f16)
        return c.bits == 8 ? launch_write<__half, __half, 8, true>(a, c.dim, sms, flags, stream)
                           : launch_write<__half, __half, 4, true>(a, c.dim, sms, flags, stream);
    return c.bits == 8 ? launch_write<float, __half, 8, true>(a, c.dim, sms, flags, stream)
                       : launch_write<float, __half, 4, true>(a, c.dim, sms, flags, stream);
}

cudaError_t launch_kvq_read(const kvq_cache_t& cc, const kvq_batch_t& bb, void* K, void* V, int y_f16, int sms,
                            unsigned flags, cudaStream_t stream) {
    const KvqCacheArg c = cache_arg(cc);
    const KvqBatchArg b = batch_arg(bb);
    const int per_cta = b.tokens >= 64 * sms ? kReadTokens : 8;
    const dim3 grid((unsigned)kvq_ctas(b.tokens, per_cta));
    auto go = [&](auto* out, auto dim, auto bits) {
        using T = std::remove_pointer_t<decltype(out)>;
        return layer_launch(kvq_read_kernel<T, decltype(dim)::value, decltype(bits)::value>, grid, kLayerThreads, 0, flags,
                            stream, c, b, per_cta, static_cast<T*>(K), static_cast<T*>(V));
    };
    auto by_bits = [&](auto* out, auto dim) {
        return cc.bits == 8 ? go(out, dim, std::integral_constant<int, 8>()) : go(out, dim, std::integral_constant<int, 4>());
    };
    auto by_dim = [&](auto* out) {
        return cc.dim == 64    ? by_bits(out, std::integral_constant<int, 64>())
               : cc.dim == 128 ? by_bits(out, std::integral_constant<int, 128>())
                               : by_bits(out, std::integral_constant<int, 256>());
    };
    return y_f16 ? by_dim(static_cast<__half*>(nullptr)) : by_dim(static_cast<float*>(nullptr));
}

cudaError_t launch_kvq_keep(const kvq_cache_t& c, const kvq_batch_t& b, const int32_t* keep, unsigned flags,
                            cudaStream_t stream) {
    const int vec_bytes = c.dim * c.bits / 8;
    return layer_launch(kvq_keep_kernel, dim3((unsigned)b.seqs, (unsigned)c.heads), kLayerThreads,
                        2 * KVQ_MAX_TREE * vec_bytes, flags, stream, cache_arg(c), batch_arg(b), keep, vec_bytes,
                        KVQ_MAX_TREE);
}

cudaError_t read_and_clear_kvq_error(unsigned* flags, cudaStream_t stream) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_kvq_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_kvq_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *flags |= v;
    return e;
}

}  // namespace w4a8
