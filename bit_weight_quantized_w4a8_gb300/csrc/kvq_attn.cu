// kvq_attn.cu -- attention of decode rows and of drafted trees over the
// quantized paged cache:
//   t_j = scale ks_j (q . kc_j),  p_j = exp(t_j - max t),  out = sum p_j vs_j vc_j / sum p_j.
//
// The rows that share a cache head (tokens x heads_q / heads of them) are taken
// in blocks of 8 or 16; a CTA of four warps walks the keys of one (sequence,
// head, row block) in units of 128, each warp its own 32, and the warps' and
// CTAs' pieces are joined by their softmax statistics (kvq_attn.cuh cuts the
// batch's units into runs).
//
// Both products run on mma.sync m16n8k16 with the cache as the M operand, so
// that 8 rows are enough to fill an instruction: S^T = K Q^T, then O^T = V^T W^T,
// W^T being S^T's weights transposed by movmatrix.  Codes are integers of
// at most 7 bits and sign, exact in binary16, and the scales stay outside the products:
// ks_j multiplies the fp32 logit, vs_j the fp32 weight before its rounding to binary16, the
// operand type of the second product (the error against 64 bits is 2.9e-4 with it, 2.1e-4
// with fp32 weights, which is the output's own rounding; fp32 weights would need a second
// product of their low halves).
//
// Bound by the cache's bytes at 8 bits: 24 sequences of up to 32768 keys (28 heads on 4,
// dim 128) 115 us in a graph, 89% of the copy rate, with three CTAs an SM (two: 120); 32 heads
// on 2 (16 rows, two CTAs an SM), up to 16384 keys: 49 us, 52% of it.
// At 4 bits by the widening of the codes: 52% of the copy rate (102 us) and
// 30% (44.5).  One token over 2048 keys: 10 us, its loads' latency and the join.
#include <atomic>
#include <type_traits>

#include "kernels.h"
#include "kvq_attn.cuh"

namespace w4a8 {
namespace {

constexpr int kAttnThreads = 128;
constexpr int kWarps = 4;
constexpr int kStep = 32;                 // keys of a warp's step
constexpr int kUnit = kStep * kWarps;     // keys of a CTA's unit of work

template <int N>
__device__ __forceinline__ void lds(uint32_t* v, uint32_t addr) {
    if constexpr (N == 4)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
    else if constexpr (N == 2)
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr));
    else
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(addr));
}
__device__ __forceinline__ float lds_f(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
    return v;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), binary16 operands.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// 8 x 8 binary16 matrix (lane 4r + c: row r, columns 2c, 2c + 1), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Layout of a warp's stage in shared memory: 32 keys, then 32 values, each
// vector W bytes, then their scales.  The 16-byte chunks of a vector are permuted
// by its key so that the reads below meet each bank once: keys are read
// 4 lanes (chunks t) x 8 rows g, values 8 lanes (runs g) x the rows 2t, so
// their permutations differ where a vector fills a 128-byte line.
template <int W, bool KEY>
__device__ __forceinline__ uint32_t chunk_off(int k, int c) {
    if constexpr (W >= 128) {
        const int f = KEY ? (((k & 1) << 2) ^ ((k >> 1) & 3)) : (k & 7);
        return k * W + (c >> 3) * 128 + (((c & 7) ^ f) << 4);
    } else if constexpr (W == 64) {
        const int line = k >> 1;
        return line * 128 + (((((k & 1) << 2) + c) ^ (2 * (line & 3))) << 4);
    } else {
        const int line = k >> 2;
        return line * 128 + (((((k & 3) << 1) + c) ^ (2 * (line & 1))) << 4);
    }
}

template <int DIM, int BITS, int NR>
struct Cfg {
    static constexpr int W = DIM * BITS / 8;                // bytes of a vector
    static constexpr int kStageBytes = 2 * kStep * W + 2 * kStep * 4;
    // three CTAs an SM where the registers of 8 rows allow it, with a stage less
    // each: 24 sequences of 28 / 4 heads of 128 114.8 -> 113.6 us, 4 bits 112 -> 106, 8 / 8
    // heads of 64 138 -> 122
    static constexpr int kCtas = NR == 1 && DIM <= 128 ? 3 : W <= 128 ? 2 : 1;
    static constexpr int kStages = W >= 256 ? 3 : W == 128 ? (kCtas == 3 ? 2 : 3) : (kCtas == 3 ? 3 : 4);
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kRows = 8 * NR;
    static constexpr int kPad = DIM + 4;
    static constexpr int kJoin = kWarps * kRows * kPad * 4;  // the warps' sums, over the ring
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static constexpr int kPart = kRows * (DIM + 2);          // floats of a CTA's piece
};

template <int DIM, int BITS, int NR>
__global__ void __launch_bounds__(kAttnThreads, Cfg<DIM, BITS, NR>::kCtas) attn_kernel(const AttnArgs a) {
    using C = Cfg<DIM, BITS, NR>;
    constexpr int W = C::W, ROWS = C::kRows;
    constexpr int KC = W / 64 > 0 ? W / 64 : 1;  // 16-byte (W = 32: 8-byte) runs of a key per lane
    constexpr int KW = W == 32 ? 2 : 4;          // words of a run
    constexpr int MT = DIM / 16;                 // 16-dim tiles of the output
    extern __shared__ __align__(128) uint8_t smem[];
    using Walk = AttnWalk<kAttnThreads, ROWS, 1, kUnit>;
    __shared__ typename Walk::Shared s_walk;
    __shared__ float s_stat[3][kWarps][ROWS];
    __shared__ unsigned s_last;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;

    Walk walk;
    if (!walk.init(a, s_walk)) return;

    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStageBytes);
    const int page_mask = (1 << a.c.shift) - 1;

    AttnTile t;
    while (walk.next(a, t)) {
        const KvqSeq& s = t.s;
        const int b = t.b, h = t.h, u0 = t.u0, u1 = t.u1, n_rows = t.rows;
        const int key_end = t.key_end;

        // queries: B operands, row 8 nr + g, in the order in which the key's runs
        // are widened
        uint32_t qf[NR][DIM / 16][2];
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int r = t.row0 + 8 * nr + g;
            const bool live = 8 * nr + g < n_rows;
            const int tok = s.first + r / a.group;
            const __half* q = a.Q + ((int64_t)tok * a.heads_q + h * a.group + r % a.group) * DIM;
            #pragma unroll
            for (int c = 0; c < KC; ++c) {
                // the run's dimensions: 16-byte runs t4 + 4c, W = 32: 8-byte run t4
                constexpr int kDims = KW * 32 / BITS;
                const int d0 = (t4 + 4 * c) * kDims;
                #pragma unroll
                for (int w = 0; w < KW; ++w) {
                    if constexpr (BITS == 8) {
                        uint2 x = make_uint2(0u, 0u);
                        if (live) x = *reinterpret_cast<const uint2*>(q + d0 + 4 * w);
                        qf[nr][c * KW + w][0] = x.x;
                        qf[nr][c * KW + w][1] = x.y;
                    } else {
                        uint4 x = make_uint4(0u, 0u, 0u, 0u);
                        if (live) x = *reinterpret_cast<const uint4*>(q + d0 + 8 * w);
                        // codes (0,4), (1,5) then (2,6), (3,7) of a word
                        uint32_t* f = qf[nr][2 * (c * KW + w)];
                        f[0] = __byte_perm(x.x, x.z, 0x5410);
                        f[1] = __byte_perm(x.x, x.z, 0x7632);
                        f[2] = __byte_perm(x.y, x.w, 0x5410);
                        f[3] = __byte_perm(x.y, x.w, 0x7632);
                    }
                }
            }
        }

        float acc[NR][MT][4];
        float m[NR][2], l[NR][2];  // references (kTop, kSlack) and sums of 2^(t - m)
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            m[nr][0] = m[nr][1] = -INFINITY;
            l[nr][0] = l[nr][1] = 0.f;
            #pragma unroll
            for (int i = 0; i < MT; ++i)
                #pragma unroll
                for (int k = 0; k < 4; ++k) acc[nr][i][k] = 0.f;
        }
        // page of this lane's key (lane = key of the step) for step u
        auto page_of = [&](int u) -> int {
            const int k = u * kUnit + warp * kStep + lane;
            if (u >= u1 || k >= key_end) return -2;  // no key
            const int p = a.b.table[b * a.b.max_pages + (k >> a.c.shift)];
            if (p < 0 || p >= a.c.pages) {
                atomicOr(&g_attn_error, kErrCacheRange);
                return -1;
            }
            return p;
        };
        auto issue = [&](int u, int page) {
            if (u < u1) {
                const int k0 = u * kUnit + warp * kStep;
                const uint32_t st = ring + ((u - u0) % C::kStages) * C::kStageBytes;
                const int64_t vec = page >= 0 ? ((((int64_t)page * a.c.heads + h) << a.c.shift) + ((k0 + lane) & page_mask)) : 0;
                constexpr int CPV = W / 16, KPI = 32 / CPV;  // chunks of a vector, keys of one warp-wide copy
                #pragma unroll
                for (int i = 0; i < CPV; ++i) {
                    const int k = i * KPI + lane / CPV, c = lane % CPV;
                    const int64_t kvec = __shfl_sync(0xFFFFFFFFu, vec, k);
                    const uint32_t bytes = __shfl_sync(0xFFFFFFFFu, page, k) >= 0 ? 16u : 0u;
                    cp_async_16_zfill(st + chunk_off<W, true>(k, c), a.c.k + kvec * W + c * 16, bytes);
                    cp_async_16_zfill(st + kStep * W + chunk_off<W, false>(k, c), a.c.v + kvec * W + c * 16, bytes);
                }
                cp_async_4_partial(st + 2 * kStep * W + 4 * lane, a.c.ks + vec, page >= 0 ? 4u : 0u);
                cp_async_4_partial(st + 2 * kStep * W + 4 * kStep + 4 * lane, a.c.vs + vec, page >= 0 ? 4u : 0u);
            }
            cp_async_commit();
        };
        // validity of the keys of the steps in flight, one ballot per stage
        unsigned valid[C::kStages];
        int pg = page_of(u0);
        #pragma unroll
        for (int i = 0; i < C::kStages - 1; ++i) {
            valid[i] = __ballot_sync(0xFFFFFFFFu, pg >= 0);
            issue(u0 + i, pg);
            pg = page_of(u0 + i + 1);
        }
        for (int u = u0; u < u1; ++u) {
            cp_async_wait<C::kStages - 2>();
            __syncwarp();
            const unsigned ok_keys = valid[0];
            #pragma unroll
            for (int i = 0; i + 2 < C::kStages; ++i) valid[i] = valid[i + 1];
            valid[C::kStages - 2] = __ballot_sync(0xFFFFFFFFu, pg >= 0);
            issue(u + C::kStages - 1, pg);
            pg = page_of(u + C::kStages);
            const int k0 = u * kUnit + warp * kStep;
            if (ok_keys == 0) continue;
            const uint32_t st = ring + ((u - u0) % C::kStages) * C::kStageBytes;
            const uint32_t sk = st + 2 * kStep * W, sv = sk + 4 * kStep;

            // S^T: 2 tiles of 16 keys x 8 rows per row group
            float sc[2][NR][4];
            #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                #pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) sc[mt][nr][k] = 0.f;
                #pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint32_t x[KW], y[KW];
                    if constexpr (W == 32) {
                        lds<KW>(x, st + chunk_off<W, true>(16 * mt + g, t4 >> 1) + 8 * (t4 & 1));
                        lds<KW>(y, st + chunk_off<W, true>(16 * mt + g + 8, t4 >> 1) + 8 * (t4 & 1));
                    } else {
                        lds<KW>(x, st + chunk_off<W, true>(16 * mt + g, t4 + 4 * c));
                        lds<KW>(y, st + chunk_off<W, true>(16 * mt + g + 8, t4 + 4 * c));
                    }
                    #pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        uint32_t f[4];
                        if constexpr (BITS == 8) {
                            widen8(x[w], f[0], f[2]);
                            widen8(y[w], f[1], f[3]);
                            #pragma unroll
                            for (int nr = 0; nr < NR; ++nr) mma_f16(sc[mt][nr], f, qf[nr][c * KW + w]);
                        } else {
                            #pragma unroll
                            for (int hw = 0; hw < 2; ++hw) {
                                widen4(x[w] >> (8 * hw), f[0], f[2]);
                                widen4(y[w] >> (8 * hw), f[1], f[3]);
                                #pragma unroll
                                for (int nr = 0; nr < NR; ++nr)
                                    mma_f16(sc[mt][nr], f, qf[nr][2 * (c * KW + w) + hw]);
                            }
                        }
                    }
                }
            }

            // logits in units of log2; keys g, g + 8 of each tile, rows 2 t4, 2 t4 + 1
            float kf[2][2], vf[2][2];
            #pragma unroll
            for (int mt = 0; mt < 2; ++mt)
                #pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    kf[mt][hf] = lds_f(sk + 4 * (16 * mt + 8 * hf + g)) * a.scale_log2;
                    vf[mt][hf] = lds_f(sv + 4 * (16 * mt + 8 * hf + g));
                }
            #pragma unroll
            for (int mt = 0; mt < 2; ++mt)
                #pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) sc[mt][nr][k] *= kf[mt][k >> 1];
            // all 32 keys cached ones in range: every row sees them
            const bool plain = ok_keys == 0xFFFFFFFFu && k0 + kStep <= s.start;
            uint32_t seen = 0xFFFFFFFFu;  // bit (mt * NR + nr) * 4 + k
            if (!plain) {
                #pragma unroll
                for (int nr = 0; nr < NR; ++nr)
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int r = 8 * nr + 2 * t4 + e;
                        const int tok = (t.row0 + min(r, n_rows - 1)) / a.group;
                        const uint64_t word = a.mask != nullptr ? a.mask[s.first + tok] : 0;
                        #pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
                            #pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const int kk = 16 * mt + 8 * hf + g;
                                const int w = k0 + kk - s.start;
                                bool see = (ok_keys >> kk) & 1;
                                if (w >= 0) see = see && (a.mask != nullptr ? w < 64 && ((word >> w) & 1) : w <= tok);
                                if (!see) {
                                    seen &= ~(1u << ((mt * NR + nr) * 4 + 2 * hf + e));
                                    sc[mt][nr][2 * hf + e] = -INFINITY;
                                }
                            }
                    }
            }

            // references: log2 of a bound of the value scales, the step's, or, where some
            // row does not see all of it, of the keys that the row and lane see (a large
            // value must cost only who sees it)
            float ve = 0.f;
            if (plain) {
                const float v = fabsf(lds_f(sv + 4 * lane));
                ve = log2_bound(__reduce_max_sync(0xFFFFFFFFu, v < INFINITY ? __float_as_uint(v) : 0u));
            }
            float top[NR][2];
            bool up = false;
            #pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(sc[0][nr][e], sc[0][nr][2 + e]), fmaxf(sc[1][nr][e], sc[1][nr][2 + e])) + ve;
                    if (!plain) {
                        float v = 0.f;
                        #pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
                            #pragma unroll
                            for (int hf = 0; hf < 2; ++hf)
                                if ((seen >> ((mt * NR + nr) * 4 + 2 * hf + e)) & 1 && fabsf(vf[mt][hf]) < INFINITY)
                                    v = fmaxf(v, fabsf(vf[mt][hf]));
                        x += log2_bound(__float_as_uint(v));
                    }
                    top[nr][e] = x;
                    up |= x - m[nr][e] > kTop + kSlack;
                }
            if (__any_sync(0xFFFFFFFFu, up)) {
                #pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float f[2];
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = top[nr][e];
                        #pragma unroll
                        for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                        const bool raise = x - m[nr][e] > kTop + kSlack;
                        f[e] = raise ? exp2_fast(m[nr][e] - (x - kTop)) : 1.f;
                        if (raise) m[nr][e] = x - kTop;
                        l[nr][e] *= f[e];
                    }
                    #pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        acc[nr][i][0] *= f[0];
                        acc[nr][i][1] *= f[1];
                        acc[nr][i][2] *= f[0];
                        acc[nr][i][3] *= f[1];
                    }
                }
            }
            uint32_t wf[2][NR][2];
            #pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                const float m0 = m[nr][0] == -INFINITY ? 0.f : m[nr][0];
                const float m1 = m[nr][1] == -INFINITY ? 0.f : m[nr][1];
                #pragma unroll
                for (int mt = 0; mt < 2; ++mt)
                    #pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float p0 = exp2_fast(sc[mt][nr][2 * hf] - m0);
                        const float p1 = exp2_fast(sc[mt][nr][2 * hf + 1] - m1);
                        l[nr][0] += p0;
                        l[nr][1] += p1;
                        float w0 = p0 * vf[mt][hf], w1 = p1 * vf[mt][hf];
                        if (!plain) {  // an unseen key's scale may be anything
                            if (!((seen >> ((mt * NR + nr) * 4 + 2 * hf)) & 1)) w0 = 0.f;
                            if (!((seen >> ((mt * NR + nr) * 4 + 2 * hf + 1)) & 1)) w1 = 0.f;
                        }
                        wf[mt][nr][hf] = transpose8(pack_half2(w0, w1));
                    }
            }

            // O^T += V^T W^T: lane's dimensions are a run of DIM / 8 (W >= 256: two of
            // 16), rows 2t, 2t+1, 2t+8, 2t+9 of each tile of 16 keys
            #pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
                constexpr int VW = W >= 128 ? 4 : W / 32;  // words of a run
                constexpr int VC = W >= 256 ? 2 : 1;
                #pragma unroll
                for (int c = 0; c < VC; ++c) {
                    uint32_t x[4][VW];
                    #pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int k = 16 * mt + 2 * t4 + (i & 1) + 8 * (i >> 1);
                        const uint32_t base = st + kStep * W;
                        if constexpr (W >= 128)
                            lds<VW>(x[i], base + chunk_off<W, false>(k, g + 8 * c));
                        else if constexpr (W == 64)
                            lds<VW>(x[i], base + chunk_off<W, false>(k, g >> 1) + 8 * (g & 1));
                        else
                            lds<VW>(x[i], base + chunk_off<W, false>(k, g >> 2) + 4 * (g & 3));
                    }
                    #pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        if constexpr (BITS == 8) {
                            // two keys' bytes side by side: dimensions 4w .. 4w + 3 of the run
                            uint32_t f[2][4];  // [dimension pair][a0, a1, a2, a3]
                            #pragma unroll
                            for (int kp = 0; kp < 2; ++kp) {
                                const uint32_t p = x[2 * kp][w], q = x[2 * kp + 1][w];
                                widen8(__byte_perm(p, q, 0x5140), f[0][2 * kp], f[0][2 * kp + 1]);
                                widen8(__byte_perm(p, q, 0x7362), f[1][2 * kp], f[1][2 * kp + 1]);
                            }
                            #pragma unroll
                            for (int dp = 0; dp < 2; ++dp)
                                #pragma unroll
                                for (int nr = 0; nr < NR; ++nr)
                                    mma_f16(acc[nr][c * 8 + w * 2 + dp], f[dp], wf[mt][nr]);
                        } else {
                            #pragma unroll
                            for (int dq = 0; dq < 4; ++dq) {  // dimensions 8w + 2 dq, + 1
                                uint32_t f[4];
                                #pragma unroll
                                for (int kp = 0; kp < 2; ++kp) {
                                    const uint32_t p = x[2 * kp][w], q = x[2 * kp + 1][w];
                                    const uint32_t z = __byte_perm(p, q, dq < 2 ? 0x5410 : 0x7632);
                                    widen4(z >> (8 * (dq & 1)), f[2 * kp], f[2 * kp + 1]);
                                }
                                #pragma unroll
                                for (int nr = 0; nr < NR; ++nr)
                                    mma_f16(acc[nr][c * 8 + w * 4 + dq], f, wf[mt][nr]);
                            }
                        }
                    }
                }
            }
        }

        // join the warps: statistics first, then the scaled sums
        cp_async_wait<0>();
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr)
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                #pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l[nr][e] += __shfl_xor_sync(0xFFFFFFFFu, l[nr][e], o);
                if (g == 0) {
                    s_stat[0][warp][8 * nr + 2 * t4 + e] = m[nr][e];
                    s_stat[1][warp][8 * nr + 2 * t4 + e] = l[nr][e];
                }
            }
        __syncthreads();  // statistics there, every warp's ring idle
        float* join = reinterpret_cast<float*>(smem);
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr)
            #pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * nr + 2 * t4 + e;
                float top = -INFINITY;
                #pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stat[0][w][r]);
                const float f = m[nr][e] == -INFINITY ? 0.f : exp2_fast(m[nr][e] - top);
                float* dst = join + (warp * ROWS + r) * C::kPad;
                constexpr int RUN = DIM >= 256 && W >= 256 ? 16 : DIM / 8;  // dimensions of a lane's run
                #pragma unroll
                for (int i = 0; i < MT; ++i) {
                    // tile i holds the run's dimensions 2 i', 2 i' + 1
                    const int run = i / (RUN / 2), d = run * 128 + g * RUN + (i % (RUN / 2)) * 2;
                    *reinterpret_cast<float2*>(dst + d) = make_float2(acc[nr][i][e] * f, acc[nr][i][2 + e] * f);
                }
            }
        __syncthreads();

        const bool whole = u0 == 0 && u1 == t.units;
        float* part = a.parts + ((int64_t)blockIdx.x * 2 + (u0 == 0 ? 1 : 0)) * C::kPart;
        for (int e = tid; e < ROWS * DIM / 4; e += kAttnThreads) {
            const int r = e / (DIM / 4), d = (e % (DIM / 4)) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            float top = -INFINITY, sum = 0.f;
            #pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_stat[0][w][r]);
            #pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float4 x = *reinterpret_cast<const float4*>(join + (w * ROWS + r) * C::kPad + d);
                o.x += x.x;
                o.y += x.y;
                o.z += x.z;
                o.w += x.w;
                const float mw = s_stat[0][w][r];
                sum += mw == -INFINITY ? s_stat[1][w][r] : s_stat[1][w][r] * exp2_fast(mw - top);
            }
            if (whole) {
                if (r < n_rows) {
                    const int row = t.row0 + r;
                    const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
                    __half* out = a.out + ((int64_t)(s.first + row / a.group) * a.heads_q + h * a.group + row % a.group) * DIM + d;
                    store4(out, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                }
            } else {
                *reinterpret_cast<float4*>(part + r * DIM + d) = o;
                if (d == 0) *reinterpret_cast<float2*>(part + ROWS * DIM + 2 * r) = make_float2(top, sum);
            }
        }
        if (!whole) {
            // the last CTA of the tile to arrive joins the pieces in their order
            __threadfence();
            __syncthreads();
            const int64_t c0 = walk.first_cta(t), c1 = walk.last_cta(t);
            if (tid == 0) {
                const unsigned n = atomicAdd(a.tickets + c0, 1u);
                s_last = n == (unsigned)(c1 - c0);
                if (s_last) a.tickets[c0] = 0u;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                // a warp takes rows in turn, its lanes first a piece each (the statistics),
                // then dimensions each, 8 or 16 pieces under way
                const int n = (int)(c1 - c0) + 1;
                constexpr int V = DIM / 32;  // dimensions of a lane
                auto piece = [&](int i) -> const float* {  // the first CTA's is its second
                    return a.parts + ((c0 + i) * 2 + (i == 0 ? 1 : 0)) * C::kPart;
                };
                for (int r = warp; r < n_rows; r += kWarps) {
                    float top = -INFINITY, sum = 0.f, o[V] = {};
                    for (int i0 = 0; i0 < n; i0 += 32) {
                        float2 st = make_float2(-INFINITY, 0.f);
                        if (i0 + lane < n) st = __ldcg(reinterpret_cast<const float2*>(piece(i0 + lane) + ROWS * DIM + 2 * r));
                        float most = st.x;
                        #pragma unroll
                        for (int x = 16; x >= 1; x >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, x));
                        const float was = top;
                        top = fmaxf(top, most);
                        const float f = was == -INFINITY ? 1.f : exp2_fast(was - top);
                        const float g = st.x == -INFINITY ? 1.f : exp2_fast(st.x - top);  // no keys: zeros (or NaN)
                        float add = st.y * g;
                        #pragma unroll
                        for (int x = 16; x >= 1; x >>= 1) add += __shfl_xor_sync(0xFFFFFFFFu, add, x);
                        sum = fmaf(sum, f, add);
                        #pragma unroll
                        for (int v = 0; v < V; ++v) o[v] *= f;
                        const int m = min(32, n - i0);
                        constexpr int Y = NR == 1 && V <= 4 ? 16 : 8;
                        #pragma unroll 1
                        for (int i = 0; i < m; i += Y) {
                            float x[Y][V];
                            #pragma unroll
                            for (int y = 0; y < Y; ++y) {
                                const float* p = piece(i0 + min(i + y, m - 1)) + r * DIM + V * lane;
                                if constexpr (V == 2) {
                                    const float2 z = __ldcg(reinterpret_cast<const float2*>(p));
                                    x[y][0] = z.x, x[y][1] = z.y;
                                } else {
                                    #pragma unroll
                                    for (int v = 0; v < V; v += 4) {
                                        const float4 z = __ldcg(reinterpret_cast<const float4*>(p + v));
                                        x[y][v] = z.x, x[y][v + 1] = z.y, x[y][v + 2] = z.z, x[y][v + 3] = z.w;
                                    }
                                }
                            }
                            #pragma unroll
                            for (int y = 0; y < Y; ++y) {
                                const float w = __shfl_sync(0xFFFFFFFFu, g, (i + y) & 31);
                                if (i + y < m) {
                                    #pragma unroll
                                    for (int v = 0; v < V; ++v) o[v] = fmaf(x[y][v], w, o[v]);
                                }
                            }
                        }
                    }
                    const int row = t.row0 + r;
                    const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
                    __half* out = a.out + ((int64_t)(s.first + row / a.group) * a.heads_q + h * a.group + row % a.group) * DIM + V * lane;
                    #pragma unroll
                    for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(out + v) = pack_half2(o[v] * inv, o[v + 1] * inv);
                }
            }
        }
        __syncthreads();  // the join buffer becomes a ring again
    }
}

template <int DIM, int BITS, int NR>
int attn_ctas(int sms) {
    using C = Cfg<DIM, BITS, NR>;
    static_assert(C::kCtas * (C::kSmem + 2048) <= 227 * 1024, "the CTAs of an SM share its memory");
    const int n = sms * C::kCtas;
    return n < kAttnMaxCtas ? n : kAttnMaxCtas;
}

// Row blocks of 8 when the rows that share a cache head fill no more on average.
bool one_group(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q) {
    return (b.tokens * (heads_q / c.heads) + b.seqs - 1) / b.seqs <= 8;
}

template <typename F>
auto by_config(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q, F f) {
    auto rows = [&](auto dim, auto bits) {
        return one_group(c, b, heads_q) ? f(dim, bits, std::integral_constant<int, 1>())
                                        : f(dim, bits, std::integral_constant<int, 2>());
    };
    auto bits = [&](auto dim) {
        return c.bits == 8 ? rows(dim, std::integral_constant<int, 8>()) : rows(dim, std::integral_constant<int, 4>());
    };
    return c.dim == 64    ? bits(std::integral_constant<int, 64>())
           : c.dim == 128 ? bits(std::integral_constant<int, 128>())
                          : bits(std::integral_constant<int, 256>());
}

}  // namespace

size_t attn_rows_workspace(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q, int sms) {
    return by_config(c, b, heads_q, [&](auto dim, auto bits, auto nr) -> size_t {
        constexpr int D = decltype(dim)::value, B = decltype(bits)::value, N = decltype(nr)::value;
        return kAttnTicketBytes + (size_t)attn_ctas<D, B, N>(sms) * 2 * Cfg<D, B, N>::kPart * sizeof(float);
    });
}

cudaError_t launch_attn_rows(const kvq_cache_t& c, const kvq_batch_t& b, const uint16_t* Q, int heads_q,
                                 const uint64_t* mask, float scale, uint16_t* out, void* ws, int sms, unsigned flags,
                                 cudaStream_t stream) {
    const AttnArgs a = {cache_arg(c), batch_arg(b), reinterpret_cast<const __half*>(Q), mask,
                        reinterpret_cast<__half*>(out), heads_q, heads_q / c.heads, scale * 1.4426950408889634f,
                        static_cast<unsigned*>(ws),
                        reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnTicketBytes)};
    return by_config(c, b, heads_q, [&](auto dim, auto bits, auto nr) {
        constexpr int D = decltype(dim)::value, B = decltype(bits)::value, N = decltype(nr)::value;
        auto* f = attn_kernel<D, B, N>;
        static std::atomic<uint64_t> ready{0};  // devices whose shared-memory limit is set
        const cudaError_t e = layer_smem(f, Cfg<D, B, N>::kSmem, ready);
        if (e != cudaSuccess) return e;
        return layer_launch(f, dim3((unsigned)attn_ctas<D, B, N>(sms)), kAttnThreads, Cfg<D, B, N>::kSmem, flags, stream, a);
    });
}

cudaError_t read_and_clear_attn_rows_error(unsigned* flags, cudaStream_t stream) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_attn_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_attn_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *flags |= v;
    return e;
}

}  // namespace w4a8
