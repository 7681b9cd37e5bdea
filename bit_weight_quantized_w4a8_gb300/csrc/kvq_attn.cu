// kvq_attn.cu -- attention of decode rows and of drafted trees over the
// quantized paged cache:
//   t_j = scale ks_j (q . kc_j),  p_j = exp(t_j - max t),  out = sum p_j vs_j vc_j / sum p_j.
//
// The rows that share a cache head (tokens x heads_q / heads of them) are taken
// in blocks of 8 or 16; a CTA of four warps walks the keys of one (sequence,
// head, row block) in units of 128, each warp its own 32, and the warps' and
// CTAs' pieces are joined by their softmax statistics.  The work of the whole
// batch, in units, is cut into equal runs for the CTAs on the device, from the
// lengths that it finds there: long and short sequences fill the GPU alike, and
// a captured graph follows its lengths.
//
// Both products run on mma.sync m16n8k16 with the cache as the M operand, so
// that 8 rows are enough to fill an instruction: S^T = K Q^T, then O^T = V^T W^T,
// W^T being S^T's weights transposed by movmatrix.  Codes are integers of
// at most 7 bits and sign, exact in binary16, and the scales stay outside the products:
// ks_j multiplies the fp32 logit, vs_j the fp32 weight before its rounding.
#include <type_traits>

#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

__device__ unsigned g_attn_error;

constexpr int kAttnThreads = 128;
constexpr int kWarps = 4;
constexpr int kStep = 32;                 // keys of a warp's step
constexpr int kUnit = kStep * kWarps;     // keys of a CTA's unit of work
constexpr int kTicketBytesAttn = 4096;    // arrival counters, one per CTA
constexpr int kMaxCtas = kTicketBytesAttn / 4;

struct AttnArgs {
    KvqCacheArg c;
    KvqBatchArg b;
    const __half* Q;
    const uint64_t* mask;
    __half* out;
    int heads_q, group;  // query heads of a cache head
    float scale_log2;
    unsigned* tickets;
    float* parts;
};

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22 relative
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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
    static constexpr int kStages = W >= 256 ? 3 : W == 128 ? 3 : 4;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kRows = 8 * NR;
    static constexpr int kPad = DIM + 4;
    static constexpr int kJoin = kWarps * kRows * kPad * 4;  // the warps' sums, over the ring
    static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
    static constexpr int kPart = kRows * (DIM + 2);          // floats of a CTA's piece
};

// Units of sequence b: row blocks x heads x units of keys (at least one, which
// writes the zeros of rows that see nothing).
struct SeqWork {
    int blocks;
    int64_t units;  // per (row block, head)
};
__device__ __forceinline__ SeqWork seq_work(const AttnArgs& a, const KvqSeq& s, int rows) {
    SeqWork w;
    w.blocks = (int)(((int64_t)s.count * a.group + rows - 1) / rows);
    const int64_t end = a.mask != nullptr && s.count > KVQ_MAX_TREE ? 0 : s.end;
    w.units = end > 0 ? (end + kUnit - 1) / kUnit : 1;
    return w;
}

template <int DIM, int BITS, int NR>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(const AttnArgs a) {
    using C = Cfg<DIM, BITS, NR>;
    constexpr int W = C::W, ROWS = C::kRows;
    constexpr int KC = W / 64 > 0 ? W / 64 : 1;  // 16-byte (W = 32: 8-byte) runs of a key per lane
    constexpr int KW = W == 32 ? 2 : 4;          // words of a run
    constexpr int MT = DIM / 16;                 // 16-dim tiles of the output
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_units[kWarps], s_find[2];
    __shared__ float s_stat[3][kWarps][ROWS];
    __shared__ unsigned s_last;
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t4 = lane & 3;

    // total work, then the run of this CTA: units [begin, end)
    int64_t total = 0;
    for (int b0 = 0; b0 < a.b.seqs; b0 += kAttnThreads) {
        if (b0 + tid < a.b.seqs) {
            const KvqSeq s = kvq_seq(a.b.cu, a.b.start, b0 + tid, a.b.tokens, a.b.max_pages, a.c.shift);
            if (!s.ok || (a.mask != nullptr && s.count > KVQ_MAX_TREE)) atomicOr(&g_attn_error, kErrCacheRange);
            const SeqWork w = seq_work(a, s, ROWS);
            total += w.units * w.blocks * a.c.heads;
        }
    }
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
    if (lane == 0) s_units[warp] = total;
    __syncthreads();
    total = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_units[w];
    const int64_t per = (total + gridDim.x - 1) / gridDim.x;
    int64_t at = per * blockIdx.x;  // next unit of the batch
    const int64_t run_end = min(at + per, total);
    if (at >= run_end) return;

    // the sequence that holds unit `at`: found by warp 0, 32 sequences a time
    if (warp == 0) {
        int64_t before = 0;
        for (int b0 = 0; b0 < a.b.seqs; b0 += 32) {
            int64_t n = 0;
            if (b0 + lane < a.b.seqs) {
                const KvqSeq s = kvq_seq(a.b.cu, a.b.start, b0 + lane, a.b.tokens, a.b.max_pages, a.c.shift);
                const SeqWork w = seq_work(a, s, ROWS);
                n = w.units * w.blocks * a.c.heads;
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
                    s_find[0] = b0 + lane;
                    s_find[1] = before + sum - n;
                }
                break;
            }
            before += __shfl_sync(0xFFFFFFFFu, sum, 31);
        }
    }
    __syncthreads();
    int b = (int)s_find[0];
    int64_t seq_first = s_find[1];  // first unit of sequence b

    const uint32_t ring = smem_u32(smem) + warp * (C::kStages * C::kStageBytes);
    const int64_t page_mask = (1 << a.c.shift) - 1;

    while (at < run_end) {
        const KvqSeq s = kvq_seq(a.b.cu, a.b.start, b, a.b.tokens, a.b.max_pages, a.c.shift);
        const SeqWork sw = seq_work(a, s, ROWS);
        const int64_t seq_units = sw.units * sw.blocks * a.c.heads;
        if (at >= seq_first + seq_units) {
            seq_first += seq_units;
            ++b;
            continue;
        }
        // tile: units [tile_first, tile_first + units) are head h, row block rb
        const int64_t tile = (at - seq_first) / sw.units;
        const int64_t tile_first = seq_first + tile * sw.units;
        const int h = (int)(tile / sw.blocks), rb = (int)(tile - (int64_t)h * sw.blocks);
        const int u0 = (int)(at - tile_first);
        const int u1 = (int)(min(run_end, tile_first + sw.units) - tile_first);
        at = tile_first + u1;
        const int n_rows = min(ROWS, s.count * a.group - rb * ROWS);
        // slots that some row of the block may see end here
        int64_t key_end = a.mask != nullptr && s.count > KVQ_MAX_TREE ? 0 : s.end;
        if (a.mask == nullptr) {
            const int64_t last = s.start + (rb * ROWS + n_rows - 1) / a.group + 1;
            if (last < key_end) key_end = last;
        }

        // queries: B operands, row 8 nr + g, in the order in which the key's runs
        // are widened
        uint32_t qf[NR][DIM / 16][2];
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int r = rb * ROWS + 8 * nr + g;
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
        float m[NR][2], l[NR][2];
        #pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            m[nr][0] = m[nr][1] = -INFINITY;
            l[nr][0] = l[nr][1] = 0.f;
            #pragma unroll
            for (int i = 0; i < MT; ++i)
                #pragma unroll
                for (int k = 0; k < 4; ++k) acc[nr][i][k] = 0.f;
        }
        // value scales are taken relative to v_unit, a power of two above all met
        // so far, times 2^-8: weights below 2^-6 of the largest keep 11 bits
        // down to 2^-22 of it
        float v_unit = 0x1p-100f;

        // page of this lane's key (lane = key of the step) for step u
        auto page_of = [&](int u) -> int {
            const int64_t k = (int64_t)u * kUnit + warp * kStep + lane;
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
                const int64_t k0 = (int64_t)u * kUnit + warp * kStep;
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
            const int64_t k0 = (int64_t)u * kUnit + warp * kStep;
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
                        const int tok = (rb * ROWS + min(r, n_rows - 1)) / a.group;
                        const uint64_t word = a.mask != nullptr ? a.mask[s.first + tok] : 0;
                        #pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
                            #pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const int kk = 16 * mt + 8 * hf + g;
                                const int64_t w = k0 + kk - s.start;
                                bool see = (ok_keys >> kk) & 1;
                                if (w >= 0) see = see && (a.mask != nullptr ? w < 64 && ((word >> w) & 1) : w <= tok);
                                if (!see) {
                                    seen &= ~(1u << ((mt * NR + nr) * 4 + 2 * hf + e));
                                    sc[mt][nr][2 * hf + e] = -INFINITY;
                                }
                            }
                    }
            }

            // running maximum per row
            float mn[NR][2];
            bool grew = false;
            #pragma unroll
            for (int nr = 0; nr < NR; ++nr)
                #pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(sc[0][nr][e], sc[0][nr][2 + e]), fmaxf(sc[1][nr][e], sc[1][nr][2 + e]));
                    #pragma unroll
                    for (int o = 4; o <= 16; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
                    mn[nr][e] = fmaxf(m[nr][e], x);
                    grew |= mn[nr][e] > m[nr][e];
                }
            // largest finite value scale of the step
            float v_old = v_unit;
            {
                const float v = fabsf(lds_f(sv + 4 * lane));
                const unsigned top = __reduce_max_sync(0xFFFFFFFFu, v < INFINITY ? __float_as_uint(v) : 0u);
                if (__uint_as_float(top) > v_unit)
                    v_unit = __uint_as_float(min((top & 0x7F800000u) + 0x00800000u, 0x7E800000u));
            }
            if (__any_sync(0xFFFFFFFFu, grew) || v_unit != v_old) {
                const float vr = v_old / v_unit;
                #pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float f[2];
                    #pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        f[e] = mn[nr][e] == -INFINITY ? 1.f : exp2_fast(m[nr][e] - mn[nr][e]);
                        l[nr][e] *= f[e];
                        f[e] *= vr;
                        m[nr][e] = mn[nr][e];
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
            const float v_inv = 256.f / v_unit;
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
                        const float vv = vf[mt][hf] * v_inv;
                        float w0 = p0 * vv, w1 = p1 * vv;
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
                const float f = m[nr][e] == -INFINITY ? 0.f : exp2_fast(m[nr][e] - top) * (v_unit * 0x1p-8f);
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

        const bool whole = u0 == 0 && u1 == (int)sw.units;
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
                    const int row = rb * ROWS + r;
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
            const int64_t c0 = tile_first / per, c1 = (tile_first + sw.units - 1) / per;
            if (tid == 0) {
                const unsigned n = atomicAdd(a.tickets + c0, 1u);
                s_last = n == (unsigned)(c1 - c0);
                if (s_last) a.tickets[c0] = 0u;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                for (int e = tid; e < n_rows * DIM / 4; e += kAttnThreads) {
                    const int r = e / (DIM / 4), d = (e % (DIM / 4)) * 4;
                    float top = -INFINITY;
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float* p = a.parts + (c * 2 + (c == c0 ? 1 : 0)) * C::kPart;
                        top = fmaxf(top, __ldcg(p + ROWS * DIM + 2 * r));
                    }
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
                    #pragma unroll 4
                    for (int64_t c = c0; c <= c1; ++c) {
                        const float* p = a.parts + (c * 2 + (c == c0 ? 1 : 0)) * C::kPart;
                        const float2 st = __ldcg(reinterpret_cast<const float2*>(p + ROWS * DIM + 2 * r));
                        const float4 x = __ldcg(reinterpret_cast<const float4*>(p + r * DIM + d));
                        const float f = st.x == -INFINITY ? 1.f : exp2_fast(st.x - top);  // no keys: zeros (or NaN)
                        o.x = fmaf(x.x, f, o.x);
                        o.y = fmaf(x.y, f, o.y);
                        o.z = fmaf(x.z, f, o.z);
                        o.w = fmaf(x.w, f, o.w);
                        sum = fmaf(st.y, f, sum);
                    }
                    const int row = rb * ROWS + r;
                    const float inv = top == -INFINITY && sum == 0.f ? 0.f : 1.f / sum;
                    __half* out = a.out + ((int64_t)(s.first + row / a.group) * a.heads_q + h * a.group + row % a.group) * DIM + d;
                    store4(out, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                }
            }
        }
        __syncthreads();  // the join buffer becomes a ring again
    }
}

template <int DIM, int BITS, int NR>
int attn_ctas(int sms) {
    // two CTAs an SM where their rings fit
    const int per_sm = 2 * (Cfg<DIM, BITS, NR>::kSmem + 2048) <= 227 * 1024 ? 2 : 1;
    const int n = sms * per_sm;
    return n < kMaxCtas ? n : kMaxCtas;
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

size_t kvq_attn_workspace(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q, int sms) {
    return by_config(c, b, heads_q, [&](auto dim, auto bits, auto nr) -> size_t {
        constexpr int D = decltype(dim)::value, B = decltype(bits)::value, N = decltype(nr)::value;
        return kTicketBytesAttn + (size_t)attn_ctas<D, B, N>(sms) * 2 * Cfg<D, B, N>::kPart * sizeof(float);
    });
}

cudaError_t launch_kvq_attention(const kvq_cache_t& c, const kvq_batch_t& b, const uint16_t* Q, int heads_q,
                                 const uint64_t* mask, float scale, uint16_t* out, void* ws, int sms, unsigned flags,
                                 cudaStream_t stream) {
    const AttnArgs a = {cache_arg(c), batch_arg(b), reinterpret_cast<const __half*>(Q), mask,
                        reinterpret_cast<__half*>(out), heads_q, heads_q / c.heads, scale * 1.4426950408889634f,
                        static_cast<unsigned*>(ws),
                        reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kTicketBytesAttn)};
    return by_config(c, b, heads_q, [&](auto dim, auto bits, auto nr) {
        constexpr int D = decltype(dim)::value, B = decltype(bits)::value, N = decltype(nr)::value;
        auto* f = attn_kernel<D, B, N>;
        cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, B, N>::kSmem);
        if (e != cudaSuccess) return e;
        return layer_launch(f, dim3((unsigned)attn_ctas<D, B, N>(sms)), kAttnThreads, Cfg<D, B, N>::kSmem, flags, stream, a);
    });
}

cudaError_t read_and_clear_attn_error(unsigned* flags, cudaStream_t stream) {
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
