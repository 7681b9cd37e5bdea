// kvq_tree.cu -- attention of many rows over the quantized paged cache (trees of
// drafted tokens times the query heads of a cache head) on the 5th-generation
// tensor cores; formulas and rounding as in kvq_attn.cu.
//
// With hundreds of rows on each key the work is the two products, which only
// tcgen05 runs at full rate, so the codes are widened to binary16 once
// per CTA, in shared memory, for up to 256 rows:
//   warps 16-23 copy the codes of 128 keys and values into shared memory, one or
//     two blocks ahead, widen them and store them in the tensor core's 128-byte swizzled
//     layout (codes held in registers came at 12.6 bytes a cycle and SM: 260 us
//     instead of 204 in the second case below);
//   warps 0-7 and 8-15 are two slots of softmax: S is read from TMEM, the
//     weights go back over it as binary16;
//   the first warp of a slot issues its products: S = Q K^T into TMEM (128 rows x
//     128 keys), and O += W V with the weights W as the TMEM operand and V with its
//     dimensions contiguous (the transposed B operand), so nothing is transposed.
// The slots take two tiles of 128 rows in turn; when a row block has only one
// tile, they take alternate keys of the same rows and are joined like two CTAs.  While
// one slot computes weights the tensor core works for the other.
//
// Softmax: row r keeps a reference M; p_j = 2^(t_j - M) is summed in fp32 and w_j
// = p_j vs_j rounded to binary16.  M is the maximum of t_j + e - 10 so far, 2^e being a bound
// of the value scales that the row sees near j, and is raised (and O and the sum
// rescaled) only when a weight would pass 2^14: so seldom that O stays in TMEM.
//
// Measured in graphs, with the join: 6 trees of 9, 32 heads on 2, 30001 keys of 4 bits 65 us;
// 4 trees of 64, 28 heads on 4, 32001 keys of 8 bits 177 us, 30% of the tensor
// cores' measured rate (kvq_attn.cu: 534), heads of 64 148.  A block of 128 keys and 256 rows takes
// 2.9 us, its products 1.07, the softmax without products and loads 2.1: bound by the chain S,
// weights, product within a slot.  (Keys of the next block widened while this one is
// at work: 84.5 -> 74.4 us for 4 trees of 16 on one tile, 194 -> 186 for those of 64.)
#include <atomic>
#include <cstddef>
#include <type_traits>

#include "kernels.h"
#include "kvq_attn.cuh"
#include "kvq_roles.h"
#include "tc.cuh"

namespace w4a8 {
namespace {

// Two slots of eight softmax warps and eight that load: six warps to a scheduler,
// 80 registers a thread.  Everything here waits for something (loads, TMEM,
// barriers), so many warps with little each.  All four forms spill (60 to 88 bytes a thread,
// -Xptxas -v), and a spilled register costs a trip to L2, as the tiles leave no
// first-level cache: what only some blocks need is kept out of the others' way (score_masked).
constexpr int kSlotWarps = 8, kSoftWarps = 2 * kSlotWarps, kLoadWarps = 8;
constexpr int kTreeThreads = (kSoftWarps + kLoadWarps) * 32;
constexpr int kRowsTile = 128;   // rows of a tile, TMEM lanes
constexpr int kBlock = 128;      // keys of a unit
constexpr int kScaleRing = 4;    // blocks whose scales are held

struct alignas(16) BlockScales {  // read as 16-byte vectors
    float k[kBlock];        // ks * scale * log2(e), never 0
    float v[kBlock];        // vs, 0 where one of the two is bad: not finite
    float vmax[8];          // largest |v| of keys 16 w .. 16 w + 15
    uint32_t odd[8];        // not 0: some of them is not there or bad
    uint16_t valid[8];      // bit i of word w: key 16 w + i is there
    uint16_t bad[8];        // it has a bad scale
};

struct TreeShared {
    uint64_t kfull[2], vfull[2];   // [block % 2]: its keys, values are in place
    uint64_t scfull[kScaleRing];   // [block % 4]: its scales are
    uint64_t sfull[2];             // [slot]: S of a job is there, and the product before it done
    uint64_t kfree[2], vfree[2];   // [block % 2]: both slots' products have used them
    uint64_t drain[2];
    BlockScales sc[kScaleRing];
    AttnWalk<kTreeThreads, kRowsTile, 2, kBlock>::Shared find;
    AttnWalk<kTreeThreads, kRowsTile, 2, kBlock> walk;  // thread 0's
    AttnTile tile;                                      // and where it is
    float ref[2][kRowsTile];      // [slot][row]: reference
    float sum[2][2][kRowsTile];   // [slot][half of the keys][row]
    float top[2][2][kRowsTile];   // a block's maxima, exchanged when a reference is raised
    uint64_t word[2][kRowsTile];  // [tile][row]: what its token sees of the drafted ones
    int tok[2][kRowsTile];        // and its place among them
    int more;
    uint32_t tmem;
    volatile int abort;
};

static_assert(offsetof(TreeShared, sc) % 16 == 0 && sizeof(BlockScales) % 16 == 0 && offsetof(BlockScales, v) % 16 == 0,
              "scales are read as 16-byte vectors");

template <int DIM, int BITS>
struct TreeCfg {
    static constexpr int W = DIM * BITS / 8;
    static constexpr int kHalf = kRowsTile * 128;            // 128 rows of 64 binary16 values
    static constexpr int kTileBytes = kHalf * (DIM / 64);
    static constexpr int kRawBytes = 16 * W;                 // codes of a loading warp's 16 keys or values
    // two tiles of Q and of K, then what fits: the raw codes of two blocks, two tiles of V
    static constexpr int kRaw = kLoadWarps * 2 * kRawBytes;  // of a block
    static constexpr int kRoom = 227 * 1024 - (int)sizeof(TreeShared) - 1024;  // - alignment
    static constexpr int kRawStages = 5 * kTileBytes + 2 * kRaw <= kRoom ? 2 : 1;
    static constexpr int kValueTiles = 6 * kTileBytes + kRawStages * kRaw <= kRoom ? 2 : 1;
    static constexpr int kOffQ = 0, kOffK = 2 * kTileBytes, kOffV = 4 * kTileBytes, kOffRaw = (4 + kValueTiles) * kTileBytes;
    static constexpr int kOffShared = kOffRaw + kRawStages * kRaw;
    static constexpr int kSmem = kOffShared + (int)sizeof(TreeShared) + 1024;
    static_assert(kSmem <= 227 * 1024, "one CTA's shared memory");
    static constexpr int kPiece = kRowsTile * (DIM + 2);     // floats: O [DIM][128], M, sum
    static constexpr uint32_t kS = 0, kO = 256;              // TMEM columns: S of slot i at 128 i, O at 256 + DIM i
    static constexpr uint32_t kCols = 512;
};

// What a CTA leaves behind its piece for the join: the row block that it began and
// that others went on with.
struct alignas(16) JoinRecord {
    int pieces;  // 1: there is none
    int rows, row0, first, h;
};
template <int DIM, int BITS>
__device__ __forceinline__ JoinRecord* join_record(const AttnArgs& a, int cta) {
    return reinterpret_cast<JoinRecord*>(a.parts + (int64_t)gridDim.x * 4 * TreeCfg<DIM, BITS>::kPiece) + cta;
}

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    #pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (;;) {
        #pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort_flag = 1;
            atomicOr(&g_attn_error, kErrFullWait);
            return false;
        }
    }
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Byte of 16-byte chunk c (8 values) of row r in a tile of 128 rows: halves of 64
// values, rows of 128 bytes, chunks permuted by chunk ^ (r % 8).
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)((c >> 3) * (kRowsTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// Draft tokens d0 .. d0 + 31 (negative: cached ones) that a row sees.
__device__ __forceinline__ uint32_t seen_bits(int d0, bool tree, uint64_t word, int tok) {
    if (d0 <= -32) return 0xFFFFFFFFu;
    if (!tree) {
        const int n = tok + 1 - d0;  // the first n
        return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
    }
    if (d0 >= 0) return d0 < 64 ? (uint32_t)(word >> d0) : 0u;
    return (uint32_t)(word << -d0) | ((1u << -d0) - 1u);
}

// Maxima of t + e over this thread's keys that its four rows see, 2^e a bound of the key's own
// value scale, for a block that some rows do not see all of: a large value must cost
// only the rows that see it.  S of an unseen key first becomes what its factor, of either
// sign, takes to -inf, S of a seen key with a bad scale NaN.  (A call of its own: written
// out, it made the other blocks slower, trees of 64 177 -> 182 us, 4 of 16 72 -> 74.)
__device__ __noinline__ float4 score_masked(uint32_t ts, const BlockScales* bs, const uint64_t* word, const int* tok, int d0,
                                            int half, bool tree) {
    const int c2 = 2 * (threadIdx.x & 3);
    const float* kf = bs->k + 64 * half + c2;
    const float* vf = bs->v + 64 * half + c2;
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    #pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t valid = reinterpret_cast<const uint32_t*>(bs->valid)[2 * half + c];
        const uint32_t bad = reinterpret_cast<const uint32_t*>(bs->bad)[2 * half + c] >> c2;
        uint64_t kk[4], ve[4];
        uint32_t none[8];  // what an unseen key's S becomes
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint2 k = *reinterpret_cast<const uint2*>(kf + 32 * c + 8 * j), v = *reinterpret_cast<const uint2*>(vf + 32 * c + 8 * j);
            kk[j] = pack2(__uint_as_float(k.x), __uint_as_float(k.y));
            ve[j] = pack2(log2_bound(v.x & 0x7FFFFFFFu), log2_bound(v.y & 0x7FFFFFFFu));
            none[2 * j] = 0xFF800000u ^ (k.x & 0x80000000u);
            none[2 * j + 1] = 0xFF800000u ^ (k.y & 0x80000000u);
        }
        #pragma unroll
        for (int hb = 0; hb < 2; ++hb) {
            uint32_t s[16], see[2];
            tmem_ld_frag32(ts + 32 * c + hb * (16u << 16), s);
            #pragma unroll
            for (int rr = 0; rr < 2; ++rr)
                see[rr] = (valid & seen_bits(d0 + 32 * c, tree, word[16 * hb + 8 * rr], tok[16 * hb + 8 * rr])) >> c2;
            tmem_ld_wait();
            #pragma unroll
            for (int x = 0; x < 16; ++x) {
                constexpr uint32_t one = 1;
                const uint32_t bit = one << (8 * (x >> 2) + (x & 1));
                if (!(see[(x >> 1) & 1] & bit)) s[x] = none[2 * (x >> 2) + (x & 1)];
                else if (bad & bit) s[x] = 0x7FFFFFFFu;
            }
            tmem_st_frag32(ts + 32 * c + hb * (16u << 16), s);
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
                #pragma unroll
                for (int rr = 0; rr < 2; ++rr) {
                    const float2 d = unpack2(fma2(pack2(__uint_as_float(s[4 * j + 2 * rr]), __uint_as_float(s[4 * j + 2 * rr + 1])), kk[j], ve[j]));
                    top[2 * hb + rr] = max3(top[2 * hb + rr], d.x, d.y);
                }
            }
        }
    }
    tmem_st_wait();
    return make_float4(top[0], top[1], top[2], top[3]);
}

// Column of dimension y in a group of eight: the widened 4-bit codes come in the
// order 0, 4, 1, 5, 2, 6, 3, 7.
template <int BITS>
__device__ __forceinline__ constexpr int column_of(int y) {
    return BITS == 8 ? y : (y < 4 ? 2 * y : 2 * y - 7);
}
__device__ __forceinline__ void store8(__half* p, const float* f) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
}

template <int DIM, int BITS>
__global__ void __launch_bounds__(kTreeThreads, 1) tree_kernel(const AttnArgs a) {
    using C = TreeCfg<DIM, BITS>;
    constexpr int KSTEPS = DIM / 16;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t base = smem_u32(smem);
    TreeShared& sh = *reinterpret_cast<TreeShared*>(smem + C::kOffShared);
    // (The join's CTAs do not fit beside this one, so that nothing after them, which might
    // hold TMEM while it waits for this kernel, starts before the allocation below.)
    griddep_launch_dependents();
    griddep_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);  // one value for the warp, known to the compiler as such

    if (tid == 0) join_record<DIM, BITS>(a, blockIdx.x)->pieces = 1;
    {
        AttnWalk<kTreeThreads, kRowsTile, 2, kBlock> walk;
        if (!walk.init(a, sh.find)) return;
        if (tid == 0) sh.walk = walk;
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.kfull[i]), kLoadWarps);
            mbar_init(smem_u32(&sh.vfull[i]), kLoadWarps);
            mbar_init(smem_u32(&sh.kfree[i]), 2);
            mbar_init(smem_u32(&sh.vfree[i]), 2);
            mbar_init(smem_u32(&sh.sfull[i]), 1);
            mbar_init(smem_u32(&sh.drain[i]), 1);
        }
        for (int i = 0; i < kScaleRing; ++i) mbar_init(smem_u32(&sh.scfull[i]), kLoadWarps);
        fence_mbar_init();
        sh.abort = 0;
    }
    if (warp == kSoftWarps) tmem_alloc(smem_u32(&sh.tmem), C::kCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const uint32_t u_tmem = __shfl_sync(0xFFFFFFFFu, tmem, 0), u_base = __shfl_sync(0xFFFFFFFFu, base, 0);
    const bool leader = elect_one();

    int blocks_done = 0;             // key blocks of earlier tiles: stage and phase go on
    int s_phase[2] = {0, 0};         // phases of sfull in earlier row blocks
    for (;;) {
        if (tid == 0) sh.more = sh.walk.next(a, sh.tile);
        __syncthreads();
        if (!sh.more) break;
        const AttnTile& t = sh.tile;  // the roles take what they need of it into registers
        const int nb = t.u1 - t.u0;
        const bool two = t.tiles == 2;
        if (warp >= kSoftWarps) {
            // codes of this warp's 16 keys of every block: copied one or two ahead as they
            // are, then widened into the tiles; lanes 0-15 have a key each for the page
            // table and the scales
            constexpr int CPR = C::W / 16;             // 16-byte chunks of codes per vector
            constexpr int N = CPR / 2;                 // of them per lane
            constexpr int R = C::kRawStages;
            const int lw = warp - kSoftWarps;
            const int u0 = t.u0, u1 = t.u1, key_end = t.key_end, h = t.h;
            const int32_t* table = a.b.table + t.b * a.b.max_pages;
            const uint32_t raw = base + C::kOffRaw + lw * 2 * R * C::kRawBytes;
            const int pmask = (1 << a.c.shift) - 1;
            const int key = 16 * lw + (lane & 15);
            auto page_of = [&](int u) -> int {  // as the table has it
                const int k = u * kBlock + key;
                return u < u1 && k < key_end ? table[k >> a.c.shift] : -1;
            };
            // a block's place: the vector of the first of the 16 keys (one page holds all),
            // this lane's, and which of them are in range
            struct Place {
                int64_t first, own;
                uint32_t there;
            };
            auto place = [&](int u, int page) -> Place {
                const int k = u * kBlock + key;
                const bool ok = page >= 0 && page < a.c.pages;
                if (!ok && u < u1 && k < key_end) atomicOr(&g_attn_error, kErrCacheRange);
                Place p;
                p.own = ok ? ((((int64_t)page * a.c.heads + h) << a.c.shift) + (k & pmask)) : 0;
                p.there = __ballot_sync(0xFFFFFFFFu, ok) & 0xFFFFu;
                p.first = __shfl_sync(0xFFFFFFFFu, p.own, 0);
                return p;
            };
            // chunk c of row r of a raw tile, permuted so that 8 rows' chunks c lie in
            // different banks
            auto raw_off = [&](int r, int c) -> uint32_t {
                if (CPR >= 8) return r * C::W + (c >> 3) * 128 + (((c & 7) ^ (r & 7)) << 4);
                if (CPR == 4) return (r >> 1) * 128 + ((((r & 1) << 2) + (c ^ ((r >> 1) & 3))) << 4);
                return (r >> 2) * 128 + ((((r & 3) << 1) + (c ^ ((r >> 2) & 1))) << 4);
            };
            auto copy = [&](int u, const Place& p, const uint8_t* codes, int kv) {
                if (u < u1) {
                    const uint32_t dst = raw + (2 * ((u - u0) % R) + kv) * C::kRawBytes;
                    #pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const int r = (32 * i + lane) / CPR, c = (32 * i + lane) % CPR;
                        cp_async_16_zfill(dst + raw_off(r, c), codes + (p.first + r) * C::W + 16 * c, (p.there >> r) & 1 ? 16u : 0u);
                    }
                }
                cp_async_commit();
            };
            // 8 lanes on 8 rows of one chunk meet each bank once, here and in the tile
            auto widen = [&](uint32_t dst, int j, int kv) {
                const uint32_t src = raw + (2 * (j % R) + kv) * C::kRawBytes;
                #pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int r = CPR >= 4 ? 8 * (i / (CPR / 4 > 0 ? CPR / 4 : 1)) + (lane & 7) : 8 * (lane >> 4) + (lane & 7);
                    const int c = CPR >= 4 ? (lane >> 3) + 4 * (i % (CPR / 4 > 0 ? CPR / 4 : 1)) : (lane >> 3) & 1;
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(src + raw_off(r, c)));
                    if constexpr (BITS == 8) {
                        uint32_t x[8];
                        #pragma unroll
                        for (int y = 0; y < 4; ++y) widen8(w[y], x[2 * y], x[2 * y + 1]);
                        sts16(dst + tile_off(16 * lw + r, 2 * c), x[0], x[1], x[2], x[3]);
                        sts16(dst + tile_off(16 * lw + r, 2 * c + 1), x[4], x[5], x[6], x[7]);
                    } else {
                        #pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t x[4];
                            widen4(w[y], x[0], x[1]);
                            widen4(w[y] >> 8, x[2], x[3]);
                            sts16(dst + tile_off(16 * lw + r, 4 * c + y), x[0], x[1], x[2], x[3]);
                        }
                    }
                }
            };
            auto freed = [&](uint64_t* bars, int blk, int tiles) -> bool {  // of the block whose tile blk takes
                const int was = blk - tiles;
                return was < 0 || __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&bars[was & 1]), (was >> 1) & 1, &sh.abort));
            };
            auto arrive = [&](uint64_t& bar) {
                fence_async_shared();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar));
            };
            auto scale_of = [&](const float* p, const Place& at) -> float { return at.there >> (lane & 15) & 1 ? p[at.own] : 0.f; };
            Place at[R + 1];  // of blocks t .. t + R
            #pragma unroll
            for (int r = 0; r < R; ++r) {
                at[r] = place(u0 + r, page_of(u0 + r));
                copy(u0 + r, at[r], a.c.k, 0);
                copy(u0 + r, at[r], a.c.v, 1);
            }
            int page = page_of(u0 + R);
            float sk = scale_of(a.c.ks, at[0]), sv = scale_of(a.c.vs, at[0]);
            // Keys of block t, then the values of the block before: the keys go into the
            // tile that block t - 2 has left while block t - 1 is at work, the values, where
            // they have one tile, follow its products.  A block's codes are copied when
            // those R before it have been widened.
            for (int t = 0; t <= nb; ++t) {
                const int blk = blocks_done + t;
                at[R] = place(u0 + t + R, page);
                page = page_of(u0 + t + R + 1);
                if (t < nb) {
                    BlockScales& bs = sh.sc[blk % kScaleRing];
                    {
                        // a factor of 0 would make NaN of an unseen key's -inf; a key of zeros
                        // has logit 0 with any
                        const float kk = sk * a.scale_log2;
                        const bool fine = fabsf(kk) < INFINITY && fabsf(sv) < INFINITY;
                        if (lane < 16) {
                            bs.k[key] = fine && kk != 0.f ? kk : 1e-30f;
                            bs.v[key] = fine ? sv : 0.f;
                        }
                        const unsigned bad = __ballot_sync(0xFFFFFFFFu, !fine) & 0xFFFFu;
                        const unsigned vmax = __reduce_max_sync(0xFFFFFFFFu, fine ? __float_as_uint(fabsf(sv)) : 0u);
                        if (lane == 0) {
                            bs.vmax[lw] = __uint_as_float(vmax);
                            bs.odd[lw] = (at[0].there ^ 0xFFFFu) | bad;
                            bs.valid[lw] = (uint16_t)at[0].there;
                            bs.bad[lw] = (uint16_t)bad;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&sh.scfull[blk % kScaleRing]));
                    sk = scale_of(a.c.ks, at[1]);
                    sv = scale_of(a.c.vs, at[1]);
                    if (t >= 1 && t <= R) cp_async_wait<2 * R - 2>();  // the first values went out before these keys
                    else cp_async_wait<2 * R - 1>();
                    __syncwarp();
                    if (!freed(sh.kfree, blk, 2)) break;
                    widen(base + C::kOffK + (blk & 1) * C::kTileBytes, t, 0);
                    arrive(sh.kfull[blk & 1]);
                    copy(u0 + t + R, at[R], a.c.k, 0);
                }
                if (t > 0) {
                    const int prev = blk - 1;
                    if (t < nb) cp_async_wait<2 * R - 1>();
                    else cp_async_wait<2 * R - 2>();
                    __syncwarp();
                    if (!freed(sh.vfree, prev, C::kValueTiles)) break;
                    widen(base + C::kOffV + prev % C::kValueTiles * C::kTileBytes, t - 1, 1);
                    arrive(sh.vfull[prev & 1]);
                    copy(u0 + t - 1 + R, at[R - 1], a.c.v, 1);
                }
                #pragma unroll
                for (int r = 0; r < R; ++r) at[r] = at[r + 1];
            }
            cp_async_wait<0>();
        } else {
            // the queries of the block's rows, in the widened keys' order of dimensions, and
            // what the rows see of the drafted tokens
            {
                constexpr int kRowsAt = kSoftWarps * 32 / (DIM / 8);  // rows of one pass
                constexpr int kPasses = 2 * kRowsTile / kRowsAt;
                const int c = tid % (DIM / 8), step_tok = kRowsAt / a.group, step_head = kRowsAt % a.group;
                int r = tid / (DIM / 8), tok = (t.row0 + r) / a.group, head = (t.row0 + r) % a.group;
                uint4 x[kPasses];
                #pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    x[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r + kRowsAt * i < t.rows)
                        x[i] = *reinterpret_cast<const uint4*>(a.Q + ((int64_t)(t.s.first + tok) * a.heads_q + t.h * a.group + head) * DIM + 8 * c);
                    tok += step_tok;
                    head += step_head;
                    if (head >= a.group) head -= a.group, ++tok;
                }
                #pragma unroll
                for (int i = 0; i < kPasses; ++i, r += kRowsAt) {
                    if (r >= t.tiles * kRowsTile) break;
                    if constexpr (BITS == 4)
                        x[i] = make_uint4(__byte_perm(x[i].x, x[i].z, 0x5410), __byte_perm(x[i].x, x[i].z, 0x7632),
                                          __byte_perm(x[i].y, x[i].w, 0x5410), __byte_perm(x[i].y, x[i].w, 0x7632));
                    sts16(base + C::kOffQ + (r / kRowsTile) * C::kTileBytes + tile_off(r % kRowsTile, c), x[i].x, x[i].y, x[i].z, x[i].w);
                }
            }
            if (tid < t.tiles * kRowsTile) {
                const int tok = (t.row0 + min(tid, t.rows - 1)) / a.group;
                sh.tok[tid / kRowsTile][tid % kRowsTile] = tok;
                sh.word[tid / kRowsTile][tid % kRowsTile] = a.mask != nullptr ? a.mask[t.s.first + tok] : 0;
            }
            fence_async_shared();
            named_bar_sync(kBarQueries, kSoftWarps * 32);

            // Softmax.  A slot's eight warps are its tile's four quarters of rows times
            // two halves of a block's keys.  S, W and O are held in fragments: rows 8 k +
            // lane / 4 of the warp's 32 (k < 4), columns 2 (lane % 4), + 1 of every 8.  A
            // thread so needs the scales of a quarter of its keys: read for whole rows
            // they took half of the shared-memory bandwidth, of which the product of Q
            // and K leaves nothing (LDS 34 cycles instead of 4).
            const int slot = warp / kSlotWarps, half = (warp >> 2) & 1, quad = warp & 3;
            const bool first = warp % kSlotWarps == 0;            // issues the slot's products
            const int tl = two ? slot : 0;
            const int tile_rows = two ? min(kRowsTile, t.rows - slot * kRowsTile) : t.rows;
            const int u0 = t.u0, start = t.s.start;
            const bool idle = 32 * quad >= tile_rows;             // the whole warp has no row
            const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
            const uint32_t ts = lanes + C::kS + 128 * slot + 64 * half;  // S of its keys; W goes over its first half
            const uint32_t to = lanes + C::kO + DIM * slot + (DIM / 2) * half;
            constexpr uint32_t kHalfLanes = 16u << 16;
            float M[4], l[4];
            #pragma unroll
            for (int k = 0; k < 4; ++k) M[k] = -INFINITY, l[k] = 0.f;
            const int my_jobs = two ? nb : (nb + 1 - slot) / 2;
            const int u_q = __shfl_sync(0xFFFFFFFFu, tl, 0);
            auto block_of = [&](int i) -> int { return blocks_done + (two ? i : 2 * i + slot); };
            // products, issued by the slot's first warp (all of it in step, so that
            // descriptors live in uniform registers; one lane issues)
            auto qk = [&](int i) {
                const uint64_t qd = sw128_desc(u_base + C::kOffQ) + u_q * (C::kTileBytes >> 4);
                const uint64_t kd = sw128_desc(u_base + C::kOffK) + (block_of(i) & 1) * (C::kTileBytes >> 4);
                if (leader) {
                    #pragma unroll
                    for (int k = 0; k < KSTEPS; ++k) {
                        const uint64_t off = ((k >> 2) * C::kHalf + (k & 3) * 32) >> 4;
                        tc_mma_f16(u_tmem + C::kS + 128 * slot, qd + off, kd + off, f16_idesc(kRowsTile, kBlock), k > 0);
                    }
                }
            };
            auto pv = [&](int i) {
                const uint64_t vd = sw128_desc_mn(u_base + C::kOffV, C::kHalf) + block_of(i) % C::kValueTiles * (C::kTileBytes >> 4);
                if (leader) {
                    #pragma unroll
                    for (int k = 0; k < kBlock / 16; ++k)
                        tc_mma_f16_tmem_a(u_tmem + C::kO + DIM * slot, u_tmem + C::kS + 128 * slot + 64 * (k >> 2) + 8 * (k & 3),
                                          vd + k * (2048 >> 4), f16_idesc(kRowsTile, DIM) | kIdescTransposeB, i > 0 || k > 0);
                }
            };
            // a stage is free when both slots have used it; of one tile, its one user
            // arrives for both
            auto release = [&](uint64_t* bars, int i) {
                if (leader) {
                    tc_commit(smem_u32(&bars[block_of(i) & 1]));
                    if (!two) tc_commit(smem_u32(&bars[block_of(i) & 1]));
                }
            };
            auto commit = [&]() {
                if (leader) tc_commit(smem_u32(&sh.sfull[slot]));
            };
            auto wait = [&](uint64_t& bar, int phase) -> bool {
                return __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&bar), phase & 1, &sh.abort));
            };
            auto wait_keys = [&](int i) -> bool {
                const int blk = block_of(i);
                return wait(sh.kfull[blk & 1], blk >> 1);
            };
            // a wait that gave up (ok false) skips the work of what follows, but each
            // warp still votes and hands over once a job (kvq_roles.h)
            bool ok = true;
            if (first && my_jobs > 0) {
                ok = wait_keys(0);
                if (ok) {
                    tc_fence_after_sync();
                    qk(0);
                    commit();
                    release(sh.kfree, 0);
                    __syncwarp();
                }
            }
            for (int i = 0; i < my_jobs; ++i) {
                const int u = u0 + (two ? i : 2 * i + slot);
                const int blk = block_of(i);
                const BlockScales& bs = sh.sc[blk % kScaleRing];
                ok = ok && wait(sh.scfull[blk % kScaleRing], blk / kScaleRing);
                const int k0 = u * kBlock;
                float ve = 0.f;  // 2^ve bounds the value scales of a plain block
                bool plain = true;
                if (ok && !idle) {
                    const float4 v = reinterpret_cast<const float4*>(bs.vmax)[0], v2 = reinterpret_cast<const float4*>(bs.vmax)[1];
                    const uint4 odd = reinterpret_cast<const uint4*>(bs.odd)[0], odd2 = reinterpret_cast<const uint4*>(bs.odd)[1];
                    ve = log2_bound(__float_as_uint(fmaxf(max3(v.x, v.y, max3(v.z, v.w, v2.x)), max3(v2.y, v2.z, v2.w))));
                    plain = k0 + kBlock <= start && (odd.x | odd.y | odd.z | odd.w | odd2.x | odd2.y | odd2.z | odd2.w) == 0u;
                }
                ok = ok && wait(sh.sfull[slot], s_phase[slot] + i);
                const bool work = ok && !idle;
                const float* kf = bs.k + 64 * half + 2 * (lane & 3);  // scales of this thread's keys, 8 apart
                const float* vf = bs.v + 64 * half + 2 * (lane & 3);
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                bool up = false;
                if (work) {
                    tc_fence_after_sync();
                    // the maxima of this thread's keys, rows k
                    if (plain) {
                        #pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int c = e >> 1, hb = e & 1;
                            uint32_t s[16];
                            tmem_ld_frag32(ts + 32 * c + hb * kHalfLanes, s);
                            tmem_ld_wait();
                            #pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint64_t kk = *reinterpret_cast<const uint64_t*>(kf + 32 * c + 8 * j);
                                #pragma unroll
                                for (int rr = 0; rr < 2; ++rr) {
                                    const float2 d = unpack2(mul2(pack2(__uint_as_float(s[4 * j + 2 * rr]), __uint_as_float(s[4 * j + 2 * rr + 1])), kk));
                                    top[2 * hb + rr] = max3(top[2 * hb + rr], d.x, d.y);
                                }
                            }
                        }
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) top[k] += ve;
                    } else {
                        const int r = 32 * quad + (lane >> 2);
                        const float4 m = score_masked(ts, &bs, sh.word[tl] + r, sh.tok[tl] + r, k0 + 64 * half - start, half, a.mask != nullptr);
                        top[0] = m.x, top[1] = m.y, top[2] = m.z, top[3] = m.w;
                    }
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) up |= top[k] - M[k] > kTop + kSlack;
                }
                // raise the references that are too low: both halves of the keys alike
                if (named_bar_or(bar_vote(slot), kSlotWarps * 32, up)) {
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], 1));
                        top[k] = fmaxf(top[k], __shfl_xor_sync(0xFFFFFFFFu, top[k], 2));
                        if ((lane & 3) == 0) sh.top[slot][half][32 * quad + 8 * k + (lane >> 2)] = top[k];
                    }
                    named_bar_sync(bar_vote(slot), kSlotWarps * 32);
                    if (work) {
                        float f[4];
                        #pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float m = fmaxf(top[k], sh.top[slot][half ^ 1][32 * quad + 8 * k + (lane >> 2)]);
                            const bool raise = m - M[k] > kTop + kSlack;
                            const float Mn = raise ? m - kTop : M[k];
                            f[k] = !raise ? 1.f : M[k] == -INFINITY ? 0.f : exp2_fast(M[k] - Mn);
                            M[k] = Mn;
                            l[k] *= f[k];
                        }
                        if (i > 0) {  // O is settled: this S was issued after the last product into it
                            #pragma unroll 1
                            for (int e = 0; e < DIM / 32; ++e) {
                                const uint32_t at = to + 32 * (e >> 1) + (e & 1) * kHalfLanes;
                                const float f0 = e & 1 ? f[2] : f[0], f1 = e & 1 ? f[3] : f[1];
                                uint32_t o[16];
                                tmem_ld_frag32(at, o);
                                tmem_ld_wait();
                                #pragma unroll
                                for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * (x & 2 ? f1 : f0));
                                tmem_st_frag32(at, o);
                            }
                            tmem_st_wait();
                        }
                    }
                }
                if (work) {
                    // weights: sums in fp32, W rounded to binary16 over S
                    uint64_t sum[4] = {0, 0, 0, 0}, nm[4];
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float x = M[k] == -INFINITY ? 0.f : -M[k];  // nothing seen yet: S is -inf throughout
                        nm[k] = pack2(x, x);
                    }
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = e >> 1, hb = e & 1;
                        uint32_t s[16], w[8];
                        tmem_ld_frag32(ts + 32 * c + hb * kHalfLanes, s);
                        tmem_ld_wait();
                        #pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint64_t kk = *reinterpret_cast<const uint64_t*>(kf + 32 * c + 8 * j);
                            const uint64_t vv = *reinterpret_cast<const uint64_t*>(vf + 32 * c + 8 * j);
                            #pragma unroll
                            for (int rr = 0; rr < 2; ++rr) {
                                const int k = 2 * hb + rr;
                                const float2 d = unpack2(fma2(pack2(__uint_as_float(s[4 * j + 2 * rr]), __uint_as_float(s[4 * j + 2 * rr + 1])), kk, nm[k]));
                                const uint64_t x = pack2(exp2_fast(d.x), exp2_fast(d.y));
                                sum[k] = add2(sum[k], x);
                                const float2 y = unpack2(mul2(x, vv));
                                w[2 * j + rr] = pack_half2(y.x, y.y);
                            }
                        }
                        tmem_st_pairs16(ts + 16 * c + hb * kHalfLanes, w);
                    }
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 f = unpack2(sum[k]);
                        l[k] += f.x + f.y;
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                }
                __syncwarp();
                if (first) {
                    // of two tiles the next keys do not depend on this product (of one,
                    // its other slot's values do, and they come in before those keys)
                    const bool more = i + 1 < my_jobs;
                    ok = ok && wait(sh.vfull[blk & 1], blk >> 1) && (!two || !more || wait_keys(i + 1));
                    named_bar_sync(bar_hand(slot), kSlotWarps * 32);
                    if (ok) {
                        tc_fence_after_sync();
                        pv(i);
                        release(sh.vfree, i);
                        if (more && (two || (ok = wait_keys(i + 1)))) {
                            tc_fence_after_sync();
                            qk(i + 1);
                            release(sh.kfree, i + 1);
                        }
                        commit();
                        __syncwarp();
                    }
                } else {
                    named_bar_arrive(bar_hand(slot), kSlotWarps * 32);
                }
            }
            // settled: the slot's last product, and what its rows' sums are relative to
            if (my_jobs > 0) ok = ok && wait(sh.sfull[slot], s_phase[slot] + my_jobs);
            #pragma unroll
            for (int k = 0; k < 4; ++k) {
                l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 1);
                l[k] += __shfl_xor_sync(0xFFFFFFFFu, l[k], 2);
                if ((lane & 3) == 0) {
                    sh.ref[slot][32 * quad + 8 * k + (lane >> 2)] = M[k];
                    sh.sum[slot][half][32 * quad + 8 * k + (lane >> 2)] = l[k];
                }
            }
        }
        blocks_done += nb;
        for (int i = 0; i < 2; ++i) {
            const int n = two ? nb : (nb + 1 - i) / 2;
            s_phase[i] += n > 0 ? n + 1 : 0;  // the first S, and one after each job
        }

        tc_fence_before_sync();
        __syncthreads();  // roles done: operands, TMEM and statistics are settled
        tc_fence_after_sync();
        if (sh.abort) break;
        if (warp == kSoftWarps && lane == 0 && t.u0 == 0 && t.u1 < t.units)
            *join_record<DIM, BITS>(a, blockIdx.x) = {(int)(sh.walk.last_cta(t) - blockIdx.x) + 1, t.rows, t.row0, t.s.first, t.h};
        // the tile's sums go out, normalized, or to this CTA's piece: a thread per
        // row (TMEM lane); the warps that hold a row share its dimensions (of one
        // tile's two slots each has a part of both)
        if (warp < kSoftWarps) {
            const int slot = warp / kSlotWarps, half = (warp >> 2) & 1, r = 32 * (warp & 3) + lane;
            const int tile_rows = two ? min(kRowsTile, t.rows - slot * kRowsTile) : t.rows;
            if (32 * (warp & 3) < tile_rows) {
                const int tl = two ? slot : 0;
                const bool whole = t.u0 == 0 && t.u1 == t.units;
                float m = sh.ref[tl][r], sum = sh.sum[tl][0][r] + sh.sum[tl][1][r], f0 = 1.f, f1 = 0.f;
                if (!two) {
                    const float m0 = m, m1 = sh.ref[1][r], l1 = sh.sum[1][0][r] + sh.sum[1][1][r];
                    m = fmaxf(m0, m1);
                    f0 = m0 == -INFINITY ? 0.f : exp2_fast(m0 - m);  // a slot of which nothing is seen: its sums are 0 or not written
                    f1 = m1 == -INFINITY ? 0.f : exp2_fast(m1 - m);
                    sum = sum * (m0 == -INFINITY ? 1.f : f0) + l1 * (m1 == -INFINITY ? 1.f : f1);
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const int row = t.row0 + tl * kRowsTile + min(r, tile_rows - 1);
                __half* out = a.out + ((int64_t)(t.s.first + row / a.group) * a.heads_q + t.h * a.group + row % a.group) * DIM;
                float* piece = a.parts + (((int64_t)blockIdx.x * 2 + (t.u0 == 0 ? 1 : 0)) * 2 + tl) * C::kPiece;
                const uint32_t to = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::kO;
                const int share = two ? DIM / 32 : DIM / 64;  // columns, by 16
                const int c0 = (two ? half : 2 * slot + half) * share;
                #pragma unroll 1
                for (int c = c0; c < c0 + share; ++c) {
                    uint32_t o[16];
                    tmem_ld16(to + (two ? DIM * slot : 0) + 16 * c, o);
                    if (!two && nb > 1) {
                        uint32_t x[16];
                        tmem_ld16(to + DIM + 16 * c, x);
                        tmem_ld_wait();
                        #pragma unroll
                        for (int y = 0; y < 16; ++y)
                            o[y] = __float_as_uint(fmaf(__uint_as_float(x[y]), f1, __uint_as_float(o[y]) * f0));
                    } else {
                        tmem_ld_wait();
                        #pragma unroll
                        for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f0);
                    }
                    if (whole) {
                        #pragma unroll
                        for (int x = 0; x < 16; x += 8) {
                            float f[8];
                            #pragma unroll
                            for (int y = 0; y < 8; ++y) f[y] = __uint_as_float(o[x + column_of<BITS>(y)]) * inv;
                            if (r < tile_rows) store8(out + 16 * c + x, f);
                        }
                    } else {
                        #pragma unroll
                        for (int x = 0; x < 16; ++x) piece[(16 * c + x) * kRowsTile + r] = __uint_as_float(o[x]);
                    }
                }
                if (!whole && half == 0 && (two || slot == 0)) {
                    piece[DIM * kRowsTile + r] = m;
                    piece[(DIM + 1) * kRowsTile + r] = sum;
                }
            }
            tc_fence_before_sync();
        }
        __syncthreads();  // the tile and TMEM have been read
        tc_fence_after_sync();
    }
    // the tensor core is idle before its memory is given back
    if (warp == 0 || warp == kSlotWarps) {
        if (leader) {
            tc_commit(smem_u32(&sh.drain[warp / kSlotWarps]));
            if (!mbar_wait(smem_u32(&sh.drain[warp / kSlotWarps]), 0)) atomicOr(&g_attn_error, kErrDrainWait);
        }
        __syncwarp();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == kSoftWarps) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kCols);
    }
}

// Joins the pieces of the row block that began in the run of CTA blockIdx.x and
// went on in the next ones, in their order: 16 dimensions of one tile a CTA, a
// thread has a row's eight and takes four pieces at a time (40 loads under
// way; one after the other they took up to 100 us).  As its own launch it
// has the whole GPU for what the last CTA to arrive would read alone.  (Its CTAs read
// what to join from a record: finding it again in the batch
// took most of their time: a call of 4 trees of 64 185.4 -> 178.5 us, 6 of 9 69.5 -> 65.1.)
constexpr int kJoinThreads = 256;
template <int DIM, int BITS>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const AttnArgs a) {
    using C = TreeCfg<DIM, BITS>;
    griddep_launch_dependents();
    griddep_wait();
    const int64_t c0 = blockIdx.x;
    const JoinRecord t = *join_record<DIM, BITS>(a, blockIdx.x);
    const int n = t.pieces;
    const int tl = blockIdx.y / (DIM / 16), r = threadIdx.x % kRowsTile, rt = tl * kRowsTile + r;
    const int c8 = blockIdx.y % (DIM / 16) * 2 + threadIdx.x / kRowsTile;
    if (n == 1 || rt >= t.rows) return;
    // the first CTA's piece is its second (of a block that it began), the others' their first
    auto piece = [&](int i) -> const float* {
        return a.parts + ((c0 + i) * 4 + (i == 0 ? 2 : 0) + tl) * C::kPiece + r;
    };
    float top = -INFINITY, sum = 0.f, o[8] = {};
    for (int i0 = 0; i0 < n; i0 += 4) {
        float m[4], l[4], x[4][8];
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* p = piece(min(i0 + i, n - 1));
            m[i] = p[DIM * kRowsTile];
            l[i] = p[(DIM + 1) * kRowsTile];
            #pragma unroll
            for (int y = 0; y < 8; ++y) x[i][y] = p[(8 * c8 + column_of<BITS>(y)) * kRowsTile];
        }
        const float was = top;
        #pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, m[i]);
        const float f = was == -INFINITY ? 0.f : exp2_fast(was - top);
        // (nothing seen so far: sums of 0, or NaN, which stays)
        sum = was == -INFINITY ? sum : sum * f;
        #pragma unroll
        for (int y = 0; y < 8; ++y) o[y] *= f;
        #pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i0 + i < n) {
                const float g = m[i] == -INFINITY ? 1.f : exp2_fast(m[i] - top);
                sum = fmaf(l[i], g, sum);
                #pragma unroll
                for (int y = 0; y < 8; ++y) o[y] = fmaf(x[i][y], g, o[y]);
            }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    #pragma unroll
    for (int y = 0; y < 8; ++y) o[y] *= inv;
    const int row = t.row0 + rt;
    store8(a.out + ((int64_t)(t.first + row / a.group) * a.heads_q + t.h * a.group + row % a.group) * DIM + 8 * c8, o);
}

template <typename F>
auto by_config(const kvq_cache_t& c, F f) {
    auto bits = [&](auto dim) {
        return c.bits == 8 ? f(dim, std::integral_constant<int, 8>()) : f(dim, std::integral_constant<int, 4>());
    };
    return c.dim == 64 ? bits(std::integral_constant<int, 64>()) : bits(std::integral_constant<int, 128>());
}

int tree_ctas(int sms) { return sms < kAttnMaxCtas ? sms : kAttnMaxCtas; }

// Whether this kernel serves a call: where it saves more than 22 us by the difference of
// what a cached token costs the two.  Measured on GB300 (8 sequences of 4 heads,
// 8192 to 32000 tokens, ps per token and cache head), at 128 dimensions: the row-block
// kernel 40 to 43 for each 16 rows, this one 88 to 94 for one tile of 128 rows and 152 to 161 for
// two, 4 and 8 bits alike; at 64 dimensions 26 to 28, and 70 to 78 and 133 to 139: nearly the same
// ratios.  At 64 tokens and up to 128 rows this one takes 10 to 19 us longer (20 to 29 us against
// 6 to 15).  22 us is high for a table as long as the sequences (over 672 calls of 8 to 448 rows and 64 to 32000
// tokens the rule takes 1.03 of the better kernel's time on average, at most 1.83;
// with 5 us 1.02, at most 1.46), but the cache is taken to be as long as the page table
// allows, as its length is on the device, and a captured step has a table for the longest.
bool tree_serves(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q) {
    if (c.dim > 128) return false;  // two tiles' O of 256 dimensions do not fit TMEM; there is no form for one
    const int64_t rows = (b.tokens * (heads_q / c.heads) + b.seqs - 1) / b.seqs, tiles = (rows + 127) / 128;
    const double here = (double)(tiles / 2) * 146e-6 + (double)(tiles % 2) * 86e-6, there = (double)((rows + 15) / 16) * 38e-6;
    const double keys = (double)b.seqs * c.heads * (double)(b.max_pages * c.page);
    return keys * (there - here) > 22.0;
}

}  // namespace

size_t kvq_attn_workspace(const kvq_cache_t& c, const kvq_batch_t& b, int heads_q, int sms) {
    if (!tree_serves(c, b, heads_q)) return attn_rows_workspace(c, b, heads_q, sms);
    return by_config(c, [&](auto dim, auto bits) -> size_t {
        return kAttnTicketBytes +
               tree_ctas(sms) * (4 * TreeCfg<decltype(dim)::value, decltype(bits)::value>::kPiece * sizeof(float) + sizeof(JoinRecord));
    });
}

cudaError_t launch_kvq_attention(const kvq_cache_t& c, const kvq_batch_t& b, const uint16_t* Q, int heads_q,
                                 const uint64_t* mask, float scale, uint16_t* out, void* ws, int sms, unsigned flags,
                                 cudaStream_t stream) {
    if (!tree_serves(c, b, heads_q)) return launch_attn_rows(c, b, Q, heads_q, mask, scale, out, ws, sms, flags, stream);
    const AttnArgs a = {cache_arg(c), batch_arg(b), reinterpret_cast<const __half*>(Q), mask,
                        reinterpret_cast<__half*>(out), heads_q, heads_q / c.heads, scale * 1.4426950408889634f,
                        static_cast<unsigned*>(ws),
                        reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kAttnTicketBytes)};
    return by_config(c, [&](auto dim, auto bits) {
        constexpr int D = decltype(dim)::value, B = decltype(bits)::value;
        static std::atomic<uint64_t> ready{0};
        cudaError_t e = layer_smem(tree_kernel<D, B>, TreeCfg<D, B>::kSmem, ready);
        if (e != cudaSuccess) return e;
        const unsigned ctas = (unsigned)tree_ctas(sms);
        e = layer_launch(tree_kernel<D, B>, dim3(ctas), kTreeThreads, TreeCfg<D, B>::kSmem, flags, stream, a);
        if (e != cudaSuccess) return e;
        return layer_launch(tree_join_kernel<D, B>, dim3(ctas, 2 * D / 16), kJoinThreads, 0, W4A8_LAUNCH_PDL, stream, a);
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
    return e == cudaSuccess ? read_and_clear_attn_rows_error(flags, stream) : e;
}

}  // namespace w4a8
