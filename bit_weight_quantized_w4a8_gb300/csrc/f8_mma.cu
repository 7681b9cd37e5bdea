// f8_mma.cu -- the product of e4m3 codes with a scale for each block of 128
// values of K, on tcgen05.
//
//   Y[m][n] = sum_kb (sa[kb][m] * sw[n / 128][kb]) * sum_{k in kb} xq[m][k] wq[n][k]
//
// One block of K is one 128-byte row of both operands: a TMA box in the 128-byte
// swizzle, four MMAs of K = 32.  The sums of a block are complete in TMEM; the
// consumer warps read them, scale them and add them to fp32 sums in registers while
// the tensor core fills the other half of TMEM with the next block.  The
// registers hold a tile's sums until its last block, so TMEM belongs to the next tile
// while a tile is written.
//
// Two kernels (figures: launches one after another in a graph, weights not in L2):
//  wide    256 rows of X x 256 (or 128: half_tiles) of W by a pair of CTAs, 128 rows of X and half of
//          W's in the shared memory of each: a thread has one row of X and half of the columns, so one
//          scale a block.  For many rows: 8192 x 3584 x 18944 473 us (2.35 PFLOP/s), 777 x 4096 x
//          4608 21.  A block takes about 1000 cycles; its four MMAs alone take 690 (512 at the nominal
//          rate).  The rest is the sums' way out of TMEM (128 x 128 a warp group, 32 columns at a
//          time): two buffers of 256 columns are all it has, so the products wait for it.  Tiles of 160
//          columns with three buffers took 554 us, halves of 128 494, 16 consumer warps 478.
//  narrow  128 rows of W x 16 .. 128 of X: the weights fill the tensor core's 128 rows
//          whatever the batch, K is cut over a cluster whose sums are joined through
//          distributed shared memory in the order of the pieces.  For few rows: 1 x 3584 x 18944
//          15.1 us (10.1 at the copy rate), 49 x 18944 x 3584 19, 1 x 3584 x 152064 87 (81): launch,
//          the first bytes' way and the join are 4 to 5 us, the rest streams.
//  goes_wide chooses between them.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <mutex>
#include <type_traits>

#include "f8.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace w4a8 {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_f8_error;

constexpr int kProducerThreads = 128;  // warp 0 copies, warp 1 issues the MMAs
constexpr int kRows = 128;             // TMEM lanes: rows of operand A
constexpr int kKBytes = 128;           // a block of K
constexpr int kABytes = kRows * kKBytes;

struct F8Args {
    CUtensorMap tm_a, tm_b;
    const float *sa, *sw;
    void* Y;
    int64_t N;
    int M, kbs, tiles_a, tiles;
    const void* X;  // values of X, where the product makes the codes itself
    int K;
};

// (Of a kernel launched dependently, warps that do not wait for the one before may wait here for those that do:
// its time does not count.)
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
    #pragma unroll 1
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    unsigned long long t0 = globaltimer_ns();
    bool alone = false;
    for (;;) {
        #pragma unroll 1
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            if (!alone) {
                griddep_wait();
                alone = true, t0 = globaltimer_ns();
                continue;
            }
            *abort_flag = 1;
            atomicOr(&g_f8_error, kErrFullWait);
            return false;
        }
    }
}
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    if (!mbar_wait(bar, parity)) atomicOr(&g_f8_error, kErrDrainWait);
}

// 32 columns of the warp's 32 lanes; the values are there after tmem_ld32_wait,
// which names them so that nothing that uses them moves in front of it.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(uint32_t (&v)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
                 :
                 : "memory");
}
// What a CTA's warps share besides the operands.
template <int S, int D>
struct Bars {
    uint64_t full[S], empty[S], d_full[D], d_empty[D];
    uint32_t tmem;
    int abort;
};

// A place in a ring of N and the parity of the pass over it.
template <int N>
struct Ring {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++at == N) at = 0, phase ^= 1;
    }
};

// One block of K: four MMAs of 32 bytes.
__device__ __forceinline__ void issue_block(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    const uint64_t ad = sw128_desc(a), bd = sw128_desc(b);
    #pragma unroll
    for (int k = 0; k < kKBytes / 32; ++k) tc_mma_e4m3(d, ad + 2 * k, bd + 2 * k, idesc, k > 0);
}

// ---------------------------------------------------------------------------
// wide
// ---------------------------------------------------------------------------

constexpr int kWideWarps = 8;  // consumers: warp w has lanes 32 (w % 4) .., half w / 4 of the columns
constexpr int kWideThreads = kProducerThreads + 32 * kWideWarps;
constexpr int kWideOut = 32 * 64;  // a warp's outputs on their way: 32 rows of 16 columns
constexpr int kWideAhead = 4;      // blocks whose scales of X a warp has or has asked for
constexpr int kWideSa = kWideAhead * 32 * 4;

template <int COLS>
struct Wide {
    static constexpr int kBufs = 512 / COLS;  // of COLS columns in TMEM
    static constexpr int kStages = COLS == 256 ? 5 : 8;
    static constexpr int kWarpCols = COLS / 2;
    static constexpr int kStage = kABytes + COLS / 2 * kKBytes;  // of one CTA
    static constexpr int kSmem = kStages * kStage + kWideWarps * (kWideOut + kWideSa) + 1024;
    static_assert(kStage % 1024 == 0 && kSmem <= 227 * 1024, "operands on 1024 bytes, one CTA's shared memory");
};

// A warp's buffer of 32 rows of 16 outputs in 16-byte chunks, swapped about so that
// 8 lanes with 8 rows, or with all chunks of a few, meet all banks.
template <typename TY>
__device__ __forceinline__ uint4* out_chunk(uint8_t* buf, int r, int c) {
    constexpr int CH = sizeof(TY);  // chunks a row
    return reinterpret_cast<uint4*>(buf + (r * CH + (c ^ (r / (8 / CH) & (CH - 1)))) * 16);
}

// The warp's rows m0 + 0..31, columns n0 + 0..15, through the buffer.
template <typename TY>
__device__ __forceinline__ void store_cols16(uint8_t* buf, const float* x, TY* Y, int m0, int M, int64_t n0, int64_t N,
                                             bool vec) {
    constexpr int CH = sizeof(TY), PER = 16 / sizeof(TY);
    const int lane = threadIdx.x % 32;
    #pragma unroll
    for (int u = 0; u < CH; ++u) {
        if constexpr (sizeof(TY) == 4) {
            *out_chunk<TY>(buf, lane, u) = make_uint4(__float_as_uint(x[4 * u]), __float_as_uint(x[4 * u + 1]),
                                                      __float_as_uint(x[4 * u + 2]), __float_as_uint(x[4 * u + 3]));
        } else {
            *out_chunk<TY>(buf, lane, u) = make_uint4(pack_half2(x[8 * u], x[8 * u + 1]), pack_half2(x[8 * u + 2], x[8 * u + 3]),
                                                      pack_half2(x[8 * u + 4], x[8 * u + 5]), pack_half2(x[8 * u + 6], x[8 * u + 7]));
        }
    }
    __syncwarp();
    const int c = lane % CH;
    const int64_t n = n0 + c * PER;
    #pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int r = 32 / CH * i + lane / CH;
        const uint4 v = *out_chunk<TY>(buf, r, c);
        if (m0 + r >= M || n >= N) continue;
        TY* y = Y + (int64_t)(m0 + r) * N + n;
        if (vec && n + PER <= N) {
            *reinterpret_cast<uint4*>(y) = v;
        } else {
            const TY* e = reinterpret_cast<const TY*>(&v);
            #pragma unroll
            for (int k = 0; k < PER; ++k)
                if (n + k < N) y[k] = e[k];
        }
    }
    __syncwarp();
}

template <int COLS, typename TY>
__global__ void __launch_bounds__(kWideThreads, 1) f8_wide_kernel(const __grid_constant__ F8Args a) {
    // of the pair's barriers, full and d_empty count in the even CTA, which issues
    // the MMAs; empty and d_full are told to both
    using C = Wide<COLS>;
    constexpr int kWarpCols = C::kWarpCols;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<C::kStages, C::kBufs> sh;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank();
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            mbar_init(smem_u32(&sh.d_full[i]), 1);
            mbar_init(smem_u32(&sh.d_empty[i]), 2 * kWideWarps);
        }
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc_pair(smem_u32(&sh.tmem), 512);
    tc_fence_before_sync();
    cl.sync();
    tc_fence_after_sync();
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t tmem = sh.tmem;
    const int first = blockIdx.x / 2, pairs = gridDim.x / 2;
    const int steps = ((a.tiles - 1 - first) / pairs + 1) * a.kbs;  // blocks of all tiles
    int issued = 0;

    if (warp == 0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        // (whole warps go along in both loops, so that descriptors and addresses are
        // uniform: one lane on its own took 100 cycles for each MMA or copy)
        const uint64_t keep = l2_evict_last_policy();
        const uint32_t full0 = cluster_addr(smem_u32(&sh.full[0]), 0);
        int kb = 0, tile = first;
        Ring<C::kStages> st;
        for (int i = 0; i < steps; ++i, st.next()) {
            if (i >= C::kStages &&
                !__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.empty[st.at]), st.phase ^ 1, &sh.abort)))
                break;
            if (elect_one()) {
                const uint32_t at = sbase + st.at * C::kStage, bar = full0 + 8 * st.at;
                if (rank == 0) mbar_arrive_expect_tx(smem_u32(&sh.full[st.at]), 2 * C::kStage);
                tma_load_2d_pair(at, &a.tm_a, kb * kKBytes, (tile % a.tiles_a * 2 + rank) * kRows, bar, keep);
                tma_load_2d_pair(at + kABytes, &a.tm_b, kb * kKBytes, (tile / a.tiles_a * 2 + rank) * (COLS / 2), bar, keep);
            }
            issued = i + 1;
            if (++kb == a.kbs) kb = 0, tile += pairs;
        }
        // nothing may come to this CTA after it has gone: copies (all have landed when
        // their stage is told to be empty; both CTAs' count in the even one) and what is told to it
        for (int i = max(0, issued - C::kStages); lane == 0 && i < issued; ++i) {
            if (!*(volatile int*)&sh.abort)
                drain(smem_u32(&sh.empty[i % C::kStages]), (i / C::kStages) & 1);
            else if (rank == 0)
                drain(smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (rank == 0) {
            const uint32_t idesc = e4m3_idesc(2 * kRows, COLS);
            Ring<C::kStages> st;
            Ring<C::kBufs> d;
            for (int i = 0; i < steps; ++i, st.next(), d.next()) {
                if (i >= C::kBufs &&
                    !__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.d_empty[d.at]), d.phase ^ 1, &sh.abort)))
                    break;
                if (!__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.full[st.at]), st.phase, &sh.abort))) break;
                tc_fence_after_sync();
                if (elect_one()) {
                    const uint32_t at = sbase + st.at * C::kStage;
                    const uint64_t ad = sw128_desc(at), bd = sw128_desc(at + kABytes);
                    #pragma unroll
                    for (int k = 0; k < kKBytes / 32; ++k)
                        tc_mma_e4m3_pair(tmem + COLS * d.at, ad + 2 * k, bd + 2 * k, idesc, k > 0);
                    tc_commit_pair(smem_u32(&sh.d_full[d.at]));
                    tc_commit_pair(smem_u32(&sh.empty[st.at]));
                }
                issued = i + 1;
            }
            // every MMA is done before TMEM is given back
            if (issued > 0 && lane == 0)
                drain(smem_u32(&sh.d_full[(issued - 1) % C::kBufs]), ((issued - 1) / C::kBufs) & 1);
            __syncwarp();
        }
    } else if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int cw = warp - 4, q = warp % 4, g = cw / 4;
        uint8_t* buf = smem + C::kStages * C::kStage + cw * kWideOut;
        const bool vec = a.N % (16 / sizeof(TY)) == 0 && reinterpret_cast<uintptr_t>(a.Y) % 16 == 0;
        const int64_t nbs = (a.N + kF8Block - 1) / kF8Block;
        const uint32_t d_empty = cluster_addr(smem_u32(&sh.d_empty[0]), 0);
        // The row's scales come by asynchronous copies, each lane's for itself, those of W
        // 32 blocks at a time, one a lane: loads into registers that far ahead all had to be
        // waited for with the nearest one.
        float* sa_ring = reinterpret_cast<float*>(smem + C::kStages * C::kStage + kWideWarps * kWideOut + cw * kWideSa) + lane;
        const float* ask_at = nullptr;
        int ask_tile = first, ask_left = 0, ask_i = 0;
        auto ask = [&]() {
            if (ask_left == 0 && ask_tile < a.tiles) {
                ask_at = a.sa + min((ask_tile % a.tiles_a * 2 + rank) * kRows + 32 * q + lane, a.M - 1);
                ask_left = a.kbs;
                ask_tile += pairs;
            }
            if (ask_left > 0) {
                cp_async_4(smem_u32(sa_ring + (ask_i & (kWideAhead - 1)) * 32), ask_at);
                ask_at += a.M;
                --ask_left;
            }
            cp_async_commit();
            ++ask_i;
        };
        for (int k = 0; k < kWideAhead - 1; ++k) ask();
        int i = 0;
        bool ok = true;
        Ring<C::kBufs> d;
        for (int tile = first; ok && tile < a.tiles; tile += pairs) {
            const int m0 = (tile % a.tiles_a * 2 + rank) * kRows + 32 * q;
            const int64_t n0 = (int64_t)(tile / a.tiles_a) * COLS + kWarpCols * g;
            const float* sw = a.sw + min(n0 / kF8Block, nbs - 1) * a.kbs;
            float acc[kWarpCols];
            #pragma unroll
            for (int j = 0; j < kWarpCols; ++j) acc[j] = 0.f;
            float sw32 = 0.f;
            for (int kb = 0; kb < a.kbs; ++kb, ++i, d.next()) {
                // (the scales belong in front of the wait: behind the loads from TMEM they
                // cost 10%, on the way from a block's sums to the release of their columns)
                if (kb % 32 == 0) sw32 = sw[min(kb + lane, a.kbs - 1)];
                cp_async_wait<kWideAhead - 2>();
                const float s = sa_ring[(i & (kWideAhead - 1)) * 32] * __shfl_sync(0xFFFFFFFFu, sw32, kb % 32);
                ask();
                ok = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.d_full[d.at]), d.phase, &sh.abort));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16) + COLS * d.at + kWarpCols * g;
                uint32_t v[2][32];
                tmem_ld32(lanes, v[0]);
                #pragma unroll
                for (int c = 0; c < kWarpCols / 32; ++c) {
                    tmem_ld32_wait(v[c & 1]);
                    if (c + 1 < kWarpCols / 32) {
                        tmem_ld32(lanes + 32 * (c + 1), v[(c + 1) & 1]);
                    } else {  // all of it is in registers
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_cluster(d_empty + 8 * d.at);
                    }
                    #pragma unroll
                    for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(__uint_as_float(v[c & 1][j]), s, acc[32 * c + j]);
                }
            }
            if (!ok) break;
            #pragma unroll
            for (int c = 0; c < kWarpCols / 16; ++c)
                store_cols16(buf, acc + 16 * c, static_cast<TY*>(a.Y), m0, a.M, n0 + 16 * c, a.N, vec);
        }
    }
    tc_fence_before_sync();
    cl.sync();  // neither CTA's shared memory or barriers are needed any more
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// narrow
// ---------------------------------------------------------------------------

constexpr int kNarrowThreads = kProducerThreads + 128;
constexpr int kNarrowCluster = 8;  // pieces of K, at most
constexpr int kNarrowAhead = 8;    // blocks whose scales have been asked for
constexpr int kOwnRows = 2;        // up to which the kernel makes X's codes itself

template <int BN>
struct Narrow {
    static constexpr int kStage = kABytes + BN * kKBytes;
    static constexpr int kCtas = BN <= 64 ? 2 : 1;  // per SM
    static constexpr int kStages = BN <= 64 ? (107 * 1024) / kStage : 6;
    static constexpr int kCols = BN < 32 ? 32 : 2 * BN;  // TMEM
    static constexpr int kSmem = kStages * kStage + 1024;
    static_assert(kStages * kStage >= BN * kRows * 4, "the sums have to fit");
};

// TX: type of X's values, of which warps 2 and 3 make the codes and scales where the tensor
// core and the consumers read them; void: codes and scales come from memory.
template <int BN, typename TY, typename TX>
__global__ void __launch_bounds__(kNarrowThreads, Narrow<BN>::kCtas) f8_narrow_kernel(const __grid_constant__ F8Args a) {
    using C = Narrow<BN>;
    constexpr bool kOwn = !std::is_void_v<TX>;
    // the values are at most kStages blocks in front of the MMAs, these two in front of the sums
    static_assert(!kOwn || (kOwnRows <= 2 && C::kStages + 2 <= kNarrowAhead), "a row half a warp; the ring of scales");
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<C::kStages, 2> sh;
    __shared__ __align__(16) float scale[2][BN];
    __shared__ float2 scale_ring[kNarrowAhead][BN];  // of X's rows and of W on their way
    __shared__ uint64_t scale_full[kOwn ? kNarrowAhead : 1];  // X's are there
    cg::cluster_group cl = cg::this_cluster();
    uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(smem_u32(&sh.full[i]), kOwn ? 2 : 1);
            mbar_init(smem_u32(&sh.empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.d_full[i]), 1);
            mbar_init(smem_u32(&sh.d_empty[i]), 4);
        }
        if constexpr (kOwn)
            for (int i = 0; i < kNarrowAhead; ++i) mbar_init(smem_u32(&scale_full[i]), 1);
        sh.abort = 0;
        fence_mbar_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(&sh.tmem), C::kCols);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    griddep_launch_dependents();
    const uint32_t tmem = sh.tmem;
    const int pieces = gridDim.x, p = blockIdx.x;  // cluster (pieces, 1, 1)
    const int kb0 = (int)((int64_t)a.kbs * p / pieces), steps = (int)((int64_t)a.kbs * (p + 1) / pieces) - kb0;
    const int64_t n0 = (int64_t)blockIdx.y * kRows;
    const int m0 = blockIdx.z * BN;
    int issued = 0;

    if (warp == 0) {
        const uint64_t once = l2_evict_first_policy(), keep = l2_evict_last_policy();
        auto load_w = [&](int i, int s) {
            if (!elect_one()) return;
            mbar_arrive_expect_tx(smem_u32(&sh.full[s]), kOwn ? kABytes : C::kStage);
            tma_load_2d_hint(sbase + s * C::kStage, &a.tm_a, (kb0 + i) * kKBytes, (int)n0, smem_u32(&sh.full[s]), once);
        };
        auto load_x = [&](int i, int s) {
            if (!kOwn && elect_one())
                tma_load_2d_hint(sbase + s * C::kStage + kABytes, &a.tm_b, (kb0 + i) * kKBytes, m0, smem_u32(&sh.full[s]), keep);
        };
        // the weights do not come from the kernel before
        const int ahead = min(steps, C::kStages);
        for (int i = 0; i < ahead; ++i) load_w(i, i);
        if constexpr (!kOwn) griddep_wait();
        for (int i = 0; i < ahead; ++i) load_x(i, i);
        issued = ahead;
        int s = 0;
        uint32_t phase = 0;
        for (int i = ahead; i < steps; ++i) {
            if (!__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.empty[s]), phase, &sh.abort))) break;
            load_w(i, s);
            load_x(i, s);
            issued = i + 1;
            if (++s == C::kStages) s = 0, phase ^= 1;
        }
        griddep_wait();  // (a full stage holds codes of X, which come behind the kernel before)
        for (int i = max(0, issued - C::kStages); lane == 0 && i < issued; ++i)
            drain(smem_u32(&sh.full[i % C::kStages]), (i / C::kStages) & 1);
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t idesc = e4m3_idesc(kRows, BN);
        int s = 0;
        uint32_t phase = 0;
        Ring<2> d;
        for (int i = 0; i < steps; ++i, d.next()) {
            if (i >= 2 && !__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.d_empty[d.at]), d.phase ^ 1, &sh.abort))) break;
            if (!__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.full[s]), phase, &sh.abort))) break;
            tc_fence_after_sync();
            if (elect_one()) {
                const uint32_t at = sbase + s * C::kStage;
                issue_block(tmem + BN * d.at, at, at + kABytes, idesc);
                tc_commit(smem_u32(&sh.d_full[d.at]));
                tc_commit(smem_u32(&sh.empty[s]));
            }
            issued = i + 1;
            if (++s == C::kStages) s = 0, phase ^= 1;
        }
        if (issued > 0 && lane == 0) drain(smem_u32(&sh.d_full[(issued - 1) & 1]), ((issued - 1) / 2) & 1);
        __syncwarp();
    } else if (warp < 4) {
        if constexpr (kOwn) {
            // one block the one warp, the next the other, sixteen lanes a row, values two blocks ahead
            // (both warps on each block: 17.7 us instead of 15.1 at 1 x 3584 x 18944, a block took as
            // long as its weights).  Rows from M on stay as they are: they only meet columns of the
            // sums that nobody writes.
            griddep_wait();
            const int l = lane % 16, r = lane / 16;
            const TX* x = static_cast<const TX*>(a.X) + (int64_t)min(r, a.M - 1) * a.K + kb0 * kF8Block + 8 * l;
            Eight<TX> now, next[2];
            auto load = [&](int i, Eight<TX>& v) {
                v = Eight<TX>();
                if (i < steps && (kb0 + i) * kF8Block + 8 * l < a.K) v.load(x + i * kF8Block);
            };
            load(warp - 2, next[0]);
            load(warp, next[1]);
            for (int i = warp - 2; i < steps; i += 2) {
                now = next[0], next[0] = next[1];
                load(i + 4, next[1]);
                const int s = i % C::kStages, round = i / C::kStages;
                float4 u, v;
                now.get(u, v);
                const float sx = f8_row_scale(u, v);
                float lo, hi;
                quant_bracket(sx, &lo, &hi);
                const uint2 codes = make_uint2(f8_codes4(u, sx, lo, hi), f8_codes4(v, sx, lo, hi));
                if (round > 0 && !__all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.empty[s]), (round & 1) ^ 1, &sh.abort))) break;
                if (r < a.M) {
                    // the 128-byte swizzle: 16-byte chunk c of row r lies at c ^ (r % 8)
                    *reinterpret_cast<uint2*>(smem + s * C::kStage + kABytes + r * kKBytes + ((l / 2) ^ r) * 16 + l % 2 * 8) = codes;
                    if (l == 0) scale_ring[i % kNarrowAhead][r].x = sx;
                }
                fence_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(smem_u32(&sh.full[s]));
                    mbar_arrive(smem_u32(&scale_full[i % kNarrowAhead]));
                }
            }
        }
    } else {
        griddep_wait();
        const int q = warp % 4, t = tid - kProducerThreads;  // t: the thread's column for scales, its lane for sums
        const uint32_t lanes = tmem + ((uint32_t)(32 * q) << 16);
        // Scales by asynchronous copies, each thread's of its column for itself, several
        // blocks ahead: loads into registers stalled every block for their latency.
        const float* sa = a.sa + (int64_t)kb0 * a.M + min(m0 + t, a.M - 1);
        const float* sw = a.sw + blockIdx.y * (int64_t)a.kbs + kb0;
        auto ask = [&](int i) {
            if (i < steps && t < BN) {
                const uint32_t at = smem_u32(&scale_ring[i % kNarrowAhead][t]);
                if constexpr (!kOwn) cp_async_4(at, sa + (int64_t)i * a.M);
                cp_async_4(at + 4, sw + i);
            }
            cp_async_commit();
        };
        for (int i = 0; i < kNarrowAhead - 1; ++i) ask(i);
        float acc[BN];
        #pragma unroll
        for (int j = 0; j < BN; ++j) acc[j] = 0.f;
        bool ok = true;
        Ring<2> d;
        for (int i = 0; i < steps; ++i, d.next()) {
            cp_async_wait<kNarrowAhead - 2>();
            if constexpr (kOwn)
                if (ok && t < 32)
                    ok = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&scale_full[i % kNarrowAhead]), i / kNarrowAhead & 1, &sh.abort));
            if (t < BN) {
                const float2 s = scale_ring[i % kNarrowAhead][t];
                scale[d.at][t] = s.x * s.y;
            }
            ask(i + kNarrowAhead - 1);
            named_bar_sync(1, 128);  // also: the block before the last has been read by all
            if (ok) ok = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&sh.d_full[d.at]), d.phase, &sh.abort));
            if (!ok) continue;  // (the others still meet at the barrier)
            tc_fence_after_sync();
            const uint32_t from = lanes + BN * d.at;
            auto add = [&](int j, const uint32_t* v, int n) {
                #pragma unroll
                for (int k = 0; k < n; k += 4) {
                    const float4 s = *reinterpret_cast<const float4*>(&scale[d.at][j + k]);
                    acc[j + k] = fmaf(__uint_as_float(v[k]), s.x, acc[j + k]);
                    acc[j + k + 1] = fmaf(__uint_as_float(v[k + 1]), s.y, acc[j + k + 1]);
                    acc[j + k + 2] = fmaf(__uint_as_float(v[k + 2]), s.z, acc[j + k + 2]);
                    acc[j + k + 3] = fmaf(__uint_as_float(v[k + 3]), s.w, acc[j + k + 3]);
                }
            };
            auto release = [&]() {
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sh.d_empty[d.at]));
            };
            if constexpr (BN == 16) {
                uint32_t v[16];
                tmem_ld16(from, v);
                tmem_ld16_wait(v);
                release();
                add(0, v, 16);
            } else {
                uint32_t v[BN > 32 ? 2 : 1][32];
                tmem_ld32(from, v[0]);
                #pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                    tmem_ld32_wait(v[c & (BN > 32)]);
                    if (c + 1 < BN / 32)
                        tmem_ld32(from + 32 * (c + 1), v[(c + 1) & (BN > 32)]);
                    else
                        release();
                    add(32 * c, v[c & (BN > 32)], 32);
                }
            }
        }
        const int64_t n = n0 + t;
        if (pieces == 1) {
            if (ok && n < a.N)
                #pragma unroll
                for (int j = 0; j < BN; ++j)
                    if (m0 + j < a.M) static_cast<TY*>(a.Y)[(int64_t)(m0 + j) * a.N + n] = (TY)acc[j];
        } else {
            // all copies have landed and all MMAs have read them (the last block's are done)
            float* sums = reinterpret_cast<float*>(smem);
            #pragma unroll
            for (int j = 0; j < BN; ++j)
                if (m0 + j < a.M) sums[j * kRows + t] = ok ? acc[j] : 0.f;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kCols);
    }
    if (pieces > 1) {
        cl.sync();
        // rows p, p + pieces, ... of the batch, a warp each, four columns a lane: the
        // pieces' sums in order
        const int rows = min(BN, a.M - m0);
        const int64_t n = n0 + 4 * lane;
        const bool vec = a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.Y) % (4 * sizeof(TY)) == 0;
        for (int j = p + pieces * warp; j < rows; j += pieces * (kNarrowThreads / 32)) {
            float4 y[kNarrowCluster];
            #pragma unroll
            for (int k = 0; k < kNarrowCluster; ++k)
                if (k < pieces) y[k] = load4(cl.map_shared_rank(reinterpret_cast<const float*>(smem), k) + j * kRows + 4 * lane);
            float4 sum = y[0];
            #pragma unroll
            for (int k = 1; k < kNarrowCluster; ++k)
                if (k < pieces) sum.x += y[k].x, sum.y += y[k].y, sum.z += y[k].z, sum.w += y[k].w;
            TY* to = static_cast<TY*>(a.Y) + (int64_t)(m0 + j) * a.N + n;
            if (vec && n < a.N) {  // then the four are inside
                store4(to, sum);
            } else {
                if (n < a.N) to[0] = (TY)sum.x;
                if (n + 1 < a.N) to[1] = (TY)sum.y;
                if (n + 2 < a.N) to[2] = (TY)sum.z;
                if (n + 3 < a.N) to[3] = (TY)sum.w;
            }
        }
        cl.sync();  // no CTA leaves while its sums may be read
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// Codes [rows][K] in boxes of one block of K and `box` rows; zeros past the ends.
bool code_map(CUtensorMap* map, const uint8_t* codes, int64_t rows, int64_t K, int box) {
    PFN_cuTensorMapEncodeTiled_v12000 fn = encode_fn();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)K};
    const cuuint32_t boxes[2] = {kKBytes, (cuuint32_t)box}, steps[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, boxes, steps,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename F>
cudaError_t cluster_launch(F* f, dim3 grid, int cluster, int threads, int smem, unsigned flags, cudaStream_t stream,
                           const F8Args& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)cluster, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = flags & 1u ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, a);
}

template <int COLS, typename TY>
cudaError_t launch_wide(F8Args& a, int64_t m_tiles, const uint8_t* Xf, int64_t K, const uint8_t* Wf, int sms, unsigned flags,
                        cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = layer_smem(f8_wide_kernel<COLS, TY>, Wide<COLS>::kSmem, ready);
    if (e != cudaSuccess) return e;
    a.tiles_a = (int)m_tiles;
    a.tiles = (int)(m_tiles * ((a.N + COLS - 1) / COLS));
    if (!code_map(&a.tm_a, Xf, a.M, K, kRows) || !code_map(&a.tm_b, Wf, a.N, K, COLS / 2)) return cudaErrorNotSupported;
    const int pairs = a.tiles < sms / 2 ? a.tiles : sms / 2;
    return cluster_launch(f8_wide_kernel<COLS, TY>, dim3((unsigned)(2 * pairs)), 2, kWideThreads, Wide<COLS>::kSmem, flags, stream, a);
}

// How many clusters of a size the GPU holds at once, with one CTA an SM: fewer than SMs / size, as a
// cluster stays within a group of SMs (46 of 3 and 15 of 7 on 152 SMs).
int max_clusters(int size) {
    constexpr int kDevices = 16;
    static std::atomic<uint64_t> ready{0};
    static std::atomic<int> known[kDevices][kNarrowCluster + 1];
    auto* f = f8_narrow_kernel<128, float, void>;
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || layer_smem(f, Narrow<128>::kSmem, ready) != cudaSuccess) return 0;
    if (dev < kDevices && (n = known[dev][size].load(std::memory_order_relaxed)) != 0) return n - 1;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {(unsigned)size, 1, 1};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kNarrowThreads);
    cfg.dynamicSmemBytes = Narrow<128>::kSmem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, f, &cfg) != cudaSuccess) {
        cudaGetLastError();  // (one piece then)
        return 0;
    }
    if (dev < kDevices) known[dev][size].store(n + 1, std::memory_order_relaxed);
    return n;
}

template <int BN, typename TY, typename TX = void>
cudaError_t launch_narrow(F8Args& a, unsigned flags, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    const cudaError_t e = layer_smem(f8_narrow_kernel<BN, TY, TX>, Narrow<BN>::kSmem, ready);
    if (e != cudaSuccess) return e;
    const int64_t tiles = a.tiles_a * (int64_t)((a.M + BN - 1) / BN);
    // Pieces of at least 4 blocks, as many as leave all clusters resident: 16 tiles in pieces of 7, counted by
    // SMs, took 21.2 us, of 6 15.0 (512 x 3584 x 512).  Two CTAs an SM up to 64 rows; one with
    // twice the stages and half the pieces was slower behind another call, whose CTAs then
    // leave no room to start in: 14.6 us a call instead of 13.5 at 1 x 3584 x 18944.
    int pieces = 1;
    for (int p = 2; p <= kNarrowCluster && a.kbs / p >= 4 && tiles <= Narrow<BN>::kCtas * (int64_t)max_clusters(p); ++p)
        pieces = p;
    const dim3 grid((unsigned)pieces, (unsigned)a.tiles_a, (unsigned)((a.M + BN - 1) / BN));
    return cluster_launch(f8_narrow_kernel<BN, TY, TX>, grid, pieces, kNarrowThreads, Narrow<BN>::kSmem, flags, stream, a);
}

// Where the narrow kernel makes X's codes itself: a launch less, 7.0 us instead of 7.9 at 1 x 3584 x
// 3584, 15.1 instead of 15.6 at 1 x 3584 x 18944 (2 rows the same; 4 rows 16.4 instead of 15.2 at
// 18944 x 3584, dependent launches).  Not where CTAs come in several waves, each with the values'
// way to go again: 88.7 us instead of 87.0 at 1 x 3584 x 152064.
bool makes_codes(int64_t M, int64_t N, int sms) { return M <= kOwnRows && (N + kRows - 1) / kRows <= 2 * (int64_t)sms; }
// More than 128 rows whose narrow tiles leave K in one piece go wide: 512 x 3584 x 3584 (112 tiles) 17.1 us
// there, 25.2 narrow, 384 x 18944 x 3584 (84) 53.9 and 82.6.  With two pieces the two are within 12% of each
// other: 256 x 18944 x 3584 (56) 53.9 and 47.8, 1500 x 3584 x 512 (48) 17.1 and 19.1; with more, narrow
// wins: 777 x 3584 x 512 (28) 17.1 and 15.0.  (Each call on its own, L2 flushed, fp16 out.)
bool goes_wide(int64_t M, int64_t N) {
    const int64_t n_tiles = (N + kRows - 1) / kRows;
    return n_tiles > 65535 || (M > 128 && n_tiles * ((M + kRows - 1) / kRows) > max_clusters(2));
}

// Tiles of 128 columns instead of 256 where the pairs of SMs go round as often: a block takes 0.77 of the
// time.  512 x 18944 x 3584 (one round) 70.3 -> 53.9 us, 512 x 4096 x 4608 23.2 -> 19.1; with a round more,
// 640 x 18944 x 3584 (two instead of one) 70.2 and 99, 1500 (three, two) 130 and 142.
bool half_tiles(int64_t m_tiles, int64_t N, int sms) {
    const int64_t pairs = sms / 2, full = m_tiles * ((N + 255) / 256), half = m_tiles * ((N + 127) / 128);
    return (half + pairs - 1) / pairs == (full + pairs - 1) / pairs;
}

// Xf and sa, or, with X, up to kOwnRows rows of values of type x_f16.
template <typename TY>
cudaError_t launch_gemm(const uint8_t* Xf, const float* sa, const void* X, int x_f16, int64_t M, int64_t K, const uint8_t* Wf,
                        const float* sw, int64_t N, void* Y, int sms, unsigned flags, cudaStream_t stream) {
    F8Args a = {};
    a.sa = sa;
    a.sw = sw;
    a.Y = Y;
    a.N = N;
    a.M = (int)M;
    a.K = (int)K;
    a.X = X;
    a.kbs = (int)((K + kF8Block - 1) / kF8Block);
    if (goes_wide(M, N)) {
        const int64_t m_tiles = (M + 2 * kRows - 1) / (2 * kRows);
        return half_tiles(m_tiles, N, sms) ? launch_wide<128, TY>(a, m_tiles, Xf, K, Wf, sms, flags, stream)
                                           : launch_wide<256, TY>(a, m_tiles, Xf, K, Wf, sms, flags, stream);
    }
    const int64_t n_tiles = (N + kRows - 1) / kRows;
    const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
    a.tiles_a = (int)n_tiles;
    if (!code_map(&a.tm_a, Wf, N, K, kRows)) return cudaErrorNotSupported;
    if (X != nullptr)
        return x_f16 ? launch_narrow<16, TY, __half>(a, flags, stream)
                     : launch_narrow<16, TY, float>(a, flags, stream);
    if (!code_map(&a.tm_b, Xf, M, K, bn)) return cudaErrorNotSupported;
    switch (bn) {
        case 16: return launch_narrow<16, TY>(a, flags, stream);
        case 32: return launch_narrow<32, TY>(a, flags, stream);
        case 64: return launch_narrow<64, TY>(a, flags, stream);
        default: return launch_narrow<128, TY>(a, flags, stream);
    }
}

}  // namespace

cudaError_t launch_f8_gemm(const uint8_t* Xf, const float* sa, int64_t M, int64_t K, const uint8_t* Wf, const float* sw,
                           int64_t N, void* Y, int y_f16, int sms, unsigned flags, cudaStream_t stream) {
    return y_f16 ? launch_gemm<__half>(Xf, sa, nullptr, 0, M, K, Wf, sw, N, Y, sms, flags, stream)
                 : launch_gemm<float>(Xf, sa, nullptr, 0, M, K, Wf, sw, N, Y, sms, flags, stream);
}

cudaError_t launch_f8_linear(const void* X, int x_f16, int64_t M, int64_t K, const uint8_t* Wf, const float* sw, int64_t N,
                             void* Y, int y_f16, uint8_t* Xf, float* sa, int sms, unsigned flags, cudaStream_t stream) {
    if (makes_codes(M, N, sms))
        return y_f16 ? launch_gemm<__half>(nullptr, nullptr, X, x_f16, M, K, Wf, sw, N, Y, sms, flags, stream)
                     : launch_gemm<float>(nullptr, nullptr, X, x_f16, M, K, Wf, sw, N, Y, sms, flags, stream);
    const cudaError_t e = launch_f8_quantize_rows(X, x_f16, M, K, Xf, sa, flags, stream);
    // (the product may start under the quantizer, whatever the caller's flags)
    return e != cudaSuccess ? e : launch_f8_gemm(Xf, sa, M, K, Wf, sw, N, Y, y_f16, sms, 1u, stream);
}

cudaError_t read_and_clear_f8_error(unsigned* flags, cudaStream_t stream) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_f8_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_f8_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *flags |= v;
    return e;
}

}  // namespace w4a8
