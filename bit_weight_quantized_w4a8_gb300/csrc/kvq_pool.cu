// kvq_pool.cu -- the cache's pages handed out and taken back on the device,
// and a step's offsets, positions and slots from request lengths.
//
// Everything is a prefix sum over the rows (requests) and a look-up per token
// or page:
//   back[b]  = pages row b gives back;  mid = top + sum back
//   need[b]  = max(ceil((lens[b] + n[b]) / page) - held[b], 0)
//   row b goes in when the rows up to it ask for no more than mid pages (or it
//   needs none) and no more tokens than there is room for
//   page k of all pages handed out (rows in order) is place mid - 1 - k of the
//   stack, page k of all pages given back goes to place mid - 1 - k: a call
//   that hands out and one that takes all of it back leave the stack as it was.
// A place from top on that a page of this same call came back to is read from
// that page's row instead of the stack, so that both directions run side by
// side: no barrier stands between them and nothing is written that is read.
//
// One cluster of CTAs scans (a thread has up to 8 rows, so 65536 rows take one
// pass) and, for short steps, writes all; for long ones a second launch writes
// with the whole GPU.  In a graph 48 requests take 4.2 us, 4093 requests of which half are
// exchanged (two calls) 27.7 to 29.4: latency, of the scan's two to three prefix sums (10 us a call under
// ncu) and of a look-up's search through the offsets, 12 loads one after the other (10 to 16).  Two requests in
// a pool of 1000, 8000 and 65536 rows: 10, 18 and 51 us, wherever they sit.  (8 rows a thread, from 8193 rows on, spill
// 400 bytes.)
#include <cooperative_groups.h>

#include <type_traits>

#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned g_pool_error;

constexpr int kPlanThreads = 1024;
constexpr int kPlanItems = 8;     // rows of a thread, at most
constexpr int kPlanCluster = 8;   // 8 x 1024 x 8 = 65536 rows
constexpr int kFillThreads = 256;

// What the scan leaves for the look-ups.
struct PlanTotals {
    int64_t back, need;  // pages given back, handed out
    int top, mid;        // of the stack before and after the former
    int tokens;
};

struct PlanArgs {
    int32_t *table, *held, *stack, *top;
    int64_t max_pages, pages;
    int seqs, shift, room;
    int32_t* lens;
    const int32_t *grow, *add;
    const uint64_t* mask;
    int32_t *cu, *pos, *seq;
    int64_t* slot;
    // workspace: first page of each row among those given back and handed out,
    // pages held before, first word of its tree (with mask), totals
    int32_t *back_at, *need_at, *old_held, *ask_at;
    PlanTotals* totals;
    const int32_t *cu_at, *len_at;  // cu and lens as the look-ups read them
    int wide;                       // pos, slot and seq on 16 bytes
};

struct Pair {
    int64_t a, b;
    __device__ __forceinline__ Pair operator+(Pair o) const { return {a + o.a, b + o.b}; }
};

struct ScanShared {
    Pair warp[32], cta[2];
};

// Exclusive prefix of v over the threads of the cluster; *total over all.  The CTAs'
// sums take turns in two places, so that one barrier a scan does: the next but one writes
// there again.
__device__ Pair cluster_scan(Pair v, ScanShared& sh, int& turn, Pair* total) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    Pair x = v;
    #pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const Pair y = {__shfl_up_sync(0xFFFFFFFFu, x.a, o), __shfl_up_sync(0xFFFFFFFFu, x.b, o)};
        if (lane >= o) x = x + y;
    }
    __syncthreads();  // the warps' sums of the scan before have been read
    if (lane == 31) sh.warp[warp] = x;
    __syncthreads();
    Pair base = {0, 0}, all = {0, 0};
    Pair w = lane < warps ? sh.warp[lane] : Pair{0, 0};
    #pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const Pair y = {__shfl_up_sync(0xFFFFFFFFu, w.a, o), __shfl_up_sync(0xFFFFFFFFu, w.b, o)};
        if (lane >= o) w = w + y;
    }
    if (warp > 0) base = {__shfl_sync(0xFFFFFFFFu, w.a, warp - 1), __shfl_sync(0xFFFFFFFFu, w.b, warp - 1)};
    all = {__shfl_sync(0xFFFFFFFFu, w.a, 31), __shfl_sync(0xFFFFFFFFu, w.b, 31)};
    cg::cluster_group cl = cg::this_cluster();
    *total = all;
    if (cl.num_blocks() > 1) {
        if (threadIdx.x == 0) sh.cta[turn] = all;
        cl.sync();
        *total = {0, 0};
        #pragma unroll
        for (unsigned r = 0; r < kPlanCluster; ++r) {
            const Pair s = *cl.map_shared_rank(&sh.cta[turn], r);
            if (r < cl.block_rank()) base = base + s;
            *total = *total + s;
        }
        turn ^= 1;
    }
    return {base.a + x.a - v.a, base.b + x.b - v.b};
}

// The last row b with at[b] <= k.
__device__ __forceinline__ int row_of(const int32_t* at, int rows, int64_t k) {
    int lo = 0, hi = rows;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (at[mid] <= k)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Page k of those given back.
__device__ __forceinline__ int32_t page_back(const PlanArgs& a, int64_t k) {
    const int b = row_of(a.back_at, a.seqs, k);
    return a.table[b * a.max_pages + (k - a.back_at[b])];
}
// Page k of those handed out.
__device__ __forceinline__ int32_t page_out(const PlanArgs& a, const PlanTotals& t, int64_t k) {
    const int64_t p = t.mid - 1 - k;
    return p < t.top ? a.stack[p] : page_back(a, (int64_t)t.top + t.back - 1 - p);
}

// Pages handed out, pages given back and tokens, by thread i of n; a thread takes
// four tokens in a row, so that one search does for them and they leave in wide stores.
// TREES: positions by mask, in variants of their own: in one, the calls without took 4.6 us instead of
// 4.2 (48 requests) and 28.7 instead of 27.7 (4093 requests, two calls).
template <bool TREES>
__device__ void plan_fill(const PlanArgs& a, const PlanTotals& t, int64_t i, int64_t n) {
    for (int64_t k = i; k < t.need; k += n) {
        const int b = row_of(a.need_at, a.seqs, k);
        a.table[b * a.max_pages + a.old_held[b] + (k - a.need_at[b])] = page_out(a, t, k);
    }
    for (int64_t k = i; k < t.back; k += n) {
        const int64_t p = (int64_t)t.top + t.back - 1 - k;
        if (p < a.pages) a.stack[p] = page_back(a, k);
    }
    if (a.pos == nullptr && a.slot == nullptr && a.seq == nullptr) return;
    for (int64_t g = 4 * i; g < a.room; g += 4 * n) {
        int pos[4], seq[4];
        int64_t slot[4];
        int row = g < t.tokens ? row_of(a.cu_at, a.seqs, g) : 0;
        #pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t k = g + e;
            pos[e] = 0;
            slot[e] = seq[e] = -1;
            if (k < t.tokens) {
                // the next row most often; another search where rows without tokens lie between (65534 of
                // them, one by one: 4.1 ms)
                if (a.cu_at[row + 1] <= k && a.cu_at[++row + 1] <= k) row = row_of(a.cu_at, a.seqs, k);
                const int len = a.len_at[row], x = len + (int)(k - a.cu_at[row]);
                pos[e] = TREES ? len + __popcll(a.mask[a.ask_at[row] + (x - len)]) - 1 : x;
                seq[e] = row;
                if (a.slot != nullptr) {
                    const int64_t j = x >> a.shift, old = a.old_held[row];
                    const int32_t page = j < old ? a.table[row * a.max_pages + j] : page_out(a, t, a.need_at[row] + j - old);
                    if (page >= 0 && page < a.pages) slot[e] = ((int64_t)page << a.shift) + (x & ((1 << a.shift) - 1));
                }
            }
        }
        if (a.wide && g + 4 <= a.room) {
            if (a.pos != nullptr) *reinterpret_cast<int4*>(a.pos + g) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            if (a.seq != nullptr) *reinterpret_cast<int4*>(a.seq + g) = make_int4(seq[0], seq[1], seq[2], seq[3]);
            if (a.slot != nullptr) {
                reinterpret_cast<longlong2*>(a.slot + g)[0] = make_longlong2(slot[0], slot[1]);
                reinterpret_cast<longlong2*>(a.slot + g)[1] = make_longlong2(slot[2], slot[3]);
            }
        } else {
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (g + e >= a.room) break;
                if (a.pos != nullptr) a.pos[g + e] = pos[e];
                if (a.slot != nullptr) a.slot[g + e] = slot[e];
                if (a.seq != nullptr) a.seq[g + e] = seq[e];
            }
        }
    }
}

// ITEMS: rows of a thread.  FILL: writes the step too; with one CTA (kOne) the look-ups stay
// in shared memory.
constexpr int kOneRows = 1024;
template <int ITEMS, bool FILL, bool kOne, bool TREES>
__global__ void __launch_bounds__(kPlanThreads) plan_scan_kernel(const __grid_constant__ PlanArgs args) {
    __shared__ ScanShared sh;
    __shared__ int32_t rows_at[kOne ? 5 + TREES : 1][kOne ? kOneRows + 1 : 1];
    PlanArgs a = args;
    if constexpr (kOne) {
        a.back_at = rows_at[0];
        a.need_at = rows_at[1];
        a.old_held = rows_at[2];
        a.cu_at = rows_at[3];
        a.len_at = rows_at[4];
        if constexpr (TREES) a.ask_at = rows_at[5];
    }
    griddep_launch_dependents();
    griddep_wait();
    const int ctas = gridDim.x, threads = blockDim.x;
    const int per = ITEMS == 1 ? 1 : (a.seqs + ctas * threads - 1) / (ctas * threads);
    const int r0 = (blockIdx.x * threads + threadIdx.x) * per;
    const int rows = max(0, min(per, a.seqs - r0));
    bool bad = false;
    const int top_in = *a.top;
    int64_t len[ITEMS], n[ITEMS];
    int held[ITEMS], back[ITEMS];
    int64_t back_sum = 0, ask_sum = 0;
    #pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        len[i] = n[i] = 0;
        held[i] = back[i] = 0;
        if (i < rows) {
            const int r = r0 + i;
            const int add = a.add[r], h = a.held[r];
            len[i] = (int64_t)a.lens[r] + (a.grow != nullptr ? a.grow[r] : 0);
            held[i] = (int)min((int64_t)max(h, 0), a.max_pages);
            bad |= held[i] != h || len[i] < 0 || len[i] > kKvqMaxSlots;
            len[i] = min(max(len[i], (int64_t)0), (int64_t)kKvqMaxSlots);
            n[i] = max(add, 0);
            if (add < 0) {
                back[i] = held[i];
                held[i] = 0;
                len[i] = 0;
            }
            back_sum += back[i];
            if constexpr (TREES) ask_sum += n[i];
        }
    }
    int turn = 0;
    Pair total;
    const Pair bp = cluster_scan({back_sum, ask_sum}, sh, turn, &total);
    PlanTotals t;
    t.top = (int)min((int64_t)max(top_in, 0), a.pages);
    t.back = total.a;
    t.mid = (int)min(t.top + total.a, a.pages);
    bad |= t.top != top_in || t.top + total.a > a.pages;

    // trees' words lie as all rows ask for tokens, whether they go in or wait: the caller
    // lays them out before the call
    int64_t need[ITEMS], ask_p = 0, ask_n = 0, words = bp.b;
    #pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        need[i] = 0;
        if (TREES && i < rows) a.ask_at[r0 + i] = (int)min(words, (int64_t)a.room);
        if (n[i] > 0) {
            const int64_t end = len[i] + n[i], want = (end + (1 << a.shift) - 1) >> a.shift;
            words += n[i];
            if (want > a.max_pages || end > kKvqMaxSlots || (TREES && words > a.room))
                n[i] = 0;
            else
                need[i] = max(want - held[i], (int64_t)0);
        }
        ask_p += need[i];
        ask_n += n[i];
    }
    Pair at = cluster_scan({ask_p, ask_n}, sh, turn, &total);
    if (total.a > t.mid || total.b > a.room) {  // some have to wait: once more over those that go in
        Pair up = at;
        int64_t got_p = 0, got_n = 0;
        #pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            up = up + Pair{need[i], n[i]};
            if ((need[i] > 0 && up.a > t.mid) || up.b > a.room) need[i] = n[i] = 0;
            got_p += need[i];
            got_n += n[i];
        }
        at = cluster_scan({got_p, got_n}, sh, turn, &total);
    }
    t.need = total.a;
    t.tokens = (int)total.b;
    int64_t b_at = bp.a, p_at = at.a, n_at = at.b;
    #pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        if (i < rows) {
            const int r = r0 + i;
            a.lens[r] = (int)len[i];
            a.held[r] = held[i] + (int)need[i];
            a.cu[r] = (int)n_at;
            if constexpr (kOne) {
                rows_at[3][r] = (int)n_at;
                rows_at[4][r] = (int)len[i];
            }
            a.back_at[r] = (int)min(b_at, (int64_t)0x7FFFFFFF);  // (more than that cannot be free pages)
            a.need_at[r] = (int)p_at;
            a.old_held[r] = held[i];
            b_at += back[i];
            p_at += need[i];
            n_at += n[i];
        }
    }
    if (t.back > 0x7FFFFFFF) t.back = 0x7FFFFFFF, bad = true;
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.cu[a.seqs] = t.tokens;
        if constexpr (kOne) rows_at[3][a.seqs] = t.tokens;
        *a.top = t.mid - (int)t.need;
        if constexpr (!FILL) *a.totals = t;
    }
    if (bad) atomicOr(&g_pool_error, kErrCacheRange);
    if (!kOne)  // (also: no CTA leaves while its sums may be read)
        cg::this_cluster().sync();
    else
        __syncthreads();
    if constexpr (FILL) plan_fill<TREES>(a, t, blockIdx.x * threads + threadIdx.x, (int64_t)ctas * threads);
}

template <bool TREES>
__global__ void __launch_bounds__(kFillThreads) plan_fill_kernel(const __grid_constant__ PlanArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    plan_fill<TREES>(a, *a.totals, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

}  // namespace

size_t kvq_plan_workspace(const kvq_pool_t& p) { return 256 + 4 * (size_t)((p.seqs + 63) / 64 * 64) * 4; }

cudaError_t launch_kvq_plan(const kvq_pool_t& p, int32_t* lens, const int32_t* grow, const int32_t* add,
                            const uint64_t* mask, int64_t tokens, int32_t* cu, int32_t* pos, int64_t* slot,
                            int32_t* seq, void* ws, int sms, unsigned flags, cudaStream_t stream) {
    PlanArgs a = {};
    a.table = p.table;
    a.held = p.held;
    a.stack = p.stack;
    a.top = p.top;
    a.max_pages = p.max_pages;
    a.pages = p.pages;
    a.seqs = (int)p.seqs;
    while ((1 << a.shift) < p.page) ++a.shift;
    a.room = (int)tokens;
    a.lens = lens;
    a.grow = grow;
    a.add = add;
    a.mask = mask;
    a.cu = cu;
    a.pos = pos;
    a.slot = slot;
    a.seq = seq;
    const int64_t pad = (p.seqs + 63) / 64 * 64;
    a.totals = static_cast<PlanTotals*>(ws);
    a.back_at = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + 256);
    a.need_at = a.back_at + pad;
    a.old_held = a.need_at + pad;
    a.ask_at = a.old_held + pad;
    a.cu_at = cu;
    a.len_at = lens;
    a.wide = reinterpret_cast<uintptr_t>(pos) % 16 == 0 && reinterpret_cast<uintptr_t>(slot) % 16 == 0 &&
             reinterpret_cast<uintptr_t>(seq) % 16 == 0;
    // One CTA where rows, tokens and the pages that may come back are few; else a cluster, and
    // for many tokens a second launch over all SMs.
    const bool one = p.seqs <= kOneRows && tokens <= 4096 && p.seqs * p.max_pages <= 1 << 17;
    const bool two = !one && tokens > 16384;
    const int threads = one ? (int)((p.seqs > tokens / 4 ? p.seqs : tokens / 4) + 127) / 128 * 128 : kPlanThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(one ? 1u : (unsigned)kPlanCluster);
    cfg.blockDim = dim3((unsigned)(threads < kPlanThreads ? threads : kPlanThreads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {cfg.gridDim.x, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = flags & 1u ? 2 : 1;
    const bool few = p.seqs <= (int64_t)kPlanCluster * kPlanThreads;  // one row a thread
    auto go = [&](auto trees) {
        constexpr bool T = decltype(trees)::value;
        const cudaError_t e = one   ? cudaLaunchKernelEx(&cfg, plan_scan_kernel<1, true, true, T>, a)
                              : two ? (few ? cudaLaunchKernelEx(&cfg, plan_scan_kernel<1, false, false, T>, a)
                                           : cudaLaunchKernelEx(&cfg, plan_scan_kernel<kPlanItems, false, false, T>, a))
                                    : (few ? cudaLaunchKernelEx(&cfg, plan_scan_kernel<1, true, false, T>, a)
                                           : cudaLaunchKernelEx(&cfg, plan_scan_kernel<kPlanItems, true, false, T>, a));
        if (e != cudaSuccess || !two) return e;
        return layer_launch(plan_fill_kernel<T>, dim3((unsigned)(4 * sms)), kFillThreads, 0, 1u, stream, a);
    };
    return mask != nullptr ? go(std::true_type{}) : go(std::false_type{});
}

cudaError_t read_and_clear_pool_error(unsigned* flags, cudaStream_t stream) {
    unsigned v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_pool_error, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbolAsync(g_pool_error, &z, sizeof(z), 0, cudaMemcpyHostToDevice, stream);
    if (e != cudaSuccess) return e;
    e = cudaStreamSynchronize(stream);
    *flags |= v;
    return e;
}

}  // namespace w4a8
