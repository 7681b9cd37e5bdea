// kvq.cu -- rotary positions and the quantized paged key/value cache: the
// write (rotation, quantization and placement in one pass), the read back,
// and the move of a tree's accepted tokens.
//
// All three are bound by memory: every value is read once and written once.
// The angle: with f = freq / (2 pi) as the 64-bit fraction of a turn F = f 2^64
// (mod 2^64), the turns of position p are p F mod 2^64, exact in integers
// whatever p; its top 32 bits, read as a signed number of 2^-32 turns, go
// through one rounding to fp32 into sincospi.
#include <type_traits>

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
    const int32_t* pos;
    const double* freqs;  // NULL: no rotation
    int rot, inter;
    float mscale;
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

__device__ __forceinline__ uint32_t codes4(float4 v, float s, float top) {
    return (uint32_t)(layer_code(v.x, s, top) & 0xFF) | (uint32_t)(layer_code(v.y, s, top) & 0xFF) << 8 |
           (uint32_t)(layer_code(v.z, s, top) & 0xFF) << 16 | (uint32_t)(layer_code(v.w, s, top) & 0xFF) << 24;
}

// Queries [0, heads_q) rotated to Y, keys and values quantized into the cache
// (HAS_KV).  A CTA takes tokens_per_cta tokens (gridDim.y CTAs share their
// vectors) and computes their cos and sin once for all heads.
template <typename TX, typename TYO, int DIM, int BITS, bool HAS_KV>
__global__ void __launch_bounds__(kLayerThreads) rope_write_kernel(const WriteArgs a) {
    constexpr int LPV = DIM / 8;
    extern __shared__ float2 cs[];  // [tokens_per_cta][rot / 2]
    __shared__ int64_t slot_row[16];
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * a.tokens_per_cta;
    const int nt = min(a.tokens_per_cta, a.b.tokens - t0);
    const int pairs = a.rope.freqs != nullptr ? a.rope.rot / 2 : 0;
    for (int e = threadIdx.x; e < nt * pairs; e += kLayerThreads) {
        const int t = e / pairs, i = e - t * pairs;
        cs[e] = turn_cos_sin(turn_fraction(a.rope.freqs[i]), a.rope.pos[t0 + t], a.rope.mscale);
    }
    if constexpr (HAS_KV) {
        if ((int)threadIdx.x < nt) {
            const int i = t0 + threadIdx.x;
            int64_t row = -1;
            const int b = kvq_find_seq(a.b.cu, a.b.seqs, i);
            if (b >= 0) {
                const int64_t st = a.b.start[b];
                if (st >= 0)
                    row = kvq_slot_row(a.b.table, a.b.max_pages, a.c.pages, a.c.shift, b, st + (i - a.b.cu[b]));
            }
            if (row < 0) atomicOr(&g_kvq_error, kErrCacheRange);
            slot_row[threadIdx.x] = row;
        }
    }
    __syncthreads();
    const int l = threadIdx.x % LPV;
    const bool half = !a.rope.inter && 8 * l < 2 * pairs;
    const int oa = half ? 4 * l : 8 * l, ob = half ? pairs + 4 * l : 8 * l + 4;
    const int vecs = a.heads_q + (HAS_KV ? 2 * a.c.heads : 0);
    // whole warps iterate together (the reductions below are warp-wide)
    const int groups = kLayerThreads / LPV;
    const int total = nt * vecs;
    for (int base = blockIdx.y * groups; base < total; base += gridDim.y * groups) {
        const int e = base + threadIdx.x / LPV;
        const bool live = e < total;
        const int t = live ? e / vecs : 0, h = live ? e - t * vecs : 0;
        const int64_t tok = t0 + t;
        const bool is_q = h < a.heads_q;
        const int kv = is_q ? 0 : (h - a.heads_q) / a.c.heads;  // 0 key, 1 value
        const int hk = is_q ? 0 : (h - a.heads_q) - kv * a.c.heads;
        const TX* x = is_q ? static_cast<const TX*>(a.Q) + tok * a.ld_q + (int64_t)h * DIM
                      : kv ? static_cast<const TX*>(a.V) + tok * a.ld_v + (int64_t)hk * DIM
                           : static_cast<const TX*>(a.K) + tok * a.ld_k + (int64_t)hk * DIM;
        float4 va = make_float4(0.f, 0.f, 0.f, 0.f), vb = va;
        const bool turned = (is_q || kv == 0) && 8 * l < 2 * pairs;
        // a value's vector has no pairs: its runs stay in order
        const int pa = turned ? oa : 8 * l, pb = turned ? ob : 8 * l + 4;
        if (live) {
            va = load4(x + pa);
            vb = load4(x + pb);
        }
        if (turned) rotate8(va, vb, cs + t * pairs + 4 * l, a.rope.inter);
        if (is_q && live) {
            TYO* y = static_cast<TYO*>(a.Y) + tok * a.ld_y + (int64_t)h * DIM;
            store4(y + pa, va);
            store4(y + pb, vb);
        }
        if constexpr (HAS_KV) {
            float m = fmaxf(absmax4(va), absmax4(vb));
            #pragma unroll
            for (int o = LPV / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            if (!is_q && live && slot_row[t] >= 0) {
                constexpr float top = BITS == 8 ? 127.f : 7.f;
                const float s = __fmul_rn(m, 1.f / top);
                const int64_t vec = kvq_vec(a.c, slot_row[t], hk);
                const uint32_t qa = codes4(va, s, top), qb = codes4(vb, s, top);
                uint8_t* codes = (kv ? a.c.v : a.c.k) + vec * (DIM * BITS / 8);
                if constexpr (BITS == 8) {
                    *reinterpret_cast<uint32_t*>(codes + pa) = qa;
                    *reinterpret_cast<uint32_t*>(codes + pb) = qb;
                } else {
                    auto pack = [](uint32_t q) {  // low nibbles of 4 bytes -> 16 bits
                        q &= 0x0F0F0F0Fu;
                        q |= q >> 4;
                        return (uint16_t)((q & 0xFFu) | ((q >> 8) & 0xFF00u));
                    };
                    *reinterpret_cast<uint16_t*>(codes + pa / 2) = pack(qa);
                    *reinterpret_cast<uint16_t*>(codes + pb / 2) = pack(qb);
                }
                if (l == 0) (kv ? a.c.vs : a.c.ks)[vec] = s;
            }
        }
    }
}

template <typename TX, typename TYO, int BITS, bool HAS_KV>
cudaError_t launch_write(const WriteArgs& a0, int dim, int sms, unsigned flags, cudaStream_t stream) {
    WriteArgs a = a0;
    const int vecs = a.heads_q + (HAS_KV ? 2 * a.c.heads : 0);
    a.tokens_per_cta = a.b.tokens >= 8 * sms ? 4 : 1;
    const int ctas = (a.b.tokens + a.tokens_per_cta - 1) / a.tokens_per_cta;
    const int groups = kLayerThreads / (dim / 8);
    int gy = 1;
    while (ctas * gy < 2 * sms && gy * groups < vecs * a.tokens_per_cta) gy *= 2;
    const dim3 grid((unsigned)ctas, (unsigned)gy);
    const int smem = a.tokens_per_cta * (a.rope.rot / 2) * (int)sizeof(float2);
    switch (dim) {
        case 64: return layer_launch(rope_write_kernel<TX, TYO, 64, BITS, HAS_KV>, grid, kLayerThreads, smem, flags, stream, a);
        case 128: return layer_launch(rope_write_kernel<TX, TYO, 128, BITS, HAS_KV>, grid, kLayerThreads, smem, flags, stream, a);
        case 256: return layer_launch(rope_write_kernel<TX, TYO, 256, BITS, HAS_KV>, grid, kLayerThreads, smem, flags, stream, a);
        default: return cudaErrorInvalidValue;
    }
}

// ---------------------------------------------------------------------------
// read back
// ---------------------------------------------------------------------------

constexpr int kReadTokens = 16;

template <typename TO, int DIM, int BITS>
__global__ void __launch_bounds__(kLayerThreads) kvq_read_kernel(const KvqCacheArg c, const KvqBatchArg b, TO* K,
                                                            TO* V) {
    constexpr int UPV = DIM / 8;  // units of 8 values per vector
    __shared__ int64_t slot_row[kReadTokens];
    griddep_launch_dependents();
    griddep_wait();
    const int t0 = blockIdx.x * kReadTokens;
    const int nt = min(kReadTokens, b.tokens - t0);
    if ((int)threadIdx.x < nt) {
        const int i = t0 + threadIdx.x;
        int64_t row = -1;
        const int s = kvq_find_seq(b.cu, b.seqs, i);
        if (s >= 0 && b.start[s] >= 0)
            row = kvq_slot_row(b.table, b.max_pages, c.pages, c.shift, s, (int64_t)b.start[s] + (i - b.cu[s]));
        if (row < 0) atomicOr(&g_kvq_error, kErrCacheRange);
        slot_row[threadIdx.x] = row;
    }
    __syncthreads();
    const int units = c.heads * UPV;
    for (int e = threadIdx.x; e < 2 * nt * units; e += kLayerThreads) {
        const int kv = e >= nt * units, r = e - kv * nt * units;
        const int t = r / units, u = r - t * units;
        if (slot_row[t] < 0) continue;
        const int64_t vec = kvq_vec(c, slot_row[t], u / UPV);
        const float s = (kv ? c.vs : c.ks)[vec];
        const uint8_t* p = (kv ? c.v : c.k) + vec * (DIM * BITS / 8) + (u % UPV) * BITS;
        float v[8];
        if constexpr (BITS == 8) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            #pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (float)(int8_t)((k < 4 ? w.x : w.y) >> (8 * (k & 3))) * s;
        } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
            #pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = (float)((int32_t)(w << (28 - 4 * k)) >> 28) * s;
        }
        TO* o = (kv ? V : K) + ((int64_t)(t0 + t) * units + u) * 8;
        store4(o, make_float4(v[0], v[1], v[2], v[3]));
        store4(o + 4, make_float4(v[4], v[5], v[6], v[7]));
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
                               const int32_t* pos, const double* freqs, int rot, int inter, float mscale, void* Y,
                               int y_f16, int64_t ld_y, int sms, unsigned flags, cudaStream_t stream) {
    WriteArgs a = {};
    a.b.tokens = (int)tokens;
    a.rope = {pos, freqs, rot, inter, mscale};
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
                             const double* freqs, int rot, int inter, float mscale, uint16_t* Q_out, int sms,
                             unsigned flags, cudaStream_t stream) {
    WriteArgs a = {};
    a.c = cache_arg(c);
    a.b = batch_arg(b);
    a.rope = {pos, freqs, freqs ? rot : 0, inter, mscale};
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

cudaError_t launch_kvq_read(const kvq_cache_t& cc, const kvq_batch_t& bb, void* K, void* V, int y_f16,
                            unsigned flags, cudaStream_t stream) {
    const KvqCacheArg c = cache_arg(cc);
    const KvqBatchArg b = batch_arg(bb);
    const dim3 grid((unsigned)((b.tokens + kReadTokens - 1) / kReadTokens));
    auto go = [&](auto* out, auto dim, auto bits) {
        using T = std::remove_pointer_t<decltype(out)>;
        return layer_launch(kvq_read_kernel<T, decltype(dim)::value, decltype(bits)::value>, grid, kLayerThreads, 0, flags,
                            stream, c, b, static_cast<T*>(K), static_cast<T*>(V));
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
