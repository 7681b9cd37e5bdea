// kvq_attn.cu -- attention of decode rows and of drafted trees over the
// quantized paged cache:
//   t_j = scale ks_j (q . kc_j),  p_j = exp(t_j - max t),  out = sum p_j vs_j vc_j / sum p_j.
//
// One CTA per (token, query head): the keys are walked in tiles of one key
// per thread with the running maximum and sum of the softmax, then each
// thread sums its output dimensions over the tile.
#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

__device__ unsigned g_attn_error;

constexpr int kAttnThreads = 128;

struct AttnArgs {
    KvqCacheArg c;
    KvqBatchArg b;
    const __half* Q;
    const uint64_t* mask;
    __half* out;
    int heads_q;
    float scale;
};

template <int BITS>
__device__ __forceinline__ float code_at(const uint8_t* p, int d) {
    if constexpr (BITS == 8) return (float)(int8_t)p[d];
    const int n = (p[d >> 1] >> (4 * (d & 1))) & 15;
    return (float)(n - ((n & 8) << 1));
}

template <int DIM, int BITS>
__global__ void __launch_bounds__(kAttnThreads) attn_kernel(const AttnArgs a) {
    __shared__ float q[DIM], p[kAttnThreads], red[kAttnThreads / 32];
    __shared__ int64_t vecs[kAttnThreads];
    griddep_launch_dependents();
    griddep_wait();
    const int i = blockIdx.x / a.heads_q, h = blockIdx.x % a.heads_q;
    const int hk = h / (a.heads_q / a.c.heads);
    const int64_t orow = ((int64_t)i * a.heads_q + h) * DIM;
    const int b = kvq_find_seq(a.b.cu, a.b.seqs, i);
    KvqSeq s = {0, 0, 0, 0, false};
    if (b >= 0) s = kvq_seq(a.b.cu, a.b.start, b, a.b.tokens, a.b.max_pages, a.c.shift);
    if (!s.ok || (a.mask != nullptr && s.count > KVQ_MAX_TREE)) {
        if (threadIdx.x == 0) atomicOr(&g_attn_error, kErrCacheRange);
        if (a.mask != nullptr && s.count > KVQ_MAX_TREE) s.end = 0;
    }
    const int64_t L = s.end;
    const uint64_t bits = a.mask != nullptr ? a.mask[i] : 0;
    for (int d = threadIdx.x; d < DIM; d += kAttnThreads) q[d] = __half2float(a.Q[orow + d]);
    __syncthreads();
    float m = -INFINITY, l = 0.f, o[(DIM + kAttnThreads - 1) / kAttnThreads] = {};
    for (int64_t j0 = 0; j0 < L; j0 += kAttnThreads) {
        const int64_t j = j0 + threadIdx.x;
        float t = -INFINITY;
        int64_t vec = -1;
        const int64_t w = j - s.start;  // place among the drafted tokens
        if (j < L && (w < 0 || (a.mask != nullptr ? (bits >> w) & 1 : w <= i - s.first))) {
            const int64_t row = kvq_slot_row(a.b.table, a.b.max_pages, a.c.pages, a.c.shift, b, j);
            if (row >= 0) {
                vec = kvq_vec(a.c, row, hk);
                const uint8_t* k = a.c.k + vec * (DIM * BITS / 8);
                float acc = 0.f;
                for (int d = 0; d < DIM; ++d) acc = fmaf(q[d], code_at<BITS>(k, d), acc);
                t = acc * a.c.ks[vec] * a.scale;
            } else {
                atomicOr(&g_attn_error, kErrCacheRange);
            }
        }
        float mt = t;
        for (int o2 = 16; o2 >= 1; o2 >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xFFFFFFFFu, mt, o2));
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mt;
        __syncthreads();
        mt = m;
        for (int w2 = 0; w2 < kAttnThreads / 32; ++w2) mt = fmaxf(mt, red[w2]);
        const float pe = vec >= 0 ? expf(t - mt) : 0.f;
        const float alpha = m == -INFINITY ? 0.f : expf(m - mt);
        float sum = pe;
        for (int o2 = 16; o2 >= 1; o2 >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o2);
        __syncthreads();
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = sum;
        p[threadIdx.x] = vec >= 0 ? pe * a.c.vs[vec] : 0.f;
        vecs[threadIdx.x] = vec;
        __syncthreads();
        sum = 0.f;
        for (int w2 = 0; w2 < kAttnThreads / 32; ++w2) sum += red[w2];
        l = l * alpha + sum;
        m = mt;
        int n = 0;
        for (int d = threadIdx.x; d < DIM; d += kAttnThreads, ++n) {
            float acc = o[n] * alpha;
            for (int k = 0; k < kAttnThreads; ++k)
                if (vecs[k] >= 0) acc = fmaf(p[k], code_at<BITS>(a.c.v + vecs[k] * (DIM * BITS / 8), d), acc);
            o[n] = acc;
        }
        __syncthreads();
    }
    int n = 0;
    for (int d = threadIdx.x; d < DIM; d += kAttnThreads, ++n)
        a.out[orow + d] = __float2half_rn(L > 0 && m > -INFINITY ? o[n] / l : (l != l ? l : 0.f));
}

}  // namespace

size_t kvq_attn_workspace(const kvq_cache_t&, const kvq_batch_t&, int, int) { return 0; }

cudaError_t launch_kvq_attention(const kvq_cache_t& c, const kvq_batch_t& b, const uint16_t* Q, int heads_q,
                                 const uint64_t* mask, float scale, uint16_t* out, void*, int, unsigned flags,
                                 cudaStream_t stream) {
    const AttnArgs a = {cache_arg(c), batch_arg(b), reinterpret_cast<const __half*>(Q), mask,
                        reinterpret_cast<__half*>(out), heads_q, scale};
    const dim3 grid((unsigned)(b.tokens * heads_q));
    auto go = [&](auto* f) { return layer_launch(f, grid, kAttnThreads, 0, flags, stream, a); };
    if (c.bits == 8)
        return c.dim == 64 ? go(attn_kernel<64, 8>) : c.dim == 128 ? go(attn_kernel<128, 8>) : go(attn_kernel<256, 8>);
    return c.dim == 64 ? go(attn_kernel<64, 4>) : c.dim == 128 ? go(attn_kernel<128, 4>) : go(attn_kernel<256, 4>);
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
