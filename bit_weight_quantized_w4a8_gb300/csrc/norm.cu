// norm.cu -- the residual update between two blocks with the norm after the
// one and the norm before the other, in one pass over the row:
//   u = y [/ rms(y) * post_w];  r' = alpha r + beta gate u;  x = r' / rms(r') w
// One CTA holds a row in registers, so every tensor is read and written once.
// Bound by memory where there are many rows (12289 x 4096, fp32 r and y: 112 us, 6.3 TB/s,
// 92% of the copy rate), by its launch and two reductions where there are few
// (one row of 3584: 2.5 us in a graph, 64 rows: 3.3).
#include "kernels.h"
#include "layer.cuh"

namespace w4a8 {
namespace {

struct NormArgs {
    const void* r;
    const void* y;
    const float *post_w, *gate, *w;
    int64_t ld_gate, M;
    int N;
    float alpha, beta, eps;
    void* r_out;
    __half* X;
    int8_t* Xq;
    float* sa;
};

// Sum (or maximum) over the CTA of one value per thread; every thread gets
// it.  `red` holds one float per warp.  The order is fixed by the thread
// count, so a row gives the same bits whatever the batch.
template <bool MAX>
__device__ __forceinline__ float cta_reduce(float v, float* red) {
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float t = __shfl_xor_sync(0xFFFFFFFFu, v, o);
        v = MAX ? fmaxf(v, t) : v + t;
    }
    const int warps = blockDim.x >> 5;
    __syncthreads();  // the last use of `red` is over
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
    #pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        const float t = __shfl_xor_sync(0xFFFFFFFFu, s, o);
        s = MAX ? fmaxf(s, t) : s + t;
    }
    return s;
}

template <typename T, int V>
__device__ __forceinline__ void load_vals(const T* p, float* v) {
    if constexpr (V == 8) {
        const float4 a = load4(p), b = load4(p + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        v[0] = static_cast<float>(p[0]);
    }
}

// V values in a row per chunk (8: vector path, 1: any size and alignment),
// CH chunks per thread.
template <typename TY, typename TR, int V, int CH>
__global__ void __launch_bounds__(1024) add_norm_kernel(const NormArgs a) {
    __shared__ float red[32];
    griddep_launch_dependents();
    griddep_wait();
    const int chunks = a.N / V;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        float v[CH][V];
        const TR* r = static_cast<const TR*>(a.r) + m * a.N;
        if (a.y != nullptr) {
            const TY* y = static_cast<const TY*>(a.y) + m * a.N;
            #pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int i = threadIdx.x + c * blockDim.x;
                if (i < chunks) {
                    load_vals<TY, V>(y + (int64_t)i * V, v[c]);
                } else {
                    #pragma unroll
                    for (int k = 0; k < V; ++k) v[c][k] = 0.f;
                }
            }
            if (a.post_w != nullptr) {
                float s = 0.f;
                #pragma unroll
                for (int c = 0; c < CH; ++c)
                    #pragma unroll
                    for (int k = 0; k < V; ++k) s = fmaf(v[c][k], v[c][k], s);
                s = cta_reduce<false>(s, red);
                const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(s, (float)a.N) + a.eps));
                #pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int i = threadIdx.x + c * blockDim.x;
                    if (i < chunks) {
                        float w[V];
                        load_vals<float, V>(a.post_w + (int64_t)i * V, w);
                        #pragma unroll
                        for (int k = 0; k < V; ++k) v[c][k] = v[c][k] * inv * w[k];
                    }
                }
            }
        }
        float s = 0.f;
        #pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < chunks) {
                float t[V], g[V];
                load_vals<TR, V>(r + (int64_t)i * V, t);
                if (a.gate != nullptr) load_vals<float, V>(a.gate + m * a.ld_gate + (int64_t)i * V, g);
                #pragma unroll
                for (int k = 0; k < V; ++k) {
                    float x = a.alpha * t[k];
                    if (a.y != nullptr) x = fmaf(a.gate != nullptr ? a.beta * g[k] : a.beta, v[c][k], x);
                    v[c][k] = x;
                    s = fmaf(x, x, s);
                }
                if (a.r_out != nullptr) {
                    TR* o = static_cast<TR*>(a.r_out) + m * a.N + (int64_t)i * V;
                    if constexpr (V == 8) {
                        store4(o, make_float4(v[c][0], v[c][1], v[c][2], v[c][3]));
                        store4(o + 4, make_float4(v[c][4], v[c][5], v[c][6], v[c][7]));
                    } else {
                        o[0] = static_cast<TR>(v[c][0]);
                    }
                }
            }
        }
        if (a.X == nullptr && a.Xq == nullptr) continue;
        s = cta_reduce<false>(s, red);
        const float inv = __fdiv_rn(1.f, __fsqrt_rn(__fdiv_rn(s, (float)a.N) + a.eps));
        float mx = 0.f;
        #pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < chunks) {
                float w[V];
                load_vals<float, V>(a.w + (int64_t)i * V, w);
                #pragma unroll
                for (int k = 0; k < V; ++k) {
                    const __half h = __float2half_rn(v[c][k] * inv * w[k]);
                    v[c][k] = __half2float(h);
                    mx = fmaxf(mx, fabsf(v[c][k]));
                }
                if (a.X != nullptr) {
                    __half* o = a.X + m * a.N + (int64_t)i * V;
                    if constexpr (V == 8)
                        *reinterpret_cast<uint4*>(o) =
                            make_uint4(pack_half2(v[c][0], v[c][1]), pack_half2(v[c][2], v[c][3]),
                                       pack_half2(v[c][4], v[c][5]), pack_half2(v[c][6], v[c][7]));
                    else
                        o[0] = __float2half_rn(v[c][0]);
                }
            }
        }
        if (a.Xq == nullptr) continue;
        const float sc = __fdiv_rn(cta_reduce<true>(mx, red), 127.f);
        if (threadIdx.x == 0) a.sa[m] = sc;
        #pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int i = threadIdx.x + c * blockDim.x;
            if (i < chunks) {
                int8_t* o = a.Xq + m * a.N + (int64_t)i * V;
                if constexpr (V == 8) {
                    uint32_t q[2] = {0u, 0u};
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        q[k >> 2] |= (uint32_t)(layer_code(v[c][k], sc, 127.f) & 0xFF) << (8 * (k & 3));
                    *reinterpret_cast<uint2*>(o) = make_uint2(q[0], q[1]);
                } else {
                    o[0] = (int8_t)layer_code(v[c][0], sc, 127.f);
                }
            }
        }
    }
}

template <typename TY, typename TR>
cudaError_t launch_types(const NormArgs& a, bool vec, unsigned flags, cudaStream_t stream) {
    const int chunks = vec ? a.N / 8 : a.N;
    const int grid = (int)(a.M < (1 << 30) ? a.M : (1 << 30));
    const int ch = (chunks + 1023) / 1024;
    const int per = (chunks + ch - 1) / ch;
    const int threads = (per + 31) / 32 * 32;
    if (vec) {
        if (ch == 1) return layer_launch(add_norm_kernel<TY, TR, 8, 1>, grid, threads, 0, flags, stream, a);
        if (ch == 2) return layer_launch(add_norm_kernel<TY, TR, 8, 2>, grid, threads, 0, flags, stream, a);
        return layer_launch(add_norm_kernel<TY, TR, 8, 4>, grid, threads, 0, flags, stream, a);
    }
    if (ch <= 4) return layer_launch(add_norm_kernel<TY, TR, 1, 4>, grid, threads, 0, flags, stream, a);
    return layer_launch(add_norm_kernel<TY, TR, 1, 32>, grid, threads, 0, flags, stream, a);
}

}  // namespace

cudaError_t launch_add_norm(const void* r, int r_f16, const void* y, int y_f16, const float* post_w,
                            const float* gate, int64_t ld_gate, const float* w, int64_t M, int N, float alpha,
                            float beta, float eps, void* r_out, uint16_t* X, int8_t* Xq, float* sa, bool vec,
                            unsigned flags, cudaStream_t stream) {
    const NormArgs a = {r, y, post_w, gate, w, ld_gate, M, N, alpha, beta, eps, r_out,
                        reinterpret_cast<__half*>(X), Xq, sa};
    if (r_f16)
        return y_f16 ? launch_types<__half, __half>(a, vec, flags, stream)
                     : launch_types<float, __half>(a, vec, flags, stream);
    return y_f16 ? launch_types<__half, float>(a, vec, flags, stream)
                 : launch_types<float, float>(a, vec, flags, stream);
}

}  // namespace w4a8
