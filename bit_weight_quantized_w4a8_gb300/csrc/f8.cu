// f8.cu -- the linear with e4m3 weights and activations and a scale for each
// block of 128: the quantizers (the product: f8_mma.cu).
#include <cuda_fp16.h>

#include "f8.cuh"
#include "kernels.h"

namespace w4a8 {
namespace {

constexpr int kF8Threads = 256;

// Sixteen lanes a (row, block of 128), 8 values a lane; a CTA has 8 rows x 2 blocks, so that the
// scales, a block's of all rows side by side, leave in runs of 32 bytes.  One launch in a graph, from
// fp16: 16 x 3584 2.7 us, 777 x 4096 4.6, 8192 x 3584 21.4 (4.1 TB/s; a warp a row and block, with the
// scales one by one, 38; codes made outside the branch that stores them 24.6).  Four blocks a group of
// lanes gain 3% there and cost 16 rows half as much again.  What bounds it is the two roundings of each
// value, to both sides of its quotient.
constexpr int kRowsTile = 8;
template <typename T>
__global__ void __launch_bounds__(kF8Threads) f8_rows_kernel(const T* X, int M, int K, int kbs, uint8_t* Xf, float* sa) {
    constexpr int BLOCKS = kF8Threads / 16 / kRowsTile;
    __shared__ float scales[BLOCKS][kRowsTile];
    griddep_launch_dependents();
    griddep_wait();
    const int g = threadIdx.x / 16, l = threadIdx.x % 16;
    const int r = g % kRowsTile, m = blockIdx.x * kRowsTile + r;
    const int kb = blockIdx.y * BLOCKS + g / kRowsTile, k = kb * kF8Block + 8 * l;
    const bool in = m < M && k < K;  // K is a multiple of 16
    Eight<T> v;
    if (in) v.load(X + (int64_t)m * K + k);
    float4 a, b;
    v.get(a, b);
    const float s = f8_row_scale(a, b);
    float lo, hi;
    quant_bracket(s, &lo, &hi);
    if (in) *reinterpret_cast<uint2*>(Xf + (int64_t)m * K + k) = make_uint2(f8_codes4(a, s, lo, hi), f8_codes4(b, s, lo, hi));
    if (l == 0) scales[g / kRowsTile][r] = s;
    __syncthreads();
    if (threadIdx.x < BLOCKS * kRowsTile) {
        const int block = blockIdx.y * BLOCKS + threadIdx.x / kRowsTile, row = blockIdx.x * kRowsTile + threadIdx.x % kRowsTile;
        if (block < kbs && row < M) sa[(int64_t)block * M + row] = scales[threadIdx.x / kRowsTile][threadIdx.x % kRowsTile];
    }
}

// One CTA a block of 128 rows x 128 values.
__global__ void __launch_bounds__(kF8Threads) f8_weights_kernel(const float* W, int64_t N, int K, int kbs, uint8_t* Wf,
                                                                float* sw) {
    __shared__ float red[kF8Threads / 32];
    const int kb = blockIdx.x % kbs;
    const int64_t n0 = (int64_t)(blockIdx.x / kbs) * kF8Block;
    const int k = kb * kF8Block + 4 * (threadIdx.x % 32), warp = threadIdx.x / 32;
    float4 v[16];
    float top = 0.f;
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = n0 + 8 * i + warp;
        v[i] = n < N && k < K ? load4(W + n * K + k) : make_float4(0.f, 0.f, 0.f, 0.f);
        top = max_nan(top, absmax4_nan(v[i]));
    }
    #pragma unroll
    for (int o = 16; o >= 1; o /= 2) top = max_nan(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (threadIdx.x % 32 == 0) red[warp] = top;
    __syncthreads();
    #pragma unroll
    for (int i = 0; i < kF8Threads / 32; ++i) top = max_nan(top, red[i]);
    const float s = f8_scale(top);
    float lo, hi;
    quant_bracket(s, &lo, &hi);
    #pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t n = n0 + 8 * i + warp;
        if (n < N && k < K) *reinterpret_cast<uint32_t*>(Wf + n * K + k) = f8_codes4(v[i], s, lo, hi);
    }
    if (threadIdx.x == 0) sw[blockIdx.x] = s;
}

int f8_blocks(int64_t k) { return (int)((k + kF8Block - 1) / kF8Block); }

}  // namespace

cudaError_t launch_f8_quantize_weights(const float* W, int64_t N, int64_t K, uint8_t* Wf, float* sw, cudaStream_t stream) {
    const int kbs = f8_blocks(K);
    const int64_t ctas = (N + kF8Block - 1) / kF8Block * kbs;
    return layer_launch(f8_weights_kernel, dim3((unsigned)ctas), kF8Threads, 0, 0u, stream, W, N, (int)K, kbs, Wf, sw);
}

cudaError_t launch_f8_quantize_rows(const void* X, int x_f16, int64_t M, int64_t K, uint8_t* Xf, float* sa, unsigned flags,
                                    cudaStream_t stream) {
    const int kbs = f8_blocks(K);
    const dim3 grid((unsigned)((M + kRowsTile - 1) / kRowsTile), (unsigned)((kbs + 1) / 2));
    return x_f16 ? layer_launch(f8_rows_kernel<__half>, grid, kF8Threads, 0, flags, stream, static_cast<const __half*>(X),
                                (int)M, (int)K, kbs, Xf, sa)
                 : layer_launch(f8_rows_kernel<float>, grid, kF8Threads, 0, flags, stream, static_cast<const float*>(X),
                                (int)M, (int)K, kbs, Xf, sa);
}

}  // namespace w4a8
