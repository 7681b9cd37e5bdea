// layer.cuh -- what the kernels of the decoder layer around the linears
// share: typed 4-value loads and stores, the quantizer's codes, the cache and
// batch descriptions as kernel arguments.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/w4a8.h"
#include "kvq_index.h"
#include "ptx.cuh"

namespace w4a8 {

constexpr unsigned kErrCacheRange = 8u;  // device error word, bit 3

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __half* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__half* p, float4 v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_half2(v.x, v.y), pack_half2(v.z, v.w));
}
// Maximum that is NaN when one of the two is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float absmax4_nan(float4 v) {
    return max_nan(max_nan(fabsf(v.x), fabsf(v.y)), max_nan(fabsf(v.z), fabsf(v.w)));
}

// clamp(round_half_away(x / s), +-top) with the IEEE quotient; 0 for s = 0.
// top 127 or 7: the codes of the framework's quantizers.
__device__ __forceinline__ int layer_code(float x, float s, float top) {
    if (s == 0.f) return 0;
    return static_cast<int>(fminf(fmaxf(roundf(__fdiv_rn(x, s)), -top), top));
}

// kvq_cache_t and kvq_batch_t as kernel arguments.
struct KvqCacheArg {
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t pages;
    int shift, heads;  // page size 1 << shift
};
struct KvqBatchArg {
    const int32_t *cu, *start, *table;
    int64_t max_pages;
    int seqs, tokens;
};

inline KvqCacheArg cache_arg(const kvq_cache_t& c) {
    int shift = 0;
    while ((1 << shift) < c.page) ++shift;
    return {static_cast<uint8_t*>(c.k), static_cast<uint8_t*>(c.v), c.ks, c.vs, c.pages, shift, c.heads};
}
inline KvqBatchArg batch_arg(const kvq_batch_t& b) {
    return {b.cu, b.start, b.table, b.max_pages, (int)b.seqs, (int)b.tokens};
}

// Vector index (row of ks, vs; times the bytes of a vector, of k, v) of
// pool row `row` (kvq_slot_row) and head h: pages are [heads][page] inside.
__device__ __forceinline__ int64_t kvq_vec(const KvqCacheArg& c, int64_t row, int h) {
    const int64_t page = row >> c.shift;
    return ((page * c.heads + h) << c.shift) + (row & ((1 << c.shift) - 1));
}

// Raises a kernel's dynamic shared-memory limit, once per device (`ready`: the
// kernel's own word of devices done; past 64 of them every time).
template <typename F>
inline cudaError_t layer_smem(F* f, int bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// One launch, with programmatic dependent launch when the flag asks for it.
template <typename F, typename... A>
inline cudaError_t layer_launch(F* f, dim3 grid, int threads, int smem, unsigned flags, cudaStream_t stream,
                                A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (flags & 1u) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    return cudaLaunchKernelEx(&cfg, f, args...);
}

}  // namespace w4a8
