// qw_ops.h - operators on caller-owned buffers: cache rows written and read back, the
// attention of drafted-token trees, logits made ready for sampling.  Launch functions take
// arguments that the ABI layer (ops_api.cu) has checked.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "qw.h"
#include "qw_internal.h"

namespace qw {

constexpr int kQGroup = 32;       // elements per scale of an 8-bit cache row
constexpr int kTreeNodesMax = 64; // drafted nodes per sequence: one bit each of a 64-bit mask
constexpr float kOpsLog2e = 1.4426950408889634f;

cudaError_t launch_kv_append(const qw_kv_view &kv, const qw_kv_rows &src, const int32_t *start, const int32_t *count,
                             cudaStream_t st);
cudaError_t launch_kv_read(const qw_kv_view &kv, const qw_kv_rows &dst, const int32_t *start, const int32_t *count,
                           cudaStream_t st);

size_t tree_attn_scratch_bytes(int n_seq, int n_kv_heads, int n_max, int n_heads, int head_dim, int max_len);
// chained: launch with programmatic stream serialization (the previous operation of the stream
// must be a kernel).
cudaError_t launch_tree_attn(const qw_kv_view &kv, const qw_tree_attention_args &a, void *scratch, cudaStream_t st,
                             bool chained = false);

cudaError_t launch_process_logits(const qw_process_logits_args &a, cudaStream_t st);

// Lets kernel K use `bytes` of dynamic shared memory on the current device; CUDA is asked once
// per kernel and device, as the answer does not change and the call costs part of a microsecond.
template <auto K>
cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned bit = dev < 32 ? 1u << dev : 0u;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---------------------------------------------------------------- element conversions

template <typename T>
__device__ __forceinline__ float elem_to_f(T v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(v);
    else return __bfloat162float(v);
}

template <typename T>
__device__ __forceinline__ T elem_from_f(float v) {
    if constexpr (sizeof(T) == 4) return v;
    else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(v);
    else return __float2bfloat16_rn(v);
}

// Eight consecutive elements (16-byte aligned for the 16-bit types, 16-byte halves for f32).
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = *reinterpret_cast<const uint4 *>(p);
        const T *e = reinterpret_cast<const T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = elem_to_f(e[i]);
    }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint4 u;
        T *e = reinterpret_cast<T *>(&u);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = elem_from_f<T>(v[i]);
        *reinterpret_cast<uint4 *>(p) = u;
    }
}

// Eight int8 codes times their group's scale.
__device__ __forceinline__ void load8_q8(const int8_t *codes, float scale, float (&v)[8]) {
    const uint2 u = *reinterpret_cast<const uint2 *>(codes);
    const int8_t *c = reinterpret_cast<const int8_t *>(&u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)c[i] * scale;
}

}  // namespace qw
