// pa_rows.cuh -- helpers of the kernels that take rows of head_dim elements
// apart over a warp's lanes: chunks of 8 elements, sums over lanes, asynchronous
// copies to shared memory.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kChunk = 8;  // elements a lane holds

// Raw bits of one chunk.
template <typename T>
struct Chunk;

template <>
struct Chunk<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = a; }
    // elements 0..3 at p, 4..7 at q
    __device__ __forceinline__ void load(const __nv_bfloat16* p, const __nv_bfloat16* q) {
        const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(q);
        a = make_uint4(x.x, x.y, y.x, y.y);
    }
    __device__ __forceinline__ void store(__nv_bfloat16* p, __nv_bfloat16* q) const {
        *reinterpret_cast<uint2*>(p) = make_uint2(a.x, a.y);
        *reinterpret_cast<uint2*>(q) = make_uint2(a.z, a.w);
    }
    __device__ __forceinline__ void to_f32(float (&x)[kChunk]) const {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo_to_f32(w[i]);
            x[2 * i + 1] = bf16_hi_to_f32(w[i]);
        }
    }
    __device__ __forceinline__ void from_f32(const float (&x)[kChunk]) {
        a.x = pack_bf16x2(x[0], x[1]);
        a.y = pack_bf16x2(x[2], x[3]);
        a.z = pack_bf16x2(x[4], x[5]);
        a.w = pack_bf16x2(x[6], x[7]);
    }
};

template <>
struct Chunk<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) { load(p, p + 4); }
    __device__ __forceinline__ void store(float* p) const { store(p, p + 4); }
    __device__ __forceinline__ void load(const float* p, const float* q) {
        a = *reinterpret_cast<const float4*>(p);
        b = *reinterpret_cast<const float4*>(q);
    }
    __device__ __forceinline__ void store(float* p, float* q) const {
        *reinterpret_cast<float4*>(p) = a;
        *reinterpret_cast<float4*>(q) = b;
    }
    __device__ __forceinline__ void to_f32(float (&x)[kChunk]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void from_f32(const float (&x)[kChunk]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
};

// log2 of a block size (8, 16 or 32): 64-bit divisions by it are a hundred
// cycles of a chain that takes a few thousand.
__device__ __forceinline__ int block_shift(int block_size) { return __popc(block_size - 1); }

// Minimum and maximum that keep a NaN of either side.
__device__ __forceinline__ float min_nan(float x, float y) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// Sums over the LANES lanes of an aligned lane group of N values each
// (N a power of two), left spread over the lanes: afterwards lane x of the
// group holds the sums of values x * N / LANES + i in v[i], i < N / LANES, or,
// where N < LANES, of value x * N / LANES in v[0] (the same in LANES / N lanes).
// About N shuffles instead of N log2(LANES).
template <int N, int LANES>
__device__ __forceinline__ void reduce_scatter(float (&v)[N]) {
    int n = N;
#pragma unroll
    for (int m = LANES / 2; m; m >>= 1) {
        if (n > 1) {
            n >>= 1;
            const bool upper = threadIdx.x & m;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i < n) {
                    const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
}

// 16 bytes from global to shared memory without a register, past L1; zeros
// without a read where `in` is false.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
}  // namespace pa
