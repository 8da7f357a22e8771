// lb_kv4.cuh -- the 4-bit key/value cache: where a token's codes and scales lie, and the host
// checks its entry points share.
#pragma once
#include "lb_common.cuh"

#include <cuda_bf16.h>

namespace lb {

// Bytes of one chunk (16 tokens of one head) and of its parts.
__host__ __device__ constexpr int kv4_chunk_bytes(int D) { return LB_KV4_CHUNK * (D + 8); }
__host__ __device__ constexpr int kv4_codes_bytes(int D) { return LB_KV4_CHUNK * (D / 2); }
constexpr int kKv4PairBytes = LB_KV4_CHUNK * 4;

// Byte offset of the chunk that holds place `in_page` of `page` for head h.
__device__ __forceinline__ int64_t kv4_chunk_offset(int64_t page, int h, int in_page, int kv_heads,
                                                    int page_shift, int D) {
    return (((page * kv_heads + h) << (page_shift - 4)) + (in_page >> 4)) *
           (int64_t)kv4_chunk_bytes(D);
}

// log2 of a page size the cache can have, or -1.
inline int page_shift_of(int page_size) {
    for (int s = 4; s <= 8; s++)
        if (page_size == 1 << s) return s;
    return -1;
}

inline bool kv4_shape_ok(int64_t pages, int page_size, int kv_heads, int head_dim) {
    return pages >= 1 && pages < (int64_t(1) << 31) && page_shift_of(page_size) > 0 &&
           kv_heads >= 1 && kv_heads <= 16384 && (head_dim == 64 || head_dim == 128);
}

inline bool aligned_to(const void *p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

inline bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && a_bytes && b_bytes && x < y + b_bytes && y < x + a_bytes;
}

// Eight consecutive values of a row as fp32.
__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = *reinterpret_cast<const float4 *>(p);
    const float4 b = *reinterpret_cast<const float4 *>(p + 4);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]),
                                               bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
}

}  // namespace lb
