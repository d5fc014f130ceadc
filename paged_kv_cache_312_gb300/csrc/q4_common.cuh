// The 4-bit cache format, as the kernels see it.
//
// A pool holds, for every physical block and KV head, one tile of
// B * D * 9 / 16 bytes (D = head_dim): B * D / 2 bytes of codes, then for every
// token and every run of 64 elements the pair (scale, minimum) in the cache's
// 16-bit type.  An element stands for minimum + code * scale.
//   K codes: token i's row is D / 2 bytes; element 2b sits in the low half of
//     byte b, element 2b + 1 in its high half.
//   V codes: tokens 2p and 2p + 1 share D bytes of 4-byte words; word j holds
//     elements 4j .. 4j + 3 of token 2p in its low half and those of token
//     2p + 1 in its high half.
// P V multiplies tokens (its k dimension) in pairs, so a V word with one
// element masked out of both halves is an operand register as it stands; a K
// word gives its pairs along head_dim, the k dimension of Q K^T.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstddef>
#include <cstdint>

namespace pkv_q4 {

constexpr int kRun = 64;  // elements that share a scale and a minimum

__host__ __device__ constexpr size_t tile_bytes(int block_size, int head_dim)
{
    return (size_t)block_size * head_dim * 9 / 16;
}

// 16-bit types: the pair of a packed word as floats, and back.
template <typename T>
struct Half16;

template <>
struct Half16<__half> {
    static constexpr uint32_t kNan = 0x7E00u;  // the quiet NaN of no payload
    static constexpr float kLeastNormal = 0x1p-14f;
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float round(float x)
    {
        return __half2float(__float2half_rn(x));
    }
    // element-wise least and greatest; a NaN in either gives NaN
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
    {
        const __half2 r = __hmin2_nan(*reinterpret_cast<const __half2*>(&a),
                                      *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        const __half2 r = __hmax2_nan(*reinterpret_cast<const __half2*>(&a),
                                      *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    // Eight elements m + c s, each rounded once: MAGIC plus a code in the low bits is a
    // whole number of the type, and the multiply-add rounds after the sum.
    static __device__ __forceinline__ uint4 dequantise(uint32_t codes, uint32_t pair)
    {
        const uint32_t ss = __byte_perm(pair, 0u, 0x1010), mm = __byte_perm(pair, 0u, 0x3232);
        const __half2 s2 = *reinterpret_cast<const __half2*>(&ss);
        const __half2 m2 = *reinterpret_cast<const __half2*>(&mm);
        const uint32_t magic = 0x64006400u;  // 1024
        uint32_t r[4];  // elements (i, i + 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = (codes >> (4 * i) & 0x000F000Fu) | magic;
            const __half2 v = __hfma2(__hsub2(*reinterpret_cast<const __half2*>(&c),
                                             *reinterpret_cast<const __half2*>(&magic)), s2, m2);
            r[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                          __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
};

template <>
struct Half16<__nv_bfloat16> {
    static constexpr uint32_t kNan = 0x7FC0u;
    static constexpr float kLeastNormal = 0x1p-100f;  // and whose reciprocal is one of fp32
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ float round(float x)
    {
        return __bfloat162float(__float2bfloat16_rn(x));
    }
    static __device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
    {
        const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                             *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
    // Eight elements m + c s, each rounded once: MAGIC plus a code in the low bits is a
    // whole number of the type, and the multiply-add rounds after the sum.
    static __device__ __forceinline__ uint4 dequantise(uint32_t codes, uint32_t pair)
    {
        const uint32_t ss = __byte_perm(pair, 0u, 0x1010), mm = __byte_perm(pair, 0u, 0x3232);
        const __nv_bfloat162 s2 = *reinterpret_cast<const __nv_bfloat162*>(&ss);
        const __nv_bfloat162 m2 = *reinterpret_cast<const __nv_bfloat162*>(&mm);
        const uint32_t magic = 0x43004300u;  // 128
        uint32_t r[4];  // elements (i, i + 4)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t c = (codes >> (4 * i) & 0x000F000Fu) | magic;
            const __nv_bfloat162 w = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c),
                                             *reinterpret_cast<const __nv_bfloat162*>(&magic));
            const __nv_bfloat162 v = __hfma2(w, s2, m2);
            r[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        return make_uint4(__byte_perm(r[0], r[1], 0x5410), __byte_perm(r[2], r[3], 0x5410),
                          __byte_perm(r[0], r[1], 0x7632), __byte_perm(r[2], r[3], 0x7632));
    }
};

}  // namespace pkv_q4
