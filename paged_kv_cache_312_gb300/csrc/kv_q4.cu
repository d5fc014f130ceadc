// Writing tokens into the 4-bit cache and reading them back.
//
// A row of head_dim elements is quantised in runs of 64:
//     m = min x,  s = round16((max x - m) / 15),
//     c = floor((x - m) / s + 1/2), held to 0 .. 15 (s = 0: c = 0),
// and an element stands for m + c s.  m is an element of the run, so it is
// exact in the cache's type.  A run that holds a NaN or an infinity stores
// s = m = NaN and reads back as NaN.
#include <cuda_runtime.h>

#include "pkv.h"
#include "pkv_kernels.h"
#include "q4_common.cuh"

namespace {

using namespace pkv_q4;

constexpr int kThreads = 256;
constexpr int kUnroll = 2;  // pairs of tokens a warp has on its way

// Whether a slot lies in the pool (its rows number below 2^31); a slot < 0 is
// padding, one past the pool is flagged.
__device__ __forceinline__ bool inside(int64_t slot, const Q4CacheParams& p)
{
    if (slot < 0) return false;
    if (slot < (int64_t)p.num_blocks * p.block_size) return true;
    atomicOr(p.status, PKV_STATUS_BAD_SLOT);
    return false;
}

__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: added, it rounds to a whole number

// The code of an element d = x - m, whatever the rounding of the reciprocal:
// k = rint(d / s - 1/4) is the code or one less; the residual d - k s, exact as
// k s has 15 bits and lies near d, decides.
__device__ __forceinline__ uint32_t exact_code(float d, float s, float inv)
{
    const float t = fmaf(d, inv, -0.25f) + kMagic;
    const uint32_t c = (__float_as_uint(t) & 31u) +
                       (fmaf(-(t - kMagic), s, d) >= 0.5f * s ? 1u : 0u);
    return min(c, 15u);
}

// Codes (8 nibbles, element e at bits 4e) and the packed (scale, minimum) of
// the 8 elements that this lane holds of a run spread over 8 lanes.
template <typename T>
__device__ __forceinline__ void quantise(const uint4& x, uint32_t& codes, uint32_t& pair)
{
    using H = Half16<T>;
    // (least, -greatest) of the run in one register: one exchange for both
    const uint32_t lo = H::min2(H::min2(x.x, x.y), H::min2(x.z, x.w));
    const uint32_t hi = H::max2(H::max2(x.x, x.y), H::max2(x.z, x.w)) ^ 0x80008000u;
    uint32_t ends = H::min2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) ends = H::min2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
    const float2 e = H::unpack(ends);
    const float m = e.x, range = -e.y - m;
    const float s = H::round(__fdiv_rn(range, 15.f));
    codes = 0u;
    pair = (H::pack(s, 0.f) & 0xFFFFu) | (ends << 16);
    if (!(s >= H::kLeastNormal)) {
        // the range of finite 16-bit values is at most twice the greatest, so a scale that
        // is not finite means an infinity or a NaN in the run (bf16 near the end of
        // fp32's own range overflows the difference, and counts as one)
        if (!(range < INFINITY)) pair = H::kNan | H::kNan << 16;
        if (!(s > 0.f)) return;
        // a scale with few bits may leave codes past 15, and its reciprocal fp32
        constexpr float up = H::kLeastNormal < 1e-30f ? 0x1p100f : 1.f;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = H::unpack(w[i / 2]);
            const float d = ((i & 1 ? v.y : v.x) - m) * up;
            codes |= exact_code(d, s * up, reciprocal(s * up)) << (4 * i);
        }
        return;
    }
    if (!(s < INFINITY)) {
        pair = H::kNan | H::kNan << 16;
        return;
    }
    // rint(d / s), and how far d / s is from it: only near the middle between two
    // codes could the reciprocal's rounding matter, and ties go up.  Codes add
    // up without a carry: a normal scale is at most half a step too small, which
    // takes the greatest element to 15.06.
    const float inv = reciprocal(s);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float off = 0.f;
    uint32_t sum = 0u, magics = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = H::unpack(w[i / 2]);
        const float d = (i & 1 ? v.y : v.x) - m;
        const float t = fmaf(d, inv, kMagic);
        off = fmaxf(off, fabsf(fmaf(d, inv, kMagic - t)));
        sum += __float_as_uint(t) << (4 * i);
        magics += 0x4B400000u << (4 * i);
    }
    codes = sum - magics;
    if (off > 0.5f - 0x1p-16f) {
        codes = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = H::unpack(w[i / 2]);
            codes |= exact_code((i & 1 ? v.y : v.x) - m, s, inv) << (4 * i);
        }
    }
}

// A warp takes kUnroll pairs of tokens 2p, 2p + 1 of the list (lanes 0-15 the
// first of a pair) and 128 elements of each token: one KV head at D = 128, two
// at D = 64.  A CTA's warps take consecutive pairs of the same heads, and the
// CTAs of one stretch of tokens, one a head group, are neighbours.
template <int D>
struct Place {
    static constexpr int CH = D / 8;      // lanes a row
    static constexpr int HPW = 128 / D;   // heads a warp
    unsigned t0;                          // token of the first pair
    int h, c;                             // KV head, 8-element chunk
    __device__ __forceinline__ Place(int head_groups)
    {
        const unsigned stretch = blockIdx.x / (unsigned)head_groups;
        const int lane = threadIdx.x & 31;
        t0 = (stretch * kUnroll * (kThreads / 32) + (threadIdx.x >> 5)) * 2 + (lane >> 4);
        h = (int)(blockIdx.x - stretch * head_groups) * HPW + (lane & 15) / CH;
        c = lane % CH;
    }
    static constexpr unsigned STEP = kThreads / 32 * 2;  // tokens from pair to pair
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
write_kernel(const Q4CacheParams p, const T* __restrict__ key, const T* __restrict__ value,
             size_t key_stride, size_t value_stride, int head_groups)
{
    const Place<D> at(head_groups);
    const int odd = (threadIdx.x >> 4) & 1;
    const bool head = at.h < p.num_kv_heads;
    const int rows = p.block_size * (D / 2);  // bytes of a tile before its pairs
    int64_t slot[kUnroll];
    uint4 kx[kUnroll], vx[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const unsigned t = at.t0 + u * Place<D>::STEP;
        slot[u] = -1;
        kx[u] = vx[u] = make_uint4(0u, 0u, 0u, 0u);
        if (head && t < (unsigned)p.num_tokens) {
            const unsigned row = at.h * D + at.c * 8;
            slot[u] = p.slot_mapping[t];
            kx[u] = *reinterpret_cast<const uint4*>(key + t * key_stride + row);
            vx[u] = *reinterpret_cast<const uint4*>(value + t * value_stride + row);
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        uint32_t kc, vc, kp, vp;
        quantise<T>(kx[u], kc, kp);
        quantise<T>(vx[u], vc, vp);
        // tokens of one V pair: each half warp stores one whole word of both
        const bool live = inside(slot[u], p);
        const uint32_t mine = live ? (uint32_t)slot[u] : 0x80000000u;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 16);
        const uint32_t vo = __shfl_xor_sync(0xffffffffu, vc, 16);
        if (!live) continue;
        const uint32_t block = mine >> p.block_shift, token = mine & (p.block_size - 1);
        const size_t tile = (size_t)(block * p.num_kv_heads + at.h) *
                            (uint32_t)tile_bytes(p.block_size, D);
        uint8_t* kt = static_cast<uint8_t*>(p.k_pool) + tile;
        uint8_t* vt = static_cast<uint8_t*>(p.v_pool) + tile;
        *reinterpret_cast<uint32_t*>(kt + token * (D / 2) + at.c * 4) = kc;
        uint8_t* vrow = vt + (token >> 1) * D + at.c * 8;
        if ((mine ^ other) == 1u && (int)(mine & 1u) == odd) {
            // words 2c (from the even token's lanes) and 2c + 1
            *reinterpret_cast<uint32_t*>(vrow + 4 * odd) =
                odd ? __byte_perm(vo, vc, 0x7632) : __byte_perm(vc, vo, 0x5410);
        } else {
            uint16_t* half = reinterpret_cast<uint16_t*>(vrow) + (token & 1);
            half[0] = (uint16_t)vc;
            half[2] = (uint16_t)(vc >> 16);
        }
        if (at.c % 8 == 0) {
            const uint32_t pairs = rows + (token * (D / kRun) + at.c / 8) * 4;
            *reinterpret_cast<uint32_t*>(kt + pairs) = kp;
            *reinterpret_cast<uint32_t*>(vt + pairs) = vp;
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(const Q4CacheParams p, T* __restrict__ key, T* __restrict__ value, int head_groups)
{
    const Place<D> at(head_groups);
    const bool head = at.h < p.num_kv_heads;
    const int rows = p.block_size * (D / 2);
    int64_t slot[kUnroll];
    uint32_t kc[kUnroll], kp[kUnroll], vp[kUnroll];
    uint2 vw[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const unsigned t = at.t0 + u * Place<D>::STEP;
        slot[u] = head && t < (unsigned)p.num_tokens ? p.slot_mapping[t] : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (!inside(slot[u], p)) {
            slot[u] = -1;
            continue;
        }
        const uint32_t place = (uint32_t)slot[u];
        const uint32_t block = place >> p.block_shift, token = place & (p.block_size - 1);
        const size_t tile = (size_t)(block * p.num_kv_heads + at.h) *
                            (uint32_t)tile_bytes(p.block_size, D);
        const uint8_t* kt = static_cast<const uint8_t*>(p.k_pool) + tile;
        const uint8_t* vt = static_cast<const uint8_t*>(p.v_pool) + tile;
        const uint32_t pairs = rows + (token * (D / kRun) + at.c / 8) * 4;
        kc[u] = *reinterpret_cast<const uint32_t*>(kt + token * (D / 2) + at.c * 4);
        vw[u] = *reinterpret_cast<const uint2*>(vt + (token >> 1) * D + at.c * 8);
        kp[u] = *reinterpret_cast<const uint32_t*>(kt + pairs);
        vp[u] = *reinterpret_cast<const uint32_t*>(vt + pairs);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        if (slot[u] < 0) continue;
        const unsigned t = at.t0 + u * Place<D>::STEP;
        const size_t dst = ((size_t)t * p.num_kv_heads + at.h) * D + at.c * 8;
        *reinterpret_cast<uint4*>(key + dst) = Half16<T>::dequantise(kc[u], kp[u]);
        *reinterpret_cast<uint4*>(value + dst) = Half16<T>::dequantise(
            __byte_perm(vw[u].x, vw[u].y, slot[u] & 1 ? 0x7632 : 0x5410), vp[u]);
    }
}

// CTAs of the head groups (CTAs side by side), and of the whole list.
int head_groups_of(const Q4CacheParams& p, int head_dim)
{
    const int hpw = 128 / head_dim;
    return (p.num_kv_heads + hpw - 1) / hpw;
}

unsigned grid_of(const Q4CacheParams& p, int head_dim)
{
    const int64_t per_cta = 2ll * kUnroll * (kThreads / 32);
    return (unsigned)((p.num_tokens + per_cta - 1) / per_cta * head_groups_of(p, head_dim));
}

template <typename T>
cudaError_t write_typed(const Q4CacheParams& p, const void* key, const void* value,
                        size_t key_stride, size_t value_stride, int head_dim, cudaStream_t stream)
{
    auto kern = head_dim == 128 ? write_kernel<T, 128> : write_kernel<T, 64>;
    kern<<<grid_of(p, head_dim), kThreads, 0, stream>>>(
        p, static_cast<const T*>(key), static_cast<const T*>(value), key_stride, value_stride,
        head_groups_of(p, head_dim));
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_typed(const Q4CacheParams& p, void* key, void* value, int head_dim,
                       cudaStream_t stream)
{
    auto kern = head_dim == 128 ? read_kernel<T, 128> : read_kernel<T, 64>;
    kern<<<grid_of(p, head_dim), kThreads, 0, stream>>>(p, static_cast<T*>(key),
                                                        static_cast<T*>(value),
                                                        head_groups_of(p, head_dim));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_write_q4(const Q4CacheParams& p, const void* key, const void* value,
                               size_t key_stride, size_t value_stride, int head_dim, int dtype,
                               cudaStream_t stream)
{
    return dtype == PKV_F16 ? write_typed<__half>(p, key, value, key_stride, value_stride, head_dim,
                                                  stream)
                            : write_typed<__nv_bfloat16>(p, key, value, key_stride, value_stride,
                                                         head_dim, stream);
}

cudaError_t launch_kv_read_q4(const Q4CacheParams& p, void* key, void* value, int head_dim,
                              int dtype, cudaStream_t stream)
{
    return dtype == PKV_F16 ? read_typed<__half>(p, key, value, head_dim, stream)
                            : read_typed<__nv_bfloat16>(p, key, value, head_dim, stream);
}
