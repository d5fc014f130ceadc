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

// Where slot `slot` lies: its block and its token in the block; false for
// padding (slot < 0) and for a slot outside the pool, which is flagged.
__device__ __forceinline__ bool locate(int64_t slot, const Q4CacheParams& p, int64_t& block,
                                       int& token)
{
    if (slot < 0) return false;
    if (slot >= (int64_t)p.num_blocks * p.block_size) {
        atomicOr(p.status, PKV_STATUS_BAD_SLOT);
        return false;
    }
    block = slot >> p.block_shift;
    token = (int)(slot & (p.block_size - 1));
    return true;
}

// Codes (8 nibbles, element e at bits 4e) and the packed (scale, minimum) of
// the 8 elements that this lane holds of a run spread over 8 lanes.
template <typename T>
__device__ __forceinline__ void quantise(const uint4& x, uint32_t& codes, uint32_t& pair)
{
    using H = Half16<T>;
    uint32_t lo = H::min2(H::min2(x.x, x.y), H::min2(x.z, x.w));
    uint32_t hi = H::max2(H::max2(x.x, x.y), H::max2(x.z, x.w));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
        lo = H::min2(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = H::max2(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    lo = H::min2(lo, __funnelshift_l(lo, lo, 16));
    hi = H::max2(hi, __funnelshift_l(hi, hi, 16));
    const float m = H::unpack(lo).x, top = H::unpack(hi).x;
    const float range = top - m;
    codes = 0u;
    // top - m of finite 16-bit values: at most twice the greatest, so only an
    // infinity or a NaN in the run gets here (bf16 near the end of fp32's own
    // range overflows the difference, and counts as one)
    if (!(range < INFINITY)) {
        pair = H::kNan | H::kNan << 16;
        return;
    }
    float s = H::round(__fdiv_rn(range, 15.f));
    pair = (H::pack(s, 0.f) & 0xFFFFu) | (lo << 16);
    if (!(s > 0.f)) return;
    // below 2^-100 the reciprocal leaves fp32: such runs are scaled up first
    const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
    s *= up;
    const float inv = __fdiv_rn(1.f, s), half = 0.5f * s;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 v = H::unpack(w[i / 2]);
        const float d = ((i & 1 ? v.y : v.x) - m) * up;
        // k = rint(d / s - 1/4) is the code or one less, whatever the rounding
        // of the reciprocal (adding 1.5 * 2^23 rounds to a whole number); the
        // residual d - k s, exact as k s has 15 bits and lies near d, decides
        const float t = fmaf(d, inv, -0.25f) + 12582912.f;
        const float k = t - 12582912.f;
        const float r = fmaf(-k, s, d);
        const int c = (int)(__float_as_uint(t) & 31u) + (r >= half ? 1 : 0);
        codes |= (uint32_t)min(c, 15) << (4 * i);
    }
}

// One warp takes tokens 2p and 2p + 1 of the list (lanes 0-15 the first) and
// 128 elements of each: one KV head at D = 128, two at D = 64.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
write_kernel(const Q4CacheParams p, const T* __restrict__ key, const T* __restrict__ value,
             size_t key_stride, size_t value_stride)
{
    constexpr int CH = D / 8;        // lanes a row
    constexpr int HPW = 128 / D;     // heads a warp
    const int lane = threadIdx.x & 31;
    const int groups = (p.num_kv_heads + HPW - 1) / HPW;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t pair_index = unit / groups;
    const int t = (int)min(pair_index * 2 + (lane >> 4), (int64_t)p.num_tokens);
    const int h = (int)(unit - pair_index * groups) * HPW + (lane & 15) / CH;
    const int c = lane % CH;
    int64_t block = 0;
    int token = 0;
    bool live = t < p.num_tokens && h < p.num_kv_heads;
    if (live) live = locate(p.slot_mapping[t], p, block, token);
    uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
    if (live) {
        kx = *reinterpret_cast<const uint4*>(key + t * key_stride + h * D + c * 8);
        vx = *reinterpret_cast<const uint4*>(value + t * value_stride + h * D + c * 8);
    }
    uint32_t kc, vc, kp, vp;
    quantise<T>(kx, kc, kp);
    quantise<T>(vx, vc, vp);
    if (!live) return;
    const size_t tile = ((size_t)block * p.num_kv_heads + h) * tile_bytes(p.block_size, D);
    uint8_t* kt = static_cast<uint8_t*>(p.k_pool) + tile;
    uint8_t* vt = static_cast<uint8_t*>(p.v_pool) + tile;
    *reinterpret_cast<uint32_t*>(kt + token * (D / 2) + c * 4) = kc;
    uint16_t* vrow = reinterpret_cast<uint16_t*>(vt + (token >> 1) * D) + 4 * c + (token & 1);
    vrow[0] = (uint16_t)vc;
    vrow[2] = (uint16_t)(vc >> 16);
    if (c % 8 == 0) {
        const int at = p.block_size * (D / 2) + (token * (D / kRun) + c / 8) * 4;
        *reinterpret_cast<uint32_t*>(kt + at) = kp;
        *reinterpret_cast<uint32_t*>(vt + at) = vp;
    }
}

// Eight elements from their codes and pair.
template <typename T>
__device__ __forceinline__ uint4 dequantise(uint32_t codes, uint32_t pair)
{
    using H = Half16<T>;
    const float2 sm = H::unpack(pair);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(0x4B000000u | ((codes >> (8 * i)) & 15u)) - 8388608.f;
        const float b = __uint_as_float(0x4B000000u | ((codes >> (8 * i + 4)) & 15u)) - 8388608.f;
        w[i] = H::pack(fmaf(a, sm.x, sm.y), fmaf(b, sm.x, sm.y));
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(const Q4CacheParams p, T* __restrict__ key, T* __restrict__ value)
{
    constexpr int CH = D / 8, HPW = 128 / D;
    const int lane = threadIdx.x & 31;
    const int groups = (p.num_kv_heads + HPW - 1) / HPW;
    const int64_t unit = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t pair_index = unit / groups;
    const int t = (int)min(pair_index * 2 + (lane >> 4), (int64_t)p.num_tokens);
    const int h = (int)(unit - pair_index * groups) * HPW + (lane & 15) / CH;
    const int c = lane % CH;
    int64_t block;
    int token;
    if (t >= p.num_tokens || h >= p.num_kv_heads || !locate(p.slot_mapping[t], p, block, token))
        return;
    const size_t tile = ((size_t)block * p.num_kv_heads + h) * tile_bytes(p.block_size, D);
    const uint8_t* kt = static_cast<const uint8_t*>(p.k_pool) + tile;
    const uint8_t* vt = static_cast<const uint8_t*>(p.v_pool) + tile;
    const int at = p.block_size * (D / 2) + (token * (D / kRun) + c / 8) * 4;
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(kt + token * (D / 2) + c * 4);
    const uint2 vw = *reinterpret_cast<const uint2*>(vt + (token >> 1) * D + c * 8);
    const uint32_t kp = *reinterpret_cast<const uint32_t*>(kt + at);
    const uint32_t vp = *reinterpret_cast<const uint32_t*>(vt + at);
    const uint32_t vc = __byte_perm(vw.x, vw.y, token & 1 ? 0x7632 : 0x5410);
    const size_t dst = ((size_t)t * p.num_kv_heads + h) * D + c * 8;
    *reinterpret_cast<uint4*>(key + dst) = dequantise<T>(kc, kp);
    *reinterpret_cast<uint4*>(value + dst) = dequantise<T>(vc, vp);
}

// CTAs for the list: one warp for every two tokens and 128 elements.
unsigned grid_of(const Q4CacheParams& p, int head_dim)
{
    const int hpw = 128 / head_dim;
    const int64_t warps =
        (int64_t)((p.num_tokens + 1) / 2) * ((p.num_kv_heads + hpw - 1) / hpw);
    return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
}

template <typename T>
cudaError_t write_typed(const Q4CacheParams& p, const void* key, const void* value,
                        size_t key_stride, size_t value_stride, int head_dim, cudaStream_t stream)
{
    auto kern = head_dim == 128 ? write_kernel<T, 128> : write_kernel<T, 64>;
    kern<<<grid_of(p, head_dim), kThreads, 0, stream>>>(
        p, static_cast<const T*>(key), static_cast<const T*>(value), key_stride, value_stride);
    return cudaGetLastError();
}

template <typename T>
cudaError_t read_typed(const Q4CacheParams& p, void* key, void* value, int head_dim,
                       cudaStream_t stream)
{
    auto kern = head_dim == 128 ? read_kernel<T, 128> : read_kernel<T, 64>;
    kern<<<grid_of(p, head_dim), kThreads, 0, stream>>>(p, static_cast<T*>(key),
                                                        static_cast<T*>(value));
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
