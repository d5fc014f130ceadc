// Writing tokens into the 4-bit cache and reading them back.
//
// A row of head_dim elements is quantised in runs of 64:
//     m = min x,  s = round16((max x - m) / 15),
//     c = floor((x - m) / s + 1/2), held to 0 .. 15 (s = 0: c = 0),
// and an element stands for m + c s.  m is an element of the run, so it is
// exact in the cache's type.  A run that holds a NaN or an infinity stores
// s = m = NaN and reads back as NaN.
//
// Both directions move 2 + 9/16 bytes an element.  32768 tokens of 8 heads of 128
// (172 MB): the write takes 33 us (5.2 TB/s; a copy reaches 6.8), bound by
// instruction issue, the read 27 us (6.3 TB/s).  A lane has 16 elements: with 8 a
// lane the pair's exchanges and the addresses weighed twice as much (write and read
// back 71 us against 63 at the time).
#include <cuda_runtime.h>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"
#include "q4_common.cuh"

namespace {

using namespace pkv_q4;
using namespace pkv_pdl;

constexpr int kThreads = 256;

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

// An element's d = x - m, rounded down: the difference of 16-bit values may need
// more than 24 bits (an x far below m), but the middles between codes do not, so
// d lies below one if x - m does.
template <typename H>
__device__ __forceinline__ float above(uint32_t w, int odd, float m)
{
    const float2 v = H::unpack(w);
    return __fsub_rd(odd ? v.y : v.x, m);
}

// The code of d, whatever the rounding of the reciprocal: k = rint(d / s - 1/4)
// is the code or one less; the residual d - k s, exact as k s has 15 bits and
// lies near d, decides.
__device__ __forceinline__ uint32_t exact_code(float d, float s, float inv)
{
    const float t = fmaf(d, inv, -0.25f) + kMagic;
    const uint32_t c = (__float_as_uint(t) & 31u) +
                       (fmaf(-(t - kMagic), s, d) >= 0.5f * s ? 1u : 0u);
    return min(c, 15u);
}

// The 16 elements that a lane holds of a run spread over four lanes: their codes
// (nibble e of codes[k] for element e of x[k]) and the run's packed (scale,
// minimum).
template <typename T>
__device__ __forceinline__ void quantise(const uint4 (&x)[2], uint32_t (&codes)[2], uint32_t& pair)
{
    using H = Half16<T>;
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    // (least, -greatest) of the run in one register: one exchange for both
    uint32_t lo = w[0], hi = w[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = H::min2(lo, w[i]);
        hi = H::max2(hi, w[i]);
    }
    hi ^= 0x80008000u;
    uint32_t ends = H::min2(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) ends = H::min2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
    const float2 e = H::unpack(ends);
    const float m = e.x, range = -e.y - m;
    const float s = H::round(__fdiv_rn(range, 15.f));
    codes[0] = codes[1] = 0u;
    pair = (H::pack(s, 0.f) & 0xFFFFu) | (ends << 16);
    if (!(s >= H::kLeastNormal)) {
        // the range of finite 16-bit values is at most twice the greatest, so a scale that
        // is not finite means an infinity or a NaN in the run (bf16 near the end of
        // fp32's own range overflows the difference, and counts as one)
        if (!(range < INFINITY)) pair = H::kNan | H::kNan << 16;
        if (!(s > 0.f)) return;
        // a scale with few bits may leave codes past 15, and its reciprocal fp32
        constexpr float up = H::kLeastNormal < 1e-30f ? 0x1p100f : 1.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            codes[i / 8] |= exact_code(above<H>(w[i / 2], i & 1, m) * up, s * up,
                                       reciprocal(s * up)) << (4 * (i % 8));
        return;
    }
    if (!(s < INFINITY)) {
        pair = H::kNan | H::kNan << 16;
        return;
    }
    // k = rint(d / s) with a reciprocal too large by more than its error (2^-21
    // against 1.5 * 2^-23): ties go up, k is never too small, and where it is one
    // too large the residual d - k s, exact as k s has 15 bits and lies near d, is
    // below -s / 2.  That is rare, but ties are not: bf16 values and scales meet in
    // them often (taking all elements near a tie the slow way: 48 us against 33 for
    // 32768 tokens of 8 heads).
    // Codes add up without a carry: a normal scale is at most half a step too
    // small, which takes the greatest element to 15.06.
    const float inv = reciprocal(s), more = fmaf(inv, 0x1p-21f, inv);
    float low = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t sum = 0u, magics = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = above<H>(w[4 * k + i / 2], i & 1, m);
            const float t = fmaf(d, more, kMagic);
            low = fminf(low, fmaf(kMagic - t, s, d));
            sum += __float_as_uint(t) << (4 * i);
            magics += 0x4B400000u << (4 * i);
        }
        codes[k] = sum - magics;
    }
    if (low < -0.5f * s) {
        codes[0] = codes[1] = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i)
            codes[i / 8] |= exact_code(above<H>(w[i / 2], i & 1, m), s, inv) << (4 * (i % 8));
    }
}

// Work is cut into (pair of tokens 2p, 2p + 1 of the list, KV head), heads
// fastest; 2 * D / 16 lanes take one, lanes 0-15 of a warp the first tokens and
// lanes 16-31 the second ones.  A lane has 16 elements of a run, 8j .. 8j + 7
// and 32 further on (j < 4), so that four lanes' 16-byte accesses are 64 bytes
// in a row.  A warp has U such stretches on its way.
template <int D>
struct Place {
    static constexpr int CH = D / 16;      // lanes a row
    static constexpr int UPW = 16 / CH;    // units a warp
    unsigned t;                            // token of the list
    int h;                                 // KV head
    bool live;
    __device__ __forceinline__ Place(const Q4CacheParams& p, int stretch)
    {
        const int lane = threadIdx.x & 31;
        const unsigned unit =
            (stretch * (kThreads / 32) + (threadIdx.x >> 5)) * UPW +
            (lane & 15) / CH;
        const unsigned pair = unit / (unsigned)p.num_kv_heads;
        t = 2 * pair + (lane >> 4);
        h = (int)(unit - pair * p.num_kv_heads);
        live = t < (unsigned)p.num_tokens;
    }
};

template <typename T, int D, int U>
__global__ void __launch_bounds__(kThreads)
write_kernel(const Q4CacheParams p, const T* key, const T* value, size_t key_stride,
             size_t value_stride)
{
    wait_for_previous();
    let_next_start();
    const int odd = (threadIdx.x >> 4) & 1;
    const int r = threadIdx.x % Place<D>::CH / 4, j = threadIdx.x % 4;  // run, place in it
    int64_t slot[U];
    int head[U];
    uint4 kx[U][2], vx[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const Place<D> at(p, blockIdx.x * U + u);
        slot[u] = -1;
        head[u] = at.h;
        kx[u][0] = kx[u][1] = vx[u][0] = vx[u][1] = make_uint4(0u, 0u, 0u, 0u);
        if (at.live) {
            const unsigned row = at.h * D + r * kRun + j * 8;
            slot[u] = p.slot_mapping[at.t];
            const uint4* k = reinterpret_cast<const uint4*>(key + at.t * key_stride + row);
            const uint4* v = reinterpret_cast<const uint4*>(value + at.t * value_stride + row);
            kx[u][0] = k[0];
            kx[u][1] = k[4];
            vx[u][0] = v[0];
            vx[u][1] = v[4];
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        uint32_t kc[2], vc[2], kp, vp;
        quantise<T>(kx[u], kc, kp);
        quantise<T>(vx[u], vc, vp);
        // tokens of one V pair: the lanes of each store two whole words of both
        const bool live = inside(slot[u], p);
        const uint32_t mine = live ? (uint32_t)slot[u] : 0x80000000u;
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 16);
        const uint32_t vo = __shfl_xor_sync(0xffffffffu, vc[odd ^ 1], 16);
        if (!live) continue;
        const uint32_t block = mine >> p.block_shift, token = mine & (p.block_size - 1);
        const size_t tile = (size_t)(block * p.num_kv_heads + head[u]) *
                            (uint32_t)tile_bytes(p.block_size, D);
        uint8_t* kt = static_cast<uint8_t*>(p.k_pool) + tile;
        uint8_t* vt = static_cast<uint8_t*>(p.v_pool) + tile;
        uint32_t* krow = reinterpret_cast<uint32_t*>(kt + token * (D / 2) + r * 32) + j;
        krow[0] = kc[0];
        krow[4] = kc[1];
        uint8_t* vrow = vt + (token >> 1) * D + r * 64 + j * 8;
        if ((mine ^ other) == 1u && (int)(mine & 1u) == odd) {
            // the words of x[0] (by the even token's lanes) and of x[1]
            const uint32_t even = odd ? vo : vc[0], odds = odd ? vc[1] : vo;
            *reinterpret_cast<uint2*>(vrow + 32 * odd) =
                make_uint2(__byte_perm(even, odds, 0x5410), __byte_perm(even, odds, 0x7632));
        } else {
            uint16_t* half = reinterpret_cast<uint16_t*>(vrow) + (token & 1);
            half[0] = (uint16_t)vc[0];
            half[2] = (uint16_t)(vc[0] >> 16);
            half[16] = (uint16_t)vc[1];
            half[18] = (uint16_t)(vc[1] >> 16);
        }
        if (j == 0) {
            const uint32_t pairs = p.block_size * (D / 2) + (token * (D / kRun) + r) * 4;
            *reinterpret_cast<uint32_t*>(kt + pairs) = kp;
            *reinterpret_cast<uint32_t*>(vt + pairs) = vp;
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(const Q4CacheParams p, T* key, T* value)
{
    wait_for_previous();
    let_next_start();
    const Place<D> at(p, blockIdx.x);
    const int r = threadIdx.x % Place<D>::CH / 4, j = threadIdx.x % 4;
    if (!at.live) return;
    const int64_t slot = p.slot_mapping[at.t];
    if (!inside(slot, p)) return;
    const uint32_t block = (uint32_t)slot >> p.block_shift;
    const uint32_t token = (uint32_t)slot & (p.block_size - 1);
    const size_t tile = (size_t)(block * p.num_kv_heads + at.h) *
                        (uint32_t)tile_bytes(p.block_size, D);
    const uint8_t* kt = static_cast<const uint8_t*>(p.k_pool) + tile;
    const uint8_t* vt = static_cast<const uint8_t*>(p.v_pool) + tile;
    const uint32_t pairs = p.block_size * (D / 2) + (token * (D / kRun) + r) * 4;
    const uint32_t* krow = reinterpret_cast<const uint32_t*>(kt + token * (D / 2) + r * 32) + j;
    const uint2* vrow = reinterpret_cast<const uint2*>(vt + (token >> 1) * D + r * 64) + j;
    const uint32_t k0 = krow[0], k1 = krow[4];
    const uint2 v0 = vrow[0], v1 = vrow[4];
    const uint32_t kp = *reinterpret_cast<const uint32_t*>(kt + pairs);
    const uint32_t vp = *reinterpret_cast<const uint32_t*>(vt + pairs);
    const size_t dst = ((size_t)at.t * p.num_kv_heads + at.h) * D + r * kRun + j * 8;
    uint4* k = reinterpret_cast<uint4*>(key + dst);
    uint4* v = reinterpret_cast<uint4*>(value + dst);
    const uint32_t sel = token & 1 ? 0x7632u : 0x5410u;
    k[0] = Half16<T>::dequantise(k0, kp);
    k[4] = Half16<T>::dequantise(k1, kp);
    v[0] = Half16<T>::dequantise(__byte_perm(v0.x, v0.y, sel), vp);
    v[4] = Half16<T>::dequantise(__byte_perm(v1.x, v1.y, sel), vp);
}

// CTAs of the list, at `unroll` stretches a warp.
unsigned grid_of(const Q4CacheParams& p, int head_dim, int unroll)
{
    const int64_t units = ((int64_t)p.num_tokens + 1) / 2 * p.num_kv_heads;
    const int64_t per_cta = (int64_t)unroll * (kThreads / 32) * (256 / head_dim);
    return (unsigned)((units + per_cta - 1) / per_cta);
}

// Two stretches a warp once there are CTAs enough to fill every SM several times
// over, one below, where the shorter chain counts.  Two against one, us: 64 CTAs
// 2.8 and 2.0, 1024 5.9 and 5.2, 2048 9.2 and 9.1, 4096 18.3 and 18.9, 8192 33.2 and
// 35.5, 32768 121 and 132; three and four are slower.  The read gains nothing from
// two (34.3 against 34.7 us for 40961 tokens).
constexpr unsigned kWriteOneMost = 16 * 152;

template <typename T, int D>
cudaError_t write_dim(const Q4CacheParams& p, const T* key, const T* value, size_t key_stride,
                      size_t value_stride, cudaStream_t stream)
{
    const unsigned one = grid_of(p, D, 1);
    if (one <= kWriteOneMost)
        return launch_dependent(write_kernel<T, D, 1>, one, kThreads, 0, stream, p, key, value,
                                key_stride, value_stride);
    return launch_dependent(write_kernel<T, D, 2>, grid_of(p, D, 2), kThreads, 0, stream, p, key,
                            value, key_stride, value_stride);
}

template <typename T>
cudaError_t write_typed(const Q4CacheParams& p, const void* key, const void* value,
                        size_t key_stride, size_t value_stride, int head_dim, cudaStream_t stream)
{
    const T *k = static_cast<const T*>(key), *v = static_cast<const T*>(value);
    return head_dim == 128 ? write_dim<T, 128>(p, k, v, key_stride, value_stride, stream)
                           : write_dim<T, 64>(p, k, v, key_stride, value_stride, stream);
}

template <typename T>
cudaError_t read_typed(const Q4CacheParams& p, void* key, void* value, int head_dim,
                       cudaStream_t stream)
{
    auto kern = head_dim == 128 ? read_kernel<T, 128> : read_kernel<T, 64>;
    return launch_dependent(kern, grid_of(p, head_dim, 1), kThreads, 0, stream, p,
                            static_cast<T*>(key), static_cast<T*>(value));
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
