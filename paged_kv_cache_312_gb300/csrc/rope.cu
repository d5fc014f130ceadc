// Rotary positions: rows rotated in place or into other rows, and the queries and
// keys of new tokens rotated on their way into the paged cache.
//
// Pair (a, b) of a row of position p becomes
//     (m (a cos t - b sin t), m (b cos t + a sin t)),  t = 2 pi p F / 2^64,
// with F the pair's frequency in units of 2^-64 turns a position: the product p F
// modulo 2^64 is the turn's fraction, exact whatever the position, so that far
// positions lose nothing and no table of angles is read.  Its top 32 bits go to
// sincospif (2^-25 of pi from the float's rounding); the rows are rotated in fp32
// and rounded once.
//
// Memory bounds it: 8192 tokens of 64 heads of 128 (268 MB in 16 bits) take 40.0 us,
// 6.7 TB/s, what a plain copy reaches; 7777 tokens of 64 query and 8 KV heads into
// rows and a cache (319 MB) 51 us, 6.2 TB/s.  The arithmetic is what comes first
// otherwise: with angles read one by one from a row of shared memory (four lanes a
// bank) and scalar multiply-adds the two took 48 and 59 us.  CTAs that live for one
// run of one token's heads, six a SM, beat CTAs that loop over tokens with the next
// one's rows on their way (60 to 75 us, two or three a SM for the registers).  Two units
// a thread against one: 40.0 and 41.1 us, 51 and 57; four: 49 and 65.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"

namespace {

using namespace pkv_pdl;

constexpr int kThreads = 256;

// Two fp32 numbers in a register pair, and what there is of packed arithmetic on them
__device__ __forceinline__ uint64_t pack2(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Two pairs (f, g) turned: f c - g s and g c + f s, cs = (cos, cos, sin, sin)
__device__ __forceinline__ void turn_two(float2& f, float2& g, const float4& cs)
{
    const uint64_t f2 = pack2(f.x, f.y), g2 = pack2(g.x, g.y);
    const uint64_t c = pack2(cs.x, cs.y), s = pack2(cs.z, cs.w);
    f = unpack2(fma2(g2, s ^ 0x8000000080000000ull, mul2(f2, c)));
    g = unpack2(fma2(f2, s, mul2(g2, c)));
}

// The N pairs of two 16-byte vectors x and y, two at a time: x[i] and y[i], or
// (interleaved) neighbours of x, then of y.  cs[k * stride] turns pairs 2k and 2k + 1.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
    static constexpr int N = 4;
    template <bool INTERLEAVED>
    static __device__ __forceinline__ void turn(uint4& x, uint4& y, const float4* cs, int stride)
    {
        float a[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z),
                      __uint_as_float(x.w)};
        float b[4] = {__uint_as_float(y.x), __uint_as_float(y.y), __uint_as_float(y.z),
                      __uint_as_float(y.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float* v = k == 0 ? a : b;
            float2 f = INTERLEAVED ? make_float2(v[0], v[2]) : make_float2(a[2 * k], a[2 * k + 1]);
            float2 g = INTERLEAVED ? make_float2(v[1], v[3]) : make_float2(b[2 * k], b[2 * k + 1]);
            turn_two(f, g, cs[k * stride]);
            if (INTERLEAVED) {
                v[0] = f.x;
                v[1] = g.x;
                v[2] = f.y;
                v[3] = g.y;
            } else {
                a[2 * k] = f.x;
                a[2 * k + 1] = f.y;
                b[2 * k] = g.x;
                b[2 * k + 1] = g.y;
            }
        }
        x = make_uint4(__float_as_uint(a[0]), __float_as_uint(a[1]), __float_as_uint(a[2]),
                       __float_as_uint(a[3]));
        y = make_uint4(__float_as_uint(b[0]), __float_as_uint(b[1]), __float_as_uint(b[2]),
                       __float_as_uint(b[3]));
    }
};
template <typename T>
struct Unit16 {
    static constexpr int N = 8;
    template <bool INTERLEAVED>
    static __device__ __forceinline__ void turn(uint4& x, uint4& y, const float4* cs, int stride)
    {
        uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint32_t& u = INTERLEAVED ? w[2 * k] : w[k];
            uint32_t& v = INTERLEAVED ? w[2 * k + 1] : w[4 + k];
            const float2 a = Unit<T>::unpack(u), b = Unit<T>::unpack(v);
            float2 f = INTERLEAVED ? make_float2(a.x, b.x) : a;
            float2 g = INTERLEAVED ? make_float2(a.y, b.y) : b;
            turn_two(f, g, cs[k * stride]);
            u = INTERLEAVED ? Unit<T>::pack(f.x, g.x) : Unit<T>::pack(f.x, f.y);
            v = INTERLEAVED ? Unit<T>::pack(f.y, g.y) : Unit<T>::pack(g.x, g.y);
        }
        x = make_uint4(w[0], w[1], w[2], w[3]);
        y = make_uint4(w[4], w[5], w[6], w[7]);
    }
};
template <>
struct Unit<__half> : Unit16<__half> {
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return __half22float2(reinterpret_cast<const __half2&>(w));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        const __half2 h = __floats2half2_rn(x, y);
        return reinterpret_cast<const uint32_t&>(h);
    }
};
template <>
struct Unit<__nv_bfloat16> : Unit16<__nv_bfloat16> {
    static __device__ __forceinline__ float2 unpack(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float x, float y)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return reinterpret_cast<const uint32_t&>(h);
    }
};

// cos and sin of the pair's turn at a position, times the magnitude
__device__ __forceinline__ float2 rotation(int32_t position, int64_t turns, float magnitude,
                                           bool inverse)
{
    const uint64_t turn = (uint64_t)(int64_t)position * (uint64_t)turns;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
}

// A unit is two 16-byte vectors of a head: N pairs' elements (rotated), or 2 N elements
// behind the rotated ones or of a value (moved as they are).  A CTA takes a run of one
// token's units, each thread U of them: all its reads are on their way before the
// token's angles are computed.
template <typename T, bool INTERLEAVED, int U>
__global__ void __launch_bounds__(kThreads, 6) rope_kernel(const RopeParams p)
{
    constexpr int N = Unit<T>::N;
    // of pairs 2k and 2k + 1 of each unit of a head: for every k, the units side by side
    __shared__ float4 turn[kRopeMaxPairs / 2];
    const int64_t t = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x - t * p.chunks);
    const int rotated = p.pairs / N;  // units of a head that are
    const uint4* src[U];
    uint4* dst[U];                    // without the slot's place in a cache
    int unit_of[U], step[U];          // unit of the head, < 0: moved as it is
    bool cached[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int at = u * blockDim.x + threadIdx.x, unit = chunk * p.chunk_units + at;
        src[u] = nullptr;
        if (at >= p.chunk_units || unit >= p.token_units) continue;
        const int row = unit / p.head_units, j = unit - row * p.head_units;
        const RopeRows& r = row < p.first.end ? p.first : row < p.second.end ? p.second : p.third;
        const int head = row - r.begin;
        const bool turned = r.turned && j < rotated;
        // element of the first vector; elements from it to the second
        const int e = turned && !INTERLEAVED ? j * N : j * 2 * N;
        unit_of[u] = turned ? j : -1;
        step[u] = turned && !INTERLEAVED ? p.pairs / N : 1;
        cached[u] = r.cache;
        src[u] = reinterpret_cast<const uint4*>(static_cast<const T*>(r.src) + t * r.src_stride +
                                                head * p.head_dim + e);
        const size_t place = r.cache ? (size_t)head * p.block_size * p.head_dim
                                     : (size_t)(t * r.dst_stride + head * p.head_dim);
        dst[u] = reinterpret_cast<uint4*>(static_cast<T*>(r.dst) + place + e);
    }
    wait_for_previous();
    let_next_start();
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (src[u] != nullptr) {
            a[u] = src[u][0];
            b[u] = src[u][step[u]];
        }
    size_t row = 0;  // of a cache, in vectors
    if (p.slots != nullptr) {
        const int64_t slot = p.slots[t];
        if (slot < 0) return;  // padding
        if (slot >= (int64_t)p.num_blocks * p.block_size) {
            if (threadIdx.x == 0 && chunk == 0) atomicOr(p.status, PKV_STATUS_BAD_SLOT);
            return;
        }
        const uint32_t block = (uint32_t)slot / (uint32_t)p.block_size;
        row = ((size_t)block * p.num_kv_heads * p.block_size +
               ((uint32_t)slot - block * (uint32_t)p.block_size)) * (p.head_dim / N);
    }
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
        const float2 cs = rotation(p.positions[(int64_t)p.axis[i] * p.num_tokens + t], p.turns[i],
                                   p.magnitude, p.inverse);
        float* at = reinterpret_cast<float*>(turn + i % N / 2 * rotated + i / N) + i % 2;
        at[0] = cs.x;
        at[2] = cs.y;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (src[u] == nullptr) continue;
        if (unit_of[u] >= 0)
            Unit<T>::template turn<INTERLEAVED>(a[u], b[u], turn + unit_of[u], rotated);
        uint4* to = dst[u] + (cached[u] ? row : 0);
        to[0] = a[u];
        to[step[u]] = b[u];
    }
}

template <typename T>
cudaError_t launch_typed(RopeParams p, cudaStream_t stream)
{
    constexpr int U = 2;
    p.head_units = p.head_dim / (2 * Unit<T>::N);
    p.token_units = p.third.end * p.head_units;
    p.chunks = (p.token_units + kThreads * U - 1) / (kThreads * U);
    p.chunk_units = (p.token_units + p.chunks - 1) / p.chunks;
    const int threads = ((p.chunk_units + U - 1) / U + 31) / 32 * 32;
    const long long grid = (long long)p.num_tokens * p.chunks;
    if (grid >= 1ll << 31) return cudaErrorInvalidConfiguration;
    auto kern = p.interleaved ? rope_kernel<T, true, U> : rope_kernel<T, false, U>;
    return launch_dependent(kern, grid, threads, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int dtype, cudaStream_t stream)
{
    return dtype == PKV_F32   ? launch_typed<float>(p, stream)
           : dtype == PKV_F16 ? launch_typed<__half>(p, stream)
                              : launch_typed<__nv_bfloat16>(p, stream);
}
