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
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"

namespace {

using namespace pkv_pdl;

// 16 bytes of a type as fp32 values and back
template <typename T>
struct Vec;
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4& w, float (&x)[4])
    {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[4])
    {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
    }
};
template <typename T, typename T2>
struct Vec16 {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4& w, float (&x)[8])
    {
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const T2 h = reinterpret_cast<const T2&>(words[i]);
            x[2 * i] = (float)h.x;
            x[2 * i + 1] = (float)h.y;
        }
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[8])
    {
        uint32_t words[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            T2 h;
            h.x = (T)x[2 * i];
            h.y = (T)x[2 * i + 1];
            words[i] = reinterpret_cast<const uint32_t&>(h);
        }
        return make_uint4(words[0], words[1], words[2], words[3]);
    }
};
template <>
struct Vec<__half> : Vec16<__half, __half2> {};
template <>
struct Vec<__nv_bfloat16> : Vec16<__nv_bfloat16, __nv_bfloat162> {};

// cos and sin of the pair's turn at a position, times the magnitude
__device__ __forceinline__ float2 rotation(int32_t position, int64_t turns, float magnitude,
                                           bool inverse)
{
    const uint64_t turn = (uint64_t)(int64_t)position * (uint64_t)turns;
    float s, c;
    sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
    return make_float2(c * magnitude, (inverse ? -s : s) * magnitude);
}

// A CTA takes a run of one token's units.  A unit is two 16-byte vectors of a head:
// N pairs' elements (rotated), or 2 N elements behind the rotated ones or of a value
// (moved as they are).
template <typename T, int U>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p)
{
    constexpr int N = Vec<T>::N;
    __shared__ float2 turn[kRopeMaxPairs];
    wait_for_previous();
    let_next_start();
    const int64_t t = blockIdx.x / p.chunks;
    const int chunk = (int)(blockIdx.x - t * p.chunks);
    int64_t slot = 0;
    if (p.slots != nullptr) {
        slot = p.slots[t];
        if (slot < 0) return;  // padding
        if (slot >= (int64_t)p.num_blocks * p.block_size) {
            if (threadIdx.x == 0 && chunk == 0) atomicOr(p.status, PKV_STATUS_BAD_SLOT);
            return;
        }
    }
    const int rotated = p.pairs / N;  // units of a head that are
    uint4 a[U], b[U];
    uint4* dst[U];
    int pair[U], step[U];  // pair < 0: moved as it is
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int unit = chunk * p.chunk_units + u * blockDim.x + threadIdx.x;
        dst[u] = nullptr;
        if (u * blockDim.x + threadIdx.x >= p.chunk_units || unit >= p.token_units) continue;
        const int row = unit / p.head_units, j = unit - row * p.head_units;
        const int set = row < p.set[0].end ? 0 : row < p.set[1].end ? 1 : 2;
        const RopeRows& r = p.set[set];
        const int head = row - r.begin;
        const bool turned = r.turned && j < rotated;
        // element of the first vector; elements from it to the second
        const int e = turned && !p.interleaved ? j * N : j * 2 * N;
        const int distance = turned && !p.interleaved ? p.pairs : N;
        pair[u] = turned ? j * N : -1;
        step[u] = distance / N;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(r.src) +
                                                          t * r.src_stride + head * p.head_dim + e);
        a[u] = src[0];
        b[u] = src[step[u]];
        size_t at;
        if (r.cache) {
            const int64_t block = slot / p.block_size;
            at = (size_t)((block * p.num_kv_heads + head) * p.block_size +
                          (slot - block * p.block_size)) * p.head_dim;
        } else {
            at = (size_t)(t * r.dst_stride + head * p.head_dim);
        }
        dst[u] = reinterpret_cast<uint4*>(static_cast<T*>(r.dst) + at + e);
    }
    for (int i = threadIdx.x; i < p.pairs; i += blockDim.x)
        turn[i] = rotation(p.positions[(int64_t)p.axis[i] * p.num_tokens + t], p.turns[i], p.magnitude,
                           p.inverse);
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (dst[u] == nullptr) continue;
        if (pair[u] >= 0) {
            float x[N], y[N];
            Vec<T>::load(a[u], x);
            Vec<T>::load(b[u], y);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 cs = turn[pair[u] + i];
                // the pair's elements: x[i], y[i], or neighbours of x, then of y
                float& first = !p.interleaved ? x[i] : i < N / 2 ? x[2 * i] : y[2 * i - N];
                float& second = !p.interleaved ? y[i] : i < N / 2 ? x[2 * i + 1] : y[2 * i - N + 1];
                const float f = first, g = second;
                first = f * cs.x - g * cs.y;
                second = g * cs.x + f * cs.y;
            }
            a[u] = Vec<T>::store(x);
            b[u] = Vec<T>::store(y);
        }
        dst[u][0] = a[u];
        dst[u][step[u]] = b[u];
    }
}

template <typename T>
cudaError_t launch_typed(RopeParams& p, cudaStream_t stream)
{
    constexpr int U = 2;
    p.head_units = p.head_dim / (2 * Vec<T>::N);
    p.token_units = p.set[2].end * p.head_units;
    p.chunks = (p.token_units + 256 * U - 1) / (256 * U);
    p.chunk_units = (p.token_units + p.chunks - 1) / p.chunks;
    const int threads = ((p.chunk_units + U - 1) / U + 31) / 32 * 32;
    return launch_dependent(rope_kernel<T, U>, (long long)p.num_tokens * p.chunks, threads, 0,
                            stream, p);
}

}  // namespace

cudaError_t launch_rope(RopeParams p, int dtype, cudaStream_t stream)
{
    return dtype == PKV_F32   ? launch_typed<float>(p, stream)
           : dtype == PKV_F16 ? launch_typed<__half>(p, stream)
                              : launch_typed<__nv_bfloat16>(p, stream);
}
