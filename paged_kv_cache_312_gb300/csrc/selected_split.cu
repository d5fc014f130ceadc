// Decode attention over selected tiles where there are few (sequence, KV head) items and
// the caller allows a split: a cluster of CTAs takes an item, each warp every so many-th
// stage of 16 tokens, and the partial results meet in distributed shared memory, without
// a work plan, a workspace or a second launch.
//
//     out = sum_i softmax_i(scale q . k_i) v_i
//
// with the running maximum and sum of each warp's tokens in fp32 (base 2), joined by
// 2^(m - M).  Every operand goes from memory to the registers it is used from, 16 bytes
// at a time.  q . k has query heads as rows and tokens as columns; its channels may be
// summed in any order, so a lane's 16-byte piece of a key is its part of two of the MMA's
// steps, with q's elements laid out the same.  Its result is what v . p (channels by
// query heads) takes as its second operand; the first one's pairs of tokens are put
// together by one instruction each.  The weights are two 16-bit numbers each, rounded
// and remainder (16 bits or more in all, as the MMA takes no wider ones with 16-bit values):
// an fp32 output of bf16 rows is 1.7e-6 off the 64-bit one (2-norms), 4e-7 with fp32 weights.
//
// Waits bound it, not memory: with eight sequences of 8 KV heads and 2048 tokens (67 MB,
// 18.0 us, 3.7 TB/s; 18.8 where they lie scattered over pools of 1.3 GB) an SM has seven
// warps, which issue a fifth of the time; the start (length, blocks, first stage) and the
// two joins are 4 us.  Three stages of 8 KB a warp and two CTAs an SM: with two stages and
// three CTAs 21.8 us (clusters of seven, to fill those, 26.6: a GPC holds few of them), with
// six and one 24.3, with a stage of keys and values in registers 23.4.  Two sums for each
// half of a stage's scores or one, the weights' remainders at once or apart: no difference.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"
#include "tc_common.cuh"

namespace {

using namespace pkv_pdl;
using namespace pkv_tc;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kHeads = 8;        // query heads of a KV head, at most
constexpr int kMostStages = 16;  // of a warp, at most

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy_if(uint4* to, const void* from, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from),
                 "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// A stage: 16 tokens of K and V, in 16-byte pieces.  A lane copies the pieces that it will
// use into places of its own, a ring of STAGES stages a warp.
template <int D>
struct Ring {
    static constexpr int KP = D / 32;  // pieces of a key row, a lane's
    static constexpr int VP = D / 64;  // of a value row
    static constexpr int PIECES = 2 * KP + 4 * VP;
    static constexpr int STAGES = 3;
    static constexpr int WARP = STAGES * PIECES * 32;  // uint4 of a warp
    static constexpr int BYTES = kWarps * WARP * 16;
    static constexpr int ROW = D + 4;  // floats of a head's partial result, over the ring
    static_assert(kHeads * ROW <= WARP * 4, "partial results fit the ring");
};

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address of CTA rank's copy of what lies at `local`
__device__ __forceinline__ uint32_t remote(const void* local, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(rank));
    return r;
}

// weight of a state with maximum m beside one with maximum `most`
__device__ __forceinline__ float weight(float m, float most)
{
    return ex2(m - (most == -INFINITY ? 0.f : most));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2) selected_split_kernel(const DecodeParams p,
                                                                     const int ways)
{
    using R = Ring<D>;
    constexpr int KP = R::KP, VP = R::VP, NS = R::STAGES, UNITS = D / 4;
    extern __shared__ __align__(16) uint4 smem[];
    __shared__ float2 state[kWarps][kHeads], joined[kHeads];  // maximum, sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = lane >> 2, col = lane & 3;  // of the MMAs' operands
    const int item = blockIdx.x / ways, rank = blockIdx.x - item * ways;
    const int G = p.num_heads, B = p.block_size;
    const int shift = B == 8 ? 3 : B == 16 ? 4 : 5;
    const int32_t* table = p.block_tables + (size_t)item * p.max_blocks;
    const T* keys = static_cast<const T*>(p.k_cache);
    const T* values = static_cast<const T*>(p.v_cache);
    uint4* ring = smem + warp * R::WARP + lane;
    const int first = rank * kWarps + warp, step = ways * kWarps;  // the warp's stages
    wait_for_previous();
    let_next_start();
    // blocks of the halves of the warp's stages, a lane's one, whatever the length will be
    int ids[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int at = ((first + lane * step) * 16 + 8 * h) >> shift;
        ids[h] = lane < kMostStages && at < p.max_blocks ? table[at] : -1;
    }
    uint32_t q[KP][4];
#pragma unroll
    for (int i = 0; i < KP; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            q[i][j] = row < G ? reinterpret_cast<const uint32_t*>(
                                    p.q)[((size_t)item * G + row) * (D / 2) + 4 * (col + 4 * i) + j]
                              : 0u;
    int len = p.context_lens[item];
    if (len < 0 || len > (int64_t)p.max_blocks << shift) {
        if (threadIdx.x == 0 && rank == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        len = 0;
    }
    const int stages = (len + 15) >> 4;
    const int count = stages > first ? (stages - first + step - 1) / step : 0;
    unsigned good = 0;  // two bits a slot: whether the halves' blocks are there
    auto copy_stage = [&](int j, int slot) {
        if (j < count) {
            const int token0 = (first + j * step) * 16;
            int block[2];
            unsigned bits = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                block[h] = __shfl_sync(0xffffffffu, ids[h], j);
                if (block[h] >= 0 && block[h] < p.num_blocks)
                    bits |= 1u << h;
                else if (lane == 0 && token0 + 8 * h < len)
                    atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
            }
            good = (good & ~(3u << 2 * slot)) | bits << 2 * slot;
            uint4* to = ring + slot * R::PIECES * 32;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int token = token0 + 8 * h + row;
                const bool ok = token < len && (bits >> h & 1);
                const T* from =
                    keys + (ok ? (((size_t)block[h] << shift) + (token & (B - 1))) * D + 8 * col
                               : 0);
#pragma unroll
                for (int i = 0; i < KP; ++i) copy_if(to + (h * KP + i) * 32, from + 32 * i, ok);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int token = token0 + 8 * (r >> 1) + 2 * col + (r & 1);
                const bool ok = token < len && (bits >> (r >> 1) & 1);
                const T* from =
                    values + (ok ? (((size_t)block[r >> 1] << shift) + (token & (B - 1))) * D +
                                       8 * row
                                 : 0);
#pragma unroll
                for (int i = 0; i < VP; ++i)
                    copy_if(to + (2 * KP + r * VP + i) * 32, from + 64 * i, ok);
            }
        }
        copies_commit();
    };
    float most = -INFINITY, sum = 0.f;  // of the row; of the lane's tokens
    float o[VP][4][4] = {};  // channel 8 (row + 8 i) + 2 j (+ 1) of heads 2 col, 2 col + 1
#pragma unroll
    for (int j = 0; j < NS - 1; ++j) copy_stage(j, j);
    int slot = 0, free = NS - 1;
    for (int j = 0; j < count; ++j) {
        copy_stage(j + NS - 1, free);
        copies_wait<NS - 1>();
        const uint4* from = ring + slot * R::PIECES * 32;
        const unsigned ok = good >> 2 * slot & 3u;
        free = slot;
        slot = slot == NS - 1 ? 0 : slot + 1;
        // two sums for each half, as one would wait for the MMA before; their last two
        // elements, of rows past the heads, stay 0
        float x[2][4] = {}, y[2][4] = {};
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const uint32_t a[4] = {q[i][0], 0u, q[i][1], 0u}, b[4] = {q[i][2], 0u, q[i][3], 0u};
            const uint4 k = from[i * 32], l = from[(KP + i) * 32];
            Mma<T>::run(x[0], a, k.x, k.y);
            Mma<T>::run(x[1], a, l.x, l.y);
            Mma<T>::run(y[0], b, k.z, k.w);
            Mma<T>::run(y[1], b, l.z, l.w);
        }
        float top = -INFINITY;
        const int left = len - (first + j * step) * 16;  // tokens from the stage on
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const bool live = (ok >> h & 1) && 8 * h + 2 * col + c < left;
                x[h][c] = live ? (x[h][c] + y[h][c]) * p.scale_log2 : -INFINITY;
                top = fmaxf(top, x[h][c]);
            }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if (__any_sync(0xffffffffu, top > most)) {
            const float now = fmaxf(top, most), w = weight(most, now);
            most = now;
            sum *= w;
            const float even = __shfl_sync(0xffffffffu, w, 8 * col);
            const float odd = __shfl_sync(0xffffffffu, w, 8 * col + 4);
#pragma unroll
            for (int i = 0; i < VP; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    o[i][c][0] *= even;
                    o[i][c][1] *= odd;
                    o[i][c][2] *= even;
                    o[i][c][3] *= odd;
                }
        }
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = weight(x[h][0], most), b = weight(x[h][1], most);
            sum += a + b;
            Mma<T>::split(a, b, hi[h], lo[h]);
        }
#pragma unroll
        for (int i = 0; i < VP; ++i) {
            uint32_t w[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint4 v = from[(2 * KP + r * VP + i) * 32];
                w[r][0] = v.x;
                w[r][1] = v.y;
                w[r][2] = v.z;
                w[r][3] = v.w;
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t a[4] = {__byte_perm(w[0][c], w[1][c], 0x5410),
                                       __byte_perm(w[0][c], w[1][c], 0x7632),
                                       __byte_perm(w[2][c], w[3][c], 0x5410),
                                       __byte_perm(w[2][c], w[3][c], 0x7632)};
                Mma<T>::run(o[i][c], a, hi[0], hi[1]);
                Mma<T>::run(o[i][c], a, lo[0], lo[1]);
            }
        }
    }
    copies_wait<0>();
    __syncwarp();

    // the warps' states, then the CTAs'
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
    if (col == 0) state[warp][row] = make_float2(most, sum);
    // a warp's partial result lies over its own ring
    auto part = [&](int w, int head, int at) {
        return reinterpret_cast<float4*>(reinterpret_cast<float*>(smem + w * R::WARP) +
                                         head * R::ROW + at);
    };
#pragma unroll
    for (int i = 0; i < VP; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                *part(warp, 2 * col + c, 8 * (row + 8 * i) + 2 * j) =
                    make_float4(o[i][j][c], o[i][j][2 + c], o[i][j + 1][c], o[i][j + 1][2 + c]);
    __syncthreads();
    for (int u = threadIdx.x; u < G * UNITS; u += kThreads) {
        const int head = u / UNITS, at = u % UNITS * 4;
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, state[w][head].x);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = weight(state[w][head].x, m);
            const float4 z = *part(w, head, at);
            l += f * state[w][head].y;
            y.x += f * z.x;
            y.y += f * z.y;
            y.z += f * z.z;
            y.w += f * z.w;
        }
        *part(0, head, at) = y;
        if (at == 0) joined[head] = make_float2(m, l);
    }
    cluster_barrier();
    const bool vec = reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
    const int units = G * UNITS, stop = units * (rank + 1) / ways;
    for (int u = units * rank / ways + (int)threadIdx.x; u < stop; u += kThreads) {
        const int head = u / UNITS, at = u % UNITS * 4;
        float m = -INFINITY, l = 0.f;
        for (int r = 0; r < ways; ++r) {
            float x;
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(x) : "r"(remote(&joined[head].x, r)) : "memory");
            m = fmaxf(m, x);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int r = 0; r < ways; ++r) {
            float2 s;
            float4 z;
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(s.x), "=f"(s.y) : "r"(remote(&joined[head], r)) : "memory");
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(z.x), "=f"(z.y), "=f"(z.z), "=f"(z.w)
                         : "r"(remote(part(0, head, at), r)) : "memory");
            const float f = weight(s.x, m);
            l += f * s.y;
            y.x += f * z.x;
            y.y += f * z.y;
            y.z += f * z.z;
            y.w += f * z.w;
        }
        const float inverse = l == 0.f ? 0.f : 1.f / l;  // no tokens: zeros
        store_out4(p.out, (size_t)item * G * D + 4 * u,
                   make_float4(y.x * inverse, y.y * inverse, y.z * inverse, y.w * inverse),
                   p.out_dtype, vec);
    }
    cluster_barrier();  // a CTA's shared memory stays until all have read it
}

template <typename T, int D>
cudaError_t launch_typed(const DecodeParams& p, int ways, cudaStream_t stream)
{
    const cudaError_t e = cudaFuncSetAttribute(
        selected_split_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::BYTES);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.dynamicSmemBytes = Ring<D>::BYTES;
    cfg.gridDim = dim3((unsigned)(p.num_seqs * ways));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ways;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, selected_split_kernel<T, D>, p, ways);
}

// Clusters of eight CTAs or four; 0: the split launch with a work plan, which is faster where
// - there are more items than clusters that a GPU of 152 SMs holds at once: with two CTAs an SM
//   (head_dim 128) and a cluster in one GPC 36 by eight and 74 by four.  Of 2048 tokens and 4
//   query heads 36 items take 14.8 us and 15.4 with a plan, 38 by eight 19.6 and 15.6, 74 by four
//   22.0 and 21.2, 76 by four 30.3 and 21.4;
// - a warp would have more than 64 KB of keys and values (128 tokens at head_dim 128), with eight
//   CTAs and more than 4 query heads, which a plan's merge through memory takes longer for,
//   128 KB.  In us, with clusters and with a plan of 128 tokens a warp, at head_dim 128:
//     items x tokens   1 x 4096     8 x 4096     32 x 4096    8 x 8192     16 x 8192    32 x 8192
//     1 query head     10.4, 11.9   11.2, 14.1   17.9, 19.8   18.4, 15.1   27.9, 19.7   31.5, 29.2
//     4                10.7, 13.6   11.6, 15.6   18.4, 20.9   18.7, 18.3   28.3, 23.0   31.8, 31.7
//     8                11.1, 16.3   11.9, 18.8   19.0, 23.8   19.2, 23.1   28.7, 28.0   32.3, 36.8
//   What is left of the plan ahead within these limits, where warps have the most tokens: 14 to
//   20 items and 36 to 50, by up to 14 % (their clusters share SMs while others have none; 19 %
//   of 16 to 20 items of 8192 tokens and more than 4 heads, in partitions of 1024); one query
//   head at head_dim 64 and 8192 tokens, by up to 15 %.
// Up to kMostStages a warp, clusters stay ahead of a plan whose partitions give a warp at least
// twice as many tokens: 8 x 8192 in partitions of 512 take 29.4 with a plan, 18.7 here.
constexpr int kMostClusters4 = 74;
constexpr int kMostChannels = 128 * 128;  // tokens of a warp times head_dim

int ways_for(const DecodeParams& p)
{
    if (p.num_seqs > kMostClusters4) return 0;
    const int ways = p.num_seqs <= (p.head_dim == 64 ? 37 : 36) ? 8 : 4;
    const int64_t tokens = (int64_t)p.max_blocks * p.block_size;
    const int64_t each = (tokens + ways * kWarps - 1) / (ways * kWarps);  // of a warp
    if (each > 16 * kMostStages) return 0;
    const bool warp_partitions = p.partition_tokens <= kWarpPartitionMaxTokens &&
                                 p.max_partitions >= kWarpPartitionMinCount;
    const int planned = warp_partitions ? p.partition_tokens : p.partition_tokens / kDecodeTcWarps;
    const int64_t most = p.num_heads > 4 && ways == 8 ? 2 * kMostChannels : kMostChannels;
    return each * p.head_dim <= most || 2 * each <= planned ? ways : 0;
}

}  // namespace

bool selected_split(const DecodeParams& p, int kv_dtype, cudaStream_t stream, cudaError_t* result)
{
    const int ways = ways_for(p);
    if (kv_dtype == PKV_F32 || p.num_heads > kHeads || ways == 0) return false;
    if (kv_dtype == PKV_F16)
        *result = p.head_dim == 128 ? launch_typed<__half, 128>(p, ways, stream)
                                    : launch_typed<__half, 64>(p, ways, stream);
    else
        *result = p.head_dim == 128 ? launch_typed<__nv_bfloat16, 128>(p, ways, stream)
                                    : launch_typed<__nv_bfloat16, 64>(p, ways, stream);
    return true;
}
