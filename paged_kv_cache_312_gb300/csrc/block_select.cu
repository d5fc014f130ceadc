// Block-sparse decode attention: what each block of a context holds at most, and
// which blocks a query attends to.
//
// Bounds: of the keys of a (block, KV head), channel by channel the greatest and the
// least, in 8 bits: 2^e is the least power of two (e >= -50) with every key within
// 127 * 2^e; the greatest is rounded up and the least down, so that
// 2^e * bounds holds every key.
//
// Selection: with a query row in 8 bits in the same way (rounded to nearest),
//     score = 2^eq * 2^e * sum_d (q_d > 0 ? q_d * greatest_d : q_d * least_d)
// bounds q . k over the block's keys; the greatest over the KV head's query heads
// counts.  The sum is a whole number below 2^21 and the factors are powers of two, so
// a score is exact in fp32: which blocks are picked does not depend on an order of
// summation, and equal scores are equal, the lowest block first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"

namespace {

using namespace pkv_pdl;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kLeastExponent = -50, kMostExponent = 50;

__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// The least e >= -50 with most <= 127 * 2^e; above 50 where there is none up to 50
// (a NaN or an infinity among them).  127 / 64 = 1.984375 is 0x7E0000 of the mantissa.
__device__ __forceinline__ int exponent_for(float most)
{
    const int bits = __float_as_int(most);
    const int e = (bits >> 23) - 127 - 6 + ((bits & 0x7FFFFF) > 0x7E0000 ? 1 : 0);
    return max(e, kLeastExponent);
}

template <typename T>
__device__ __forceinline__ float to_float(T x) { return (float)x; }

// ---- bounds ------------------------------------------------------------------

// One warp takes one (sequence, block, KV head); a lane has V channels of every
// ROWS-th token.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) bounds_kernel(const BoundsParams p)
{
    constexpr int V = 16 / sizeof(T);       // elements of a 16-byte load
    constexpr int LANES = D / V < 32 ? D / V : 32;  // lanes of a row
    constexpr int VECS = D / V / LANES;     // loads of a lane for a row
    constexpr int ROWS = 32 / LANES;        // rows that a warp loads at once
    wait_for_previous();
    let_next_start();
    const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int h = (int)(item % p.num_kv_heads);
    const int64_t rest = item / p.num_kv_heads;
    const int j = (int)(rest % p.blocks_each);
    const int64_t s = rest / p.blocks_each;
    if (s >= p.num_seqs) return;
    const int len = p.context_lens[s], fresh = p.new_tokens[s];
    if (fresh <= 0) return;
    const int lane = threadIdx.x & 31;
    if (len < fresh || fresh > p.max_new_tokens ||
        len > (int64_t)p.max_blocks << p.block_shift) {
        if (lane == 0 && h == 0 && j == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        return;
    }
    const int column = ((len - fresh) >> p.block_shift) + j;
    const int held = len - (column << p.block_shift);  // of the context's tokens from here on
    if (held <= 0) return;
    const int block = p.block_tables[s * p.max_blocks + column];
    if (block < 0 || block >= p.num_blocks) {
        if (lane == 0) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        return;
    }
    const int tokens = min(held, p.block_size);
    const size_t tile = (size_t)block * p.num_kv_heads + h;
    const uint4* rows = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_cache) +
                                                       tile * p.block_size * D);
    float hi[VECS][V], lo[VECS][V];
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            hi[v][i] = -INFINITY;
            lo[v][i] = INFINITY;
        }
    bool odd = false;  // a NaN among them
#pragma unroll 4
    for (int t = lane / LANES; t < tokens; t += ROWS)
#pragma unroll
        for (int v = 0; v < VECS; ++v) {
            const uint4 w = rows[t * (D / V) + v * LANES + lane % LANES];
            const T* x = reinterpret_cast<const T*>(&w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float f = to_float(x[i]);
                odd |= f != f;
                hi[v][i] = fmaxf(hi[v][i], f);
                lo[v][i] = fminf(lo[v][i], f);
            }
        }
    float most = 0.f;
#pragma unroll
    for (int v = 0; v < VECS; ++v)
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) {
                hi[v][i] = fmaxf(hi[v][i], __shfl_xor_sync(0xffffffffu, hi[v][i], o));
                lo[v][i] = fminf(lo[v][i], __shfl_xor_sync(0xffffffffu, lo[v][i], o));
            }
            most = fmaxf(most, fmaxf(fabsf(hi[v][i]), fabsf(lo[v][i])));
        }
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const int e = exponent_for(most);
    const bool unbounded = e > kMostExponent || __any_sync(0xffffffffu, odd);
    const float inverse = power_of_two(-(e > kMostExponent ? 0 : e));
    if (lane == 0) p.scales[tile] = unbounded ? INFINITY : power_of_two(e);
    if (lane >= LANES) return;
    int8_t* out = p.bounds + tile * (2 * D);
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
        uint32_t up[V / 4] = {}, down[V / 4] = {};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            int u = __float2int_ru(hi[v][i] * inverse), d = __float2int_rd(lo[v][i] * inverse);
            // a product that underflows still lies above zero, or below
            if (hi[v][i] > 0.f) u = max(u, 1);
            if (lo[v][i] < 0.f) d = min(d, -1);
            if (unbounded) u = d = 0;
            up[i / 4] |= (uint32_t)(u & 255) << (8 * (i % 4));
            down[i / 4] |= (uint32_t)(d & 255) << (8 * (i % 4));
        }
        const int at = (v * LANES + lane) * V;
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            reinterpret_cast<uint32_t*>(out + at)[i] = up[i];
            reinterpret_cast<uint32_t*>(out + D + at)[i] = down[i];
        }
    }
}

// ---- selection ---------------------------------------------------------------

// fp32 in an order that whole numbers have
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

constexpr int kBins = 1024;  // of a histogram over the range that is left
constexpr int kBinBits = 10;

// One CTA takes one (sequence, KV head): the scores of its blocks, the least score
// that is picked, and the picked blocks in ascending order.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p)
{
    constexpr int QUADS = D / 8;   // 16-byte pieces of a tile's bounds
    constexpr int PIECES = QUADS / 4;  // of a lane: four lanes take a tile
    extern __shared__ uint4 smem[];
    int8_t* q8 = reinterpret_cast<int8_t*>(smem);  // [G][q where > 0 | q where < 0]
    const int G = p.num_heads / p.num_kv_heads;
    float* unit = reinterpret_cast<float*>(q8 + G * 2 * D);  // [G]
    __shared__ unsigned hist[kBins];
    __shared__ unsigned part[2][kWarps];
    __shared__ unsigned ends[2], found[2];
    wait_for_previous();
    let_next_start();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = blockIdx.x;
    const int s = (int)(item / p.num_kv_heads), h = (int)(item - (int64_t)s * p.num_kv_heads);
    int len = p.context_lens[s];
    if (len < 0 || len > (int64_t)p.max_blocks << p.block_shift) {
        if (threadIdx.x == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        len = 0;
    }
    const int n = (len + p.block_size - 1) >> p.block_shift;
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
    float* scores = p.scores + item * p.max_blocks;
    int32_t* selected = p.selected + item * p.max_selected;
    const int count = min(n, p.max_selected);
    if (threadIdx.x == 0)  // the context's last block is always among them
        p.selected_lens[item] = n == 0 ? 0 : (count << p.block_shift) -
                                                 ((n << p.block_shift) - len);
    for (int i = count + threadIdx.x; i < p.max_selected; i += kThreads) selected[i] = -1;
    auto emit = [&](int at, int i) {
        const int block = table[i];
        const bool good = block >= 0 && block < p.num_blocks;
        if (!good) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        selected[at] = good ? block * p.num_kv_heads + h : -1;
    };
    if (n <= p.max_selected) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            scores[i] = INFINITY;
            emit(i, i);
        }
        return;
    }
    // q in 8 bits, positive and negative elements apart
    for (int g = warp; g < G; g += kWarps) {
        const T* row = static_cast<const T*>(p.q) +
                       ((int64_t)s * p.num_heads + h * G + g) * D;
        float x[D / 32], most = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = to_float(row[lane + 32 * i]);
            most = fmaxf(most, fabsf(x[i]));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
        const int e = min(exponent_for(most), kMostExponent);
        const float inverse = power_of_two(-e);
        if (lane == 0) unit[g] = power_of_two(e);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            // halves up; what lies above the whole number below is exact near a half
            const float y = x[i] * inverse, whole = floorf(y);
            const int c = max(-127, min(127, __float2int_rn(whole) + (y - whole >= 0.5f ? 1 : 0)));
            q8[g * 2 * D + lane + 32 * i] = (int8_t)max(c, 0);
            q8[g * 2 * D + D + lane + 32 * i] = (int8_t)min(c, 0);
        }
    }
    if (threadIdx.x < 2) ends[threadIdx.x] = threadIdx.x == 0 ? 0xFFFFFFFFu : 0u;
    __syncthreads();

    const int first = p.first_blocks, last = n - p.recent_blocks;  // candidates: [first, last)
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (i < first || i >= last) scores[i] = INFINITY;
    uint32_t least = 0xFFFFFFFFu, greatest = 0u;
    const int sub = lane & 3;
    for (int i0 = first + warp * 8; i0 < last; i0 += kWarps * 8) {
        const int i = i0 + (lane >> 2);
        int block = -1;
        if (i < last) {
            block = table[i];
            if (block < 0 || block >= p.num_blocks) {
                if (sub == 0) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
                block = -1;
            }
        }
        uint4 piece[PIECES];
        float scale = 0.f;
#pragma unroll
        for (int k = 0; k < PIECES; ++k) piece[k] = make_uint4(0u, 0u, 0u, 0u);
        if (block >= 0) {
            const size_t tile = (size_t)block * p.num_kv_heads + h;
            const uint4* t = reinterpret_cast<const uint4*>(p.bounds) + tile * QUADS;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) piece[k] = t[k * 4 + sub];
            scale = p.scales[tile];
        }
        float best = -INFINITY;
        for (int g = 0; g < G; ++g) {
            const uint4* q = smem + g * QUADS;
            int dot = 0;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                const uint4 w = q[k * 4 + sub];
                dot = __dp4a((int)piece[k].x, (int)w.x, dot);
                dot = __dp4a((int)piece[k].y, (int)w.y, dot);
                dot = __dp4a((int)piece[k].z, (int)w.z, dot);
                dot = __dp4a((int)piece[k].w, (int)w.w, dot);
            }
            dot += __shfl_xor_sync(0xffffffffu, dot, 1);
            dot += __shfl_xor_sync(0xffffffffu, dot, 2);
            best = fmaxf(best, (float)dot * unit[g]);
        }
        if (i < last && sub == 0) {
            // a block that is not there is picked last; one without bounds first
            const float score = block < 0 ? -INFINITY : scale < INFINITY ? best * scale : INFINITY;
            scores[i] = score;
            least = min(least, ordered(score));
            greatest = max(greatest, ordered(score));
        }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    greatest = __reduce_max_sync(0xffffffffu, greatest);
    if (lane == 0) {
        atomicMin(&ends[0], least);
        atomicMax(&ends[1], greatest);
    }
    __syncthreads();

    // the least key that is picked, `threshold`, and how many of those equal to it
    const unsigned want = (unsigned)(p.max_selected - p.first_blocks - p.recent_blocks);
    unsigned above = 0, equal = 0;
    uint32_t lo = ends[0], hi = ends[1], threshold = 0xFFFFFFFFu;
    while (want > 0) {
        if (lo == hi) {
            threshold = lo;
            equal = want - above;
            break;
        }
        const int shift = max(0, 32 - __clz(hi - lo) - kBinBits);
        for (int i = threadIdx.x; i < kBins; i += kThreads) hist[i] = 0u;
        __syncthreads();
        for (int i = first + threadIdx.x; i < last; i += kThreads) {
            const uint32_t key = ordered(scores[i]);
            if (key >= lo && key <= hi) atomicAdd(&hist[(key - lo) >> shift], 1u);
        }
        __syncthreads();
        // the bin with the last one wanted, counted from the top
        constexpr int EACH = kBins / kThreads;
        const int top = kBins - 1 - (int)threadIdx.x * EACH;
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < EACH; ++i) mine += hist[top - i];
        unsigned upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) part[0][warp] = upto;
        __syncthreads();
        unsigned before = above + upto - mine;
        for (int w = 0; w < warp; ++w) before += part[0][w];
        if (before < want && before + mine >= want) {
            int bin = top;
            while (before + hist[bin] < want) before += hist[bin--];
            found[0] = (unsigned)bin;
            found[1] = before;
        }
        __syncthreads();
        const unsigned bin = found[0], inside = hist[bin];
        above = found[1];
        lo += bin << shift;
        hi = min(hi, lo + ((1u << shift) - 1u));
        __syncthreads();
        if (inside == want - above || shift == 0) {  // the whole bin, or one key
            threshold = lo;
            equal = inside == want - above ? 0xFFFFFFFFu : want - above;
            break;
        }
    }

    // each warp has a run of blocks: picked for certain, and equal to the threshold
    const int run = (n + kWarps - 1) / kWarps;
    const int begin = min(n, warp * run), end = min(n, begin + run);
    unsigned sure = 0, ties = 0;
    auto kind = [&](int i) {  // 2: picked, 1: equal
        if (i >= end) return 0;
        if (i < first || i >= last) return 2;
        const uint32_t key = ordered(scores[i]);
        return want == 0 ? 0 : key > threshold ? 2 : key == threshold ? 1 : 0;
    };
    for (int i = begin; i < end; i += 32) {
        const int k = kind(i + lane);
        sure += __popc(__ballot_sync(0xffffffffu, k == 2));
        ties += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    if (lane == 0) {
        part[0][warp] = sure;
        part[1][warp] = ties;
    }
    __syncthreads();
    sure = ties = 0;
    for (int w = 0; w < warp; ++w) {
        sure += part[0][w];
        ties += part[1][w];
    }
    const unsigned below = (1u << lane) - 1u;
    for (int i = begin; i < end; i += 32) {
        const int k = kind(i + lane);
        const unsigned picked = __ballot_sync(0xffffffffu, k == 2);
        const unsigned same = __ballot_sync(0xffffffffu, k == 1);
        const unsigned rank = ties + __popc(same & below);
        if (k == 2 || (k == 1 && rank < equal))
            emit((int)(sure + __popc(picked & below) + min(rank, equal)), i + lane);
        sure += __popc(picked);
        ties += __popc(same);
    }
}

template <typename T, int D>
cudaError_t bounds_typed(const BoundsParams& p, cudaStream_t stream)
{
    const long long warps = (long long)p.num_seqs * p.blocks_each * p.num_kv_heads;
    return launch_dependent(bounds_kernel<T, D>, (warps + kWarps - 1) / kWarps, kThreads, 0, stream,
                            p);
}

template <typename T, int D>
cudaError_t select_typed(const SelectParams& p, cudaStream_t stream)
{
    const int smem = p.num_heads / p.num_kv_heads * (2 * D + 4);
    return launch_dependent(select_kernel<T, D>, (long long)p.num_seqs * p.num_kv_heads, kThreads,
                            smem, stream, p);
}

}  // namespace

cudaError_t launch_block_bounds(const BoundsParams& p, int head_dim, int dtype,
                                cudaStream_t stream)
{
    if (head_dim == 128)
        return dtype == PKV_F32   ? bounds_typed<float, 128>(p, stream)
               : dtype == PKV_F16 ? bounds_typed<__half, 128>(p, stream)
                                  : bounds_typed<__nv_bfloat16, 128>(p, stream);
    return dtype == PKV_F32   ? bounds_typed<float, 64>(p, stream)
           : dtype == PKV_F16 ? bounds_typed<__half, 64>(p, stream)
                              : bounds_typed<__nv_bfloat16, 64>(p, stream);
}

cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, int dtype,
                                 cudaStream_t stream)
{
    if (head_dim == 128)
        return dtype == PKV_F32   ? select_typed<float, 128>(p, stream)
               : dtype == PKV_F16 ? select_typed<__half, 128>(p, stream)
                                  : select_typed<__nv_bfloat16, 128>(p, stream);
    return dtype == PKV_F32   ? select_typed<float, 64>(p, stream)
           : dtype == PKV_F16 ? select_typed<__half, 64>(p, stream)
                              : select_typed<__nv_bfloat16, 64>(p, stream);
}
