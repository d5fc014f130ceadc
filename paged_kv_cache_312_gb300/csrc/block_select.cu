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
// bounds (that row) . k over the block's keys, q . k but for the row's rounding; the
// greatest over the KV head's query heads counts.  The sum is a whole number below 2^21
// and the factors are powers of two, so a score is exact in fp32: which blocks are picked
// does not depend on an order of summation, and equal scores are equal, the lowest block
// first.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
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

// ---- bounds ------------------------------------------------------------------

// 4-byte words of keys: element-wise greatest and least, a NaN in either giving NaN
template <typename T>
struct Words;
template <>
struct Words<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b)
    {
        float r;
        asm("max.NaN.f32 %0, %1, %2;"
            : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(r);
    }
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b)
    {
        float r;
        asm("min.NaN.f32 %0, %1, %2;"
            : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
        return __float_as_uint(r);
    }
    static __device__ __forceinline__ void unpack(uint32_t w, float* x)
    {
        x[0] = __uint_as_float(w);
    }
};
template <typename T2>
struct Pairs {
    static constexpr int N = 2;
    static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t b)
    {
        const T2 r = __hmax2_nan(reinterpret_cast<T2&>(a), reinterpret_cast<T2&>(b));
        return reinterpret_cast<const uint32_t&>(r);
    }
    static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b)
    {
        const T2 r = __hmin2_nan(reinterpret_cast<T2&>(a), reinterpret_cast<T2&>(b));
        return reinterpret_cast<const uint32_t&>(r);
    }
    static __device__ __forceinline__ void unpack(uint32_t w, float* x)
    {
        x[0] = (float)reinterpret_cast<T2&>(w).x;
        x[1] = (float)reinterpret_cast<T2&>(w).y;
    }
};
template <>
struct Words<__half> : Pairs<__half2> {};
template <>
struct Words<__nv_bfloat16> : Pairs<__nv_bfloat162> {};

// Bounds of one tile, a warp's: block `block` of the pool for KV head h, of which the
// context holds `held` tokens or more.  A lane has four words of every ROWS-th token, all
// read before the first is used (up to eight).
template <typename T, int D, int B>
__device__ __forceinline__ void bound_tile(const BoundsParams& p, int block, int h, int held)
{
    using W = Words<T>;
    constexpr int V = 4 * W::N;          // channels of a lane
    constexpr int LANES = D / V;         // lanes of a row
    constexpr int ROWS = 32 / LANES;     // rows that a warp reads at once
    constexpr int READS = B / ROWS;      // reads of a lane
    constexpr int BATCH = READS < 8 ? READS : 8;
    const int lane = threadIdx.x & 31;
    if (block < 0 || block >= p.num_blocks) {
        if (lane == 0) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        return;
    }
    const size_t tile = (size_t)block * p.num_kv_heads + h;
    const uint4* rows = reinterpret_cast<const uint4*>(static_cast<const T*>(p.k_cache) +
                                                       tile * B * D) + lane % LANES;
    // a token past the context stands for its last one
    const int last = min(held, B) - 1;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int first = 0; first < READS; first += BATCH) {
        uint4 w[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            w[i] = rows[min((first + i) * ROWS + lane / LANES, last) * LANES];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                hi[k] = first + i == 0 ? x[k] : W::most(hi[k], x[k]);
                lo[k] = first + i == 0 ? x[k] : W::least(lo[k], x[k]);
            }
        }
    }
    float top[V], bottom[V], most = 0.f;
    bool odd = false;  // a NaN among them
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            hi[k] = W::most(hi[k], __shfl_xor_sync(0xffffffffu, hi[k], o));
            lo[k] = W::least(lo[k], __shfl_xor_sync(0xffffffffu, lo[k], o));
        }
        W::unpack(hi[k], top + k * W::N);
        W::unpack(lo[k], bottom + k * W::N);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        odd |= top[i] != top[i];
        most = fmaxf(most, fmaxf(fabsf(top[i]), fabsf(bottom[i])));
    }
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    const int e = exponent_for(most);
    const bool unbounded = __any_sync(0xffffffffu, odd) || e > kMostExponent;
    const float inverse = unbounded ? 0.f : power_of_two(-e);
    if (lane == 0) p.scales[tile] = unbounded ? INFINITY : power_of_two(e);
    // the first lanes of a row write the greatest, the next ones (or the same) the least
    uint32_t up[V / 4] = {}, down[V / 4] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        int u = __float2int_ru(top[i] * inverse), d = __float2int_rd(bottom[i] * inverse);
        // a product that underflows still lies above zero, or below
        if (top[i] > 0.f) u = max(u, 1);
        if (bottom[i] < 0.f) d = min(d, -1);
        if (unbounded) u = d = 0;
        up[i / 4] |= (uint32_t)(u & 255) << (8 * (i % 4));
        down[i / 4] |= (uint32_t)(d & 255) << (8 * (i % 4));
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(p.bounds + tile * (2 * D)) + lane % LANES * (V / 4);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
        if (lane < LANES) out[i] = up[i];
        if (lane / LANES == (ROWS > 1 ? 1 : 0)) out[D / 4 + i] = down[i];
    }
}

// Blocks of a sequence that hold new tokens; of a bad length none.
template <int B>
__device__ __forceinline__ int blocks_to_bound(const BoundsParams& p, int len, int fresh, bool flag)
{
    if (fresh <= 0) return 0;
    if (len < fresh || fresh > p.max_new_tokens || len > (int64_t)p.max_blocks * B) {
        if (flag) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        return 0;
    }
    return (len - 1) / B - (len - fresh) / B + 1;
}

// A warp for each (sequence, block that new tokens may lie in, KV head).  Four loads that
// wait for one another bound it where there are few, memory else.
template <typename T, int D, int B>
__global__ void __launch_bounds__(kThreads, 6) bounds_kernel(const BoundsParams p)
{
    wait_for_previous();
    let_next_start();
    const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const unsigned rest = item / (unsigned)p.num_kv_heads;
    const int h = (int)(item - rest * p.num_kv_heads);
    const unsigned s = rest / (unsigned)p.blocks_each;
    const int j = (int)(rest - s * p.blocks_each);
    if (s >= (unsigned)p.num_seqs) return;
    const int len = p.context_lens[s], fresh = p.new_tokens[s];
    if (j >= blocks_to_bound<B>(p, len, fresh, j == 0 && h == 0 && (threadIdx.x & 31) == 0)) return;
    const int column = (len - fresh) / B + j;
    bound_tile<T, D, B>(p, p.block_tables[(size_t)s * p.max_blocks + column], h, len - column * B);
}

// The same where most such warps would find no tile: the sequences may have very different
// numbers of new tokens (a prompt among decoding ones).  Each CTA counts the blocks, a thread
// those of every 256th sequence; a warp takes an equal run of the tiles, in the order of the
// threads, their sequences, the blocks and the heads, and finds its first by the counts.
// A block's number is read before the block ahead of it is worked on.  Few CTAs, as each
// counts: three an SM; every block of 64 prompts of 32 KV heads (572 MB) takes 89 us, 6.4 TB/s
// (two 92, four 91, six 99; a second wave of four 89, but 7.9 instead of 5.6 us below).
// 255 sequences of one new token and one of 8192, 8 KV heads, take 6 us, and with a warp for
// each possible tile 134.
template <typename T, int D, int B>
__global__ void __launch_bounds__(kThreads, 3) bounds_many_kernel(const BoundsParams p)
{
    __shared__ unsigned before[kThreads + 1];  // blocks of the threads before
    __shared__ unsigned part[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int share = (p.num_seqs + kThreads - 1) / kThreads;
    wait_for_previous();
    let_next_start();
    unsigned mine = 0;
#pragma unroll 4
    for (int i = 0; i < share; ++i) {
        const int s = i * kThreads + threadIdx.x;
        if (s < p.num_seqs)
            mine += blocks_to_bound<B>(p, p.context_lens[s], p.new_tokens[s], blockIdx.x == 0);
    }
    unsigned upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) part[warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < warp ? part[lane % kWarps] : 0u);
    before[threadIdx.x + 1] = upto;
    if (threadIdx.x == 0) before[0] = 0;
    __syncthreads();
    const unsigned heads = (unsigned)p.num_kv_heads, tiles = before[kThreads] * heads;
    const unsigned part_of = blockIdx.x * kWarps + warp, parts = gridDim.x * kWarps;
    const unsigned end = (unsigned)((uint64_t)tiles * (part_of + 1) / parts);
    unsigned t = (unsigned)((uint64_t)tiles * part_of / parts);
    while (t < end) {
        const unsigned x = t / heads;  // of the blocks
        int at = 0;                    // the last thread with at most x blocks before it
#pragma unroll
        for (int step = kThreads / 2; step > 0; step /= 2)
            if (before[at + step] <= x) at += step;
        // of its sequences the one with block x, 32 at a time
        unsigned j = x - before[at];
        int s, len = 0, fresh = 0;
        for (int i = 0;; i += 32) {
            s = (i + lane) * kThreads + at;
            if (s < p.num_seqs) {
                len = p.context_lens[s];
                fresh = p.new_tokens[s];
            }
            const unsigned blocks = s < p.num_seqs ? blocks_to_bound<B>(p, len, fresh, false) : 0;
            unsigned sum = blocks;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            const unsigned past = __ballot_sync(0xffffffffu, sum > j);
            if (past) {
                const int from = __ffs(past) - 1;
                j -= __shfl_sync(0xffffffffu, sum - blocks, from);
                s = __shfl_sync(0xffffffffu, s, from);
                len = __shfl_sync(0xffffffffu, len, from);
                fresh = __shfl_sync(0xffffffffu, fresh, from);
                break;
            }
            if (i + 32 >= share) return;  // (only if the lengths change meanwhile)
            j -= __shfl_sync(0xffffffffu, sum, 31);
        }
        const int* ids = p.block_tables + (size_t)s * p.max_blocks;
        const int last = (len - 1) / B;
        int column = (len - fresh) / B + (int)j, id = ids[column];
        for (int h = (int)(t - x * heads); t < end && column <= last; ++column, h = 0) {
            const int next = ids[min(column + 1, last)];
            for (; h < p.num_kv_heads && t < end; ++h, ++t)
                bound_tile<T, D, B>(p, id, h, len - column * B);
            id = next;
        }
    }
}

// ---- selection ---------------------------------------------------------------

// Whether a sequence's length fits its table
__device__ __forceinline__ bool fits(int len, const SelectParams& p)
{
    return len >= 0 && len <= (int64_t)p.max_blocks << p.block_shift;
}

// dot += A B: 16 rows and 8 columns of 16 fp16 elements, sums in fp32
__device__ __forceinline__ void mma_f16(float (&dot)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(dot[0]), "+f"(dot[1]), "+f"(dot[2]), "+f"(dot[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void copy_async(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

// Query rows in 8 bits, as fp16 whole numbers: positive elements, then negative ones.
// Rows lie 64 bytes further apart than they are long, so that the MMA's eight heads
// read other banks.
template <int D>
struct QueryRows {
    static constexpr int STRIDE = 2 * D + 32;  // fp16 elements
};

template <int D>
__device__ __forceinline__ void load_query(const void* q, int64_t row, int dtype,
                                           float (&x)[D / 32])
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        const int64_t at = row * D + lane + 32 * i;
        x[i] = dtype == PKV_F32   ? static_cast<const float*>(q)[at]
               : dtype == PKV_F16 ? __half2float(static_cast<const __half*>(q)[at])
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(q)[at]);
    }
}

// One row, a warp's: into `to`, and the terms (2^24 unit, -128 unit sum of q) that turn
// an MMA's sum into q times the bounds, see below.
template <int D>
__device__ __forceinline__ void quantise_query(const float (&x)[D / 32], __half* to, float2* terms)
{
    const int lane = threadIdx.x & 31;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) most = fmaxf(most, fabsf(x[i]));
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    const int e = min(exponent_for(most), kMostExponent);
    const float inverse = power_of_two(-e);
    int sum = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        // halves up; what lies above the whole number below is exact near a half
        const float y = x[i] * inverse, whole = floorf(y);
        const int c = max(-127, min(127, __float2int_rn(whole) + (y - whole >= 0.5f ? 1 : 0)));
        sum += c;
        to[lane + 32 * i] = __int2half_rn(max(c, 0));
        to[D + lane + 32 * i] = __int2half_rn(min(c, 0));
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0)
        *terms = make_float2(power_of_two(24 + e), (float)(-128 * sum) * power_of_two(e));
}

// Scores: a CTA takes every so many-th turn of 64 of the blocks of one (sequence, KV head),
// a warp 16 of them as the rows of an MMA whose columns are 8 HT query heads.  A lane has the
// blocks of row lane / 4 and of row lane / 4 + 8, every fourth 16-byte piece of their
// bounds, and ends with the score of one of the two.  Its pieces come by asynchronous
// copies into places of its own, a turn ahead; their blocks' ids a turn before that.
//
// A bound's byte c, taken as an fp16 number (c + 128) * 2^-24, needs no arithmetic; the
// MMA's sum of whole numbers below 2^22 times 2^-24 is exact, and 128 times the sum of
// q comes off it.  Up to 8 query heads' elements stay in registers.
//
// 64 contexts of up to 32768 tokens, 8 KV heads of 8 query heads (495 thousand tiles,
// 132 MB): 30 us, 4.4 TB/s.  The copies alone take 28 (a plain gather of as many bytes
// 22, by 256 bytes or by 2048), the arithmetic alone 24; issue slots are 37 % busy, loads' latency is what
// warps wait for most.  8-bit MMAs need nothing taken apart, but run at 62 cycles each
// on an SM quarter (16 fp16 ones in 8 each for the same work): 37 us for the call against
// 36.  Without tensor cores (dp4a, 32 instructions for 16 tiles and a query head and
// the sums across lanes) a CTA a row took 97 us.
// Copies of whole rows by the bulk-copy engine in these ones' place: 40 us for the call
// against 36.  A place that is given no block is left alone: one tile read in its stead
// by every CTA made that tile's memory the whole call's bottleneck (65 us).
constexpr int kScoreThreads = 128;
constexpr int kNoCandidate = -2147483647 - 1;  // in place of a block's id

// Bytes of shared memory of score_run, up to the terms' end
template <int D>
__host__ __device__ constexpr int score_bytes(int threads, int group)
{
    return 2 * threads * D + group * (QueryRows<D>::STRIDE * 2 + 8);
}

// Scores of every `ways`-th turn of one (sequence, KV head)'s blocks from the `way`-th on,
// into p.scores and (where there is one) kept.  length() is waited for only once what else
// comes first is on its way; returns what it gives.  Nothing is scored where all blocks
// are picked.
template <int D, int HT, int NT, typename Length>
__device__ __forceinline__ int score_run(const SelectParams& p, uint4* smem, int s, int h,
                                         int way, int ways, float* kept, Length&& length)
{
    constexpr int QUADS = D / 8;       // 16-byte pieces of a tile's bounds
    constexpr int PIECES = QUADS / 4;  // of a lane: four lanes take a tile
    constexpr int NW = NT / 32;
    const int step = ways * (NT / 2);  // blocks from turn to turn
    const int G = p.num_heads / p.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4* places = smem + threadIdx.x;  // [2 turns][2 rows][PIECES][NT]
    __half* query = reinterpret_cast<__half*>(smem + 4 * PIECES * NT);
    float2* terms = reinterpret_cast<float2*>(query + G * QueryRows<D>::STRIDE);
    const int64_t row = (int64_t)s * p.num_heads + (int64_t)h * G;
    float x[D / 32] = {};  // on its way while the length and the first ids are
    if (warp < G) load_query<D>(p.q, row + warp, p.dtype, x);
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
    const int sub = lane & 3, odd = lane & 1;
    auto read_ids = [&](int i0, int from, int to, int (&id)[2]) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = i0 + (lane >> 2) + 8 * r;
            id[r] = i >= from && i < to ? table[i] : kNoCandidate;
        }
    };
    int i0 = way * (NT / 2) + warp * 16, id[2];
    read_ids(i0, 0, p.max_blocks, id);  // whatever the length will be
    const int len = length();
    const int n = (len + p.block_size - 1) >> p.block_shift;
    if (n <= p.max_selected || way * (NT / 2) >= n) return len;
    const int first = p.first_blocks, last = n - p.recent_blocks;  // candidates: [first, last)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        const int i = i0 + (lane >> 2) + 8 * r;
        if (i < first || i >= last) id[r] = kNoCandidate;
    }
    float* scores = p.scores + ((int64_t)s * p.num_kv_heads + h) * p.max_blocks;
    // copies of the two rows' bounds; where no block is, the place keeps what it holds,
    // and the score counts for nothing
    auto is_block = [&](int id) { return id >= 0 && id < p.num_blocks; };
    auto copy_bounds = [&](const int (&id)[2], int turn) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (is_block(id[r])) {
                const uint4* t = reinterpret_cast<const uint4*>(p.bounds) +
                                 (size_t)(id[r] * p.num_kv_heads + h) * QUADS + sub;
#pragma unroll
                for (int k = 0; k < PIECES; ++k)
                    copy_async(places + ((turn * 2 + r) * PIECES + k) * NT, t + 4 * k);
            }
        copies_commit();
    };
    // a lane's own row: its id and, if it is a block, its scale
    auto own_scale = [&](const int (&id)[2], int& mine) {
        mine = odd ? id[1] : id[0];
        return is_block(mine) ? p.scales[mine * p.num_kv_heads + h] : 0.f;
    };
    int mine, next_mine;
    copy_bounds(id, 0);
    float scale = own_scale(id, mine);
    read_ids(i0 + step, first, last, id);
    for (int g = warp; g < G; g += NW) {
        if (g != warp) load_query<D>(p.q, row + g, p.dtype, x);
        quantise_query<D>(x, query + g * QueryRows<D>::STRIDE, terms + g);
    }
    __syncthreads();
    uint4 held[HT == 1 ? 2 * PIECES : 1];
    if constexpr (HT == 1) {
        const uint4* q = reinterpret_cast<const uint4*>(
                             query + min(lane >> 2, G - 1) * QueryRows<D>::STRIDE) + 2 * sub;
#pragma unroll
        for (int k = 0; k < 2 * PIECES; ++k) held[k] = q[8 * (k / 2) + k % 2];
    }
    for (int turn = 0; i0 < n; turn ^= 1, i0 += step) {
        copy_bounds(id, turn ^ 1);
        const float next_scale = own_scale(id, next_mine);
        read_ids(i0 + 2 * step, first, last, id);
        copies_wait<1>();
        float best[2] = {-INFINITY, -INFINITY};
        for (int g0 = 0; g0 < G; g0 += 8 * HT) {
            // column lane / 4 of the MMA's other operand: a query head's elements
            const uint4* q[HT];
            float dot[HT][2][4] = {};
#pragma unroll
            for (int t = 0; t < HT; ++t)
                q[t] = reinterpret_cast<const uint4*>(
                           query + min(g0 + 8 * t + (lane >> 2), G - 1) * QueryRows<D>::STRIDE) +
                       2 * sub;
#pragma unroll
            for (int k = 0; k < PIECES; ++k) {
                const uint4 u = places[(turn * 2 * PIECES + k) * NT];
                const uint4 v = places[((turn * 2 + 1) * PIECES + k) * NT];
                const uint32_t up[4] = {u.x, u.y, u.z, u.w}, down[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint4 w[HT];
#pragma unroll
                    for (int t = 0; t < HT; ++t)
                        w[t] = HT == 1 ? held[2 * k + half] : q[t][8 * k + half];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t a = up[2 * half + j] ^ 0x80808080u;
                        const uint32_t b = down[2 * half + j] ^ 0x80808080u;
                        const uint32_t rows[4] = {
                            __byte_perm(a, 0u, 0x4140), __byte_perm(b, 0u, 0x4140),
                            __byte_perm(a, 0u, 0x4342), __byte_perm(b, 0u, 0x4342)};
#pragma unroll
                        for (int t = 0; t < HT; ++t)
                            mma_f16(dot[t][j], rows, j == 0 ? w[t].x : w[t].z,
                                    j == 0 ? w[t].y : w[t].w);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c) {  // columns past the last head repeat it
                    const float2 f = terms[min(g0 + 8 * t + 2 * sub + c, G - 1)];
                    best[0] = fmaxf(best[0], fmaf(dot[t][0][c] + dot[t][1][c], f.x, f.y));
                    best[1] = fmaxf(best[1], fmaf(dot[t][0][2 + c] + dot[t][1][2 + c], f.x, f.y));
                }
        }
        // odd lanes take the second row, even ones the first
        float score = fmaxf(odd ? best[1] : best[0],
                            __shfl_xor_sync(0xffffffffu, odd ? best[0] : best[1], 1));
        score = fmaxf(score, __shfl_xor_sync(0xffffffffu, score, 2));
        const int i = i0 + (lane >> 2) + 8 * odd;
        if (sub < 2 && i < n) {
            // a block that is not there is picked last; one without bounds first
            // (or with what is no scale)
            // (+ 0: of a scale of zero -0 and 0, which are equal, would have two keys)
            score = scale >= 0.f && scale < INFINITY ? score * scale + 0.f : INFINITY;
            if (mine == kNoCandidate) {
                score = INFINITY;
            } else if (!is_block(mine)) {
                atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
                score = -INFINITY;
            }
            scores[i] = score;
            if (kept != nullptr) kept[i] = score;
        }
        __syncwarp();
        scale = next_scale;
        mine = next_mine;
    }
    copies_wait<0>();
    return len;
}

template <int D, int HT>
__global__ void __launch_bounds__(kScoreThreads, 5) score_kernel(const SelectParams p)
{
    extern __shared__ uint4 smem[];
    const int64_t item = blockIdx.x / p.ways;
    const int way = (int)(blockIdx.x - item * p.ways);
    const int s = (int)(item / p.num_kv_heads), h = (int)(item - (int64_t)s * p.num_kv_heads);
    wait_for_previous();
    let_next_start();
    score_run<D, HT, kScoreThreads>(p, smem, s, h, way, p.ways, nullptr, [&] {
        const int len = p.context_lens[s];
        return fits(len, p) ? len : 0;
    });
}

// fp32 in an order that whole numbers have: infinity is 0xFF800000, -infinity 0x7FFFFF
__device__ __forceinline__ uint32_t ordered(float x)
{
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The picked blocks: a CTA takes one (sequence, KV head).  The least score that is
// picked comes from histograms over a range that narrows by the number of bins a
// round (one or two rounds, mostly); then each warp writes the picked blocks of its run
// of the context behind those of the warps before it.  Latency bounds it: 5 us alone,
// after the scores 6 to 8 with the wait for their end.  One kernel for both, clusters
// of CTAs that read one another's histograms, took 49 us against 36 for 64 contexts of
// up to 32768 and 19 against 13 for one of 131072.
constexpr int kBinsEach = 4;  // histogram bins a thread
constexpr int kFewBlocks = 4 * kScoreThreads;

// A block's key: its score in order, or one of these for a block that is kept whatever
// its score and for none.
constexpr uint32_t kKeptKey = 0xFFFFFFFFu, kNoKey = 0u;

// The range [lo, hi] that is left of the keys and the number above it; at the end the
// threshold that picked keys lie above, and how many of those equal to it are picked.
struct Cut {
    uint32_t lo, hi, threshold;
    unsigned above, equal;
};

template <int NT>
struct Histogram {
    static constexpr int NW = NT / 32;
    static constexpr int BINS = kBinsEach * NT;
    static constexpr int BITS = NT == 1024 ? 12 : NT == 512 ? 11 : NT == 256 ? 10 : 9;
    static constexpr int ROUNDS = (31 + BITS) / BITS;
    static_assert(BINS == 1 << BITS, "NT is 128, 256, 512 or 1024");
    __align__(16) unsigned bins[BINS];
    unsigned part[2][NW];
    unsigned found[3];

    __device__ __forceinline__ void clear()
    {
        reinterpret_cast<uint4*>(bins)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
    }
    // The sums over the warps before this one
    __device__ __forceinline__ void sums_before(unsigned a, unsigned b, unsigned& a_before,
                                                unsigned& b_before)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();
        if (lane == 0) {
            part[0][warp] = a;
            part[1][warp] = b;
        }
        __syncthreads();
        a_before = __reduce_add_sync(0xffffffffu, lane < warp ? part[0][lane % NW] : 0u);
        b_before = __reduce_add_sync(0xffffffffu, lane < warp ? part[1][lane % NW] : 0u);
    }
    // All threads' least and greatest key
    __device__ __forceinline__ void range(uint32_t lo, uint32_t hi, Cut& cut)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (lane == 0) {
            part[0][warp] = lo;
            part[1][warp] = hi;
        }
        __syncthreads();
        cut.lo = __reduce_min_sync(0xffffffffu, part[0][lane % NW]);
        cut.hi = __reduce_max_sync(0xffffffffu, part[1][lane % NW]);
        __syncthreads();
    }
    // The bin with the last key wanted, of bins that hold every key of the range; clears
    // them.  True once the threshold is known.
    __device__ __forceinline__ bool narrow(unsigned want, int shift, Cut& cut)
    {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();
        const int top = BINS - kBinsEach * (1 + (int)threadIdx.x);  // counted from the top
        const uint4 sum = *reinterpret_cast<const uint4*>(bins + top);
        *reinterpret_cast<uint4*>(bins + top) = make_uint4(0u, 0u, 0u, 0u);
        const unsigned each[kBinsEach] = {sum.w, sum.z, sum.y, sum.x};
        const unsigned own = sum.x + sum.y + sum.z + sum.w;
        unsigned upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) part[0][warp] = upto;
        __syncthreads();
        unsigned before = cut.above + upto - own +
                          __reduce_add_sync(0xffffffffu, lane < warp ? part[0][lane % NW] : 0u);
        if (before < want && before + own >= want) {
            int k = 0;
#pragma unroll
            for (int i = 0; i < kBinsEach - 1; ++i)
                if (k == i && before + each[i] < want) {
                    before += each[i];
                    ++k;
                }
            found[0] = (unsigned)(top + kBinsEach - 1 - k);
            found[1] = before;
            found[2] = k == 0 ? each[0] : k == 1 ? each[1] : k == 2 ? each[2] : each[3];
        }
        __syncthreads();
        const unsigned inside = found[2];
        cut.above = found[1];
        cut.lo += found[0] << shift;
        cut.hi = min(cut.hi, cut.lo + ((1u << shift) - 1u));
        if (inside == want - cut.above) {  // the whole bin
            cut.threshold = cut.lo - 1u;
            return true;
        }
        if (shift > 0) return false;
        cut.threshold = cut.lo;  // one key
        cut.equal = want - cut.above;
        return true;
    }
};

__device__ __forceinline__ int shift_for(const Cut& cut, int bits)
{
    return max(0, 32 - __clz(cut.hi - cut.lo) - bits);
}

// The blocks of a context that has more than are picked: PER > 0: a warp's 32 `each` of
// them from `mark`, a lane has every 32nd, their scores (as bits) and ids in key and ids;
// PER = 0: any number, read from memory each time.
template <int NT, int PER>
__device__ __forceinline__ void pick_among(const SelectParams& p, Histogram<NT>& hist, int64_t item,
                                           int h, int n, int each, const float* from,
                                           const int32_t* table, uint32_t* key, const int* ids)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mark = warp * 32 * each;
    int32_t* selected = p.selected + item * p.max_selected;
    auto emit = [&](unsigned at, int block) {
        const bool good = block >= 0 && block < p.num_blocks;
        if (!good) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        // (past the row only if another call writes the scores meanwhile)
        if (at < (unsigned)p.max_selected) selected[at] = good ? block * p.num_kv_heads + h : -1;
    };
    const int first = p.first_blocks, last = n - p.recent_blocks;  // candidates: [first, last)
    const int stop = min(n, mark + 32 * each);  // of the warp's run
    auto key_of = [&](int i, float score) {
        return i >= stop ? kNoKey : i < first || i >= last ? kKeptKey : ordered(score);
    };
    if constexpr (PER > 0) {
#pragma unroll
        for (int u = 0; u < PER; ++u)
            key[u] = u < each ? key_of(mark + 32 * u + lane, __uint_as_float(key[u])) : kNoKey;
    }
    // f(key, id) for the lane's blocks, all lanes of the warp together
    auto for_each = [&](auto&& f) {
        if constexpr (PER > 0) {
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                if (u >= each) break;
                f(key[u], ids[u]);
            }
        } else {
            for (int i0 = mark; i0 < stop; i0 += 128) {
                float x[4];
                int id[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int i = i0 + 32 * u + lane;
                    x[u] = i < stop ? from[i] : 0.f;
                    id[u] = i < stop ? table[i] : 0;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) f(key_of(i0 + 32 * u + lane, x[u]), id[u]);
            }
        }
    };
    // none but kept blocks lie above this threshold
    Cut cut = {0u, 0u, kKeptKey - 1u, 0u, 0u};
    const unsigned want = (unsigned)(p.max_selected - p.first_blocks - p.recent_blocks);
    if (want > 0) {
        uint32_t lo = 0xFFFFFFFFu, hi = 0u;
        for_each([&](uint32_t k, int) {
            if (k - 1u < kKeptKey - 1u) {  // neither kept nor none
                lo = min(lo, k);
                hi = max(hi, k);
            }
        });
        hist.range(lo, hi, cut);
    }
    for (int round = 0; want > 0 && round < Histogram<NT>::ROUNDS; ++round) {
        if (cut.lo == cut.hi) {
            cut.threshold = cut.lo;
            cut.equal = want - cut.above;
            break;
        }
        const int shift = shift_for(cut, Histogram<NT>::BITS);
        const uint32_t span = cut.hi - cut.lo;
        for_each([&](uint32_t k, int) {
            if (k - cut.lo <= span) atomicAdd(&hist.bins[(k - cut.lo) >> shift], 1u);
        });
        if (hist.narrow(want, shift, cut)) break;
    }

    unsigned sure = 0, ties = 0;
    if (cut.equal == 0) {  // the usual case: no equal keys to choose from
        for_each([&](uint32_t k, int) {
            sure += __popc(__ballot_sync(0xffffffffu, k > cut.threshold));
        });
    } else {
        for_each([&](uint32_t k, int) {
            sure += __popc(__ballot_sync(0xffffffffu, k > cut.threshold));
            ties += __popc(__ballot_sync(0xffffffffu, k == cut.threshold));
        });
    }
    hist.sums_before(sure, ties, sure, ties);
    const unsigned below = (1u << lane) - 1u;
    if (cut.equal == 0) {
        for_each([&](uint32_t k, int id) {
            const unsigned picked = __ballot_sync(0xffffffffu, k > cut.threshold);
            if (k > cut.threshold) emit(sure + __popc(picked & below), id);
            sure += __popc(picked);
        });
    } else {
        for_each([&](uint32_t k, int id) {
            const unsigned picked = __ballot_sync(0xffffffffu, k > cut.threshold);
            const unsigned same = __ballot_sync(0xffffffffu, k == cut.threshold);
            const unsigned rank = ties + __popc(same & below);
            if (k > cut.threshold || (k == cut.threshold && rank < cut.equal))
                emit(sure + __popc(picked & below) + min(rank, cut.equal), id);
            sure += __popc(picked);
            ties += __popc(same);
        });
    }
}

// The scores come from `from`; the length from length().  PER blocks a thread are held:
// of a table that is no wider than that (or WIDE is false), read before the length is
// known; of a wider one, those of a context of no more blocks.
template <int NT, int PER, bool WIDE, typename Length>
__device__ __forceinline__ void pick_blocks(const SelectParams& p, Histogram<NT>& hist, int s,
                                            int h, const float* from, Length&& length)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t item = (int64_t)s * p.num_kv_heads + h;
    const int32_t* table = p.block_tables + (int64_t)s * p.max_blocks;
    int32_t* selected = p.selected + item * p.max_selected;
    uint32_t key[PER];
    int ids[PER];
    auto read = [&](int each, int blocks) {
#pragma unroll
        for (int u = 0; u < PER; ++u) {
            const int i = warp * 32 * each + 32 * u + lane;
            const bool there = u < each && i < blocks;
            key[u] = there ? __float_as_uint(from[i]) : 0u;
            ids[u] = there ? table[i] : 0;
        }
    };
    int each = (p.max_blocks + NT - 1) / NT;
    if constexpr (!WIDE) read(each, p.max_blocks);
    const int len = length();
    const int n = (len + p.block_size - 1) >> p.block_shift;
    const int count = min(n, p.max_selected);
    if (threadIdx.x == 0)  // the context's last block is always among them
        p.selected_lens[item] = n == 0 ? 0 : (count << p.block_shift) -
                                                 ((n << p.block_shift) - len);
    for (int i = count + threadIdx.x; i < p.max_selected; i += NT) selected[i] = -1;
    if (n <= p.max_selected) {
        for (int i = threadIdx.x; i < n; i += NT) {
            const int block = table[i];
            const bool good = block >= 0 && block < p.num_blocks;
            if (!good) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
            p.scores[item * p.max_blocks + i] = INFINITY;
            selected[i] = good ? block * p.num_kv_heads + h : -1;
        }
        return;
    }
    if constexpr (WIDE) {
        each = (n + NT - 1) / NT;
        if (each > PER) {
            pick_among<NT, 0>(p, hist, item, h, n, each, from, table, key, ids);
            return;
        }
        read(each, n);
    }
    pick_among<NT, PER>(p, hist, item, h, n, each, from, table, key, ids);
}

__device__ __forceinline__ int checked_length(const SelectParams& p, int s)
{
    const int len = p.context_lens[s];
    if (fits(len, p)) return len;
    if (threadIdx.x == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
    return 0;
}

template <int NT, int PER, bool WIDE>
__global__ void __launch_bounds__(NT) pick_kernel(const SelectParams p)
{
    __shared__ Histogram<NT> hist;
    const int64_t item = blockIdx.x;
    const int s = (int)(item / p.num_kv_heads), h = (int)(item - (int64_t)s * p.num_kv_heads);
    hist.clear();
    wait_for_previous();
    let_next_start();
    pick_blocks<NT, PER, WIDE>(p, hist, s, h, p.scores + item * p.max_blocks,
                               [&] { return checked_length(p, s); });
}

// Both for contexts of at most kFewBlocks blocks: a CTA takes one (sequence, KV head) and
// keeps its scores.  From Python one launch less is 2.5 us of a call; on the GPU the two
// ways are near: 64 contexts of 512 blocks 11.8 us against 13.2 in two kernels, 256 short ones
// 17.6 and 18.2, four of up to 256 blocks 4.9 and 4.5.  With up to 1024 blocks in one
// CTA of 256 threads eight contexts of 1024 took 13.0 against 9.8.
template <int D, int HT>
__global__ void __launch_bounds__(kScoreThreads) select_kernel(const SelectParams p)
{
    extern __shared__ uint4 smem[];
    __shared__ Histogram<kScoreThreads> hist;
    const int64_t item = blockIdx.x;
    const int s = (int)(item / p.num_kv_heads), h = (int)(item - (int64_t)s * p.num_kv_heads);
    float* kept = reinterpret_cast<float*>(
        reinterpret_cast<char*>(smem) +
        score_bytes<D>(kScoreThreads, p.num_heads / p.num_kv_heads));
    hist.clear();
    wait_for_previous();
    let_next_start();
    const int len = score_run<D, HT, kScoreThreads>(p, smem, s, h, 0, 1, kept,
                                                    [&] { return checked_length(p, s); });
    __syncthreads();
    pick_blocks<kScoreThreads, kFewBlocks / kScoreThreads, false>(p, hist, s, h, kept,
                                                                  [&] { return len; });
}

// The counts of CTAs and rows from here on are those of a GPU of 152 SMs; others give the same
// results.
//
// Turns of a score CTA at most (of a full table), what its start takes in turns, CTAs that
// the GPU holds, and the waves of them past which a row gets fewer CTAs of more turns.
// The call in us with 2, 4, 8 and 16 turns: 64 contexts of up to 2048 blocks and 8 KV heads
// 45.6, 37.9, 36.6, 36.5; 16 of 1024 blocks and 32 KV heads 37.0, 34.8, 36.6, 39.0; 32 of 2048
// blocks, 4 KV heads of 16 query heads 37.2, 31.0, 28.3, 28.2.  256 contexts of 94 blocks and 8
// KV heads in tables of 8192 with the limit of waves and without it: 29.6 and 117 (with
// kManyRows' choice), in tables of 512 23.4.
constexpr int kMostTurns = 8;
constexpr int kStartTurns = 5;
constexpr int kScoreSlots = 5 * 152;
constexpr int kMostWaves = 8;
// Rows from which on a wide table's selection is by 256 threads, many to an SM, that hold a
// context of up to 2048 blocks and read a longer one again; fewer rows by 1024 threads.
constexpr int kManyRows = 2 * 152;

// A warp for each possible tile where most of them exist (one sequence, or at most four
// blocks of each: 1024 sequences of one new token, 8 KV heads, 5.1 us and 8.2 the other way)
// or where they are two waves at most: 8 KV heads, 31 sequences of one new token and one
// of 512 (8448 warps) 3.2 and 3.4, one of 2048 (33024) 6.2 and 3.6.
constexpr long long kFewTiles = 2ll * 6 * 152 * kWarps;
constexpr int kEachFew = 4;

template <typename T, int D, int B>
cudaError_t bounds_block(const BoundsParams& p, cudaStream_t stream)
{
    const long long tiles = (long long)p.num_seqs * p.blocks_each * p.num_kv_heads;
    if (p.num_seqs == 1 || p.blocks_each <= kEachFew || tiles <= kFewTiles)
        return launch_dependent(bounds_kernel<T, D, B>, (tiles + kWarps - 1) / kWarps, kThreads, 0,
                                stream, p);
    return launch_dependent(bounds_many_kernel<T, D, B>, 3 * 152, kThreads, 0, stream, p);
}

template <typename T, int D>
cudaError_t bounds_typed(const BoundsParams& p, cudaStream_t stream)
{
    return p.block_size == 8    ? bounds_block<T, D, 8>(p, stream)
           : p.block_size == 16 ? bounds_block<T, D, 16>(p, stream)
                                : bounds_block<T, D, 32>(p, stream);
}

// A launch with `smem` bytes of dynamic shared memory, of which `room` are there anyway.  A
// kernel's limit is one for all threads of the process: every call that needs one sets the same,
// `most`, since one of its own size could lower it between another thread's and its launch.
template <typename K>
cudaError_t launch_select(K kern, const SelectParams& p, long long grid, int threads, int smem,
                          int room, int most, cudaStream_t stream)
{
    if (smem > room) {  // many query heads
        const cudaError_t e =
            cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(kern, grid, threads, smem, stream, p);
}

template <int D>
cudaError_t select_few(const SelectParams& p, cudaStream_t stream)
{
    const int group = p.num_heads / p.num_kv_heads;
    auto kern = group <= 8 ? select_kernel<D, 1> : select_kernel<D, 2>;
    return launch_select(kern, p, (long long)p.num_seqs * p.num_kv_heads, kScoreThreads,
                         score_bytes<D>(kScoreThreads, group) + 4 * p.max_blocks,
                         48 * 1024 - (int)sizeof(Histogram<kScoreThreads>),
                         score_bytes<D>(kScoreThreads, kSelectMaxGroup) + 4 * kFewBlocks, stream);
}

template <int NT, int PER, bool WIDE>
cudaError_t pick_threads(const SelectParams& p, cudaStream_t stream)
{
    return launch_dependent(pick_kernel<NT, PER, WIDE>, (long long)p.num_seqs * p.num_kv_heads, NT,
                            0, stream, p);
}

template <int D>
cudaError_t score_dim(SelectParams p, cudaStream_t stream)
{
    const long long items = (long long)p.num_seqs * p.num_kv_heads;
    const int turns = (p.max_blocks + kScoreThreads / 2 - 1) / (kScoreThreads / 2);  // of a row
    auto ways = [&](int each) { return (turns + each - 1) / each; };
    // turns of a CTA: those that take the GPU the fewest, its waves of CTAs times their
    // turns and their start; more for so many rows that CTAs without work (of rows
    // shorter than the table) would weigh
    auto cost = [&](int each) {
        return (items * ways(each) + kScoreSlots - 1) / kScoreSlots * (each + kStartTurns);
    };
    int each = 1;
    for (int e = 2; e <= kMostTurns; e *= 2)
        if (cost(e) < cost(each)) each = e;
    p.ways = (int)std::min<long long>(ways(each), std::max(1ll, kMostWaves * kScoreSlots / items));
    const long long grid = items * p.ways;
    const int group = p.num_heads / p.num_kv_heads;
    auto kern = group <= 8 ? score_kernel<D, 1> : score_kernel<D, 2>;
    return launch_select(kern, p, grid, kScoreThreads, score_bytes<D>(kScoreThreads, group),
                         48 * 1024, score_bytes<D>(kScoreThreads, kSelectMaxGroup), stream);
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

cudaError_t launch_select_blocks(const SelectParams& p, int head_dim, cudaStream_t stream)
{
    if (p.max_blocks > p.max_selected && p.max_blocks <= kFewBlocks)
        return head_dim == 128 ? select_few<128>(p, stream) : select_few<64>(p, stream);
    if (p.max_blocks > p.max_selected) {  // else nothing is scored
        const cudaError_t e =
            head_dim == 128 ? score_dim<128>(p, stream) : score_dim<64>(p, stream);
        if (e != cudaSuccess) return e;
    }
    // the fewest threads that hold the scores, four each (a call over 512 rows of 2048
    // blocks: 35.7 us, with eight each 36.4; over 64 rows of 1024: 9.8 and 10.8)
    if (p.max_blocks <= 4 * 128) return pick_threads<128, 4, false>(p, stream);
    if (p.max_blocks <= 4 * 256) return pick_threads<256, 4, false>(p, stream);
    if (p.max_blocks <= 4 * 512) return pick_threads<512, 4, false>(p, stream);
    if ((long long)p.num_seqs * p.num_kv_heads >= kManyRows)
        return pick_threads<256, 8, true>(p, stream);
    return p.max_blocks <= 8 * 1024 ? pick_threads<1024, 8, false>(p, stream)
                                    : pick_threads<1024, 8, true>(p, stream);
}
