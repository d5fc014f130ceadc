// Paged decode attention over the 4-bit cache for sm_103a.
//
// A token's key and value stand for k = m_r + c s_r and v = m'_r + c' s'_r in
// each run r of 64 elements (q4_common.cuh), so that with A_r = sum_d q_d c_d
// over the run's elements
//     score = scale * sum_r (s_r A_r + m_r sum_d q_d),
//     out   = sum_i p_i (m'_r + c' s'_r) / sum_i p_i,   p_i = 2^(score_i - max).
// Both products run on mma.sync m16n8k16 over the bare codes, tokens (or
// head_dim) on M and up to 8 NT query heads on N; scales and minima are applied
// in fp32 to the few numbers that come out of Q K^T or go into P V, not to the
// codes.
//
//  * A code is an fp16 operand as it stands: the bits of c in the low mantissa
//    bits of an otherwise empty half are the subnormal c * 2^-24 (or, four bits
//    higher, c * 2^-20), exact, and the MMA takes subnormals at full speed
//    (measured).  Eight codes become four operand registers with four ANDs and a
//    shift (K), or two byte permutes and two ANDs (V).  q is scaled by a power of
//    two that takes the row's greatest element to 2^10 .. 2^11 of fp16, the odd code
//    positions by another 2^-4: exact down to 2^-20 of the greatest, and below that,
//    where fp16 is subnormal, off by at most 2^-31 of it.
//  * P V gets w_i = p_i s'_i * kappa in fp16: one rounding (2^-11 of w_i; below 2^-14
//    of the greatest w, 2^-25 of that), besides small elements of q the only one below
//    32 bits.  kappa, kept for each head and run, holds the greatest
//    w near 1 whatever the scales' size: it moves, with O rescaled, when a w
//    passes 2^12 or the reference maximum rises.  The codes are centred by
//    c = 7.5 + (c - 7.5): an extra MMA with all operands 7.5 sums the rounded w,
//    and p_i (m' + 7.5 s') is summed in fp32, so that the rounding of w weighs
//    on elements around zero and not on the minimum's offset.
//  * Online softmax in base 2 against a per-head reference maximum that moves
//    only when a score passes it by more than 8.
//
// One CTA of four warps takes a (sequence, KV head, head slice, partition) item
// of the grid or of the work plan (decode_plan.cu); a warp takes every fourth
// stage of 32 tokens, through a ring in shared memory that 16-byte cp.async
// copies fill one stage ahead.  The warps' states are merged in shared memory;
// partials of a split item go to the workspace, and a second kernel merges them.
//
// What bounds it (bf16, D = 128, 8 contexts of 32768, 8 KV heads, 302 MB, 62.2 us
// a call; 44.5 at the copy rate): plan, copies and merge alone take 56 us, and the
// arithmetic alone about as long as the copies.  16 tokens of one KV head are 248
// instructions of a warp (276 with five to eight heads a group), half of them on
// the half-rate integer pipe (72 to take the codes apart), and 17 MMAs of 8
// cycles, which keep that pipe waiting; to start and end a warp takes about 970.
// No pipe is full (issue 57 %, integer 51 %, tensor 25 %, DRAM 64 %): four warps a
// scheduler wait for one another's latencies.
// Four warps a CTA and four CTAs a SM (128 registers): two warps leave a ragged
// batch waiting for its longest sequences (64 x 8 heads over 256 sequences: 88 us
// against 59), eight spend more on starting and merging (78).  Two tiles between
// votes (TT): 68 us against 70.5 when it came in.  e4m3 codes on the fp8 mma.sync
// would halve the unpacking, but that instruction runs as conversions and fp16
// MMAs on this architecture (80 us against 68).
#include <cuda_runtime.h>

#include <climits>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"
#include "q4_common.cuh"
#include "tc_common.cuh"

namespace {

using namespace pkv_tc;
using namespace pkv_q4;
using namespace pkv_pdl;

constexpr int NW = kDecodeQ4Warps;
constexpr int ST = kDecodeQ4StageTokens;
constexpr int NS = 2;  // stages of a warp's ring

// 16 bytes from src + SRC to shared address dst + DST.
template <int DST, int SRC>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src),
                 "n"(DST), "n"(SRC));
}
// Calls f with Index<0>() .. Index<N - 1>().
template <int I>
struct Index {
    static constexpr int value = I;
};
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unrolled(F&& f)
{
    if constexpr (I < N) {
        f(Index<I>());
        unrolled<N, I + 1>(f);
    }
}
__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;");
}
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// floor(log2 x) of a normal x > 0 (below: -127; infinity and NaN: 128)
__device__ __forceinline__ int exponent(float x)
{
    return (int)(__float_as_uint(x) >> 23 & 255u) - 127;
}

// The operand registers of a K word of eight codes: c * 2^-24 of elements i, i + 4 in
// registers i = 0 and 2, c * 2^-20 in 1 and 3.
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&r)[4])
{
    const uint32_t u = w >> 8;
    r[0] = w & 0x000F000Fu;
    r[1] = w & 0x00F000F0u;
    r[2] = u & 0x000F000Fu;
    r[3] = u & 0x00F000F0u;
}

// The same of a V word (elements i of two tokens), with one instruction less:
// registers 1 and 3 hold (c_even + 16 c_odd) * 2^-24, from whose sums the even
// codes' are taken off at the end.
__device__ __forceinline__ void spread_v(uint32_t w, uint32_t (&r)[4])
{
    r[1] = __byte_perm(w, 0u, 0x4240);
    r[3] = __byte_perm(w, 0u, 0x4341);
    r[0] = r[1] & 0x000F000Fu;
    r[2] = r[3] & 0x000F000Fu;
}

// d += A B.
__device__ __forceinline__ void mma_acc(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = A B: the first MMA of a chain.
__device__ __forceinline__ void mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The reference maximum of a warp (or partial) that saw no token: below every
// score, and finite, so that two of them differ by zero.
constexpr float kNone = -1e38f;

template <typename T, int D, int NT>
struct Shape {
    static constexpr int R = D / kRun;       // runs of a row
    static constexpr int NC = 8 * NT;        // query-head columns
    static constexpr int GROUP_BYTES = 8 * (D / 2);        // codes of 8 tokens
    static constexpr int CODE_BYTES = 4 * GROUP_BYTES;     // K (or V) codes of a stage
    static constexpr int PAIR_BYTES = ST * R * 4;          // K (or V) pairs of a stage
    static constexpr int STAGE_BYTES = 2 * (CODE_BYTES + PAIR_BYTES);
    static constexpr int FLOAT_BYTES = ST * R * 16;        // a stage's pairs as fp32
    static constexpr int RING_BYTES = NS * STAGE_BYTES + FLOAT_BYTES;
    static constexpr int GPC = 512 / GROUP_BYTES;          // groups a warp-wide copy brings
    static constexpr int K_CHUNKS = D / 32, V_CHUNKS = D / 16;  // of a K row, of a V pair's row
    static constexpr int MERGE_BYTES = NW * NC * (D + 2) * 4;
    static constexpr int SMEM_BYTES =
        NW * RING_BYTES > MERGE_BYTES ? NW * RING_BYTES : MERGE_BYTES;
};

// T: the cache's type; NT: column tiles of eight query heads.  FOLD (up to four
// heads, NT = 1): columns 0 .. 3 hold the heads and stand for the first of two
// tiles of tokens, columns 4 .. 7 the same heads for the second, so that no lane
// weighs columns that are not there.  Each lane keeps the scores of its columns'
// tile; the V products of both tiles run into the same accumulators, with weights
// of zero in the other tile's columns; a column is a state of its own until the
// end.  8 contexts of 32768, 4 heads a group: 61.4 us against 64.1; 32 heads of
// their own K over 64 sequences: 62.5 against 65.8.
template <typename T, int D, int B, int NT, bool FOLD>
__global__ void __launch_bounds__(NW * 32, decode_q4_ctas_per_sm(D, 8 * NT))
decode_q4_kernel(const DecodeParams p)
{
    using Sh = Shape<T, D, NT>;
    using H = Half16<T>;
    constexpr int R = Sh::R, NC = Sh::NC;
    constexpr int TT = NT == 1 ? 2 : 1;  // tiles of 16 tokens taken together
    constexpr int XT = FOLD ? 1 : TT;    // sets of scores that makes
    constexpr int CS = FOLD ? 2 : 1;     // columns, and states, of a head
    static_assert(!FOLD || NT == 1, "four heads at most");
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const int G = p.num_heads / p.num_kv_heads, HS = p.head_slices;
    // A call that is not split lets the next one's CTAs in as early as there is room
    // (62.5 us against 64.2 where the loop ends, 64 sequences of 32 heads); the merge
    // of a split call would then sit beside the last attention CTAs, and the next
    // call's behind it (8 contexts of 32768 69 us against 61).
    const bool early = p.max_partitions <= 1;
    wait_for_previous();
    if (early) let_next_start();  // by now all that came before is visible to it

    // ---- the item: record or grid slot (((s * Hkv) + g) * parts + part) * HS + hs
    int sg, part, L, piece = -1, npieces = 0;
    if (p.items != nullptr) {
        const int4 it = p.items[blockIdx.x];  // read with the count: past it, stale
        if ((int)blockIdx.x >= *p.item_count) return;
        sg = it.x * (p.num_kv_heads * HS) + it.z;
        L = it.y;
        part = it.w;
        if (it.w & kPlanPieceFlag) {
            piece = it.w & kPlanPieceMask;
            npieces = (it.w >> kPlanPieceBits) & kPlanPieceMask;
        }
    } else {
        const int hs_b = blockIdx.x % HS, t = blockIdx.x / HS;
        part = t % p.max_partitions;
        sg = (t / p.max_partitions) * HS + hs_b;
        L = p.context_lens[sg / (HS * p.num_kv_heads)];
    }
    const int sgk = sg / HS, hs = sg - sgk * HS;
    const int s = sgk / p.num_kv_heads, g = sgk - s * p.num_kv_heads;
    const int GC = (G + HS - 1) / HS, hb = hs * GC, ncol = min(GC, G - hb);
    if (L < 0 || (int64_t)L > (int64_t)p.max_blocks * B) {
        if (threadIdx.x == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        L = 0;
    }
    int begin, end, nparts;
    if (piece >= 0) {
        const int nsq = (L + ST - 1) / ST;
        begin = (int)((int64_t)piece * nsq / npieces) * ST;
        end = min(L, (int)((int64_t)(piece + 1) * nsq / npieces) * ST);
        nparts = npieces;
        part = piece;
    } else {
        nparts = (L + p.partition_tokens - 1) / p.partition_tokens;
        if (part >= max(nparts, 1)) return;
        begin = part * p.partition_tokens;
        end = min(L, begin + p.partition_tokens);
    }
    const int nst = end > begin ? (end - begin + ST - 1) / ST : 0;

    // ---- this warp's stages: j < cnt, tokens begin + (warp + 4 j) * 32 on, in a
    // ring of NS.  A stage is four groups of 8 tokens, each inside one block;
    // lane 4 (j % 8) + u keeps the block id of group u of stage j for a window
    // of eight stages, and the next window's is on its way.
    uint8_t* ring = smem + warp * Sh::RING_BYTES;
    float2* k_pairs = reinterpret_cast<float2*>(ring + NS * Sh::STAGE_BYTES);  // [32][R]
    float2* v_pairs = k_pairs + ST * R;
    const int cnt = nst > warp ? (nst - warp + NW - 1) / NW : 0;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    constexpr size_t tile = tile_bytes(B, D);
    const uint32_t block_stride = (uint32_t)(tile * p.num_kv_heads);
    const uint8_t* kp = static_cast<const uint8_t*>(p.k_cache) + g * tile;
    const uint8_t* vp = static_cast<const uint8_t*>(p.v_cache) + g * tile;
    auto load_ids = [&](int j0) {
        const int tok = begin + (warp + (j0 + (lane >> 2)) * NW) * ST + (lane & 3) * 8;
        int id = -1;
        if (tok < end) {
            id = table[tok / B];
            if (id < 0 || id >= p.num_blocks) {
                atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
                id = -1;
            }
        }
        return id;
    };
    int ids = load_ids(0), ids_next = -1;
    if (cnt > 8) ids_next = load_ids(8);
    uint32_t there = __ballot_sync(0xffffffffu, ids >= 0);  // the window's groups with a block
    // where this lane's 16 bytes of a copy come from and go: the groups of one
    // copy are GPC; chunks are swizzled so that the reads below hit every bank
    constexpr int GPC = Sh::GPC, LPG = 32 / GPC;  // groups a copy, lanes a group
    const int cl = lane % LPG;
    const int k_write = lane / LPG * Sh::GROUP_BYTES + (cl / Sh::K_CHUNKS) * (D / 2) +
                        ((cl % Sh::K_CHUNKS) ^ (D == 128 ? (cl >> 3 & 1) << 1 : 0)) * 16;
    const int v_write = lane / LPG * Sh::GROUP_BYTES + (cl / Sh::V_CHUNKS) * D +
                        ((cl % Sh::V_CHUNKS) ^
                         (D == 128 ? (cl >> 3) << 1 : (cl >> 3 & 1) << 1)) * 16;
    int k_read[R], v_read[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        k_read[r] = gq * (D / 2) + (r ^ (D == 128 ? gq >> 1 & 1 : 0)) * 32 + tq * 8;
        v_read[r] = tq * D +
                    ((4 * r + (gq >> 1)) ^ (D == 128 ? tq << 1 : (tq >> 1) << 1)) * 16 +
                    (gq & 1) * 8;
    }
    // pairs: lanes 0 .. PL - 1 copy K's, as many after them V's
    constexpr int PL = 8 * R;  // 16-byte chunks of a stage's K (or V) pairs
    const int pu = (lane % PL) / (2 * R), pc = lane % (2 * R);  // group and chunk
    const uint8_t* pp =
        (lane < PL ? kp : vp) + B * (D / 2) + (8 * pu) % B * (R * 4) + pc * 16;
    // codes: this lane's 16 bytes of a copy's groups within a block
    kp += (GPC * 8 > B ? cl : lane) * 16;
    vp += (GPC * 8 > B ? cl : lane) * 16;
    const uint32_t ring_at = smem_u32(ring);
    const uint32_t k_dst = ring_at + k_write, v_dst = ring_at + Sh::CODE_BYTES + v_write;
    // Starts the copies of stage j; returns which of its groups have a block (the
    // others' copies bring block 0, which nothing reads).
    auto issue = [&](int j) -> uint32_t {
        uint32_t groups = 0;
        if (j < cnt) {
            if (j != 0 && (j & 7) == 0) {
                ids = ids_next;
                there = __ballot_sync(0xffffffffu, ids >= 0);
                ids_next = load_ids(j + 8);
            }
            const int lane0 = (j & 7) * 4;
            const uint32_t slot = (j % NS) * Sh::STAGE_BYTES;
            groups = there >> lane0 & 15u;
            const uint8_t *k_at = nullptr, *v_at = nullptr;
            unrolled<4 / GPC>([&](auto tag) {
                constexpr int k = decltype(tag)::value, IN = (k * GPC * 8) % B * (D / 2);
                // a copy's groups lie in one block, or (B = 8, two groups a copy) in two
                if (IN == 0) {
                    const uint32_t id = (uint32_t)max(
                        0, __shfl_sync(0xffffffffu, ids,
                                       lane0 + k * GPC + (GPC * 8 > B ? lane / LPG : 0)));
                    k_at = kp + (size_t)id * block_stride;
                    v_at = vp + (size_t)id * block_stride;
                }
                cp_async16<k * 512, IN>(k_dst + slot, k_at);
                cp_async16<k * 512, IN>(v_dst + slot, v_at);
            });
            const uint32_t ip = (uint32_t)max(0, __shfl_sync(0xffffffffu, ids, lane0 + pu));
            if (lane < 2 * PL)
                cp_async16<2 * Sh::CODE_BYTES, 0>(ring_at + slot + lane * 16,
                                                  pp + (size_t)ip * block_stride);
        }
        cp_async_commit();
        return groups;
    };
    static_assert(NS == 2, "one stage on its way while one is worked on");
    uint32_t groups_next = issue(0);

    // ---- Q as the B operand: column n = query head g * G + hb + n.  k-step
    // 4r + i pairs elements 64r + 16tq + {i, 4 + i} and + {8 + i, 12 + i}: the
    // order in which spread() leaves a K word's codes.
    uint32_t qb[NT][R * 4][2];
    // columns 2tq, 2tq + 1: scale * 2^24 / q's scaling, sum q * that scaling / 2^24
    float su[NT][2], sq[NT][R][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = FOLD ? gq & 3 : 8 * t + gq;
        float v[R][16], top = 0.f, sum[R];
        const T* row = static_cast<const T*>(p.q) +
                       ((size_t)s * p.num_heads + g * G + hb + (n < ncol ? n : 0)) * D;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[r] = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 x = n < ncol ? H::unpack(*reinterpret_cast<const uint32_t*>(
                                                row + 64 * r + 16 * tq + 2 * j))
                                          : make_float2(0.f, 0.f);
                v[r][2 * j] = x.x;
                v[r][2 * j + 1] = x.y;
                top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                sum[r] += x.x + x.y;
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
            for (int r = 0; r < R; ++r) sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], o);
        }
        // greatest element to 2^10 .. 2^11
        const int e = min(max(exponent(top), -100), 112);
        const float f = pow2(10 - e);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float fi = i & 1 ? f * 0.0625f : f;
                qb[t][4 * r + i][0] = Half16<__half>::pack(v[r][i] * fi, v[r][4 + i] * fi);
                qb[t][4 * r + i][1] = Half16<__half>::pack(v[r][8 + i] * fi, v[r][12 + i] * fi);
            }
        // a row's constants sit with lanes 4 * column ..; this lane's accumulators hold columns
        // 2tq and 2tq + 1
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int from = 4 * (2 * tq + c);
            su[t][c] = p.scale_log2 * pow2(__shfl_sync(0xffffffffu, e, from) + 14);
#pragma unroll
            for (int r = 0; r < R; ++r)
                sq[t][r][c] = __shfl_sync(0xffffffffu, sum[r] * (f * 0x1p-24f), from);
        }
    }

    // ---- state of columns 8t + 2tq + c: reference maximum, sum of p, kappa,
    // sum of p (m' + 7.5 s'), sum of 7.5 w, sum of w c' (elements 64r + 8gq + n
    // in [0], [1] and + 4 in [2], [3])
    float mr[NT][2], l[NT][2], kap[NT][R][2], oz[NT][R][2], aw[NT][R][4], acc[NT][R * 4][4];
    bool fresh = true;  // no token seen yet: the first ones set mr and kappa
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        mr[t][0] = mr[t][1] = 0.f;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            kap[t][r][0] = kap[t][r][1] = 1.f;
            oz[t][r][0] = oz[t][r][1] = 0.f;
            aw[t][r][0] = aw[t][r][1] = aw[t][r][2] = aw[t][r][3] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < R * 4; ++i)
            acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
    }

    // ---- stages
    for (int j = 0; j < cnt; ++j) {
        cp_async_wait<NS - 2>();
        __syncwarp();  // every lane's copies of stage j are in, and stage j - 1 is consumed
        const uint32_t groups = groups_next;
        const int tok_s = begin + (warp + j * NW) * ST;
        const uint8_t* st = ring + (j % NS) * Sh::STAGE_BYTES;
        // ---- the stage's pairs as floats, one token a lane: K's (s, m) of each run, V's
        // (s', m' + 7.5 s'), zero for a token that is not there
        uint32_t seen = 0xffffffffu;
        if (tok_s + ST > end || groups != 15u)
            seen = __ballot_sync(0xffffffffu,
                                 tok_s + lane < end && (groups >> (lane >> 3) & 1u));
        const bool mine = seen >> lane & 1u;
        {
            const uint8_t* pt = st + 2 * Sh::CODE_BYTES + lane * (R * 4);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float2 k = H::unpack(*reinterpret_cast<const uint32_t*>(pt + 4 * r));
                const uint32_t w = *reinterpret_cast<const uint32_t*>(pt + Sh::PAIR_BYTES + 4 * r);
                const float2 v = H::unpack(mine ? w : 0u);
                k_pairs[lane * R + r] = k;
                v_pairs[lane * R + r] = make_float2(v.x, fmaf(7.5f, v.x, v.y));
            }
        }
        __syncwarp();
        groups_next = issue(j + 1);
        // bits 8u of this lane's tokens gq + 8u
        const uint32_t seen_l = seen >> (gq + (FOLD ? tq >> 1 << 4 : 0));
        // TT tiles of 16 tokens at a time (two of them where the registers allow:
        // twice the independent work between the votes)
#pragma unroll 1
        for (int hf = 0; hf < 2; hf += TT) {
            if (tok_s + hf * 16 >= end) break;
            // ---- X = sum_r s_r A_r + m_r sum q, in units of su: rows gq, gq + 8 of a tile
            float x[XT][NT][4];
#pragma unroll
            for (int hx = 0; hx < XT; ++hx) {
                const float2* kpr = k_pairs + ((FOLD ? tq >> 1 : hf + hx) * 16 + gq) * R;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float sc[TT][NT][4];
#pragma unroll
                    for (int h = hx; h < hx + (FOLD ? TT : 1); ++h) {
                        const uint8_t* at = st + 2 * (hf + h) * Sh::GROUP_BYTES;
                        const uint2 w0 = *reinterpret_cast<const uint2*>(at + k_read[r]);
                        const uint2 w1 =
                            *reinterpret_cast<const uint2*>(at + Sh::GROUP_BYTES + k_read[r]);
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        spread(w0.x, a0);
                        spread(w1.x, a1);
                        spread(w0.y, a2);
                        spread(w1.y, a3);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {a0[i], a1[i], a2[i], a3[i]};
#pragma unroll
                            for (int t = 0; t < NT; ++t)
                                if (i == 0)
                                    mma_first(sc[h][t], a, qb[t][4 * r][0], qb[t][4 * r][1]);
                                else
                                    mma_acc(sc[h][t], a, qb[t][4 * r + i][0],
                                            qb[t][4 * r + i][1]);
                        }
                    }
                    const float2 sm0 = kpr[r], sm1 = kpr[8 * R + r];
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 sm = e < 2 ? sm0 : sm1;
                            const float z = r ? fmaf(sm.y, sq[t][r][e & 1], x[hx][t][e])
                                              : sm.y * sq[t][r][e & 1];
                            const float a =
                                FOLD && tq >= 2 ? sc[TT - 1][t][e] : sc[hx][t][e];
                            x[hx][t][e] = fmaf(sm.x, a, z);
                        }
                }
            }
            // ---- p, and w = p s' kappa, against the references as they stand (the scores
            // are kept as they are: less the old reference they would round to its size)
            float pr[XT][NT][4];
            uint32_t wb[XT][NT][R][2];
            float2 sm[XT][2][R];  // (s', m' + 7.5 s') of tokens gq, gq + 8
            float high = -INFINITY;
            uint32_t most = 0u;
            float y[XT][NT][4];  // the scores
#pragma unroll
            for (int h = 0; h < XT; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[h][t][e] = x[h][t][e] * su[t][e & 1];
            if (seen != 0xffffffffu) {
#pragma unroll
                for (int h = 0; h < XT; ++h)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (!(seen_l >> (16 * (hf + h) + 8 * (e >> 1)) & 1u))
                                y[h][t][e] = -INFINITY;
            }
            auto weigh = [&]() {
#pragma unroll
                for (int h = 0; h < XT; ++h)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int u = 0; u < 2; ++u)
                                // p s' first: a p of zero keeps a large s' kappa from the sum
                                wb[h][t][r][u] = Half16<__half>::pack(
                                    pr[h][t][2 * u] * sm[h][u][r].x * kap[t][r][0],
                                    pr[h][t][2 * u + 1] * sm[h][u][r].x * kap[t][r][1]);
            };
#pragma unroll
            for (int h = 0; h < XT; ++h) {
                const float2* vpr = v_pairs + ((FOLD ? tq >> 1 : hf + h) * 16 + gq) * R;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < R; ++r) sm[h][u][r] = vpr[8 * u * R + r];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float z = y[h][t][e] - mr[t][e & 1];
                        high = fmaxf(high, z);
                        pr[h][t][e] = ex2(z);
                    }
            }
            weigh();
#pragma unroll
            for (int h = 0; h < XT; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            most = Half16<__half>::max2(most, wb[h][t][r][u]);
            // w > 2^12: as bits, as w >= 0 (a NaN counts too)
            const bool up = high > 8.f || ((most + 0x13FF13FFu) & 0x80008000u) != 0u;
            if (fresh || __any_sync(0xffffffffu, up)) {
                if (seen >> (16 * hf) << (32 - 16 * TT)) {  // of these tokens
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            // the reference moves to the greatest score (up only, once set;
                            // a score that overflowed to -infinity is below any), and the
                            // scores are taken afresh: y rounds to the old reference's size
                            float to = fresh ? kNone : mr[t][c];
#pragma unroll
                            for (int h = 0; h < XT; ++h)
                                to = fmaxf(to, fmaxf(y[h][t][c], y[h][t][2 + c]));
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
                            const float al = fresh ? 0.f : ex2(mr[t][c] - to);
                            mr[t][c] = to;
                            l[t][c] *= al;
#pragma unroll
                            for (int h = 0; h < XT; ++h) {
                                pr[h][t][c] = ex2(y[h][t][c] - to);
                                pr[h][t][2 + c] = ex2(y[h][t][2 + c] - to);
                            }
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                // kappa: the greatest p s' of these tokens, or what a w of 1
                                // of the tokens before stands for now, to 1 .. 2; none of
                                // either: a kappa that any w will overflow
                                const float one =
                                    __uint_as_float((254u << 23) - __float_as_uint(kap[t][r][c]));
                                float top = al * one;
#pragma unroll
                                for (int h = 0; h < XT; ++h)
                                    top = fmaxf(top, fmaxf(pr[h][t][c] * sm[h][0][r].x,
                                                           pr[h][t][2 + c] * sm[h][1][r].x));
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                                const float kn = pow2(-min(max(exponent(top), -120), 120));
                                const float f = al * one * kn;
                                kap[t][r][c] = kn;
                                if (!fresh) {
                                    oz[t][r][c] *= al;
                                    aw[t][r][c] *= f;
                                    aw[t][r][2 + c] *= f;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        acc[t][4 * r + i][c] *= f;
                                        acc[t][4 * r + i][2 + c] *= f;
                                    }
                                }
                            }
                        }
                    fresh = false;
                    weigh();
                }
            }
            // ---- sums, and O^T += codes of V^T times w: pairs tq, tq + 4 of a tile
            const uint32_t mid[4] = {0x47804780u, 0x47804780u, 0x47804780u, 0x47804780u};  // 7.5
#pragma unroll
            for (int hx = 0; hx < XT; ++hx) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) l[t][c] += pr[hx][t][c] + pr[hx][t][2 + c];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float z0 = sm[hx][0][r].y, z1 = sm[hx][1][r].y;
                    uint32_t b[NT][2];
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            oz[t][r][c] =
                                fmaf(pr[hx][t][c], z0, fmaf(pr[hx][t][2 + c], z1, oz[t][r][c]));
                        b[t][0] = movmatrix_trans(wb[hx][t][r][0]);
                        b[t][1] = movmatrix_trans(wb[hx][t][r][1]);
                        mma_acc(aw[t][r], mid, b[t][0], b[t][1]);
                    }
#pragma unroll
                    for (int h = hx; h < hx + (FOLD ? TT : 1); ++h) {
                        const uint8_t* at = st + Sh::CODE_BYTES + 2 * (hf + h) * Sh::GROUP_BYTES;
                        const uint2 w0 = *reinterpret_cast<const uint2*>(at + v_read[r]);
                        const uint2 w1 =
                            *reinterpret_cast<const uint2*>(at + Sh::GROUP_BYTES + v_read[r]);
                        uint32_t a0[4], a1[4], a2[4], a3[4];
                        spread_v(w0.x, a0);
                        spread_v(w0.y, a1);
                        spread_v(w1.x, a2);
                        spread_v(w1.y, a3);
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            // FOLD: of column gq, the other tile's weights left out
                            const bool keep = !FOLD || gq >> 2 == h;
                            const uint32_t b0 = keep ? b[t][0] : 0u, b1 = keep ? b[t][1] : 0u;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t a[4] = {a0[i], a1[i], a2[i], a3[i]};
                                mma_acc(acc[t][4 * r + i], a, b0, b1);
                            }
                        }
                    }
                }
            }
        }
    }

    if (!early) let_next_start();
    // ---- the warp's sums over its row groups, and its O in plain units
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l[t][c] += __shfl_xor_sync(0xffffffffu, l[t][c], o);
#pragma unroll
                for (int r = 0; r < R; ++r)
                    oz[t][r][c] += __shfl_xor_sync(0xffffffffu, oz[t][r][c], o);
            }
        }
    cp_async_wait<0>();
    __syncthreads();  // the rings are free
    float* merge = reinterpret_cast<float*>(smem);
    float* wm = merge + warp * NC * (D + 2);  // [NC][D], m[NC], l[NC]
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int n = 8 * t + 2 * tq + c;
            if ((FOLD ? n & 3 : n) >= ncol) continue;
            if (gq == 0) {
                wm[NC * D + n] = fresh ? kNone : mr[t][c];
                wm[NC * D + NC + n] = l[t][c];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float inv = 1.f / kap[t][r][c];
#pragma unroll
                for (int e = c; e < 4; e += 2) {  // elements 8gq .. + 3, then + 4 .. + 7
                    const float (*a)[4] = &acc[t][4 * r];
                    const float v[4] = {a[0][e] * 0x1p24f, (a[1][e] - a[0][e]) * 0x1p20f,
                                        a[2][e] * 0x1p24f, (a[3][e] - a[2][e]) * 0x1p20f};
                    float4 o;
                    o.x = fmaf(v[0] - aw[t][r][e], inv, oz[t][r][c]);
                    o.y = fmaf(v[1] - aw[t][r][e], inv, oz[t][r][c]);
                    o.z = fmaf(v[2] - aw[t][r][e], inv, oz[t][r][c]);
                    o.w = fmaf(v[3] - aw[t][r][e], inv, oz[t][r][c]);
                    *reinterpret_cast<float4*>(wm + n * D + 64 * r + 8 * gq + 2 * (e - c)) = o;
                }
            }
        }
    __syncthreads();

    // ---- merge the warps
    const size_t hbase = (size_t)s * p.num_heads + (size_t)g * G + hb;
    const bool vec_out = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
    for (int idx = threadIdx.x; idx < ncol * D / 4; idx += NW * 32) {
        const int n = idx / (D / 4), d = (idx - n * (D / 4)) * 4;
        float M = kNone;
#pragma unroll
        for (int k = 0; k < NW * CS; ++k)  // FOLD: columns n and n + 4 of a warp
            M = fmaxf(M, merge[k / CS * NC * (D + 2) + NC * D + n + k % CS * 4]);
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NW * CS; ++k) {
            const float* ww = merge + k / CS * NC * (D + 2);
            const int nk = n + k % CS * 4;
            const float wt = ex2(ww[NC * D + nk] - M);  // 1, of nothing, where no warp saw a token
            den = fmaf(wt, ww[NC * D + NC + nk], den);
            const float4 o = *reinterpret_cast<const float4*>(ww + nk * D + d);
            num.x = fmaf(wt, o.x, num.x);
            num.y = fmaf(wt, o.y, num.y);
            num.z = fmaf(wt, o.z, num.z);
            num.w = fmaf(wt, o.w, num.w);
        }
        if (nparts <= 1) {
            // a sum of zero: no token was seen; a NaN stays one
            const float inv = den == 0.f ? 0.f : 1.f / den;
            store_out4(p.out, (hbase + n) * D + d,
                       make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv),
                       p.out_dtype, vec_out);
        } else {
            const size_t slot = (hbase + n) * p.max_partitions + part;
            *reinterpret_cast<float4*>(p.ws_o + slot * D + d) = num;
            if (d == 0) p.ws_ml[slot] = make_float2(M, den);
        }
    }
    if (p.done != nullptr && part == 0 && threadIdx.x == 0) p.done[sg] = nparts;
}

// Split calls: one CTA merges the partials of one query head by log-sum-exp,
//     M = max_i m_i,  w_i = 2^(m_i - M),  out = sum_i w_i O_i / sum_i w_i l_i,
// its warps (and at D = 64 their halves) each every so many partials.  A kernel
// of its own spreads a lone long request's merge (64 partials of 16 heads, 0.5
// MB) over as many SMs as there are heads; the last attention CTA alone took
// 40 us for it.  It is all latency, so the first partials are read along with
// their number (what lies past it is in the workspace, and ignored).
template <int D>
__global__ void __launch_bounds__(128) merge_q4_kernel(const DecodeParams p)
{
    constexpr int V4 = D / 4, LANES = 128 / V4;  // threads a row, partials at once
    constexpr int AHEAD = 32 / LANES;
    __shared__ float4 sum[128];
    const int row = blockIdx.x, s = row / p.num_heads, h = row - s * p.num_heads;
    const int G = p.num_heads / p.num_kv_heads, HS = p.head_slices, GC = (G + HS - 1) / HS;
    const int lane = threadIdx.x & 31, first = threadIdx.x / V4;
    const unsigned* count = p.done + (s * p.num_kv_heads + h / G) * HS + h % G / GC;
    const float2* ml = p.ws_ml + (size_t)row * p.max_partitions;
    const float4* src = reinterpret_cast<const float4*>(
                            p.ws_o + (size_t)row * p.max_partitions * D) + threadIdx.x % V4;
    let_next_start();
    wait_for_previous();
    float4 o[AHEAD];
    float2 x[2];  // of partials lane, lane + 32
    const unsigned n = __ldcg(count);
#pragma unroll
    for (int k = 0; k < 2; ++k)
        x[k] = __ldcg(ml + min(lane + 32 * k, p.max_partitions - 1));
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        o[k] = __ldcg(src + (size_t)min(first + k * LANES, p.max_partitions - 1) * V4);
    if (n <= 1u) return;  // the attention CTA wrote the output
    const int nparts = (int)min(n, (unsigned)p.max_partitions);
    float M = kNone, den = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k)
        if (lane + 32 * k < nparts) M = fmaxf(M, x[k].x);
    for (int i = lane + 64; i < nparts; i += 32) M = fmaxf(M, __ldcg(ml + i).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        w[k] = lane + 32 * k < nparts ? ex2(x[k].x - M) : 0.f;
        if (lane + 32 * k < nparts) den = fmaf(w[k], x[k].y, den);
    }
    for (int i = lane + 64; i < nparts; i += 32) {
        const float2 y = __ldcg(ml + i);
        den = fmaf(ex2(y.x - M), y.y, den);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float wi, const float4& v) {
        num.x = fmaf(wi, v.x, num.x);
        num.y = fmaf(wi, v.y, num.y);
        num.z = fmaf(wi, v.z, num.z);
        num.w = fmaf(wi, v.w, num.w);
    };
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        const int i = first + k * LANES;  // < 32
        const float wi = __shfl_sync(0xffffffffu, w[0], i);
        if (i < nparts) add(wi, o[k]);
    }
#pragma unroll 8
    for (int i = first + AHEAD * LANES; i < nparts; i += LANES)
        add(ex2(__ldcg(ml + i).x - M), __ldcg(src + (size_t)i * V4));
    sum[threadIdx.x] = num;
    __syncthreads();
    if (threadIdx.x >= V4) return;
#pragma unroll
    for (int k = 1; k < LANES; ++k) add(1.f, sum[threadIdx.x + k * V4]);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    store_out4(p.out, (size_t)row * D + threadIdx.x * 4,
               make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv), p.out_dtype,
               (reinterpret_cast<uintptr_t>(p.out) & 15) == 0);
}

// The same for many rows, few of them split perhaps: a warp a row, which reads
// nothing before it knows the number of partials.
template <int D>
__global__ void __launch_bounds__(128) merge_rows_q4_kernel(const DecodeParams p)
{
    constexpr int V4 = D / 4, LANES = 32 / V4;  // lanes a row, partials at once
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int s = row / p.num_heads, h = row - s * p.num_heads;
    const int G = p.num_heads / p.num_kv_heads, HS = p.head_slices, GC = (G + HS - 1) / HS;
    let_next_start();
    wait_for_previous();
    if (s >= p.num_seqs) return;
    const unsigned n = __ldcg(p.done + (s * p.num_kv_heads + h / G) * HS + h % G / GC);
    if (n <= 1u) return;  // the attention CTA wrote the output
    const int nparts = (int)min(n, (unsigned)p.max_partitions);
    const float2* ml = p.ws_ml + (size_t)row * p.max_partitions;
    const float4* src = reinterpret_cast<const float4*>(
                            p.ws_o + (size_t)row * p.max_partitions * D) + lane % V4;
    float M = kNone, den = 0.f;
    for (int i = lane; i < nparts; i += 32) M = fmaxf(M, __ldcg(ml + i).x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < nparts; i0 += 32) {
        float w = 0.f;
        if (i0 + lane < nparts) {
            const float2 y = __ldcg(ml + i0 + lane);
            w = ex2(y.x - M);
            den = fmaf(w, y.y, den);
        }
        const int here = min(32, nparts - i0);
#pragma unroll 4
        for (int j = 0; j < here; j += LANES) {
            const int i = j + lane / V4;
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (i >= here) continue;
            const float4 v = __ldcg(src + (size_t)(i0 + i) * V4);
            num.x = fmaf(wi, v.x, num.x);
            num.y = fmaf(wi, v.y, num.y);
            num.z = fmaf(wi, v.z, num.z);
            num.w = fmaf(wi, v.w, num.w);
        }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
#pragma unroll
    for (int d = 16; d >= V4; d >>= 1) {
        num.x += __shfl_xor_sync(0xffffffffu, num.x, d);
        num.y += __shfl_xor_sync(0xffffffffu, num.y, d);
        num.z += __shfl_xor_sync(0xffffffffu, num.z, d);
        num.w += __shfl_xor_sync(0xffffffffu, num.w, d);
    }
    if (lane >= V4) return;
    const float inv = den == 0.f ? 0.f : 1.f / den;
    store_out4(p.out, (size_t)row * D + lane * 4,
               make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv), p.out_dtype,
               (reinterpret_cast<uintptr_t>(p.out) & 15) == 0);
}

template <typename T, int D, int B, int NT, bool FOLD>
cudaError_t launch(const DecodeParams& p, long long grid, cudaStream_t stream)
{
    constexpr int smem = Shape<T, D, NT>::SMEM_BYTES;
    static_assert(smem <= 48 * 1024, "what a kernel may have without asking");
    return launch_dependent(decode_q4_kernel<T, D, B, NT, FOLD>, grid, NW * 32, smem, stream, p);
}

template <typename T, int D, int NT, bool FOLD>
cudaError_t launch_block(const DecodeParams& p, long long grid, cudaStream_t stream)
{
    if (p.block_size == 8) return launch<T, D, 8, NT, FOLD>(p, grid, stream);
    if (p.block_size == 16) return launch<T, D, 16, NT, FOLD>(p, grid, stream);
    return launch<T, D, 32, NT, FOLD>(p, grid, stream);
}

template <typename T, int D>
cudaError_t launch_dim(const DecodeParams& p, long long grid, int columns, cudaStream_t stream)
{
    return columns > 8   ? launch_block<T, D, 2, false>(p, grid, stream)
           : columns > 4 ? launch_block<T, D, 1, false>(p, grid, stream)
                         : launch_block<T, D, 1, true>(p, grid, stream);
}

template <typename T>
cudaError_t launch_typed(const DecodeParams& p, long long grid, int columns, cudaStream_t stream)
{
    return p.head_dim == 128 ? launch_dim<T, 128>(p, grid, columns, stream)
                             : launch_dim<T, 64>(p, grid, columns, stream);
}

// A CTA a row while the GPU holds them all at once (16 on each of 152 SMs), a warp a
// row past that.  CTA against warp, us a call: 16 rows of 64 partials 10.3 and 22.6,
// 256 rows of 19 61.6 and 68.9, 2048 rows of 8 49.4 and 50.0, 4096 rows of ragged
// contexts 35.4 and 32.5, 16384 75.5 and 62.5.
constexpr long long kMergeCtaRows = 16 * 152;

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams& p, int kv_dtype, long long grid, int columns,
                             cudaStream_t stream)
{
    const cudaError_t e = kv_dtype == PKV_F16
                              ? launch_typed<__half>(p, grid, columns, stream)
                              : launch_typed<__nv_bfloat16>(p, grid, columns, stream);
    if (e != cudaSuccess || p.max_partitions <= 1) return e;
    const long long rows = (long long)p.num_seqs * p.num_heads;
    if (rows <= kMergeCtaRows)
        return launch_dependent(p.head_dim == 128 ? merge_q4_kernel<128> : merge_q4_kernel<64>,
                                rows, 128, 0, stream, p);
    return launch_dependent(
        p.head_dim == 128 ? merge_rows_q4_kernel<128> : merge_rows_q4_kernel<64>, (rows + 3) / 4,
        128, 0, stream, p);
}
