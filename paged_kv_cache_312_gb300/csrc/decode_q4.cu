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
//    higher, c * 2^-20), exact.  Eight codes become four operand registers with
//    four ANDs and a shift.  q is scaled by a power of two into fp16's range
//    (exact but for elements below 2^-34 of the row's greatest), the odd code
//    positions by another 2^-4.
//  * P V gets w_i = p_i s'_i * kappa in fp16: one rounding (2^-11), the only
//    one below 32 bits.  kappa, kept for each head and run, holds the greatest
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
// copies fill two stages ahead.  The warps' states are merged in shared memory; partials
// of a split item go to the workspace and the CTA that completes an item's
// count merges them by log-sum-exp.
#include <cuda_runtime.h>

#include <climits>

#include "pkv.h"
#include "pkv_kernels.h"
#include "q4_common.cuh"
#include "tc_common.cuh"

namespace {

using namespace pkv_tc;
using namespace pkv_q4;

constexpr int NW = kDecodeQ4Warps;
constexpr int ST = kDecodeQ4StageTokens;
constexpr int NS = 3;  // stages of a warp's ring

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^e for e in [-126, 127]
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// floor(log2 x) of a normal x > 0 (below: -127; infinity and NaN: 128)
__device__ __forceinline__ int exponent(float x) { return (int)(__float_as_uint(x) >> 23 & 255u) - 127; }

// The four operand registers of a word of eight codes (values c * 2^-24 in
// registers 0 and 2, c * 2^-20 in 1 and 3).
__device__ __forceinline__ void spread(uint32_t w, uint32_t (&r)[4])
{
    const uint32_t u = w >> 8;
    r[0] = w & 0x000F000Fu;
    r[1] = w & 0x00F000F0u;
    r[2] = u & 0x000F000Fu;
    r[3] = u & 0x00F000F0u;
}

template <typename T, int D, int NT>
struct Shape {
    static constexpr int R = D / kRun;       // runs of a row
    static constexpr int NC = 8 * NT;        // query-head columns
    static constexpr int GROUP_BYTES = 8 * (D / 2);        // codes of 8 tokens
    static constexpr int CODE_BYTES = 4 * GROUP_BYTES;     // K (or V) codes of a stage
    static constexpr int PAIR_BYTES = ST * R * 4;          // K (or V) pairs of a stage
    static constexpr int STAGE_BYTES = 2 * (CODE_BYTES + PAIR_BYTES);
    static constexpr int RING_BYTES = NS * STAGE_BYTES;
    static constexpr int GPC = 512 / GROUP_BYTES;          // groups a warp-wide copy brings
    static constexpr int K_CHUNKS = D / 32, V_CHUNKS = D / 16;  // of a K row, of a V pair's row
    static constexpr int MERGE_BYTES = NW * NC * (D + 2) * 4;
    static constexpr int SMEM_BYTES =
        NW * RING_BYTES > MERGE_BYTES ? NW * RING_BYTES : MERGE_BYTES;
};

template <typename T, int D, int NT>
__global__ void __launch_bounds__(NW * 32, decode_q4_ctas_per_sm(D, 8 * NT)) decode_q4_kernel(const DecodeParams p)
{
    using Sh = Shape<T, D, NT>;
    using H = Half16<T>;
    constexpr int R = Sh::R, NC = Sh::NC;
    extern __shared__ __align__(16) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tq = lane & 3;
    const int G = p.num_heads / p.num_kv_heads, HS = p.head_slices;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the item: record or grid slot (((s * Hkv) + g) * parts + part) * HS + hs
    int sg, part, L, piece = -1, npieces = 0;
    if (p.items != nullptr) {
        if ((int)blockIdx.x >= *p.item_count) return;
        const int4 it = p.items[blockIdx.x];
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
    if (L < 0 || (int64_t)L > (int64_t)p.max_blocks * p.block_size) {
        if (threadIdx.x == 0) atomicOr(p.status, PKV_STATUS_BAD_LEN);
        L = 0;
    }
    const int block_shift = 31 - __clz(p.block_size);
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
    const int cnt = nst > warp ? (nst - warp + NW - 1) / NW : 0;
    const int32_t* table = p.block_tables + (size_t)s * p.max_blocks;
    const size_t tile = tile_bytes(p.block_size, D);
    const uint32_t block_stride = (uint32_t)(tile * p.num_kv_heads);
    const uint8_t* kp = static_cast<const uint8_t*>(p.k_cache) + g * tile;
    const uint8_t* vp = static_cast<const uint8_t*>(p.v_cache) + g * tile;
    auto load_ids = [&](int j0) {
        const int tok = begin + (warp + (j0 + (lane >> 2)) * NW) * ST + (lane & 3) * 8;
        int id = -1;
        if (tok < end) {
            id = table[tok >> block_shift];
            if (id < 0 || id >= p.num_blocks) {
                atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
                id = -1;
            }
        }
        return id;
    };
    int ids = load_ids(0), ids_next = load_ids(8);
    // where this lane's 16 bytes of a copy come from and go: the groups of one
    // copy are GPC; chunks are swizzled so that the reads below hit every bank
    constexpr int GPC = Sh::GPC, LPG = 32 / GPC;  // groups a copy, lanes a group
    const int cl = lane % LPG;
    const int k_write = (cl / Sh::K_CHUNKS) * (D / 2) +
                        ((cl % Sh::K_CHUNKS) ^ (D == 128 ? (cl >> 3 & 1) << 1 : 0)) * 16;
    const int v_write = (cl / Sh::V_CHUNKS) * D +
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
    // pairs: lanes 0 .. 4 R * 4 / 4 - 1 copy K's, as many after them V's
    constexpr int PL = 8 * R;  // 16-byte chunks of a stage's K (or V) pairs
    const int pu = (lane % PL) / (2 * R), pc = lane % (2 * R);  // group and chunk
    const uint8_t* pp = (lane < PL ? kp : vp) + p.block_size * (D / 2) + pc * 16;
    const int in_block = p.block_size - 1;
    uint32_t live = 0;  // four bits a stage in flight: its groups with a block
    auto issue = [&](int j) {
        if (j < cnt) {
            if (j != 0 && (j & 7) == 0) {
                ids = ids_next;
                ids_next = load_ids(j + 8);
            }
            const int lane0 = (j & 7) * 4;
            uint8_t* st = ring + (j % NS) * Sh::STAGE_BYTES;
            const uint32_t have = __ballot_sync(0xffffffffu, ids >= 0) >> lane0 & 15u;
            live |= have << (4 * (NS - 1));
#pragma unroll
            for (int k = 0; k < 4 / GPC; ++k) {
                const int u = k * GPC + lane / LPG;
                const int id = __shfl_sync(0xffffffffu, ids, lane0 + u);
                if (id >= 0) {
                    const size_t off = (size_t)(uint32_t)id * block_stride +
                                       ((8 * u) & in_block) * (D / 2) + cl * 16;
                    uint8_t* dst = st + u * Sh::GROUP_BYTES;
                    cp_async16(smem_u32(dst + k_write), kp + off);
                    cp_async16(smem_u32(dst + Sh::CODE_BYTES + v_write), vp + off);
                }
            }
            const int id = __shfl_sync(0xffffffffu, ids, lane0 + pu);
            if (lane < 2 * PL && id >= 0)
                cp_async16(smem_u32(st + 2 * Sh::CODE_BYTES + lane * 16),
                           pp + (size_t)(uint32_t)id * block_stride +
                               ((8 * pu) & in_block) * (R * 4));
        }
        cp_async_commit();
    };
    for (int j = 0; j < NS - 1; ++j) {
        issue(j);
        live >>= 4;
    }

    // ---- Q as the B operand: column n = query head g * G + hb + n.  k-step
    // 4r + i pairs elements 64r + 16tq + {i, 4 + i} and + {8 + i, 12 + i}: the
    // order in which spread() leaves a K word's codes.
    uint32_t qb[NT][R * 4][2];
    float su[NT][2], sq[NT][R][2];  // scale * 2^24 / q's scaling, scale * sum q: columns 2tq, 2tq + 1
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const int n = 8 * t + gq;
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
                sq[t][r][c] = p.scale_log2 * __shfl_sync(0xffffffffu, sum[r], from);
        }
    }

    // ---- state of columns 8t + 2tq + c: reference maximum, sum of p, kappa,
    // sum of p (m' + 7.5 s'), sum of 7.5 w, sum of w c' (elements 64r + 8gq + n
    // in [0], [1] and + 4 in [2], [3])
    float mr[NT][2], l[NT][2], kap[NT][R][2], oz[NT][R][2], aw[NT][R][4], acc[NT][R * 4][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        mr[t][0] = mr[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            // any w overflows this kappa: the first tokens set it
            kap[t][r][0] = kap[t][r][1] = 0x1p120f;
            oz[t][r][0] = oz[t][r][1] = 0.f;
            aw[t][r][0] = aw[t][r][1] = aw[t][r][2] = aw[t][r][3] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < R * 4; ++i) acc[t][i][0] = acc[t][i][1] = acc[t][i][2] = acc[t][i][3] = 0.f;
    }

    // ---- stages
    for (int j = 0; j < cnt; ++j) {
        cp_async_wait<NS - 2>();
        __syncwarp();  // every lane's copies of stage j are in, and stage j - 1 is consumed
        issue(j + NS - 1);
        const int tok_s = begin + (warp + j * NW) * ST;
        const uint8_t* st = ring + (j % NS) * Sh::STAGE_BYTES;
        const uint32_t groups = live & 15u;
        live >>= 4;
#pragma unroll(NT == 1 ? 2 : 1)
        for (int hf = 0; hf < 2; ++hf) {
            const int tok0 = tok_s + hf * 16;
            if (tok0 >= end) break;
            // ---- this lane's tokens: K rows gq and gq + 8, V pairs tq and tq + 4
            uint2 kw[2][R], vw[2][R];
            uint32_t ks[2][R], vs[2][R];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* at = st + (2 * hf + u) * Sh::GROUP_BYTES;
                const uint8_t* pt = st + 2 * Sh::CODE_BYTES + ((2 * hf + u) * 8 + gq) * (R * 4);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    kw[u][r] = *reinterpret_cast<const uint2*>(at + k_read[r]);
                    vw[u][r] = *reinterpret_cast<const uint2*>(at + Sh::CODE_BYTES + v_read[r]);
                    ks[u][r] = *reinterpret_cast<const uint32_t*>(pt + 4 * r);
                    vs[u][r] = *reinterpret_cast<const uint32_t*>(pt + Sh::PAIR_BYTES + 4 * r);
                }
            }
            const bool full = tok0 + 16 <= end && (groups >> (2 * hf) & 3u) == 3u;
            bool valid[2] = {true, true};
            if (!full) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    valid[u] = tok0 + gq + 8 * u < end && (groups >> (2 * hf + u) & 1u);
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        if (!valid[u]) vs[u][r] = 0u;
                }
            }
            // ---- A_r = codes of K times Q, then the scores
            float x[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) x[t][0] = x[t][1] = x[t][2] = x[t][3] = 0.f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t a0[4], a1[4], a2[4], a3[4];
                spread(kw[0][r].x, a0);
                spread(kw[1][r].x, a1);
                spread(kw[0][r].y, a2);
                spread(kw[1][r].y, a3);
                float sc[NT][4];
#pragma unroll
                for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a[4] = {a0[i], a1[i], a2[i], a3[i]};
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        Mma<__half>::run(sc[t], a, qb[t][4 * r + i][0], qb[t][4 * r + i][1]);
                }
                const float2 sm0 = H::unpack(ks[0][r]), sm1 = H::unpack(ks[1][r]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        x[t][c] += sm0.x * (sc[t][c] * su[t][c]) + sm0.y * sq[t][r][c];
                        x[t][2 + c] += sm1.x * (sc[t][2 + c] * su[t][c]) + sm1.y * sq[t][r][c];
                    }
            }
            if (!full) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        if (!valid[0]) x[t][c] = -INFINITY;
                        if (!valid[1]) x[t][2 + c] = -INFINITY;
                    }
            }
            // ---- p, and w = p s' kappa, against the references as they stand
            float pr[NT][4], w[NT][R][4];
            float2 sm[2][R];  // (s', m') of tokens gq, gq + 8; masked ones are zero
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < R; ++r) sm[u][r] = H::unpack(vs[u][r]);
            bool up = false;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int c = e & 1, u = e >> 1;
                    const float m = mr[t][c];
                    pr[t][e] = ex2(x[t][e] - (m == -INFINITY ? 0.f : m));
                    up = up || x[t][e] > m + 8.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        w[t][r][e] = pr[t][e] * sm[u][r].x * kap[t][r][c];
                        up = up || w[t][r][e] > 4096.f;
                    }
                }
            if (__any_sync(0xffffffffu, up)) {
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(x[t][c], x[t][2 + c]);
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1)
                            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                        const float mn = fmaxf(mr[t][c], mx);
                        const float al = mn == -INFINITY ? 1.f : ex2(mr[t][c] - mn);
                        const float ms = mn == -INFINITY ? 0.f : mn;
                        mr[t][c] = mn;
                        l[t][c] *= al;
                        pr[t][c] = ex2(x[t][c] - ms);
                        pr[t][2 + c] = ex2(x[t][2 + c] - ms);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            // the greatest p s' of these tokens, or what the ones before weigh now
                            const float w0 = pr[t][c] * sm[0][r].x, w1 = pr[t][2 + c] * sm[1][r].x;
                            float top = fmaxf(w0, w1);
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1)
                                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                            const float was = al / kap[t][r][c];
                            top = fmaxf(top, was);
                            const float kn =
                                top > 0.f ? pow2(-min(max(exponent(top), -120), 120)) : kap[t][r][c];
                            const float f = was * kn;
                            kap[t][r][c] = kn;
                            oz[t][r][c] *= al;
                            aw[t][r][c] *= f;
                            aw[t][r][2 + c] *= f;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                acc[t][4 * r + i][c] *= f;
                                acc[t][4 * r + i][2 + c] *= f;
                            }
                            w[t][r][c] = w0 * kn;
                            w[t][r][2 + c] = w1 * kn;
                        }
                    }
            }
            uint32_t wb[NT][R][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int c = 0; c < 2; ++c) l[t][c] += pr[t][c] + pr[t][2 + c];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float z0 = fmaf(7.5f, sm[0][r].x, sm[0][r].y);
                    const float z1 = fmaf(7.5f, sm[1][r].x, sm[1][r].y);
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        oz[t][r][c] = fmaf(pr[t][c], z0, fmaf(pr[t][2 + c], z1, oz[t][r][c]));
                    wb[t][r][0] = movmatrix_trans(Half16<__half>::pack(w[t][r][0], w[t][r][1]));
                    wb[t][r][1] = movmatrix_trans(Half16<__half>::pack(w[t][r][2], w[t][r][3]));
                }
            }
            // ---- O^T += codes of V^T times w
            const uint32_t mid[4] = {0x47804780u, 0x47804780u, 0x47804780u, 0x47804780u};  // 7.5
#pragma unroll
            for (int r = 0; r < R; ++r) {
                uint32_t a0[4], a1[4], a2[4], a3[4];
                spread(vw[0][r].x, a0);
                spread(vw[0][r].y, a1);
                spread(vw[1][r].x, a2);
                spread(vw[1][r].y, a3);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    Mma<__half>::run(aw[t][r], mid, wb[t][r][0], wb[t][r][1]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a[4] = {a0[i], a1[i], a2[i], a3[i]};
                        Mma<__half>::run(acc[t][4 * r + i], a, wb[t][r][0], wb[t][r][1]);
                    }
                }
            }
        }
    }

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
            if (gq == 0) {
                wm[NC * D + n] = mr[t][c];
                wm[NC * D + NC + n] = l[t][c];
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float inv = 1.f / kap[t][r][c];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float unit = i & 1 ? 0x1p20f : 0x1p24f;
                    float* o = wm + n * D + 64 * r + 8 * gq + i;
                    o[0] = fmaf(fmaf(acc[t][4 * r + i][c], unit, -aw[t][r][c]), inv, oz[t][r][c]);
                    o[4] = fmaf(fmaf(acc[t][4 * r + i][2 + c], unit, -aw[t][r][2 + c]), inv,
                                oz[t][r][c]);
                }
            }
        }
    __syncthreads();

    // ---- merge the warps
    const size_t hbase = (size_t)s * p.num_heads + (size_t)g * G + hb;
    const bool vec_out = (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
    for (int idx = threadIdx.x; idx < ncol * D / 4; idx += NW * 32) {
        const int n = idx / (D / 4), d = (idx - n * (D / 4)) * 4;
        float M = -INFINITY;
#pragma unroll
        for (int k = 0; k < NW; ++k) M = fmaxf(M, merge[k * NC * (D + 2) + NC * D + n]);
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            const float* ww = merge + k * NC * (D + 2);
            const float mw = ww[NC * D + n];
            const float wt = mw == -INFINITY ? 0.f : ex2(mw - M);
            den = fmaf(wt, ww[NC * D + NC + n], den);
            const float4 o = *reinterpret_cast<const float4*>(ww + n * D + d);
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
    if (nparts <= 1) return;

    // ---- split: the CTA that completes the item's count merges its partials
    __shared__ int is_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        unsigned prev;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
                     : "=r"(prev)
                     : "l"(&p.done[sg]), "r"(1u)
                     : "memory");
        is_last = prev == (unsigned)(nparts - 1);
    }
    __syncthreads();
    if (!is_last) return;
    for (int idx = threadIdx.x; idx < ncol * D / 4; idx += NW * 32) {
        const int n = idx / (D / 4), d = (idx - n * (D / 4)) * 4;
        const size_t base = (hbase + n) * p.max_partitions;
        float M = -INFINITY;
        for (int i = 0; i < nparts; ++i) M = fmaxf(M, __ldcg(&p.ws_ml[base + i]).x);
        float den = 0.f;
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < nparts; ++i) {
            const float2 ml = __ldcg(&p.ws_ml[base + i]);
            const float wt = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
            den = fmaf(wt, ml.y, den);
            const float4 o = __ldcg(reinterpret_cast<const float4*>(p.ws_o + (base + i) * D + d));
            num.x = fmaf(wt, o.x, num.x);
            num.y = fmaf(wt, o.y, num.y);
            num.z = fmaf(wt, o.z, num.z);
            num.w = fmaf(wt, o.w, num.w);
        }
        const float inv = den == 0.f ? 0.f : 1.f / den;
        store_out4(p.out, (hbase + n) * D + d,
                   make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv), p.out_dtype,
                   vec_out);
    }
}

template <typename T, int D, int NT>
cudaError_t launch(const DecodeParams& p, long long grid, cudaStream_t stream)
{
    auto kern = decode_q4_kernel<T, D, NT>;
    constexpr int smem = Shape<T, D, NT>::SMEM_BYTES;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename T>
cudaError_t launch_typed(const DecodeParams& p, long long grid, int columns, cudaStream_t stream)
{
    if (p.head_dim == 128)
        return columns > 8 ? launch<T, 128, 2>(p, grid, stream) : launch<T, 128, 1>(p, grid, stream);
    return columns > 8 ? launch<T, 64, 2>(p, grid, stream) : launch<T, 64, 1>(p, grid, stream);
}

}  // namespace

cudaError_t launch_decode_q4(const DecodeParams& p, int kv_dtype, long long grid, int columns,
                             cudaStream_t stream)
{
    return kv_dtype == PKV_F16 ? launch_typed<__half>(p, grid, columns, stream)
                               : launch_typed<__nv_bfloat16>(p, grid, columns, stream);
}
