// Work plan of a split decode launch: the longest sequences first, no empty
// grid slots.
//
// A split launch's rectangular grid gives every (sequence, KV head, head
// slice) as many CTA slots as the longest context needs; with ragged
// lengths most of them are empty and exit at once, and the long items start
// wherever the caller put their sequence, so the launch often ends on a
// long item that started late.  This one-CTA kernel runs in place of the
// memset that zeroes the split's completion counters: it zeroes them, orders
// the sequences by context length, longest first (a counting sort on
// length buckets), and writes one record per CTA that has work -- (sequence,
// context length, KV head x head slice, partition group) -- consecutive in
// that order, plus their count.  The decode kernel's CTA b takes record b,
// or exits if b is past the count.  The order changes no result: every
// partition's softmax state and every merge are the same whichever CTA runs
// first.
//
// Both launches are programmatic dependent launches: the plan kernel starts
// while the previous decode launch's last CTAs still run (decode CTAs let
// dependents launch as they start) and makes a plan for the lengths as it finds
// them.  What the kernels before it wrote is visible only once they have completed,
// so it then waits for that, reads the lengths again, plans afresh if any differs
// (the kernel before was an extend of the block tables, say), and only now writes
// counters and records.  The decode CTAs are resident while the plan kernel
// finishes and wait for it to complete before they read a record.
#include <cuda_runtime.h>

#include <climits>

#include "pkv_kernels.h"

namespace {

constexpr int kPlanThreads = 1024;

struct PlanSmem {
    static constexpr int LENS = 0;                               // int [kPlanMaxSeqs]
    static constexpr int SORTED = LENS + kPlanMaxSeqs;           // int [kPlanMaxSeqs]
    static constexpr int OFF = SORTED + kPlanMaxSeqs;            // int [kPlanMaxSeqs]
    static constexpr int HIST = OFF + kPlanMaxSeqs;              // int [kPlanBuckets]
    static constexpr int WSUM = HIST + kPlanBuckets;             // int [32]
    static constexpr int INFO = WSUM + 32;                       // int [8], below
    static constexpr int INTS = INFO + 8;
    static constexpr int BYTES = INTS * 4;
    // INFO: over the non-empty sequences, the fewest and most stages, the
    // fewest partitions, their count; then the pieces per sequence (0: groups)
    static constexpr int MIN_NST = 0, MAX_NST = 1, MIN_PARTS = 2, NONEMPTY = 3, PIECES = 4,
                         TOTAL = 5, TARGET = 6;
};

// Pieces per sequence for near-equal contexts: the fewest c <= cmax whose
// items * c CTAs fill their last wave of `slots` to kPlanWaveFillPct; else
// the c with the fullest last wave (the fewest of equals).  One warp calls
// it, lane l trying c = l + 1, l + 33.  No c qualifies only when items is
// below ~20 waves of CTAs, so the products below stay far inside 64 bits.
__device__ int choose_pieces(long long items, int slots, int cmax)
{
    const int lane = threadIdx.x & 31;
    for (int c0 = 1; c0 <= cmax; c0 += 32) {
        const int c = c0 + lane;
        bool ok = false;
        if (c <= cmax) {
            const long long ctas = items * c;
            const long long room = (ctas + slots - 1) / slots * slots;
            ok = 100 * ctas >= (long long)kPlanWaveFillPct * room;
        }
        const unsigned m = __ballot_sync(0xffffffffu, ok);
        if (m != 0u) return c0 + __ffs(m) - 1;
    }
    int best = 1;
    long long bc = 0, br = 1;  // fill of `best`: bc / br
    for (int c = 1 + lane; c <= cmax; c += 32) {
        const long long ctas = items * c;
        const long long room = (ctas + slots - 1) / slots * slots;
        if (ctas * br > bc * room) {
            best = c;
            bc = ctas;
            br = room;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int b2 = __shfl_xor_sync(0xffffffffu, best, o);
        const long long c2 = __shfl_xor_sync(0xffffffffu, bc, o);
        const long long r2 = __shfl_xor_sync(0xffffffffu, br, o);
        const long long lhs = c2 * br, rhs = bc * r2;
        if (lhs > rhs || (lhs == rhs && b2 < best)) {
            best = b2;
            bc = c2;
            br = r2;
        }
    }
    return best;
}

// Exclusive prefix sum over the block of one value per thread; *total gets
// the sum.  Every thread of the block calls it.
__device__ int block_exclusive_scan(int v, int* wsum, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int w = lane < kPlanThreads / 32 ? wsum[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        wsum[lane] = w;  // inclusive over warps
    }
    __syncthreads();
    const int before = warp > 0 ? wsum[warp - 1] : 0;
    *total = wsum[kPlanThreads / 32 - 1];
    __syncthreads();  // wsum may be reused by the caller's next scan
    return before + x - v;
}

__global__ void __launch_bounds__(kPlanThreads) decode_plan_kernel(const DecodePlanParams pp)
{
    extern __shared__ int psm[];
    int* lens = psm + PlanSmem::LENS;
    int* sorted = psm + PlanSmem::SORTED;
    int* off = psm + PlanSmem::OFF;
    int* hist = psm + PlanSmem::HIST;
    int* wsum = psm + PlanSmem::WSUM;
    const int tid = threadIdx.x;
    const int S = pp.num_seqs;
    // the decode launch that follows may start now: its CTAs wait for this
    // grid to complete (griddepcontrol.wait) before they read anything it
    // writes
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    int* info = psm + PlanSmem::INFO;
    __shared__ unsigned long long stages;  // of all sequences
    const int P = pp.partition_tokens;
    const int per_seq = pp.num_kv_heads * pp.head_slices;
    int run = 0;  // records so far
    // a sequence with no tokens (or a bad length) keeps one record, whose
    // CTA writes its zero rows
    auto groups_of = [&](int L, int pieces, int target) {
        const int Lc = (L < 0 || L > pp.max_len) ? 0 : L;
        if (pieces > 0) return Lc > 0 ? pieces : 1;
        const int np = max(1, (Lc + pp.partition_tokens - 1) / pp.partition_tokens);
        if (target > 0) {
            const int nst = (Lc + pp.stage_tokens - 1) / pp.stage_tokens;
            return max(1, min(min(np, min(pp.max_groups, kPlanPieceMask)),
                              (nst + target - 1) / target));
        }
        return (np + pp.cta_parts - 1) / pp.cta_parts;
    };
    // How the sequences are cut, (pieces, target), by one warp: of the `ne` non-empty
    // ones the fewest and most stages and the fewest partitions, and all their stages.
    //
    // When the split contexts hold within 10 % the same number of stages, each gives
    // the same number of records a (KV head, head slice): `pieces` equal runs of stages,
    // as many as fill the GPU's waves (at most the partitions, and the groups, a
    // sequence has room for).
    //
    // Contexts of many lengths where the launch has room for pp.spare records beyond
    // one each (at least pp.slots): runs of at most `target` stages, what each of
    // the slots has to do on average, so that a long context does not outlast the
    // others and a short one is not cut for nothing.  4-bit attention of 256 ragged
    // contexts, 64 query heads on 8: partitions of 512 tokens 88 us, such runs 67; of
    // 1024 tokens 70 and 67 (twice, three times as many runs: 68, 72).
    //
    // Neither (0, 0): a record a partition group.
    auto choose = [&](int ne, int least, int most, int parts, long long stages) {
        int2 cut = make_int2(0, 0);
        if (pp.slots > 0 && ne > 0 && 10LL * most <= 11LL * least) {
            const int cmax = min(min(parts, pp.max_groups), min(kPlanMaxPieces, kPlanPieceMask));
            cut.x = choose_pieces((long long)ne * per_seq, pp.slots, max(cmax, 1));
            if (pp.spare > 0) cut.x = min(cut.x, pp.spare / (ne * per_seq) + 1);
        } else if (pp.spare > 0) {
            const long long each = (stages * per_seq + pp.slots - 1) / pp.slots;
            cut.y = (int)min(max(each, (long long)kPlanLeastStages), (long long)INT_MAX);
        }
        return cut;
    };
    // the lengths as they stand; read through L2, as are those below: what an earlier
    // read left in this SM's L1 would hide a change
    for (int s = tid; s < S; s += kPlanThreads) lens[s] = __ldcg(pp.context_lens + s);
    __syncthreads();
    // The order, the records of each sequence and their total, of lens[]; again if
    // the lengths turn out to be others
    for (bool known = false;; known = true) {
        if (S <= 32) {
            // few sequences: one warp, a sequence a lane, does what follows without a
            // histogram or a barrier
            if (tid < 32) {
                const int L = tid < S ? lens[tid] : 0;
                const int Lc = (L < 0 || L > pp.max_len) ? 0 : L;
                const bool there = tid < S && Lc > 0 && P > 0;
                const int nst = (Lc + pp.stage_tokens - 1) / pp.stage_tokens;
                const int least = __reduce_min_sync(0xffffffffu, there ? nst : INT_MAX);
                const int most = __reduce_max_sync(0xffffffffu, there ? nst : 0);
                const int parts =
                    __reduce_min_sync(0xffffffffu, there ? (Lc + P - 1) / P : INT_MAX);
                const int ne = __popc(__ballot_sync(0xffffffffu, there));
                const int all = __reduce_add_sync(0xffffffffu, there ? nst : 0);
                const int2 cut = choose(ne, least, most, parts, all);
                const int c = tid < S ? per_seq * groups_of(L, cut.x, cut.y) : 0;
                int rank = 0, before = 0;
                for (int o = 0; o < S; ++o) {  // longest first, then in their own order
                    const int Lo = __shfl_sync(0xffffffffu, Lc, o);
                    const int co = __shfl_sync(0xffffffffu, c, o);
                    if (Lo > Lc || (Lo == Lc && o < tid)) {
                        ++rank;
                        before += co;
                    }
                }
                const int total = __reduce_add_sync(0xffffffffu, c);
                if (tid < S) {
                    sorted[rank] = tid;
                    off[rank] = before;
                }
                if (tid == 0) {
                    info[PlanSmem::PIECES] = cut.x;
                    info[PlanSmem::TARGET] = cut.y;
                    info[PlanSmem::TOTAL] = total;
                }
            }
            __syncthreads();
            run = info[PlanSmem::TOTAL];
        } else {
            for (int k = tid; k < kPlanBuckets; k += kPlanThreads) hist[k] = 0;
            if (tid == 0) {
                info[PlanSmem::MIN_NST] = INT_MAX;
                info[PlanSmem::MAX_NST] = 0;
                info[PlanSmem::MIN_PARTS] = INT_MAX;
                info[PlanSmem::NONEMPTY] = 0;
                stages = 0;
            }
            __syncthreads();
            // histogram of length buckets, longest bucket first (index 0); the
            // spread and the sum of the non-empty sequences' stage counts
            unsigned long long mine = 0;
            for (int s = tid; s < S; s += kPlanThreads) {
                const int L = lens[s];
                const int Lc = (L < 0 || L > pp.max_len) ? 0 : L;  // the decode kernel flags it
                const int key = min(Lc >> pp.bucket_shift, kPlanBuckets - 1);
                atomicAdd(&hist[kPlanBuckets - 1 - key], 1);
                if (Lc > 0 && P > 0) {
                    const int nst = (Lc + pp.stage_tokens - 1) / pp.stage_tokens;
                    atomicMin(&info[PlanSmem::MIN_NST], nst);
                    atomicMax(&info[PlanSmem::MAX_NST], nst);
                    atomicMin(&info[PlanSmem::MIN_PARTS], (Lc + P - 1) / P);
                    atomicAdd(&info[PlanSmem::NONEMPTY], 1);
                    mine += nst;
                }
            }
            if (pp.spare > 0) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
                if ((tid & 31) == 0) atomicAdd(&stages, mine);
            }
            __syncthreads();
            if (tid < 32) {
                const int2 cut = choose(info[PlanSmem::NONEMPTY], info[PlanSmem::MIN_NST],
                                        info[PlanSmem::MAX_NST], info[PlanSmem::MIN_PARTS],
                                        (long long)stages);
                if (tid == 0) {
                    info[PlanSmem::PIECES] = cut.x;
                    info[PlanSmem::TARGET] = cut.y;
                }
            }
            // bucket starts: exclusive scan, two buckets per thread
            {
                static_assert(kPlanBuckets == 2 * kPlanThreads, "two buckets a thread");
                const int a = hist[2 * tid], b = hist[2 * tid + 1];
                int total;
                const int ex = block_exclusive_scan(a + b, wsum, &total);
                __syncthreads();
                hist[2 * tid] = ex;
                hist[2 * tid + 1] = ex + a;
            }
            __syncthreads();
            // rank of each sequence (any order within a bucket)
            for (int s = tid; s < S; s += kPlanThreads) {
                const int L = lens[s];
                const int Lc = (L < 0 || L > pp.max_len) ? 0 : L;
                const int key = min(Lc >> pp.bucket_shift, kPlanBuckets - 1);
                sorted[atomicAdd(&hist[kPlanBuckets - 1 - key], 1)] = s;
            }
            __syncthreads();
            // written before the barrier above
            const int pieces = info[PlanSmem::PIECES], target = info[PlanSmem::TARGET];
            for (int r0 = 0; r0 < S; r0 += kPlanThreads) {
                const int r = r0 + tid;
                const int c = r < S ? per_seq * groups_of(lens[sorted[r]], pieces, target) : 0;
                int total;
                const int ex = block_exclusive_scan(c, wsum, &total);
                if (r < S) off[r] = run + ex;
                run += total;
            }
            __syncthreads();
        }
        if (known) break;
        // what came before has completed and is visible: the lengths as they are
        asm volatile("griddepcontrol.wait;" ::: "memory");
        bool changed = false;
        for (int s = tid; s < S; s += kPlanThreads) {
            const int L = __ldcg(pp.context_lens + s);
            changed |= L != lens[s];
            lens[s] = L;
        }
        if (!__syncthreads_or(changed)) break;
        run = 0;
    }
    const int pieces = info[PlanSmem::PIECES], target = info[PlanSmem::TARGET];
    for (int i = tid; i < pp.num_counters; i += kPlanThreads) pp.done[i] = 0u;
    // a sequence's records: KV head, then partition group (or piece), then
    // head slice (the slices of one group adjacent: their reads of a K/V tile
    // meet in L2).  Few sequences have many threads each: one thread wrote a lone
    // sequence's 256 records in 18 us.
    const int HS = pp.head_slices;
    const int share = max(1, kPlanThreads / S);
    for (int r = tid / share; r < S; r += kPlanThreads / share) {
        const int s = sorted[r], L = lens[s];
        const int ng = groups_of(L, pieces, target), n = per_seq * ng;
        int4* out = pp.items + off[r];
        for (int i = tid % share; i < n; i += share) {
            const int hs = i % HS, t = i / HS, g = t / ng, grp = t - g * ng;
            const int w = pieces > 0 || target > 0
                              ? kPlanPieceFlag | grp | (ng << kPlanPieceBits)
                              : grp;
            out[i] = make_int4(s, L, g * HS + hs, w);
        }
    }
    if (tid == 0) *pp.item_count = run;
}

}  // namespace

cudaError_t launch_decode_plan(const DecodePlanParams& pp, cudaStream_t stream)
{
    cudaError_t e = cudaFuncSetAttribute(decode_plan_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         PlanSmem::BYTES);
    if (e != cudaSuccess) return e;
    // a programmatic dependent launch: it starts when the previous kernel on
    // the stream lets its dependents launch and waits for that kernel to complete
    // before it writes anything
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = PlanSmem::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_plan_kernel, pp);
}
