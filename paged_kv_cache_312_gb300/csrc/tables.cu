// Block tables and slot map of a step, built on the GPU from the requests'
// lengths, and the release of finished requests.
//
// The pool's free blocks are a stack in device memory, so that a decode loop
// needs no host round trip and one graph serves every step.  Request s holds
// ceil(len / B) blocks; a step that adds n tokens needs
//     need_s = ceil((len + n) / B) - ceil(len / B)
// more, and takes them from the stack's top in request order:
//     fresh block k of request s = stack[count - 1 - (first_s + k)],
//     first_s = sum of need over the requests before s.
// Row r of the step belongs to the request with query_start[s] <= r <
// query_start[s + 1], sits at position len + r - query_start[s], and its slot
// is block * B + position % B.  Everything follows from two prefix sums, so
// one CTA scans the requests and then each row is on its own: the row at a
// block's first position also writes the block's table entry.
//
// The host allocator takes and gives back blocks in the same order, so both
// hand out the same blocks from the same stack.
//
// The scan of a step or release in two launches lets its second kernel become
// resident early; that one waits for the scan, as every kernel of this library
// waits for the one before it before it takes a length or a table entry as given.
//
// All of it is latency: a step of 64 rows takes 3.1 us (two dependent loads, a
// scan, a search in shared memory, two more loads), one of 518,000 rows of 1000
// requests 8.4 us, of which its 6.8 MB are 1.0 at the copy rate.
#include <cuda_runtime.h>

#include "pdl.cuh"
#include "pkv.h"
#include "pkv_kernels.h"

namespace {

using namespace pkv_pdl;

constexpr int kThreads = 1024;
// Small steps and releases run in one CTA and one launch, others as a scan and a
// grid.  One launch against two, us: steps of 64 rows of 16 requests 2.8 and 4.3,
// of 2048 rows 3.9 and 4.5 (256 requests: 4.4 and 5.1; 2048: 7.8 and 9.4), of 4096
// rows of 256 requests 6.3 and 4.9 (2048: 9.6 and 7.9); releases over 1024 table
// entries 3.0 and 3.5, over 1152 3.6 and 3.6, over 4096 5.2 and 3.5.
constexpr int kSmallRows = 2048;
constexpr int kSmallSeqs = 2048;
constexpr int kSmallEntries = 1024;

// Exclusive prefix sums over the block of two values per thread; totals in
// *ta, *tb.  Every thread of the block calls it.
__device__ void scan2(long long a, long long b, long long& ea, long long& eb, long long& ta,
                      long long& tb)
{
    __shared__ long long wa[32], wb[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, x, o);
        const long long v = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x += u;
            y += v;
        }
    }
    if (lane == 31) {
        wa[warp] = x;
        wb[warp] = y;
    }
    __syncthreads();
    if (warp == 0) {
        long long p = wa[lane], q = wb[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, p, o);
            const long long v = __shfl_up_sync(0xffffffffu, q, o);
            if (lane >= o) {
                p += u;
                q += v;
            }
        }
        wa[lane] = p;
        wb[lane] = q;
    }
    __syncthreads();
    ea = (warp ? wa[warp - 1] : 0) + x - a;
    eb = (warp ? wb[warp - 1] : 0) + y - b;
    ta = wa[31];
    tb = wb[31];
    __syncthreads();  // the caller's next scan writes wa and wb again
}

// What request s asks for: its tokens and fresh blocks, none (and the flag)
// for a length that is negative or would pass the table.
__device__ __forceinline__ void request(const TablesParams& p, int s, int& len, int& tokens,
                                        int& blocks)
{
    len = p.context_lens[s];
    tokens = p.new_tokens[s];
    blocks = 0;
    const long long after = (long long)len + tokens;
    if (len < 0 || tokens < 0 || after > (long long)p.max_blocks * p.block_size) {
        atomicOr(p.status, PKV_STATUS_BAD_LEN);
        tokens = 0;
        return;
    }
    blocks = (int)((after + p.block_size - 1) / p.block_size -
                   ((long long)len + p.block_size - 1) / p.block_size);
}

// What the rows of a step need of its requests, in shared memory where they
// fit: first row, length before the step, stack place of block 0 (fresh block j
// is at place - j).
struct Requests {
    int *start, *len, *place;  // [num_seqs + 1], [num_seqs], [num_seqs]
};

// Scans the requests: query_start, first fresh block (ws), lengths and count,
// and a small step's copies (r.start not NULL).  A step that needs more blocks
// or rows than there are changes nothing: all its rows are padding.
__device__ void scan_requests(const TablesParams& p, const Requests& r)
{
    const int tid = threadIdx.x;
    const int count = *p.free_count;
    long long tokens_before = 0, blocks_before = 0;
    int len = 0, tokens = 0, blocks = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kThreads) {
        const int s = s0 + tid;
        len = tokens = blocks = 0;
        if (s < p.num_seqs) request(p, s, len, tokens, blocks);
        long long et, eb, tt, tb;
        scan2(tokens, blocks, et, eb, tt, tb);
        if (s < p.num_seqs) {
            // beyond the limits these are never used: the step is refused
            const int first = (int)min(blocks_before + eb, (long long)p.num_blocks);
            const int row = (int)min(tokens_before + et, (long long)p.max_tokens);
            p.query_start[s] = row;
            if (r.start) {
                r.start[s] = row;
                r.len[s] = len;
                r.place[s] = count - 1 - first + (len + p.block_size - 1) / p.block_size;
            } else {
                p.ws[s] = first;
            }
        }
        tokens_before += tt;
        blocks_before += tb;
    }
    const bool refused = count < 0 || count > p.num_blocks || blocks_before > count ||
                         tokens_before > p.max_tokens;
    // every length was read above; each is read again only by the thread that
    // writes it, so lens_out may be context_lens
    for (int s = tid; s < p.num_seqs; s += kThreads) {
        if (p.num_seqs > kThreads) request(p, s, len, tokens, blocks);
        p.lens_out[s] = refused ? len : len + tokens;
        if (refused) p.query_start[s] = 0;
    }
    __syncthreads();  // all threads have read the count
    if (tid == 0) {
        const int total = refused ? 0 : (int)tokens_before;
        p.query_start[p.num_seqs] = total;
        if (r.start) r.start[p.num_seqs] = total;
        p.ws[p.num_seqs] = count;
        *p.count_out = refused ? count : count - (int)blocks_before;
        if (refused) atomicOr(p.status, PKV_STATUS_REFUSED);
    }
    __syncthreads();
}

// The request of row r: the last s with start[s] <= r.
__device__ __forceinline__ int find(const int* start, int num_seqs, int r)
{
    int lo = 0, hi = num_seqs;  // start[lo] <= r < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Rows r0 .. r0 + 3 of the step: one search, then on from row to row.  `start`
// is query_start, or its copy in shared memory.
__device__ __forceinline__ void fill_four(const TablesParams& p, const int* start, int total,
                                          int count, int r0, bool vector)
{
    int64_t slot[4];
    int32_t pos[4];
    int s = -1, end = 0, p0 = 0, held = 0, fresh = 0, j = -1, at = 0, id = -1;
    const int32_t* row = nullptr;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + i;
        slot[i] = -1;
        pos[i] = 0;
        if (r >= total) continue;
        const bool next = r >= end;
        if (next) {
            s = find(start, p.num_seqs, r);
            const int q0 = start[s];
            end = start[s + 1];
            const int len = p.lens_out[s] - (end - q0);
            held = len / p.block_size + (len % p.block_size != 0);
            p0 = len - q0;
            fresh = count - 1 - p.ws[s] + held;  // stack place of block j: fresh - j
            row = p.block_tables + (size_t)s * p.max_blocks;
            j = (p0 + r) / p.block_size;
            at = p0 + r - j * p.block_size;
        } else if (++at == p.block_size) {
            at = 0;
            ++j;
        }
        if (next || at == 0) {
            id = j >= held ? p.free_list[fresh - j] : row[j];
            // the block's first row is in this step, and writes its entry
            if (j >= held && at == 0) const_cast<int32_t*>(row)[j] = id;
            if (id < 0 || id >= p.num_blocks) {
                atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
                id = -1;
            }
        }
        pos[i] = p0 + r;
        if (id >= 0) slot[i] = (int64_t)id * p.block_size + at;
    }
    if (vector && r0 + 4 <= p.max_tokens) {
        longlong2* out = reinterpret_cast<longlong2*>(p.slot_mapping + r0);
        out[0] = make_longlong2(slot[0], slot[1]);
        out[1] = make_longlong2(slot[2], slot[3]);
        if (p.positions)
            *reinterpret_cast<int4*>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (r0 + i < p.max_tokens) {
            p.slot_mapping[r0 + i] = slot[i];
            if (p.positions) p.positions[r0 + i] = pos[i];
        }
}

// Threads first, first + step, ... of the step's rows, four rows each.  The
// searches go through shared memory where the starts fit.
constexpr int kSharedStarts = 4096;

__device__ void fill_rows(const TablesParams& p, int* shared, int first, int step)
{
    const bool vector = (reinterpret_cast<uintptr_t>(p.slot_mapping) & 15) == 0 &&
                        (reinterpret_cast<uintptr_t>(p.positions) & 15) == 0;
    const int* start = p.query_start;
    if (p.num_seqs < kSharedStarts) {
        for (int s = threadIdx.x; s <= p.num_seqs; s += blockDim.x) shared[s] = p.query_start[s];
        __syncthreads();
        start = shared;
    }
    const int total = start[p.num_seqs], count = p.ws[p.num_seqs];
    for (long long r0 = 4ll * first; r0 < p.max_tokens; r0 += 4ll * step)
        fill_four(p, start, total, count, (int)r0, vector);
}

// A small step in one CTA: scan, then a thread a row.
__global__ void __launch_bounds__(kThreads) extend_small_kernel(const TablesParams p)
{
    __shared__ int start[kSmallSeqs + 1], len[kSmallSeqs], place[kSmallSeqs];
    wait_for_previous();
    scan_requests(p, Requests{start, len, place});
    const int total = start[p.num_seqs];
    for (int r = threadIdx.x; r < p.max_tokens; r += kThreads) {
        int64_t slot = -1;
        int pos = 0;
        if (r < total) {
            const int s = find(start, p.num_seqs, r);
            pos = len[s] + r - start[s];
            const int j = pos / p.block_size, at = pos - j * p.block_size;
            int32_t* entry = p.block_tables + (size_t)s * p.max_blocks + j;
            const bool fresh = j >= (len[s] + p.block_size - 1) / p.block_size;
            const int id = fresh ? p.free_list[place[s] - j] : *entry;
            // the block's first row is in this step, and writes its entry
            if (fresh && at == 0) *entry = id;
            if (id >= 0 && id < p.num_blocks)
                slot = (int64_t)id * p.block_size + at;
            else
                atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        }
        p.slot_mapping[r] = slot;
        if (p.positions) p.positions[r] = pos;
    }
}

__global__ void __launch_bounds__(kThreads) extend_scan_kernel(const TablesParams p)
{
    let_next_start();  // the rows' kernel: resident when the scan ends
    wait_for_previous();
    scan_requests(p, Requests{nullptr, nullptr, nullptr});
}

__global__ void __launch_bounds__(256) extend_rows_kernel(const TablesParams p)
{
    __shared__ int starts[kSharedStarts];
    wait_for_previous();
    fill_rows(p, starts, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
}

// ---- release -----------------------------------------------------------------

// Blocks that request s gives back (0 if it stays, or for a bad length).
__device__ __forceinline__ int given_back(const ReleaseParams& p, int s)
{
    if (p.release[s] == 0) return 0;
    const int len = p.context_lens[s];
    if (len < 0 || (long long)len > (long long)p.max_blocks * p.block_size) {
        atomicOr(p.status, PKV_STATUS_BAD_LEN);
        return 0;
    }
    return len / p.block_size + (len % p.block_size != 0);
}

// Stack place of each request's last block (ws): the last request is pushed
// first, and of a request its last block, so that releasing what an extend
// took puts the stack back as it was.
__device__ void scan_release(const ReleaseParams& p)
{
    const int tid = threadIdx.x;
    const int count = *p.free_count;
    long long before = 0;
    for (int i0 = 0; i0 < p.num_seqs; i0 += kThreads) {
        const int s = p.num_seqs - 1 - (i0 + tid);
        const int n = s >= 0 ? given_back(p, s) : 0;
        long long e, eb, t, tb;
        scan2(n, 0, e, eb, t, tb);
        if (s >= 0) p.ws[s] = (int)min(before + e, (long long)p.num_blocks);
        before += t;
    }
    __syncthreads();  // all threads have read the count
    if (tid == 0) {
        const bool refused = count < 0 || count + before > p.num_blocks;
        p.ws[p.num_seqs] = refused ? -1 : count;
        if (refused)
            atomicOr(p.status, PKV_STATUS_REFUSED);
        else
            *p.free_count = count + (int)before;
    }
    __syncthreads();
}

// Block j of request s goes onto the stack, and out of the table.
__device__ __forceinline__ void give_back(const ReleaseParams& p, int s, int j, int n, int base)
{
    int32_t* entry = p.block_tables + (size_t)s * p.max_blocks + j;
    const int id = *entry;
    if (id < 0 || id >= p.num_blocks) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
    p.free_list[base + n - 1 - j] = id;
    *entry = -1;
}

// A small release in one CTA: the scan, then a thread an entry.
__global__ void __launch_bounds__(kThreads) release_small_kernel(const ReleaseParams p)
{
    wait_for_previous();
    scan_release(p);
    const int count = p.ws[p.num_seqs];
    if (count < 0) return;
    for (int i = threadIdx.x; i < p.num_seqs * p.max_blocks; i += kThreads) {
        const int s = i / p.max_blocks, j = i - s * p.max_blocks;
        const int n = given_back(p, s);
        if (j < n) give_back(p, s, j, n, count + p.ws[s]);
    }
    __syncthreads();  // all threads have read the lengths
    for (int s = threadIdx.x; s < p.num_seqs; s += kThreads)
        if (given_back(p, s) > 0) p.context_lens[s] = 0;
}

__global__ void __launch_bounds__(kThreads) release_scan_kernel(const ReleaseParams p)
{
    let_next_start();
    wait_for_previous();
    scan_release(p);
}

// One CTA per request.
__global__ void __launch_bounds__(128) release_rows_kernel(const ReleaseParams p)
{
    wait_for_previous();
    const int s = blockIdx.x, count = p.ws[p.num_seqs];
    if (count < 0) return;
    const int n = given_back(p, s);
    for (int j = threadIdx.x; j < n; j += blockDim.x) give_back(p, s, j, n, count + p.ws[s]);
    __syncthreads();  // all threads have read the length
    if (threadIdx.x == 0 && n > 0) p.context_lens[s] = 0;
}

}  // namespace

cudaError_t launch_tables_extend(const TablesParams& p, cudaStream_t stream)
{
    if (p.max_tokens <= kSmallRows && p.num_seqs <= kSmallSeqs)
        return launch_dependent(extend_small_kernel, 1, kThreads, 0, stream, p);
    const cudaError_t e = launch_dependent(extend_scan_kernel, 1, kThreads, 0, stream, p);
    if (e != cudaSuccess) return e;
    const int ctas = (p.max_tokens - 1) / 1024 + 1;
    return launch_dependent(extend_rows_kernel, ctas < 4096 ? ctas : 4096, 256, 0, stream, p);
}

cudaError_t launch_tables_release(const ReleaseParams& p, cudaStream_t stream)
{
    if ((int64_t)p.num_seqs * p.max_blocks <= kSmallEntries)
        return launch_dependent(release_small_kernel, 1, kThreads, 0, stream, p);
    const cudaError_t e = launch_dependent(release_scan_kernel, 1, kThreads, 0, stream, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(release_rows_kernel, p.num_seqs, 128, 0, stream, p);
}
