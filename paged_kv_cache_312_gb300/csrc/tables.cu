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
#include <cuda_runtime.h>

#include "pkv.h"
#include "pkv_kernels.h"

namespace {

constexpr int kThreads = 1024;

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

// Scans the requests: query_start, first fresh block (ws), lengths and count.
// A step that needs more blocks or rows than there are changes nothing: all
// its rows are padding.
__device__ void scan_requests(const TablesParams& p)
{
    const int tid = threadIdx.x;
    const int count = *p.free_count;
    long long tokens_before = 0, blocks_before = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kThreads) {
        const int s = s0 + tid;
        int len = 0, tokens = 0, blocks = 0;
        if (s < p.num_seqs) request(p, s, len, tokens, blocks);
        long long et, eb, tt, tb;
        scan2(tokens, blocks, et, eb, tt, tb);
        if (s < p.num_seqs) {
            // beyond the limits these are never used: the step is refused
            p.query_start[s] = (int)min(tokens_before + et, (long long)p.max_tokens);
            p.ws[s] = (int)min(blocks_before + eb, (long long)p.num_blocks);
        }
        tokens_before += tt;
        blocks_before += tb;
    }
    const bool refused = count < 0 || count > p.num_blocks || blocks_before > count ||
                         tokens_before > p.max_tokens;
    // every length was read above; each is read again only by the thread that
    // writes it, so lens_out may be context_lens
    for (int s = tid; s < p.num_seqs; s += kThreads) {
        int len, tokens, blocks;
        request(p, s, len, tokens, blocks);
        p.lens_out[s] = refused ? len : len + tokens;
        if (refused) p.query_start[s] = 0;
    }
    __syncthreads();  // all threads have read the count
    if (tid == 0) {
        p.query_start[p.num_seqs] = refused ? 0 : (int)tokens_before;
        p.ws[p.num_seqs] = count;
        *p.count_out = refused ? count : count - (int)blocks_before;
        if (refused) atomicOr(p.status, PKV_STATUS_REFUSED);
    }
    __syncthreads();
}

// The request of row r: the last s with query_start[s] <= r.
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

// Rows first, first + step, ... of the step.
__device__ void fill_rows(const TablesParams& p, int first, int step)
{
    const int total = p.query_start[p.num_seqs];
    const int count = p.ws[p.num_seqs];
    for (long long rr = first; rr < p.max_tokens; rr += step) {
        const int r = (int)rr;
        if (r >= total) {
            p.slot_mapping[r] = -1;
            if (p.positions) p.positions[r] = 0;
            continue;
        }
        const int s = find(p.query_start, p.num_seqs, r);
        const int q0 = p.query_start[s];
        const int len = p.lens_out[s] - (p.query_start[s + 1] - q0);
        const int pos = len + (r - q0);
        const int j = pos / p.block_size, at = pos - j * p.block_size;
        const int held = len / p.block_size + (len % p.block_size != 0);
        int32_t* entry = p.block_tables + (size_t)s * p.max_blocks + j;
        int id;
        if (j >= held) {
            id = p.free_list[count - 1 - (p.ws[s] + j - held)];
            if (at == 0) *entry = id;
        } else {
            id = *entry;
        }
        const bool ok = id >= 0 && id < p.num_blocks;
        if (!ok) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        p.slot_mapping[r] = ok ? (int64_t)id * p.block_size + at : -1;
        if (p.positions) p.positions[r] = pos;
    }
}

__global__ void __launch_bounds__(kThreads) extend_scan_kernel(const TablesParams p)
{
    scan_requests(p);
}

__global__ void __launch_bounds__(256) extend_rows_kernel(const TablesParams p)
{
    fill_rows(p, blockIdx.x * blockDim.x + threadIdx.x, gridDim.x * blockDim.x);
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
__global__ void __launch_bounds__(kThreads) release_scan_kernel(const ReleaseParams p)
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
    __syncthreads();
    if (tid == 0) {
        const bool refused = count < 0 || count + before > p.num_blocks;
        p.ws[p.num_seqs] = refused ? -1 : count;
        if (refused)
            atomicOr(p.status, PKV_STATUS_REFUSED);
        else
            *p.free_count = count + (int)before;
    }
}

// One CTA per request copies its table row onto the stack and empties it.
__global__ void __launch_bounds__(128) release_rows_kernel(const ReleaseParams p)
{
    const int s = blockIdx.x;
    const int count = p.ws[p.num_seqs];
    if (count < 0) return;
    const int n = given_back(p, s);
    const int base = count + p.ws[s];
    int32_t* row = p.block_tables + (size_t)s * p.max_blocks;
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int id = row[j];
        if (id < 0 || id >= p.num_blocks) atomicOr(p.status, PKV_STATUS_BAD_BLOCK);
        p.free_list[base + n - 1 - j] = id;
        row[j] = -1;
    }
    __syncthreads();  // all threads have read the length
    if (threadIdx.x == 0 && n > 0) p.context_lens[s] = 0;
}

}  // namespace

cudaError_t launch_tables_extend(const TablesParams& p, cudaStream_t stream)
{
    extend_scan_kernel<<<1, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || p.max_tokens == 0) return e;
    const int ctas = (p.max_tokens + 255) / 256;
    extend_rows_kernel<<<ctas < 4096 ? ctas : 4096, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_tables_release(const ReleaseParams& p, cudaStream_t stream)
{
    release_scan_kernel<<<1, kThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    release_rows_kernel<<<p.num_seqs, 128, 0, stream>>>(p);
    return cudaGetLastError();
}
