// Host program: the library's entry points (api.cu, api_q4.cu, compiled as they
// are) over stand-ins for the launches and for the few CUDA runtime calls they
// make.  It calls them on a stack filled with a pattern, and prints what the work
// plan and the attention kernel would have been launched with:
//     call pattern rc spare slots max_groups partition cta_parts stage counters parts grid
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdio>
#include <cstring>

#include "pkv.h"
#include "pkv_kernels.h"

namespace {

DecodePlanParams plan;
bool planned = false;
int parts = 0;
long long ctas = 0;

cudaError_t seen(const DecodeParams& p, long long grid)
{
    parts = p.max_partitions;
    ctas = grid;
    return cudaSuccess;
}

CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)
{
    return CUDA_SUCCESS;
}

}  // namespace

// ---- the runtime calls on the way to a launch ------------------------------
extern "C" {
cudaError_t cudaGetDevice(int* d)
{
    *d = 0;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int)
{
    *v = 152;
    return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned int,
                                             unsigned long long,
                                             cudaDriverEntryPointQueryResult* q)
{
    *fn = reinterpret_cast<void*>(&encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
}

// ---- the launches ----------------------------------------------------------
unsigned int* pkv_status_word_ptr()
{
    static unsigned int word;
    return &word;
}
cudaError_t launch_decode_plan(const DecodePlanParams& pp, cudaStream_t)
{
    plan = pp;
    planned = true;
    return cudaSuccess;
}
cudaError_t launch_decode_tensor_core(const DecodeParams& p, int, const void*, const void*,
                                      long long grid, cudaStream_t)
{
    return seen(p, grid);
}
cudaError_t launch_decode_tensor_core_wide(const DecodeParams& p, int, const void*, const void*,
                                           long long grid, cudaStream_t)
{
    return seen(p, grid);
}
cudaError_t launch_decode_tensor_core_deep(const DecodeParams& p, int, const void*, const void*,
                                           long long grid, bool, cudaStream_t)
{
    return seen(p, grid);
}
cudaError_t launch_decode_grouped(const DecodeParams& p, int, const void*, const void*,
                                  long long grid, bool, cudaStream_t)
{
    return seen(p, grid);
}
bool decode_wide_tcgen05_supported(int, int, int, int group, const void*)
{
    return group % kDecodeWideHeads == 0;
}
int decode_wide_tcgen05_heads(int group) { return group % 64 == 0 ? 64 : 32; }
cudaError_t launch_decode_wide_tcgen05(const DecodeParams& p, int, const void*, const void*,
                                       int items, int, cudaStream_t)
{
    return seen(p, items);
}
cudaError_t launch_decode_cuda_core(const DecodeParams& p, int, cudaStream_t) { return seen(p, 0); }
cudaError_t launch_decode_q4(const DecodeParams& p, int, long long grid, int, cudaStream_t)
{
    return seen(p, grid);
}
cudaError_t launch_lse_reduce(const DecodeParams&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_prefill_tensor_core(const PrefillParams&, int, const void*, const void*,
                                       cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_prefill_tcgen05(const PrefillParams&, int, const void*, const void*,
                                   cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_write(void*, void*, const void*, const void*, const int64_t*, int, int, int,
                            int, int, int, unsigned int*, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_append(void*, void*, const void*, const void*, const int32_t*, const int32_t*,
                             int, int, int, int, int, int, int, unsigned int*, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_copy_blocks(void*, void*, const int64_t*, int, int, size_t, unsigned int*,
                                  cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_swap_blocks(void*, void*, const void*, const void*, const int64_t*, int, int,
                                  int, size_t, unsigned int*, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_write_q4(const Q4CacheParams&, const void*, const void*, size_t, size_t, int,
                               int, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_kv_read_q4(const Q4CacheParams&, void*, void*, int, int, cudaStream_t)
{
    return cudaSuccess;
}
cudaError_t launch_tables_extend(const TablesParams&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_tables_release(const ReleaseParams&, cudaStream_t) { return cudaSuccess; }

namespace {

// Leaves `pattern` in every word of the stack below the caller's frame.
__attribute__((noinline)) int dirty(int pattern)
{
    volatile int words[16384];
    for (int i = 0; i < 16384; ++i) words[i] = pattern;
    return words[77];
}

struct Call {
    const char* name;
    bool q4;
    int heads, kv_heads, seqs, width, partition;
};

}  // namespace

int main()
{
    static char bytes[4096] __attribute__((aligned(256)));
    const Call calls[] = {
        {"split-warp-partitions", false, 64, 8, 4, 1024, 512},
        {"split-many", false, 32, 8, 64, 256, 1024},
        {"unsplit", false, 64, 8, 256, 256, 0},
        {"wide-group", false, 256, 8, 16, 256, 0},
        {"q4-split", true, 64, 8, 64, 256, 512},
        {"q4-unsplit", true, 64, 8, 1024, 256, 0},
        // the greatest partition of whole blocks: one a context
        {"huge-partition", false, 32, 8, 4, 64, INT_MAX / 32 * 32},
        {"q4-huge-partition", true, 32, 8, 4, 64, INT_MAX / 32 * 32},
    };
    const int block = 16, dim = 128, blocks = 1 << 16;
    for (const Call& c : calls)
        for (int pattern : {0, 5, 1000, 7777, 32729, -1}) {
            std::memset(&plan, 0, sizeof plan);
            planned = false;
            parts = 0;
            ctas = 0;
            const size_t need = pkv_decode_workspace_bytes(c.seqs, c.heads, dim, c.width * block,
                                                           c.partition);
            dirty(pattern);
            const int rc =
                (c.q4 ? pkv_paged_decode_attention_q4 : pkv_paged_decode_attention)(
                    bytes, bytes, bytes, bytes, reinterpret_cast<const int32_t*>(bytes),
                    reinterpret_cast<const int32_t*>(bytes), 0.1f, block, c.kv_heads, c.seqs,
                    c.heads, dim, c.width, blocks, PKV_BF16, PKV_BF16, c.partition, bytes, need,
                    nullptr);
            std::printf("%s %d %d %d %d %d %d %d %d %d %d %lld %d\n", c.name, pattern, rc,
                        plan.spare, plan.slots, plan.max_groups, plan.partition_tokens,
                        plan.cta_parts, plan.stage_tokens, plan.num_counters, parts, ctas,
                        (int)planned);
        }
    return 0;
}
