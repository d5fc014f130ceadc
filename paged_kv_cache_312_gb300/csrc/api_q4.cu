// C-ABI entry points of the 4-bit cache and of the GPU block tables (declared
// in include/pkv.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "pkv.h"
#include "pkv_internal.h"
#include "pkv_kernels.h"
#include "q4_common.cuh"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_fail(cudaError_t e, const char* where)
{
    return pkv_fail(PKV_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

// log2 of a block size of 8, 16 or 32
int block_shift(int block_size) { return block_size == 8 ? 3 : block_size == 16 ? 4 : 5; }

// Checks that a write into a 4-bit pool and a read from it share.
int check_cache(const char* fn, int num_tokens, int num_blocks, int num_kv_heads, int head_dim,
                int block_size, int dtype)
{
    if (!pkv_dtype_bytes(dtype)) return pkv_fail(PKV_ERR_DTYPE, "%s: dtype %d", fn, dtype);
    if (dtype == PKV_F32)
        return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: the 4-bit cache holds 16-bit types only", fn);
    if (head_dim != 64 && head_dim != 128)
        return pkv_fail(PKV_ERR_SHAPE, "%s: head_dim %d not in {64,128}", fn, head_dim);
    if (block_size != 8 && block_size != 16 && block_size != 32)
        return pkv_fail(PKV_ERR_SHAPE, "%s: block_size %d not in {8,16,32}", fn, block_size);
    if (num_tokens < 0 || num_blocks < 0 || num_kv_heads <= 0 || num_kv_heads > 65535)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d tokens, %d blocks, %d KV heads", fn, num_tokens,
                        num_blocks, num_kv_heads);
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: cache has >= 2^31 rows", fn);
    if ((int64_t)num_tokens * num_kv_heads >= (1ll << 32))
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d tokens of %d heads are >= 2^32 rows", fn, num_tokens,
                        num_kv_heads);
    return PKV_OK;
}

}  // namespace

extern "C" {

size_t pkv_q4_tile_bytes(int block_size, int head_dim)
{
    if ((block_size != 8 && block_size != 16 && block_size != 32) ||
        (head_dim != 64 && head_dim != 128))
        return 0;
    return pkv_q4::tile_bytes(block_size, head_dim);
}

int pkv_kv_write_q4(void* k_pool, void* v_pool, const void* key, const void* value,
                    const int64_t* slot_mapping, int num_tokens, int64_t key_stride,
                    int64_t value_stride, int num_blocks, int num_kv_heads, int head_dim,
                    int block_size, int dtype, void* stream)
{
    static const char* fn = "pkv_kv_write_q4";
    const int rc =
        check_cache(fn, num_tokens, num_blocks, num_kv_heads, head_dim, block_size, dtype);
    if (rc != PKV_OK) return rc;
    const int64_t row = (int64_t)num_kv_heads * head_dim;
    if (num_tokens > 1 && (key_stride < row || value_stride < row || key_stride % 8 != 0 ||
                           value_stride % 8 != 0))
        return pkv_fail(PKV_ERR_SHAPE,
                        "%s: token strides %lld, %lld must be multiples of 8 of at least %lld", fn,
                        (long long)key_stride, (long long)value_stride, (long long)row);
    if (num_tokens == 0) return PKV_OK;
    if (!k_pool || !v_pool || !key || !value || !slot_mapping)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(key, 16) || !aligned(value, 16) ||
        !aligned(slot_mapping, 8))
        return pkv_fail(PKV_ERR_ALIGN, "%s: pools, key and value need 16-byte alignment", fn);
    Q4CacheParams p{k_pool,     v_pool,       slot_mapping, num_tokens,
                    num_blocks, num_kv_heads, block_size,   block_shift(block_size),
                    pkv_status_word_ptr()};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e =
        launch_kv_write_q4(p, key, value, (size_t)key_stride, (size_t)value_stride, head_dim,
                           dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_kv_read_q4(void* key, void* value, const void* k_pool, const void* v_pool,
                   const int64_t* slot_mapping, int num_tokens, int num_blocks, int num_kv_heads,
                   int head_dim, int block_size, int dtype, void* stream)
{
    static const char* fn = "pkv_kv_read_q4";
    const int rc =
        check_cache(fn, num_tokens, num_blocks, num_kv_heads, head_dim, block_size, dtype);
    if (rc != PKV_OK) return rc;
    if (num_tokens == 0) return PKV_OK;
    if (!k_pool || !v_pool || !key || !value || !slot_mapping)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(key, 16) || !aligned(value, 16) ||
        !aligned(slot_mapping, 8))
        return pkv_fail(PKV_ERR_ALIGN, "%s: pools, key and value need 16-byte alignment", fn);
    Q4CacheParams p{const_cast<void*>(k_pool),
                    const_cast<void*>(v_pool),
                    slot_mapping,
                    num_tokens,
                    num_blocks,
                    num_kv_heads,
                    block_size,
                    block_shift(block_size),
                    pkv_status_word_ptr()};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_kv_read_q4(p, key, value, head_dim, dtype,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

size_t pkv_tables_workspace_bytes(int num_seqs)
{
    return num_seqs <= 0 ? 0 : ((size_t)(num_seqs + 1) * 4 + 255) / 256 * 256;
}

}  // extern "C"

namespace {

// Checks that an extend and a release share.
int check_tables(const char* fn, int num_seqs, int max_blocks, int block_size, int num_blocks)
{
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv_fail(PKV_ERR_SHAPE, "%s: num_seqs %d outside [0, 65535]", fn, num_seqs);
    if (max_blocks <= 0 || block_size <= 0 || num_blocks <= 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d blocks a sequence of %d tokens, pool of %d", fn,
                        max_blocks, block_size, num_blocks);
    if ((int64_t)max_blocks * block_size > (1ll << 30))
        return pkv_fail(PKV_ERR_SHAPE, "%s: max context too long", fn);
    return PKV_OK;
}

int check_workspace(const char* fn, const void* ws, size_t bytes, int num_seqs)
{
    const size_t need = pkv_tables_workspace_bytes(num_seqs);
    if (!ws || bytes < need)
        return pkv_fail(PKV_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                        ws ? bytes : (size_t)0);
    if (!aligned(ws, 256))
        return pkv_fail(PKV_ERR_ALIGN, "%s: workspace needs 256-byte alignment", fn);
    return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_tables_extend(int32_t* block_tables, const int32_t* context_lens,
                      const int32_t* new_tokens, const int32_t* free_list,
                      const int32_t* free_count, int32_t* query_start, int64_t* slot_mapping,
                      int32_t* positions, int32_t* lens_out, int32_t* free_count_out, int num_seqs,
                      int max_blocks_per_seq, int block_size, int num_blocks, int max_tokens,
                      void* workspace, size_t workspace_bytes, void* stream)
{
    static const char* fn = "pkv_tables_extend";
    int rc = check_tables(fn, num_seqs, max_blocks_per_seq, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (max_tokens < 0 || max_tokens > 1 << 30)
        return pkv_fail(PKV_ERR_SHAPE, "%s: max_tokens %d outside [0, 2^30]", fn, max_tokens);
    if (num_seqs == 0 && max_tokens > 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d rows of no sequence", fn, max_tokens);
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !context_lens || !new_tokens || !free_list || !free_count ||
        !query_start || (max_tokens > 0 && !slot_mapping) || !lens_out || !free_count_out)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(slot_mapping, 8) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(new_tokens, 4) || !aligned(free_list, 4) || !aligned(free_count, 4) ||
        !aligned(query_start, 4) || !aligned(positions, 4) || !aligned(lens_out, 4) ||
        !aligned(free_count_out, 4))
        return pkv_fail(PKV_ERR_ALIGN, "%s: misaligned pointer", fn);
    rc = check_workspace(fn, workspace, workspace_bytes, num_seqs);
    if (rc != PKV_OK) return rc;
    TablesParams p{block_tables, context_lens, new_tokens,  free_list,
                   free_count,   query_start,  slot_mapping, positions,
                   lens_out,     free_count_out, num_seqs,   max_blocks_per_seq,
                   block_size,   num_blocks,   max_tokens,  static_cast<int32_t*>(workspace),
                   pkv_status_word_ptr()};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_tables_extend(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_tables_release(int32_t* block_tables, int32_t* context_lens, const int32_t* release,
                       int32_t* free_list, int32_t* free_count, int num_seqs,
                       int max_blocks_per_seq, int block_size, int num_blocks, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    static const char* fn = "pkv_tables_release";
    int rc = check_tables(fn, num_seqs, max_blocks_per_seq, block_size, num_blocks);
    if (rc != PKV_OK) return rc;
    if (num_seqs == 0) return PKV_OK;
    if (!block_tables || !context_lens || !release || !free_list || !free_count)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(release, 4) ||
        !aligned(free_list, 4) || !aligned(free_count, 4))
        return pkv_fail(PKV_ERR_ALIGN, "%s: misaligned pointer", fn);
    rc = check_workspace(fn, workspace, workspace_bytes, num_seqs);
    if (rc != PKV_OK) return rc;
    ReleaseParams p{block_tables, context_lens, release,    free_list, free_count, num_seqs,
                    max_blocks_per_seq, block_size, num_blocks, static_cast<int32_t*>(workspace),
                    pkv_status_word_ptr()};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_tables_release(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

}  // extern "C"

namespace {

int decode_q4(const char* fn, void* out, const void* q, const void* k_pool, const void* v_pool,
              const int32_t* block_tables, const int32_t* context_lens, float scale,
              int block_size, int num_kv_heads, int num_seqs, int num_heads, int head_dim,
              int max_blocks_per_seq, int num_blocks, int kv_dtype, int out_dtype,
              int partition_size, void* workspace, size_t workspace_bytes, void* stream)
{
    const int chk = pkv_decode_check(fn, kv_dtype, out_dtype, num_seqs, num_heads, num_kv_heads,
                                     head_dim, block_size, max_blocks_per_seq, num_blocks,
                                     partition_size, scale);
    if (chk != PKV_OK) return chk;
    if (kv_dtype == PKV_F32)
        return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: the 4-bit cache holds 16-bit types only", fn);
    if (num_seqs == 0) return PKV_OK;
    if (!out || !q || !k_pool || !v_pool || !block_tables || !context_lens)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(q, 4) ||
        !aligned(out, pkv_dtype_bytes(out_dtype)) || !aligned(block_tables, 4) ||
        !aligned(context_lens, 4))
        return pkv_fail(PKV_ERR_ALIGN, "%s: pools need 16-byte, q 4-byte alignment", fn);

    const int max_ctx = max_blocks_per_seq * block_size;
    // one partition a context, whose end passes 31 bits no more than the context's
    partition_size = std::min(partition_size, max_ctx);
    DecodeParams p = {};
    p.out = out;
    p.q = q;
    p.k_cache = k_pool;
    p.v_cache = v_pool;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
    p.block_size = block_size;
    p.num_kv_heads = num_kv_heads;
    p.num_heads = num_heads;
    p.head_dim = head_dim;
    p.num_seqs = num_seqs;
    p.max_blocks = max_blocks_per_seq;
    p.num_blocks = num_blocks;
    p.out_dtype = out_dtype;
    p.cta_parts = 1;
    p.partition_tokens = partition_size ? partition_size : max_ctx;
    p.max_partitions = (max_ctx + p.partition_tokens - 1) / p.partition_tokens;
    const int G = num_heads / num_kv_heads;
    p.head_slices = (G + kDecodeQ4MaxColumns - 1) / kDecodeQ4MaxColumns;
    const int columns = (G + p.head_slices - 1) / p.head_slices;
    const int64_t rows = (int64_t)num_seqs * num_kv_heads * p.head_slices;
    if (rows * p.max_partitions >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: more than 2^31 work items", fn);

    int* plan_count = nullptr;
    int4* plan_items = nullptr;
    if (partition_size > 0 || workspace != nullptr) {
        const size_t need = pkv_decode_workspace_bytes(num_seqs, num_heads, head_dim, max_ctx,
                                                       partition_size);
        if (!workspace || workspace_bytes < need)
            return pkv_fail(PKV_ERR_WORKSPACE, "%s: workspace of %zu bytes needed, %zu given", fn,
                            need, workspace ? workspace_bytes : (size_t)0);
        if (!aligned(workspace, 256))
            return pkv_fail(PKV_ERR_ALIGN, "%s: workspace needs 256-byte alignment", fn);
        char* base = static_cast<char*>(workspace);
        size_t count_at = 0, items_at = 256;
        if (partition_size > 0) {
            const DecodeWorkspace w = decode_workspace(num_seqs, num_heads, p.max_partitions,
                                                       head_dim);
            p.done = reinterpret_cast<unsigned*>(base);
            p.ws_ml = reinterpret_cast<float2*>(base + w.ml);
            p.ws_o = reinterpret_cast<float*>(base + w.o);
            count_at = w.count;
            items_at = w.items;
        }
        plan_count = reinterpret_cast<int*>(base + count_at);
        plan_items = reinterpret_cast<int4*>(base + items_at);
    }
    p.status = pkv_status_word_ptr();
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);

    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        sms = 0;
    const int slots = decode_q4_ctas_per_sm(head_dim, columns) * sms;
    int64_t grid = rows * p.max_partitions;
    // A plan lists the CTAs with work, longest sequence first.  A grid that the GPU
    // holds at once needs none (one context of 16384 in 256 CTAs: 11.8 us against
    // 13.7; 76 ragged ones in 608, not split: 46 against 55); past that it pays
    // (256 ragged contexts in 2048 CTAs: 58.6 us against 76 without; 8 of 32768 in
    // equal pieces: 61 against 76).
    if (plan_items != nullptr && num_seqs <= kPlanMaxSeqs && grid > slots) {
        DecodePlanParams pp = {};
        pp.context_lens = context_lens;
        pp.num_seqs = num_seqs;
        pp.num_kv_heads = num_kv_heads;
        pp.head_slices = p.head_slices;
        pp.partition_tokens = p.partition_tokens;
        pp.cta_parts = 1;
        pp.stage_tokens = kDecodeQ4StageTokens;
        pp.slots = p.max_partitions > 1 ? slots : 0;
        pp.spare = kDecodeQ4PiecesPerSlot * pp.slots;
        pp.max_groups = p.max_partitions;
        pp.max_len = max_ctx;
        while ((max_ctx >> pp.bucket_shift) >= kPlanBuckets) ++pp.bucket_shift;
        pp.items = plan_items;
        pp.item_count = plan_count;
        const cudaError_t e = launch_decode_plan(pp, st);
        if (e != cudaSuccess) return cuda_fail(e, fn);
        p.items = plan_items;
        p.item_count = plan_count;
        if (pp.spare > 0 && grid > rows + pp.spare) grid = rows + pp.spare;
    }
    const cudaError_t e = launch_decode_q4(p, kv_dtype, grid, columns, st);
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

}  // namespace

extern "C" {

int pkv_paged_decode_attention_q4(void* out, const void* q, const void* k_pool, const void* v_pool,
                                  const int32_t* block_tables, const int32_t* context_lens,
                                  float scale, int block_size, int num_kv_heads, int num_seqs,
                                  int num_heads, int head_dim, int max_blocks_per_seq,
                                  int num_blocks, int kv_dtype, int out_dtype, int partition_size,
                                  void* workspace, size_t workspace_bytes, void* stream)
{
    return decode_q4("pkv_paged_decode_attention_q4", out, q, k_pool, v_pool, block_tables,
                     context_lens, scale, block_size, num_kv_heads, num_seqs, num_heads, head_dim,
                     max_blocks_per_seq, num_blocks, kv_dtype, out_dtype, partition_size,
                     workspace, workspace_bytes, stream);
}

int pkv_paged_decode_attention_selected_q4(
    void* out, const void* q, const void* k_pool, const void* v_pool, const int32_t* selected,
    const int32_t* selected_lens, float scale, int block_size, int num_kv_heads, int num_seqs,
    int num_heads, int head_dim, int max_selected, int num_blocks, int kv_dtype, int out_dtype,
    int partition_size, void* workspace, size_t workspace_bytes, void* stream)
{
    static const char* fn = "pkv_paged_decode_attention_selected_q4";
    const int rc = pkv_selected_check(fn, kv_dtype, out_dtype, num_seqs, num_heads, num_kv_heads,
                                      head_dim, block_size, max_selected, num_blocks,
                                      partition_size, scale);
    if (rc != PKV_OK) return rc;
    return decode_q4(fn, out, q, k_pool, v_pool, selected, selected_lens, scale, block_size, 1,
                     num_seqs * num_kv_heads, num_heads / num_kv_heads, head_dim, max_selected,
                     num_blocks * num_kv_heads, kv_dtype, out_dtype, partition_size, workspace,
                     workspace_bytes, stream);
}

}  // extern "C"
