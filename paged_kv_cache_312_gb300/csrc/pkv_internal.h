// Internal host-side helpers of libpkv (not part of the C ABI).
#pragma once

#include <cstddef>
#include <cstdint>

// Records a formatted message as the calling thread's last error and returns
// `code`, so that call sites read `return pkv_fail(PKV_ERR_SHAPE, "...")`.
int pkv_fail(int code, const char* fmt, ...)
#if defined(__GNUC__)
    __attribute__((format(printf, 2, 3)))
#endif
    ;

// Element size in bytes of a PKV_* dtype code, 0 if unknown.
inline int pkv_dtype_bytes(int dtype)
{
    return dtype == 0 ? 4 : (dtype == 1 || dtype == 2) ? 2 : 0;
}

// Checks of a decode request's dtypes and sizes that need no pointer:
// dtypes, num_seqs in [0, 65535], head_dim in {64, 128}, block_size in
// {8, 16, 32}, num_heads a multiple of num_kv_heads, positive table and pool
// sizes, a maximum context of at most 2^30 tokens, fewer than 2^31 cache
// rows, partition_size 0 or a multiple of block_size, a finite scale.
// Returns PKV_OK or the failing code (with the message recorded).
int pkv_decode_check(const char* fn, int kv_dtype, int out_dtype, int num_seqs, int num_heads,
                     int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                     int num_blocks, int partition_size, float scale);

// The same of an attention over selected blocks, whose launch takes each (sequence,
// KV head) for a sequence of one KV head over a pool of (block, KV head) tiles:
// at most 65535 of them.
int pkv_selected_check(const char* fn, int kv_dtype, int out_dtype, int num_seqs, int num_heads,
                       int num_kv_heads, int head_dim, int block_size, int max_selected,
                       int num_blocks, int partition_size, float scale);

// Split workspace of a decode launch, in order (each part 256-byte aligned):
//   done  : u32 [S][H]           partitions finished per (sequence, KV head)
//   ml    : float2 [S][H][P]     per-partition (max, sum), base 2
//   o     : float [S][H][P][D]   per-partition unnormalised output
//   count : int                  work records in the plan
//   items : int4 [S][H][P]       the plan's records, one per CTA with work
// with H the number of query heads (an upper bound for the KV heads times
// the head slices, so S*H*P bounds every split launch's grid).
struct DecodeWorkspace {
    size_t ml, o, count, items, total;
};

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

inline DecodeWorkspace decode_workspace(size_t S, size_t H, size_t P, size_t D)
{
    DecodeWorkspace w;
    w.ml = align256(S * H * 4);
    w.o = w.ml + align256(S * H * P * 8);
    w.count = w.o + align256(S * H * P * D * 4);
    w.items = w.count + 256;
    w.total = w.items + S * H * P * 16;
    return w;
}

// Optional workspace of an unsplit launch, the work plan alone: the record
// count at byte 0, the wide-group kernel's record counter at byte 64, then
// one record per (sequence, KV head x head slice) from byte 256.
inline size_t decode_plan_bytes(size_t S, size_t H) { return 256 + S * H * 16; }
