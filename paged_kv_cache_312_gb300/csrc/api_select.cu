// C-ABI entry points of the rotary positions, of the blocks' bounds and of the
// selection of blocks, and the one of the attention over them (declared in
// include/pkv.h): argument checks and launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <tuple>
#include <type_traits>

#include "pkv.h"
#include "pkv_internal.h"
#include "pkv_kernels.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int cuda_fail(cudaError_t e, const char* where)
{
    return pkv_fail(PKV_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

int block_shift(int block_size) { return block_size == 8 ? 3 : block_size == 16 ? 4 : 5; }

// Checks that both rotations share; fills the rotation's part of p.
int check_rotation(const char* fn, RopeParams& p, const int32_t* positions, const int64_t* turns,
                   const uint8_t* pair_axis, int num_axes, int num_tokens, int head_dim,
                   int rotary_dim, float magnitude, int interleaved, int inverse, int dtype)
{
    if (!pkv_dtype_bytes(dtype)) return pkv_fail(PKV_ERR_DTYPE, "%s: dtype %d", fn, dtype);
    if (head_dim <= 0 || head_dim > 2 * kRopeMaxPairs || head_dim % 16 != 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: head_dim %d is no multiple of 16 up to %d", fn,
                        head_dim, 2 * kRopeMaxPairs);
    if (rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % 16 != 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: rotary_dim %d is no multiple of 16 up to head_dim %d",
                        fn, rotary_dim, head_dim);
    if (num_axes < 1 || num_axes > kRopeMaxAxes)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d axes, not 1 to %d", fn, num_axes, kRopeMaxAxes);
    if (num_tokens < 0) return pkv_fail(PKV_ERR_SHAPE, "%s: %d tokens", fn, num_tokens);
    if (!std::isfinite(magnitude))
        return pkv_fail(PKV_ERR_SHAPE, "%s: the magnitude is not finite", fn);
    if (num_axes > 1 && !pair_axis)
        return pkv_fail(PKV_ERR_NULL, "%s: %d axes, and no axis of each pair", fn, num_axes);
    p.pairs = rotary_dim / 2;
    for (int i = 0; i < kRopeMaxPairs; ++i) {
        p.axis[i] = pair_axis != nullptr && i < p.pairs ? pair_axis[i] : 0;
        if (p.axis[i] >= num_axes)
            return pkv_fail(PKV_ERR_SHAPE, "%s: pair %d turns on axis %d of %d", fn, i, p.axis[i],
                            num_axes);
    }
    p.positions = positions;
    p.turns = turns;
    p.num_tokens = num_tokens;
    p.head_dim = head_dim;
    p.magnitude = magnitude;
    p.interleaved = interleaved != 0;
    p.inverse = inverse != 0;
    if (num_tokens == 0) return PKV_OK;
    if (!positions || !turns) return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(positions, 4) || !aligned(turns, 8))
        return pkv_fail(PKV_ERR_ALIGN, "%s: misaligned positions or turns", fn);
    return PKV_OK;
}

// A tensor [num_tokens][heads][head_dim] whose tokens lie `stride` elements apart.
int check_rows(const char* fn, const char* name, const void* rows, int64_t stride, int num_tokens,
               int64_t heads, int head_dim, int dtype)
{
    const int vec = 16 / pkv_dtype_bytes(dtype);
    if (num_tokens > 1 && (stride < heads * head_dim || stride % vec != 0))
        return pkv_fail(PKV_ERR_SHAPE,
                        "%s: token stride %lld of %s must be a multiple of %d of at least %lld", fn,
                        (long long)stride, name, vec, (long long)(heads * head_dim));
    if (num_tokens == 0) return PKV_OK;
    if (!rows) return pkv_fail(PKV_ERR_NULL, "%s: %s is NULL", fn, name);
    if (!aligned(rows, 16))
        return pkv_fail(PKV_ERR_ALIGN, "%s: %s needs 16-byte alignment", fn, name);
    return PKV_OK;
}

// Checks of a pool of blocks and of tables over it.
int check_blocks(const char* fn, int num_seqs, int max_blocks, int num_blocks, int num_kv_heads,
                 int head_dim, int block_size, int dtype)
{
    if (!pkv_dtype_bytes(dtype)) return pkv_fail(PKV_ERR_DTYPE, "%s: dtype %d", fn, dtype);
    if (num_seqs < 0 || num_seqs > 65535)
        return pkv_fail(PKV_ERR_SHAPE, "%s: num_seqs %d outside [0, 65535]", fn, num_seqs);
    if (head_dim != 64 && head_dim != 128)
        return pkv_fail(PKV_ERR_SHAPE, "%s: head_dim %d not in {64,128}", fn, head_dim);
    if (block_size != 8 && block_size != 16 && block_size != 32)
        return pkv_fail(PKV_ERR_SHAPE, "%s: block_size %d not in {8,16,32}", fn, block_size);
    if (max_blocks <= 0 || num_blocks <= 0 || num_kv_heads <= 0 || num_kv_heads > 65535)
        return pkv_fail(PKV_ERR_SHAPE, "%s: max_blocks_per_seq %d, %d blocks of %d KV heads", fn,
                        max_blocks, num_blocks, num_kv_heads);
    if ((int64_t)max_blocks * block_size > (1ll << 30))
        return pkv_fail(PKV_ERR_SHAPE, "%s: max context too long", fn);
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: cache has >= 2^31 rows", fn);
    return PKV_OK;
}

// The arguments of a call, one after the other from 8-byte words; the only `const
// uint8_t*` among them is the pairs' axes.
struct Words {
    const int64_t* at;
    bool fit = true;  // every `int` is one

    template <typename A>
    A next(const uint8_t* pair_axis)
    {
        if constexpr (std::is_same_v<A, const uint8_t*>) {
            return pair_axis;
        } else if constexpr (std::is_floating_point_v<A>) {
            double x;
            std::memcpy(&x, at++, sizeof x);
            return (A)x;
        } else if constexpr (std::is_pointer_v<A>) {
            return reinterpret_cast<A>((uintptr_t)*at++);
        } else {
            const int64_t x = *at++;
            fit = fit && (sizeof(A) == 8 || x == (int)x);
            return (A)x;
        }
    }
    template <typename... A>
    int call(int (*fn)(A...), const uint8_t* pair_axis)
    {
        std::tuple<A...> args{next<A>(pair_axis)...};  // braces: in order
        if (!fit) return pkv_fail(PKV_ERR_SHAPE, "pkv_call_words: a number past 32 bits");
        return std::apply(fn, args);
    }
};

}  // namespace

extern "C" {

int pkv_rope_turns(const double* inv_freq, int num_pairs, int64_t* turns)
{
    static const char* fn = "pkv_rope_turns";
    // 1 / (2 pi) as the sum of two doubles
    constexpr double kHigh = 0x1.45f306dc9c883p-3, kLow = -0x1.6b01ec5417056p-57;
    if (num_pairs < 0) return pkv_fail(PKV_ERR_SHAPE, "%s: %d pairs", fn, num_pairs);
    if (num_pairs > 0 && (!inv_freq || !turns)) return pkv_fail(PKV_ERR_NULL, "%s: NULL", fn);
    for (int i = 0; i < num_pairs; ++i)
        if (!(std::fabs(inv_freq[i]) <= 0x1p20))
            return pkv_fail(PKV_ERR_SHAPE, "%s: frequency %d is not within 2^20", fn, i);
    for (int i = 0; i < num_pairs; ++i) {
        const double f = std::fabs(inv_freq[i]), high = f * kHigh;
        const double low = std::fma(f, kHigh, -high) + f * kLow;  // high + low: the turns
        // the fraction of high in units of 2^-64, exact but for what lies below one
        const double units = std::ldexp(high - std::floor(high), 64), whole = std::floor(units);
        const uint64_t part = (uint64_t)whole + (uint64_t)(int64_t)std::llrint(
                                                    (units - whole) + std::ldexp(low, 64));
        turns[i] = (int64_t)(inv_freq[i] < 0 ? 0 - part : part);
    }
    return PKV_OK;
}

int pkv_rope(void* out, const void* x, const int32_t* positions, const int64_t* turns,
             const uint8_t* pair_axis, int num_axes, int num_tokens, int num_heads, int head_dim,
             int rotary_dim, int64_t out_stride, int64_t x_stride, float magnitude,
             int interleaved, int inverse, int dtype, void* stream)
{
    static const char* fn = "pkv_rope";
    RopeParams p = {};
    int rc = check_rotation(fn, p, positions, turns, pair_axis, num_axes, num_tokens, head_dim,
                            rotary_dim, magnitude, interleaved, inverse, dtype);
    if (rc != PKV_OK) return rc;
    if (num_heads <= 0 || num_heads > 65535)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d heads", fn, num_heads);
    rc = check_rows(fn, "x", x, x_stride, num_tokens, num_heads, head_dim, dtype);
    if (rc == PKV_OK)
        rc = check_rows(fn, "out", out, out_stride, num_tokens, num_heads, head_dim, dtype);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    if (out == x && num_tokens > 1 && out_stride != x_stride)
        return pkv_fail(PKV_ERR_SHAPE, "%s: in place, but with other strides", fn);
    p.first = RopeRows{x, out, x_stride, out_stride, 0, num_heads, true, false};
    p.second.begin = p.second.end = p.third.begin = p.third.end = num_heads;
    const cudaError_t e = launch_rope(p, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_rope_write(void* q_out, void* k_cache, void* v_cache, const void* q, const void* key,
                   const void* value, const int32_t* positions, const int64_t* turns,
                   const uint8_t* pair_axis, int num_axes, const int64_t* slot_mapping,
                   int num_tokens, int64_t q_out_stride, int64_t q_stride, int64_t key_stride,
                   int64_t value_stride, int num_blocks, int num_heads, int num_kv_heads,
                   int head_dim, int rotary_dim, int block_size, float magnitude, int interleaved,
                   int dtype, void* stream)
{
    static const char* fn = "pkv_rope_write";
    RopeParams p = {};
    int rc = check_rotation(fn, p, positions, turns, pair_axis, num_axes, num_tokens, head_dim,
                            rotary_dim, magnitude, interleaved, 0, dtype);
    if (rc != PKV_OK) return rc;
    if (num_heads < 0 || num_heads > 65535 || num_kv_heads <= 0 || num_kv_heads > 65535 ||
        num_blocks < 0 || block_size <= 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: %d heads on %d KV heads, %d blocks of %d tokens", fn,
                        num_heads, num_kv_heads, num_blocks, block_size);
    if ((int64_t)num_blocks * num_kv_heads * block_size >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: cache has >= 2^31 rows", fn);
    if (num_heads > 0) {
        rc = check_rows(fn, "q", q, q_stride, num_tokens, num_heads, head_dim, dtype);
        if (rc == PKV_OK)
            rc = check_rows(fn, "q_out", q_out, q_out_stride, num_tokens, num_heads, head_dim,
                            dtype);
        if (rc == PKV_OK && q_out == q && num_tokens > 1 && q_out_stride != q_stride)
            rc = pkv_fail(PKV_ERR_SHAPE, "%s: q in place, but with other strides", fn);
    }
    if (rc == PKV_OK)
        rc = check_rows(fn, "key", key, key_stride, num_tokens, num_kv_heads, head_dim, dtype);
    if (rc == PKV_OK)
        rc = check_rows(fn, "value", value, value_stride, num_tokens, num_kv_heads, head_dim,
                        dtype);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    if (!k_cache || !v_cache || !slot_mapping)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(slot_mapping, 8))
        return pkv_fail(PKV_ERR_ALIGN, "%s: caches need 16-byte alignment", fn);
    p.first = RopeRows{q, q_out, q_stride, q_out_stride, 0, num_heads, true, false};
    p.second = RopeRows{key, k_cache, key_stride, 0, num_heads, num_heads + num_kv_heads, true,
                        true};
    p.third = RopeRows{value, v_cache, value_stride, 0, num_heads + num_kv_heads,
                        num_heads + 2 * num_kv_heads, false, true};
    p.slots = slot_mapping;
    p.num_blocks = num_blocks;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.status = pkv_status_word_ptr();
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_rope(p, dtype, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_block_bounds(int8_t* bounds, float* bound_scales, const void* k_cache,
                     const int32_t* block_tables, const int32_t* context_lens,
                     const int32_t* new_tokens, int num_seqs, int max_blocks_per_seq,
                     int num_blocks, int num_kv_heads, int head_dim, int block_size,
                     int max_new_tokens, int dtype, void* stream)
{
    static const char* fn = "pkv_block_bounds";
    const int rc = check_blocks(fn, num_seqs, max_blocks_per_seq, num_blocks, num_kv_heads,
                                head_dim, block_size, dtype);
    if (rc != PKV_OK) return rc;
    if (max_new_tokens < 0 || max_new_tokens > 1 << 30)
        return pkv_fail(PKV_ERR_SHAPE, "%s: max_new_tokens %d outside [0, 2^30]", fn,
                        max_new_tokens);
    // a run of tokens that starts in a block's last place
    const int blocks_each =
        std::min((max_new_tokens + block_size - 2) / block_size + 1, max_blocks_per_seq);
    if ((int64_t)num_seqs * blocks_each * num_kv_heads >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: more than 2^31 tiles", fn);
    if (num_seqs == 0 || max_new_tokens == 0) return PKV_OK;
    if (!bounds || !bound_scales || !k_cache || !block_tables || !context_lens || !new_tokens)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(bounds, 16) || !aligned(k_cache, 16) || !aligned(bound_scales, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(new_tokens, 4))
        return pkv_fail(PKV_ERR_ALIGN, "%s: bounds and cache need 16-byte alignment", fn);
    BoundsParams p{bounds, bound_scales, k_cache, block_tables, context_lens, new_tokens, num_seqs,
                   max_blocks_per_seq, num_blocks, num_kv_heads, block_size,
                   block_shift(block_size), max_new_tokens, blocks_each, pkv_status_word_ptr()};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_block_bounds(p, head_dim, dtype,
                                              static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_select_blocks(int32_t* selected, int32_t* selected_lens, float* scores, const void* q,
                      const int8_t* bounds, const float* bound_scales,
                      const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim, int block_size,
                      int max_blocks_per_seq, int num_blocks, int max_selected, int first_blocks,
                      int recent_blocks, int dtype, void* stream)
{
    static const char* fn = "pkv_select_blocks";
    const int rc = check_blocks(fn, num_seqs, max_blocks_per_seq, num_blocks, num_kv_heads,
                                head_dim, block_size, dtype);
    if (rc != PKV_OK) return rc;
    if (num_heads <= 0 || num_heads > 65535 || num_heads % num_kv_heads != 0)
        return pkv_fail(PKV_ERR_SHAPE, "%s: num_heads %d / num_kv_heads %d", fn, num_heads,
                        num_kv_heads);
    if (num_heads / num_kv_heads > kSelectMaxGroup)
        return pkv_fail(PKV_ERR_UNSUPPORTED, "%s: more than %d query heads a KV head", fn,
                        kSelectMaxGroup);
    if ((int64_t)num_seqs * num_kv_heads >= (1ll << 31))
        return pkv_fail(PKV_ERR_SHAPE, "%s: more than 2^31 rows", fn);
    if (first_blocks < 0 || recent_blocks < 1 || max_selected > 1 << 30 ||
        (int64_t)first_blocks + recent_blocks > max_selected)
        return pkv_fail(PKV_ERR_SHAPE,
                        "%s: the first %d and the %d (at least 1) most recent of %d blocks", fn,
                        first_blocks, recent_blocks, max_selected);
    if (num_seqs == 0) return PKV_OK;
    if (!selected || !selected_lens || !scores || !q || !bounds || !bound_scales ||
        !block_tables || !context_lens)
        return pkv_fail(PKV_ERR_NULL, "%s: NULL pointer", fn);
    if (!aligned(bounds, 16) || !aligned(q, 16) || !aligned(bound_scales, 4) ||
        !aligned(selected, 4) || !aligned(selected_lens, 4) || !aligned(scores, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4))
        return pkv_fail(PKV_ERR_ALIGN, "%s: bounds and q need 16-byte alignment", fn);
    SelectParams p{selected, selected_lens, scores, q, bounds, bound_scales, block_tables,
                   context_lens, num_seqs, num_heads, num_kv_heads, max_blocks_per_seq, num_blocks,
                   block_size, block_shift(block_size), max_selected, first_blocks, recent_blocks,
                   dtype, pkv_status_word_ptr(), 0};
    if (!p.status) return pkv_fail(PKV_ERR_CUDA, "%s: no device status word", fn);
    const cudaError_t e = launch_select_blocks(p, head_dim, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PKV_OK : cuda_fail(e, fn);
}

int pkv_paged_decode_attention_selected(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* selected,
    const int32_t* selected_lens, float scale, int block_size, int num_kv_heads, int num_seqs,
    int num_heads, int head_dim, int max_selected, int num_blocks, int kv_dtype, int out_dtype,
    int partition_size, void* workspace, size_t workspace_bytes, void* stream)
{
    return pkv_decode_selected("pkv_paged_decode_attention_selected", selected_split, out, q,
                               k_cache, v_cache, selected, selected_lens, scale, block_size,
                               num_kv_heads, num_seqs, num_heads, head_dim, max_selected,
                               num_blocks, kv_dtype, out_dtype, partition_size, workspace,
                               workspace_bytes, stream);
}

int pkv_call_words(const int64_t* words, const uint8_t* pair_axis)
{
    if (!words) return pkv_fail(PKV_ERR_NULL, "pkv_call_words: NULL");
    Words w{words + 1};
    switch (words[0]) {
    case PKV_CALL_ROPE: return w.call(pkv_rope, pair_axis);
    case PKV_CALL_ROPE_WRITE: return w.call(pkv_rope_write, pair_axis);
    case PKV_CALL_BLOCK_BOUNDS: return w.call(pkv_block_bounds, pair_axis);
    case PKV_CALL_SELECT_BLOCKS: return w.call(pkv_select_blocks, pair_axis);
    case PKV_CALL_ATTENTION_SELECTED:
        return w.call(pkv_paged_decode_attention_selected, pair_axis);
    case PKV_CALL_ATTENTION_SELECTED_Q4:
        return w.call(pkv_paged_decode_attention_selected_q4, pair_axis);
    }
    return pkv_fail(PKV_ERR_SHAPE, "pkv_call_words: call %lld", (long long)words[0]);
}

}  // extern "C"
