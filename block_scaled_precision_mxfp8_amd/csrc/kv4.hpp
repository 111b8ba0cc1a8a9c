// kv4.hpp -- geometry of the paged MXFP4 key/value cache (internal).
//
// One layer of the cache is `pages` pages of one run of bytes each,
// page_stride bytes apart.  A page holds `page` tokens (a multiple of 16) of
// every head, in four sections:
//   K codes   [heads][page][dim/2]           a token's row as mxfp4_quantize packs it
//   V codes   [heads][page/16][dim/2][16]    16 tokens of each byte (dim pair) together
//   K scales  [heads][page/16][dim/32][16]   E8M0 bytes, 16 tokens together
//   V scales  [heads][page/16][dim/32][16]
// The product P V contracts over tokens, so attention wants V with the tokens
// of one dim side by side: in blocks of 16 tokens a lane gets them with one
// 16-byte load, and a token can still be written alone.  The scales of 16
// tokens come with one load as well.  Every section starts 16-byte aligned.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

struct Kv4Geom {
    int64_t pages, page_stride;
    int32_t heads, dim, page;

    __host__ __device__ int64_t code_bytes() const { return (int64_t)heads * page * (dim >> 1); }
    __host__ __device__ int64_t scale_bytes() const { return (int64_t)heads * page * (dim >> 5); }
    __host__ __device__ int64_t page_bytes() const { return 2 * (code_bytes() + scale_bytes()); }
    __host__ __device__ int64_t v_codes() const { return code_bytes(); }
    __host__ __device__ int64_t k_scales() const { return 2 * code_bytes(); }
    __host__ __device__ int64_t v_scales() const { return 2 * code_bytes() + scale_bytes(); }
    // inside a section: token `in` of the page, byte b (= dim / 2) or group g (= dim / 32)
    __host__ __device__ int64_t k_code(int h, int in) const
    {
        return ((int64_t)h * page + in) * (dim >> 1);
    }
    __host__ __device__ int64_t v_code(int h, int in, int b) const
    {
        return (int64_t)h * page * (dim >> 1) + ((int64_t)(in >> 4) * (dim >> 1) + b) * 16 + (in & 15);
    }
    __host__ __device__ int64_t scale(int h, int in, int g) const
    {
        return (int64_t)h * page * (dim >> 5) + ((int64_t)(in >> 4) * (dim >> 5) + g) * 16 + (in & 15);
    }
};

// Arguments of the attention kernels.
struct Kv4Attn {
    Kv4Geom geo;
    const uint8_t *cache;
    const uint16_t *q;
    int64_t q_seq, q_tok, q_head;  // element strides of q
    const int32_t *table;          // [seqs, width] page of each run of `page` tokens
    int64_t table_stride;
    const int32_t *lengths;
    int32_t seqs, tokens, q_heads, width;
    float scale;
    int32_t causal, window;
    uint16_t *out;  // [seqs, tokens, q_heads, dim]
    float *lse;     // [seqs, tokens, q_heads] or NULL
    // split over the context: per split, unnormalised sums [rows, dim], then
    // (maximum, sum) pairs [rows, 2] of the softmax in powers of two
    float *part;
    int32_t splits;
    int32_t ranked;  // start sequences longest first (set by the launcher)
};

hipError_t launch_kv4_append(const Kv4Geom &geo, uint8_t *cache, const uint16_t *k, int64_t k_tok,
                             int64_t k_head, const uint16_t *v, int64_t v_tok, int64_t v_head,
                             const int64_t *slots, int64_t tokens, uint16_t *k_fq, uint16_t *v_fq,
                             hipStream_t stream);

hipError_t launch_kv4_copy(uint8_t *cache, int64_t layers, int64_t layer_stride, int64_t pages,
                           int64_t page_stride, int64_t page_bytes, const int32_t *src,
                           const int32_t *dst, int64_t n, hipStream_t stream);

// Splits of the context an attention call uses (1 needs no workspace); never
// more with a window than without (0).
int32_t kv4_attention_splits(int64_t seqs, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                             int64_t dim, int64_t page, int64_t width, int64_t window);

// Most rows (query tokens x query heads of one kv head) an attention call takes.
int64_t kv4_attention_most_rows(int64_t dim);

hipError_t launch_kv4_attention(const Kv4Attn &a, hipStream_t stream);

}  // namespace mxq
