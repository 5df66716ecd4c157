// gdn_kv4.cuh - the 4-bit key/value cache: its number format, the geometry of
// its pages, and the arguments of the calls that write, read and attend to it.
//
// Format. 16 values along the head dimension share one scale s; each value is
// an e2m1 code (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
// 6) times s. The scale is one byte b, the fp16 number with the bits b << 7
// (5 exponent bits, 3 mantissa bits, no sign), at most 10240 (b = 226), so
//   s = RNE(min(max|x| / 6, 10240)) to that grid,  code = RNE(x / s) to e2m1.
// A product of a code and a scale has at most 6 significant bits, is a multiple
// of 2^-18 and at most 61440: fp16, bf16 and fp32 all hold it exactly, so reading
// the cache never rounds. The exponent range of fp16 is why no per-tensor scale is
// needed beside the blocks'.
//
// Page. For each kv head P tokens: [K codes P x D/2 | K scales P x D/16 |
// V codes P x D/2 | V scales P x D/16]. The 8-byte code block i of token row r
// lies at block i ^ swizzle(r): with it, the 8 token rows that the lanes of one
// quarter warp read for K, and the 4 token rows they read for V, fall into
// different shared-memory banks after a plain contiguous copy of the page.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "gdn_launch.h"

namespace gdn {

constexpr float kKv4MaxScale = 10240.0f;
constexpr uint32_t kErrBadPage = 2u;  // a needed block_table entry was missing or out of range

enum class DType : int { kF32 = 0, kF16 = 1, kBF16 = 2 };

__host__ __device__ constexpr int kv4_swizzle(int row, int n_blocks) {
    return (((row & 1) << 3) | (((row >> 2) & 1) << 2)) & (n_blocks - 1);
}

// Bytes of one kv head's part of a page; its V half starts in the middle.
__host__ __device__ constexpr size_t kv4_head_bytes(int page, int head_dim) {
    return static_cast<size_t>(2) * page * (head_dim / 2 + head_dim / 16);
}

constexpr int kKv4MaxTokens = 1 << 20;  // of a window

// Where sequence b's window lies: its first position, its valid tokens, and the end of
// the positions that the block table can hold. A first position below 0 stays so (no lower than
// -kKv4MaxTokens, where no token reaches position 0): its tokens before position 0 are missing.
struct Kv4Window {
    int start, n, cap;
};

struct Kv4Cache {
    uint8_t* cache;
    const int32_t* block_table;
    const int32_t* kv_start;
    const int32_t* seq_len;  // may be NULL: every sequence has T tokens
    int B, L, T, kv_heads, head_dim;
    int n_pages, max_pages, page_shift;
};

#ifdef __CUDACC__
__device__ __forceinline__ Kv4Window kv4_window(const Kv4Cache& c, int b) {
    Kv4Window w;
    w.cap = c.max_pages << c.page_shift;
    w.start = min(max(__ldg(c.kv_start + b), -kKv4MaxTokens), w.cap);
    w.n = c.seq_len != nullptr ? min(max(__ldg(c.seq_len + b), 0), c.T) : c.T;
    return w;
}

// The page that holds position pos of sequence b, or -1.
__device__ __forceinline__ int kv4_page(const Kv4Cache& c, int b, int pos) {
    const int slot = pos >> c.page_shift;
    if (static_cast<uint32_t>(slot) >= static_cast<uint32_t>(c.max_pages)) return -1;
    const int page = __ldg(c.block_table + static_cast<size_t>(b) * c.max_pages + slot);
    return page >= 0 && page < c.n_pages ? page : -1;
}

// First byte of (layer, page, kv head).
__device__ __forceinline__ size_t kv4_head_offset(const Kv4Cache& c, int l, int page, int h) {
    return ((static_cast<size_t>(l) * c.n_pages + page) * c.kv_heads + h) *
           kv4_head_bytes(1 << c.page_shift, c.head_dim);
}

// Whether tokens of the window lie outside the positions that the block table can hold.
__device__ __forceinline__ bool kv4_runs_out(const Kv4Window& w) { return w.n > 0 && (w.start < 0 || w.n > w.cap - w.start); }

#endif  // __CUDACC__

struct Kv4AttnArgs {
    Kv4Cache c;
    const void* q;
    void* out;
    void* workspace;
    int q_heads;
    DType dtype;
    float scale;
};

cudaError_t launch_kv4_append(const Kv4Cache& c, const void* k, const void* v, DType dtype, cudaStream_t stream);
cudaError_t launch_kv4_read(const Kv4Cache& c, void* k, void* v, DType dtype, cudaStream_t stream);

size_t kv4_attention_workspace_bytes(int B, int L, int T, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t stream);

struct LogprobArgs {
    const void* logits;
    const int32_t* tokens;
    float* logprob;
    float* entropy;
    int32_t* top_ids;
    float* top_logprobs;
    long long n_rows, vocab, ld;
    int k;
    DType dtype;
};

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream);

}  // namespace gdn
