// gdn_prompt.cuh - arguments of the operators that take a prompt's queries, keys and values before they are cached:
// rotary positions and causal attention.
#pragma once

#include "gdn_kv4.cuh"

namespace gdn {

constexpr uint32_t kRopeInterleaved = 1u;  // match GDN_ROPE_* in gdn.h
constexpr uint32_t kRopeInverse = 2u;

// One side of a rotation: tokens of `heads` heads, their rows `in_stride` and `out_stride` elements apart.
struct RopeSide {
    const void* in;
    void* out;
    long long in_stride, out_stride;
    int heads;
};

struct RopeArgs {
    RopeSide side[2];  // queries, keys (0 heads: none)
    const uint64_t* turns;
    const int32_t* start;      // [B], or
    const int32_t* positions;  // [B][T]
    const int32_t* seq_len;    // may be NULL
    int B, L, T, head_dim, rotary_dim;
    float gain;
    uint32_t flags;
    DType dtype;
};

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream);

struct PromptArgs {
    const void* q;
    const void* k;
    const void* v;
    void* out;
    void* workspace;
    const int32_t* offsets;  // [B + 1]
    const int32_t* seq_len;  // may be NULL
    long long q_stride, k_stride, v_stride, out_stride;  // elements from token to token
    int B, n_tokens, q_heads, kv_heads, head_dim;
    DType dtype;
    float scale;
};

size_t prompt_workspace_bytes(int B, int n_tokens, int q_heads, int kv_heads, int head_dim, DType dtype);
cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream);

#ifdef __CUDACC__
// Rows [first, first + n) of sequence b.
struct PromptRows {
    int first, n;
};

__device__ __forceinline__ PromptRows prompt_rows(const PromptArgs& a, int b) {
    PromptRows r;
    r.first = min(max(__ldg(a.offsets + b), 0), a.n_tokens);
    r.n = min(max(__ldg(a.offsets + b + 1), r.first), a.n_tokens) - r.first;
    if (a.seq_len != nullptr) r.n = min(r.n, max(__ldg(a.seq_len + b), 0));
    return r;
}

// Whether they fall: the sequence may then share rows with others.
__device__ __forceinline__ bool prompt_rows_fall(const PromptArgs& a, int b) {
    return min(max(__ldg(a.offsets + b + 1), 0), a.n_tokens) < min(max(__ldg(a.offsets + b), 0), a.n_tokens);
}

// Whether sequence b's borders fall or lie outside the rows.
__device__ __forceinline__ bool prompt_borders_bad(const PromptArgs& a, int b) {
    const int lo = __ldg(a.offsets + b), hi = __ldg(a.offsets + b + 1);
    return lo < 0 || hi < lo || hi > a.n_tokens;
}
#endif

}  // namespace gdn
