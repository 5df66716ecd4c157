// gdn_kv4_attention.cuh - what the two kernels of attention over the 4-bit cache
// share: their parameters, the split of the work over the CTAs, unpacking,
// and the queries' and outputs' types.
#pragma once

#include "gdn_kv4.cuh"

namespace gdn {

constexpr float kPShift = 9.0f;  // probabilities are kept relative to 2^-9 of the reference maximum's ...
constexpr float kSlack = 6.0f;   // ... which is raised when a score exceeds it by 6: none is above 2^15
constexpr float kNone = 1e30f;   // the shift of a column that has seen no key

// The unit, if there is one, whose first rounds a CTA did and whose last ones other CTAs did: what the joining kernel
// needs to know. `parts` CTAs, this one first, have a partial result of it each.
struct JoinRecord {
    int b, block, pair, parts;  // block: of the window kernel; pair: layer and kv head
};

struct AttnParams {
    Kv4Cache c;
    const void* q;
    void* out;
    float* part;    // per CTA two partial results: [columns][D] sums, then maxima and sums of the columns
    void* records;  // per CTA a JoinRecord
    int q_heads, group;
    float* sums;    // of the window kernel: per CTA the sums of earlier tiles
    int unit_rows, col_blocks, tile_shift;  // of the window kernel: rows of a unit, units of a window, log2 of a tile's tokens
    DType dtype;
    float scale;
};

// A unit: its layer, kv head, first column (0 but in the window kernel), and the positions its columns see.
struct Unit {
    int l, h, col0, start, n, end;  // end: first position that no column sees (not above 0: there is none that one sees)
};

// ------------------------------------------------------------ work split --
// a b / c, in 32 bits where they suffice.
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
    const unsigned long long x = static_cast<unsigned long long>(a) * b;
    if ((x | static_cast<unsigned long long>(c)) >> 32) return x / static_cast<unsigned long long>(c);
    return static_cast<uint32_t>(x) / static_cast<uint32_t>(c);
}

// Places [lo, hi) of CTA i of n <= total: each has one at least.
__device__ __forceinline__ void cta_range(long long total, int i, int n, long long& lo, long long& hi) {
    lo = mul_div(total, i, n);
    hi = mul_div(total, i + 1, n);
}

// The CTA of n that has place x: the largest i with total i / n <= x.
__device__ __forceinline__ int cta_of(long long total, long long x, int n) {
    return static_cast<int>(((x + 1) * n - 1) / total);
}

// ---------------------------------------------------------------- pieces --
// The 8 codes of a word as four fp16 pairs, times a pair of scales.
__device__ __forceinline__ void unpack(uint32_t w, uint32_t s, uint32_t (&v)[4]) {
    asm("{\n\t.reg .b8 c0, c1, c2, c3;\n\t"
        "mov.b32 {c0, c1, c2, c3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, c1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, c3;\n\t}"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
        : "r"(w));
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(s));
}

// Byte i (0 or 1) of a as both halves of an fp16 pair of scales.
__device__ __forceinline__ uint32_t scale_twice(uint32_t a, int i) { return __byte_perm(a, 0, i ? 0x4141 : 0x4040) << 7; }
__device__ __forceinline__ float exp2_approx(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// What rounding to fp16 left of two floats, rounded to fp16.
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    return pack_half2(a - f.x, b - f.y);
}

constexpr float kLeastScale = 1.17549435e-38f;  // the factor of raw scores is never 0: 0 times a masked -inf

// 2^(11 - exponent of a row's largest magnitude): scaled by it the row fills fp16's range, exactly.
__device__ __forceinline__ float row_factor(float a) {
    const int e = min(max(static_cast<int>(__float_as_uint(a) >> 23) - 127, -115), 127);
    return a > 0.0f && a < INFINITY ? __uint_as_float(static_cast<uint32_t>(138 - e) << 23) : 1.0f;
}

// Factor of the raw scores of a row that was scaled by f, for exponentials of base 2. The scale is divided first: its
// product with log2(e) may be out of range where the queries are small.
__device__ __forceinline__ float score_factor(float scale, float f) {
    return fmaxf(scale / f * 1.4426950408889634f, kLeastScale);
}

__device__ __forceinline__ float4 load_q4(const AttnParams& p, size_t i) {
    if (p.dtype == DType::kF32) return *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + i);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.q) + i);
    if (p.dtype == DType::kF16) {
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xFFFF0000u));
}

__device__ __forceinline__ void store_out2(const AttnParams& p, size_t i, float a, float b) {
    if (p.dtype == DType::kF32) {
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + i) = make_float2(a, b);
    } else if (p.dtype == DType::kF16) {
        *reinterpret_cast<uint32_t*>(static_cast<__half*>(p.out) + i) = pack_half2(a, b);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + i) = *reinterpret_cast<const uint32_t*>(&v);
    }
}

// Row (t, query head) of column col of a unit: its first element in q and out.
__device__ __forceinline__ size_t q_row(const AttnParams& p, int b, const Unit& x, int col) {
    const int t = p.c.T == 1 ? 0 : col / p.group;
    const int head = x.h * p.group + (col - t * p.group);
    return (((static_cast<size_t>(b) * p.c.L + x.l) * p.c.T + t) * p.q_heads + head) * p.c.head_dim;
}

// Windows with many rows, on the tensor cores (gdn_kv4_window.cu); sets the fields of its units itself.
cudaError_t launch_kv4_window(AttnParams p, cudaStream_t stream);
size_t kv4_window_workspace_bytes(int head_dim);

}  // namespace gdn
