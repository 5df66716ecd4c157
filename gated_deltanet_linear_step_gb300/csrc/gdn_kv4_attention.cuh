// gdn_kv4_attention.cuh - what the two kernels of attention over the 4-bit cache
// share: their parameters, the split of the work over the CTAs, unpacking,
// and the queries' and outputs' types.
#pragma once

#include "gdn_kv4.cuh"
#include "gdn_tc.cuh"

namespace gdn {

constexpr float kPShift = 9.0f;  // probabilities are kept relative to 2^-9 of the reference maximum's ...
constexpr float kSlack = 6.0f;   // ... which is raised when a score exceeds it by 6: none is above 2^15
constexpr float kNone = 3.402823466e38f;  // the shift of a column that has seen no key: any finite score is above its negative
// An exponential's argument is one fused product and sum, s mul + shift, so the largest score's misses 9 by what its product was
// rounded by when it became the reference maximum. From 2^27 on (in base 2), where fp32 scores are 8 or more apart, that may be more than probabilities have
// room for: their sum would be 0 or infinite.
constexpr float kBig = 134217728.0f;

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
    // Shared prefixes take two passes. The first, over the prefixes: its sequence g is the rows of a group of sequences, which
    // all see the kv_start[g] tokens of its block table, and leaves normalised outputs and their maxima and sums
    // in prefix_out and prefix_sums. The second, over the sequences' own caches, joins its results with those.
    const int32_t* groups;  // of the first pass: [c.B + 1], the groups' first sequences
    int batch, window;      // of the first pass: sequences, and tokens of a sequence's window (c.T: batch x window)
    float* prefix_out;      // fp32, like q; both NULL without shared prefixes
    float2* prefix_sums;    // per row of prefix_out: maximum, sum
};

// Kernels for calls without shared prefixes are compiled of their own: what those never ask costs 5 to 7 % otherwise (64 sequences
// of up to 8192 tokens, 20 heads of 128: 45.0 and 48.4 us; 2 x 1024 tokens after 8000, 32 heads: 317 and 339 us).
struct PlainParams : AttnParams {};

#ifdef __CUDACC__
// Whether this is the pass over the prefixes; whether the call has any.
__device__ __forceinline__ bool over_prefixes(const AttnParams& p) { return p.groups != nullptr; }
__device__ __forceinline__ bool shares(const AttnParams& p) { return p.prefix_sums != nullptr; }
__device__ __forceinline__ int causal(const AttnParams& p) { return p.groups == nullptr ? 1 : 0; }  // 1: row t sees positions up to kv_start + t
__device__ __forceinline__ constexpr bool over_prefixes(const PlainParams&) { return false; }
__device__ __forceinline__ constexpr bool shares(const PlainParams&) { return false; }
__device__ __forceinline__ constexpr int causal(const PlainParams&) { return 1; }

// Sequences [lo, hi) of group g. The first and last borders are 0 and the batch, so every sequence is in one group, whatever
// the others hold (in two where they fall, which is reported).
template <class P>
__device__ __forceinline__ int group_begin(const P& p, int g) {
    return g == 0 ? 0 : g == p.c.B ? p.batch : min(max(__ldg(p.groups + g), 0), p.batch);
}

// The window of sequence b, or of the group of rows that it is in the pass over the prefixes: there `start` is the last position
// that all of them see (-1: none).
template <class P>
__device__ __forceinline__ Kv4Window attn_window(const P& p, int b) {
    if (!over_prefixes(p)) return kv4_window(p.c, b);
    Kv4Window w;
    w.cap = p.c.max_pages << p.c.page_shift;
    w.start = min(max(__ldg(p.c.kv_start + b), 0), w.cap) - 1;
    w.n = max(group_begin(p, b + 1) - group_begin(p, b), 0) * p.window;
    return w;
}

// Whether tokens lie outside the positions that the block table can hold.
template <class P>
__device__ __forceinline__ bool attn_runs_out(const P& p, int b) {
    if (!over_prefixes(p)) return kv4_runs_out(kv4_window(p.c, b));
    const int n = __ldg(p.c.kv_start + b);
    return n < 0 || n > p.c.max_pages << p.c.page_shift;
}

// Whether borders of the groups are out of order: the first CTA's threads look at some each.
template <class P>
__device__ __forceinline__ bool some_group_falls(const P& p) {
    bool falls = false;
    if (over_prefixes(p) && blockIdx.x == 0) {
        for (int g = threadIdx.x; g <= p.c.B; g += blockDim.x)
            falls = falls || __ldg(p.groups + g) != group_begin(p, g) || (g > 0 && group_begin(p, g) < group_begin(p, g - 1));
    }
    return falls;
}
#endif

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
    const unsigned long long y = static_cast<unsigned long long>(x + 1) * n - 1;
    if ((y | static_cast<unsigned long long>(total)) >> 32) return static_cast<int>(y / static_cast<unsigned long long>(total));
    return static_cast<int>(static_cast<uint32_t>(y) / static_cast<uint32_t>(total));
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

__device__ __forceinline__ bool is_big(float m) { return fabsf(m) >= kBig && fabsf(m) < INFINITY; }

// Whether a score exceeds the reference maximum by more than kSlack.
__device__ __forceinline__ bool is_over(float top, float mul, float shift) { return fmaf(top, mul, shift) > kPShift + kSlack; }

// The factor of the raw scores of a row whose maximum is big, see kBig: a power of two, which rounds nothing, by which the largest one is 2^31 or
// more and the others are 128 or more below it. The row's softmax is taken as that score alone (and its equals).
__device__ __forceinline__ float big_factor(float top) {
    const int e = static_cast<int>(__float_as_uint(fabsf(top)) >> 23) - 127;
    return __uint_as_float(static_cast<uint32_t>(min(31 - e, 127) + 127) << 23);
}

// Raises a row's reference maximum m, and with it its shift, to its largest raw score `top`; returns the factor of what was added up before.
// `first_mul` gives the factor of the row's raw scores, which `mul` is but for rows that are big. (Big rows cost the tensor-core kernels 1 to 2 % of every call:
// chunks of 1024 tokens after 8000, 318 -> 323 us; done over at the unit's end, as gdn_prompt.cu does it for nothing, 2 to 3 %.)
template <class F>
__device__ __forceinline__ float raise(float top, float& m, float& mul, float& shift, F first_mul) {
    float al = 0.0f;
    if (__builtin_expect(is_big(m), 0)) {
        if (!is_over(top, mul, shift)) return 1.0f;
        mul = first_mul();
        m = fmaxf(m, top * mul);
    } else {
        const float v = fmaxf(m, top * mul);
        al = v == m ? 1.0f : exp2_approx(m - v);
        m = v;
    }
    shift = m == -INFINITY ? kNone : kPShift - m;
    if (__builtin_expect(is_big(m), 0)) {
        mul = big_factor(top);
        shift = -top * mul;
    }
    return al;
}

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

template <class P>
__device__ __forceinline__ float4 load_q4(const P& p, size_t i) {
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

// The pass over the sequences' own caches starts while the prefixes' results are still being joined: every CTA waits for those
// before its first use of them, and before its end, so that whatever follows in the stream follows both.
template <class P>
__device__ __forceinline__ void wait_for_prefixes(const P& p) {
    if (shares(p) && !over_prefixes(p)) griddep_wait();
}

// Launches a pass's main kernel, that of the own caches early (wait_for_prefixes).
template <class P>
inline cudaError_t launch_pass(void (*kernel)(P), int ctas, int threads, size_t smem, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = p.prefix_sums != nullptr && p.groups == nullptr ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// The factors of a row's sums (relative to 2^(m - kPShift), their probabilities' sum l) and of its prefix_out. A row that sees no
// key at all is zeros.
struct OutFactors {
    float own, prefix;
};

template <class P>
__device__ __forceinline__ OutFactors out_factors(const P& p, size_t first, float m, float l) {
    if (over_prefixes(p) || !shares(p)) return {l > 0.0f || l != l ? 1.0f / l : 0.0f, 0.0f};
    const float2 before = p.prefix_sums[first / p.c.head_dim];
    const float top = fmaxf(before.x, m);
    if (top == -INFINITY) return {0.0f, 0.0f};
    const float a = exp2_approx(before.x - top) * before.y, b = exp2_approx(m - top);
    const float inv = 1.0f / fmaf(b, l, a);
    return {b * inv, a * inv};
}

// The pass over the prefixes leaves a row's maximum and sum for the other.
template <class P>
__device__ __forceinline__ void keep_sums(const P& p, size_t first, float m, float l) {
    if (over_prefixes(p)) p.prefix_sums[first / p.c.head_dim] = make_float2(m, l);
}

// Outputs i and i + 1 from a row's sums, in the call's type; in the pass over the prefixes fp32 in prefix_out.
template <class P>
__device__ __forceinline__ void store_out2(const P& p, size_t i, float a, float b, const OutFactors& f) {
    a *= f.own;
    b *= f.own;
    if (over_prefixes(p)) {
        *reinterpret_cast<float2*>(p.prefix_out + i) = make_float2(a, b);
        return;
    }
    if (f.prefix != 0.0f) {
        const float2 y = *reinterpret_cast<const float2*>(p.prefix_out + i);
        a = fmaf(y.x, f.prefix, a);
        b = fmaf(y.y, f.prefix, b);
    }
    if (p.dtype == DType::kF32) {
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + i) = make_float2(a, b);
    } else if (p.dtype == DType::kF16) {
        *reinterpret_cast<uint32_t*>(static_cast<__half*>(p.out) + i) = pack_half2(a, b);
    } else {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.out) + i) = *reinterpret_cast<const uint32_t*>(&v);
    }
}

// 16 outputs from a row's sums, in the call's type; in the pass over the prefixes fp32 in prefix_out.
template <class P>
__device__ __forceinline__ void store_out16(const P& p, size_t i, float (&o)[16], const OutFactors& f) {
#pragma unroll
    for (int j = 0; j < 16; ++j) o[j] *= f.own;
    if (f.prefix != 0.0f) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            const float4 y = *reinterpret_cast<const float4*>(p.prefix_out + i + j);
            o[j] = fmaf(y.x, f.prefix, o[j]), o[j + 1] = fmaf(y.y, f.prefix, o[j + 1]);
            o[j + 2] = fmaf(y.z, f.prefix, o[j + 2]), o[j + 3] = fmaf(y.w, f.prefix, o[j + 3]);
        }
    }
    if (p.dtype == DType::kF32 || over_prefixes(p)) {
        float* out = over_prefixes(p) ? p.prefix_out : static_cast<float*>(p.out);
#pragma unroll
        for (int j = 0; j < 16; j += 4) *reinterpret_cast<float4*>(out + i + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        return;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (p.dtype == DType::kF16) {
            w[j] = pack_half2(o[2 * j], o[2 * j + 1]);
        } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * j], o[2 * j + 1]);
            w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + i);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Row (t, query head) of column col of a unit: its first element in q and out.
template <class P>
__device__ __forceinline__ size_t q_row(const P& p, int b, const Unit& x, int col) {
    const int t = p.c.T == 1 ? 0 : col / p.group;
    const int head = x.h * p.group + (col - t * p.group);
    if (over_prefixes(p)) {
        const int s = t / p.window;
        return (((static_cast<size_t>(group_begin(p, b) + s) * p.c.L + x.l) * p.window + (t - s * p.window)) * p.q_heads + head) * p.c.head_dim;
    }
    return (((static_cast<size_t>(b) * p.c.L + x.l) * p.c.T + t) * p.q_heads + head) * p.c.head_dim;
}

// Windows with many rows, on the tensor cores (gdn_kv4_window.cu); sets the fields of its units itself.
cudaError_t launch_kv4_window(AttnParams p, cudaStream_t stream);
size_t kv4_window_workspace_bytes(int head_dim);

// The pass over shared prefixes of 16-bit calls with head_dim <= 128, on the tensor cores (gdn_kv4_prefix.cu); the same workspace.
cudaError_t launch_kv4_prefix(AttnParams p, cudaStream_t stream);

}  // namespace gdn
