// gdn_kv4_cache.cu - writing keys and values into the 4-bit cache and reading
// them back (the format and the page layout are in gdn_kv4.cuh).
//
// Both are one pass over the data: HBM is the floor. Writing: one thread per
// block of 16 values, K and V of the same block one after the other, so that
// both loads are in flight together; consecutive threads take the blocks of a
// token and then the next token of the same head, so a warp's codes and scales
// land in contiguous 256- and 32-byte pieces. Reading: 16 bytes of output
// per place, so every store of a warp is one contiguous 512-byte piece.
//
// Measured: 16 x 1024 ragged tokens of 4 layers, 8 heads of 128, bf16 (127 MB in, 36 MB of cache written): 35 us, 0.69 of
// the measured HBM rate; with correctly rounded quotients, as fp32 values still take, 13 us more. One token of 64
// sequences, written and read back: 5 us, two launches and the latency of three dependent reads each.

#include "gdn_kv4.cuh"

namespace gdn {
namespace {

constexpr int kCacheThreads = 256;

__device__ unsigned int g_kv4_cache_error = 0;

// Unsigned division by a number fixed at launch: n / d = (n * m) >> 32 >> s, exact for n < 2^31.
struct FastDiv {
    uint32_t d, m, s;
    void set(uint32_t div) {
        d = div;
        s = 0;
        while ((1u << s) < div) ++s;
        m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - div)) / div + 1);
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

struct CacheParams {
    Kv4Cache c;
    const void* in_k;
    const void* in_v;
    void* out_k;
    void* out_v;
    FastDiv by_t, by_heads, by_layers;
    uint32_t rows;  // B L kv_heads T
};

template <typename T>
__device__ __forceinline__ float2 pair_of(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_of<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 pair_of<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// 16 consecutive values, as they are and as floats.
template <typename T>
struct Raw16 {
    uint4 v[sizeof(T)];
    __device__ __forceinline__ explicit Raw16(const T* p) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) v[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void floats(float (&x)[16]) const {
#pragma unroll
        for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (sizeof(T) == 4) {
                    x[4 * i + j] = __uint_as_float(w[j]);
                } else {
                    const float2 f = pair_of<T>(w[j]);
                    x[8 * i + 2 * j] = f.x;
                    x[8 * i + 2 * j + 1] = f.y;
                }
            }
        }
    }
};

// max of two magnitudes; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// a >= 0 to the nearest scale byte, ties to even.
__device__ __forceinline__ uint32_t scale_byte(float a) {
    a = fminf(a, kKv4MaxScale);
    if (a < 6.103515625e-05f) return static_cast<uint32_t>(__float2int_rn(a * 131072.0f));  // below 2^-14: steps of 2^-17
    uint32_t u = __float_as_uint(a);
    u += 0x7FFFFu + ((u >> 20) & 1u);
    return (u >> 20) - (112u << 3);
}

__device__ __forceinline__ float scale_value(uint32_t b) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}

// Two floats as e2m1 codes, a in the low nibble.
__device__ __forceinline__ uint32_t e2m1_pair(float a, float b) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}" : "=r"(r) : "f"(a), "f"(b));
    return r;
}

// Two quotients x / s as e2m1 codes. fp32 values take the correctly rounded quotient. A 16-bit value's quotient is
// either exactly half way between two codes or off it by 2^-11 of itself at least (x has 11 significant bits, half way
// points times s have 7), so the product with 1 / s, within 2^-22 of the quotient, decides as well once it is rounded
// to 16 bits, which makes a half way point exact again: 5 operations for a pair instead of about 18.
template <typename T>
__device__ __forceinline__ uint32_t code_pair(float a, float b, float s, float r) {
    if constexpr (sizeof(T) == 4) return e2m1_pair(__fdiv_rn(a, s), __fdiv_rn(b, s));
    const float2 y = __fmul2_rn(make_float2(a, b), make_float2(r, r));
    const float2 c = __fmul2_rn(y, make_float2(257.0f, 257.0f));  // c - (c - y) is y to 16 bits (Dekker's splitting)
    const float2 d = __fadd2_rn(c, make_float2(-y.x, -y.y));
    return e2m1_pair(c.x - d.x, c.y - d.y);
}

// The block's codes (8 bytes, value 0 in the lowest nibble) and its scale byte.
// The codes are those of the exact quotients, so they do not depend on
// the order of work: a plain restatement gives the same bytes.
template <typename T>
__device__ __forceinline__ uint32_t quantise16(float (&x)[16], uint2& codes) {
    float a = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) a = max_nan(a, fabsf(x[i]));
    if (!(a <= 6.0f * kKv4MaxScale)) {  // NaN counts as 0, what is larger saturates
        a = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            x[i] = x[i] == x[i] ? fminf(fmaxf(x[i], -6.0f * kKv4MaxScale), 6.0f * kKv4MaxScale) : 0.0f;
            a = fmaxf(a, fabsf(x[i]));
        }
    }
    const uint32_t byte = scale_byte(a / 6.0f);
    if (byte == 0u) {
        codes = make_uint2(0u, 0u);
        return 0u;
    }
    const float s = scale_value(byte), r = __frcp_rn(s);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= code_pair<T>(x[2 * i], x[2 * i + 1], s, r) << (8 * (i & 3));
    codes = make_uint2(w[0], w[1]);
    return byte;
}

// Six CTAs per SM for 16-bit values, 40 registers (fp32 ones, which wait for their correctly rounded quotients, are
// slower so: 128 against 117 us): 16 x 1024 ragged tokens of 4 layers, 8 heads of 128, written and read back, 74.2 -> 69.9 us.
template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads, sizeof(T) == 4 ? 1 : 6) kv4_append_kernel(const __grid_constant__ CacheParams p) {
    constexpr int kBlocks = D / 16;
    const unsigned long long item = static_cast<unsigned long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
    const int blk = static_cast<int>(item) & (kBlocks - 1);
    if (item / kBlocks >= p.rows) return;
    const uint32_t row = static_cast<uint32_t>(item / kBlocks);
    const uint32_t bhl = p.by_t.div(row);
    const int t = static_cast<int>(row - bhl * p.by_t.d);
    const uint32_t bl = p.by_heads.div(bhl);
    const int h = static_cast<int>(bhl - bl * p.by_heads.d);
    const int b = static_cast<int>(p.by_layers.div(bl));
    const int l = static_cast<int>(bl - b * p.by_layers.d);
    const Kv4Window w = kv4_window(p.c, b);
    if (t >= w.n) return;
    const size_t src = ((static_cast<size_t>(bl) * p.c.T + t) * p.c.kv_heads + h) * D + blk * 16;
    const Raw16<T> k(static_cast<const T*>(p.in_k) + src), v(static_cast<const T*>(p.in_v) + src);
    const int page = t < w.cap - w.start ? kv4_page(p.c, b, w.start + t) : -1;
    if (page < 0) {
        if (blk == 0) atomicOr(&g_kv4_cache_error, kErrBadPage);
        return;
    }
    const int psize = 1 << p.c.page_shift;
    const int r = (w.start + t) & (psize - 1);
    uint8_t* kc = p.c.cache + kv4_head_offset(p.c, l, page, h);
    uint8_t* vc = kc + kv4_head_bytes(psize, D) / 2;
    const int code_at = r * (D / 2) + (blk ^ kv4_swizzle(r, kBlocks)) * 8;
    const int scale_at = psize * (D / 2) + r * kBlocks + blk;
    uint2 codes;
    float x[16];
    k.floats(x);
    uint32_t s = quantise16<T>(x, codes);
    *reinterpret_cast<uint2*>(kc + code_at) = codes;
    kc[scale_at] = static_cast<uint8_t>(s);
    v.floats(x);
    s = quantise16<T>(x, codes);
    *reinterpret_cast<uint2*>(vc + code_at) = codes;
    vc[scale_at] = static_cast<uint8_t>(s);
}

// The two codes of a byte as fp16 values, the low nibble's in the low half.
__device__ __forceinline__ __half2 e2m1_values(uint32_t byte) {
    uint32_t r;
    asm("{\n\t.reg .b8 c;\n\tcvt.u8.u32 c, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(byte));
    return *reinterpret_cast<const __half2*>(&r);
}

// kPer consecutive values (16 bytes of output) from their codes and scale.
__device__ __forceinline__ void store_values(float* out, uint32_t codes, __half2 s) {
    const float2 a = __half22float2(__hmul2(e2m1_values(codes & 255u), s));
    const float2 b = __half22float2(__hmul2(e2m1_values(codes >> 8), s));
    __stcs(reinterpret_cast<float4*>(out), make_float4(a.x, a.y, b.x, b.y));
}

template <typename T>
__device__ __forceinline__ uint32_t pack_pair(__half2 v);
template <>
__device__ __forceinline__ uint32_t pack_pair<__half>(__half2 v) {
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack_pair<__nv_bfloat16>(__half2 v) {
    const float2 f = __half22float2(v);
    const __nv_bfloat162 o = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&o);
}

template <typename T>
__device__ __forceinline__ void store_values(T* out, uint32_t codes, __half2 s) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_pair<T>(__hmul2(e2m1_values((codes >> (8 * i)) & 255u), s));
    __stcs(reinterpret_cast<uint4*>(out), make_uint4(o[0], o[1], o[2], o[3]));
}

// kReadItems places per thread, kCacheThreads apart, step by step: what a place needs is found by three
// dependent loads (the window, the page's number, the codes). 65536 tokens of 8 heads of 128, bf16 / fp32: 64 / 111 us
// with one place per thread, 61 / 94 with two (0.84 / 0.96 of the measured HBM rate), 69 / 106 with four.
constexpr int kReadItems = 2;

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) kv4_read_kernel(const __grid_constant__ CacheParams p) {
    constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // values per place
    constexpr int kChunks = D / kPer;
    const int psize = 1 << p.c.page_shift;
    const unsigned long long item0 = static_cast<unsigned long long>(blockIdx.x) * (kCacheThreads * kReadItems) + threadIdx.x;
    const int d = (static_cast<int>(item0) & (kChunks - 1)) * kPer;  // kCacheThreads is a multiple of kChunks
    uint32_t row[kReadItems];
    int h[kReadItems], l[kReadItems], b[kReadItems], t[kReadItems], pos[kReadItems], page[kReadItems];
    bool on[kReadItems];
#pragma unroll
    for (int i = 0; i < kReadItems; ++i) {
        const unsigned long long r = (item0 + i * kCacheThreads) / kChunks;  // ((b L + l) T + t) kv_heads + h
        on[i] = r < p.rows;
        row[i] = on[i] ? static_cast<uint32_t>(r) : 0u;
        const uint32_t blt = p.by_heads.div(row[i]);
        h[i] = static_cast<int>(row[i] - blt * p.by_heads.d);
        const uint32_t bl = p.by_t.div(blt);
        t[i] = static_cast<int>(blt - bl * p.by_t.d);
        b[i] = static_cast<int>(p.by_layers.div(bl));
        l[i] = static_cast<int>(bl - b[i] * p.by_layers.d);
    }
#pragma unroll
    for (int i = 0; i < kReadItems; ++i) {
        const Kv4Window w = kv4_window(p.c, b[i]);
        on[i] = on[i] && t[i] < w.n;
        pos[i] = t[i] < w.cap - w.start ? w.start + t[i] : -1;  // below 0: not in the table
    }
#pragma unroll
    for (int i = 0; i < kReadItems; ++i) page[i] = on[i] && pos[i] >= 0 ? kv4_page(p.c, b[i], pos[i]) : -1;
    uint32_t kw[kReadItems], vw[kReadItems], ks[kReadItems], vs[kReadItems];
#pragma unroll
    for (int i = 0; i < kReadItems; ++i) {
        kw[i] = vw[i] = ks[i] = vs[i] = 0u;  // a token that is not there reads as zeros
        if (page[i] < 0) continue;
        const int r = pos[i] & (psize - 1);
        const uint8_t* kc = p.c.cache + kv4_head_offset(p.c, l[i], page[i], h[i]);
        const uint8_t* vc = kc + kv4_head_bytes(psize, D) / 2;
        const int code_at = r * (D / 2) + ((d >> 4) ^ kv4_swizzle(r, D / 16)) * 8 + ((d & 15) >> 1);
        const int scale_at = psize * (D / 2) + r * (D / 16) + (d >> 4);
        if constexpr (kPer == 8) {
            kw[i] = *reinterpret_cast<const uint32_t*>(kc + code_at);
            vw[i] = *reinterpret_cast<const uint32_t*>(vc + code_at);
        } else {
            kw[i] = *reinterpret_cast<const uint16_t*>(kc + code_at);
            vw[i] = *reinterpret_cast<const uint16_t*>(vc + code_at);
        }
        ks[i] = kc[scale_at];
        vs[i] = vc[scale_at];
    }
#pragma unroll
    for (int i = 0; i < kReadItems; ++i) {
        if (!on[i]) continue;
        if (page[i] < 0 && d == 0) atomicOr(&g_kv4_cache_error, kErrBadPage);
        const size_t at = static_cast<size_t>(row[i]) * D + d;
        store_values(static_cast<T*>(p.out_k) + at, kw[i], __half2half2(__ushort_as_half(static_cast<unsigned short>(ks[i] << 7))));
        store_values(static_cast<T*>(p.out_v) + at, vw[i], __half2half2(__ushort_as_half(static_cast<unsigned short>(vs[i] << 7))));
    }
}

template <typename T, int D>
cudaError_t launch_one(bool append, const CacheParams& p, cudaStream_t stream) {
    const unsigned long long per_row = append ? D / 16 : D * sizeof(T) / 16;
    const unsigned long long per_block = append ? kCacheThreads : kCacheThreads * kReadItems;
    const unsigned long long blocks = (p.rows * per_row + per_block - 1) / per_block;
    if (append)
        kv4_append_kernel<T, D><<<static_cast<unsigned>(blocks), kCacheThreads, 0, stream>>>(p);
    else
        kv4_read_kernel<T, D><<<static_cast<unsigned>(blocks), kCacheThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(bool append, const CacheParams& p, cudaStream_t stream) {
    switch (p.c.head_dim) {
        case 64: return launch_one<T, 64>(append, p, stream);
        case 128: return launch_one<T, 128>(append, p, stream);
        case 256: return launch_one<T, 256>(append, p, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_cache(bool append, CacheParams& p, DType dtype, cudaStream_t stream) {
    p.by_t.set(p.c.T);
    p.by_heads.set(p.c.kv_heads);
    p.by_layers.set(p.c.L);
    p.rows = static_cast<uint32_t>(p.c.B) * p.c.L * p.c.T * p.c.kv_heads;
    switch (dtype) {
        case DType::kF32: return launch_typed<float>(append, p, stream);
        case DType::kF16: return launch_typed<__half>(append, p, stream);
        case DType::kBF16: return launch_typed<__nv_bfloat16>(append, p, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Cache& c, const void* k, const void* v, DType dtype, cudaStream_t stream) {
    CacheParams p{};
    p.c = c;
    p.in_k = k;
    p.in_v = v;
    return launch_cache(true, p, dtype, stream);
}

cudaError_t launch_kv4_read(const Kv4Cache& c, void* k, void* v, DType dtype, cudaStream_t stream) {
    CacheParams p{};
    p.c = c;
    p.out_k = k;
    p.out_v = v;
    return launch_cache(false, p, dtype, stream);
}

cudaError_t read_kv4_cache_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_cache_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_cache_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace gdn
