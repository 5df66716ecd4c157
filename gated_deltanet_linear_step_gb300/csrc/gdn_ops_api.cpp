// gdn_ops_api.cpp - the C entry points of the operators beside the decode step
// (declared in include/gdn.h): the 4-bit key/value cache, attention over it, and
// log probabilities. Argument checks on the host, then the launch.

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gdn.h"
#include "gdn_kv4.cuh"

static_assert(GDN_DTYPE_F32 == static_cast<int>(gdn::DType::kF32) && GDN_DTYPE_F16 == static_cast<int>(gdn::DType::kF16) &&
                  GDN_DTYPE_BF16 == static_cast<int>(gdn::DType::kBF16),
              "data type mismatch");
static_assert(GDN_KV4_MAX_T == gdn::kKv4MaxTokens, "window size mismatch");

namespace gdn {
gdn_status report_status(gdn_status s, const char* msg);  // gdn_api.cpp
}

namespace {

using u64 = unsigned long long;

gdn_status fail(gdn_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return gdn::report_status(s, buf);
}

gdn_status launched(cudaError_t e, const char* fn) {
    if (e != cudaSuccess) return fail(GDN_ERR_CUDA, "%s: CUDA error: %s", fn, cudaGetErrorString(e));
    return gdn::report_status(GDN_OK, "");
}

// A buffer of a call: where it lies, how it has to be aligned, and whether it may be NULL.
struct Buffer {
    const char* name;
    const void* p;
    u64 bytes;
    unsigned align;
    bool required, output;
};

gdn_status check_pointers(const char* fn, const Buffer* b, int n) {
    for (int i = 0; i < n; ++i) {
        if (b[i].p == nullptr) {
            if (b[i].required) return fail(GDN_ERR_NULL, "%s: %s is NULL", fn, b[i].name);
            continue;
        }
        if ((reinterpret_cast<u64>(b[i].p) & (b[i].align - 1)) != 0)
            return fail(GDN_ERR_ALIGN, "%s: %s is not %u-byte aligned", fn, b[i].name, b[i].align);
    }
    return GDN_OK;
}

gdn_status check_overlaps(const char* fn, const Buffer* b, int n) {
    for (int i = 0; i < n; ++i) {
        if (!b[i].output || b[i].p == nullptr) continue;
        for (int k = 0; k < n; ++k) {
            if (k == i || b[k].p == nullptr) continue;
            const u64 x = reinterpret_cast<u64>(b[i].p), y = reinterpret_cast<u64>(b[k].p);
            if (x < y + b[k].bytes && y < x + b[i].bytes)
                return fail(GDN_ERR_ALIAS, "%s: output %s overlaps %s", fn, b[i].name, b[k].name);
        }
    }
    return GDN_OK;
}

int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

bool cache_geometry_ok(int kv_heads, int head_dim, int page_size) {
    return kv_heads >= 1 && kv_heads <= 1024 && (head_dim == 64 || head_dim == 128 || head_dim == 256) && page_size >= 16 &&
           page_size <= 256 && (page_size & (page_size - 1)) == 0;
}

bool window_ok(int B, int L, int T, int heads) {
    if (B < 1 || L < 1 || T < 1 || T > GDN_KV4_MAX_T) return false;
    const u64 bl = static_cast<u64>(B) * L;
    return bl < (1ull << 31) && bl * T < (1ull << 31) && bl * T * heads < (1ull << 31);
}

u64 type_size(int dtype) { return dtype == GDN_DTYPE_F32 ? 4 : 2; }

gdn_status check_cache(const char* fn, int B, int L, int T, int kv_heads, int head_dim, int n_pages, int max_pages,
                       int page_size, int dtype) {
    if (dtype < GDN_DTYPE_F32 || dtype > GDN_DTYPE_BF16) return fail(GDN_ERR_DTYPE, "%s: unknown data type %d", fn, dtype);
    if (!cache_geometry_ok(kv_heads, head_dim, page_size))
        return fail(GDN_ERR_SHAPE, "%s: kv_heads=%d in [1, 1024], head_dim=%d in {64, 128, 256}, page_size=%d a power of two in "
                    "[16, 256]", fn, kv_heads, head_dim, page_size);
    if (!window_ok(B, L, T, kv_heads))
        return fail(GDN_ERR_SHAPE, "%s: B=%d, L=%d, T=%d (at most %d) out of range, or too many rows", fn, B, L, T, GDN_KV4_MAX_T);
    if (n_pages < 1 || max_pages < 1 || static_cast<u64>(max_pages) * page_size > (1ull << 30))
        return fail(GDN_ERR_SHAPE, "%s: n_pages=%d, max_pages=%d out of range", fn, n_pages, max_pages);
    return GDN_OK;
}

gdn::Kv4Cache cache_args(const void* cache, const int32_t* block_table, const int32_t* kv_start, const int32_t* seq_len,
                         int B, int L, int T, int kv_heads, int head_dim, int n_pages, int max_pages, int page_size) {
    gdn::Kv4Cache c;
    c.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
    c.block_table = block_table;
    c.kv_start = kv_start;
    c.seq_len = seq_len;
    c.B = B;
    c.L = L;
    c.T = T;
    c.kv_heads = kv_heads;
    c.head_dim = head_dim;
    c.n_pages = n_pages;
    c.max_pages = max_pages;
    c.page_shift = log2_of(page_size);
    return c;
}

// gdn_kv4_append (append) and gdn_kv4_read: the same buffers, the other way round.
gdn_status run_cache(const char* fn, bool append, const void* k, const void* v, const void* cache,
                     const int32_t* block_table, const int32_t* kv_start, const int32_t* seq_len, int B, int L, int T,
                     int kv_heads, int head_dim, int n_pages, int max_pages, int page_size, int dtype, void* stream) {
    gdn_status s = check_cache(fn, B, L, T, kv_heads, head_dim, n_pages, max_pages, page_size, dtype);
    if (s != GDN_OK) return s;
    const u64 rows = static_cast<u64>(B) * L * T * kv_heads * head_dim * type_size(dtype);
    const u64 cache_bytes = static_cast<u64>(L) * n_pages * kv_heads * gdn::kv4_head_bytes(page_size, head_dim);
    const Buffer b[] = {{"k", k, rows, 16, true, !append},
                        {"v", v, rows, 16, true, !append},
                        {"cache", cache, cache_bytes, 16, true, append},
                        {"block_table", block_table, static_cast<u64>(B) * max_pages * 4, 4, true, false},
                        {"kv_start", kv_start, static_cast<u64>(B) * 4, 4, true, false},
                        {"seq_len", seq_len, static_cast<u64>(B) * 4, 4, false, false}};
    const int n = static_cast<int>(sizeof(b) / sizeof(b[0]));
    if ((s = check_pointers(fn, b, n)) != GDN_OK || (s = check_overlaps(fn, b, n)) != GDN_OK) return s;
    const gdn::Kv4Cache c = cache_args(cache, block_table, kv_start, seq_len, B, L, T, kv_heads, head_dim, n_pages,
                                       max_pages, page_size);
    const gdn::DType d = static_cast<gdn::DType>(dtype);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launched(append ? gdn::launch_kv4_append(c, k, v, d, st)
                           : gdn::launch_kv4_read(c, const_cast<void*>(k), const_cast<void*>(v), d, st), fn);
}

// Whether the query side of an attention call is in range.
bool queries_ok(int B, int L, int T, int q_heads, int kv_heads) {
    if (q_heads < 1 || q_heads > 4096 || q_heads % kv_heads != 0) return false;
    // units (layer, kv head, block of at least 8 columns) stay below 2^30
    return window_ok(B, L, T, q_heads) && static_cast<u64>(L) * kv_heads * (static_cast<u64>(T) * q_heads / kv_heads / 8 + 1) < (1ull << 30);
}

}  // namespace

extern "C" {

size_t gdn_kv4_page_bytes(int kv_heads, int head_dim, int page_size) {
    if (!cache_geometry_ok(kv_heads, head_dim, page_size)) return 0;
    return kv_heads * gdn::kv4_head_bytes(page_size, head_dim);
}

gdn_status gdn_kv4_append(const void* k, const void* v, void* cache, const int32_t* block_table, const int32_t* kv_start,
                          const int32_t* seq_len, int B, int L, int T, int kv_heads, int head_dim, int n_pages,
                          int max_pages, int page_size, int dtype, void* stream) {
    return run_cache("gdn_kv4_append", true, k, v, cache, block_table, kv_start, seq_len, B, L, T, kv_heads, head_dim,
                     n_pages, max_pages, page_size, dtype, stream);
}

gdn_status gdn_kv4_read(const void* cache, const int32_t* block_table, const int32_t* kv_start, const int32_t* seq_len,
                        void* k, void* v, int B, int L, int T, int kv_heads, int head_dim, int n_pages, int max_pages,
                        int page_size, int dtype, void* stream) {
    return run_cache("gdn_kv4_read", false, k, v, cache, block_table, kv_start, seq_len, B, L, T, kv_heads, head_dim,
                     n_pages, max_pages, page_size, dtype, stream);
}

size_t gdn_kv4_attention_workspace_size(int B, int L, int T, int q_heads, int kv_heads, int head_dim) {
    if (!cache_geometry_ok(kv_heads, head_dim, 16) || !queries_ok(B, L, T, q_heads, kv_heads)) return 0;
    return gdn::kv4_attention_workspace_bytes(B, L, T, q_heads, kv_heads, head_dim);
}

gdn_status gdn_kv4_attention(const void* q, const void* cache, const int32_t* block_table, const int32_t* kv_start,
                             const int32_t* seq_len, void* out, void* workspace, size_t workspace_bytes, int B, int L,
                             int T, int q_heads, int kv_heads, int head_dim, int n_pages, int max_pages, int page_size,
                             int dtype, float scale, void* stream) {
    const char* fn = "gdn_kv4_attention";
    gdn_status s = check_cache(fn, B, L, T, kv_heads, head_dim, n_pages, max_pages, page_size, dtype);
    if (s != GDN_OK) return s;
    if (!queries_ok(B, L, T, q_heads, kv_heads))
        return fail(GDN_ERR_SHAPE, "%s: q_heads=%d must be a multiple of kv_heads=%d, at most 4096, with fewer than 2^31 rows", fn,
                    q_heads, kv_heads);
    if (!(scale > 0.0f) || !std::isfinite(scale)) return fail(GDN_ERR_SHAPE, "%s: scale=%g must be positive", fn, scale);
    const size_t need = gdn::kv4_attention_workspace_bytes(B, L, T, q_heads, kv_heads, head_dim);
    const u64 rows = static_cast<u64>(B) * L * T * q_heads * head_dim * type_size(dtype);
    const u64 cache_bytes = static_cast<u64>(L) * n_pages * kv_heads * gdn::kv4_head_bytes(page_size, head_dim);
    const Buffer b[] = {{"q", q, rows, 16, true, false},
                        {"cache", cache, cache_bytes, 16, true, false},
                        {"block_table", block_table, static_cast<u64>(B) * max_pages * 4, 4, true, false},
                        {"kv_start", kv_start, static_cast<u64>(B) * 4, 4, true, false},
                        {"seq_len", seq_len, static_cast<u64>(B) * 4, 4, false, false},
                        {"out", out, rows, 16, true, true},
                        {"workspace", workspace, need, 16, true, true}};
    const int n = static_cast<int>(sizeof(b) / sizeof(b[0]));
    if ((s = check_pointers(fn, b, n)) != GDN_OK) return s;
    if (workspace_bytes < need)
        return fail(GDN_ERR_SHAPE, "%s: workspace of %zu bytes, %zu needed", fn, workspace_bytes, need);
    if ((s = check_overlaps(fn, b, n)) != GDN_OK) return s;
    gdn::Kv4AttnArgs a;
    a.c = cache_args(cache, block_table, kv_start, seq_len, B, L, T, kv_heads, head_dim, n_pages, max_pages, page_size);
    a.q = q;
    a.out = out;
    a.workspace = workspace;
    a.q_heads = q_heads;
    a.dtype = static_cast<gdn::DType>(dtype);
    a.scale = scale;
    return launched(gdn::launch_kv4_attention(a, static_cast<cudaStream_t>(stream)), fn);
}

gdn_status gdn_logprobs(const void* logits, const int32_t* tokens, float* logprob, float* entropy, int32_t* top_ids,
                        float* top_logprobs, int64_t n_rows, int64_t vocab, int64_t row_stride, int k, int dtype,
                        void* stream) {
    const char* fn = "gdn_logprobs";
    if (dtype < GDN_DTYPE_F32 || dtype > GDN_DTYPE_BF16) return fail(GDN_ERR_DTYPE, "%s: unknown data type %d", fn, dtype);
    if (n_rows < 1 || n_rows > (1 << 26) || vocab < 1 || vocab > (1ll << 31) - 1 || row_stride < vocab ||
        row_stride > (1ll << 40) / n_rows)
        return fail(GDN_ERR_SHAPE, "%s: n_rows=%lld, vocab=%lld, row_stride=%lld out of range", fn,
                    static_cast<long long>(n_rows), static_cast<long long>(vocab), static_cast<long long>(row_stride));
    if (k < 0 || k > GDN_LOGPROBS_MAX_K || k > vocab)
        return fail(GDN_ERR_SHAPE, "%s: k=%d must be in [0, min(vocab, %d)]", fn, k, GDN_LOGPROBS_MAX_K);
    const u64 es = type_size(dtype), rows = static_cast<u64>(n_rows);
    const Buffer b[] = {
        {"logits", logits, ((rows - 1) * row_stride + vocab) * es, static_cast<unsigned>(es), true, false},
        {"tokens", tokens, rows * 4, 4, logprob != nullptr, false},
        {"logprob", logprob, rows * 4, 4, false, true},
        {"entropy", entropy, rows * 4, 4, false, true},
        {"top_ids", top_ids, rows * k * 4, 4, k > 0, k > 0},
        {"top_logprobs", top_logprobs, rows * k * 4, 4, k > 0, k > 0}};
    const int n = static_cast<int>(sizeof(b) / sizeof(b[0]));
    gdn_status s;
    if ((s = check_pointers(fn, b, n)) != GDN_OK || (s = check_overlaps(fn, b, n)) != GDN_OK) return s;
    gdn::LogprobArgs a;
    a.logits = logits;
    a.tokens = tokens;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.n_rows = n_rows;
    a.vocab = vocab;
    a.ld = row_stride;
    a.k = k;
    a.dtype = static_cast<gdn::DType>(dtype);
    return launched(gdn::launch_logprobs(a, static_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
