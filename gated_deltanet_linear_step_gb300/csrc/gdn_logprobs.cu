// gdn_logprobs.cu - log probabilities of given tokens, entropy and the k most
// likely tokens of rows of logits, in one pass over the logits:
//
//   lse = m + log sum exp(x - m),  logprob = x[token] - lse,
//   H = lse - sum p x = log S - W / S  with  S = sum exp(x - m), W = sum exp(x - m) (x - m)
//
// Bound by HBM: a logit is read once, and each costs about 8 issue slots of a lane,
// of the 11 that an SM has for a 16-bit value at the HBM rate. Every thread keeps the running (m, S, W) of
// its own elements; a batch of 16-byte loads first raises m, so the
// exponentials of the batch need no rescaling. A row is shared by a cluster of up to 16
// CTAs that push their results into the first one's shared memory, so one row
// already keeps 16 SMs busy and no workspace is needed.
//
// Measured: 2048 rows of 131072 bf16, k = 4: 105 us (0.76 of the measured HBM rate; 93 us without the top k, 150 us at
// k = 32); 128 rows of 200001 fp32, k = 20: 29 us (0.52); one row of 131072 fp32: 7.4 us. What is left over is
// the end of a CTA: all eight of an SM reach it together, so the reads and joins of the top k are not hidden.
//
// Top k without a second pass: the threads' own maxima are known after the
// pass. With tau the k-th largest of a CTA's maxima (to 16 bits, from below), at
// least k elements are >= tau, and only the threads whose maximum is >= tau, about
// k of them, can hold one: their elements are read again (from L2, by all threads) and
// what is >= tau is listed. The list, a little over k long, is ranked by value and
// then by lowest index; its order of writing does not matter. A list that runs over (many equal
// values) is replaced by k rounds of an exact search, each a pass over the CTA's share. A mask that leaves a CTA's
// threads fewer than k maxima is such a case: 128 rows of 131072 fp32, k = 20, 498 us with 60 tokens left, 21 us without a mask.
//
// Sums are fp32, one per thread over ceil(V / 256 / CTAs of the row) elements (512 for many rows of 131072, 32 for one) and then
// by trees. x - m is taken before the factor log2(e) of the exponential: scaled by it,
// a mask of the type's lowest value would overflow, and a row of such masks alone has a distribution.

#include <cooperative_groups.h>

#include <algorithm>
#include <atomic>

#include "gdn_kv4.cuh"

namespace cg = cooperative_groups;

namespace gdn {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxK = 32;
constexpr int kList = 512;       // candidates of a CTA
static_assert(kMaxK * 16 <= kList, "the lists of a cluster fit too");
constexpr int kMaxCluster = 16;
constexpr int kBatch = 2;        // 16-byte loads of a batch; two batches of a thread are in flight
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -700.0f;  // exp of less is 0 anyway; keeps 0 * inf out of W

struct Sums {
    float m, s, w;  // maximum, sum, weighted sum relative to it
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ Sums join(Sums a, Sums b) {
    Sums r;
    r.m = max_nan(a.m, b.m);
    const float da = fmaxf(a.m - r.m, kLeast), db = fmaxf(b.m - r.m, kLeast);  // -inf - -inf: no elements, s = 0
    const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
    r.s = a.s * fa + b.s * fb;
    r.w = (a.w + da * a.s) * fa + (b.w + db * b.s) * fb;
    return r;
}

// The sums of lanes 0 .. n - 1 (n a power of two; the others hold none), in every lane.
__device__ __forceinline__ Sums join_lanes(Sums s, int lane, int n) {
    for (int o = n / 2; o > 0; o >>= 1) {
        Sums y;
        y.m = __shfl_xor_sync(~0u, s.m, o);
        y.s = __shfl_xor_sync(~0u, s.s, o);
        y.w = __shfl_xor_sync(~0u, s.w, o);
        s = (lane & o) ? join(y, s) : join(s, y);
    }
    return s;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Order of values as unsigned numbers: NaN above all, both zeros equal.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) return 0xFFFFFFFEu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Candidate order: larger value first, then lower index; as one number, larger is better.
__device__ __forceinline__ unsigned long long rank_key(uint32_t key, uint32_t index) {
    return (static_cast<unsigned long long>(key) << 32) | (0xFFFFFFFFu - index);
}

template <typename T>
__device__ __forceinline__ void widen(const uint4& v, float* x);
template <>
__device__ __forceinline__ void widen<float>(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void widen<__half>(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
template <>
__device__ __forceinline__ void widen<__nv_bfloat16>(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(w[i] << 16), x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
// The largest of a vector's elements; NaN if one is.
template <typename T>
__device__ __forceinline__ float vector_max(const uint4& v);
template <>
__device__ __forceinline__ float vector_max<float>(const uint4& v) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
}
template <>
__device__ __forceinline__ float vector_max<__half>(const uint4& v) {
    const __half2* h = reinterpret_cast<const __half2*>(&v);
    const float2 f = __half22float2(__hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])));
    return max_nan(f.x, f.y);
}
template <>
__device__ __forceinline__ float vector_max<__nv_bfloat16>(const uint4& v) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
    const float2 f = __bfloat1622float2(__hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3])));
    return max_nan(f.x, f.y);
}
__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }

// A row as 16-byte vectors of its aligned-down address: elements outside [0, vocab) are -inf.
template <typename T>
struct Row {
    static constexpr int kPer = 16 / static_cast<int>(sizeof(T));
    const T* base;    // aligned down
    int skip;         // elements of the first vector before the row
    long long vocab;
    __device__ __forceinline__ long long vectors() const { return (skip + vocab + kPer - 1) / kPer; }
    __device__ __forceinline__ long long index(long long v, int e) const { return v * kPer + e - skip; }
    __device__ __forceinline__ bool inside(long long v) const {
        return v * kPer >= skip && (v + 1) * kPer <= skip + vocab;
    }
    __device__ __forceinline__ void load(long long v, float* x) const {
        if (inside(v)) {
            widen<T>(__ldg(reinterpret_cast<const uint4*>(base) + v), x);
            return;
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const long long i = index(v, e);
            x[e] = i >= 0 && i < vocab ? to_float(base[v * kPer + e]) : -INFINITY;
        }
    }
};

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 8) logprobs_kernel(const LogprobArgs a) {
    using R = Row<T>;
    constexpr int kPer = R::kPer;
    __shared__ Sums part[kLpWarps];
    __shared__ Sums parts[kMaxCluster];  // in rank 0: every CTA's sums
    __shared__ Sums whole;
    __shared__ unsigned long long floor_s;
    __shared__ unsigned long long list[kList];
    __shared__ unsigned long long best[kMaxK];     // this CTA's top k
    __shared__ unsigned long long joined[kMaxCluster * kMaxK];
    __shared__ unsigned long long warp_best[kLpWarps];
    __shared__ uint32_t keys[kLpThreads];
    __shared__ int holders[kLpThreads];
    __shared__ uint32_t tau_s;
    __shared__ int count, n_holders;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const long long row = blockIdx.x / ranks;
    cluster_arrive();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    R r;
    {
        const T* p = static_cast<const T*>(a.logits) + row * a.ld;
        r.skip = static_cast<int>((reinterpret_cast<unsigned long long>(p) & 15u) / sizeof(T));
        r.base = p - r.skip;
        r.vocab = a.vocab;
    }
    const long long nv = r.vectors(), per = (nv + ranks - 1) / ranks;
    const long long v0 = rank * per, v1 = min(v0 + per, nv);

    // --- one pass: the thread's maximum and sums
    Sums t{-INFINITY, 0.0f, 0.0f};
    auto raise = [&](float bm) {
        if (!(bm <= t.m)) {  // raised (or NaN)
            const float m = max_nan(t.m, bm);
            const float d = fmaxf(t.m - m, kLeast), f = ex2(d * kLog2e);
            t.w = (t.w + d * t.s) * f;
            t.s *= f;
            t.m = m;
        }
    };
    auto take = [&](const float* x) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const float d = fmaxf(x[e] - t.m, kLeast), p = ex2(d * kLog2e);
            t.s += p;
            t.w = fmaf(p, d, t.w);
        }
    };
    // vector u is thread (u - w0) mod kLpThreads's; [w0, w1) lie in the row as a whole and come a batch of loads at a time
    const long long w0 = max(v0, r.skip > 0 ? 1ll : 0ll), w1 = min(v1, (r.skip + r.vocab) / kPer);
    const uint4* vec = reinterpret_cast<const uint4*>(r.base);
    long long v = w0 + tid;
    // the next batch is requested before the current one is worked on
    constexpr long long kStep = static_cast<long long>(kBatch) * kLpThreads;
    auto fetch = [&](uint4 (&w)[kBatch], long long at) {
        if (at + kStep - kLpThreads < w1) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i) w[i] = __ldg(vec + at + i * kLpThreads);
        }
    };
    auto work = [&](const uint4 (&w)[kBatch]) {
        float bm = vector_max<T>(w[0]);
#pragma unroll
        for (int i = 1; i < kBatch; ++i) bm = max_nan(bm, vector_max<T>(w[i]));
        raise(bm);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            float x[kPer];
            widen<T>(w[i], x);
            take(x);
        }
    };
    uint4 wa[kBatch], wb[kBatch];
    fetch(wa, v);
    while (v + kStep - kLpThreads < w1) {
        fetch(wb, v + kStep);
        work(wa);
        v += kStep;
        if (v + kStep - kLpThreads >= w1) break;
        fetch(wa, v + kStep);
        work(wb);
        v += kStep;
    }
    for (; v < w1; v += kLpThreads) {
        const uint4 w = __ldg(vec + v);
        float x[kPer];
        widen<T>(w, x);
        raise(vector_max<T>(w));
        take(x);
    }
    // the row's first and last vector, if they are not whole
    auto edge = [&](long long u) {
        if (static_cast<int>((u - w0 + kLpThreads) % kLpThreads) != tid) return;
        float x[kPer], bm = -INFINITY;
        r.load(u, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) bm = max_nan(bm, x[e]);
        raise(bm);
        take(x);
    };
    if (v0 < w0 && v0 < v1) edge(v0);
    if (w1 < v1 && v1 - 1 >= w0) edge(v1 - 1);

    // --- the CTA's sums
    const Sums s = join_lanes(t, lane, 32);
    if (lane == 0) part[warp] = s;
    if (tid == 0) count = n_holders = 0;
    __syncthreads();

    // --- the CTA's top k
    const int k = a.k;
    if (k > 0) {
        // tau: the largest multiple of 2^16 that at least k maxima reach (0 if there are fewer)
        keys[tid] = order_key(t.m);
        __syncthreads();
        if (warp == 0) {
            uint32_t key[kLpThreads / 32];
#pragma unroll
            for (int i = 0; i < kLpThreads / 32; ++i) key[i] = keys[32 * i + lane];
            uint32_t c = 0;
            for (int bit = 31; bit >= 16; --bit) {
                const uint32_t next = c | (1u << bit);
                int n = 0;
#pragma unroll
                for (int i = 0; i < kLpThreads / 32; ++i) n += key[i] >= next;
                if (__reduce_add_sync(~0u, n) >= k) c = next;
            }
            if (lane == 0) tau_s = c;
        }
        __syncthreads();
        const uint32_t tau = tau_s;
        if (keys[tid] >= tau) holders[atomicAdd(&n_holders, 1)] = tid;
        __syncthreads();
        // the holders' vectors are read again, by all threads
        const int turns = static_cast<int>((v1 - w0 + kLpThreads - 1) / kLpThreads) + 1;  // vectors of a thread, at most
        for (int i = tid; i < n_holders * turns; i += kLpThreads) {
            const int h = i / turns;
            const long long u = w0 + holders[h] + (i - h * turns - 1ll) * kLpThreads;
            if (u < v0 || u >= v1) continue;
            float x[kPer];
            r.load(u, x);
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                const long long j = r.index(u, e);
                const uint32_t xk = order_key(x[e]);
                if (xk >= tau && j >= 0 && j < r.vocab) {
                    const int at = atomicAdd(&count, 1);
                    if (at < kList) list[at] = rank_key(xk, static_cast<uint32_t>(j));
                }
            }
        }
        if (tid < kMaxK) best[tid] = 0;
        __syncthreads();
        const int n = count;
        if (n <= kList) {
            auto rank = [&](int j) {
                const unsigned long long me = list[j];
                int place = 0;
                for (int i = 0; i < n; ++i) place += list[i] > me;
                if (place < k) best[place] = me;
            };
            if (n <= kLpThreads) {  // nearly always; as one loop: one row of 131072 fp32 7.47 us instead of 7.40
                if (tid < n) rank(tid);
            } else {
#pragma unroll 1
                for (int j = tid; j < n; j += kLpThreads) rank(j);
            }
        } else {  // many equal values: one exact search per place
            unsigned long long last = ~0ull;
            for (int place = 0; place < k; ++place) {
                unsigned long long top = 0;
                for (long long u = v0 + tid; u < v1; u += kLpThreads) {
                    float x[kPer];
                    r.load(u, x);
#pragma unroll
                    for (int e = 0; e < kPer; ++e) {
                        const long long i = r.index(u, e);
                        if (i < 0 || i >= r.vocab) continue;
                        const unsigned long long c = rank_key(order_key(x[e]), static_cast<uint32_t>(i));
                        if (c < last && c > top) top = c;
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
                if (lane == 0) warp_best[warp] = top;
                __syncthreads();
                top = warp_best[0];
                for (int w = 1; w < kLpWarps; ++w) top = max(top, warp_best[w]);
                __syncthreads();
                if (tid == 0) best[place] = top;
                last = top;
            }
        }
    }

    // --- the row: every CTA puts its results in rank 0's shared memory, and rank 0 joins them
    __syncthreads();  // best is complete
    cluster_wait();   // rank 0 has started
    if (tid < k) *cluster.map_shared_rank(&joined[rank * k + tid], 0) = best[tid];
    if (warp == 1) {
        Sums c = lane < kLpWarps ? part[lane] : Sums{-INFINITY, 0.0f, 0.0f};
        c = join_lanes(c, lane, kLpWarps);
        if (lane == 0) *cluster.map_shared_rank(&parts[rank], 0) = c;
    }
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) {
        Sums c = lane < ranks ? parts[lane] : Sums{-INFINITY, 0.0f, 0.0f};
        c = join_lanes(c, lane, kMaxCluster);
        if (lane == 0) whole = c;
    }
    // k candidates at least are not below the lists' smallest ceil(k / ranks)-th entry, nor below a list's k-th
    if (warp == 1) {
        unsigned long long least = ~0ull, kth = 0;
        if (k > 0 && lane < ranks) {
            least = joined[lane * k + (k + ranks - 1) / ranks - 1];
            kth = joined[lane * k + k - 1];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            least = min(least, __shfl_xor_sync(~0u, least, o));
            kth = max(kth, __shfl_xor_sync(~0u, kth, o));
        }
        if (lane == 0) {
            floor_s = max(max(least, kth), 1ull);  // 0: no element
            count = 0;
        }
    }
    __syncthreads();
    const Sums c = whole;
    const float nan = __uint_as_float(0x7FC00000u);
    const bool none = !(fabsf(c.m) < INFINITY);  // no finite maximum: no distribution
    const float log_s = logf(c.s);
    if (tid == 0) {
        if (a.logprob != nullptr) {
            const long long tok = a.tokens[row];
            const bool ok = tok >= 0 && tok < a.vocab && !none;
            a.logprob[row] = ok ? (to_float(r.base[r.skip + tok]) - c.m) - log_s : nan;
        }
        if (a.entropy != nullptr) a.entropy[row] = none ? nan : log_s - c.w / c.s;
    }
    if (k == 0) return;
    for (int i = tid; i < ranks * k; i += kLpThreads)
        if (joined[i] >= floor_s) list[atomicAdd(&count, 1)] = joined[i];
    __syncthreads();
    for (int i = tid; i < count; i += kLpThreads) {
        const unsigned long long me = list[i];
        int place = 0;
        for (int j = 0; j < count; ++j) place += list[j] > me;
        if (place >= k) continue;
        const uint32_t id = 0xFFFFFFFFu - static_cast<uint32_t>(me);
        a.top_ids[row * k + place] = static_cast<int32_t>(id);
        a.top_logprobs[row * k + place] = none ? nan : (to_float(r.base[r.skip + id]) - c.m) - log_s;
    }
}

template <typename T>
cudaError_t launch_typed(const LogprobArgs& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may form clusters of 16
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    // CTAs per row: doubled while the launch has fewer than 5 CTAs per SM and each would keep two batches of loads per
    // thread. Up to 8 fit an SM, but a row's last steps are the same for any share of it: 128 rows of 200001 fp32 took
    // 29 us on clusters of 8 and 36 us on clusters of 16.
    const long long batch = static_cast<long long>(kLpThreads) * kBatch * 16 * 2;
    int ranks = 1;
    while (ranks < kMaxCluster && a.n_rows * ranks < 5ll * sms &&
           a.vocab * static_cast<long long>(sizeof(T)) > batch * ranks)
        ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows * ranks));
    cfg.blockDim = dim3(kLpThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, a);
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::kF32: return launch_typed<float>(a, stream);
        case DType::kF16: return launch_typed<__half>(a, stream);
        case DType::kBF16: return launch_typed<__nv_bfloat16>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
