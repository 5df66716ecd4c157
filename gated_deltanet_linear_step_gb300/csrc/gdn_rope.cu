// gdn_rope.cu - rotary positions of queries and keys.
//
//   (a, b) -> gain (a cos - b sin, a sin + b cos),  angle = position x frequency
//
// for the pairs (i, i + r/2) or (2 i, 2 i + 1) of a head's first r dims; the others are copied. The inverse turns by the
// negative angle (times the same gain): the transpose, which is what gradients need.
//
// Angles. A frequency comes as the fraction of a turn per position in 64-bit fixed point, so position x frequency modulo a
// whole turn is one integer multiplication whatever the position, exact but for the table's own rounding (2^-53 of a turn for each
// position); the angle is rounded to 2^-28 of a turn when it becomes a float. fp32 products of position and frequency would be off by a radian
// near position 2^24.
//
// What bounds it: HBM, every element read and written once. Persistent CTAs take tokens in turn. A token's rows (whole heads, up to kPiece
// bytes at a time) come by bulk copies into a ring of stages, turn in place and leave by bulk copies; the cosines and sines of the next token
// are computed beside them, once for all of its heads and layers. 16773 packed tokens of 40 heads of 128 in bf16: 58 us through the public call (56
// in a graph), 0.87 of the measured copy rate; 16004 tokens of 18 heads of 256, 96 dims turning, fp16: 49 us (47), 0.89. Plain loads and stores
// reached 71 and 82 us; a table of the pairs in their own order had four-way bank conflicts, 73 us.

#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_prompt.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 256;
// Stages, bytes of one, CTAs per SM. Against 4, 12288, 4, 16773 tokens of 40 heads of 128 in bf16 take 2 % longer with three stages, 15 % with
// three CTAs, 30 to 60 % with five (fewer registers).
constexpr int kStages = 4;
constexpr int kPiece = 12288;
constexpr int kCtas = 4;

__device__ unsigned int g_rope_error = 0;

struct RopeParams {
    RopeArgs a;
    int heads;     // of both sides
    int at_once;   // heads of a piece
    int pieces;    // of a token in a layer
    int n_tokens;  // B T
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float x) { return __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T x[V];
};

// Cosine and sine of a fraction of a turn, 2^-64 each unit. Its upper 32 bits count; of what is left within an eighth of a turn a float keeps 24 bits.
__device__ __forceinline__ void turn_cos_sin(uint64_t turn, float& c, float& s) {
    const int hi = static_cast<int>(turn >> 32);
    const int quarter = static_cast<int>((static_cast<uint32_t>(hi) + 0x20000000u) >> 30);
    const int rest = hi - static_cast<int>(static_cast<uint32_t>(quarter) << 30);  // within an eighth of a turn either way
    float s0, c0;
    sincospif(static_cast<float>(rest) * 4.656612873077393e-10f, &s0, &c0);       // 2^-31: in half turns
    c = quarter & 1 ? -s0 : c0;
    s = quarter & 1 ? c0 : s0;
    if (quarter & 2) c = -c, s = -s;
}

// Where a CTA is: piece `piece` of layer l of token t of sequence b; b < 0: at the end.
struct Walk {
    int token, b, t, l, piece;
};

// From `token` on the first that is to be turned, of every gridDim.x-th.
__device__ __forceinline__ void settle(const RopeParams& p, Walk& w) {
    for (;; w.token += gridDim.x) {
        if (w.token < 0 || w.token >= p.n_tokens) {
            w.b = -1;
            return;
        }
        w.b = static_cast<int>(static_cast<uint32_t>(w.token) / static_cast<uint32_t>(p.a.T));
        w.t = w.token - w.b * p.a.T;
        if (p.a.seq_len == nullptr || w.t < __ldg(p.a.seq_len + w.b)) return;
    }
}

// On to the next piece; true if it is of another token.
__device__ __forceinline__ bool advance(const RopeParams& p, Walk& w) {
    if (++w.piece < p.pieces) return false;
    w.piece = 0;
    if (++w.l < p.a.L) return false;
    w.l = 0;
    w.token = w.token > 0x7FFFFFFF - static_cast<int>(gridDim.x) ? -1 : w.token + static_cast<int>(gridDim.x);
    settle(p, w);
    return true;
}

// The parts of a piece: heads [lo, hi) of each side, and its row.
template <typename T, typename F>
__device__ __forceinline__ void each_side(const RopeParams& p, const Walk& w, F f) {
    const int first = w.piece * p.at_once, end = min(first + p.at_once, p.heads), nq = p.a.side[0].heads;
    const long long row = (static_cast<long long>(w.b) * p.a.L + w.l) * p.a.T + w.t;
    if (first < nq) f(p.a.side[0], row, first, min(end, nq), 0);
    if (end > nq) f(p.a.side[1], row, max(first, nq) - nq, end - nq, max(nq - first, 0));
}

template <typename T, int V, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads, kCtas) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ __align__(128) unsigned char sm[];
    __shared__ float2 table[2][kRopeThreads + 8];  // cosines and sines of this token and the next
    __shared__ __align__(8) uint64_t full_s[kStages];
    const RopeArgs& a = p.a;
    const int pairs = a.rotary_dim / 2, tid = threadIdx.x;
    const uint32_t full = smem_addr(full_s), stage0 = smem_addr(sm);
    const uint32_t piece_bytes = static_cast<uint32_t>(p.at_once) * a.head_dim * sizeof(T);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, 1);
        fence_mbar_init();
    }
    // a thread stays at its place of a head and steps through the heads; the table goes by the pairs' places within a thread's first, so that
    // neighbouring threads read neighbouring pairs
    constexpr int kPairs = INTERLEAVED ? V / 2 : V;
    const int chunks = (pairs + kPairs - 1) / kPairs, step = kRopeThreads / chunks;
    const int chunk = tid % chunks, head0 = tid / chunks;
    const uint64_t my_turns = tid < pairs ? __ldg(reinterpret_cast<const unsigned long long*>(a.turns) + tid) : 0;
    auto position = [&](const Walk& w) -> int {
        if (w.b < 0) return 0;
        return a.positions != nullptr ? __ldg(a.positions + w.token) : __ldg(a.start + w.b);
    };
    auto fill = [&](int buffer, const Walk& w, int pos) {
        if (tid >= pairs) return;
        float c, s;
        const long long at = static_cast<long long>(pos) + (a.positions != nullptr ? 0 : w.t);
        turn_cos_sin(static_cast<uint64_t>(at) * my_turns, c, s);
        table[buffer][tid % kPairs * chunks + tid / kPairs] = make_float2(c * a.gain, (a.flags & kRopeInverse ? -s : s) * a.gain);
    };
    // the pieces that are requested, by thread 0
    Walk ahead{static_cast<int>(blockIdx.x), 0, 0, 0, 0};
    settle(p, ahead);
    Walk w = ahead, next = ahead;  // the piece at hand, and the next token
    int issued = 0;
    auto request = [&]() {
        if (ahead.b < 0) return;
        const int s = issued % kStages;
        uint32_t bytes = 0;
        each_side<T>(p, ahead, [&](const RopeSide&, long long, int lo, int hi, int) { bytes += (hi - lo) * a.head_dim * sizeof(T); });
        mbar_arrive_expect_tx(full + 8 * s, bytes);
        each_side<T>(p, ahead, [&](const RopeSide& side, long long row, int lo, int hi, int at) {
            bulk_load(stage0 + s * piece_bytes + at * a.head_dim * sizeof(T),
                      static_cast<const T*>(side.in) + row * side.in_stride + static_cast<long long>(lo) * a.head_dim,
                      (hi - lo) * a.head_dim * sizeof(T), full + 8 * s);
        });
        ++issued;
        advance(p, ahead);
    };
    if (w.b < 0) return;
    int pos = position(next);
    if (tid == 0)
        for (int i = 0; i < kStages - 1; ++i) request();
    fill(0, next, pos);
    auto step_token = [&]() {
        next.token = next.token > 0x7FFFFFFF - static_cast<int>(gridDim.x) ? -1 : next.token + static_cast<int>(gridDim.x);
        settle(p, next);
        pos = position(next);
    };
    step_token();
    __syncthreads();

    bool bad = false;
    int n = 0, buffer = 0;
    for (bool fresh = true;; ++n) {
        const int s = n % kStages;
        bad = !mbar_wait_bounded(full + 8 * s, static_cast<uint32_t>(n / kStages) & 1u);
        const int heads = min(p.at_once, p.heads - w.piece * p.at_once);
        T* rows = reinterpret_cast<T*>(sm + s * piece_bytes);
        if (head0 < step && !bad) {
            for (int h = head0; h < heads; h += step) {
                T* x = rows + h * a.head_dim + chunk * V;
                if constexpr (INTERLEAVED) {
                    const float2* cs = table[buffer] + chunk;
                    Vec<T, V> v = *reinterpret_cast<Vec<T, V>*>(x);
#pragma unroll
                    for (int j = 0; j < V; j += 2) {
                        if (chunk * V + j >= a.rotary_dim) break;
                        const float y = to_float(v.x[j]), z = to_float(v.x[j + 1]);
                        const float2 f = cs[j / 2 * chunks];
                        v.x[j] = from_float<T>(fmaf(y, f.x, -(z * f.y)));
                        v.x[j + 1] = from_float<T>(fmaf(y, f.y, z * f.x));
                    }
                    *reinterpret_cast<Vec<T, V>*>(x) = v;
                } else {
                    const float2* cs = table[buffer] + chunk;
                    Vec<T, V> v = *reinterpret_cast<Vec<T, V>*>(x), u = *reinterpret_cast<Vec<T, V>*>(x + pairs);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float y = to_float(v.x[j]), z = to_float(u.x[j]);
                        const float2 f = cs[j * chunks];
                        v.x[j] = from_float<T>(fmaf(y, f.x, -(z * f.y)));
                        u.x[j] = from_float<T>(fmaf(y, f.y, z * f.x));
                    }
                    *reinterpret_cast<Vec<T, V>*>(x) = v;
                    *reinterpret_cast<Vec<T, V>*>(x + pairs) = u;
                }
            }
        }
        if (fresh && next.b >= 0) {  // the next token's
            fill(buffer ^ 1, next, pos);
            step_token();
        }
        fence_proxy_async_smem();
        if (__syncthreads_or(bad)) {
            bad = true;
            break;
        }
        if (tid == 0) {
            each_side<T>(p, w, [&](const RopeSide& side, long long row, int lo, int hi, int at) {
                bulk_store(static_cast<T*>(side.out) + row * side.out_stride + static_cast<long long>(lo) * a.head_dim,
                           stage0 + s * piece_bytes + at * a.head_dim * sizeof(T), (hi - lo) * a.head_dim * sizeof(T));
            });
            bulk_commit();
            bulk_wait_read_one();  // the stage before this one has left
            request();
        }
        fresh = advance(p, w);
        if (fresh) buffer ^= 1;
        if (w.b < 0) break;
    }
    if (tid == 0) {
        if (bad) {  // whatever is in flight lands before the CTA ends
            atomicOr(&g_rope_error, kErrWaitTimeout);
            for (int i = n; i < issued; ++i) (void)mbar_wait_bounded(full + 8 * (i % kStages), static_cast<uint32_t>(i / kStages) & 1u);
        }
        bulk_wait_all();
    }
}

template <typename T, int V, bool INTERLEAVED>
cudaError_t launch_one(const RopeArgs& a, cudaStream_t stream) {
    RopeParams p;
    p.a = a;
    p.heads = a.side[0].heads + a.side[1].heads;
    const int most = std::max<int>(kPiece / (a.head_dim * sizeof(T)), 1);
    p.pieces = (p.heads + most - 1) / most;
    p.at_once = (p.heads + p.pieces - 1) / p.pieces;
    p.n_tokens = a.B * a.T;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(rope_kernel<T, V, INTERLEAVED>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStages * kPiece);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    const size_t smem = static_cast<size_t>(kStages) * p.at_once * a.head_dim * sizeof(T);
    rope_kernel<T, V, INTERLEAVED><<<std::min(p.n_tokens, kCtas * sms), kRopeThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream) {
    constexpr int V = 16 / sizeof(T);
    if (a.flags & kRopeInterleaved) return launch_one<T, V, true>(a, stream);
    // the widest items that both halves begin at
    const int pairs = a.rotary_dim / 2;
    if (pairs % V == 0) return launch_one<T, V, false>(a, stream);
    if (pairs % (V / 2) == 0) return launch_one<T, V / 2, false>(a, stream);
    if (pairs % 2 == 0) return launch_one<T, 2, false>(a, stream);
    return launch_one<T, 1, false>(a, stream);
}

}  // namespace

cudaError_t read_rope_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_rope_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::kF32: return launch_type<float>(a, stream);
        case DType::kF16: return launch_type<__half>(a, stream);
        case DType::kBF16: return launch_type<__nv_bfloat16>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
