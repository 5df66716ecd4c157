// gdn_prompt.cu - causal attention over whole prompts: packed sequences of different lengths, grouped heads, on the 5th-generation
// tensor cores.
//
//   out_i = sum_{j <= i} p_j v_j / sum_{j <= i} p_j,  p_j = exp(scale q_i . k_j)
//
//   S = Q K^T   128 rows x kTok keys x D,   O += P V   128 rows x D x kTok keys
//
// in one pass over the keys with the running reference maximum and sum of a softmax. A row is a (token, query head) pair: a block of 128
// rows holds as many heads of one kv head's group as the largest power of two in the group's size (128 at most), of 128 / heads tokens: a tile of
// keys and values serves all of a group of 4 or 8, and one head of a group of 5. A unit is NB blocks of consecutive tokens; two blocks take
// turns on the tensor cores, one's softmax beside the other's products.
//
//   warp 0      finds the CTA's units and loads their tiles by TMA
//   warp 1      issues the products
//   warps 2, 3  look through the values of the tiles that not all rows see, see "What is masked"
//   4 NB warps  a row per thread: scores from tensor memory, maximum, exponentials, probabilities back over the scores (as the A operand of
//               the second product), at the end outputs
//
// Work. The units of all sequences are taken by falling length (that of block index l in its sequence goes by l), dealt out to the CTAs forth
// and back; each CTA goes through its own, the loads of the next unit beside the products of the last.
//
// What is masked. A causal row does not see later keys of its tile, nor does a unit's last tile end where its sequence does. Scores of such
// keys are set to -inf by a select, so whatever keys hold there does not matter; but 0 times a NaN or an infinite value would. So in the tiles that
// not every row of the unit sees, values that are not finite are set to 0 in shared memory, the keys of the sequence that had any are
// noted, and the rows that do see those add them to their outputs at the end.
//
// Numerics. Scores, maxima, sums and the accumulation are fp32. Probabilities are rounded to the inputs' 16-bit type (half a step as the
// outputs' own rounding), relative to 2^9 of the reference maximum, which is raised when a score exceeds it by kSlack (in base 2). fp32
// inputs are split by a kernel before into fp16 hi + lo (22 bits), scaled by powers of two to fill fp16's range (queries per row, keys and values
// per sequence and head; fp16's smallest step leaves 2^-40 of the largest), and so are their probabilities: three products each instead of one. The
// tensor cores cut a running sum off at every step instead of rounding it, so sums start afresh every 16384 keys (fp32: 256) and are added
// up with fp32 instructions in the workspace (fp32 outputs of 2500 normal tokens against 64 bits: 1.5e-6 of their size and 112 us with 512 keys, 1.1e-6 and
// 119 us with 256, 0.8e-6 and 139 us with 128).
//
// Waits are bounded. One that gives up makes its warp leave its loops; the others run into their own limits, the device error word is set,
// and the tensor memory is freed after the last product has completed.

#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_kv4_attention.cuh"
#include "gdn_prompt.cuh"
#include "gdn_tc_attention.cuh"

namespace gdn {
namespace {

constexpr int kRows = kMmaRows;
constexpr int kMaxSms = 192;     // the workspace is sized for cards of up to as many
constexpr int kRing = 4;         // units that are under way at most: one in each role's hands, and one found ahead
constexpr int kCheckWarps = 2;

__device__ unsigned int g_prompt_error = 0;

struct PromptParams {
    PromptArgs a;
    CUtensorMap q, k, v;
    float* sums;           // per CTA, of earlier runs of tiles: [dim / 4][row][4]
    const float* q_mul;    // fp32 calls: factor of a row's raw scores, but for the keys' own
    const uint32_t* most;  // fp32 calls: [sequence][kv head][2] bits of the largest finite key and value
    int heads, tokens;     // of a block: query heads, tokens
    int chunks;            // of a kv head's query heads
};

// A unit: rows first + token .. of a sequence of n, query heads head0 .., and the tiles of its blocks.
struct PromptUnit {
    int first, n, token, kv_head, head0, seq;
    int tiles[2];
};

template <typename T, int D>
struct Prompt {
    static constexpr bool kSplit = sizeof(T) == 4;
    static constexpr int kParts = kSplit ? 2 : 1;
    static constexpr int kBlocks = !kSplit && D <= 128 ? 2 : 1;      // tensor memory has room for two blocks' scores and sums at D <= 128
    static constexpr int kTok = kSplit ? (D == 64 ? 128 : D == 128 ? 64 : 32) : D == 256 ? 64 : 128;
    static constexpr int kStages = kSplit && D == 256 ? 1 : !kSplit && D == 64 ? 3 : 2;
    static constexpr int kBuffers = kBlocks == 2 ? 1 : 2;            // of a block's scores
    static constexpr int kSoftWarps = 4 * kBlocks;
    static constexpr int kThreads = 32 * (2 + kCheckWarps + kSoftWarps);
    static constexpr int kBlk = D / 64;                              // 64-dim blocks of a row (128 bytes)
    static constexpr uint32_t kQBlock = kRows * 128;
    static constexpr uint32_t kQPart = kBlk * kQBlock;               // of hi, then lo
    static constexpr uint32_t kQBytes = kParts * kQPart;             // of a block
    static constexpr uint32_t kKvBlock = kTok * 128;
    static constexpr uint32_t kKvPart = kBlk * kKvBlock;
    static constexpr uint32_t kKvBytes = kParts * kKvPart;
    static constexpr uint32_t kOffK = kBlocks * kQBytes;
    static constexpr uint32_t kOffV = kOffK + kStages * kKvBytes;
    static constexpr uint32_t kOffUnits = kOffV + kStages * kKvBytes;
    static constexpr int kMasked = (2 * kRows + kTok - 2) / kTok + 1;  // tiles of a unit that not all rows see
    static constexpr uint32_t kOffNote = kOffUnits + kRing * sizeof(PromptUnit);           // keys with values that are not finite
    static constexpr uint32_t kOffSome = kOffNote + kRing * kMasked * (kTok / 16) * 2;     // whether there are any, per check warp
    static constexpr uint32_t kOffBar = (kOffSome + kRing * kCheckWarps * 4 + 7) / 8 * 8;
    static constexpr uint32_t kBars = 2 * kRing + 2 * kBlocks + 5 * kStages + 4 * kBlocks * kBuffers + 2;
    static constexpr uint32_t kOffOut = (kOffBar + kBars * 8 + 16 + 15) / 16 * 16;  // per softmax warp: 128 bytes of each of its rows
    static constexpr uint32_t kUsed = kOffOut + kSoftWarps * 32 * 128;
    static constexpr uint32_t kLeast = 118 * 1024;                   // one CTA per SM: the tensor memory is its own
    static constexpr uint32_t kSmem = kUsed + 1024 > kLeast ? kUsed + 1024 : kLeast;
    static constexpr int kFreshTiles = (kSplit ? 256 : 16384) / kTok;
    // Tensor memory. One block: its scores in two buffers in turn, the probabilities over the scores they came from, then the sums. Two
    // blocks: [first block's probabilities | scores of either | second block's probabilities | sums of both]. A block's scores are in
    // registers long before its probabilities are ready, so the other block's next scores can take their place, and no product waits for
    // another one to complete (with scores and probabilities of each block in one place it has to: 16384 tokens of 32 heads take 6 % longer).
    static constexpr uint32_t kTmO = 256;
    __host__ __device__ static constexpr uint32_t tm_scores(int t) { return kBlocks == 2 ? 64 : kTok * (t % kBuffers); }
    __host__ __device__ static constexpr uint32_t tm_probs(int block, int t) { return kBlocks == 2 ? 192 * block : kTok * (t % kBuffers); }
    static_assert((kBlocks == 1 ? kBuffers * kTok <= 256 : kTok == 128 && !kSplit) && kTmO + kBlocks * D <= 512, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
};

constexpr uint32_t kTmCols = 512;

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* tm, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// --------------------------------------------------------------- the units --
// By one warp. Blocks of sequences b = lane + 32 i are kept in registers for i < kKept.
constexpr int kKept = 4;

struct Finder {
    int kept[kKept];
    int total;   // units of a kv head and a chunk
    int levels;  // of the sequence with the most
};

__device__ __forceinline__ int blocks_of(const PromptArgs& a, int b, int tokens) {
    return b < a.B ? (prompt_rows(a, b).n + tokens - 1) / tokens : 0;
}

// Units of block index `level` or more.
__device__ __forceinline__ int units_from(const PromptArgs& a, const Finder& f, int level, int tokens, int lane) {
    int s = 0;
#pragma unroll
    for (int i = 0; i < kKept; ++i) s += max(f.kept[i] - level, 0);
    for (int b = lane + 32 * kKept; b < a.B; b += 32) s += max(blocks_of(a, b, tokens) - level, 0);
    return __reduce_add_sync(~0u, s);
}

__device__ __forceinline__ Finder find_all(const PromptArgs& a, int tokens, int lane) {
    Finder f;
    int most = 0;
    bool fall = false;  // borders that fall could make any number of sequences of the same rows: none has units then
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
        f.kept[i] = blocks_of(a, lane + 32 * i, tokens);
        most = max(most, f.kept[i]);
        fall = fall || (lane + 32 * i < a.B && prompt_rows_fall(a, lane + 32 * i));
    }
    for (int b = lane + 32 * kKept; b < a.B; b += 32) {
        most = max(most, blocks_of(a, b, tokens));
        fall = fall || prompt_rows_fall(a, b);
    }
    f.levels = __reduce_max_sync(~0u, most);
    f.total = __any_sync(~0u, fall) ? 0 : units_from(a, f, 0, tokens, lane);
    return f;
}

// Where the search for a CTA's units has come to, by falling block index and rising sequence: the units asked for rise, so it goes on from there.
// (Started afresh for each unit it took longer than the units: 4096 prompts of 1 to 4 tokens 3750 us, now 980.)
struct Search {
    int level;   // block index
    int above;   // units of larger ones
    int upto;    // and of this one
    int b0;      // sequences below it ..
    int before;  // .. have so many units of this block index
};

// Sequence of the x-th unit, whose block index is then s.level.
__device__ __forceinline__ int find_unit(const PromptArgs& a, const Finder& f, int x, int tokens, int lane, Search& s) {
    if (x >= s.upto) {
        int hi = s.level, above = s.upto, step = 1, lo, upto;  // above: units_from(hi)
        for (;; step *= 2) {
            lo = max(hi - step, 0);
            upto = units_from(a, f, lo, tokens, lane);
            if (upto > x || lo == 0) break;
            hi = lo;
            above = upto;
        }
        while (hi - lo > 1) {  // units_from(lo) > x >= units_from(hi)
            const int mid = (lo + hi) >> 1, n = units_from(a, f, mid, tokens, lane);
            if (n > x) {
                lo = mid;
                upto = n;
            } else {
                hi = mid;
                above = n;
            }
        }
        s = Search{lo, above, upto, 0, 0};
    }
    int rank = x - s.above - s.before;
    for (; s.b0 < a.B; s.b0 += 32) {
        const int b0 = s.b0;
        int mine = f.kept[0];
        if (b0 > 0) {
            mine = 0;
#pragma unroll
            for (int i = 1; i < kKept; ++i)
                if (b0 == 32 * i) mine = f.kept[i];
            if (b0 >= 32 * kKept) mine = blocks_of(a, b0 + lane, tokens);
        }
        unsigned hit = __ballot_sync(~0u, mine > s.level);
        const int count = __popc(hit);
        if (rank >= count) {
            rank -= count;
            s.before += count;
            continue;
        }
        for (; rank > 0; --rank) hit &= hit - 1;
        return b0 + __ffs(hit) - 1;
    }
    return 0;
}

// ------------------------------------------------------------------ pieces --
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (sizeof(T) == 2 && !__is_same(T, __half)) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    } else {
        return pack_half2(a, b);
    }
}

template <typename T>
__device__ __forceinline__ float value_of(T x) {
    if constexpr (sizeof(T) == 4) return x;
    else return static_cast<float>(x);
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// 2^(14 - exponent of the largest magnitude): scaled by it values fill fp16's range, exactly.
__device__ __forceinline__ float fill_factor(uint32_t most) {
    const int e = max(static_cast<int>(most >> 23) - 127, -112);
    return most > 0 ? __uint_as_float(static_cast<uint32_t>(141 - e) << 23) : 1.0f;
}

// Two blocks: the 12 warps start with 168 registers each; the first four give up 64 for the softmax warps' 32 more (384 x 168 = 128 x 104 +
// 256 x 200), which then hold a row's 128 scores without spills (without that 16384 tokens of 32 heads take 14 % longer).
template <int BLOCKS, bool MORE>
__device__ __forceinline__ void take_registers() {
    if constexpr (BLOCKS == 2) {
        if constexpr (MORE) asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    }
}

// 16 bytes of a row as floats.
template <typename T>
__device__ __forceinline__ void read16(const T* p, float (&x)[16 / sizeof(T)]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const T* v = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x[i] = value_of(v[i]);
}

// The outputs of the rows in `rows` (a lane's row: token `last` of the sequence whose rows begin at `first`, and a query head of kv_head), by a warp, eight rows
// at a time, in two passes over their keys: for rows with a reference maximum that is big, see kBig. Where every row of a call is, that takes 340 ms instead of 1.3
// for 16384 tokens of 32 heads of 128 in bf16 (row by row 1340). (Raising such maxima with a factor that changes, as the kernels over the cache do, took 2 to 4 % of every call.)
template <typename T, int D>
__device__ __noinline__ void big_rows(const PromptArgs& a, unsigned rows, int first, int kv_head, int last, int head, int lane) {
    constexpr int V = 16 / sizeof(T), kMine = D / 32, kAtOnce = 8, kKeys = 4;
    const T* k = static_cast<const T*>(a.k) + static_cast<long long>(first) * a.k_stride + static_cast<long long>(kv_head) * D;
    const T* v = static_cast<const T*>(a.v) + static_cast<long long>(first) * a.v_stride + static_cast<long long>(kv_head) * D + kMine * lane;
    const float scale = a.scale;
    while (rows != 0) {
        const T* q[kAtOnce];
        int ends[kAtOnce], at[kAtOnce], end = -1;  // the rows' last keys (-1: no row), their lanes, the largest of the former
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
            at[r] = rows != 0 ? __ffs(rows) - 1 : 0;
            ends[r] = __shfl_sync(~0u, last, at[r]);
            q[r] = static_cast<const T*>(a.q) + (static_cast<long long>(first) + max(ends[r], 0)) * a.q_stride + static_cast<long long>(__shfl_sync(~0u, head, at[r])) * D;
            if (rows == 0) ends[r] = -1;
            end = max(end, ends[r]);
            rows &= rows - 1;
        }
        auto scores = [&](int key, float (&s)[kAtOnce]) {
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) s[r] = 0.0f;
            const T* row = k + min(key, end) * a.k_stride;
#pragma unroll 1
            for (int c = 0; c < D; c += V) {
                float y[V];
                read16(row + c, y);
#pragma unroll
                for (int r = 0; r < kAtOnce; ++r) {
                    float x[V];
                    read16(q[r] + c, x);
#pragma unroll
                    for (int i = 0; i < V; ++i) s[r] = fmaf(x[i], y[i], s[r]);
                }
            }
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) s[r] = key <= ends[r] ? s[r] : -INFINITY;
        };
        float s[kAtOnce], top[kAtOnce], l[kAtOnce], o[kAtOnce][kMine];
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
            top[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < kMine; ++i) o[r][i] = 0.0f;
        }
#pragma unroll 1
        for (int key = 0; key <= end; key += 32) {
            scores(key + lane, s);
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) top[r] = fmaxf(top[r], s[r]);
        }
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r)
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(~0u, top[r], i));
#pragma unroll 1
        for (int key = 0; key <= end; key += 32) {
            scores(key + lane, s);
#pragma unroll
            for (int r = 0; r < kAtOnce; ++r) {
                s[r] = key + lane <= ends[r] ? exp2_approx((s[r] - top[r]) * scale * 1.4426950408889634f) : 0.0f;
                l[r] += s[r];
            }
#pragma unroll 1
            for (int j0 = 0; j0 < 32 && key + j0 <= end; j0 += kKeys) {
                float y[kKeys][kMine];
#pragma unroll
                for (int j = 0; j < kKeys; ++j)
#pragma unroll
                    for (int i = 0; i < kMine; ++i) y[j][i] = value_of(v[min(key + j0 + j, end) * a.v_stride + i]);
#pragma unroll
                for (int r = 0; r < kAtOnce; ++r)
#pragma unroll
                    for (int j = 0; j < kKeys; ++j) {
                        const float f = __shfl_sync(~0u, s[r], j0 + j);
                        if (key + j0 + j > ends[r]) continue;
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            o[r][i] = finite(y[j][i]) ? fmaf(f, y[j][i], o[r][i]) : o[r][i] + y[j][i];  // (0 times infinity, where a probability is too small)
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < kAtOnce; ++r) {
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) l[r] += __shfl_xor_sync(~0u, l[r], i);
            if (ends[r] < 0) continue;
            T* out = static_cast<T*>(a.out) + (static_cast<long long>(first) + ends[r]) * a.out_stride + static_cast<long long>(__shfl_sync(~0u, head, at[r])) * D + kMine * lane;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                if constexpr (sizeof(T) == 4) out[i] = o[r][i] / l[r];
                else if constexpr (__is_same(T, __half)) out[i] = __float2half_rn(o[r][i] / l[r]);
                else out[i] = __float2bfloat16_rn(o[r][i] / l[r]);
            }
        }
    }
}

// ------------------------------------------------------------------ kernel --
template <typename T, int D>
__global__ void __launch_bounds__(Prompt<T, D>::kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    using W = Prompt<T, D>;
    constexpr int kTok = W::kTok, kStages = W::kStages, kBlocks = W::kBlocks, kBuffers = W::kBuffers;
    constexpr bool kHalves = kTok >= 64;  // a tile's product with the values begins when half of the probabilities are there
    constexpr bool kSplit = W::kSplit, kBf16 = !kSplit && !__is_same(T, __half);
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sm = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    PromptUnit* units = reinterpret_cast<PromptUnit*>(sm + W::kOffUnits);
    uint16_t* note = reinterpret_cast<uint16_t*>(sm + W::kOffNote);
    volatile uint32_t* some_noted = reinterpret_cast<volatile uint32_t*>(sm + W::kOffSome);
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(sm + W::kOffBar + W::kBars * 8);
    const uint32_t unit_full = base + W::kOffBar, unit_free = unit_full + 8 * kRing;
    const uint32_t q_full = unit_free + 8 * kRing, q_free = q_full + 8 * kBlocks;  // per block
    const uint32_t k_full = q_free + 8 * kBlocks, v_full = k_full + 8 * kStages, v_ok = v_full + 8 * kStages, k_free = v_ok + 8 * kStages,
                   v_free = k_free + 8 * kStages;
    // per block and buffer: a softmax warp may be done with a tile before the product of the tile before it has completed
    const uint32_t s_done = v_free + 8 * kStages, p_ready = s_done + 8 * kBlocks * kBuffers;
    const uint32_t p_rest = p_ready + 8 * kBlocks * kBuffers;  // (probabilities of the first half of a tile, and of the others)
    const uint32_t o_done = p_rest + 8 * kBlocks * kBuffers, s_free = o_done + 8 * kBlocks * kBuffers, drained = s_free + 8;
    // where and in which phase the block's tile t is
    auto place = [](int block, int t) -> uint32_t { return 8u * static_cast<uint32_t>(kBuffers * block + t % kBuffers); };
    auto phase = [](int t) -> uint32_t { return static_cast<uint32_t>(t / kBuffers) & 1u; };

    if (warp == 0) {
        if (lane == 0) {
            for (int i = 0; i < kRing; ++i) {
                mbar_init(unit_full + 8 * i, 1);
                mbar_init(unit_free + 8 * i, 1 + kCheckWarps + W::kSoftWarps);
            }
            for (int i = 0; i < kBlocks; ++i) {
                mbar_init(q_full + 8 * i, 1);
                mbar_init(q_free + 8 * i, 1);
            }
            for (int i = 0; i < kStages; ++i) {
                mbar_init(k_full + 8 * i, 1);
                mbar_init(v_full + 8 * i, 1);
                mbar_init(v_ok + 8 * i, kCheckWarps);
                mbar_init(k_free + 8 * i, 1);
                mbar_init(v_free + 8 * i, 1);
            }
            for (int i = 0; i < kBlocks * kBuffers; ++i) {
                mbar_init(s_done + 8 * i, 1);
                mbar_init(p_ready + 8 * i, 4);
                mbar_init(p_rest + 8 * i, 4);
                mbar_init(o_done + 8 * i, 1);
            }
            mbar_init(s_free, 4);  // (two blocks: the scores have been read)
            mbar_init(drained, 1);
            fence_mbar_init();
        }
    } else if (warp == 1) {
        tmem_alloc(smem_addr(tmem_s), kTmCols);
    }
    if (blockIdx.x == 0)
        for (int b = tid; b < p.a.B; b += W::kThreads)
            if (prompt_borders_bad(p.a, b)) atomicOr(&g_prompt_error, kErrBadBorders);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if constexpr (kSplit) griddep_wait();  // for the inputs' parts: the kernel is launched while they are made
    const uint32_t tmem = *tmem_s;
    bool failed = false;
    // the u-th unit of this CTA, by a warp or (products) by one lane; false at the end, or when the wait gave up
    auto take = [&](int u, PromptUnit& x, bool alone) -> bool {
        const uint32_t bar = unit_full + 8 * (u % kRing), parity = static_cast<uint32_t>(u / kRing) & 1u;
        if (!(alone ? wait_for(bar, parity) : warp_wait(bar, parity))) {
            failed = true;
            return false;
        }
        x = units[u % kRing];
        return x.n > 0;
    };

    if (warp < 2 + kCheckWarps) {
        take_registers<kBlocks, false>();  // (the warps of a warpgroup execute one and the same instruction)
        if (warp == 0) {
            // ------------------------------------------------------------- loads
            const int step = kBlocks * p.tokens;
            const Finder f = find_all(p.a, step, lane);
            Search search{f.levels, 0, 0, 0, 0};
            const int pairs = p.a.kv_heads * p.chunks;
            const long long total = static_cast<long long>(f.total) * pairs;
            int n = 0, u = 0, k_issued = 0, v_issued = 0, q_issued[2] = {0, 0};  // tiles, units; loads, as the elected lane counts them
            auto load_tile = [&](uint32_t at, const CUtensorMap* map, uint32_t full, int head, int row) {
                mbar_arrive_expect_tx(full, W::kKvBytes);
#pragma unroll
                for (int c = 0; c < W::kParts * W::kBlk; ++c) tma_load(at + c * W::kKvBlock, map, 64 * c, head, row, full);
            };
            auto look = [&](int i) -> PromptUnit {  // the i-th unit of this CTA
                PromptUnit x{};
                const long long at = static_cast<long long>(i) * gridDim.x + ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                if (at >= total) return x;
                const int index = static_cast<int>(at / pairs), pair = static_cast<int>(at - static_cast<long long>(index) * pairs);
                x.seq = find_unit(p.a, f, index, step, lane, search);
                const PromptRows r = prompt_rows(p.a, x.seq);
                x.first = r.first;
                x.n = r.n;
                x.token = search.level * step;
                x.kv_head = pair / p.chunks;
                x.head0 = x.kv_head * (p.a.q_heads / p.a.kv_heads) + (pair - x.kv_head * p.chunks) * p.heads;
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    const int t0 = x.token + b * p.tokens;
                    x.tiles[b] = b < kBlocks && t0 < x.n ? (min(x.n, t0 + p.tokens) + kTok - 1) / kTok : 0;
                }
                return x;
            };
            const bool elected = elect_one();  // the same lane throughout: it counts
            PromptUnit next = look(0);
            for (;; ++u) {
                const PromptUnit x = next;
                if (u >= kRing && !warp_wait(unit_free + 8 * (u % kRing), static_cast<uint32_t>(u / kRing - 1) & 1u)) {
                    failed = true;
                    break;
                }
                if (lane == 0) {
                    units[u % kRing] = x;
                    mbar_arrive_local(unit_full + 8 * (u % kRing));
                }
                if (x.n == 0) break;
                const int tiles = max(x.tiles[0], x.tiles[1]);
                bool ok = true;
                auto load_k = [&](int t, int j) -> bool {
                    const int s = t % kStages;
                    if (t >= kStages && !wait_for(k_free + 8 * s, static_cast<uint32_t>(t / kStages - 1) & 1u)) return false;
                    load_tile(base + W::kOffK + s * W::kKvBytes, &p.k, k_full + 8 * s, x.kv_head, x.first + j * kTok);
                    ++k_issued;
                    return true;
                };
                auto load_v = [&](int t, int j) -> bool {
                    const int s = t % kStages;
                    if (t >= kStages && !wait_for(v_free + 8 * s, static_cast<uint32_t>(t / kStages - 1) & 1u)) return false;
                    load_tile(base + W::kOffV + s * W::kKvBytes, &p.v, v_full + 8 * s, x.kv_head, x.first + j * kTok);
                    ++v_issued;
                    return true;
                };
                auto load_q = [&](int b) -> bool {  // (a block's place is free once its last scores of the unit before are done)
                    if (x.tiles[b] == 0) return true;
                    if (q_issued[b] > 0 && !wait_for(q_free + 8 * b, static_cast<uint32_t>(q_issued[b] - 1) & 1u)) return false;
                    mbar_arrive_expect_tx(q_full + 8 * b, static_cast<uint32_t>(W::kParts * W::kBlk * p.heads * p.tokens * 128));
#pragma unroll
                    for (int c = 0; c < W::kParts * W::kBlk; ++c)
                        tma_load(base + b * W::kQBytes + c * W::kQBlock, &p.q, 64 * c, x.head0, x.first + x.token + b * p.tokens, q_full + 8 * b);
                    ++q_issued[b];
                    return true;
                };
                // in the order in which their places become free; the next unit is looked up once this one's first loads are under way
                if (elected) ok = load_k(n, 0) && load_q(0) && load_v(n, 0) && (kBlocks == 1 || load_q(1));
                __syncwarp();
                next = look(u + 1);
                if (elected) {
                    for (int j = 1; j < tiles && ok; ++j) ok = load_k(n + j, j) && load_v(n + j, j);
                }
                __syncwarp();
                n += tiles;
                if (__any_sync(~0u, !ok)) {
                    failed = true;
                    break;
                }
            }
            k_issued = __reduce_max_sync(~0u, k_issued);
            v_issued = __reduce_max_sync(~0u, v_issued);
            // whatever is in flight has landed before the CTA ends
            for (int s = 0; s < kStages; ++s) {
                const int k = (k_issued - s + kStages - 1) / kStages, v = (v_issued - s + kStages - 1) / kStages;  // of this stage
                if (k > 0) (void)warp_wait(k_full + 8 * s, static_cast<uint32_t>(k - 1) & 1u);
                if (v > 0) (void)warp_wait(v_full + 8 * s, static_cast<uint32_t>(v - 1) & 1u);
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int q = __reduce_max_sync(~0u, q_issued[b]);
                if (q > 0) (void)warp_wait(q_full + 8 * b, static_cast<uint32_t>(q - 1) & 1u);
            }
        } else if (warp == 1) {
            // (its waits poll: the hardware wakes a suspended thread later, 16384 tokens of 32 heads took 1.4 % longer)
            // ---------------------------------------------------------- products
            if (elect_one()) {
                const uint32_t type = kBf16 ? (1u << 7) | (1u << 10) : 0u;
                const uint32_t idesc_s = idesc_f16(kTok) | type, idesc_o = idesc_f16(D) | type | kIdescBMnMajor;
                const uint32_t q_desc = desc_k(base), k_desc = desc_k(base + W::kOffK), v_desc = desc_mn(base + W::kOffV, W::kKvBlock);
                int n = 0;                  // tiles so far
                int m[kBlocks] = {};        // tiles of each block ...
                int scored = 0;             // ... and of both
                int queries[kBlocks] = {};  // units of each block
                // S = Q K of block i, the CTA's tile t
                auto first = [&](int i, int t) -> bool {
                    if constexpr (kBlocks == 2) {
                        if (scored > 0 && !mbar_wait_bounded(s_free, static_cast<uint32_t>(scored - 1) & 1u)) return false;
                        ++scored;
                    } else {  // the buffer's last reader
                        if (m[i] >= kBuffers && !mbar_wait_bounded(o_done + place(i, m[i]), phase(m[i] - kBuffers))) return false;
                    }
                    tc_fence_after();
                    const uint32_t k = k_desc + (t % kStages) * (W::kKvBytes >> 4), q = q_desc + i * (W::kQBytes >> 4);
                    const uint32_t d = tmem + W::tm_scores(m[i]);
                    // the products of the rests come first, so that half of what the tensor cores cut off is of small numbers
#pragma unroll
                    for (int part = kSplit ? 0 : 2; part < 3; ++part) {
                        const uint32_t qp = q + (part == 0 ? W::kQPart >> 4 : 0), kp = k + (part == 1 ? W::kKvPart >> 4 : 0);
#pragma unroll
                        for (int c = 0; c < 4 * W::kBlk; ++c) {
                            const uint32_t ko = kp + (c >> 2) * (W::kKvBlock >> 4) + 2 * (c & 3), qo = qp + (c >> 2) * (W::kQBlock >> 4) + 2 * (c & 3);
                            if (c == 0 && part == (kSplit ? 0 : 2))
                                mma_ss<true>(d, qo, ko, idesc_s);
                            else
                                mma_ss<false>(d, qo, ko, idesc_s);
                        }
                    }
                    mma_commit(s_done + place(i, m[i]));
                    ++m[i];
                    return true;
                };
                // O += P V of block i, the CTA's tile t, the block's tile before its last score product (or that one's own)
                auto second = [&](int i, int t, int mine, bool fresh) -> bool {
                    if (!mbar_wait_bounded(v_ok + 8 * (t % kStages), static_cast<uint32_t>(t / kStages) & 1u)) return false;
                    if (!mbar_wait_bounded(p_ready + place(i, mine), phase(mine))) return false;
                    tc_fence_after();
                    const uint32_t v = v_desc + (t % kStages) * (W::kKvBytes >> 4), d = tmem + W::kTmO + i * D;
                    const uint32_t pr = tmem + W::tm_probs(i, mine);
#pragma unroll
                    for (int c = 0; c < kTok / 16; ++c) {
                        if (kHalves && c == kTok / 32) {
                            if (!mbar_wait_bounded(p_rest + place(i, mine), phase(mine))) return false;
                            tc_fence_after();
                        }
                        const uint32_t vo = v + c * (2048 >> 4);
                        if constexpr (kSplit) {  // 32 keys' probabilities from the first of their 32 columns, their rests from the 16th
                            const uint32_t pc = pr + 32 * (c >> 1) + 8 * (c & 1);
                            mma_ts(d, pc + 16, vo, idesc_o, fresh && c == 0 ? 0u : 1u);
                            mma_ts(d, pc, vo + (W::kKvPart >> 4), idesc_o, 1u);
                            mma_ts(d, pc, vo, idesc_o, 1u);
                        } else {
                            mma_ts(d, pr + 8 * c, vo, idesc_o, fresh && c == 0 ? 0u : 1u);
                        }
                    }
                    mma_commit(o_done + place(i, mine));
                    return true;
                };
                // Tile by tile over all units: a block's product with the values of the tile before, then its scores; so a unit's first scores are
                // under way while the last tile of the unit before is in the softmax. (One block with two buffers: scores first, but for a unit's first
                // tile, whose queries come late.)
                bool open[kBlocks] = {}, fresh[kBlocks] = {};  // the block's tile before awaits its product with the values; the product starts its sums
                auto close = [&](int i, int t, int mine) -> bool {
                    if (!open[i]) return true;
                    open[i] = false;
                    return second(i, t, mine, fresh[i]);
                };
                PromptUnit x;
                for (int u = 0; !failed && take(u, x, true); ++u) {
                    mbar_arrive_local(unit_free + 8 * (u % kRing));
                    const int tiles = max(x.tiles[0], x.tiles[1]);
                    for (int j = 0; j < tiles && !failed; ++j, ++n) {
                        if (!mbar_wait_bounded(k_full + 8 * (n % kStages), static_cast<uint32_t>(n / kStages) & 1u)) {
                            failed = true;
                            break;
                        }
#pragma unroll
                        for (int i = 0; i < kBlocks; ++i) {
                            const bool scores = j < x.tiles[i], ahead = kBuffers == 2 && j > 0;
                            bool ok = ahead || close(i, n - 1, m[i] - 1);
                            if (scores) {
                                ok = ok && (j > 0 || mbar_wait_bounded(q_full + 8 * i, static_cast<uint32_t>(queries[i]++) & 1u)) && first(i, n);
                                if (ok && j == x.tiles[i] - 1) mma_commit(q_free + 8 * i);
                            }
                            if (ok && i == kBlocks - 1) mma_commit(k_free + 8 * (n % kStages));
                            ok = ok && (!ahead || close(i, n - 1, m[i] - (scores ? 2 : 1)));
                            if (ok && i == kBlocks - 1 && n > 0) mma_commit(v_free + 8 * ((n - 1) % kStages));
                            open[i] = scores;
                            fresh[i] = j % W::kFreshTiles == 0;
                            if (!ok) {
                                failed = true;
                                break;
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
                    if (!failed && !close(i, n - 1, m[i] - 1)) failed = true;
                // whatever was issued has completed before the tensor memory is freed
                mma_commit(drained);
                (void)mbar_wait_bounded(drained, 0);
            }
        } else {
            // ----------------------------------------------------- masked values
            constexpr int kMine = kTok / kCheckWarps;  // keys of a tile that this warp looks at
            constexpr uint32_t kExponent = kBf16 ? 0x7F80u : 0x7C00u;
            const int me = warp - 2;
            int n = 0;
            PromptUnit x;
            for (int u = 0; !failed && take(u, x, false); ++u) {
                const int slot = u % kRing, tiles = max(x.tiles[0], x.tiles[1]), whole = (x.token + 1) / kTok;  // tiles that every row sees
                bool any = false;
                for (int j = 0; j < tiles; ++j, ++n) {
                    const int s = n % kStages;
                    if (!warp_wait(v_full + 8 * s, static_cast<uint32_t>(n / kStages) & 1u)) {
                        failed = true;
                        break;
                    }
                    if (j >= whole) {
                        unsigned char* tile = sm + W::kOffV + s * W::kKvBytes;
#pragma unroll
                        for (int r0 = 0; r0 < kMine; r0 += 32) {
                            const int row = me * kMine + r0 + lane;
                            uint32_t most = 0;
                            if (kMine >= 32 || lane < kMine) {
#pragma unroll
                                for (int c = 0; c < 8 * W::kBlk; ++c) {
                                    const uint4 w = *reinterpret_cast<const uint4*>(tile + (c >> 3) * W::kKvBlock + row * 128 + (((c & 7) ^ (lane & 7)) << 4));
                                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu)));
                                }
                            }
                            const bool bad = (most & 0xFFFFu) >= kExponent || (most >> 16) >= kExponent;
                            if (bad) {
#pragma unroll 1
                                for (int c = 0; c < 32 * W::kBlk; ++c) {  // pairs of 16-bit values of the row
                                    uint32_t* at = reinterpret_cast<uint32_t*>(tile + (c >> 5) * W::kKvBlock + row * 128) + (c & 31);
                                    uint32_t w = *at;
                                    if ((w & kExponent) == kExponent) w &= 0xFFFF0000u;
                                    if ((w >> 16 & kExponent) == kExponent) w &= 0x0000FFFFu;
                                    *at = w;
                                }
                            }
                            const unsigned keys = __ballot_sync(~0u, bad && j * kTok + row < x.n);
                            any = any || keys != 0;
                            if (lane == 0) {
                                uint16_t* to = note + (slot * W::kMasked + (j - whole)) * (kTok / 16) + (me * kMine + r0) / 16;
                                to[0] = static_cast<uint16_t>(keys);
                                if (kMine >= 32) to[1] = static_cast<uint16_t>(keys >> 16);
                            }
                        }
                        fence_proxy_async_smem();
                    }
                    if ((j == 0 || j >= whole) && lane == 0) some_noted[slot * kCheckWarps + me] = any ? 1u : 0u;  // (the first block may end before this unit)
                    __syncwarp();
                    if (lane == 0) mbar_arrive_local(v_ok + 8 * s);
                }
                if (lane == 0) mbar_arrive_local(unit_free + 8 * slot);
            }
        }
    } else {
        take_registers<kBlocks, true>();
        // -------------------------------------------------------------- rows
        const int block = (warp - 2 - kCheckWarps) >> 2, quarter = warp & 3;  // (a warp reaches lanes 32 (warp mod 4) ..)
        const int row = 32 * quarter + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t o_at = lanes + W::kTmO + block * D;
        const int row_token = row / p.heads, row_head = row - row_token * p.heads;
        int m_tiles = 0;  // of this block so far
        PromptUnit x;
        for (int u = 0; !failed && take(u, x, false); ++u) {
            const int tiles = x.tiles[block], token = x.token + block * p.tokens;
            const bool valid = token + row_token < x.n;
            const bool some = __any_sync(~0u, valid);
            const int lim = valid ? token + row_token : -1;
            const long long out_row = static_cast<long long>(x.first) + lim;
            float mul = p.a.scale * 1.4426950408889634f, unscale = 1.0f;
            if constexpr (kSplit) {
                const uint32_t* most = p.most + (static_cast<size_t>(x.seq) * p.a.kv_heads + x.kv_head) * 2;
                mul = valid ? p.q_mul[out_row * p.a.q_heads + x.head0 + row_head] / fill_factor(most[0]) : 0.0f;
                unscale = 1.0f / fill_factor(most[1]);
            }
            mul = fmaxf(mul, kLeastScale);
            float m = -INFINITY, shift = kNone, l = 0.0f, sum_m = -INFINITY, worst = 0.0f;  // the largest size of m
            auto four_sums = [&](int c) -> float4& {  // of dims c .. c + 3
                return *reinterpret_cast<float4*>(p.sums + static_cast<size_t>(blockIdx.x) * D * (kBlocks * kRows) + c * (kBlocks * kRows) + 4 * (block * kRows + row));
            };
            // the sums in tensor memory and the earlier ones
            auto with_earlier = [&](int c, auto& o, float f) {
#pragma unroll
                for (int i = 0; i < static_cast<int>(sizeof(o) / 4); i += 4) {
                    const float4 y = four_sums(c + i);
                    o[i] = fmaf(y.x, f, o[i]), o[i + 1] = fmaf(y.y, f, o[i + 1]);
                    o[i + 2] = fmaf(y.z, f, o[i + 2]), o[i + 3] = fmaf(y.w, f, o[i + 3]);
                }
            };
            for (int r = 0; r < tiles && !failed; ++r, ++m_tiles) {
                if (!warp_wait(s_done + place(block, m_tiles), phase(m_tiles))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (some) {
                    const uint32_t p_at = lanes + W::tm_probs(block, m_tiles);
                    float s[kTok];
                    tmem_read(lanes + W::tm_scores(m_tiles), s);
                    if constexpr (kBlocks == 2) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_local(s_free);
                    }
                    if ((r + 1) * kTok > token + 1) {
                        const int seen = lim - r * kTok;
#pragma unroll
                        for (int i = 0; i < kTok; ++i) s[i] = i <= seen ? s[i] : -INFINITY;
                    }
                    float t0 = max3(s[0], s[1], s[2]), t1 = max3(s[3], s[4], s[5]), t2 = max3(s[6], s[7], s[8]), t3 = max3(s[9], s[10], s[11]);
#pragma unroll
                    for (int i = 12; i + 8 <= kTok; i += 8) {
                        t0 = max3(t0, s[i], s[i + 1]);
                        t1 = max3(t1, s[i + 2], s[i + 3]);
                        t2 = max3(t2, s[i + 4], s[i + 5]);
                        t3 = max3(t3, s[i + 6], s[i + 7]);
                    }
                    t0 = max3(t0, s[kTok - 4], s[kTok - 3]);
                    t1 = max3(t1, s[kTok - 2], s[kTok - 1]);
                    const float top = max3(fmaxf(t0, t1), t2, t3);
                    const bool fresh = r % W::kFreshTiles == 0;
                    if (fresh && r > 0) {  // the sums of the tiles so far leave the tensor memory
                        if (!warp_wait(o_done + place(block, m_tiles - 1), phase(m_tiles - 1))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        const float f = sum_m == -INFINITY ? 0.0f : exp2_approx(sum_m - m);
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            __syncwarp();
                            tmem_read(o_at + c, o);
                            if (valid) {
                                if (r > W::kFreshTiles) with_earlier(c, o, f);
#pragma unroll
                                for (int i = 0; i < 32; i += 4) four_sums(c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            }
                        }
                        __syncwarp();
                        sum_m = m;
                    }
                    const bool over = fmaf(top, mul, shift) > kPShift + kSlack;
                    if (__any_sync(~0u, over)) {
                        const float v = over ? fmaxf(m, top * mul) : m;  // (a row's bits do not depend on its neighbours)
                        const float al = v == m ? 1.0f : exp2_approx(m - v);
                        m = v;
                        worst = fmaxf(worst, v == -INFINITY ? 0.0f : fabsf(v));
                        shift = v == -INFINITY ? kNone : kPShift - v;
                        l *= al;
                        if (!fresh) {  // the sums so far: after the product that is adding to them
                            if (!warp_wait(o_done + place(block, m_tiles - 1), phase(m_tiles - 1))) {
                                failed = true;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                uint32_t w[16];
                                tmem_read16(o_at + c, w);
#pragma unroll
                                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * al);
                                tmem_st16(o_at + c, w);
                            }
                        }
                    }
                    // (two blocks: the last reader of the probabilities' place is the product before these scores, and a commit stands for every
                    // product that was issued before it)
                    float2 sum = make_float2(0.0f, 0.0f);
                    const float2 mul2 = make_float2(mul, mul), shift2 = make_float2(shift, shift);
#pragma unroll
                    for (int c = 0; c < kTok; c += 32) {
                        uint32_t hi[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 e = __ffma2_rn(make_float2(s[c + 2 * i], s[c + 2 * i + 1]), mul2, shift2);
                            s[c + 2 * i] = exp2_approx(e.x);
                            s[c + 2 * i + 1] = exp2_approx(e.y);
                            sum = __fadd2_rn(sum, make_float2(s[c + 2 * i], s[c + 2 * i + 1]));
                            hi[i] = pack2<T>(s[c + 2 * i], s[c + 2 * i + 1]);
                        }
                        tmem_st16(p_at + (kSplit ? c : c / 2), hi);
                        if constexpr (kSplit) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) hi[i] = pack_rest(s[c + 2 * i], s[c + 2 * i + 1], hi[i]);
                            tmem_st16(p_at + c + 16, hi);
                        }
                        if (kHalves && c + 32 == kTok / 2) {
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_local(p_ready + place(block, m_tiles));
                        }
                    }
                    l += sum.x + sum.y;
                    tmem_st_wait();
                } else if (lane == 0) {
                    if (kBlocks == 2) mbar_arrive_local(s_free);
                    if (kHalves) mbar_arrive_local(p_ready + place(block, m_tiles));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_local((kHalves ? p_rest : p_ready) + place(block, m_tiles));
            }
            if (failed) break;
            if (tiles > 0) {
                if (!warp_wait(o_done + place(block, m_tiles - 1), phase(m_tiles - 1))) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (some) {
                    const float inv = 1.0f / l;
                    const float f = sum_m == -INFINITY ? 0.0f : exp2_approx(sum_m - m);
                    const int whole = (x.token + 1) / kTok;
                    const bool odd = (some_noted[(u % kRing) * kCheckWarps] | some_noted[(u % kRing) * kCheckWarps + 1]) != 0;
                    T* out = static_cast<T*>(p.a.out) + out_row * p.a.out_stride + static_cast<long long>(x.head0 + row_head) * D;
                    const unsigned rows = __ballot_sync(~0u, valid);
                    unsigned char* stage = sm + W::kOffOut + (warp - 2 - kCheckWarps) * 4096;
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
                        float o[64];
                        __syncwarp();
                        tmem_read(o_at + c, o);
                        if (valid) {
                            if (tiles > W::kFreshTiles) with_earlier(c, o, f);
#pragma unroll
                            for (int i = 0; i < 64; ++i) o[i] = kSplit ? o[i] * inv * unscale : o[i] * inv;
                            if (odd) {
#pragma unroll 1
                                for (int key = whole * kTok; key <= lim; ++key) {
                                    const int j = key - whole * kTok;
                                    if ((note[(u % kRing) * W::kMasked * (kTok / 16) + (j >> 4)] >> (j & 15) & 1) == 0) continue;
                                    const T* v = static_cast<const T*>(p.a.v) + (static_cast<long long>(x.first) + key) * p.a.v_stride +
                                                 static_cast<long long>(x.kv_head) * D + c;
#pragma unroll
                                    for (int i = 0; i < 64; ++i) {
                                        const float y = value_of(v[i]);
                                        if (!finite(y)) o[i] += y;
                                    }
                                }
                            }
                        }
                        // 128 bytes of each row at a time go through shared memory, so that a warp writes whole lines (rows straight from their
                        // threads, 32 bytes each, took 2500 clocks of a unit's end)
#pragma unroll
                        for (int part = 0; part < static_cast<int>(sizeof(T)) / 2; ++part) {
                            constexpr int kDims = 128 / static_cast<int>(sizeof(T));
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                uint32_t w[4];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    if constexpr (kSplit) w[k] = __float_as_uint(o[part * kDims + 4 * i + k]);
                                    else w[k] = pack2<T>(o[8 * i + 2 * k], o[8 * i + 2 * k + 1]);
                                }
                                *reinterpret_cast<uint4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = 4 * i + (lane >> 3), at = lane & 7;
                                const uint4 w = *reinterpret_cast<const uint4*>(stage + r * 128 + ((at ^ (r & 7)) << 4));
                                T* to = reinterpret_cast<T*>(__shfl_sync(~0u, reinterpret_cast<unsigned long long>(out), r));
                                if (rows >> r & 1u) *reinterpret_cast<uint4*>(to + c + part * kDims + at * (16 / static_cast<int>(sizeof(T)))) = w;
                            }
                        }
                    }
                    __syncwarp();
                    const unsigned big = __ballot_sync(~0u, valid && worst >= kBig && fabsf(m) < INFINITY);
                    if (big != 0) big_rows<T, D>(p.a, big, x.first, x.kv_head, lim, x.head0 + row_head, lane);
                }
                tc_fence_before();
            }
            if (lane == 0) mbar_arrive_local(unit_free + 8 * (u % kRing));
        }
    }
    __syncwarp();
    // (in the issuing warp the elected lane alone knows, whichever it is)
    if (__any_sync(~0u, failed) && lane == 0) atomicOr(&g_prompt_error, kErrWaitTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
    }
}

// ------------------------------------------------------------ fp32 inputs --
struct SplitParams {
    PromptArgs a;
    uint32_t* most;
    float* q_mul;
    __half* q;  // [token][head][2][D]
    __half* k;
    __half* v;
};

// The sequence that a row belongs to as a valid row, or -1.
__device__ __forceinline__ int sequence_of(const PromptArgs& a, int row) {
    int lo = 0, hi = a.B;  // the last sequence that begins at or before the row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.offsets + mid) <= row) lo = mid;
        else hi = mid;
    }
    const PromptRows r = prompt_rows(a, lo);
    return row >= r.first && row < r.first + r.n ? lo : -1;
}

template <int D>
__device__ __forceinline__ uint32_t row_most(const float (&x)[D / 32]) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        if (finite(x[i])) most = max(most, __float_as_uint(fabsf(x[i])));
    return __reduce_max_sync(~0u, most);
}

template <int D>
__device__ __forceinline__ void read_row(const float* p, int lane, float (&x)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
        const float2 v = *reinterpret_cast<const float2*>(p + 2 * lane + 32 * i);
        x[i] = v.x, x[i + 1] = v.y;
    }
}

template <int D>
__device__ __forceinline__ void write_split(__half* p, int lane, const float (&x)[D / 32], float f) {
#pragma unroll
    for (int i = 0; i < D / 32; i += 2) {
        const float a = x[i] * f, b = x[i + 1] * f;
        const uint32_t hi = pack_half2(a, b);
        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        *reinterpret_cast<uint32_t*>(p + 2 * lane + 32 * i) = hi;
        *reinterpret_cast<uint32_t*>(p + D + 2 * lane + 32 * i) = pack_half2(finite(back.x) ? a - back.x : 0.0f, finite(back.y) ? b - back.y : 0.0f);
    }
}

constexpr int kMostRows = 4;  // of a warp

// The largest finite key and value of every sequence and head: a warp for a few tokens of a head, whose reads do not wait for the search of
// their sequences (16 tokens of a warp one after the other: 22 us for 3016 tokens of 4 heads of 128).
template <int D>
__global__ void __launch_bounds__(256) prompt_most_kernel(const __grid_constant__ SplitParams p) {
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int head = static_cast<int>(item % p.a.kv_heads);
    const long long row0 = item / p.a.kv_heads * kMostRows;
    griddep_launch_dependents();
    if (row0 >= p.a.n_tokens) return;
    float x[2][kMostRows][D / 32];
    int seq[kMostRows];
#pragma unroll
    for (int i = 0; i < kMostRows; ++i) {
        const long long row = min(row0 + i, static_cast<long long>(p.a.n_tokens) - 1);
        read_row<D>(static_cast<const float*>(p.a.k) + row * p.a.k_stride + head * D, lane, x[0][i]);
        read_row<D>(static_cast<const float*>(p.a.v) + row * p.a.v_stride + head * D, lane, x[1][i]);
    }
#pragma unroll
    for (int i = 0; i < kMostRows; ++i) seq[i] = row0 + i < p.a.n_tokens ? sequence_of(p.a, static_cast<int>(row0) + i) : -1;
#pragma unroll
    for (int part = 0; part < 2; ++part) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < kMostRows; ++i) {
            const uint32_t mine = row_most<D>(x[part][i]);
            if (seq[i] >= 0) most = max(most, mine);
            if (i + 1 < kMostRows && seq[i + 1] == seq[i]) continue;  // (the last of its sequence here)
            if (seq[i] >= 0 && lane == 0 && most > 0) atomicMax(p.most + (static_cast<size_t>(seq[i]) * p.a.kv_heads + head) * 2 + part, most);
            most = 0;
        }
    }
}

constexpr int kSplitHeads = 4;  // of a warp at once

// Queries, keys and values as fp16 hi + lo, a CTA per token (and 32 of its heads); rows of no sequence are zeros.
template <int D>
__global__ void __launch_bounds__(256) prompt_split_kernel(const __grid_constant__ SplitParams p) {
    const int lane = threadIdx.x & 31, heads = p.a.q_heads + 2 * p.a.kv_heads;
    const long long row = blockIdx.x;
    const int head0 = (blockIdx.y * 8 + (threadIdx.x >> 5)) * kSplitHeads;
    griddep_launch_dependents();
    if (head0 >= heads) return;
    float x[kSplitHeads][D / 32];
#pragma unroll
    for (int i = 0; i < kSplitHeads; ++i) {
        const int head = min(head0 + i, heads - 1), kv = head - p.a.q_heads;
        const float* from = kv < 0 ? static_cast<const float*>(p.a.q) + row * p.a.q_stride + head * D
                                   : kv < p.a.kv_heads ? static_cast<const float*>(p.a.k) + row * p.a.k_stride + kv * D
                                                       : static_cast<const float*>(p.a.v) + row * p.a.v_stride + (kv - p.a.kv_heads) * D;
        read_row<D>(from, lane, x[i]);
    }
    const int seq = sequence_of(p.a, static_cast<int>(row));
    griddep_wait();  // for the largest values
#pragma unroll
    for (int i = 0; i < kSplitHeads; ++i) {
        const int head = head0 + i;
        if (head >= heads) break;
        const int part = head >= p.a.q_heads + p.a.kv_heads, kv = head - p.a.q_heads - (part ? p.a.kv_heads : 0);
        float f = 1.0f;
        if (seq < 0) {
#pragma unroll
            for (int j = 0; j < D / 32; ++j) x[i][j] = 0.0f;
        } else if (head < p.a.q_heads) {
            f = fill_factor(row_most<D>(x[i]));
            if (lane == 0) p.q_mul[row * p.a.q_heads + head] = p.a.scale / f * 1.4426950408889634f;
        } else {
            f = fill_factor(p.most[(static_cast<size_t>(seq) * p.a.kv_heads + kv) * 2 + part]);
        }
        write_split<D>(head < p.a.q_heads ? p.q + (row * p.a.q_heads + head) * 2 * D : (part ? p.v : p.k) + (row * p.a.kv_heads + kv) * 2 * D, lane, x[i], f);
    }
}

// ---------------------------------------------------------------- launches --
size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Where the workspace's parts lie.
struct Workspace {
    size_t most, q_mul, q, k, v, sums, bytes;
};

template <typename T, int D>
Workspace workspace_of(int B, int n_tokens, int q_heads, int kv_heads) {
    using W = Prompt<T, D>;
    Workspace w{};
    const size_t n = n_tokens;
    if (W::kSplit) {
        w.q_mul = align256(static_cast<size_t>(B) * kv_heads * 2 * 4);
        w.q = align256(w.q_mul + n * q_heads * 4);
        w.k = align256(w.q + n * q_heads * D * 4);
        w.v = align256(w.k + n * kv_heads * D * 4);
        w.sums = align256(w.v + n * kv_heads * D * 4);
    }
    // sums of earlier runs of tiles, where there can be any
    w.bytes = w.sums + (n_tokens > W::kFreshTiles * W::kTok ? static_cast<size_t>(kMaxSms) * W::kBlocks * kRows * D * 4 : 0);
    return w;
}

bool encode(CUtensorMap* map, const void* p, CUtensorMapDataType type, int dims, int heads, int tokens, long long stride_bytes, int box_heads, int box_tokens) {
    const auto fn = tensor_map_encoder();
    if (fn == nullptr) return false;
    const cuuint64_t size[3] = {static_cast<cuuint64_t>(dims), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
    const cuuint64_t stride[2] = {static_cast<cuuint64_t>(dims) * 2, static_cast<cuuint64_t>(stride_bytes)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)}, one[3] = {1, 1, 1};
    return fn(map, type, 3, const_cast<void*>(p), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query heads of a block, which share its tiles of keys: as many of the group's as divide it and the 128 rows, so that no row is empty. A group of
// five or three has one.
int block_heads(int group) { return std::min(group & -group, kRows); }

// Launches a kernel, `early`: as soon as every CTA of the one before has begun (the three kernels of fp32 calls: 116.7 -> 114.7 us).
template <class P>
cudaError_t launch_early(void (*kernel)(P), dim3 grid, int threads, size_t smem, bool early, const P& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int D>
cudaError_t launch_one(const PromptArgs& a, cudaStream_t stream) {
    using W = Prompt<T, D>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    const int group = a.q_heads / a.kv_heads;
    const Workspace w = workspace_of<T, D>(a.B, a.n_tokens, a.q_heads, a.kv_heads);
    char* ws = static_cast<char*>(a.workspace);
    PromptParams p{};
    p.a = a;
    p.heads = block_heads(group);
    p.tokens = kRows / p.heads;
    p.chunks = group / p.heads;
    p.sums = reinterpret_cast<float*>(ws + w.sums);
    CUtensorMapDataType type = __is_same(T, __nv_bfloat16) ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const void *q = a.q, *k = a.k, *v = a.v;
    long long qs = a.q_stride * 2, ks = a.k_stride * 2, vs = a.v_stride * 2;
    if constexpr (W::kSplit) {
        SplitParams s;
        s.a = a;
        s.most = reinterpret_cast<uint32_t*>(ws + w.most);
        s.q_mul = reinterpret_cast<float*>(ws + w.q_mul);
        q = s.q = reinterpret_cast<__half*>(ws + w.q);
        k = s.k = reinterpret_cast<__half*>(ws + w.k);
        v = s.v = reinterpret_cast<__half*>(ws + w.v);
        qs = static_cast<long long>(a.q_heads) * D * 4;
        ks = vs = static_cast<long long>(a.kv_heads) * D * 4;
        p.most = s.most;
        p.q_mul = s.q_mul;
        e = cudaMemsetAsync(s.most, 0, static_cast<size_t>(a.B) * a.kv_heads * 8, stream);
        if (e != cudaSuccess) return e;
        const long long most = (static_cast<long long>(a.n_tokens) + kMostRows - 1) / kMostRows * a.kv_heads;
        prompt_most_kernel<D><<<static_cast<unsigned>((most + 7) / 8), 256, 0, stream>>>(s);
        const int heads = a.q_heads + 2 * a.kv_heads;
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        e = launch_early(prompt_split_kernel<D>, dim3(static_cast<unsigned>(a.n_tokens), static_cast<unsigned>((heads + 8 * kSplitHeads - 1) / (8 * kSplitHeads))), 256,
                         0, true, s, stream);
        if (e != cudaSuccess) return e;
    }
    if (!encode(&p.q, q, type, W::kParts * D, a.q_heads, a.n_tokens, qs, p.heads, p.tokens) ||
        !encode(&p.k, k, type, W::kParts * D, a.kv_heads, a.n_tokens, ks, 1, W::kTok) ||
        !encode(&p.v, v, type, W::kParts * D, a.kv_heads, a.n_tokens, vs, 1, W::kTok))
        return cudaErrorInvalidValue;
    const int step = W::kBlocks * p.tokens;
    const long long units = (static_cast<long long>(a.n_tokens) / step + a.B) * a.kv_heads * p.chunks;  // at most
    return launch_early(prompt_kernel<T, D>, dim3(static_cast<unsigned>(std::min<long long>(units, std::min(sms, kMaxSms)))), W::kThreads, W::kSmem, W::kSplit, p,
                        stream);
}

template <typename T>
cudaError_t launch_type(const PromptArgs& a, cudaStream_t stream) {
    switch (a.head_dim) {
        case 64: return launch_one<T, 64>(a, stream);
        case 128: return launch_one<T, 128>(a, stream);
        case 256: return launch_one<T, 256>(a, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <typename T>
size_t bytes_of(int B, int n_tokens, int q_heads, int kv_heads, int head_dim) {
    switch (head_dim) {
        case 64: return workspace_of<T, 64>(B, n_tokens, q_heads, kv_heads).bytes;
        case 128: return workspace_of<T, 128>(B, n_tokens, q_heads, kv_heads).bytes;
        case 256: return workspace_of<T, 256>(B, n_tokens, q_heads, kv_heads).bytes;
        default: return 0;
    }
}

}  // namespace

size_t prompt_workspace_bytes(int B, int n_tokens, int q_heads, int kv_heads, int head_dim, DType dtype) {
    return dtype == DType::kF32 ? bytes_of<float>(B, n_tokens, q_heads, kv_heads, head_dim)
                                : bytes_of<__half>(B, n_tokens, q_heads, kv_heads, head_dim);
}

cudaError_t launch_prompt_attention(const PromptArgs& a, cudaStream_t stream) {
    switch (a.dtype) {
        case DType::kF32: return launch_type<float>(a, stream);
        case DType::kF16: return launch_type<__half>(a, stream);
        case DType::kBF16: return launch_type<__nv_bfloat16>(a, stream);
    }
    return cudaErrorInvalidValue;
}

cudaError_t read_prompt_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_prompt_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_prompt_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace gdn
