// gdn_kv4_window.cu - attention over the 4-bit cache for windows with many query
// rows (verify windows, prompt chunks): the same mathematics as
// gdn_kv4_attention.cu, on the 5th-generation tensor cores.
//
//   S = Q K^T   128 rows x 64 tokens x D,   O += P V   128 rows x D x 64 tokens
//
// A row is a (token, query head) pair of one kv head's group, so one unpacked tile of
// keys and values serves the whole group of a block of tokens, and two blocks of 128 rows
// (256 rows per CTA) where a window has them.
//
// What bounds it. 2 x 1024 tokens behind 8000, 32 query heads of 128, bf16: 310 us, 0.92 PFLOP/s, 0.46 of the
// measured bf16 rate (four sequences 605 us, 0.94 PFLOP/s). For a 64-token tile of both blocks (2750 clocks of an SM) the
// tensor pipe works 1500 clocks (a product of 64 columns takes as long as one of 128), the special-function unit 1024
// (16384 exponentials), and the schedulers issue 0.57 of the time; the longest chain is a softmax warp's own: scores
// from tensor memory, maximum, exchange, exponentials, probabilities back, about 2200 clocks. Windows of few rows (a
// verify window, 17 query heads) are bound by the latency of one tile's steps, about 2600 clocks, which is why up to 16
// rows go to gdn_kv4_attention.cu (64 sequences of 4096, 16 rows: 62 us there, 104 us here).
//
//   warp 0     issues the products, by an elected lane (a lane chosen by its number had each product's operands moved to
//              uniform registers by a loop over the lanes, and issuing took longer than everything else: 411 us)
//   8 warps    half a row per thread (for each 128 rows; warps w and w + 4 share rows and exchange their
//              halves' maxima): queries in, the softmax of a tile from tensor
//              memory, probabilities back to tensor memory (fp16, over the scores they
//              came from, as the A operand of the second product), outputs out
//   4-8 warps  unpack the next tiles: 16 bytes of codes per thread from global
//              memory, a tile ahead in registers, to fp16 in the swizzled
//              K-major rows that both products read (V with its rows as K: MN-major)
//
// Scores have two buffers in tensor memory, K and V tiles two stages each, so
// the product of tile j + 1 runs during the softmax of tile j (at D = 64 with two blocks: one buffer and longer tiles). The
// running maximum is a reference that is raised only when a score exceeds it by
// kSlack (in base 2): then the row's sums are read, scaled and written back,
// which is rare after the first tile. fp32 calls take Q and P as fp16 hi + lo, two products each.
//
// Numerics, masks and missing pages: as in gdn_kv4_attention.cu. Tokens past a
// block's end and those of missing pages are unpacked as zeros.
//
// Work split: blocks of rows have different numbers of tiles (causal), so the
// line that is dealt out to the CTAs has the blocks of each sequence in turn, each times its (layer, kv head) pairs.
// Waits are bounded. One that gives up makes the issuing and unpacking roles leave their loops, while a softmax warp goes on
// without waiting, so that its other half still meets it; the others run into their own limits, the device
// error word is set, and the tensor memory is freed after the last product has completed.

#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_kv4_attention.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kRows = 128;       // of a block
// A unit's start (queries in, outputs out) takes as many places on the line as this many tokens. 2 x 1024 tokens from
// position 0, 32 heads: 131 / 104 / 86 us for 128 / 256 / 512; 16 ragged windows of 8: 57 / 47 / 47 us.
constexpr int kStartTokens = 512;

__device__ unsigned int g_kv4_window_error = 0;

// NB blocks of 128 rows per CTA share the unpacked tiles: two where a window has as many rows and the tensor memory
// has room for their sums (D <= 128), one CTA per SM then; otherwise one, and two CTAs per SM where they fit. fp32 calls
// always take one block, whose sums fit shared memory: 1024 tokens after 8000, two sequences with 32 heads, 559 us (D =
// 128) and 449 us (D = 64), with two 605 and 469 us.
template <int D, bool SPLIT, int NB>
struct Win {
    static constexpr int kSoftWarps = 8 * NB;
    static constexpr int kUnpackWarps = D == 128 ? 4 * NB : 4;
    static constexpr int kThreads = 32 * (1 + kSoftWarps + kUnpackWarps);
    static constexpr int kUnitRows = NB * kRows;
    // Tiles of 64 tokens with two buffers of scores, or of 128 tokens, for which the first product runs at twice the rate,
    // with one (there is no more tensor memory): 2 x 1024 tokens behind 8000, 32 heads, take 328 us with the former and
    // 354 us with the latter at D = 128, 280 and 257 us at D = 64.
    static constexpr int kTok = NB == 2 && D == 64 ? 128 : 64;
    static constexpr int kBuffers = kTok == 128 ? 1 : 2;
    static constexpr int kStages = D == 256 && SPLIT ? 1 : 2;
    static constexpr int kBlk = D / 64;                        // 64-dim blocks of a row (128 bytes)
    static constexpr uint32_t kQBlock = kRows * 128;           // bytes of a block of Q
    static constexpr uint32_t kQBytes = kBlk * kQBlock;        // of Q hi (then lo) of 128 rows
    static constexpr uint32_t kQRows = kQBytes * (SPLIT ? 2 : 1);
    static constexpr uint32_t kKvBlock = kTok * 128;           // of a block of K or V
    static constexpr uint32_t kKvBytes = kBlk * kKvBlock;
    static constexpr uint32_t kOffK = kQRows * NB;
    static constexpr uint32_t kOffV = kOffK + kStages * kKvBytes;
    static constexpr uint32_t kOffMul = kOffV + kStages * kKvBytes;  // factor of a row's raw scores
    static constexpr uint32_t kOffBad = kOffMul + kUnitRows * 4;     // missing pages of tiles j mod 4
    static constexpr uint32_t kOffXch = kOffBad + 4 * 4;             // what the two halves of a row tell each other
    static constexpr uint32_t kOffBar = kOffXch + 2 * 2 * kUnitRows * 4;
    static constexpr uint32_t kBars = 2 + 2 + 1 + 1 + 3 * 2 * NB;   // see below
    static constexpr uint32_t kOffSum = kOffBar + kBars * 8 + 64;    // + cursor, tensor memory address
    // Sums in tensor memory start afresh every 512 tokens (16-bit calls: 16384) and are added up with fp32 instructions,
    // in shared memory where it has room, otherwise in the workspace ([dim / 4][row][4], which a warp reads in whole
    // lines): the tensor cores cut off a running sum at every step instead of rounding it, so the error grows with the
    // steps. fp32, equal values at 16000 tokens: 1.7e-4 without, 7e-6 with. 16 random windows of 8 tokens after up to
    // 4096: 2.3e-6 without, 1.6e-6 at every 1024, 1.0e-6 here (an fp32 softmax over the unpacked cache has 1.1e-6), time
    // 47.5 -> 48 us; D = 256, two sequences of 1024 tokens after 8000 with 16 heads: 764 -> 826 us. 16-bit calls round
    // their probabilities to 2^-12; at every 16384 the sums lose less, and it costs nothing. The fp32 additions round too, in
    // step with each other on data that repeats itself: fp32, equal values over 2^20 tokens in a pattern of 1024, 1.8e-5 on
    // average and 1.3e-4 at most.
    static constexpr int kFreshTiles = SPLIT ? 512 / kTok : 16384 / kTok;
    static constexpr bool kSumInSmem = SPLIT && D <= 128;
    static_assert(!kSumInSmem || kOffSum % 16 == 0, "read by fours");
    static constexpr uint32_t kUsed = kOffSum + (kSumInSmem ? kUnitRows * D * 4 : 0);
    static constexpr int kCtas = NB == 1 && D <= 128 && 2 * (kUsed + 2048) <= 232448 ? 2 : 1;
    // no more CTAs than the tensor memory has room for: a third (second) would wait in its allocation
    static constexpr uint32_t kLeast = kCtas == 2 ? 80 * 1024 : 118 * 1024;
    static constexpr uint32_t kSmem = (kUsed + 1024 > kLeast ? kUsed + 1024 : kLeast);
    static constexpr uint32_t kTmCols = NB * (128 + D) <= 256 ? 256 : 512;
    static constexpr uint32_t kTmO = NB * 128;                       // scores of block i from 128 i, buffers kTok apart
    static_assert(NB * (128 + D) <= 512, "scores and sums fit the tensor memory");
};

// Where a CTA is: unit (b, block, pair of layer and kv head), at place `at` of its `cost`, `left` places to go.
struct WinCursor {
    int b, blk, lh, cost, at;
    int left;
};

constexpr int kNoRow = -2147483647 - 1;

// First position that no row of block blk sees, or kNoRow.
__device__ __forceinline__ int block_end(const AttnParams& p, const Kv4Window& w, int blk) {
    const int row = blk * p.unit_rows;  // T group < 2^31
    if (row >= w.n * p.group) return kNoRow;
    const int t_hi = min(static_cast<int>((static_cast<uint32_t>(row) + p.unit_rows - 1) / p.group), w.n - 1);
    return w.start + min(t_hi + 1, w.cap - w.start);
}

__device__ __forceinline__ int block_cost(const AttnParams& p, const Kv4Window& w, int blk) {
    const int end = block_end(p, w, blk);
    // one tile at least: rows that see no position get their zeros
    return end == kNoRow ? 0 : (kStartTokens + max(end, 1) + (1 << p.tile_shift) - 1) >> p.tile_shift;
}

// Cost of block i % col_blocks of sequence i / col_blocks.
__device__ __forceinline__ int item_cost(const AttnParams& p, int i) {
    const int b = i / p.col_blocks;
    return block_cost(p, kv4_window(p.c, b), i - b * p.col_blocks);
}

__device__ __forceinline__ long long line_length(const AttnParams& p, int pairs, int lane) {
    long long s = 0;
    for (int i = lane; i < p.c.B * p.col_blocks; i += 32) s += item_cost(p, i);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    return s * pairs;
}

// The unit and place in it of place x of the line, by one warp.
__device__ __forceinline__ WinCursor find(const AttnParams& p, int pairs, long long x, int lane) {
    WinCursor k{p.c.B, 0, 0, 0, 0, 0};
    const int items = p.c.B * p.col_blocks;
    for (int i0 = 0; i0 < items; i0 += 32) {
        const int cost = i0 + lane < items ? item_cost(p, i0 + lane) : 0;
        long long sum = static_cast<long long>(cost) * pairs;
        const long long mine = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += y;
        }
        const unsigned hit = __ballot_sync(~0u, sum > x);
        if (hit == 0) {
            x -= __shfl_sync(~0u, sum, 31);
            continue;
        }
        const int src = __ffs(hit) - 1;
        k.b = (i0 + src) / p.col_blocks;
        k.blk = i0 + src - k.b * p.col_blocks;
        k.cost = __shfl_sync(~0u, cost, src);
        x -= __shfl_sync(~0u, sum - mine, src);
        k.lh = static_cast<int>(mul_div(x, 1, k.cost));
        k.at = static_cast<int>(x - static_cast<long long>(k.lh) * k.cost);
        return k;
    }
    return k;
}

__device__ __forceinline__ void next_unit(const AttnParams& p, int pairs, WinCursor& k) {
    k.left -= k.cost - k.at;
    k.at = 0;
    if (++k.lh < pairs || k.left <= 0) return;
    k.lh = 0;
    ++k.blk;
    while (k.b < p.c.B) {
        if (k.blk < p.col_blocks && (k.cost = block_cost(p, kv4_window(p.c, k.b), k.blk)) > 0) return;
        k.blk = 0;
        ++k.b;
    }
}

// The tiles [r0, r1) of the cursor's unit that are its CTA's.
__device__ __forceinline__ void unit_tiles(const AttnParams& p, const WinCursor& k, int& r0, int& r1) {
    const int start = kStartTokens >> p.tile_shift;
    r0 = max(k.at - start, 0);
    r1 = min(k.cost, k.at + k.left) - start;
}

__device__ __forceinline__ Unit win_unit(const AttnParams& p, const WinCursor& k) {
    Unit x;
    const Kv4Window w = kv4_window(p.c, k.b);
    x.h = k.lh % p.c.kv_heads;
    x.l = k.lh / p.c.kv_heads;
    x.col0 = k.blk * p.unit_rows;
    x.start = w.start;
    x.n = w.n;
    x.end = block_end(p, w, k.blk);
    return x;
}

// fp16 by fp16, fp32 accumulation, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

// One product step, D (tensor memory) = or += A B, with the descriptors' halves apart: their upper halves are one
// constant and their lower ones differ by constants, so a step costs the issuing thread an addition or two.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, version, 128-byte swizzle

// Lower halves: K-major rows, and rows read as K (MN-major) with 64-wide blocks `stride` bytes apart.
__device__ __forceinline__ uint32_t desc_k(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t saddr, uint32_t stride) {
    return ((saddr & 0x3FFFFu) >> 4) | ((stride >> 4) << 16);
}

template <bool FIRST>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(kDescHi), "n"(FIRST ? 0 : 1)
        : "memory");
}

// A from tensor memory (fp16 pairs, 8 columns of 32 bits per k-step of 16).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %4};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_lo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
        : "memory");
}

// 32 consecutive columns of this warp's lanes, one lane per thread, complete when it returns.
__device__ __forceinline__ void tmem_read32(uint32_t taddr, float (&v)[32]) {
    uint32_t u[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
          "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
          "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(u[i]);
}

// 16 consecutive columns of this warp's lanes, one lane per thread, complete when it returns.
__device__ __forceinline__ void tmem_read16(uint32_t taddr, uint32_t (&u)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
          "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(taddr)
        : "memory");
}

// 16 outputs of a row, times a factor.
__device__ __forceinline__ void store_out16(const AttnParams& p, size_t i, const float (&o)[16], float f) {
    if (p.dtype == DType::kF32) {
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4*>(static_cast<float*>(p.out) + i + j) =
                make_float4(o[j] * f, o[j + 1] * f, o[j + 2] * f, o[j + 3] * f);
        return;
    }
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (p.dtype == DType::kF16) {
            w[j] = pack_half2(o[2 * j] * f, o[2 * j + 1] * f);
        } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * j] * f, o[2 * j + 1] * f);
            w[j] = *reinterpret_cast<const uint32_t*>(&v);
        }
    }
    uint4* out = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + i);
    out[0] = make_uint4(w[0], w[1], w[2], w[3]);
    out[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Stores 16 consecutive columns of this warp's lanes, one lane per thread.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Waits for phase `parity` of the mbarrier, giving up after kWaitLimitNs. The hardware suspends the thread for up to
// 20 us at a time: five waits per tile and warp that polled took a tenth of the SM's issue slots.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity) {
    unsigned long long t0 = 0;
    for (;;) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        const unsigned long long t = global_timer_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kWaitLimitNs) return false;
    }
}

// Every lane of a warp waits; false, for all of them, if one gave up.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
    const bool late = !wait_for(bar, parity);
    return !__any_sync(~0u, late);
}

template <int D, bool SPLIT, int NB>
__global__ void __launch_bounds__(Win<D, SPLIT, NB>::kThreads, Win<D, SPLIT, NB>::kCtas)
    kv4_window_kernel(const __grid_constant__ AttnParams p) {
    using W = Win<D, SPLIT, NB>;
    constexpr int kStages = W::kStages, kSoftWarps = W::kSoftWarps, kUnpackWarps = W::kUnpackWarps;
    constexpr int kUnitRows = W::kUnitRows, kTok = W::kTok, kBuffers = W::kBuffers;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), base = (raw + 1023u) & ~1023u;
    unsigned char* sm = smem_raw + (base - raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* mul_s = reinterpret_cast<float*>(sm + W::kOffMul);
    uint32_t* bad_s = reinterpret_cast<uint32_t*>(sm + W::kOffBad);
    WinCursor* cur_s = reinterpret_cast<WinCursor*>(sm + W::kOffBar + W::kBars * 8);
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(cur_s + 1);
    const uint32_t bars = base + W::kOffBar;
    const uint32_t k_full = bars, v_full = bars + 16;      // per stage: unpacked
    const uint32_t q_full = bars + 32, drained = bars + 40;
    // per block and parity of the tile
    const uint32_t s_done = bars + 48, p_ready = s_done + 16 * NB, o_done = p_ready + 16 * NB;
    float* xch = reinterpret_cast<float*>(sm + W::kOffXch);
    const int pairs = p.c.L * p.c.kv_heads;

    long long total = 0;
    int ctas = 0;
    if (warp < 2) {
        total = line_length(p, pairs, lane);
        ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    }
    if (warp == 0) {
        long long lo = 0, hi = 0;
        WinCursor k{};
        if (static_cast<int>(blockIdx.x) < ctas) {
            cta_range(total, blockIdx.x, ctas, lo, hi);
            k = find(p, pairs, lo, lane);
        }
        k.left = static_cast<int>(hi - lo);
        if (lane == 0) *cur_s = k;
    } else if (tid == 32) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(k_full + 8 * i, kUnpackWarps);
            mbar_init(v_full + 8 * i, kUnpackWarps);
            for (int j = 0; j < NB; ++j) {
                mbar_init(o_done + 16 * j + 8 * i, 1);
                mbar_init(s_done + 16 * j + 8 * i, 1);
                mbar_init(p_ready + 16 * j + 8 * i, 8);
            }
        }
        mbar_init(q_full, kSoftWarps);
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    __syncthreads();
    WinCursor cur = *cur_s;
    griddep_launch_dependents();
    JoinRecord* record = reinterpret_cast<JoinRecord*>(p.records) + blockIdx.x;
    if (tid == 32) *record = JoinRecord{0, 0, 0, 0};
    if (cur.left <= 0) return;
    if (warp == 0) tmem_alloc(smem_addr(tmem_s), W::kTmCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_s;

    // Tile n of the CTA (counted over all its units) uses stage n mod kStages of K and V and buffer n mod kBuffers of the
    // scores; barriers per tile alternate by its parity.
    auto stage_parity = [](int n) -> uint32_t { return static_cast<uint32_t>(n / kStages) & 1u; };
    auto tile_parity = [](int n) -> uint32_t { return static_cast<uint32_t>(n >> 1) & 1u; };
    bool failed = false;
    int n = 0;

    if (warp > 0 && warp <= kSoftWarps) {
        // ------------------------------------------------------------------ rows
        const int block = (warp - 1) >> 3, quarter = warp & 3, half = ((warp - 1) >> 2) & 1;  // (a warp reaches lanes 32 (warp mod 4) ..)
        const int row = 128 * block + 32 * quarter + lane;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t o_at = lanes + W::kTmO + block * D;  // the row's sums
        int met = 0;  // times the two halves have met
        // This half's value of the row to the other half; returns the other's. A warp that has given up waiting still comes
        // here as often as its other half does, so this barrier needs no limit of its own.
        auto exchange = [&](float v) -> float {
            float* x = xch + (met & 1) * 2 * kUnitRows + row;
            ++met;
            x[half * kUnitRows] = v;
            asm volatile("bar.sync %0, 64;" ::"r"(1 + 4 * block + quarter) : "memory");
            return x[(half ^ 1) * kUnitRows];
        };
        for (; cur.left > 0; next_unit(p, pairs, cur)) {
            int r0, r1;
            unit_tiles(p, cur, r0, r1);
            if (r1 <= r0) break;
            const Unit x = win_unit(p, cur);
            const int b = cur.b;
            const int rows = min(x.n * p.group - x.col0, kUnitRows);
            if (tid == 32 && kv4_runs_out(kv4_window(p.c, b))) atomicOr(&g_kv4_window_error, kErrBadPage);
            // queries, scaled to fill fp16's range: row 8 i + this warp of the block's eight, kAtOnce rows in flight
            constexpr int kAtOnce = D > 128 ? 2 : 4;
            const int mine = 128 * block + ((warp - 1) & 7);
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += kAtOnce) {
                if (mine + 8 * i0 >= rows) break;
                constexpr int kChunks = D > 128 ? D / 128 : 1;
                float4 v[kAtOnce][kChunks];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const int rr = mine + 8 * (i0 + i);
                        v[i][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (rr < rows && 4 * lane + 128 * c < D) v[i][c] = load_q4(p, q_row(p, b, x, x.col0 + rr) + 128 * c + 4 * lane);
                    }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int rr = mine + 8 * (i0 + i);
                    float a = 0.0f;
#pragma unroll
                    for (int c = 0; c < kChunks; ++c)
                        a = fmaxf(fmaxf(a, fmaxf(fabsf(v[i][c].x), fabsf(v[i][c].y))), fmaxf(fabsf(v[i][c].z), fabsf(v[i][c].w)));
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
                    const float f = row_factor(a);
                    if (lane == 0) mul_s[rr] = score_factor(p.scale, f);
#pragma unroll
                    for (int c = 0; c < kChunks; ++c) {
                        const int d = 4 * lane + 128 * c;
                        if (d >= D) continue;
                        const uint32_t at = block * W::kQRows + (d >> 6) * W::kQBlock + sw128_offset(rr & 127, (d & 63) >> 3) + (d & 7) * 2;
                        const float q0 = v[i][c].x * f, q1 = v[i][c].y * f, q2 = v[i][c].z * f, q3 = v[i][c].w * f;
                        const uint2 hi = make_uint2(pack_half2(q0, q1), pack_half2(q2, q3));
                        *reinterpret_cast<uint2*>(sm + at) = hi;
                        if constexpr (SPLIT)
                            *reinterpret_cast<uint2*>(sm + W::kQBytes + at) =
                                make_uint2(pack_rest(q0, q1, hi.x), pack_rest(q2, q3, hi.y));
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_local(q_full);
            asm volatile("bar.sync %0, 256;" ::"r"(1 + 4 * NB + block) : "memory");  // the block's rows have their factors

            const bool some = 128 * block + 32 * quarter < rows;  // this warp has rows
            const float mul = row < rows ? mul_s[row] : kLeastScale;
            const int lim = row < rows ? min(x.start + (x.col0 + row) / p.group, x.end - 1) : -1;
            const int seen_by_all = min(x.start + x.col0 / p.group + 1, x.end);
            float m = -INFINITY, shift = kNone, l = 0.0f;
            // sums of earlier tiles, relative to sum_m
            auto four_sums = [&](int c) -> float4& {  // of dims c .. c + 3
                float* sums = W::kSumInSmem ? reinterpret_cast<float*>(sm + W::kOffSum)
                                            : p.sums + static_cast<size_t>(blockIdx.x) * D * W::kUnitRows;
                return *reinterpret_cast<float4*>(sums + c * W::kUnitRows + 4 * row);
            };
            float sum_m = -INFINITY;
            for (int r = r0; r < r1;) {
                const int first = r, last = min(first + W::kFreshTiles, r1);
                for (; r < last; ++r, ++n) {
                    if (!failed && !warp_wait(s_done + 16 * block + 8 * (n & 1), tile_parity(n))) failed = true;
                    tc_fence_after();
                    if (some) {
                        constexpr int kHalf = kTok / 2, kChunks = kHalf / 32;
                        // the half's scores, then, per 32 of them, 16 columns of probabilities and 16 of their rests
                        const uint32_t s_at = lanes + 128 * block + kTok * (n % kBuffers) + kHalf * half;
                        const int p0 = r * kTok + kHalf * half;  // its first position
                        const uint32_t bad = (bad_s[n & 3] >> (kHalf / 16 * half)) & ((1u << (kHalf / 16)) - 1u);
                        const bool part = p0 + kHalf > seen_by_all || bad != 0;
                        float s[32];
                        auto scores = [&](int c) {
                            tmem_read32(s_at + 32 * c, s);
                            if (part) {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (p0 + 32 * c + i > lim || ((bad >> (2 * c + (i >> 4))) & 1u)) s[i] = -INFINITY;
                            }
                        };
                        float top = -INFINITY;
#pragma unroll
                        for (int c = 0; c < kChunks; ++c) {
                            scores(c);
                            float t0 = max3(s[0], s[1], s[2]), t1 = max3(s[3], s[4], s[5]);
#pragma unroll
                            for (int i = 6; i < 30; i += 4) {
                                t0 = max3(t0, s[i], s[i + 1]);
                                t1 = max3(t1, s[i + 2], s[i + 3]);
                            }
                            top = max3(top, max3(t0, s[30], s[31]), t1);
                        }
                        top = fmaxf(top, exchange(top));
                        if (__any_sync(~0u, fmaf(top, mul, shift) > kPShift + kSlack)) {
                            const float v = fmaxf(m, top * mul);
                            const float al = v == m ? 1.0f : exp2_approx(m - v);
                            m = v;
                            shift = v == -INFINITY ? kNone : kPShift - v;
                            l *= al;
                            if (r > first) {  // this half of the sums so far: after the product that is adding to them
                                if (!failed && !warp_wait(o_done + 16 * block + 8 * ((n - 1) & 1), tile_parity(n - 1))) failed = true;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                                    uint32_t w[16];
                                    tmem_read16(o_at + c, w);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * al);
                                    tmem_st16(o_at + c, w);
                                }
                            }
                        }
                        float2 sum = make_float2(0.0f, 0.0f);
                        const float2 mul2 = make_float2(mul, mul), shift2 = make_float2(shift, shift);
#pragma unroll
                        for (int c = kChunks - 1; c >= 0; --c) {  // the last chunk is still in registers
                            if (c < kChunks - 1) scores(c);
                            uint32_t hi[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), mul2, shift2);
                                s[2 * i] = exp2_approx(e.x);
                                s[2 * i + 1] = exp2_approx(e.y);
                                sum = __fadd2_rn(sum, make_float2(s[2 * i], s[2 * i + 1]));
                                hi[i] = pack_half2(s[2 * i], s[2 * i + 1]);
                            }
                            tmem_st16(s_at + 32 * c, hi);
                            if constexpr (SPLIT) {
#pragma unroll
                                for (int i = 0; i < 16; ++i) hi[i] = pack_rest(s[2 * i], s[2 * i + 1], hi[i]);
                                tmem_st16(s_at + 32 * c + 16, hi);
                            }
                        }
                        l += sum.x + sum.y;
                        tmem_st_wait();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_local(p_ready + 16 * block + 8 * (n & 1));
                }
                if (!failed && !warp_wait(o_done + 16 * block + 8 * ((n - 1) & 1), tile_parity(n - 1))) failed = true;
                tc_fence_after();
                if (some && r1 - r0 > W::kFreshTiles) {  // these sums and the earlier ones; the last time in tensor memory
                    const float f = sum_m == -INFINITY ? 0.0f : exp2_approx(sum_m - m);
#pragma unroll 1
                    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                        uint32_t w[16];
                        __syncwarp();
                        tmem_read16(o_at + c, w);
                        if (row < rows) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4) {
                                const float4 y = first > r0 ? four_sums(c + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                const float4 v = make_float4(fmaf(y.x, f, __uint_as_float(w[i])), fmaf(y.y, f, __uint_as_float(w[i + 1])),
                                                             fmaf(y.z, f, __uint_as_float(w[i + 2])), fmaf(y.w, f, __uint_as_float(w[i + 3])));
                                w[i] = __float_as_uint(v.x), w[i + 1] = __float_as_uint(v.y);
                                w[i + 2] = __float_as_uint(v.z), w[i + 3] = __float_as_uint(v.w);
                                if (last < r1) four_sums(c + i) = v;
                            }
                        }
                        __syncwarp();
                        if (last == r1) tmem_st16(o_at + c, w);
                    }
                    tmem_st_wait();
                    sum_m = m;
                }
            }
            // outputs: each half its dims
            const float other = exchange(l);
            l = half == 0 ? l + other : other + l;
            const bool done = r0 == 0 && r1 == cur.cost - (kStartTokens >> p.tile_shift);
            if (some) {
                float* slot = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (r0 == 0 ? 1 : 0)) * (kUnitRows * (D + 2));
                const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;  // no key at all: zeros
                const size_t out = row < rows ? q_row(p, b, x, x.col0 + row) : 0;
#pragma unroll 1
                for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
                    uint32_t w[16];
                    __syncwarp();
                    tmem_read16(o_at + c, w);
                    float o[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(w[i]);
                    if (row < rows && done) {
                        store_out16(p, out + c, o, inv);
                    } else if (row < rows) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<float4*>(slot + (NB == 2 ? (c + i) * kUnitRows + 4 * row : row * D + c + i)) =
                                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (!done && half == 0 && row < rows) {
                    slot[kUnitRows * D + row] = m;
                    slot[kUnitRows * D + kUnitRows + row] = l;
                }
                __syncwarp();
            }
            if (tid == 32 && !done && r0 == 0)  // this CTA's block of the join has it
                *record = JoinRecord{cur.b, cur.blk, cur.lh,
                                     cta_of(total, mul_div(total, blockIdx.x + 1, ctas) - cur.at - cur.left + cur.cost - 1, ctas) -
                                         static_cast<int>(blockIdx.x) + 1};
            tc_fence_before();
        }
    } else if (warp > kSoftWarps) {
        // ---------------------------------------------------------------- unpack
        constexpr int kChunksPerRow = D / 32;            // 16 bytes of codes: 32 dims, two scales
        constexpr int kMine = kTok * kChunksPerRow / (32 * kUnpackWarps);  // chunks of K (and of V) per thread
        const int uw = warp - 1 - kSoftWarps;
        const int psize = 1 << p.c.page_shift;
        constexpr int kTokShift = kTok == 128 ? 7 : 6;
        const int shift = min(p.c.page_shift, kTokShift);
        const uint32_t head_bytes = static_cast<uint32_t>(kv4_head_bytes(psize, D)), page_bytes = head_bytes * p.c.kv_heads;
        // a thread's chunks are the same place of rows kStep apart
        constexpr int kStep = 8 * (4 * kUnpackWarps / kChunksPerRow);
        const int place = 4 * uw + (lane >> 3);
        const int pc = place % kChunksPerRow, row0 = (place / kChunksPerRow) * 8 + (lane & 7);
        const int lc = pc ^ (kv4_swizzle(row0, D / 16) >> 1);  // the dims: 32 lc ..
        uint32_t dst[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = (lc >> 1) * W::kKvBlock + sw128_offset(row0, (lc & 1) * 4 + j);
        const uint32_t code_off = row0 * (D / 2) + pc * 16, scale_off = psize * (D / 2) + row0 * (D / 16) + 2 * lc;
        WinCursor ahead = cur;   // of the tile whose data is requested next
        int a_r = 0, a_r1 = 0;
        int a_end = 0;
        const int32_t* a_table = nullptr;  // the sequence's pages
        const uint8_t* a_head = nullptr;
        bool more = true;
        // steps to the next tile; false at the end of the CTA's places
        auto step = [&]() {
            if (++a_r < a_r1) return;
            for (;;) {
                if (ahead.left <= 0) {
                    more = false;
                    return;
                }
                int r0, r1;
                unit_tiles(p, ahead, r0, r1);
                const Unit x = win_unit(p, ahead);
                a_r = r0;
                a_r1 = r1;
                a_end = x.end;
                a_table = p.c.block_table + static_cast<size_t>(ahead.b) * p.c.max_pages;
                a_head = p.c.cache + (static_cast<size_t>(x.l) * p.c.n_pages * p.c.kv_heads + x.h) * head_bytes;
                next_unit(p, pairs, ahead);
                if (r1 > r0) return;
            }
        };
        a_r1 = -1;
        step();
        uint4 kc[kMine], vc[kMine];
        uint32_t ks[kMine], vs[kMine];
        uint32_t bad = 0;
        auto fetch = [&]() {
            const int p0 = a_r * kTok;
            if (shift == kTokShift && p0 + kTok <= a_end) {  // a whole tile of one page
                int page = __ldg(a_table + (p0 >> p.c.page_shift));
                if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.n_pages)) page = -1;
                bad = page < 0 ? (1u << (kTok / 16)) - 1u : 0u;
                const int in_page = p0 & (psize - 1);
                const uint8_t* k = a_head + static_cast<unsigned long long>(static_cast<uint32_t>(max(page, 0))) * page_bytes;
                const uint8_t* v = k + head_bytes / 2;
                const uint32_t co = code_off + in_page * (D / 2), so = scale_off + in_page * (D / 16);
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    kc[i] = __ldg(reinterpret_cast<const uint4*>(k + co + i * kStep * (D / 2)));
                    vc[i] = __ldg(reinterpret_cast<const uint4*>(v + co + i * kStep * (D / 2)));
                    ks[i] = __ldg(reinterpret_cast<const uint16_t*>(k + so + i * kStep * (D / 16)));
                    vs[i] = __ldg(reinterpret_cast<const uint16_t*>(v + so + i * kStep * (D / 16)));
                    if (page < 0) ks[i] = vs[i] = 0u;
                }
                return;
            }
            // lane j looks up page j of the tile
            const int pos = p0 + (lane << shift);
            const bool want = lane < (kTok >> shift) && pos < a_end;
            int page = want ? __ldg(a_table + (pos >> p.c.page_shift)) : 0;
            if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.c.n_pages)) page = -1;
            const unsigned gone = __ballot_sync(~0u, page == -1);
            // the missing pages as 16-token groups, whatever the page size
            bad = 0;
#pragma unroll
            for (int q = 0; q < kTok / 16; ++q) bad |= ((gone >> ((16 * q) >> shift)) & 1u) << q;
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int row = row0 + i * kStep, j = row >> shift;
                const int pg = __shfl_sync(~0u, page, j);
                kc[i] = vc[i] = make_uint4(0u, 0u, 0u, 0u);
                ks[i] = vs[i] = 0u;
                if (pg >= 0 && p0 + row < a_end) {
                    const int off = (p0 & (psize - 1)) - (j << shift) + i * kStep;  // rows from row0's offsets
                    const uint8_t* k = a_head + static_cast<unsigned long long>(static_cast<uint32_t>(pg)) * page_bytes;
                    const uint8_t* v = k + head_bytes / 2;
                    kc[i] = __ldg(reinterpret_cast<const uint4*>(k + static_cast<int>(code_off) + off * (D / 2)));
                    vc[i] = __ldg(reinterpret_cast<const uint4*>(v + static_cast<int>(code_off) + off * (D / 2)));
                    ks[i] = __ldg(reinterpret_cast<const uint16_t*>(k + static_cast<int>(scale_off) + off * (D / 16)));
                    vs[i] = __ldg(reinterpret_cast<const uint16_t*>(v + static_cast<int>(scale_off) + off * (D / 16)));
                }
            }
        };
        // one chunk of 32 values, as fp16 in its swizzled row
        auto put = [&](unsigned char* tile, const uint4& code, uint32_t scales) {
            const uint32_t w[4] = {code.x, code.y, code.z, code.w};
            const uint32_t s0 = scale_twice(scales, 0), s1 = scale_twice(scales, 1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t v[4];
                unpack(w[j], j < 2 ? s0 : s1, v);
                *reinterpret_cast<uint4*>(tile + dst[j]) = make_uint4(v[0], v[1], v[2], v[3]);
            }
        };
        if (more) fetch();
        while (more) {
            const int s = n % kStages;
            if (n >= kStages && !warp_wait(s_done + 16 * (NB - 1) + 8 * ((n - kStages) & 1), tile_parity(n - kStages))) {
                failed = true;
                break;
            }
            unsigned char* kt = sm + W::kOffK + s * W::kKvBytes;
            unsigned char* vt = sm + W::kOffV + s * W::kKvBytes;
            if (uw == 0 && lane == 0) {
                bad_s[n & 3] = bad;
                if (bad != 0) atomicOr(&g_kv4_window_error, kErrBadPage);
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) put(kt + i * (kStep / 8) * 1024, kc[i], ks[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_local(k_full + 8 * s);
            if (n >= kStages && !warp_wait(o_done + 16 * (NB - 1) + 8 * ((n - kStages) & 1), tile_parity(n - kStages))) {
                failed = true;
                break;
            }
#pragma unroll
            for (int i = 0; i < kMine; ++i) put(vt + i * (kStep / 8) * 1024, vc[i], vs[i]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_local(v_full + 8 * s);
            ++n;
            step();
            if (more) {
                fetch();
            }
        }
    } else if (elect_one()) {
        // -------------------------------------------------------------- products
        const uint32_t idesc_s = idesc_f16(kTok), idesc_o = idesc_f16(D) | kIdescBMnMajor;
        const uint32_t q_desc = desc_k(base), k_desc = desc_k(base + W::kOffK), v_desc = desc_mn(base + W::kOffV, W::kKvBlock);
        int units = 0;
        // S = Q K of block j, tile t
        auto first = [&](int j, int t) {
            const uint32_t k = k_desc + (t % kStages) * (W::kKvBytes >> 4);
            const uint32_t q = q_desc + j * (W::kQRows >> 4), d = tmem + 128 * j + kTok * (t % kBuffers);
            // k-steps of 16 dims, 32 bytes of a row. The rests come first: the tensor cores cut each sum off at fp32, and
            // so half of the cuts are of small numbers (error of fp32 outputs 1.7e-6 -> 1.25e-6 at 4096 tokens).
            if constexpr (SPLIT) {
#pragma unroll
                for (int i = 0; i < 4 * W::kBlk; ++i) {
                    const uint32_t ko = k + (i >> 2) * (W::kKvBlock >> 4) + 2 * (i & 3);
                    const uint32_t qo = q + (W::kQBytes >> 4) + (i >> 2) * (W::kQBlock >> 4) + 2 * (i & 3);
                    if (i == 0)
                        mma_ss<true>(d, qo, ko, idesc_s);
                    else
                        mma_ss<false>(d, qo, ko, idesc_s);
                }
            }
#pragma unroll
            for (int i = 0; i < 4 * W::kBlk; ++i) {
                const uint32_t ko = k + (i >> 2) * (W::kKvBlock >> 4) + 2 * (i & 3);
                const uint32_t qo = q + (i >> 2) * (W::kQBlock >> 4) + 2 * (i & 3);
                if (i == 0 && !SPLIT)
                    mma_ss<true>(d, qo, ko, idesc_s);
                else
                    mma_ss<false>(d, qo, ko, idesc_s);
            }
            mma_commit(s_done + 16 * j + 8 * (t & 1));
        };
        // O += P V of block j, tile t, once its probabilities are there
        auto second = [&](int j, int t, bool start) -> bool {
            if (j == 0 && !wait_for(v_full + 8 * (t % kStages), stage_parity(t))) return false;
            if (!wait_for(p_ready + 16 * j + 8 * (t & 1), tile_parity(t))) return false;
            tc_fence_after();
            const uint32_t v = v_desc + (t % kStages) * (W::kKvBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk) {
                // 32 tokens' probabilities from the first of their 32 columns, their rests from the 16th
                const uint32_t pr = tmem + 128 * j + kTok * (t % kBuffers) + 32 * (kk >> 1) + 8 * (kk & 1);
                mma_ts(tmem + W::kTmO + j * D, pr, v + kk * (2048 >> 4), idesc_o, start && kk == 0 ? 0u : 1u);
                if constexpr (SPLIT) mma_ts(tmem + W::kTmO + j * D, pr + 16, v + kk * (2048 >> 4), idesc_o, 1u);
            }
            mma_commit(o_done + 16 * j + 8 * (t & 1));
            return true;
        };
        for (; cur.left > 0 && !failed; next_unit(p, pairs, cur)) {
            int r0, r1;
            unit_tiles(p, cur, r0, r1);
            if (r1 <= r0) break;
            if (!wait_for(q_full, static_cast<uint32_t>(units) & 1u)) {
                failed = true;
                break;
            }
            ++units;
            for (int r = r0; r < r1 && !failed; ++r, ++n) {
                if (!wait_for(k_full + 8 * (n % kStages), stage_parity(n))) {
                    failed = true;
                    break;
                }
                if constexpr (kBuffers == 2) {  // the next tile's scores before this one's product with V
                    for (int j = 0; j < NB && !failed; ++j) {
                        // (the buffer's last reader, the second product of tile n - 2, has completed)
                        if (n >= 2 && !wait_for(o_done + 16 * j + 8 * (n & 1), tile_parity(n - 2))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        first(j, n);
                    }
                    for (int j = 0; j < NB && !failed; ++j)
                        if (r > r0 && !second(j, n - 1, (r - 1 - r0) % W::kFreshTiles == 0)) failed = true;
                } else {  // a block's product with V, then its next scores, while the other block's softmax runs
                    for (int j = 0; j < NB && !failed; ++j) {
                        if ((r > r0 && !second(j, n - 1, (r - 1 - r0) % W::kFreshTiles == 0)) ||
                            (n >= 1 && !wait_for(o_done + 16 * j + 8 * ((n - 1) & 1), tile_parity(n - 1)))) {
                            failed = true;
                            break;
                        }
                        tc_fence_after();
                        first(j, n);
                    }
                }
            }
            for (int j = 0; j < NB && !failed; ++j)
                if (!second(j, n - 1, (r1 - 1 - r0) % W::kFreshTiles == 0)) failed = true;
        }
        // whatever was issued has completed before the tensor memory is freed
        mma_commit(drained);
        (void)wait_for(drained, 0);
    }
    __syncwarp();
    // (in the issuing warp the elected lane alone knows, whichever it is)
    if (__any_sync(~0u, failed) && lane == 0) atomicOr(&g_kv4_window_error, kErrWaitTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, W::kTmCols);
    }
}

// Joins the partial results of the units that several CTAs shared: a column of blocks for each CTA that such a unit
// starts in. Two blocks of rows: a warp for 32 rows and 16 dims, the sums lying as [dim / 4][row][4], so that a warp here
// reads, and the softmax warps wrote, whole lines. One block: a warp for each row, the sums lying as [row][dim]; units of
// few rows have more parts. 2 x 1024 tokens after 8000, 32 heads of 128: 310 us by the first way, 321 us by the second
// (of 64: 234 and 241, from position 0: 76 and 82); 16 ragged windows of 8 tokens with 5 heads: 51 and 49 us, 32 tokens
// after 30000: 64 and 60 us. By rows, CTAs per unit: the last case takes 137 / 95 / 74 us with 4 / 8 / 16, and 61 us with
// a part's factor computed once, by one lane.
template <int D, int NB>
__global__ void __launch_bounds__(256) kv4_window_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr size_t unit = NB * kRows, slot_floats = unit * (D + 2);
    const int lane = threadIdx.x & 31;
    griddep_wait();
    const JoinRecord rec = reinterpret_cast<const JoinRecord*>(p.records)[blockIdx.x];
    if (rec.parts == 0) return;
    WinCursor k{rec.b, rec.block, rec.pair, 0, 0, 0};
    const Unit x = win_unit(p, k);
    const int rows = min(x.n * p.group - x.col0, p.unit_rows);
    const float* base = p.part + static_cast<size_t>(blockIdx.x) * 2 * slot_floats;
    auto slot = [&](int i) -> const float* {
        return base + (i == 0 ? 1 : 2 * static_cast<size_t>(i)) * slot_floats;
    };
    if constexpr (NB == 2) {
        const int items = (rows + 31) / 32 * (D / 16);
        for (int item = blockIdx.y * 8 + (threadIdx.x >> 5); item < items; item += gridDim.y * 8) {
            const int row = item / (D / 16) * 32 + lane, c = item % (D / 16) * 16;
            if (row >= rows) continue;
            float mm = -INFINITY;
#pragma unroll 8
            for (int i = 0; i < rec.parts; ++i) mm = fmaxf(mm, slot(i)[unit * D + row]);
            float o[16] = {}, l = 0.0f;
#pragma unroll 4
            for (int i = 0; i < rec.parts; ++i) {
                const float* s = slot(i);
                const float ms = s[unit * D + row];
                const float f = ms == -INFINITY ? 0.0f : exp2_approx(ms - mm);
                l += s[unit * D + unit + row] * f;
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(s + (c + j) * unit + 4 * row);
                    o[j] += y.x * f;
                    o[j + 1] += y.y * f;
                    o[j + 2] += y.z * f;
                    o[j + 3] += y.w * f;
                }
            }
            store_out16(p, q_row(p, k.b, x, x.col0 + row) + c, o, l > 0.0f || l != l ? 1.0f / l : 0.0f);
        }
        return;
    }
    for (int row = blockIdx.y * 8 + (threadIdx.x >> 5); row < rows; row += gridDim.y * 8) {
        // a lane has the maximum and sum of every 32nd part; a part's factor is asked of its lane
        float ms = lane < rec.parts ? slot(lane)[unit * D + row] : -INFINITY;
        float ls = lane < rec.parts ? slot(lane)[unit * D + unit + row] : 0.0f;
        float mm = ms;
        for (int i = lane + 32; i < rec.parts; i += 32) mm = fmaxf(mm, slot(i)[unit * D + row]);
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
        float2 v[D / 64];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) v[c] = make_float2(0.0f, 0.0f);
        float l = 0.0f;
        for (int first = 0; first < rec.parts; first += 32) {
            const int n = min(32, rec.parts - first);
            if (first > 0) {
                ms = lane < n ? slot(first + lane)[unit * D + row] : -INFINITY;
                ls = lane < n ? slot(first + lane)[unit * D + unit + row] : 0.0f;
            }
            const float factor = ms == -INFINITY ? 0.0f : exp2_approx(ms - mm);
            l += ls * factor;
#pragma unroll 8
            for (int i = 0; i < n; ++i) {
                const float f = __shfl_sync(~0u, factor, i);
                const float* s = slot(first + i) + row * D + 2 * lane;
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    const float2 y = *reinterpret_cast<const float2*>(s + 64 * c);
                    v[c].x += y.x * f;
                    v[c].y += y.y * f;
                }
            }
        }
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
        const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
        const size_t out = q_row(p, k.b, x, x.col0 + row) + 2 * lane;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) store_out2(p, out + 64 * c, v[c].x * inv, v[c].y * inv);
    }
}

constexpr int kMaxSms = 192;  // the workspace is sized for cards of up to as many

template <int D, bool SPLIT, int NB>
cudaError_t launch_one(AttnParams p, cudaStream_t stream) {
    using W = Win<D, SPLIT, NB>;
    p.unit_rows = W::kUnitRows;
    p.tile_shift = W::kTok == 128 ? 7 : 6;
    p.col_blocks = static_cast<int>((static_cast<long long>(p.c.T) * p.group + W::kUnitRows - 1) / W::kUnitRows);
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(kv4_window_kernel<D, SPLIT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    static_assert(W::kCtas * (W::kSmem + 1024) <= 233472, "the CTAs of an SM fit its shared memory");
    const int ctas = W::kCtas * std::min(sms, kMaxSms);
    kv4_window_kernel<D, SPLIT, NB><<<ctas, W::kThreads, W::kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long rows = std::min<long long>(static_cast<long long>(p.c.T) * p.group, W::kUnitRows);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, static_cast<unsigned>(NB == 2
                                                       ? ((rows + 31) / 32 * (D / 16) + 7) / 8
                                                       : std::min<long long>((rows + 7) / 8, 16)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_window_join_kernel<D, NB>, p);
}

template <int D>
cudaError_t launch_dim(const AttnParams& p, cudaStream_t stream) {
    const bool split = p.dtype == DType::kF32;
    if constexpr (D <= 128) {
        if (!split && static_cast<long long>(p.c.T) * p.group > kRows) return launch_one<D, false, 2>(p, stream);
    }
    return split ? launch_one<D, true, 1>(p, stream) : launch_one<D, false, 1>(p, stream);
}

}  // namespace

size_t kv4_window_workspace_bytes(int head_dim) {
    return static_cast<size_t>(2 * kMaxSms) * ((2 * kRows * (head_dim + 2) + kRows * head_dim) * sizeof(float) + sizeof(JoinRecord));
}

cudaError_t launch_kv4_window(AttnParams p, cudaStream_t stream) {
    p.sums = p.part + static_cast<size_t>(2 * kMaxSms) * 2 * kRows * (p.c.head_dim + 2);
    p.records = p.sums + static_cast<size_t>(2 * kMaxSms) * kRows * p.c.head_dim;
    switch (p.c.head_dim) {
        case 64: return launch_dim<64>(p, stream);
        case 128: return launch_dim<128>(p, stream);
        case 256: return launch_dim<256>(p, stream);
        default: return cudaErrorInvalidValue;
    }
}

cudaError_t read_kv4_window_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_window_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_window_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace gdn
