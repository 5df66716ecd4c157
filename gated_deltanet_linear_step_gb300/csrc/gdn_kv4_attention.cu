// gdn_kv4_attention.cu - attention of a window's queries over the 4-bit cache
// (format and pages: gdn_kv4.cuh), streaming the cache once:
//
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q . k_j,  j <= start + t
//
// with the running maximum m and sum of a softmax, in one pass over the keys.
//
// What bounds it. A cached element is 4.5 bits, so at the HBM rate an SM takes in
// about 42 of them per clock and has about 3 issue slots of a lane for each: the
// unpacking is what has to be cheap. One warp owns a tile of tokens; its lanes
// unpack codes in registers in exactly the fragment order of mma.m16n8k16, with
// the cache as the A operand and the (few) queries as the 8 columns of B: a
// single token's query heads waste less of an 8-wide side than of a 128-row
// tile of the tensor memory, which would also need the unpacked values written
// to shared memory first. A code byte becomes an fp16 pair by one conversion and
// is scaled by one multiplication; both are exact (6 significant bits).
//
// Fragment orders (lane = 4 g + t4). Which head dimension or token a fragment's
// index stands for is free as long as both operands agree, so they are chosen for
// 16-byte contiguous reads:
//  - S^T = K Q^T: row r of an 8-row half is token pi8(r); of a row lane t4 holds the
//    contiguous dims 32 t4 .. (D = 128), 4 per k-step.
//  - O^T = V^T P^T: k index pair (2 t4, 2 t4 + 1) is the token pair (pi8(2 t4), pi8(2 t4 + 1));
//    lane g holds the D/8 contiguous dims from g D/8 of both tokens, and interleaving
//    the nibbles of the two tokens' words gives bytes that convert straight to the
//    (token, next token) pairs of A. The P fragment comes from the S accumulators by movmatrix.
//
// Numerics. Queries are scaled by a power of two per row to fill fp16's range
// (16-bit inputs stay exact down to 2^-25 of the row's largest, bf16 ones to 2^-28; fp32 ones are split into fp16 hi + lo, 22
// bits; fp16's smallest step leaves 2^-36 of the row's largest of any element);
// scores, maxima, sums and outputs are fp32. Probabilities are rounded to fp16
// (half a step is 2^-12 of the value, below the 2^-9 of a bf16 output; the reference maximum stands for 2^9, so that small ones
// keep their bits) or, for fp32, split into hi + lo. Below 2^-23 (hi + lo: 2^-12) of the row's largest they lose bits to fp16's
// smallest step, 2^-34 of the largest at most. Masked keys take no part: their
// scores are set to -inf by a select, and the scales of tokens past the end
// are set to zero, so whatever such bytes hold (infinities, NaN) does not matter.
//
// Work split. A unit is (sequence, layer, kv head) with all its query rows (16 at most: one or two column tiles), its
// tiles are cut into rounds of one tile per warp, and the rounds of all units are
// laid end to end and dealt out evenly to the CTAs, whatever the mix of lengths.
// A unit that crosses a CTA boundary leaves partial sums in the workspace, and a
// second small kernel joins them in order: no atomics, so results do not
// depend on timing.
//
// Each warp fills its own ring of tiles by 16-byte asynchronous copies (four bulk copies of a tile's pieces, each by
// its own lane, cost more instructions). No warp waits for another but at the joins, and nothing spins.
//
// Measured: 64 sequences of 16384 tokens, 8 kv heads of 128, fp16: 207 us, 0.86 of the time that the cache alone takes
// at the measured HBM rate; 4 x 131000 tokens, 2 heads of 256: 64 us (0.69); 64 sequences of mixed lengths up to 8192:
// 42 us (0.49: the start of the kernel, of each unit and the joins take about 15 us); one sequence of 500: 10 us
// with the joining kernel, a chain of dependent reads (lengths, block table, tile) and the joins.

#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_kv4_attention.cuh"
#include "gdn_tc.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = 32 * kWarps;

__device__ unsigned int g_kv4_attn_error = 0;

// A warp's tile: kTokens tokens of one kv head, K codes | V codes | K scales | V scales.
template <int D>
struct Tile {
    static constexpr int kTokens = D == 256 ? 32 : 64;
    static constexpr int kRow = D / 2;      // code bytes of a token
    static constexpr int kBlocks = D / 16;  // scales of a token
    static constexpr uint32_t kCodeBytes = kTokens * kRow;
    static constexpr uint32_t kScaleBytes = kTokens * kBlocks;
    static constexpr uint32_t kBytes = 2 * (kCodeBytes + kScaleBytes);
};

// Token of row r of an 8-row half tile.
__device__ __forceinline__ int pi8(int r) { return r ^ ((r >> 1) & 1); }

// ------------------------------------------------------------ work split --
// The units lie end to end on a line: each takes kUnitCost places for its start (its queries are read, its
// warps joined) and then one per round. CTA i of n has the places [total i / n, total (i + 1) / n) and does the
// rounds among them. Without the places for starts a CTA of 20 rounds could get 20 one-round sequences. A batch of
// 64 sequences of mixed lengths up to 8192 takes 45 / 42 / 43 us with 1 / 2 / 3 places.
constexpr int kUnitCost = 2;

// raise() without branches but for a warp's (three answers to one question of 1500 tokens, fp32: 28.7 us, with branches 30.0).
template <class F>
__device__ __forceinline__ float raise_column(float top, float& m, float& mul, float& shift, F first_mul) {
    const float old = m, v = fmaxf(m, top * mul);
    float al = v == m ? 1.0f : exp2_approx(m - v), next = v == -INFINITY ? kNone : kPShift - v;
    m = v;
    const bool was = is_big(old);
    if (__any_sync(~0u, was || is_big(v))) {
        const float first = first_mul();
        const bool stays = was && !is_over(top, mul, shift);
        m = !was ? v : stays ? old : fmaxf(old, top * first);
        al = !was ? al : stays ? 1.0f : 0.0f;
        const float power = big_factor(top);
        next = stays ? shift : is_big(m) ? -top * power : was ? kPShift - m : next;
        mul = stays ? mul : is_big(m) ? power : first;
    }
    shift = next;
    return al;
}

// Places of one unit of sequence b (0: no token).
template <int D, class P>
__device__ __forceinline__ int seq_cost(const P& p, int b) {
    const Kv4Window w = attn_window(p, b);
    if (w.n == 0) return 0;
    const int end = max(w.start + min(causal(p) ? w.n : 1, w.cap - w.start), 1);  // one round at least: its rows get their zeros
    constexpr int kRound = Tile<D>::kTokens * kWarps;
    return kUnitCost + (end + kRound - 1) / kRound;
}

// Where a CTA is: unit u of sequence b (cost places long), at place `at` of it, with `left` places to go.
struct Cursor {
    int b, u, cost, at;
    long long left;
};

// Places of all sequences' units (of one unit each), by one warp.
template <int D, class P>
__device__ __forceinline__ long long all_costs(const P& p, int lane) {
    long long s = 0;
    for (int b = lane; b < p.c.B; b += 32) s += seq_cost<D>(p, b);
    if (p.c.B == 1) return __shfl_sync(~0u, s, 0);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    return s;
}

// The unit and place in it of place x of the line (units per sequence: `units`), by one warp.
template <int D, class P>
__device__ __forceinline__ Cursor locate(const P& p, int units, long long x, int lane) {
    Cursor k;
    k.b = p.c.B;
    k.u = k.cost = k.at = 0;
    k.left = 0;
    long long before = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const int mine = b0 + lane < p.c.B ? seq_cost<D>(p, b0 + lane) : 0;
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(~0u, (before + sum) * units > x);
        if (hit != 0) {
            const int src = __ffs(hit) - 1;
            k.b = b0 + src;
            k.cost = __shfl_sync(~0u, mine, src);
            const long long base = (before + __shfl_sync(~0u, sum, src) - k.cost) * units;
            k.u = static_cast<int>(mul_div(x - base, 1, k.cost));
            k.at = static_cast<int>((x - base) - static_cast<long long>(k.u) * k.cost);
            return k;
        }
        before += __shfl_sync(~0u, sum, 31);
    }
    return k;
}

// The rounds [r0, r1) of the cursor's unit that are its CTA's.
__device__ __forceinline__ void unit_rounds(const Cursor& k, int& r0, int& r1) {
    r0 = max(k.at - kUnitCost, 0);
    r1 = static_cast<int>(min(static_cast<long long>(k.cost), k.at + k.left)) - kUnitCost;
}

// On to the next unit.
template <int D, class P>
__device__ __forceinline__ void advance(const P& p, int units, Cursor& k) {
    k.left -= k.cost - k.at;
    k.at = 0;
    if (++k.u < units || k.left <= 0) return;
    k.u = 0;
    do {
        ++k.b;
    } while (k.b < p.c.B && (k.cost = seq_cost<D>(p, k.b)) == 0);
}

template <class P>
__device__ __forceinline__ Unit unit_of(const P& p, int b, int u) {
    Unit x;
    x.h = u % p.c.kv_heads;
    x.l = u / p.c.kv_heads;
    x.col0 = 0;
    const Kv4Window w = attn_window(p, b);
    x.start = w.start;
    x.n = w.n;
    x.end = w.start + min(causal(p) ? w.n : 1, w.cap - w.start);
    return x;
}

// ---------------------------------------------------------------- pieces --
// Waits until at most N of this thread's committed cp.async groups are still in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Byte i (0 or 1) of a and of b as the halves of an fp16 pair of scales.
template <int D>
__device__ __forceinline__ uint32_t scale_both(uint32_t a, uint32_t b, int i) {
    if constexpr (D < 256) return __byte_perm(a, b, 0x5410) << 7;  // a and b have one byte each
    return (__byte_perm(a, b, i ? 0x5511 : 0x4400) & 0x00FF00FFu) << 7;
}

// Output sums lie permuted: pair (i, g) of the dims (D/8) g + 2 i + {0, 1} is at 16 i + 2 g.
template <int D>
__device__ __forceinline__ int dim_of(int pos) {
    return (D / 8) * ((pos >> 1) & 7) + 2 * (pos >> 4) + (pos & 1);
}

// ---------------------------------------------------------------- kernel --
// Resident CTAs per SM, as a block's registers and shared memory allow, and tiles in a warp's ring. 64 sequences of
// 16384 tokens, 8 heads of 128, one query token: tiles of 32 tokens 223 us (3 CTAs, 3 tiles) and 228 us (4 CTAs,
// 2 tiles, 128 registers), of 64 tokens 210 us (2 CTAs, 2 tiles) and 204 us (3 CTAs, 2 tiles): the work per tile that
// does not depend on its length is a third of a 32-token tile's instructions.
template <int D, int NT, bool SPLIT>
struct Shape {
    static constexpr int kCtas = D <= 128 && NT == 1 && !SPLIT ? 3 : 2;
    static constexpr int kStages = 2;
};

template <int D, int NT, bool SPLIT>
struct Smem {
    static constexpr int kStages = Shape<D, NT, SPLIT>::kStages;
    static constexpr int kCols = 8 * NT;
    static constexpr uint32_t kRedStride = D + 8;  // floats: bank spread of the lanes' pairs
    static constexpr uint32_t kQBytes = kCols * D * 2 * (SPLIT ? 2 : 1);
    static constexpr uint32_t kOffQ = kWarps * kStages * Tile<D>::kBytes;
    static constexpr uint32_t kOffCol = kOffQ + kQBytes;                   // maxima and sums: [warp][col] twice
    static constexpr uint32_t kOffMul = kOffCol + 2 * kWarps * kCols * 4;  // per column: scale of the raw scores
    static constexpr uint32_t kOffBad = kOffMul + kCols * 4;               // per stage: pages that are not there
    static constexpr uint32_t kOffRed = kOffBad + kWarps * kStages * 4;    // per warp: its stage with its sums, or -1
    static constexpr uint32_t kOffRuns = kOffRed + kWarps * 4;             // maxima and sums of the columns over earlier runs, twice; runs
    static constexpr uint32_t kBytes = kOffRuns + 2 * 2 * kCols * 4 + 16;
    static_assert(8 * kRedStride * 4 <= Tile<D>::kBytes, "eight columns of sums fit a stage");
};

template <int D, int NT, bool SPLIT, class P>
__global__ void __launch_bounds__(kAttnThreads, Shape<D, NT, SPLIT>::kCtas)
    kv4_attention_kernel(const __grid_constant__ P p) {
    using S = Smem<D, NT, SPLIT>;
    using TL = Tile<D>;
    constexpr int kStages = S::kStages;
    constexpr int kCols = S::kCols;
    constexpr int kTokens = TL::kTokens, kHalfTiles = kTokens / 16;  // m16 tiles of a tile
    constexpr int kRound = kTokens * kWarps;
    constexpr int kMTiles = D / 16;
    // Sums start afresh every 1024 steps of 16 tokens (65536 tokens of a unit) and are added up with fp32 instructions in the
    // CTA's part of the workspace: what the tensor cores cut off at every step, and what rounding leaves of a lane's sum of
    // probabilities, would grow with the row otherwise. Rows of equal values, not split: fp16 outputs over 2^20 keys 2.2e-3
    // without, 7.4e-4 with (half of fp16's step and the probabilities' are 7.3e-4); fp32 over 2^19 keys 7.7e-5 and 6.8e-6.
    constexpr int kFreshRounds = 1024 / kHalfTiles;
    constexpr bool kQRegs = NT == 1 && !SPLIT && D <= 128;  // the query fragments stay in registers
    extern __shared__ __align__(128) unsigned char sm[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    float* col_m = reinterpret_cast<float*>(sm + S::kOffCol);
    float* col_l = col_m + kWarps * kCols;
    float* mul_s = reinterpret_cast<float*>(sm + S::kOffMul);
    float* runs_s = reinterpret_cast<float*>(sm + S::kOffRuns);
    int* run_s = reinterpret_cast<int*>(runs_s + 2 * 2 * kCols);
    uint32_t* bad_s = reinterpret_cast<uint32_t*>(sm + S::kOffBad) + warp * kStages;
    int* red_s = reinterpret_cast<int*>(sm + S::kOffRed);
    unsigned char* ring = sm + warp * kStages * TL::kBytes;
    if (some_group_falls(p)) atomicOr(&g_kv4_attn_error, kErrBadBorders);
    const int units = p.c.L * p.c.kv_heads;
    const long long total = all_costs<D>(p, lane) * units;
    const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    JoinRecord* record = reinterpret_cast<JoinRecord*>(p.records) + blockIdx.x;
    if (tid == 0) {
        *record = JoinRecord{0, 0, 0, 0};
        *run_s = 0;
    }
    if (static_cast<int>(blockIdx.x) >= ctas) {
        wait_for_prefixes(p);
        return;
    }
    long long lo, hi;
    cta_range(total, blockIdx.x, ctas, lo, hi);
    Cursor cur = locate<D>(p, units, lo, lane);
    cur.left = hi - lo;

    // --- requests: 16 bytes per lane and copy, 512 of codes at a time; lane j looks up page j of the tile
    const int psize = 1 << p.c.page_shift;
    const int piece_shift = min(p.c.page_shift, 31 - __clz(kTokens));
    const int n_pages = kTokens >> piece_shift;  // of a tile
    const uint32_t head_bytes = static_cast<uint32_t>(kv4_head_bytes(psize, D)), page_bytes = head_bytes * p.c.kv_heads;
    // a lane's place in the first copy of the scales: of K in the lower half (D < 256: K and V in one copy)
    const uint32_t scale_lane = TL::kScaleBytes == 256 ? (lane & 15) * 16 + (lane >> 4) * (head_bytes / 2) : lane * 16;
    const uint32_t ring_addr = smem_addr(ring) + lane * 16;
    Cursor ahead = cur;     // unit of the next tile
    int a_seg = 0;          // rounds of that unit left in this CTA
    int a_p0 = 0, a_end = 0;
    int a_page = -1;        // block table entry of the tile's page; of page `lane` if it has several
    const int32_t* a_table = nullptr;
    const uint8_t* a_head = nullptr;
    bool ready = false;     // there is a next tile
    // The warp's next tile: its page's number is read here, a tile ahead of its use.
    auto look = [&]() {
        while (a_p0 >= a_end || a_seg <= 0) {  // on to the next unit in which the warp has a tile
            if (ahead.left <= 0) {
                ready = false;
                return;
            }
            const Unit u = unit_of(p, ahead.b, ahead.u);
            a_end = u.end;
            a_head = p.c.cache + (static_cast<size_t>(u.l) * p.c.n_pages * p.c.kv_heads + u.h) * head_bytes;
            a_table = p.c.block_table + static_cast<size_t>(ahead.b) * p.c.max_pages;
            int r0, r1;
            unit_rounds(ahead, r0, r1);
            a_seg = r1 - r0;
            a_p0 = r0 * kRound + warp * kTokens;
            advance<D>(p, units, ahead);
        }
        ready = true;
        const int slot = (a_p0 >> p.c.page_shift) + (n_pages == 1 ? 0 : lane);
        a_page = n_pages == 1 || (lane < n_pages && a_p0 + (lane << piece_shift) < a_end) ? __ldg(a_table + slot) : 0;
    };
    uint32_t issued = 0, used = 0;  // this warp's tiles
    auto issue = [&]() {
        if (ready) {
            const uint32_t s = issued % kStages;
            const bool gone = static_cast<uint32_t>(a_page) >= static_cast<uint32_t>(p.c.n_pages);
            const int a_row = a_p0 & (psize - 1);
            const unsigned bad = n_pages == 1 ? (gone ? 1u : 0u) : __ballot_sync(~0u, gone);
            if (lane == 0) bad_s[s] = bad;
            if (gone) a_page = -1;
            const uint32_t dst = ring_addr + s * TL::kBytes;
            const uint32_t half = static_cast<uint32_t>(head_bytes / 2), scales = psize * TL::kRow;
            constexpr int kCopies = TL::kCodeBytes / 512, kRows = 512 / TL::kRow;  // of K or V codes; rows of a copy
            constexpr int kScaleCopies = 2 * TL::kScaleBytes / 512;                // K's, then V's
            if (n_pages == 1) {
                if (!gone) {
                    const uint8_t* src = a_head + static_cast<unsigned long long>(static_cast<uint32_t>(a_page)) * page_bytes;
                    const uint8_t* k = src + a_row * TL::kRow + lane * 16;
                    const uint8_t* v = k + half;
#pragma unroll
                    for (int i = 0; i < kCopies; ++i) {
                        cp_async16(dst + i * 512, k + i * 512);
                        cp_async16(dst + TL::kCodeBytes + i * 512, v + i * 512);
                    }
                    const uint8_t* c = src + scales + a_row * TL::kBlocks + scale_lane;
#pragma unroll
                    for (int i = 0; i < kScaleCopies; ++i)
                        cp_async16(dst + 2 * TL::kCodeBytes + i * 512, kScaleCopies == 1 ? c : c + i * half);
                }
            } else {  // pages end between copies
#pragma unroll 1
                for (int i = 0; i < kCopies; ++i) {
                    const int j = (i * kRows) >> piece_shift;
                    const int page = __shfl_sync(~0u, a_page, j);
                    const uint8_t* k = a_head + static_cast<unsigned long long>(static_cast<uint32_t>(page)) * page_bytes +
                                       (i * kRows - (j << piece_shift)) * TL::kRow + lane * 16;
                    if (page >= 0) {
                        cp_async16(dst + i * 512, k);
                        cp_async16(dst + TL::kCodeBytes + i * 512, k + half);
                    }
                }
#pragma unroll 1
                for (int i = 0; i < kScaleCopies; ++i) {
                    const int at = (i * 512 + lane * 16) & (TL::kScaleBytes - 1), part = (i * 512 + lane * 16) / TL::kScaleBytes;
                    const int row = at / TL::kBlocks, j = row >> piece_shift;
                    const int page = __shfl_sync(~0u, a_page, j);
                    if (page >= 0)
                        cp_async16(dst + 2 * TL::kCodeBytes + i * 512,
                                   a_head + static_cast<unsigned long long>(static_cast<uint32_t>(page)) * page_bytes +
                                       part * half + scales + (row - (j << piece_shift)) * TL::kBlocks + (at & (TL::kBlocks - 1)));
                }
            }
            ++issued;
            a_p0 += kRound;
            --a_seg;
            look();
        }
        cp_async_commit();  // one group per place in the ring, empty or not
    };
    look();
    for (int s = 0; s < kStages; ++s) issue();
    griddep_launch_dependents();  // the join's CTAs may come up; they wait for this grid's end

    // --- where this lane reads a tile (rows 8 and 16 further have the same swizzle)
    const int ka = pi8(g), v0 = pi8(2 * t4), v1 = pi8(2 * t4 + 1);
    const uint32_t k_off = ka * TL::kRow + (D >= 128 ? ((2 * t4) ^ kv4_swizzle(ka, TL::kBlocks)) * 8 : t4 * 8);
    const uint32_t k_off2 = ka * TL::kRow + ((8 + 2 * t4) ^ kv4_swizzle(ka, TL::kBlocks)) * 8;  // D = 256: its second half
    const uint32_t ks_off = 2 * TL::kCodeBytes + ka * TL::kBlocks + (D >= 128 ? 2 * t4 : t4);
    auto v_at = [&](int row) -> uint32_t {
        if constexpr (D == 256) return row * TL::kRow + ((2 * g) ^ kv4_swizzle(row, TL::kBlocks)) * 8;
        if constexpr (D == 128) return row * TL::kRow + (g ^ kv4_swizzle(row, TL::kBlocks)) * 8;
        return row * TL::kRow + g * 4;
    };
    const uint32_t v_off0 = TL::kCodeBytes + v_at(v0), v_off1 = TL::kCodeBytes + v_at(v1);
    const int vs_lane = D == 256 ? 2 * g : D == 128 ? g : g >> 1;
    const uint32_t vs_off0 = 2 * TL::kCodeBytes + TL::kScaleBytes + v0 * TL::kBlocks + vs_lane;
    const uint32_t vs_off1 = 2 * TL::kCodeBytes + TL::kScaleBytes + v1 * TL::kBlocks + vs_lane;

    while (cur.left > 0) {
        const Unit x = unit_of(p, cur.b, cur.u);
        const int b = cur.b;
        int r0, r1;
        unit_rounds(cur, r0, r1);
        if (r1 <= r0) break;  // its start alone, at the end of the CTA's places
        r1 = min(r1, r0 + kFreshRounds);

        // --- queries of the unit: B fragments in shared memory, or straight in registers
        const int all_cols = x.n * p.group;  // columns that exist
        if (tid == 0 && attn_runs_out(p, b)) atomicOr(&g_kv4_attn_error, kErrBadPage);
        uint2 qr[kQRegs ? D / 16 : 1];
        float col_mul = 0.0f;  // of column g
        if constexpr (kQRegs) {
            constexpr int kSpan = D / 4;  // contiguous dims of a lane
            float4 v[D / 16];
            float a = 0.0f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (g < all_cols) v[i] = load_q4(p, q_row(p, b, x, g) + kSpan * t4 + 4 * i);
                a = fmaxf(fmaxf(a, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
            }
            a = fmaxf(a, __shfl_xor_sync(~0u, a, 1));
            a = fmaxf(a, __shfl_xor_sync(~0u, a, 2));
            const float f = row_factor(a);
            col_mul = score_factor(p.scale, f);
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                qr[i] = make_uint2(pack_half2(v[i].x * f, v[i].y * f), pack_half2(v[i].z * f, v[i].w * f));
        } else {
            __syncthreads();
            for (int c = warp; c < kCols; c += kWarps) {
                constexpr int kChunks = D > 128 ? D / 128 : 1;
                float4 v[kChunks];
                float a = 0.0f;
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (c < all_cols && 4 * lane + 128 * i < D) v[i] = load_q4(p, q_row(p, b, x, c) + 128 * i + 4 * lane);
                    a = fmaxf(fmaxf(a, fmaxf(fabsf(v[i].x), fabsf(v[i].y))), fmaxf(fabsf(v[i].z), fabsf(v[i].w)));
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
                const float f = row_factor(a);
                if (lane == 0) mul_s[c] = score_factor(p.scale, f);
#pragma unroll
                for (int i = 0; i < kChunks; ++i) {
                    if (4 * lane + 128 * i >= D) continue;
                    constexpr int kPerT4 = D >= 128 ? 8 : 4;  // k-steps of a lane's contiguous dims
                    const int st = 8 * i + (lane & (kPerT4 - 1)), tt = lane / kPerT4;
                    const float q0 = v[i].x * f, q1 = v[i].y * f, q2 = v[i].z * f, q3 = v[i].w * f;
                    const uint32_t at = ((st * NT + (c >> 3)) * 32 + (c & 7) * 4 + tt) * 8;
                    uint2 w = make_uint2(pack_half2(q0, q1), pack_half2(q2, q3));
                    *reinterpret_cast<uint2*>(sm + S::kOffQ + at) = w;
                    if constexpr (SPLIT)
                        *reinterpret_cast<uint2*>(sm + S::kOffQ + kCols * D * 2 + at) =
                            make_uint2(pack_rest(q0, q1, w.x), pack_rest(q2, q3, w.y));
                }
            }
            __syncthreads();
        }

        auto first_mul = [&](int c) -> float { return kQRegs ? __shfl_sync(~0u, col_mul, (c & 7) * 4) : mul_s[c]; };  // of column c's raw scores
        float m[NT][2], shift[NT][2], ls[NT][2], mul[NT][2];
        int lim[NT][2];  // last position that the column sees
        float o[kMTiles][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = 8 * nt + 2 * t4 + j;
                m[nt][j] = -INFINITY;
                shift[nt][j] = kNone;
                ls[nt][j] = 0.0f;
                mul[nt][j] = first_mul(c);
                lim[nt][j] = c < all_cols ? min(x.start + causal(p) * (c / p.group), x.end - 1) : -1;
            }
#pragma unroll
        for (int i = 0; i < kMTiles; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;
        // positions below this are seen by every column that exists (the others' results are not used)
        const int seen_by_all = min(x.start + 1, x.end);
        bool owed = false;  // a consumed stage is not yet refilled
        int freed = -1;     // the last consumed stage

        for (int r = r0; r < r1; ++r) {
            const int p0 = r * kRound + warp * kTokens;
            if (p0 >= x.end) break;
            if (owed) issue();
            owed = false;
            const uint32_t s = used % kStages;
            cp_async_wait<kStages - 1>();
            __syncwarp();  // every lane's copies of the stage have landed
            const unsigned char* st = ring + s * TL::kBytes;
            const uint32_t bad = bad_s[s];
            const bool whole = p0 + kTokens <= seen_by_all && bad == 0;

            // --- S^T = K Q^T
            float sc[kHalfTiles][NT][4];
#pragma unroll
            for (int mt = 0; mt < kHalfTiles; ++mt) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sc[mt][nt][j] = 0.0f;
                constexpr int kHalves = D > 128 ? D / 128 : 1;
#pragma unroll
                for (int hf = 0; hf < kHalves; ++hf) {
                    constexpr int kWords = D >= 128 ? 4 : 2;
                    uint32_t wa[kWords], wb[kWords];
                    uint32_t da, db;  // scale bytes of the lane's blocks
                    const unsigned char* kp = st + (hf == 0 ? k_off : k_off2) + mt * 16 * TL::kRow;
                    const unsigned char* sp = st + ks_off + 8 * hf + mt * 16 * TL::kBlocks;
                    if constexpr (D >= 128) {
                        const uint4 va = *reinterpret_cast<const uint4*>(kp);
                        const uint4 vb = *reinterpret_cast<const uint4*>(kp + 8 * TL::kRow);
                        wa[0] = va.x, wa[1] = va.y, wa[2] = va.z, wa[3] = va.w;
                        wb[0] = vb.x, wb[1] = vb.y, wb[2] = vb.z, wb[3] = vb.w;
                        da = *reinterpret_cast<const uint16_t*>(sp);
                        db = *reinterpret_cast<const uint16_t*>(sp + 8 * TL::kBlocks);
                    } else {
                        const uint2 va = *reinterpret_cast<const uint2*>(kp);
                        const uint2 vb = *reinterpret_cast<const uint2*>(kp + 8 * TL::kRow);
                        wa[0] = va.x, wa[1] = va.y;
                        wb[0] = vb.x, wb[1] = vb.y;
                        da = sp[0];
                        db = sp[8 * TL::kBlocks];
                    }
#pragma unroll
                    for (int w = 0; w < kWords; ++w) {
                        uint32_t a[4], c[4];
                        unpack(wa[w], scale_twice(da, w >> 1), a);
                        unpack(wb[w], scale_twice(db, w >> 1), c);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const int step = 8 * hf + 2 * w + k;
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                const uint32_t at = ((step * NT + nt) * 32 + lane) * 8;
                                uint2 qh;
                                if constexpr (kQRegs)
                                    qh = qr[step];
                                else
                                    qh = *reinterpret_cast<const uint2*>(sm + S::kOffQ + at);
                                mma_f16(sc[mt][nt], a[2 * k], c[2 * k], a[2 * k + 1], c[2 * k + 1], qh.x, qh.y);
                                if constexpr (SPLIT) {
                                    const uint2 ql = *reinterpret_cast<const uint2*>(sm + S::kOffQ + kCols * D * 2 + at);
                                    mma_f16(sc[mt][nt], a[2 * k], c[2 * k], a[2 * k + 1], c[2 * k + 1], ql.x, ql.y);
                                }
                            }
                        }
                    }
                }
            }

            // --- masks; the reference maximum is raised when a score is well above it
            if (!whole) {
#pragma unroll
                for (int mt = 0; mt < kHalfTiles; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const int row = 16 * mt + 8 * hf + ka;
                        const bool gone = (bad >> (row >> piece_shift)) & 1u;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                if (p0 + row > lim[nt][j] || gone) sc[mt][nt][2 * hf + j] = -INFINITY;
                    }
            }
            float top[NT][2];
            bool over = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v = fmaxf(sc[0][nt][j], sc[0][nt][2 + j]);
#pragma unroll
                    for (int mt = 1; mt < kHalfTiles; ++mt) v = fmaxf(v, fmaxf(sc[mt][nt][j], sc[mt][nt][2 + j]));
                    top[nt][j] = v;
                    over = over || is_over(v, mul[nt][j], shift[nt][j]);
                }
            if (__any_sync(~0u, over)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float al[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float v = top[nt][j];
#pragma unroll
                        for (int q = 4; q < 32; q <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, q));
                        al[j] = raise_column(v, m[nt][j], mul[nt][j], shift[nt][j], [&]() { return first_mul(8 * nt + 2 * t4 + j); });
                        ls[nt][j] *= al[j];
                    }
#pragma unroll
                    for (int i = 0; i < kMTiles; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) o[i][nt][j] *= al[j & 1];
                }
            }
            uint32_t ph[kHalfTiles][NT][2], pl[kHalfTiles][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int mt = 0; mt < kHalfTiles; ++mt)
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const float e0 = exp2_approx(fmaf(sc[mt][nt][2 * hf], mul[nt][0], shift[nt][0]));
                        const float e1 = exp2_approx(fmaf(sc[mt][nt][2 * hf + 1], mul[nt][1], shift[nt][1]));
                        ls[nt][0] += e0;
                        ls[nt][1] += e1;
                        const uint32_t w = pack_half2(e0, e1);
                        ph[mt][nt][hf] = transpose8(w);
                        if constexpr (SPLIT) pl[mt][nt][hf] = transpose8(pack_rest(e0, e1, w));
                    }

            // --- O^T += V^T P^T
#pragma unroll
            for (int mt = 0; mt < kHalfTiles; ++mt) {
                // the lane's four tokens: k indices 2 t4, 2 t4 + 1, and both + 8
                constexpr int kWords = D / 64;  // words of a lane's D/8 dims
                uint32_t w[4][kWords];
                uint32_t sb[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const unsigned char* v = st + ((k & 1) ? v_off1 : v_off0) + (16 * mt + 8 * (k >> 1)) * TL::kRow;
                    const unsigned char* sv = st + ((k & 1) ? vs_off1 : vs_off0) + (16 * mt + 8 * (k >> 1)) * TL::kBlocks;
                    if constexpr (D == 256) {
                        const uint4 u = *reinterpret_cast<const uint4*>(v);
                        w[k][0] = u.x, w[k][1] = u.y, w[k][2] = u.z, w[k][3] = u.w;
                        sb[k] = *reinterpret_cast<const uint16_t*>(sv);
                    } else if constexpr (D == 128) {
                        const uint2 u = *reinterpret_cast<const uint2*>(v);
                        w[k][0] = u.x, w[k][1] = u.y;
                        sb[k] = *sv;
                    } else {
                        w[k][0] = *reinterpret_cast<const uint32_t*>(v);
                        sb[k] = *sv;
                    }
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int row = 16 * mt + 8 * (k >> 1) + ((k & 1) ? v1 : v0);
                        const bool gone = (bad >> (row >> piece_shift)) & 1u;
                        if (p0 + row >= x.end || gone) sb[k] = 0;
                    }
                }
                uint32_t s01 = 0, s23 = 0;
#pragma unroll
                for (int wi = 0; wi < kWords; ++wi) {
                    if (wi == 0 || wi == 2) {
                        s01 = scale_both<D>(sb[0], sb[1], wi / 2);
                        s23 = scale_both<D>(sb[2], sb[3], wi / 2);
                    }
                    uint32_t e01[4], o01[4], e23[4], o23[4];
                    unpack((w[0][wi] & 0x0F0F0F0Fu) | ((w[1][wi] << 4) & 0xF0F0F0F0u), s01, e01);
                    unpack(((w[0][wi] >> 4) & 0x0F0F0F0Fu) | (w[1][wi] & 0xF0F0F0F0u), s01, o01);
                    unpack((w[2][wi] & 0x0F0F0F0Fu) | ((w[3][wi] << 4) & 0xF0F0F0F0u), s23, e23);
                    unpack(((w[2][wi] >> 4) & 0x0F0F0F0Fu) | (w[3][wi] & 0xF0F0F0F0u), s23, o23);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if constexpr (SPLIT) {
                                // The tensor cores cut a running sum off at every step, so fp32 calls add each step's
                                // products to it with fp32 instructions: 4.3e-5 -> 1.7e-6 at 16000 equal values, 49 -> 52 us
                                // for single tokens of 64 sequences of up to 8192 tokens with 20 heads.
                                float step[4] = {};
                                mma_f16(step, e01[i], o01[i], e23[i], o23[i], pl[mt][nt][0], pl[mt][nt][1]);
                                mma_f16(step, e01[i], o01[i], e23[i], o23[i], ph[mt][nt][0], ph[mt][nt][1]);
#pragma unroll
                                for (int j = 0; j < 4; ++j) o[4 * wi + i][nt][j] += step[j];
                            } else {
                                mma_f16(o[4 * wi + i][nt], e01[i], o01[i], e23[i], o23[i], ph[mt][nt][0], ph[mt][nt][1]);
                            }
                        }
                }
            }
            if (bad != 0 && lane == 0) atomicOr(&g_kv4_attn_error, kErrBadPage);
            ++used;
            freed = static_cast<int>(s);
            owed = true;
            __syncwarp();  // every lane has read the stage
        }

        // --- join the warps: each puts its sums, 8 columns at a time, where its last tile was
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) ls[nt][j] += __shfl_xor_sync(~0u, ls[nt][j], q);
                if (g == 0) {
                    col_m[warp * kCols + 8 * nt + 2 * t4 + j] = m[nt][j];
                    col_l[warp * kCols + 8 * nt + 2 * t4 + j] = ls[nt][j];
                }
            }
        if (lane == 0) red_s[warp] = freed;
        __syncthreads();
        const int run = *run_s;
        const bool begins = r0 == run * kFreshRounds;  // the unit's first rounds are this CTA's
        const bool done = begins && r1 == cur.cost - kUnitCost;
        float* slot = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * (kCols * (D + 2));
        if (done) wait_for_prefixes(p);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (freed >= 0) {
                float f[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int c = 8 * nt + 2 * t4 + j;
                    float mm = col_m[c];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, col_m[w * kCols + c]);
                    f[j] = m[nt][j] == -INFINITY ? 0.0f : exp2_approx(m[nt][j] - mm);
                }
                float* mine = reinterpret_cast<float*>(ring + freed * TL::kBytes) + 2 * t4 * S::kRedStride + 2 * g;
#pragma unroll
                for (int i = 0; i < kMTiles; ++i) {
                    *reinterpret_cast<float2*>(mine + 16 * i) = make_float2(o[i][nt][0] * f[0], o[i][nt][2] * f[0]);
                    *reinterpret_cast<float2*>(mine + S::kRedStride + 16 * i) = make_float2(o[i][nt][1] * f[1], o[i][nt][3] * f[1]);
                }
            }
            __syncthreads();
            for (int e = tid; e < 8 * D / 2; e += kAttnThreads) {
                const int c8 = e / (D / 2), pos = 2 * (e % (D / 2)), c = 8 * nt + c8;
                if (c >= all_cols) continue;
                float2 v = make_float2(0.0f, 0.0f);
                float mm = -INFINITY, l = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, col_m[w * kCols + c]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    if (red_s[w] < 0) continue;
                    const float* theirs = reinterpret_cast<const float*>(sm + (w * kStages + red_s[w]) * TL::kBytes);
                    const float2 y = *reinterpret_cast<const float2*>(theirs + c8 * S::kRedStride + pos);
                    v.x += y.x;
                    v.y += y.y;
                    const float mw = col_m[w * kCols + c];
                    l += col_l[w * kCols + c] * (mw == -INFINITY ? 0.0f : exp2_approx(mw - mm));
                }
                if (run > 0) {  // and the earlier runs
                    const float* before = runs_s + (run & 1) * 2 * kCols + c;
                    const float now = mm;
                    mm = fmaxf(mm, before[0]);
                    const float f0 = before[0] == -INFINITY ? 0.0f : exp2_approx(before[0] - mm);
                    const float f1 = now == -INFINITY ? 0.0f : exp2_approx(now - mm);
                    const float2 y = *reinterpret_cast<const float2*>(slot + c * D + pos);
                    v = make_float2(y.x * f0 + v.x * f1, y.y * f0 + v.y * f1);
                    l = before[kCols] * f0 + l * f1;
                }
                if (done) {
                    const size_t out = q_row(p, b, x, c);
                    store_out2(p, out + dim_of<D>(pos), v.x, v.y, out_factors(p, out, mm, l));
                    if (pos == 0) keep_sums(p, out, mm, l);
                } else {
                    *reinterpret_cast<float2*>(slot + c * D + pos) = v;
                    if (pos == 0) {
                        float* next = runs_s + ((run & 1) ^ 1) * 2 * kCols + c;  // others may still read this run's
                        slot[kCols * D + c] = next[0] = mm;
                        slot[kCols * D + kCols + c] = next[kCols] = l;
                    }
                }
            }
            __syncthreads();
        }
        if (owed) issue();
        const int places = r1 + kUnitCost - cur.at;
        if (places < cur.left && r1 < cur.cost - kUnitCost) {  // the unit's next run
            cur.at += places;
            cur.left -= places;
            if (tid == 0) *run_s = run + 1;
            continue;
        }
        if (tid == 0 && !done && begins)  // this CTA's blocks of the join have it
            *record = JoinRecord{cur.b, 0, cur.u,
                                 cta_of(total, hi - cur.left - cur.at + cur.cost - 1, ctas) - static_cast<int>(blockIdx.x) + 1};

        // --- the next unit
        advance<D>(p, units, cur);
        if (tid == 0) *run_s = 0;
    }
    wait_for_prefixes(p);
}

constexpr int kJoinThreads = 256;

// Joins the partial results of the units that several CTAs shared, one column per block.
template <int D, int NT, class P>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(const __grid_constant__ P p) {
    constexpr int kCols = 8 * NT;
    constexpr size_t kSlot = kCols * (D + 2);
    __shared__ float2 sums[kJoinThreads];
    __shared__ float lsum[kJoinThreads];
    const int lane = threadIdx.x & 31, c = blockIdx.y;
    if (shares(p)) griddep_launch_dependents();  // the pass over the own caches follows
    griddep_wait();
    const JoinRecord rec = reinterpret_cast<const JoinRecord*>(p.records)[blockIdx.x];
    if (rec.parts == 0) return;
    const Unit x = unit_of(p, rec.b, rec.pair);
    if (c >= x.n * p.group) return;
    const int parts = rec.parts;
    const float* base = p.part + static_cast<size_t>(blockIdx.x) * 2 * kSlot;
    auto slot = [&](int i) -> const float* { return i == 0 ? base + kSlot : base + static_cast<size_t>(i) * 2 * kSlot; };
    float mm = -INFINITY;
    for (int i = lane; i < parts; i += 32) mm = fmaxf(mm, slot(i)[kCols * D + c]);
    for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
    constexpr int kPairs = D / 2, kWays = kJoinThreads / kPairs;
    const int pair = threadIdx.x % kPairs, way = threadIdx.x / kPairs;
    float2 v = make_float2(0.0f, 0.0f);
    float l = 0.0f;
#pragma unroll 8
    for (int i = way; i < parts; i += kWays) {
        const float* s = slot(i);
        const float ms = s[kCols * D + c];
        const float f = ms == -INFINITY ? 0.0f : exp2_approx(ms - mm);
        const float2 y = *reinterpret_cast<const float2*>(s + c * D + 2 * pair);
        v.x += y.x * f;
        v.y += y.y * f;
        l += s[kCols * D + kCols + c] * f;
    }
    sums[threadIdx.x] = v;
    lsum[threadIdx.x] = l;
    __syncthreads();
    if (way != 0) return;
    for (int w = 1; w < kWays; ++w) {
        v.x += sums[w * kPairs + pair].x;
        v.y += sums[w * kPairs + pair].y;
        l += lsum[w * kPairs + pair];
    }
    const size_t out = q_row(p, rec.b, x, c);
    store_out2(p, out + dim_of<D>(2 * pair), v.x, v.y, out_factors(p, out, mm, l));
    if (pair == 0) keep_sums(p, out, mm, l);
}

// Windows of more query rows per kv head than this go to the tensor cores (gdn_kv4_window.cu). 64 sequences of 4096
// tokens, 4 kv heads: 57 / 59 / 62 us here for 9 / 12 / 16 rows against 103 us there; with a third and a fourth column tile
// 20 to 24 and 20 to 32 rows took 94 to 97 and 137 to 147 us here against 104 us there.
constexpr int kMostColumns = 16;

bool on_tensor_cores(int T, int group) { return static_cast<long long>(T) * group > kMostColumns; }

int column_tiles(int T, int group) { return T * group <= 8 ? 1 : 2; }

constexpr int kMaxCtas = 4 * 192;  // the workspace is sized for cards of up to 192 SMs

template <int D, int NT, bool SPLIT, class P>
cudaError_t launch_one(const P& p, cudaStream_t stream) {
    using S = Smem<D, NT, SPLIT>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(kv4_attention_kernel<D, NT, SPLIT, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 S::kBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    constexpr int kFit = Shape<D, NT, SPLIT>::kCtas;
    static_assert(kFit * (S::kBytes + 1024) <= 233472, "the CTAs of an SM fit its shared memory");
    // no more CTAs than there can be places, as far as the tables' lengths say (three answers to one question of 1500 tokens, fp32: 30.9 -> 26.7 us)
    constexpr int kRound = Tile<D>::kTokens * kWarps;
    const long long rounds = ((static_cast<long long>(p.c.max_pages) << p.c.page_shift) + kRound - 1) / kRound;
    const long long places = static_cast<long long>(p.c.B) * p.c.L * p.c.kv_heads * (kUnitCost + rounds);
    const int ctas = static_cast<int>(std::min<long long>(places, std::min(kFit * sms, kMaxCtas)));
    e = launch_pass(kv4_attention_kernel<D, NT, SPLIT, P>, ctas, kAttnThreads, S::kBytes, p, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, static_cast<unsigned>(std::min<long long>(8 * NT, static_cast<long long>(p.c.T) * p.group)));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, NT, P>, p);
}

template <int D, int NT, class P>
cudaError_t launch_split(const P& p, cudaStream_t stream) {
    return p.dtype == DType::kF32 ? launch_one<D, NT, true>(p, stream) : launch_one<D, NT, false>(p, stream);
}

template <int D, class P>
cudaError_t launch_dim(const P& p, int nt, cudaStream_t stream) {
    if (nt == 1) return launch_split<D, 1>(p, stream);
    return launch_split<D, 2>(p, stream);
}

}  // namespace

size_t kv4_attention_workspace_bytes(int B, int L, int T, int q_heads, int kv_heads, int head_dim) {
    (void)B;
    (void)L;
    const int group = q_heads / kv_heads;
    if (on_tensor_cores(T, group)) return kv4_window_workspace_bytes(head_dim);
    const int nt = column_tiles(T, group);
    return static_cast<size_t>(kMaxCtas) * (2 * (8 * nt) * (head_dim + 2) * sizeof(float) + sizeof(JoinRecord));
}

namespace {

AttnParams attn_params(const Kv4AttnArgs& a) {
    AttnParams p{};
    p.c = a.c;
    p.q = a.q;
    p.out = a.out;
    p.part = static_cast<float*>(a.workspace);
    p.q_heads = a.q_heads;
    p.group = a.q_heads / a.c.kv_heads;
    p.dtype = a.dtype;
    p.scale = a.scale;
    return p;
}

cudaError_t launch_attention(AttnParams p, cudaStream_t stream) {
    if (on_tensor_cores(p.c.T, p.group))
        return p.groups != nullptr && p.dtype != DType::kF32 && p.c.head_dim <= 128 ? launch_kv4_prefix(p, stream) : launch_kv4_window(p, stream);
    const int nt = column_tiles(p.c.T, p.group);
    p.records = p.part + static_cast<size_t>(kMaxCtas) * 2 * (8 * nt) * (p.c.head_dim + 2);
    switch (p.c.head_dim) {
        case 64: return p.prefix_sums != nullptr ? launch_dim<64>(p, nt, stream) : launch_dim<64>(PlainParams{p}, nt, stream);
        case 128: return p.prefix_sums != nullptr ? launch_dim<128>(p, nt, stream) : launch_dim<128>(PlainParams{p}, nt, stream);
        case 256: return p.prefix_sums != nullptr ? launch_dim<256>(p, nt, stream) : launch_dim<256>(PlainParams{p}, nt, stream);
        default: return cudaErrorInvalidValue;
    }
}

// What one pass of the attention needs, in whole 16-byte units.
size_t pass_bytes(int B, int L, int T, int q_heads, int kv_heads, int head_dim) {
    return (kv4_attention_workspace_bytes(B, L, T, q_heads, kv_heads, head_dim) + 15) / 16 * 16;
}

}  // namespace

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, cudaStream_t stream) { return launch_attention(attn_params(a), stream); }

// The passes' workspaces, that of the own caches first, then the outputs over the prefixes, then their maxima and sums.
size_t kv4_attention_shared_workspace_bytes(int B, int L, int T, int q_heads, int kv_heads, int head_dim) {
    const size_t rows = static_cast<size_t>(B) * L * T * q_heads;
    return pass_bytes(B, L, T, q_heads, kv_heads, head_dim) + pass_bytes(1, L, B * T, q_heads, kv_heads, head_dim) +
           rows * (head_dim * sizeof(float) + sizeof(float2));
}

cudaError_t launch_kv4_attention_shared(const Kv4SharedArgs& a, cudaStream_t stream) {
    AttnParams own = attn_params(a.own);
    const Kv4Cache& c = a.own.c;
    const size_t rows = static_cast<size_t>(c.B) * c.L * c.T * own.q_heads;
    const size_t own_bytes = pass_bytes(c.B, c.L, c.T, own.q_heads, c.kv_heads, c.head_dim);
    AttnParams prefix = own;
    prefix.part = own.part + own_bytes / sizeof(float);  // (the passes overlap)
    own.prefix_out = prefix.prefix_out = prefix.part + pass_bytes(1, c.L, c.B * c.T, own.q_heads, c.kv_heads, c.head_dim) / sizeof(float);
    own.prefix_sums = prefix.prefix_sums = reinterpret_cast<float2*>(own.prefix_out + rows * c.head_dim);
    prefix.c.block_table = a.prefix_table;
    prefix.c.kv_start = a.prefix_len;
    prefix.c.seq_len = nullptr;
    prefix.c.B = a.n_groups;
    prefix.c.T = c.B * c.T;
    prefix.c.max_pages = a.max_prefix_pages;
    prefix.groups = a.groups;
    prefix.batch = c.B;
    prefix.window = c.T;
    const cudaError_t e = launch_attention(prefix, stream);
    return e != cudaSuccess ? e : launch_attention(own, stream);
}

cudaError_t read_kv4_attention_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_attn_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_attn_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace gdn
