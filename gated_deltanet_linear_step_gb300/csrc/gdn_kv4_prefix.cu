// gdn_kv4_prefix.cu - attention of many rows over a shared prefix of the 4-bit cache: the first pass of gdn_kv4_attention_shared for
// 16-bit calls, on the 5th-generation tensor cores. Mathematics, numerics and missing pages are those of gdn_kv4_window.cu; what is
// different is that every row sees every key.
//
//   S = Q K^T   128 rows x 128 keys x D,   O += P V   128 rows x D x 128 keys
//
// A unit is up to 256 rows, (sequence, token, query head) of one kv head's group: two blocks of 128 that share the unpacked tiles and take turns on the
// tensor cores, one's softmax beside the other's products. A unit of up to 128 rows has its tiles dealt to two blocks of the same
// rows instead, which are joined at its end, so that it does not wait for its own softmax at every tile.
//
//   warp 0     issues the products
//   warp 1     looks up pages and copies the tiles' codes and scales to shared memory, 4.5 bits a value, by bulk copies
//   8 warps    a row per thread: queries in, scores from tensor memory, maximum, exponentials, probabilities back, sums out
//   4 warps    unpack the tiles to fp16 in the swizzled rows that the products read
//
// Tensor memory: [first block's probabilities | scores of either | second block's probabilities | sums of both], as in gdn_prompt.cu.
//
// Work split: all units of all groups lie on a line, a tile three places long, in units of up to 128 rows two; it is dealt out
// evenly to the CTAs. Units that several CTAs share leave partial sums in the workspace, which a second kernel joins in order.
// Waits are bounded, as there.
//
// What bounds it: two blocks' tile takes some 3600 clocks, of which the tensor cores need 2600 (128 x 128 x 128 some 650 in practice), a
// block's softmax 1900 beside the other's products; one block's takes 2700. A CTA spends 9 us before its first scores (its place in the line, page
// numbers, tiles and queries one after the other) and 4 on its sums. The raw tiles wait in three places because a copy takes 2000 clocks
// and a turn to unpack 700: with one place each for keys and values a tile of one block took 3600 clocks.

#include <algorithm>
#include <atomic>

#include "gdn_device.cuh"
#include "gdn_kv4_attention.cuh"
#include "gdn_tc_attention.cuh"

namespace gdn {
namespace {

constexpr int kRows = kMmaRows;
constexpr int kTok = 128;
constexpr int kBlocks = 2;
constexpr int kUnitRows = kBlocks * kRows;
constexpr int kStages = 2;
constexpr int kUnpackWarps = 4;
constexpr int kThreads = 512;
constexpr int kDual = 3, kSingle = 2;  // places of a tile of two blocks' rows and of one's
constexpr int kLeastPlaces = 8;  // of a CTA: the call for 40 rows over 1500 tokens takes 39 / 32 / 30 / 27 / 29 us with 24 / 16 / 12 / 8 / 4, 100 rows over 32000 52 / 45 / 47 / 47 / 47
constexpr int kMaxSms = 192;     // the workspace is sized for cards of up to as many
constexpr int kFreshTiles = 16384 / kTok;  // sums start afresh, see gdn_kv4_window.cu
constexpr uint32_t kTmCols = 512, kTmScores = 64, kTmO = 256;

__device__ unsigned int g_kv4_prefix_error = 0;

template <int D>
struct Prefix {
    static constexpr int kBlk = D / 64;                          // 64-dim blocks of a row (128 bytes)
    static constexpr int kRaw = D == 64 ? 6 : 3;                 // tiles' keys or values as they are cached, in turn
    static constexpr uint32_t kQBlock = kRows * 128, kQBytes = kBlk * kQBlock;
    static constexpr uint32_t kKvBlock = kTok * 128, kKvBytes = kBlk * kKvBlock;
    static constexpr uint32_t kCodes = kTok * D / 2, kScales = kTok * D / 16, kRawBytes = kCodes + kScales;  // of keys, or of values
    static constexpr uint32_t kOffK = kBlocks * kQBytes;
    static constexpr uint32_t kOffV = kOffK + kStages * kKvBytes;
    static constexpr uint32_t kOffRaw = kOffV + kStages * kKvBytes;
    static constexpr uint32_t kOffMul = kOffRaw + kRaw * kRawBytes;
    static constexpr uint32_t kOffBad = kOffMul + kUnitRows * 4;     // missing pages of tiles j mod 8
    static constexpr uint32_t kOffBar = kOffBad + 8 * 4;
    static constexpr uint32_t kBars = 4 * kStages + 2 * kRaw + 6 * kBlocks + 3;
    static constexpr uint32_t kUsed = kOffBar + kBars * 8 + 64;
    static constexpr uint32_t kLeast = 118 * 1024;                   // one CTA per SM: the tensor memory is its own
    static constexpr uint32_t kSmem = kUsed + 1024 > kLeast ? kUsed + 1024 : kLeast;
    static_assert(kSmem <= 232448 && kTmO + kBlocks * D <= kTmCols, "shared and tensor memory");
};

// The unit, if there is one, whose first tiles a CTA did and whose last ones other CTAs did (rows 0: there is none): `parts` CTAs, this one first, have
// a partial result of it each.
struct PrefixRecord {
    int g, pair, block;
    short rows, parts;
};
static_assert(sizeof(PrefixRecord) == sizeof(JoinRecord), "the workspace holds one per CTA");

// Places of a unit's start: queries in, sums out, some 7 us of it that nothing hides where a CTA goes from one unit to the next. The whole call
// for 64 samples after 32000 tokens, 20 heads of 128: 80 us with 9 places, 75 with 18, 73 with 24; 20 samples 48 with 24, 46 with 20; 64 requests
// in four groups after 4000 tokens 83 and 81. Verify windows of 64-dim heads: 67 us with 9 or 12, 70 with 18.
__host__ __device__ __forceinline__ int start_places(const AttnParams& p) { return p.c.head_dim == 64 ? 12 : 20; }

// A group's units for one layer and kv head: `dual` of more than 128 rows, then `single` (0 or 1) of up to 128.
struct Group {
    int n, end, rows, tiles, dual, single;  // n: tokens of its sequences; end: of the prefix
};

__device__ __forceinline__ Group group_of(const AttnParams& p, int g) {
    const Kv4Window w = attn_window(p, g);
    Group x;
    x.n = w.n;
    x.end = w.start + 1;
    x.rows = w.n * p.group;
    x.tiles = max((w.start + kTok) / kTok, 1);  // one at least: rows that see no key get their zeros
    const int rest = x.rows % kUnitRows;
    x.dual = x.rows / kUnitRows + (rest > kRows ? 1 : 0);
    x.single = rest > 0 && rest <= kRows ? 1 : 0;
    return x;
}

__device__ __forceinline__ long long group_cost(const AttnParams& p, const Group& x, int pairs) {
    return static_cast<long long>(pairs) * (x.dual * (start_places(p) + static_cast<long long>(kDual) * x.tiles) + x.single * (start_places(p) + static_cast<long long>(kSingle) * x.tiles));
}

// Where a CTA is: unit `index` of group g, at place `at` of its `cost`, `left` places to go.
struct PrefixCursor {
    int g, index, at, cost;
    long long left;
};

// What a role needs to know of the cursor's unit: its rows, their tiles [r0, r1) that are this CTA's, whether they are all of them.
struct PrefixUnit {
    Unit x;
    int rows, r0, r1, tiles, weight, block, pair;
};

__device__ __forceinline__ void set_cost(const AttnParams& p, int pairs, PrefixCursor& k) {
    const Group x = group_of(p, k.g);
    k.cost = start_places(p) + (k.index < pairs * x.dual ? kDual : kSingle) * x.tiles;
}

__device__ __forceinline__ PrefixUnit unit_at(const AttnParams& p, int pairs, const PrefixCursor& k) {
    PrefixUnit u;
    const Group x = group_of(p, k.g);
    const bool dual = k.index < pairs * x.dual;
    u.weight = dual ? kDual : kSingle;
    u.block = dual ? k.index / pairs : x.dual;
    u.pair = k.index - u.block * pairs;
    u.tiles = x.tiles;
    auto first = [&](int place) -> int {
        const int x = max(place - start_places(p), 0);
        return dual ? (x + kDual - 1) / kDual : (x + kSingle - 1) / kSingle;
    };
    u.r0 = first(k.at);
    u.r1 = first(static_cast<int>(min(static_cast<long long>(k.cost), k.at + k.left)));
    u.x.h = u.pair % p.c.kv_heads;
    u.x.l = u.pair / p.c.kv_heads;
    u.x.col0 = u.block * kUnitRows;
    u.x.start = x.end - 1;
    u.x.n = x.n;
    u.x.end = x.end;
    u.rows = min(x.rows - u.x.col0, kUnitRows);
    return u;
}

__device__ __forceinline__ void next_unit(const AttnParams& p, int pairs, PrefixCursor& k) {
    k.left -= k.cost - k.at;
    k.at = 0;
    if (k.left <= 0) return;
    ++k.index;
    for (; k.g < p.c.B; ++k.g, k.index = 0) {
        const Group x = group_of(p, k.g);
        if (k.index < pairs * (x.dual + x.single)) {
            set_cost(p, pairs, k);
            return;
        }
    }
}

// The unit and place in it of place x of the line, by one warp.
__device__ __forceinline__ PrefixCursor find(const AttnParams& p, int pairs, long long x, int lane) {
    PrefixCursor k{0, 0, 0, 0, 0};
    for (int g0 = 0; g0 < p.c.B; g0 += 32) {
        const long long mine = g0 + lane < p.c.B ? group_cost(p, group_of(p, g0 + lane), pairs) : 0;
        long long sum = mine;
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
        x -= __shfl_sync(~0u, sum - mine, src);
        k.g = g0 + src;
        const Group u = group_of(p, k.g);
        const int dual = start_places(p) + kDual * u.tiles, single = start_places(p) + kSingle * u.tiles;
        const long long duals = static_cast<long long>(pairs) * u.dual * dual;
        if (x < duals) {
            k.index = static_cast<int>(mul_div(x, 1, dual));
            k.at = static_cast<int>(x - static_cast<long long>(k.index) * dual);
            k.cost = dual;
        } else {
            x -= duals;
            k.index = static_cast<int>(mul_div(x, 1, single));
            k.at = static_cast<int>(x - static_cast<long long>(k.index) * single);
            k.index += pairs * u.dual;
            k.cost = single;
        }
        return k;
    }
    return k;
}

__device__ __forceinline__ long long line_length(const AttnParams& p, int pairs, int lane) {
    long long s = 0;
    for (int g = lane; g < p.c.B; g += 32) s += group_cost(p, group_of(p, g), pairs);
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    return s;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefix_kernel(const __grid_constant__ AttnParams p) {
    using W = Prefix<D>;
    constexpr int kRaw = W::kRaw;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    const uint32_t raw_addr = smem_addr(smem_raw), base = (raw_addr + 1023u) & ~1023u;
    unsigned char* sm = smem_raw + (base - raw_addr);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float* mul_s = reinterpret_cast<float*>(sm + W::kOffMul);
    volatile uint32_t* bad_s = reinterpret_cast<volatile uint32_t*>(sm + W::kOffBad);
    PrefixCursor* cur_s = reinterpret_cast<PrefixCursor*>(sm + W::kOffBar + W::kBars * 8);
    uint32_t* tmem_s = reinterpret_cast<uint32_t*>(cur_s + 1);
    const uint32_t k_full = base + W::kOffBar, v_full = k_full + 8 * kStages, k_free = v_full + 8 * kStages, v_free = k_free + 8 * kStages;
    const uint32_t raw_full = v_free + 8 * kStages, raw_free = raw_full + 8 * kRaw;
    const uint32_t q_full = raw_free + 8 * kRaw, q_free = q_full + 8 * kBlocks;  // per block
    const uint32_t s_done = q_free + 8 * kBlocks, p_ready = s_done + 8 * kBlocks, p_rest = p_ready + 8 * kBlocks, o_done = p_rest + 8 * kBlocks;
    const uint32_t s_free = o_done + 8 * kBlocks, joined = s_free + 8, drained = joined + 8;
    const int pairs = p.c.L * p.c.kv_heads;

    if (some_group_falls(p)) atomicOr(&g_kv4_prefix_error, kErrBadBorders);
    if (blockIdx.x == 0)
        for (int g = tid; g < p.c.B; g += kThreads)
            if (attn_runs_out(p, g)) atomicOr(&g_kv4_prefix_error, kErrBadPage);
    long long total = 0;
    int ctas = 0;
    if (warp < 2 || (warp >= 4 && warp < 12)) {
        total = line_length(p, pairs, lane);
        ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), max(total / kLeastPlaces, 1ll)));
    }
    if (warp == 0) {
        long long lo = 0, hi = 0;
        PrefixCursor k{};
        if (static_cast<int>(blockIdx.x) < ctas && total > 0) {
            cta_range(total, blockIdx.x, ctas, lo, hi);
            k = find(p, pairs, lo, lane);
        }
        k.left = hi - lo;
        if (lane == 0) *cur_s = k;
    } else if (tid == 32) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(k_full + 8 * i, kUnpackWarps);
            mbar_init(v_full + 8 * i, kUnpackWarps);
            mbar_init(k_free + 8 * i, 1);
            mbar_init(v_free + 8 * i, 1);
        }
        for (int i = 0; i < kRaw; ++i) {
            mbar_init(raw_full + 8 * i, 1);
            mbar_init(raw_free + 8 * i, kUnpackWarps);
        }
        for (int i = 0; i < kBlocks; ++i) {
            mbar_init(q_full + 8 * i, 4);
            mbar_init(q_free + 8 * i, 1);
            mbar_init(s_done + 8 * i, 1);
            mbar_init(p_ready + 8 * i, 4);
            mbar_init(p_rest + 8 * i, 4);
            mbar_init(o_done + 8 * i, 1);
        }
        mbar_init(s_free, 4);
        mbar_init(joined, 4);
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    __syncthreads();
    PrefixCursor cur = *cur_s;
    PrefixRecord* record = reinterpret_cast<PrefixRecord*>(p.records) + blockIdx.x;
    if (tid == 32) *record = PrefixRecord{0, 0, 0, 0, 0};
    if (cur.left <= 0) return;
    if (warp == 0) tmem_alloc(smem_addr(tmem_s), kTmCols);
    tc_fence_before();
    __syncthreads();
    griddep_launch_dependents();  // (this grid has its tensor memory: whatever waits for some, waits for CTAs that end by themselves)
    tc_fence_after();
    const uint32_t tmem = *tmem_s;
    // Tile n of the CTA (counted over all its units) uses stage n mod kStages of K and V; its keys and values as they are cached are the 2 n-th and
    // (2 n + 1)-th use of the raw places.
    bool failed = false;
    int n = 0;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");  // (512 x 128 = 128 x 48 + 256 x 208 + 128 x 48)
        if (warp == 1) {
            // --------------------------------------------------------- loads
            const int psize = 1 << p.c.page_shift, shift = min(p.c.page_shift, 7), pieces = kTok >> shift;
            const uint32_t head_bytes = static_cast<uint32_t>(kv4_head_bytes(psize, D));
            const unsigned long long page_bytes = static_cast<unsigned long long>(head_bytes) * p.c.kv_heads;
            int uses = 0;  // of the raw places
            for (; cur.left > 0 && !failed; next_unit(p, pairs, cur)) {
                const PrefixUnit u = unit_at(p, pairs, cur);
                const int32_t* table = p.c.block_table + static_cast<size_t>(cur.g) * p.c.max_pages;
                const uint8_t* head = p.c.cache + (static_cast<size_t>(u.x.l) * p.c.n_pages * p.c.kv_heads + u.x.h) * head_bytes;
                // lane j looks up page j of a tile, a tile ahead
                auto wanted = [&](int r) { return lane < pieces && r * kTok + (lane << shift) < u.x.end; };
                auto look = [&](int r) { return wanted(r) ? __ldg(table + ((r * kTok + (lane << shift)) >> p.c.page_shift)) : -1; };
                int next = u.r0 < u.r1 ? look(u.r0) : -1;
                for (int r = u.r0; r < u.r1; ++r, ++n) {
                    const bool want = wanted(r);
                    const int page = static_cast<uint32_t>(next) < static_cast<uint32_t>(p.c.n_pages) ? next : -1;
                    const unsigned gone = __ballot_sync(~0u, want && page < 0), there = __ballot_sync(~0u, page >= 0);
                    if (r + 1 < u.r1) next = look(r + 1);
                    uint32_t bad = 0;  // the missing pages as 16-token groups, whatever the page size
#pragma unroll
                    for (int q = 0; q < kTok / 16; ++q) bad |= ((gone >> ((16 * q) >> shift)) & 1u) << q;
                    const int rows = 1 << shift;
                    const uint8_t* k = head + static_cast<unsigned long long>(static_cast<uint32_t>(max(page, 0))) * page_bytes;
                    const uint32_t in_page = (r * kTok + (lane << shift)) & (psize - 1), row = lane << shift;
                    const uint32_t bytes = static_cast<uint32_t>(__popc(there)) * rows * (D / 2 + D / 16);
                    for (int part = 0; part < 2; ++part) {
                        const int s = uses % kRaw;
                        if (uses >= kRaw && !warp_wait(raw_free + 8 * s, static_cast<uint32_t>(uses / kRaw - 1) & 1u)) {
                            failed = true;
                            break;
                        }
                        ++uses;
                        const uint32_t full = raw_full + 8 * s, to = base + W::kOffRaw + s * W::kRawBytes;
                        if (lane == 0) {
                            if (part == 0) bad_s[n & 7] = bad;
                            mbar_arrive_expect_tx(full, bytes);
                        }
                        __syncwarp();
                        if (page >= 0) {
                            const uint8_t* from = k + part * (head_bytes / 2);
                            bulk_load(to + row * (D / 2), from + in_page * (D / 2), rows * (D / 2), full);
                            bulk_load(to + W::kCodes + row * (D / 16), from + psize * (D / 2) + in_page * (D / 16), rows * (D / 16), full);
                        }
                    }
                    if (bad != 0 && lane == 0) atomicOr(&g_kv4_prefix_error, kErrBadPage);
                    if (failed) break;
                }
            }
            // whatever is in flight has landed before the CTA ends
            for (int s = 0; s < kRaw; ++s) {
                const int c = (uses - s + kRaw - 1) / kRaw;
                if (c > 0) (void)warp_wait(raw_full + 8 * s, static_cast<uint32_t>(c - 1) & 1u);
            }
        } else if (warp == 0) {
            if (elect_one()) {
                // -------------------------------------------------- products (its waits poll, as in gdn_prompt.cu)
                constexpr uint32_t idesc_s = idesc_f16(kTok), idesc_o = idesc_f16(D) | kIdescBMnMajor;
                const uint32_t q_desc = desc_k(base), k_desc = desc_k(base + W::kOffK), v_desc = desc_mn(base + W::kOffV, W::kKvBlock);
                // Per block: tiles; units whose queries its place held; whether its last tile awaits its product with the values, whether that starts
                // its sums, and the tile. 16 bits a count: parities and neighbours are all that is asked of them. The code is there once for both
                // blocks: what is run for the first time is waited for.
                uint32_t m = 0, queries = 0, tiles = 0, open = 0, fresh = 0;
                int scored = 0;  // tiles of both blocks
                auto low = [](uint32_t x, int i) -> uint32_t { return (x >> (16 * i)) & 0xFFFFu; };
                auto put = [](uint32_t x, int i, uint32_t v) -> uint32_t { return i ? (x & 0xFFFFu) | (v << 16) : (x & 0xFFFF0000u) | (v & 0xFFFFu); };
                auto close = [&](int i) -> bool {
                    if (!((open >> i) & 1u)) return true;
                    open ^= 1u << i;
                    const uint32_t t = low(tiles, i), mine = low(m, i) - 1;
                    if (!mbar_wait_bounded(v_full + 8 * (t % kStages), (t / kStages) & 1u)) return false;
                    if (!mbar_wait_bounded(p_ready + 8 * i, mine & 1u)) return false;
                    tc_fence_after();
                    const uint32_t v = v_desc + (t % kStages) * (W::kKvBytes >> 4), d = tmem + kTmO + i * D, pr = tmem + 192 * i;
#pragma unroll
                    for (int c = 0; c < kTok / 16; ++c) {
                        if (c == kTok / 32) {
                            if (!mbar_wait_bounded(p_rest + 8 * i, mine & 1u)) return false;
                            tc_fence_after();
                        }
                        mma_ts(d, pr + 8 * c, v + c * (2048 >> 4), idesc_o, c == 0 && ((fresh >> i) & 1u) ? 0u : 1u);
                    }
                    mma_commit(o_done + 8 * i);
                    if (!(((open >> (i ^ 1)) & 1u) && low(tiles, i ^ 1) == t)) mma_commit(v_free + 8 * (t % kStages));  // the tile's last product
                    return true;
                };
                for (; cur.left > 0 && !failed; next_unit(p, pairs, cur)) {
                    const PrefixUnit u = unit_at(p, pairs, cur);
                    const bool dual = u.weight == kDual;
                    for (int r = u.r0; r < u.r1 && !failed; ++r, ++n) {
                        const int j = r - u.r0;
                        // (a product with values that is due goes ahead of the wait for new keys)
                        bool ok = (dual || close(j & 1)) && mbar_wait_bounded(k_full + 8 * (n % kStages), static_cast<uint32_t>(n / kStages) & 1u);
#pragma unroll 1
                        for (int i = dual ? 0 : j & 1; ok && i < (dual ? kBlocks : (j & 1) + 1); ++i) {
                            ok = !dual || close(i);
                            const int qb = dual ? i : 0;  // whose queries
                            if (ok && j == 0) {
                                ok = mbar_wait_bounded(q_full + 8 * qb, low(queries, qb) & 1u);
                                queries = put(queries, qb, low(queries, qb) + 1);
                            }
                            // (the scores of the tile before have been read)
                            ok = ok && (scored == 0 || mbar_wait_bounded(s_free, static_cast<uint32_t>(scored - 1) & 1u));
                            if (!ok) break;
                            ++scored;
                            tc_fence_after();
                            const uint32_t k = k_desc + (n % kStages) * (W::kKvBytes >> 4), q = q_desc + qb * (W::kQBytes >> 4);
#pragma unroll
                            for (int c = 0; c < 4 * W::kBlk; ++c) {
                                const uint32_t ko = k + (c >> 2) * (W::kKvBlock >> 4) + 2 * (c & 3), qo = q + (c >> 2) * (W::kQBlock >> 4) + 2 * (c & 3);
                                if (c == 0)
                                    mma_ss<true>(tmem + kTmScores, qo, ko, idesc_s);
                                else
                                    mma_ss<false>(tmem + kTmScores, qo, ko, idesc_s);
                            }
                            mma_commit(s_done + 8 * i);
                            const uint32_t bit = 1u << i;
                            fresh = (dual ? j : j >> 1) % kFreshTiles == 0 ? fresh | bit : fresh & ~bit;
                            open |= bit;
                            tiles = put(tiles, i, static_cast<uint32_t>(n));
                            m = put(m, i, low(m, i) + 1);
                            if (r == u.r1 - 1) mma_commit(q_free + 8 * qb);
                        }
                        if (ok)
                            mma_commit(k_free + 8 * (n % kStages));
                        else
                            failed = true;
                    }
                    // a unit of one block's rows: its tiles' products before those of the next unit begin in the other block; and the CTA's last ones
                    const bool last = cur.left <= cur.cost - cur.at;
#pragma unroll 1
                    for (int i = 0; i < kBlocks; ++i)
                        if (!failed && (!dual || last) && !close(i)) failed = true;
                }
                // whatever was issued has completed before the tensor memory is freed
                mma_commit(drained);
                (void)mbar_wait_bounded(drained, 0);
            }
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        // -------------------------------------------------------------- rows
        const int block = (warp - 4) >> 2, quarter = warp & 3, row = 32 * quarter + lane;  // (a warp reaches lanes 32 (warp mod 4) ..)
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
        const uint32_t o_at = lanes + kTmO + block * D, p_at = lanes + 192 * block;
        int m_tiles = 0, held = 0, seen = 0, joins = 0;  // tiles of this block; units whose queries its place held, and the first block's; joined units
        for (; cur.left > 0 && !failed; next_unit(p, pairs, cur)) {
            const PrefixUnit u = unit_at(p, pairs, cur);
            if (u.r1 <= u.r0) continue;
            const bool dual = u.weight == kDual;
            const int b = cur.g;
            const int rows = dual ? u.rows - kRows * block : u.rows;  // of this block
            // queries, scaled to fill fp16's range
            if (dual || block == 0) {
                if (held > 0 && !warp_wait(q_free + 8 * block, static_cast<uint32_t>(held - 1) & 1u)) {
                    failed = true;
                    break;
                }
                ++held;
                // a thread its own row (rows by all lanes of a warp, 8 at a time, took 14 us: a row's place and factor are divisions)
                const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (row < rows ? q_row(p, b, u.x, u.x.col0 + kRows * block + row) : 0));
                uint4 w[D / 8];
                uint32_t most = 0;
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    w[i] = row < rows ? __ldg(from + i) : make_uint4(0u, 0u, 0u, 0u);
                    most = __vmaxu2(most, __vmaxu2(__vmaxu2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu), __vmaxu2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu)));
                }
                most = max(most & 0xFFFFu, most >> 16);  // (16-bit magnitudes are in the order of their bits)
                const bool half = p.dtype == DType::kF16;
                const float f = row_factor(half ? __half2float(__ushort_as_half(static_cast<uint16_t>(most))) : __uint_as_float(most << 16));
                mul_s[kRows * block + row] = score_factor(p.scale, f);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                    uint32_t y[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 v = half ? __half22float2(*reinterpret_cast<const __half2*>(&x[j]))
                                              : make_float2(__uint_as_float(x[j] << 16), __uint_as_float(x[j] & 0xFFFF0000u));
                        y[j] = pack_half2(v.x * f, v.y * f);
                    }
                    *reinterpret_cast<uint4*>(sm + block * W::kQBytes + (i >> 3) * W::kQBlock + sw128_offset(row, i & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive_local(q_full + 8 * block);
            } else if (!warp_wait(q_full, static_cast<uint32_t>(seen) & 1u)) {  // the rows' factors are the first block's
                failed = true;
                break;
            }
            ++seen;
            const bool some = 32 * quarter < rows;  // this warp has rows
            auto first_mul = [&]() -> float { return row < rows ? mul_s[(dual ? kRows * block : 0) + row] : kLeastScale; };
            float mul = first_mul();
            float m = -INFINITY, shift = kNone, l = 0.0f, sum_m = -INFINITY;
            float* slot = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (u.r0 == 0 ? 1 : 0)) * (kUnitRows * (D + 2));
            auto four_sums = [&](int c) -> float4& {  // of earlier runs of tiles, of dims c .. c + 3
                return *reinterpret_cast<float4*>(p.sums + static_cast<size_t>(blockIdx.x) * D * kUnitRows + c * kUnitRows + 4 * (kRows * block + row));
            };
            int mine = 0;  // tiles of this block in this unit
            for (int r = u.r0 + (dual ? 0 : block); r < u.r1; r += dual ? 1 : 2, ++m_tiles, ++mine) {
                if (!warp_wait(s_done + 8 * block, static_cast<uint32_t>(m_tiles) & 1u)) {
                    failed = true;
                    break;
                }
                tc_fence_after();
                if (some) {
                    float s[kTok];
                    tmem_read(lanes + kTmScores, s);
                    const uint32_t bad = bad_s[(n + (r - u.r0)) & 7];
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_local(s_free);
                    const int there = u.x.end - r * kTok;
                    if (there < kTok || bad != 0) {
#pragma unroll
                        for (int i = 0; i < kTok; ++i)
                            if (i >= there || ((bad >> (i >> 4)) & 1u)) s[i] = -INFINITY;
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
                    const bool starts = mine % kFreshTiles == 0;
                    if (starts && mine > 0) {  // the sums of the tiles so far leave the tensor memory
                        if (!warp_wait(o_done + 8 * block, static_cast<uint32_t>(m_tiles - 1) & 1u)) {
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
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 y = mine > kFreshTiles ? four_sums(c + i) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                                four_sums(c + i) = make_float4(fmaf(y.x, f, o[i]), fmaf(y.y, f, o[i + 1]), fmaf(y.z, f, o[i + 2]), fmaf(y.w, f, o[i + 3]));
                            }
                        }
                        __syncwarp();
                        sum_m = m;
                    }
                    const bool over = is_over(top, mul, shift);
                    if (__any_sync(~0u, over)) {
                        const float al = over ? raise(top, m, mul, shift, first_mul) : 1.0f;  // (a row's bits do not depend on its neighbours)
                        l *= al;
                        if (!starts) {  // the sums so far: after the product that is adding to them
                            if (!warp_wait(o_done + 8 * block, static_cast<uint32_t>(m_tiles - 1) & 1u)) {
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
                    // (the last reader of the probabilities' place is the product before these scores, and a commit stands for every
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
                            hi[i] = pack_half2(s[c + 2 * i], s[c + 2 * i + 1]);
                        }
                        tmem_st16(p_at + c / 2, hi);
                        if (c + 32 == kTok / 2) {
                            tmem_st_wait();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_local(p_ready + 8 * block);
                        }
                    }
                    l += sum.x + sum.y;
                    tmem_st_wait();
                } else if (lane == 0) {
                    mbar_arrive_local(s_free);
                    mbar_arrive_local(p_ready + 8 * block);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_local(p_rest + 8 * block);
            }
            n += u.r1 - u.r0;
            if (failed || (mine > 0 && !warp_wait(o_done + 8 * block, static_cast<uint32_t>(m_tiles - 1) & 1u))) {
                failed = true;
                break;
            }
            tc_fence_after();
            const float f = sum_m == -INFINITY ? 0.0f : exp2_approx(sum_m - m);  // of the sums of earlier runs
            // 16 sums of dims c .., all runs together
            auto read16 = [&](int c, float (&o)[16]) {
                uint32_t w[16];
                __syncwarp();
                tmem_read16(o_at + c, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(w[i]);
                if (mine > kFreshTiles) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 y = four_sums(c + i);
                        o[i] = fmaf(y.x, f, o[i]), o[i + 1] = fmaf(y.y, f, o[i + 1]);
                        o[i + 2] = fmaf(y.z, f, o[i + 2]), o[i + 3] = fmaf(y.w, f, o[i + 3]);
                    }
                }
            };
            auto part = [&](int c, int at) -> float4& { return *reinterpret_cast<float4*>(slot + c * kUnitRows + 4 * at); };
            if (!dual && block == 1) {  // to the first block, through the other half of the unit's place in the workspace
                if (some && mine > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float o[16];
                        read16(c, o);
#pragma unroll
                        for (int i = 0; i < 16; i += 4) part(c + i, kRows + row) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                slot[kUnitRows * D + kRows + row] = m;
                slot[kUnitRows * D + kUnitRows + kRows + row] = l;
                __syncwarp();
                if (lane == 0) mbar_arrive_local(joined);
                tc_fence_before();
                continue;
            }
            float own = 1.0f, others = 0.0f;
            if (!dual) {
                if (!warp_wait(joined, static_cast<uint32_t>(joins) & 1u)) {
                    failed = true;
                    break;
                }
                ++joins;
                const float m1 = slot[kUnitRows * D + kRows + row], l1 = slot[kUnitRows * D + kUnitRows + kRows + row];
                const float v = fmaxf(m, m1);
                own = m == -INFINITY ? 0.0f : exp2_approx(m - v);
                others = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - v);
                l = l != 0.0f || l1 != 0.0f ? l * own + l1 * others : 0.0f;
                m = v;
            }
            const bool done = u.r0 == 0 && u.r1 == u.tiles;
            if (some) {
                const size_t out = row < rows ? q_row(p, b, u.x, u.x.col0 + (dual ? kRows * block : 0) + row) : 0;
                const OutFactors factors = done && row < rows ? out_factors(p, out, m, l) : OutFactors{0.0f, 0.0f};
                if (done && row < rows) keep_sums(p, out, m, l);
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                    float o[16];
                    read16(c, o);
                    if (!dual) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 y = others != 0.0f ? part(c + i, kRows + row) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            o[i] = fmaf(y.x, others, o[i] * own), o[i + 1] = fmaf(y.y, others, o[i + 1] * own);
                            o[i + 2] = fmaf(y.z, others, o[i + 2] * own), o[i + 3] = fmaf(y.w, others, o[i + 3] * own);
                        }
                    }
                    if (row < rows && done) {
                        store_out16(p, out + c, o, factors);
                    } else if (row < rows) {
#pragma unroll
                        for (int i = 0; i < 16; i += 4) part(c + i, kRows * block + row) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    }
                }
                if (!done && row < rows) {
                    slot[kUnitRows * D + kRows * block + row] = m;
                    slot[kUnitRows * D + kUnitRows + kRows * block + row] = l;
                }
                __syncwarp();
            }
            if (warp == 4 && lane == 0 && !done && u.r0 == 0)  // this CTA's blocks of the join have it: the last tile's CTA is its last
                *record = PrefixRecord{cur.g, u.pair, u.block, static_cast<short>(u.rows),
                                       static_cast<short>(cta_of(total, mul_div(total, blockIdx.x + 1, ctas) - cur.left - cur.at + start_places(p) +
                                                                            static_cast<long long>(u.weight) * (u.tiles - 1), ctas) - static_cast<int>(blockIdx.x) + 1)};
            tc_fence_before();
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        // ------------------------------------------------------------ unpack
        // A thread's chunks (16 bytes of codes: 32 dims, two scales) are the same place of rows kStep apart.
        constexpr int kPerRow = D / 32, kStep = 32 * kUnpackWarps / kPerRow, kChunks = kTok / kStep, kAtOnce = kChunks < 4 ? kChunks : 4;
        const int row0 = (tid - 384) / kPerRow, pc = (tid - 384) % kPerRow;
        const int lc = pc ^ (kv4_swizzle(row0, D / 16) >> 1);  // the dims: 32 lc .. (rows 8 apart have the same order)
        uint32_t dst[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) dst[j] = (lc >> 1) * W::kKvBlock + sw128_offset(row0, (lc & 1) * 4 + j);
        const uint32_t code_off = row0 * (D / 2) + pc * 16, scale_off = W::kCodes + row0 * (D / 16) + 2 * lc;
        for (; cur.left > 0 && !failed; next_unit(p, pairs, cur)) {
            const PrefixUnit u = unit_at(p, pairs, cur);
            for (int r = u.r0; r < u.r1 && !failed; ++r, ++n) {
                const int s = n % kStages, there = u.x.end - r * kTok;
                for (int part = 0; part < 2; ++part) {
                    const int use = 2 * n + part, raw = use % kRaw;
                    if (!warp_wait(raw_full + 8 * raw, static_cast<uint32_t>(use / kRaw) & 1u) ||
                        (n >= kStages && !warp_wait((part ? v_free : k_free) + 8 * s, static_cast<uint32_t>(n / kStages - 1) & 1u))) {
                        failed = true;
                        break;
                    }
                    const uint32_t bad = bad_s[n & 7];
                    const unsigned char* codes = sm + W::kOffRaw + raw * W::kRawBytes;
                    unsigned char* tile = sm + (part ? W::kOffV : W::kOffK) + s * W::kKvBytes;
                    const bool whole = there >= kTok && bad == 0;
#pragma unroll
                    for (int c0 = 0; c0 < kChunks; c0 += kAtOnce) {
                        uint4 w[kAtOnce];
                        uint32_t scales[kAtOnce];
#pragma unroll
                        for (int c = 0; c < kAtOnce; ++c) {
                            w[c] = *reinterpret_cast<const uint4*>(codes + code_off + (c0 + c) * kStep * (D / 2));
                            scales[c] = *reinterpret_cast<const uint16_t*>(codes + scale_off + (c0 + c) * kStep * (D / 16));
                        }
                        if (!whole) {
#pragma unroll
                            for (int c = 0; c < kAtOnce; ++c) {
                                const int row = row0 + (c0 + c) * kStep;
                                if (row >= there || ((bad >> (row >> 4)) & 1u)) scales[c] = 0, w[c] = make_uint4(0u, 0u, 0u, 0u);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < kAtOnce; ++c) {
                            const uint32_t s0 = scale_twice(scales[c], 0), s1 = scale_twice(scales[c], 1), word[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                uint32_t v[4];
                                unpack(word[j], j < 2 ? s0 : s1, v);
                                *reinterpret_cast<uint4*>(tile + dst[j] + (c0 + c) * (kStep / 8) * 1024) = make_uint4(v[0], v[1], v[2], v[3]);
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_local(raw_free + 8 * raw);
                        mbar_arrive_local((part ? v_full : k_full) + 8 * s);
                    }
                }
            }
        }
    }
    __syncwarp();
    // (in the issuing warp the elected lane alone knows, whichever it is)
    if (__any_sync(~0u, failed) && lane == 0) atomicOr(&g_kv4_prefix_error, kErrWaitTimeout);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmCols);
    }
}

// Joins the partial results of the units that several CTAs shared. An item is 32 rows and four dims of such a unit (a warp reads whole lines);
// the items of all units are dealt out to the warps, each of which finds its own in the CTAs' records: a unit over 19 CTAs has as many warps
// as one over two.
template <int D>
__global__ void __launch_bounds__(256) kv4_prefix_join_kernel(const __grid_constant__ AttnParams p, int ctas) {
    constexpr size_t slot_floats = kUnitRows * (D + 2);
    constexpr int kPerLane = kMaxSms / 32;
    const int lane = threadIdx.x & 31;
    griddep_launch_dependents();  // the pass over the own caches
    griddep_wait();
    const PrefixRecord* records = reinterpret_cast<const PrefixRecord*>(p.records);
    int mine = 0, counts[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int at = lane * kPerLane + i;
        counts[i] = at < ctas ? ((records[at].rows + 31) >> 5) * (D / 4) : 0;
        mine += counts[i];
    }
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, sum, o);
        if (lane >= o) sum += y;
    }
    const int total = __shfl_sync(~0u, sum, 31);
    for (int item = blockIdx.x * 8 + (threadIdx.x >> 5); item < total; item += gridDim.x * 8) {
        const int src = __ffs(__ballot_sync(~0u, sum > item)) - 1;
        int left = item - __shfl_sync(~0u, sum - mine, src), first = src * kPerLane;
#pragma unroll
        for (int i = 0; i < kPerLane - 1; ++i) {
            const int c = __shfl_sync(~0u, counts[i], src);
            if (first == src * kPerLane + i && left >= c) left -= c, ++first;
        }
        const PrefixRecord rec = records[first];
        const int row = left / (D / 4) * 32 + lane, c = left % (D / 4) * 4;
        if (row >= rec.rows) continue;
        const float* base = p.part + static_cast<size_t>(first) * 2 * slot_floats;
        auto slot = [&](int i) -> const float* { return base + (i == 0 ? 1 : 2 * static_cast<size_t>(i)) * slot_floats; };
        // the parts one by one, with the running maximum: one round of reads
        float mm = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int i = 0; i < rec.parts; ++i) {
            const float* s = slot(i);
            const float ms = s[kUnitRows * D + row], ls = s[kUnitRows * D + kUnitRows + row];
            const float4 y = *reinterpret_cast<const float4*>(s + c * kUnitRows + 4 * row);
            const float v = fmaxf(mm, ms), f = mm == v ? 1.0f : exp2_approx(mm - v), g = ms == -INFINITY ? 0.0f : exp2_approx(ms - v);
            mm = v;
            l = fmaf(l, f, ls * g);
            o.x = fmaf(o.x, f, y.x * g), o.y = fmaf(o.y, f, y.y * g), o.z = fmaf(o.z, f, y.z * g), o.w = fmaf(o.w, f, y.w * g);
        }
        Unit x{};
        x.l = rec.pair / p.c.kv_heads;
        x.h = rec.pair % p.c.kv_heads;
        const size_t out = q_row(p, rec.g, x, rec.block * kUnitRows + row);
        const OutFactors f = out_factors(p, out, mm, l);
        *reinterpret_cast<float4*>(p.prefix_out + out + c) = make_float4(o.x * f.own, o.y * f.own, o.z * f.own, o.w * f.own);
        if (c == 0) keep_sums(p, out, mm, l);
    }
}

template <int D>
cudaError_t launch_one(const AttnParams& p, cudaStream_t stream) {
    using W = Prefix<D>;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use its shared memory
    if (dev >= 64 || !(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        e = cudaFuncSetAttribute(kv4_prefix_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, W::kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    // no more CTAs than there can be work for, as far as the tables' lengths say
    const long long tiles = std::max<long long>(((static_cast<long long>(p.c.max_pages) << p.c.page_shift) + kTok - 1) / kTok, 1);
    const long long units = (static_cast<long long>(p.c.T) * p.group / kUnitRows + p.c.B) * p.c.L * p.c.kv_heads;
    const long long places = units * (start_places(p) + kDual * tiles);
    const int ctas = static_cast<int>(std::min<long long>(std::max<long long>(places / kLeastPlaces, 1), std::min(sms, kMaxSms)));
    kv4_prefix_kernel<D><<<ctas, kThreads, W::kSmem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * ctas);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv4_prefix_join_kernel<D>, p, ctas);
}

}  // namespace

// The workspace is that of the window kernel: two partial results of 256 rows for each of up to 192 CTAs, a set of sums, a record.
cudaError_t launch_kv4_prefix(AttnParams p, cudaStream_t stream) {
    p.sums = p.part + static_cast<size_t>(2 * kMaxSms) * 2 * kRows * (p.c.head_dim + 2);
    p.records = p.sums + static_cast<size_t>(2 * kMaxSms) * kRows * p.c.head_dim;
    return p.c.head_dim == 64 ? launch_one<64>(p, stream) : launch_one<128>(p, stream);
}

cudaError_t read_kv4_prefix_error(uint32_t* out) {
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_kv4_prefix_error, sizeof(v));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_kv4_prefix_error, &zero, sizeof(zero));
    *out = v;
    return e;
}

}  // namespace gdn
