// paged_attention_prefill: the attention of a ragged batch of new tokens over
// the paged cache, on the fifth-generation tensor cores (tcgen05).
//
// What is computed.  Sequence s has L_s cached positions, the last n_s of them
// its new tokens' own; new token i attends over positions t < L_s - n_s + i + 1:
//     out = sum_t p_t V_t,   p = softmax(scale * q . K_t).
// Rows are (token, query head) pairs of one KV head, token-major, so a KV
// head's whole group shares every K/V byte that reaches the SM.
//
// How.  A work item is 256 rows (two tiles of 128, the MMA's M) over a run of
// 128-position steps.  The items are listed longest first, by the plan kernel or
// (a single call of moderate size) by every CTA for itself, and one persistent
// CTA per SM takes them in snake order.  Per step and tile i
//     S_i = Q_i K^T    tcgen05.mma 128 x 128, Q_i and K from shared memory, S_i
//                      fp32 in tensor memory (TMEM)
//     P_i = 2^(S_i - ref)   one thread a row; the reference maximum moves only
//                      when a score passes it by more than 2^8 (O_i is then
//                      rescaled in TMEM); P_i, rounded to the input type (the
//                      MMA's operand type, the price of its rate: bf16 outputs
//                      are 2.3e-3 from 64 bits where a form in fp32, rounded
//                      once, is 1.7e-3; f16 2.5e-4 and 1.9e-4), takes S_i's
//                      place in TMEM; the row sum stays fp32 and sums the
//                      weights before rounding
//     O_i += P_i V     tcgen05.mma, A from TMEM, V from shared memory read as an
//                      MN-major operand, O_i fp32 in TMEM
// The two tiles are a step's ping and pong: while one tile's softmax runs, the
// tensor cores work on the other's products, in turns.  TMEM is full: S_0 S_1 O_0
// O_1 of 128 columns each.  At head_dim 64 the O take half of that, P has columns
// of its own and the next S is issued as soon as this one is in registers, without
// turns (99 to 97 us over 24 ragged prompts of 5 to 2000 tokens, 12 heads over 4).
//
// What bounds it.  A step of two tiles is 2048 tensor cycles at head_dim 128 and
// takes 2650 to 2850: a tile's S, softmax, P V and next S are a serial chain, under
// which only the other tile's products run.  One prompt of 8192 tokens, 64 heads
// over 8: 690 us, 1590 TFLOP/s, 83% of the rate measured for a large bf16 matrix
// product, in the first milliseconds; 754 us, 1460 TFLOP/s, once the power cap
// holds the clock down, 86% of that product's own rate then.  Start-up takes 7 us without a plan, 9 with one
// (plan 3 to 4, first S 5, second 1.6: latencies and instruction fetch), and the
// items' ends spread by a tenth of a call.  Tiles of up to 128 rows compute half as
// much over the same K and V: where all CTAs run such, a step takes 1.41 us, the HBM
// rate.  At head_dim 64 there are as many exponentials for half the products: 950 to
// 990 TFLOP/s over 16384 tokens, 16 heads over 4.  No unit is the bound there either
// (8192 tokens: tensor pipe 40% busy, exponentials' unit 40%, issue slots 52%): the
// softmax is two warps a scheduler, waiting for TMEM and for each other.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1 (they also write the output),
// 13 loads Q tiles, 8 and 10 stream the K and V blocks (TMA, one
// box per block and 128-byte column plane), 9 and 11 issue tile 0's and 1's
// MMAs (a warp's program order is what orders S_i after the O_i that reads P_i),
// 12 and 14 clean V tiles, 15 decodes the work items.
//
// Masked positions.  A masked score is replaced before the maximum, whatever K
// holds there.  A masked position's weight is 0, but 0 * V is NaN where V is
// not finite, so on the steps that some row sees only in part, and on a
// sequence's last, two warps look through the V rows that not every row sees:
// slots past the end become zeros, non-finite elements too, after their first
// position per column is noted; the epilogue then adds inf or NaN to exactly
// the rows that see them.
//
// E4M3 pools.  Warp 8 streams tiles of codes, and three warps (10, 12, 13: one a scheduler) expand
// them into the ring as f16, where every code is exact, and clean V on the way;
// K's scale multiplies the scores, V's the output.  The products run in f16: a
// bf16 query tile is converted in place by its softmax warps.  A step takes 1.7 us
// (1.45 over 16-bit pools), which the three warps' expansion sets: 16 groups of eight
// rows, two a warp at a time, are three trips (issue slots 45%, tensor pipe 48% busy).
//
// Trees (paged_attention_tree).  The last n_s <= 64 positions are a tree's nodes, and
// token i sees of them those of its 64-bit mask, none after itself: tiles, steps and
// plan stay those of the causal call.  On the one or two steps that hold nodes a
// thread masks its row by its word, and V's non-finite elements are noted as a word of
// nodes a column, since what two rows see is no longer one a part of the other.  64
// trees of 16 over 512 to 4096 positions, 32 heads over 8: 98.5 us, 5.6 TB/s (steps at
// the HBM rate, 1.5 us; start-up 9 us; blocks read once leave L2 first, 102 without);
// 128 ragged trees of 1 to 64, 64 heads over 8: 156 us, where a step of two tiles takes
// 1.72 us from HBM and an item 3.4 us beside.  At head_dim 64 the first batch takes
// 74 us, 54% of the HBM rate: 0.9 us a step, the chain of a lone tile's S, softmax, P V.
// Over E4M3 pools: 64 trees of 60, 149 us, two tiles, whose steps the expansion sets
// (1.7 us).  Where no tree of the batch has more than 128 rows (LONE), the second tile's
// softmax warps would be idle, so they expand codes too (eight warps in all, one trip a
// tile) and S of the next step runs under the softmax, in the other tile's columns: 64
// trees of 26, 115 to 101 us, 1.35 us a step.  No pipe is full there and no one part is
// the bound: without the expansion 94 us, without the exponentials 96, without the first
// pass over S 91, without its wait for the last P V where nothing is rescaled 102.  Two
// warpgroups on even and odd steps, 640 threads, took 111 to 125.
//
// Every wait is bounded in wall time; a CTA that gives up raises the error
// word, gives its copies and products in flight time to land and frees its TMEM.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "pkv_decode_common.cuh"
#include "pkv_prefill_common.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

namespace {

constexpr int kStep = kPrefillStep;
constexpr int kSub = kPrefillSub;

template <int D, bool KV8 = false, bool TREE = false, bool LONE = false>
struct PfGeo {
    static constexpr int kThreads = 512;
    static constexpr int kLoadK = 8, kLoadV = 10, kMma = 9, kClean = 12, kLoadQ = KV8 ? 14 : 13, kPlan = 15;   // (9 and 11: MMAs; 12 and 14: cleaning; E4M3: 10, 12 and 13 expand)
    static constexpr int kHalves = D * 2 / 128;             // 128-byte column planes of a tile
    static constexpr int kPlane = 128 * 128;                // bytes of a plane: 128 rows
    static constexpr int kTile = kHalves * kPlane;          // a K, V or Q tile
    // ring of K and V tiles, in turn; over an E4M3 pool a tile less in favour of two tiles of codes (a tree's words of nodes
    // leave no room for those: three of each)
    static constexpr int kStages = KV8 ? (TREE && !LONE ? 3 : 4) : D == 128 ? 5 : 10;
    static constexpr int kCodes = KV8 ? (TREE ? 3 : 2) : 0;   // staged tiles of codes (128 rows of D bytes)
    static constexpr int kCodeTile = 128 * D;
    static constexpr int kTiles = LONE ? 1 : 2;             // an item's tiles of rows at most, a softmax warpgroup each
    static constexpr int kConverters = LONE ? 8 : 3;        // warps 4-7 and 10-13, a trip a tile; else warps 10, 12 and 13: on two of the schedulers (10, 12, 14) 120 us, on three 117 (8 chunks of 256 to 512)
    static constexpr size_t kRing = kTiles * size_t(kTile); // after the Q tiles
    static constexpr size_t kCode = kRing + size_t(kStages) * kTile;
    static constexpr size_t kBars = kCode + size_t(kCodes) * kCodeTile;
    static constexpr int kItems = 4;                        // items decoded ahead
    static constexpr int kItemReaders = 15;                 // warps that read each
    static constexpr int kNumBars = 3 * kStages + 21 + 2 * kItems + 2 * kCodes;
    static constexpr int kTags = LONE ? 8 : 3;              // warps that list non-finite V elements, at most
    static constexpr size_t kMisc = kBars + kNumBars * 8;   // TMEM address, abort flag, tags [kTags], epilogues [8]
    static constexpr size_t kBad = (kMisc + 40 + 4 * kTags + 15) / 16 * 16;   // first positions of non-finite V elements: [2 warps][+inf, -inf][D], or [3 warps][NaN][D]
    // a tree's: the nodes that hold them, 64 bits, [+inf, -inf][D] (a warp cleans half the columns), or [kTags][NaN][D]
    static constexpr size_t kList = kBad + size_t(TREE && KV8 ? 2 * kTags : 4) * D * 4;    // [kItems] decoded items
    static constexpr size_t kBytes = kList + kItems * 64;
    static_assert(!KV8 || D == 128, "E4M3 pools: a row of codes is one 128-byte plane");
    static constexpr uint32_t kColS = 0, kColO = 256, kTmemCols = 512;
    // P's columns: its own at head_dim 64, where they are left over; S's at 128
    static constexpr bool kOwnP = D == 64;
    static constexpr uint32_t kColP = kOwnP ? 384 : kColS, kStrideP = kOwnP ? 64 : 128;
    // registers a thread: 512 threads start with 128; the softmax warpgroups take 192, the others keep 64
    static constexpr int kRegsSoftmax = 192, kRegsOther = 64;
    static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= kThreads * 128, "the split fits the launch's registers");
    static_assert(kBytes <= 232448, "fits one SM");
};

// A bounded wait (false: gave up, or another role did).  Short code: every role waits in its inner loop,
// and the roles share the instruction cache.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, unsigned parity, volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs) return false;
    return true;
}

// One work item, decoded by the plan warp into shared memory and read by every other role.
struct alignas(16) Item {
    int s, kvh, tile, step0;
    int qs, n, L, split;
    int rows;                        // query rows of the item (0: an entry to skip; -1: no more items)
    int nst[2];                      // steps of each tile
    int lim0;                        // positions every row of the item sees
    int end[2];                      // position after the last one each tile sees in the item
    int pad[2];
    __device__ __forceinline__ int steps_of(int i) const { return i ? nst[1] : nst[0]; }
    __device__ __forceinline__ int end_of(int i) const { return i ? end[1] : end[0]; }
    __device__ __forceinline__ int steps() const { return max(nst[0], nst[1]); }
    __device__ __forceinline__ int stop() const { return max(end[0], end[1]); }
    // V rows [lo, nv16) of step j that not every row sees (nv: the item's positions in the step)
    __device__ __forceinline__ void partial(int j, int& lo, int& nv, int& nv16) const {
        const int tok0 = (step0 + j) * kStep;
        nv = min(kStep, stop() - tok0);
        nv16 = (nv + 15) & ~15;
        lo = max(0, lim0 - tok0);
    }
};

// (Plan, tables and q are read with ld.cg, never ld.nc: the compiler may move an ld.nc above the
// wait for the kernel that writes them.)
// The entry of this CTA's item in a round: fetched a round ahead of its use.
struct Entry {
    int4 x, y;
    int kvh;
    bool live;
};
__device__ __forceinline__ Entry fetch_entry(const PrefillArgs& a, int total, int round) {
    const int g = gridDim.x, b = blockIdx.x;
    const long long w = static_cast<long long>(round) * g + ((round & 1) ? g - 1 - b : b);
    Entry n{};
    n.live = w < total;
    if (n.live) {
        const int e = pf::div(static_cast<int>(w), a.by_kv_heads);
        n.kvh = static_cast<int>(w) - e * a.num_kv_heads;
        n.x = __ldcg(a.items + 2 * e);
        n.y = __ldcg(a.items + 2 * e + 1);
    }
    return n;
}
// The same without a plan: this CTA's item is tile blockIdx.x / KV heads of the batch, counted by a warp over the
// sequences.
__device__ __forceinline__ Entry find_entry(const PrefillArgs& a) {
    Entry n{};
    const int lane = threadIdx.x & 31;
    const int e = pf::div(static_cast<int>(blockIdx.x), a.by_kv_heads);
    int before = 0;
    for (int s0 = 0; s0 < a.num_seqs; s0 += 32) {
        pf::Seq q{0, 0, 0};
        if (s0 + lane < a.num_seqs) q = pf::load_seq(a, s0 + lane, blockIdx.x == 0);
        const int mine = pf::tiles_of(q, a.group), upto = before + pf::warp_scan(mine);
        const unsigned m = __ballot_sync(0xffffffffu, upto > e);
        if (!n.live && m) {
            const int k = __ffs(m) - 1;
            n.live = true;
            n.kvh = static_cast<int>(blockIdx.x) - e * a.num_kv_heads;
            n.x = make_int4(s0 + k, e - __shfl_sync(0xffffffffu, upto - mine, k), 0, 1 << 23);
            n.y = make_int4(__shfl_sync(0xffffffffu, q.start, k), __shfl_sync(0xffffffffu, q.n, k),
                            __shfl_sync(0xffffffffu, q.len, k), 0);
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return n;
}
template <bool TREE, bool LONE>
__device__ __forceinline__ void read_item(const PrefillArgs& a, const Entry& n, Item& it) {
    const int4 x = n.x, y = n.y;
    it.kvh = n.kvh;
    it.s = x.x;
    it.tile = x.y;
    it.step0 = x.z;
    const int step1 = x.w;
    it.qs = y.x;
    it.n = y.y;
    it.L = y.z;
    it.split = y.w;
    it.rows = 0;
    it.nst[0] = it.nst[1] = it.end[0] = it.end[1] = 0;
    it.lim0 = 0;
    const int nparts = it.split & 255, part = (it.split >> 8) & 255, base = it.split >> 16;
    // a plan of other arguments: skip the entry rather than leave the buffers
    if (it.s < 0 || it.s >= a.num_seqs || it.tile < 0 || it.step0 < 0 || step1 < it.step0 || it.qs < 0 || it.n <= 0 ||
        it.qs + static_cast<long long>(it.n) > a.num_tokens || it.L < 0 || it.L > a.max_seq_len ||
        static_cast<long long>(it.tile) * kPrefillRows >= static_cast<long long>(it.n) * a.group || it.split < 0 ||
        (it.split != 0 && (part >= nparts || base + nparts > a.part_cap)) || (TREE && it.n > kTreeNodes) ||
        (LONE && it.n * a.group > kSub)) {
        if ((threadIdx.x & 31) == 0) raise_error(a.err, kErrBounds);
        return;
    }
    const int row0 = it.tile * kPrefillRows;
    it.rows = min(kPrefillRows, it.n * a.group - row0);
    const int past = it.L - it.n;
    it.lim0 = max(0, TREE ? past : past + pf::div(row0, a.by_group) + 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = min(kSub, it.rows - i * kSub);
        if (r > 0) {
            const int lim = past + pf::div(row0 + i * kSub + r - 1, a.by_group) + 1;      // the tile's last row's
            it.end[i] = max(0, min(step1 < (1 << 23) ? step1 * kStep : it.L, min(lim, it.L)));
            it.nst[i] = max(0, (it.end[i] + kStep - 1) / kStep - it.step0);
        }
    }
}

__device__ __forceinline__ uint64_t pack64(float x, float y) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack64(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// One lane of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// A place in the ring: its slot, and the parity its barriers have there.
template <int N>
struct Ring {
    int slot = 0;
    unsigned phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == N) {
            slot = 0;
            phase ^= 1u;
        }
    }
};
template <typename T>
__device__ __forceinline__ T from_float(float x) {
    const uint32_t w = Mma<T>::pack(x, x);
    return *reinterpret_cast<const T*>(&w);
}
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool keep) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(keep ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t x) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
    return r;
}
// 4 x 4 transposition over a quad: lane q's register i becomes lane i's register q.
__device__ __forceinline__ void quad_transpose(uint32_t (&w)[4]) {
    const int q = threadIdx.x & 3;
#pragma unroll
    for (int s = 1; s <= 2; s <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i & s) continue;
            const uint32_t give = (q & s) ? w[i] : w[i ^ s];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, give, s);
            if (q & s) w[i] = got;
            else w[i ^ s] = got;
        }
    }
}

// Evict first, or the usual policy.  Blocks that no other item of their sequence reads leave L2 first: 64 trees of 16 over
// 512 to 4096 positions of their own, 110.4 us instead of 112.4.  Prefixes that sequences share keep their place all the
// same, since all that competes with them is loaded alike: 64 sequences with 2048 common positions of 2100 to 5000, 150.6
// instead of 153.2; of 2049 to 2300, 107.1 and 108.2; with 8192 common ones 359.9 and 360.9; 128 with 512 of 600 to 4000,
// 197.2 and 196.5.
__device__ __forceinline__ uint64_t l2_policy(bool first) {
    uint64_t f, n;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(f));
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(n));
    return first ? f : n;
}

// Element offset / D of row r of the item's tile in q / out.
__device__ __forceinline__ int64_t qo_row(const PrefillArgs& a, const Item& it, int r) {
    const int rr = it.tile * kPrefillRows + r;
    const int tok = pf::div(rr, a.by_group);
    return (static_cast<int64_t>(it.qs) + tok) * a.num_heads + it.kvh * a.group + (rr - tok * a.group);
}

// A Q tile into shared memory by one warp's 16-byte asynchronous copies (128-byte swizzle, zeros past the
// rows): the form for group sizes that no TMA box fits.
template <typename T, int D>
__device__ __forceinline__ void copy_q(const PrefillArgs& a, const Item& it, int tile, uint32_t qtile) {
    using G = PfGeo<D>;
    constexpr int kCh = D / 8;                               // 16-byte chunks of a row
    constexpr int kRowsAt = 32 / kCh;                        // rows the warp copies at once
    const int lane = threadIdx.x & 31;
    const int ch = lane % kCh, sub = lane / kCh;
    const uint4* q = static_cast<const uint4*>(a.q) + ch;
#pragma unroll 1
    for (int r0 = 0; r0 < kSub; r0 += 32) {
        const int mine = tile * kSub + r0 + lane;            // each lane places one row, the others ask it
        const int at = mine < it.rows ? static_cast<int>(qo_row(a, it, mine)) : -1;
#pragma unroll 4
        for (int u = 0; u < 32; u += kRowsAt) {
            const int row = __shfl_sync(0xffffffffu, at, u + sub);
            cp_async_16_or_zero(dec::swz(qtile + (ch >> 3) * G::kPlane, r0 + u + sub, ch & 7),
                                q + static_cast<int64_t>(max(row, 0)) * kCh, row >= 0);
        }
    }
    cp_async_commit();
    cp_async_wait_all();
    fence_proxy_async_smem();
    __syncwarp();
}

// ---------------------------------------------------------------- planning by the CTA itself
struct LocalPlan {
    int start[kPrefillLocal], n[kPrefillLocal], len[kPrefillLocal];      // sequences
    int first[kPrefillLocal + 1];                                        // their first tiles
    int steps[kPrefillLocal], seq[kPrefillLocal], slot[kPrefillLocal];   // tiles
    alignas(16) int key[kPrefillLocalItems];                             // items: length and order
    int ref[kPrefillLocalItems];                                         // tile, part
    int order[kPrefillLocalItems];                                       // by rank
    int scan[16], wmax[16], wsum[16];
    pf::Choice choice;
};

// Exclusive scan of v over the block; *total: its sum.
__device__ __forceinline__ int block_scan(int v, int* scan, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int inc = pf::warp_scan(v);
    __syncthreads();
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    const int w = pf::warp_scan(lane < 16 ? scan[lane] : 0);
    const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
    *total = __shfl_sync(0xffffffffu, w, 15);
    return inc - v + (warp > 0 ? before : 0);
}

// The plan kernel's plan (pkv_prefill_plan.cu), made by a CTA of 512 threads in its own shared memory and so ordered
// without atomics, the same in every CTA: an item's rank is the number of longer ones and of equally long ones
// before it.  Returns the number of items a KV head.  CTA 0 reports bad bounds and lists the split tiles.
__device__ __forceinline__ int local_plan(const PrefillArgs& a, LocalPlan& lp) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const bool report = blockIdx.x == 0;
    pf::Seq q{0, 0, 0};
    if (t < a.num_seqs) q = pf::load_seq(a, t, report);
    lp.start[t] = q.start;
    lp.n[t] = q.n;
    lp.len[t] = q.len;
    int tiles;
    lp.first[t] = block_scan(pf::tiles_of(q, a.group), lp.scan, &tiles);
    if (t == 0) lp.first[kPrefillLocal] = tiles;
    tiles = min(tiles, kPrefillLocal);                       // (more only where the starts decrease: reported)
    __syncthreads();
    int st = 0, k = 0;
    if (t < tiles) {
#pragma unroll 1
        for (int w = kPrefillLocal / 2; w > 0; w >>= 1)
            if (lp.first[k + w] <= t) k += w;
        st = pf::tile_steps(a, pf::Seq{lp.start[k], lp.n[k], lp.len[k]}, t - lp.first[k]);
    }
    lp.steps[t] = st;
    lp.seq[t] = k;
    const int wm = __reduce_max_sync(0xffffffffu, st), ws = __reduce_add_sync(0xffffffffu, st);
    if (lane == 0) {
        lp.wmax[warp] = wm;
        lp.wsum[warp] = ws;
    }
    __syncthreads();
    const int maxs = __reduce_max_sync(0xffffffffu, lane < 16 ? lp.wmax[lane] : 0);
    unsigned long long sum = 0;
    for (int w = 0; w < 16; ++w) sum += lp.wsum[w];
    const int P = pf::choose_part<16>(a, lp.choice, lp.steps, tiles, maxs, static_cast<float>(sum));
    // items, partial slots and split tiles before this tile, in one scan (11, 11 and 10 bits)
    const int parts = t < tiles ? pf::parts_of(st, P) : 0;
    int total;
    const int at = block_scan(parts | (parts > 1 ? parts << 11 | 1 << 22 : 0), lp.scan, &total);
    const int item0 = at & 2047, slot = at >> 11 & 2047, merge = static_cast<unsigned>(at) >> 22;
    const int items = total & 2047;
    lp.slot[t] = slot;
    const int len = pf::part_len(st, parts);
    for (int p = 0; p < parts; ++p) {
        const int s0 = min(st, p * len);
        lp.key[item0 + p] = min(min(st, s0 + len) - s0, (1 << 21) - 1) << 10 | (kPrefillLocalItems - 1 - item0 - p);
        lp.ref[item0 + p] = t << 8 | p;
    }
    if (report) {
        if (parts > 1) a.merges[merge] = make_int4(prefill_split(parts, 0, slot), t - lp.first[k], lp.start[k], lp.n[k]);
        if (t == 0) a.header[1] = static_cast<unsigned>(total) >> 22;
    }
    if (t < 3 && items + t < kPrefillLocalItems) lp.key[items + t] = -1;      // (the last four are read whole)
    __syncthreads();
    const bool alone = items * a.num_kv_heads <= static_cast<int>(gridDim.x);       // an item a CTA at most: in any order
    const int n = alone ? 0 : items;
#pragma unroll 1
    for (int i = t; i < items; i += 512) {
        const int key = lp.key[i];
        int rank = alone ? i : 0;
        const int4* all = reinterpret_cast<const int4*>(lp.key);
#pragma unroll 4
        for (int j = 0; 4 * j < n; ++j) {
            const int4 o = all[j];
            rank += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
        }
        lp.order[rank] = i;
    }
    lp.wsum[warp] = P;                                       // (for the entries)
    __syncthreads();
    return items;
}

// The entry of rank e of a local plan.
__device__ __forceinline__ Entry local_entry(const LocalPlan& lp, int e, int kvh) {
    const int P = lp.wsum[0], ref = lp.ref[lp.order[e]], t = ref >> 8, p = ref & 255, k = lp.seq[t], st = lp.steps[t];
    const int parts = pf::parts_of(st, P), len = pf::part_len(st, parts), s0 = min(st, p * len);
    Entry n;
    n.x = make_int4(k, t - lp.first[k], s0, min(st, s0 + len));
    n.y = make_int4(lp.start[k], lp.n[k], lp.len[k], parts > 1 ? prefill_split(parts, p, lp.slot[t]) : 0);
    n.kvh = kvh;
    n.live = true;
    return n;
}

// T: the products' type; KV8: E4M3 pools (codes expanded to f16, every one exact there); OT: q's and out's.
// TREE: the last n positions are a tree's nodes, of which row (token i, head) sees those of token i's mask.
// LONE (E4M3 pools): no tree has more than 128 rows of a KV head, every item is a single tile.
template <typename T, int D, bool KV8, typename OT, bool TREE, bool LONE>
__device__ __forceinline__ void prefill_cta(const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                                            const PrefillArgs& a) {
    using G = PfGeo<D, KV8, TREE, LONE>;
    constexpr int ST = G::kStages;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr bool kConvertQ = !std::is_same<T, OT>::value;     // bf16 queries over an E4M3 pool: to f16 in place
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* ring = smem + G::kRing;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + G::kBars);
    uint64_t* full = bars;                          // [ST] a tile landed (TMA bytes)
    uint64_t* empty = bars + ST;                    // [ST] the products that read it are done (both MMA warps' commits), the cleaning warps past it
    uint64_t* clean = bars + 2 * ST;                // [ST] the cleaning warps are past the tile
    uint64_t* q_full = bars + 3 * ST;               // [2] an item's Q tile is in shared memory (TMA bytes, or the Q warp)
    uint64_t* q_empty = q_full + 2;                 // [2] an item's last S product done: its Q is read (MMA commit)
    uint64_t* s_full = q_full + 4;                  // [2] a step's S in TMEM, all earlier products done (MMA commit)
    uint64_t* p_full = q_full + 6;                  // [2][2] half a step's P (kOwnP: [2][0], all of it) in TMEM, O rescaled (softmax threads)
    uint64_t* o_full = q_full + 10;                 // [2] an item's last O product done (MMA commit)
    uint64_t* turn = q_full + 12;                   // [2] the tile may issue its next round (the other's MMA warp)
    uint64_t* q_raw = q_full + 14;                  // [2] the tile before its conversion to f16 (kConvertQ)
    uint64_t* fin = q_full + 16;                    // every product issued is done (both MMA warps' commits)
    uint64_t* s_read = q_full + 17;                 // [2] kOwnP: a step's S in registers (softmax threads)
    uint64_t* o_step = q_full + 19;                 // [2] kOwnP: a step's O product done (MMA commit)
    uint64_t* item_full = q_full + 21;              // [kItems] an item is decoded (plan warp)
    uint64_t* item_empty = item_full + G::kItems;   // [kItems] every reader has read it
    uint64_t* code_full = item_empty + G::kItems;   // [kCodes] a tile of codes landed (TMA bytes)
    uint64_t* code_empty = code_full + G::kCodes;   // [kCodes] it is expanded (converter warps)
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + G::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + G::kMisc + 4);
    volatile int* epilogues = abort_flag + 1 + G::kTags;       // [8] items a softmax warp is through with
    volatile int* bad_tag = abort_flag + 1;         // [kTags] the item whose non-finite V elements a warp's table lists (-1: none)
    int* bad = reinterpret_cast<int*>(smem + G::kBad);      // (kBad)
    unsigned long long* bad_nodes = reinterpret_cast<unsigned long long*>(smem + G::kBad);      // (TREE)
    static_assert(G::kBad % 8 == 0, "the node masks are 64-bit words");

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], KV8 ? G::kConverters : 1);
            mbar_init(&empty[i], KV8 ? G::kTiles : 4);
            mbar_init(&clean[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], kConvertQ ? kSub : 1);
            mbar_init(&q_raw[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[2 * i], kSub);
            mbar_init(&p_full[2 * i + 1], kSub);
            mbar_init(&o_full[i], 1);
            mbar_init(&turn[i], 1);
            mbar_init(&s_read[i], kSub);
            mbar_init(&o_step[i], 1);
        }
        for (int i = 0; i < G::kItems; ++i) {
            mbar_init(&item_full[i], 1);
            mbar_init(&item_empty[i], G::kItemReaders);
        }
        for (int i = 0; i < G::kCodes; ++i) {
            mbar_init(&code_full[i], 1);
            mbar_init(&code_empty[i], G::kConverters);
        }
        mbar_init(fin, G::kTiles);
        for (int i = 0; i < 8; ++i) epilogues[i] = 0;
        for (int i = 0; i < G::kTags; ++i) bad_tag[i] = -1;
        // the 128B swizzle and the MMA descriptors assume 1 KB aligned tiles
        const bool misaligned = (smem_u32(smem) & 1023u) != 0;
        if (misaligned) raise_error(a.err, kErrTimeout);
        *abort_flag = misaligned;
        fence_barrier_init();
    }
    if (warp == G::kMma) tc::tmem_alloc(tmem_slot, G::kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependency_wait();
    // ---- without a plan kernel: the CTA plans here, over the still idle tiles, and lane r of the plan warp takes
    // round r's entry
    Entry mine{};
    if (a.local) {
        LocalPlan& lp = *reinterpret_cast<LocalPlan*>(smem);
        static_assert(sizeof(LocalPlan) <= G::kBars, "the scratch lies in the tiles");
        const int total = local_plan(a, lp) * a.num_kv_heads;
        if (warp == G::kPlan) {
            const int g = gridDim.x, b = blockIdx.x, w = lane * g + ((lane & 1) ? g - 1 - b : b);
            const int e = pf::div(w, a.by_kv_heads);
            if (w < total) mine = local_entry(lp, e, w - e * a.num_kv_heads);
        }
        fence_proxy_async_smem();                   // the scratch before the tiles' copies
        __syncthreads();
    }
    Item* list = reinterpret_cast<Item*>(smem + G::kList);
    // The round's item for one warp; false: none is left, or a wait gave up.
    auto get_item = [&](int r, Item& it, bool& ok) {
        const int k = r % G::kItems;
        ok = wait_bar(&item_full[k], (r / G::kItems) & 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        const int4* src = reinterpret_cast<const int4*>(list + k);
        int4* dst = reinterpret_cast<int4*>(&it);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = src[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(&item_empty[k]);
        return it.rows >= 0;
    };

    // Before a cleaning warp writes item r's first entry into its table: every softmax warp is through with the items
    // before r, whose entries it may still read.  Each by itself: a warp whose tile has no steps in several items runs
    // ahead of the others by as many.  False: the wait gave up, or another role did.
    auto table_free = [&](int r) {
        const unsigned long long t0 = globaltimer_ns();
        for (;;) {
            if (!__any_sync(0xffffffffu, lane < 4 * G::kTiles && epilogues[lane] < r)) break;
            if (__any_sync(0xffffffffu, *abort_flag || globaltimer_ns() - t0 > kWaitLimitNs)) return false;
            __nanosleep(200);
        }
        __threadfence_block();
        return true;
    };

    if (warp >= 4 * G::kTiles) {
        regs_dec<G::kRegsOther>();
        if (KV8 && warp == G::kLoadK) {
            // ======================================================== tiles of E4M3 codes, K and V in turn
            const int bs = a.block_size;
            const bool leader = elect_one();
            Ring<G::kCodes> c;
            Item it;
            bool ok = !*abort_flag;
            if (leader) {
                prefetch_tensormap(&tmk);
                prefetch_tensormap(&tmv);
            }
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
                const int n = it.steps(), stop = it.stop();
                // (a KV head that is one item: no other item of the sequence reads its blocks, they leave L2 first)
                [[maybe_unused]] const uint64_t once = TREE ? l2_policy(LONE || it.n * a.group <= kPrefillRows) : 0ull;
                const int32_t* trow = a.block_tables + static_cast<int64_t>(it.s) * a.max_blocks_per_seq;
                auto id_of = [&](int j) {                    // block id `lane` of step j (-1: no block)
                    const int pos = (it.step0 + j) * kStep + lane * bs;
                    return lane * bs < kStep && j < n && pos < stop ? __ldcg(trow + (pos >> a.block_shift)) : -1;
                };
                int nxt = id_of(0);
                for (int j = 0; j < n && ok; ++j) {
                    int id = nxt;
                    nxt = id_of(j + 1);
                    const int tok0 = (it.step0 + j) * kStep;
                    const int nb = (min(stop, tok0 + kStep) - tok0 + bs - 1) >> a.block_shift;
                    if (lane < nb && (id < 0 || static_cast<int64_t>(id) >= a.num_blocks)) {
                        raise_error(a.err, kErrBounds);
                        id = -1;
                    }
                    for (int kv = 0; kv < 2; ++kv) {
                        ok = wait_bar(&code_empty[c.slot], c.phase ^ 1, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const int slot = __shfl_sync(0xffffffffu, c.slot, 0);
                        if (leader) mbar_arrive_expect_tx(&code_full[slot], static_cast<unsigned>(nb * bs * D));
                        uint8_t* dst = smem + G::kCode + slot * G::kCodeTile;
                        for (int b = 0; b < nb; ++b) {
                            const int pb = __shfl_sync(0xffffffffu, id, b);
                            if (leader) {
                                if constexpr (TREE) tma_load_4d_hint(dst + b * bs * D, kv ? &tmv : &tmk, 0, it.kvh, 0, pb, &code_full[slot], once);
                                else tma_load_4d(dst + b * bs * D, kv ? &tmv : &tmk, 0, it.kvh, 0, pb, &code_full[slot]);
                            }
                        }
                        c.next();
                    }
                }
            }
            if (!ok && lane == 0) {
                dec::raise_abort(a.err, abort_flag);
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
            }
        } else if (KV8 && (warp == G::kLoadV || warp == G::kClean || warp == G::kClean + 1 || (LONE && (warp < 8 || warp == G::kMma + 2)))) {
            // ======================================================== codes to f16, V cleaned on the way
            // A lane takes 16 codes, 32 bytes of f16 in one column plane.  A load or store instruction covers
            // eight rows by four lanes a row, and every eight lanes two rows whose numbers differ in bits 0
            // and 2 (q and q ^ 5): the swizzles then put the eight pieces into different banks both times.  A
            // lane's row in a group of eight, and so its swizzle, never changes: addresses advance by 1 KB.
            const int cw = LONE ? (warp < 8 ? warp - 4 : warp - 6) : warp == G::kLoadV ? 0 : warp - G::kClean + 1;
            [[maybe_unused]] int* mine = bad + cw * D;
            const int l3 = lane & 3, rl = (lane >> 3) ^ ((lane >> 2) & 1 ? 5 : 0);
            Ring<ST> c;
            Ring<G::kCodes> q;
            Item it;
            bool ok = !*abort_flag;
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
                const int n = it.steps();
                for (int t = 0; t < 2 * n && ok; ++t) {      // K and V of step t / 2
                    int lo, nv, nv16;
                    it.partial(t >> 1, lo, nv, nv16);
                    const bool look = (t & 1) && lo < nv;    // V that some row does not see
                    const int tok0 = (it.step0 + (t >> 1)) * kStep;
                    ok = wait_bar(&code_full[q.slot], q.phase, abort_flag) && wait_bar(&empty[c.slot], c.phase ^ 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const uint32_t src = smem_u32(smem + G::kCode + q.slot * G::kCodeTile), dst = smem_u32(ring + c.slot * G::kTile);
#pragma unroll 1
                    for (int g0 = cw; g0 < kStep / 8; g0 += 2 * G::kConverters) {      // two groups of eight rows at a time
                        uint32_t x[4][4];                    // [group, plane]
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = 8 * (g0 + (u >> 1) * G::kConverters) + rl;
                            x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0u;                        // slots past the end
                            if (row < nv)
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(x[u][0]), "=r"(x[u][1]), "=r"(x[u][2]), "=r"(x[u][3])
                                             : "r"(dec::swz(src, row, 4 * (u & 1) + l3)));
                        }
                        if (look && 8 * (g0 + G::kConverters) + 7 >= lo) {
                            uint32_t hit = 0;                // (a code of seven ones is NaN)
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                uint32_t any = 0;
#pragma unroll
                                for (int e = 0; e < 4; ++e) any |= ((x[u][e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                                if (any && 8 * (g0 + (u >> 1) * G::kConverters) + rl >= lo) hit |= 1u << u;
                            }
                            if (__any_sync(0xffffffffu, hit != 0)) {                           // rare
                                if (bad_tag[cw] != r) {
                                    ok = table_free(r);
                                    for (int k = lane; k < D; k += 32) {
                                        if constexpr (TREE) bad_nodes[cw * D + k] = 0ull;
                                        else mine[k] = 0x7fffffff;
                                    }
                                    __syncwarp();
                                    if (lane == 0) bad_tag[cw] = r;
                                    __syncwarp();
                                }
#pragma unroll
                                for (int u = 0; u < 4; ++u) {
                                    if (!(hit >> u & 1u)) continue;
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
#pragma unroll 1
                                        for (int b = 0; b < 4; ++b) {
                                            if ((x[u][e] >> (8 * b) & 0x7fu) != 0x7fu) continue;
                                            const int col = 64 * (u & 1) + 16 * l3 + 4 * e + b;
                                            const int pos = tok0 + 8 * (g0 + (u >> 1) * G::kConverters) + rl;
                                            if constexpr (TREE) atomicOr(&bad_nodes[cw * D + col], 1ull << (pos - it.L + it.n));
                                            else atomicMin(&mine[col], pos);
                                            x[u][e] &= ~(0xffu << (8 * b));
                                        }
                                }
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const int row = 8 * (g0 + (u >> 1) * G::kConverters) + rl;
                            if (row >= kStep) break;
                            const uint32_t plane = dst + (u & 1) * G::kPlane;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) h[e] = e4m3x2_to_f16x2(x[u][2 * half + (e >> 1)] >> (16 * (e & 1)));
                                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dec::swz(plane, row, 2 * l3 + half)),
                                             "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                                             : "memory");
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&full[c.slot]);
                        mbar_arrive(&code_empty[q.slot]);
                    }
                    c.next();
                    q.next();
                }
            }
            if (!ok && lane == 0) dec::raise_abort(a.err, abort_flag);
        } else if (warp == G::kLoadK || warp == G::kLoadV) {
            // ======================================================== the K/V ring: one warp for K, one for V
            // An elected lane issues the boxes one after another (some 40 cycles each; left to the lanes
            // side by side the compiler serialises them at 65, and one warp for both K and V then took
            // 2100 cycles a step, as long as the step's products).
            const int kv = warp == G::kLoadV;
            const CUtensorMap* tm = kv ? &tmv : &tmk;
            const int bs = a.block_size;
            const bool leader = elect_one();
            Ring<ST> c;
            if (kv) c.next();
            Item it;
            bool ok = !*abort_flag;
            if (leader) prefetch_tensormap(tm);
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
                const int n = it.steps(), stop = it.stop();
                // (a KV head that is one item: no other item of the sequence reads its blocks, they leave L2 first)
                [[maybe_unused]] const uint64_t once = TREE ? l2_policy(LONE || it.n * a.group <= kPrefillRows) : 0ull;
                const int32_t* trow = a.block_tables + static_cast<int64_t>(it.s) * a.max_blocks_per_seq;
                auto id_of = [&](int j) {                    // block id `lane` of step j (-1: no block)
                    const int pos = (it.step0 + j) * kStep + lane * bs;
                    return lane * bs < kStep && j < n && pos < stop ? __ldcg(trow + (pos >> a.block_shift)) : -1;
                };
                int nxt = id_of(0);
                for (int j = 0; j < n; ++j) {
                    int id = nxt;
                    nxt = id_of(j + 1);
                    const int tok0 = (it.step0 + j) * kStep;
                    const int nb = (min(stop, tok0 + kStep) - tok0 + bs - 1) >> a.block_shift;
                    if (lane < nb && (id < 0 || static_cast<int64_t>(id) >= a.num_blocks)) {
                        raise_error(a.err, kErrBounds);
                        id = -1;                             // outside the tensor map: TMA fills zeros
                    }
                    ok = wait_bar(&empty[c.slot], c.phase ^ 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    const int slot = __shfl_sync(0xffffffffu, c.slot, 0);
                    if (leader) mbar_arrive_expect_tx(&full[slot], static_cast<unsigned>(nb * bs * D * 2));
                    uint8_t* dst = ring + slot * G::kTile;
                    for (int b = 0; b < nb; ++b) {
                        const int pb = __shfl_sync(0xffffffffu, id, b);
                        if (leader) {
#pragma unroll
                            for (int hf = 0; hf < G::kHalves; ++hf) {
                                if constexpr (TREE) tma_load_4d_hint(dst + hf * G::kPlane + b * bs * 128, tm, hf * 64, it.kvh, 0, pb, &full[slot], once);
                                else tma_load_4d(dst + hf * G::kPlane + b * bs * 128, tm, hf * 64, it.kvh, 0, pb, &full[slot]);
                            }
                        }
                    }
                    c.next();
                    c.next();
                }
            }
            if (!ok && lane == 0) {
                dec::raise_abort(a.err, abort_flag);
                const unsigned long long t0 = globaltimer_ns();       // copies in flight land before the CTA ends
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
            }
        } else if (warp == G::kMma || (!LONE && warp == G::kMma + 2)) {
            // ======================================================== one warp a tile issues its MMAs
            // The warp runs the control flow together and one elected lane issues.  These warps run a few
            // hundred instructions a step between the softmax warps' thousands on the same schedulers, so
            // nearly every instruction line is fetched anew; with a warp for each tile one's waits and
            // bookkeeping run beside the other's products.
            const uint32_t kIdS = tc::idesc_f16(kSub, kStep, kBf16, false) | (a.negate_q ? tc::kNegateA : 0u);
            constexpr uint32_t kIdO = tc::idesc_f16(kSub, D, kBf16, true);        // O += P V
            const int i = warp != G::kMma;
            const uint64_t dq = tc::smem_desc_sw128(smem_u32(smem) + i * G::kTile, 16, 1024);
            const uint64_t dk = tc::smem_desc_sw128(smem_u32(ring), 16, 1024);            // ring slot 0 as K
            const uint64_t dv = tc::smem_desc_sw128(smem_u32(ring), G::kPlane, 1024);     // and as V
            const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
            const uint32_t ts = tm + G::kColS + i * 128, to = tm + G::kColO + i * D, tp = tm + G::kColP + i * G::kStrideP;
            const bool leader = elect_one();
            Ring<ST> c;                                      // the next tile of the ring
            unsigned np = 0, nq = 0, nr = 0, nturn = i == 0;   // parities (tile 0 goes first: its turn's phase before the first)
            Item it;
            bool ok = !*abort_flag;
            auto wait = [&](uint64_t* bar, unsigned parity) { return wait_bar(bar, parity, abort_flag); };
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
                const int n = it.steps(), ni = it.steps_of(i);
                // S = Q K^T, or -Q K^T where scale and K's scale together are negative (the softmax takes their magnitude)
                uint32_t id_s = kIdS;
                if (KV8 && __ldcg(a.k_scale + it.kvh) < 0.0f) id_s ^= tc::kNegateA;
                if constexpr (LONE) {
                    // S of the next step before this step's P: into the other tile's columns, so that it runs under the
                    // softmax.  (That buffer's last P is read by a product issued before: in order.)
                    for (int j = -1; j < n; ++j) {
                        Ring<ST> v = c;                      // this step's V (c: its K; in round -1 the first K)
                        if (j >= 0) v.next();
                        Ring<ST> k = v;
                        if (j >= 0) k.next();
                        if (j + 1 < n) {
                            ok = wait(&full[k.slot], k.phase);
                            if (ok && j < 0) {
                                ok = wait(&q_full[0], nq);
                                nq ^= 1u;
                            }
                            if (!ok) break;
                            tc::fence_after_sync();
                            if (leader) {
                                const uint64_t d = dk + static_cast<uint64_t>(k.slot * (G::kTile >> 4));
                                const uint32_t to_s = ts + ((j + 1) & 1) * 128;
#pragma unroll
                                for (int ks = 0; ks < D / 16; ++ks) {
                                    const uint64_t off = ((ks >> 2) * G::kPlane + (ks & 3) * 32) >> 4;
                                    tc::mma_ss(to_s, dq + off, d + off, id_s, ks > 0);
                                }
                                tc::commit(&s_full[(j + 1) & 1]);
                                tc::commit(&empty[k.slot]);
                                if (j + 2 == n) tc::commit(&q_empty[0]);
                            }
                        }
                        if (j < 0) continue;
                        const int b = j & 1, left = it.end_of(0) - (it.step0 + j) * kStep;
                        const uint64_t d = dv + static_cast<uint64_t>(v.slot * (G::kTile >> 4));
                        ok = wait(&full[v.slot], v.phase);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            ok = ok && wait(&p_full[2 * b + half], np >> b & 1u);
                            tc::fence_after_sync();
                            if (ok && leader) {
#pragma unroll
                                for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                                    if (kk * 16 < left)      // (16 a product, none wholly past the end)
                                        tc::mma_ts(to, ts + b * 128 + kk * 8, d + kk * 128, kIdO, (j > 0 || kk > 0) ? 1u : 0u);
                            }
                        }
                        np ^= 1u << b;
                        if (!ok) break;
                        if (leader) {
                            tc::commit(&o_step[0]);
                            if (j == n - 1) tc::commit(&o_full[0]);
                            tc::commit(&empty[v.slot]);
                        }
                        c = k;
                    }
                } else {
                    // round j: O += P V of step j, then S of step j + 1 (round -1: the first S alone)
#pragma unroll 1
                    for (int j = -1; j < n; ++j) {
                        const Ring<ST> v = c;                    // V of this step, then K of the next
                        if (j >= 0) {
                            c.next();
                            ok = wait(&full[v.slot], v.phase);
                            int lo, nv, nv16;
                            it.partial(j, lo, nv, nv16);
                            if (!KV8 && ok && lo < nv16) {       // V that some row sees only in part
                                ok = wait(&clean[v.slot], v.phase);
                            }
                        }
                        const bool more_k = j + 1 < n;
                        if (ok && more_k) ok = wait(&full[c.slot], c.phase);
                        if (!ok) break;
                        auto issue_s = [&]() {                   // (leader) S of step j + 1
                            const uint64_t d = dk + static_cast<uint64_t>(c.slot * (G::kTile >> 4));
#pragma unroll
                            for (int ks = 0; ks < D / 16; ++ks) {
                                const uint64_t off = ((ks >> 2) * G::kPlane + (ks & 3) * 32) >> 4;
                                tc::mma_ss(ts, dq + off, d + off, id_s, ks > 0);
                            }
                            tc::commit(&s_full[i]);
                            if (j + 2 == ni) tc::commit(&q_empty[i]);
                        };
                        if constexpr (G::kOwnP) {
                            // S of the next step as soon as this one's is in registers: it runs under the softmax
                            if (j + 1 < ni) {
                                ok = j < 0 ? wait(&q_full[i], nq) : wait(&s_read[i], nr);
                                if (!ok) break;
                                if (j < 0) nq ^= 1u;
                                else nr ^= 1u;
                                tc::fence_after_sync();
                                if (leader) issue_s();
                            }
                            // (the item's last S is read too before the next item's first replaces it: by the softmax
                            // threads that wrote the P this waits for)
                            if (j >= 0 && j == ni - 1) nr ^= 1u;
                            if (leader && more_k) tc::commit(&empty[c.slot]);
                        } else {
                            // the tiles take turns, a round's O product and S product at a time: left to themselves
                            // they fall into step, both on the tensor cores, then both in their softmax
                            ok = wait(&turn[i], nturn);
                            nturn ^= 1u;
                            if (!ok) break;
                        }
                        if (j >= 0 && j < ni) {
                            const int left = it.end_of(i) - (it.step0 + j) * kStep;   // (16 a product, none wholly past the end)
                            const uint64_t d = dv + static_cast<uint64_t>(v.slot * (G::kTile >> 4));
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (!G::kOwnP || half == 0) {    // (kOwnP: both halves come at once)
                                    ok = ok && wait(&p_full[2 * i + half], np);
                                    tc::fence_after_sync();
                                }
                                if (ok && leader) {
                                    if (left >= kStep - 15) {
#pragma unroll
                                        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                                            tc::mma_ts(to, tp + kk * 8, d + kk * 128, kIdO, (j > 0 || kk > 0) ? 1u : 0u);
                                    } else {
#pragma unroll 1
                                        for (int kk = 4 * half; kk < 4 * half + 4 && kk * 16 < left; ++kk)
                                            tc::mma_ts(to, tp + kk * 8, d + kk * 128, kIdO, (j > 0 || kk > 0) ? 1u : 0u);
                                    }
                                }
                            }
                            np ^= 1u;
                            if (!ok) break;
                            if (G::kOwnP && leader) tc::commit(&o_step[i]);
                        }
                        if constexpr (G::kOwnP) {
                            if (leader && j >= 0) {
                                if (j == ni - 1) tc::commit(&o_full[i]);
                                tc::commit(&empty[v.slot]);
                            }
                        } else {
                            if (j < 0 && ni > 0) {
                                ok = wait(&q_full[i], nq);
                                nq ^= 1u;
                                if (!ok) break;
                                tc::fence_after_sync();
                            }
                            if (leader) {
                                if (j + 1 < ni) issue_s();
                                mbar_arrive(&turn[1 - i]);
                                if (j >= 0 && j == ni - 1) tc::commit(&o_full[i]);
                                if (j >= 0) tc::commit(&empty[v.slot]);
                                if (more_k) tc::commit(&empty[c.slot]);
                            }
                        }
                        if (more_k) c.next();
                    }
                }
            }
            if (!ok && leader) dec::raise_abort(a.err, abort_flag);
            if (leader) tc::commit(fin);
            wait_bar(fin, 0, abort_flag);
            if (*abort_flag) {                               // (an abort may leave MMAs running: give them a moment)
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
            }
            __syncwarp();
        } else if (warp == G::kLoadQ) {
            // ======================================================== Q tiles, as soon as the last S product read them
            const bool leader = elect_one();
            Item it;
            const int sub_tokens = kSub / a.group;           // (when the group divides a tile)
            unsigned ph = 3u;                                // parities of q_empty (a bit a tile): both tiles start empty
            bool ok = !*abort_flag;
            if (leader && a.q_tma) prefetch_tensormap(&tmq);
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
#pragma unroll 1
                for (int i = 0; i < G::kTiles; ++i) {
                    if (it.steps_of(i) == 0) continue;
                    ok = wait_bar(&q_empty[i], (ph >> i) & 1u, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    ph ^= 1u << i;
                    if (!ok) break;
                    uint8_t* dst = smem + i * G::kTile;
                    if (a.q_tma) {
                        // (rows of the box past the item's are other tokens' queries, or zeros past the last:
                        // their scores go nowhere)
                        const int tok = it.qs + (2 * it.tile + i) * sub_tokens;
                        if (leader) {
                            uint64_t* bar = kConvertQ ? &q_raw[i] : &q_full[i];
                            mbar_arrive_expect_tx(bar, G::kTile);
#pragma unroll
                            for (int hf = 0; hf < G::kHalves; ++hf)
                                tma_load_4d(dst + hf * G::kPlane, &tmq, hf * 64, it.kvh * a.group, tok, 0, bar);
                        }
                    } else {
                        copy_q<T, D>(a, it, i, smem_u32(dst));
                        if (leader) mbar_arrive(kConvertQ ? &q_raw[i] : &q_full[i]);
                    }
                }
            }
            if (!ok && leader) {
                dec::raise_abort(a.err, abort_flag);
                const unsigned long long t0 = globaltimer_ns();
                while (globaltimer_ns() - t0 < 10000000ull) __nanosleep(100000);
            }
        } else if (warp == G::kPlan) {
            // ======================================================== items, decoded a few ahead
            // (the first entry is read beside the count of items, not after it: entries past the count are stale)
            Entry next{};
            int total = 0;
            auto round_entry = [&](int r) {                  // (local plan)
                Entry n;
                n.x = make_int4(__shfl_sync(0xffffffffu, mine.x.x, r), __shfl_sync(0xffffffffu, mine.x.y, r),
                                __shfl_sync(0xffffffffu, mine.x.z, r), __shfl_sync(0xffffffffu, mine.x.w, r));
                n.y = make_int4(__shfl_sync(0xffffffffu, mine.y.x, r), __shfl_sync(0xffffffffu, mine.y.y, r),
                                __shfl_sync(0xffffffffu, mine.y.z, r), __shfl_sync(0xffffffffu, mine.y.w, r));
                n.kvh = __shfl_sync(0xffffffffu, mine.kvh, r);
                n.live = __shfl_sync(0xffffffffu, static_cast<int>(mine.live), r) != 0;
                return n;
            };
            if (a.direct) {
                next = find_entry(a);
            } else if (a.local) {
                next = round_entry(0);
            } else {
                next = fetch_entry(a, a.capacity * a.num_kv_heads, 0);
                total = min(max(__ldcg(a.header), 0), a.capacity) * a.num_kv_heads;
                next.live = static_cast<int>(blockIdx.x) < total;
            }
            bool ok = !*abort_flag, more = true;
            for (int r = 0; ok && more; ++r) {
                const int k = r % G::kItems;
                Item it;
                more = next.live;
                if (more) {
                    read_item<TREE, LONE>(a, next, it);
                    if (!a.local) next = fetch_entry(a, total, r + 1);
                    else if (r < 31) next = round_entry(r + 1);
                    else next.live = false;
                } else {
                    it.rows = -1;
                }
                ok = wait_bar(&item_empty[k], ((r / G::kItems) & 1) ^ 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    list[k] = it;
                    mbar_arrive(&item_full[k]);
                }
                __syncwarp();
            }
            if (!ok && lane == 0) dec::raise_abort(a.err, abort_flag);
        } else if (warp == G::kClean || warp == G::kClean + 2) {
            // ======================================================== V tiles that some row sees only in part
            const int fw = warp != G::kClean;
            [[maybe_unused]] int* mine = bad + fw * 2 * D;
            // the 16-byte pieces of a row, which two warps share: alternating runs of rows, or (TREE) half the columns
            // each, so that a column's node masks are one warp's
            constexpr int kCh = TREE ? D / 16 : D / 8;
            const int ch0 = TREE ? fw * kCh : 0;
            constexpr int kApart = TREE ? 1 : 2;             // runs of rows side by side
            constexpr int kBatch = 4;                        // loads in flight a lane
            constexpr uint32_t kCarry = kBf16 ? 0x00800080u : 0x04000400u;   // exponent all ones -> bit 15
            Ring<ST> c;
            Item it;
            bool ok = !*abort_flag;
            for (int r = 0; ok && get_item(r, it, ok); ++r) {
                const int n = it.steps();
                for (int j = 0; j < n && ok; ++j) {
                    // (these warps pass every slot of the ring in order, so that they clean V as it lands)
                    ok = wait_bar(&full[c.slot], c.phase, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive(&clean[c.slot]);
                        mbar_arrive(&empty[c.slot]);
                    }
                    c.next();
                    const int slot = c.slot;
                    ok = wait_bar(&full[slot], c.phase, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    c.next();
                    int lo, nv, nv16;
                    it.partial(j, lo, nv, nv16);
                    if (lo >= nv16) {
                        if (lane == 0) {
                            mbar_arrive(&clean[slot]);
                            mbar_arrive(&empty[slot]);
                        }
                        continue;
                    }
                    const uint32_t vt = smem_u32(ring + slot * G::kTile);
                    const int tok0 = (it.step0 + j) * kStep;
                    auto addr_of = [&](int i) {
                        const int ch = ch0 + i % kCh;
                        return dec::swz(vt + (ch >> 3) * G::kPlane, i / kCh, ch & 7);
                    };
                    const int end = nv16 * kCh;
#pragma unroll 1
                    for (int i0 = lo * kCh + (TREE ? 0 : fw * 32 * kBatch); i0 < end; i0 += 32 * kApart * kBatch) {       // (warp-uniform)
                        uint32_t hit = 0;                    // bit u: piece u holds a non-finite element
#pragma unroll
                        for (int u = 0; u < kBatch; ++u) {
                            const int i = i0 + 32 * u + lane, row = i / kCh;
                            uint32_t x[4] = {0u, 0u, 0u, 0u}, any = 0;
                            if (row < nv)
                                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                             : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                             : "r"(addr_of(i)));
#pragma unroll
                            for (int e = 0; e < 4; ++e) any |= ((x[e] & 0x7fff7fffu) + kCarry) & 0x80008000u;
                            hit |= any ? 1u << u : 0u;
                        }
                        if (i0 + 32 * kBatch > nv * kCh) {   // slots past the end
                            for (int u = 0; u < kBatch; ++u) {
                                const int i = i0 + 32 * u + lane;
                                if (i / kCh >= nv && i < end)
                                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr_of(i)), "r"(0u) : "memory");
                            }
                        }
                        if (__any_sync(0xffffffffu, hit != 0)) {             // rare
                            if (bad_tag[fw] != r) {          // (warp-uniform: this warp alone writes it)
                                ok = table_free(r);
                                if constexpr (TREE) {
                                    for (int k = lane; k < D; k += 32) bad_nodes[(k / (D / 2)) * D + fw * (D / 2) + k % (D / 2)] = 0ull;
                                } else {
                                    for (int k = lane; k < 2 * D; k += 32) mine[k] = 0x7fffffff;
                                }
                                __syncwarp();
                                if (lane == 0) bad_tag[fw] = r;
                                __syncwarp();
                            }
#pragma unroll 1
                            for (int e = 0; e < 8 * kBatch && hit != 0; ++e) {
                                if (!(hit >> (e >> 3) & 1u)) continue;
                                const int i = i0 + 32 * (e >> 3) + lane;
                                const uint32_t addr = addr_of(i) + 2 * (e & 7);
                                uint16_t h;
                                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
                                const uint32_t mag = h & 0x7fffu, inf = 0x8000u - (kCarry & 0xffffu);
                                if (mag < inf) continue;
                                const int col = 8 * (ch0 + i % kCh) + (e & 7), pos = tok0 + i / kCh;
                                const bool up = mag > inf || h < 0x8000u, down = mag > inf || h >= 0x8000u;
                                if constexpr (TREE) {
                                    const unsigned long long node = 1ull << (pos - it.L + it.n);
                                    if (up) atomicOr(&bad_nodes[col], node);
                                    if (down) atomicOr(&bad_nodes[D + col], node);
                                } else {
                                    if (up) atomicMin(&mine[col], pos);
                                    if (down) atomicMin(&mine[D + col], pos);
                                }
                                asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(uint16_t(0)) : "memory");
                            }
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&clean[slot]);
                        mbar_arrive(&empty[slot]);
                    }
                }
            }
            if (!ok && lane == 0) dec::raise_abort(a.err, abort_flag);
        }
    } else {
        // ============================================================ softmax: one row a thread
        regs_inc<G::kRegsSoftmax>();
        const int wg = warp >> 2;
        const int t = threadIdx.x & 127;
        const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        uint32_t ts = tl + G::kColS + wg * 128, tp = tl + G::kColP + wg * G::kStrideP;
        const uint32_t to = tl + G::kColO + wg * D;
        OT* out = static_cast<OT*>(a.out);
        unsigned ns = 0, no = 0, nraw = 0, nstep = 0;       // (LONE: ns holds a parity bit for each S buffer)
        Item it;
        bool ok = !*abort_flag;
#pragma unroll 1
        for (int r = 0; ok && get_item(r, it, ok); ++r) {
            const int myrow = wg * kSub + t;                 // row of the item
            const bool has = myrow < it.rows;
            const int rr = it.tile * kPrefillRows + myrow, tok = pf::div(rr, a.by_group);
            const int at = has ? (it.qs + tok) * a.num_heads + it.kvh * a.group + (rr - tok * a.group) : -1;   // row of out
            // positions this row sees (rows past the end: all, their weights go nowhere)
            const int lim = has ? max(0, min(it.L, it.L - it.n + tok + 1)) : 0x7fffffff;
            const int n = it.steps_of(wg);
            // the warp has no row of the item: single tokens beside prompts leave most warps without (177 -> 175 us for 60
            // of them beside 4 chunks; at head_dim 64 the code more cost 4%)
            const bool idle = wg * kSub + (warp & 3) * 32 >= it.rows;
            const int seen = min(lim, it.end_of(wg));           // (dummy rows too stop at the tile's end)
            // TREE: the nodes the row sees (dummy rows: all), none after its own nor of a position below 0
            const int past = it.L - it.n;
            unsigned long long nodes = 0ull;
            if constexpr (TREE) {
                if (it.rows > 0) {
                    nodes = ~0ull >> (kTreeNodes - it.n);
                    if (has) nodes &= __ldcg(a.tree_mask + it.qs + tok) & ~0ull >> (kTreeNodes - 1 - tok);
                    if (past < 0) nodes = past > -kTreeNodes ? nodes & ~0ull << -past : 0ull;
                }
            }
            float m_ref = -INFINITY, l = 0.0f;
            float sl2 = a.scale_log2;
            if (KV8) {
                sl2 *= fabsf(__ldcg(a.k_scale + it.kvh));
                if (sl2 == 0.0f) sl2 = 0x1p-149f;            // (a masked score, -inf, stays -inf)
            }
            const uint64_t sl2x2 = pack64(sl2, sl2);
            if constexpr (kConvertQ) {
                if (n > 0) {                                 // the tile's bf16 queries to f16, in place
                    ok = wait_bar(&q_raw[wg], nraw & 1, abort_flag);
                    ok = __all_sync(0xffffffffu, ok);
                    ++nraw;
                    if (!ok) break;
                    const uint32_t tile = smem_u32(smem + wg * G::kTile) + 16 * t;
#pragma unroll 4
                    for (int i = 0; i < G::kTile; i += 16 * kSub) {
                        uint32_t x[4];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                     : "r"(tile + i));
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = Mma<OT>::unpack(x[e]);
                            x[e] = Mma<T>::pack(f.x, f.y);
                        }
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile + i), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                                     "r"(x[3])
                                     : "memory");
                    }
                    fence_proxy_async_smem();
                    mbar_arrive(&q_full[wg]);
                }
            }
            for (int j = 0; j < n; ++j) {
                const int sb = LONE ? j & 1 : wg;            // S's buffer
                if constexpr (LONE) {
                    ts = tp = tl + G::kColS + sb * 128;
                    ok = wait_bar(&s_full[sb], ns >> sb & 1u, abort_flag);
                    ns ^= 1u << sb;
                } else {
                    ok = wait_bar(&s_full[wg], ns & 1, abort_flag);
                    ++ns;
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc::fence_after_sync();
                if constexpr (!G::kOwnP) {
                    if (idle) {                              // (what P holds there reaches rows of no token alone)
                        mbar_arrive(&p_full[2 * sb]);
                        mbar_arrive(&p_full[2 * sb + 1]);
                        if (LONE && j > 0) ++nstep;
                        continue;
                    }
                }
                // Two passes over S, a rolled loop of two halves each, S read from TMEM again for the second: half
                // the code of one pass with S in registers, and the code of the loops is what the schedulers'
                // instruction caches must hold beside the MMA warps'.
                [[maybe_unused]] const int vis = seen - (it.step0 + j) * kStep;
                float top = -INFINITY;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[2][32];
                    tc::ld32(x[0], ts + 64 * h);
                    tc::ld32(x[1], ts + 64 * h + 32);
                    tc::wait_ld();
                    if constexpr (TREE) {
                        const int j0 = (it.step0 + j) * kStep + 64 * h - past;    // the node of the first column
                        if (j0 > -64) {                      // (the same in every thread) masked scores go back as -inf
                            const unsigned long long word = j0 >= kTreeNodes ? 0ull
                                                            : j0 >= 0        ? nodes >> j0
                                                                             : nodes << -j0 | ((1ull << -j0) - 1ull);
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t half = static_cast<uint32_t>(word >> (32 * c));
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(half >> e & 1u)) x[c][e] = 0xff800000u;
                                tc::st32(ts + 64 * h + 32 * c, x[c]);
                            }
                            tc::wait_st();
                        }
                    } else if (__any_sync(0xffffffffu, vis < 64 * h + 64)) {     // masked scores go back as -inf
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (64 * h + 32 * c + e >= vis) x[c][e] = 0xff800000u;
                            tc::st32(ts + 64 * h + 32 * c, x[c]);
                        }
                        tc::wait_st();
                    }
                    float mx[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        mx[c] = max3(__uint_as_float(x[c][0]), __uint_as_float(x[c][1]), __uint_as_float(x[c][2]));
#pragma unroll
                        for (int e = 3; e < 31; e += 2) mx[c] = max3(mx[c], __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
                        mx[c] = fmaxf(mx[c], __uint_as_float(x[c][31]));
                    }
                    top = max3(top, mx[0], mx[1]);
                }
                top *= sl2;
                float alpha = 1.0f;
                if (top > m_ref + 8.0f) {
                    if (m_ref != -INFINITY) alpha = fast_exp2(m_ref - top);
                    m_ref = top;
                }
                if constexpr (G::kOwnP || LONE) {
                    // the last step's O product reads P's columns (kOwnP) and writes O (LONE: only a warp that rescales
                    // O has to wait, but with the wait in such warps alone 64 trees of 26 took 102.3 us instead of 101.1)
                    if (j > 0) {
                        ok = wait_bar(&o_step[wg], nstep & 1, abort_flag);
                        ok = __all_sync(0xffffffffu, ok);
                        ++nstep;
                        if (!ok) break;
                        tc::fence_after_sync();
                    }
                }
                if (__any_sync(0xffffffffu, alpha != 1.0f)) {
                    // (where P takes S's place, S of this step was issued after the last O product: that is done)
                    l *= alpha;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 16) {
                        uint32_t o[16];
                        tc::ld16(o, to + c0);
                        tc::wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tc::st16(to + c0, o);
                    }
                }
                // (a row that has seen nothing keeps ref = -inf: every weight 2^-inf = 0)
                const float off = m_ref == -INFINITY ? -INFINITY : -m_ref;
                const uint64_t offx2 = pack64(off, off);
                uint64_t sum0 = 0, sum1 = 0;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[2][32], w[32];
                    tc::ld32(x[0], ts + 64 * h);
                    tc::ld32(x[1], ts + 64 * h + 32);
                    tc::wait_ld();
                    if constexpr (G::kOwnP) {
                        if (h == 1) {
                            tc::fence_before_sync();
                            mbar_arrive(&s_read[wg]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t* y = &x[e >> 4][2 * (e & 15)];
                        const float2 z = unpack64(fma2(pack64(__uint_as_float(y[0]), __uint_as_float(y[1])), sl2x2, offx2));
                        const float p0 = fast_exp2(z.x), p1 = fast_exp2(z.y);
                        if (e & 1) sum1 = add2(sum1, pack64(p0, p1));
                        else sum0 = add2(sum0, pack64(p0, p1));
                        w[e] = Mma<T>::pack(p0, p1);
                    }
                    tc::st32(tp + 32 * h, w);
                    // (at head_dim 64 one hand-over of the whole step: S of the next runs under the softmax anyway,
                    // and a wait fewer in the MMA warp is worth more than half a product's head start: 92.2 to 90.8 us
                    // over 24 ragged prompts of 5 to 2000 tokens, 12 heads over 4)
                    if (!G::kOwnP || h == 1) {
                        tc::wait_st();
                        tc::fence_before_sync();
                        mbar_arrive(&p_full[2 * sb + (G::kOwnP ? 0 : h)]);
                    }
                }
                const float2 sm = unpack64(add2(sum0, sum1));
                l += sm.x + sm.y;
            }
            if (!ok) break;

            // ---- the output, or a split tile's partial one
            const bool split = it.split != 0;
            const int64_t slot = static_cast<int64_t>(it.kvh) * a.part_cap + (it.split >> 16) + ((it.split >> 8) & 255);
            float4* prow = a.part_o + slot * (D / 4) * a.part_rows + myrow;      // [column / 4][row]
            if (n > 0) {
                if (G::kOwnP || LONE) ++nstep;               // (the last step's, of which this is the completion)
                ok = wait_bar(&o_full[wg], no & 1, abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                ++no;
                if (!ok) break;
                tc::fence_after_sync();
                const float vs = KV8 ? __ldcg(a.v_scale + it.kvh) : 1.0f;
                // (no weight: zeros for a row that sees nothing, NaN where every score it sees is -inf; a NaN sum stays)
                const bool sees = TREE ? past > 0 || nodes != 0ull : lim > 0;
                const float inv = l > 0.0f ? vs / l : l == 0.0f ? (sees ? NAN : 0.0f) : l;
                if (split) {
                    // a row a thread, 16 bytes of 32 neighbouring rows side by side
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc::ld32(o, to + c0);
                        tc::wait_ld();
                        if (has) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                prow[static_cast<int64_t>(c0 / 4 + k) * a.part_rows] =
                                    make_float4(__uint_as_float(o[4 * k]) * vs, __uint_as_float(o[4 * k + 1]) * vs,
                                                __uint_as_float(o[4 * k + 2]) * vs, __uint_as_float(o[4 * k + 3]) * vs);
                        }
                    }
                } else {
                    // The 16x256b shape gives a quad two rows' columns; transposed over the quad, four lanes
                    // write 64 contiguous bytes of a row (a row a thread would touch 32 lines a store, 2 us
                    // an item in the load-store unit).
#pragma unroll 1
                    for (int hh = 0; hh < 2; ++hh) {
                        const int ra = 16 * hh + (lane >> 2);                                 // rows ra and ra + 8 of the warp
                        const float ia = __shfl_sync(0xffffffffu, inv, ra), ib = __shfl_sync(0xffffffffu, inv, ra + 8);
                        const uint64_t ia2 = pack64(ia, ia), ib2 = pack64(ib, ib);
                        const int aa = __shfl_sync(0xffffffffu, at, ra), ab = __shfl_sync(0xffffffffu, at, ra + 8);
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 64) {
                            uint32_t o[32];
                            tc::ld16x256_x8(o, to + (static_cast<uint32_t>(16 * hh) << 16) + c0);
                            tc::wait_ld();
#pragma unroll
                            for (int g = 0; g < 8; g += 4) {
                                uint32_t wa[4], wb[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t* y = &o[4 * (g + e)];
                                    const float2 fa = unpack64(mul2(pack64(__uint_as_float(y[0]), __uint_as_float(y[1])), ia2));
                                    const float2 fb = unpack64(mul2(pack64(__uint_as_float(y[2]), __uint_as_float(y[3])), ib2));
                                    wa[e] = Mma<OT>::pack(fa.x, fa.y);
                                    wb[e] = Mma<OT>::pack(fb.x, fb.y);
                                }
                                quad_transpose(wa);
                                quad_transpose(wb);
                                const int col = c0 + 8 * (g + (lane & 3));
                                if (aa >= 0)
                                    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(aa) * D + col) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
                                if (ab >= 0)
                                    *reinterpret_cast<uint4*>(out + static_cast<int64_t>(ab) * D + col) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
                            }
                        }
                    }
                }
                // rare: V elements that were cleaned away are added to what the products gave, which may hold an
                // infinity or NaN of its own from a position that every row sees
                const bool bad0 = __any_sync(0xffffffffu, bad_tag[0] == r), bad1 = __any_sync(0xffffffffu, bad_tag[1] == r),
                           bad2 = KV8 && __any_sync(0xffffffffu, bad_tag[2] == r);
                [[maybe_unused]] unsigned bads = 0;          // the warps that list some (TREE over E4M3 pools)
                if constexpr (TREE && KV8) bads = __ballot_sync(0xffffffffu, lane < G::kTags && bad_tag[min(lane, G::kTags - 1)] == r);
                if (bads || bad0 || bad1 || bad2) {
                    __syncwarp();
#pragma unroll 1
                    for (int c = 0; c < D; ++c) {
                        bool up, down;
                        if constexpr (TREE) {
                            if constexpr (KV8) {
                                unsigned long long listed = 0ull;
                                for (unsigned m = bads; m; m &= m - 1) listed |= bad_nodes[(__ffs(m) - 1) * D + c];
                                up = down = (listed & nodes) != 0ull;
                            } else {
                                const bool listed = c < D / 2 ? bad0 : bad1;
                                up = listed && (bad_nodes[c] & nodes);
                                down = listed && (bad_nodes[D + c] & nodes);
                            }
                        } else if (KV8) {
                            up = (bad0 && bad[c] < seen) || (bad1 && bad[D + c] < seen) || (bad2 && bad[2 * D + c] < seen);
                            down = up;
                        } else {
                            up = (bad0 && bad[c] < seen) || (bad1 && bad[2 * D + c] < seen);
                            down = (bad0 && bad[D + c] < seen) || (bad1 && bad[3 * D + c] < seen);
                        }
                        const bool add = has && (up || down);
                        if (__any_sync(0xffffffffu, add)) {
                            const uint32_t o = tc::ld1(to + c);
                            tc::wait_ld();
                            const float x = (up ? INFINITY : 0.0f) + (down ? -INFINITY : 0.0f);
                            if (add) {
                                if (split) reinterpret_cast<float*>(prow + static_cast<int64_t>(c / 4) * a.part_rows)[c & 3] += x;
                                else out[static_cast<int64_t>(at) * D + c] = from_float<OT>(__uint_as_float(o) * inv + x);
                            }
                        }
                    }
                    __threadfence_block();                   // (the table is read)
                }
                tc::fence_before_sync();
            } else if (has && !split) {                      // rows that see nothing
                uint4* o = reinterpret_cast<uint4*>(out + static_cast<int64_t>(at) * D);
#pragma unroll
                for (int k = 0; k < D / 8; ++k) o[k] = make_uint4(0u, 0u, 0u, 0u);
            }
            // (a part whose every score the row sees is -inf: its sum is -1, told from a part it sees nothing of; its weight
            // in the merge is 2^(-inf - m), 0 beside a part with a finite score and NaN without one)
            if (split && has) {
                bool some = seen > it.step0 * kStep;
                if constexpr (TREE) {
                    const int from = it.step0 * kStep - past, to = it.end_of(wg) - past;     // the part's nodes
                    some = from < 0 && n > 0;
                    if (from < kTreeNodes && to > 0)
                        some |= ((nodes & ~0ull >> (kTreeNodes - min(to, kTreeNodes))) >> max(from, 0)) != 0ull;
                }
                a.part_ml[slot * a.part_rows + myrow] = make_float2(m_ref, l == 0.0f && some ? -1.0f : l);
            }
            __syncwarp();
            if (lane == 0) atomicAdd(const_cast<int*>(epilogues) + warp, 1);
        }
        if (!ok && lane == 0) dec::raise_abort(a.err, abort_flag);
    }
    tc::fence_before_sync();
    __syncthreads();                                // every role is through: TMEM is no longer used
    launch_dependents();
    if (warp == G::kMma) {
        tc::fence_after_sync();
        tc::tmem_dealloc(tmem, G::kTmemCols);
    }
}

// Whether no tree of the call has more than a tile of rows of a KV head, so that every item is a single one: the same in
// every CTA.  The query starts alone decide: padding rows behind the last tree and sequences without nodes count for
// nothing, and a replayed graph goes by its own trees.  Looking takes 1 us.
__device__ __forceinline__ bool lone_trees(const PrefillArgs& a) {
    if (a.lone_nodes >= kTreeNodes) return true;
    grid_dependency_wait();
    bool more = false;
    for (int s = threadIdx.x; s < a.num_seqs; s += blockDim.x)
        more |= static_cast<long long>(__ldcg(a.query_starts + s + 1)) - __ldcg(a.query_starts + s) > a.lone_nodes;
    return !__syncthreads_or(more);
}

// Trees over E4M3 pools: both forms, the one the host expects (LONE_FIRST) first.  The second in the code runs 2 to 5%
// slower: 64 trees of 26, 32 heads over 8, 101.1 us as the first and 103.3 as the second, of 33 144.3 and 146.7, 128 trees of 1
// to 64, 64 heads over 8, 194.1 and 202.6.  (In kernels of their own 101.0, 143.0 and 192.7; one after the other, the one
// that does not apply ending at once, 3 us more a call.)
template <typename T, int D, bool KV8, typename OT, bool TREE, bool LONE_FIRST>
__global__ void __launch_bounds__(PfGeo<D, KV8, TREE>::kThreads, 1) prefill_kernel(const __grid_constant__ CUtensorMap tmq,
                                                                        const __grid_constant__ CUtensorMap tmk,
                                                                        const __grid_constant__ CUtensorMap tmv,
                                                                        const __grid_constant__ PrefillArgs a) {
    if constexpr (TREE && KV8) {
        if (lone_trees(a) == LONE_FIRST) {
            prefill_cta<T, D, KV8, OT, TREE, LONE_FIRST>(tmq, tmk, tmv, a);
            return;
        }
    }
    prefill_cta<T, D, KV8, OT, TREE, TREE && KV8 && !LONE_FIRST>(tmq, tmk, tmv, a);
}

// The split tiles' parts merged: 32 rows by 64 columns a CTA, a row a lane, its columns over the warps.
//     m = max_p m_p,  out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p
// summed in part order.  Launched for every call whose plan may split, since the host does not know whether it did
// (without a split tile its CTAs end at once).  A kernel of its own, since the merge of a 256-row tile is a megabyte of reads:
// by the last CTA to finish it took 70 us of a 177 us call (33 tokens x 64 heads over 65549 positions).
// Bound by latency: the next call waits for the last of these CTAs.  So the parts' weights are found first, a part a
// warp, and kept in shared memory; then every load of the partial outputs is independent of the others, 16 in flight
// a lane.
constexpr int kMergeThreads = 256, kMergeRows = 32, kMergeCols = 64;
template <typename T, int D>
__global__ void __launch_bounds__(kMergeThreads) prefill_merge_kernel(const PrefillArgs a) {
    constexpr int kWarps = kMergeThreads / 32;
    constexpr int kQuads = kMergeCols / 4 / kWarps;           // 4-column pieces a thread merges
    __shared__ uint2 tile[kMergeRows][kMergeCols / 4 + 1];
    __shared__ int rows_at[kMergeRows];
    __shared__ float2 weight[kPrefillMaxParts][kMergeRows];   // (reference, sum), then (2^(m_p - m), times the sum); below 0: nothing seen
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    grid_dependency_wait();
    launch_dependents();
    const int groups = a.part_rows / kMergeRows, pieces = groups * (D / kMergeCols);
    const long long units = static_cast<long long>(min(__ldcg(a.header + 1), a.part_cap / 2)) * a.num_kv_heads * pieces;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int piece = static_cast<int>(u % pieces), g = piece / (D / kMergeCols), cols = piece % (D / kMergeCols);
        const int kvh = static_cast<int>((u / pieces) % a.num_kv_heads);
        const int4 e = __ldcg(a.merges + u / pieces / a.num_kv_heads);
        const int nparts = e.x & 255, base = e.x >> 16;
        Item it;
        it.tile = e.y;
        it.qs = e.z;
        it.n = e.w;
        it.kvh = kvh;
        if (nparts < 1 || nparts > kPrefillMaxParts || base < 0 || base + nparts > a.part_cap || it.tile < 0 || it.qs < 0 ||
            it.n <= 0 || it.qs + static_cast<long long>(it.n) > a.num_tokens) {
            if (threadIdx.x == 0) raise_error(a.err, kErrBounds);
            continue;
        }
        const long long left = static_cast<long long>(it.n) * a.group - static_cast<long long>(it.tile) * kPrefillRows - g * kMergeRows;
        if (left <= 0) continue;
        const bool has = lane < left;
        const int row = g * kMergeRows + lane;
        const int64_t slot = static_cast<int64_t>(kvh) * a.part_cap + base;
        const float2* ml = a.part_ml + slot * a.part_rows + row;
        const float4* po = a.part_o + (slot * (D / 4) + cols * (kMergeCols / 4) + warp) * a.part_rows + row;
#pragma unroll 4
        for (int p = warp; p < nparts; p += kWarps)
            weight[p][lane] = has ? __ldcg(ml + static_cast<int64_t>(p) * a.part_rows) : make_float2(-INFINITY, 0.0f);
        if (warp == 0) rows_at[lane] = has ? static_cast<int>(qo_row(a, it, row)) : -1;
        __syncthreads();
        float m = -INFINITY;
#pragma unroll 8
        for (int p = 0; p < nparts; ++p) m = fmaxf(m, weight[p][lane].x);
        __syncthreads();
        for (int p = warp; p < nparts; p += kWarps) {
            const float2 x = weight[p][lane];
            // (a part the row sees nothing of: its O was not written)
            const float w = x.x == -INFINITY && x.y == 0.0f ? -1.0f : fast_exp2(x.x - m);
            weight[p][lane] = make_float2(w, w < 0.0f ? 0.0f : w * x.y);
        }
        __syncthreads();
        float den = 0.0f;
        float4 acc[kQuads];
#pragma unroll
        for (int k = 0; k < kQuads; ++k) acc[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
        for (int p = 0; p < nparts; ++p) {
            const float2 x = weight[p][lane];
            const bool none = x.x < 0.0f;
            den += x.y;
#pragma unroll
            for (int k = 0; k < kQuads; ++k) {
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (!none) v = __ldcg(po + (static_cast<int64_t>(p) * (D / 4) + k * kWarps) * a.part_rows);
                const float w = none ? 0.0f : x.x;
                acc[k].x += w * v.x;
                acc[k].y += w * v.y;
                acc[k].z += w * v.z;
                acc[k].w += w * v.w;
            }
        }
        const float inv = den > 0.0f ? 1.0f / den : den == 0.0f ? 0.0f : den;
#pragma unroll
        for (int k = 0; k < kQuads; ++k)
            tile[lane][warp + k * kWarps] =
                make_uint2(Mma<T>::pack(acc[k].x * inv, acc[k].y * inv), Mma<T>::pack(acc[k].z * inv, acc[k].w * inv));
        __syncthreads();
        for (int i = threadIdx.x; i < kMergeRows * (kMergeCols / 4); i += kMergeThreads) {
            const int r = i / (kMergeCols / 4), c = i % (kMergeCols / 4);
            if (rows_at[r] >= 0)
                reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(rows_at[r]) * D + cols * kMergeCols)[c] = tile[r][c];
        }
        __syncthreads();
    }
}

template <typename T, int D, bool KV8, typename OT, bool TREE, bool LONE_FIRST = false>
cudaError_t launch_t(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                     cudaStream_t s) {
    using G = PfGeo<D, KV8, TREE>;
    using GL = PfGeo<D, KV8, TREE, TREE && KV8>;            // (its other form's)
    constexpr size_t kShared = std::max(G::kBytes, GL::kBytes);
    static_assert(G::kRing % 1024 == 0 && GL::kRing % 1024 == 0 && G::kTile % 1024 == 0, "tiles start on a swizzle atom");
    static_assert(G::kRegsSoftmax == GL::kRegsSoftmax && G::kRegsOther == GL::kRegsOther, "one register split");
    auto kern = prefill_kernel<T, D, KV8, OT, TREE, LONE_FIRST>;
    // once a device: the shared memory, and that the warpgroups' register split fits what a block is launched with
    // (or it would wait for ever)
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1u)) {
        cudaFuncAttributes fa{};
        if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
        if (fa.numRegs * G::kThreads < 256 * G::kRegsSoftmax + 256 * G::kRegsOther) return cudaErrorLaunchOutOfResources;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kShared));
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(
        std::min<int64_t>(a.slots, static_cast<int64_t>(a.direct ? a.capacity - a.part_cap : a.capacity) * a.num_kv_heads)));
    cfg.blockDim = dim3(G::kThreads);
    cfg.dynamicSmemBytes = kShared;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, tmq, tmk, tmv, a);
    if (e != cudaSuccess || !a.may_split) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * a.slots));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, prefill_merge_kernel<OT, D>, a);
}

template <bool TREE>
cudaError_t launch(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv, int dtype,
                   int head_dim, cudaStream_t s) {
    using bf16 = __nv_bfloat16;
    if constexpr (TREE) {
        // (trees that fill a tile on average or less are expected to be one each)
        if (a.k_scale && a.num_tokens * a.group <= int64_t(kPrefillSub) * a.num_seqs)
            return dtype == 0 ? launch_t<__half, 128, true, __half, true, true>(a, tmq, tmk, tmv, s)
                              : launch_t<__half, 128, true, bf16, true, true>(a, tmq, tmk, tmv, s);
    }
    if (a.k_scale)
        return dtype == 0 ? launch_t<__half, 128, true, __half, TREE>(a, tmq, tmk, tmv, s)
                          : launch_t<__half, 128, true, bf16, TREE>(a, tmq, tmk, tmv, s);
    if (dtype == 0)
        return head_dim == 128 ? launch_t<__half, 128, false, __half, TREE>(a, tmq, tmk, tmv, s)
                               : launch_t<__half, 64, false, __half, TREE>(a, tmq, tmk, tmv, s);
    return head_dim == 128 ? launch_t<bf16, 128, false, bf16, TREE>(a, tmq, tmk, tmv, s)
                           : launch_t<bf16, 64, false, bf16, TREE>(a, tmq, tmk, tmv, s);
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                           int dtype, int head_dim, cudaStream_t s) {
    return a.tree_mask ? launch<true>(a, tmq, tmk, tmv, dtype, head_dim, s) : launch<false>(a, tmq, tmk, tmv, dtype, head_dim, s);
}

}  // namespace pkv
