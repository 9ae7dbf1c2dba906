// Launchers shared between the C-ABI translation unit and the kernel units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pkv {

constexpr int kMaxCopyLayers = 64;   // layer pointers carried per copy_blocks launch

struct AppendArgs {
    const uint4* k;          // [T][row_vecs]
    const uint4* v;
    uint4* key_cache;        // [num_blocks * block_size][row_vecs]
    uint4* value_cache;
    const int64_t* slots;
    int64_t num_tokens;
    int64_t num_slots;       // num_blocks * block_size
    int row_vecs;            // num_kv_heads * head_dim * 2 / 16
    unsigned* err;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);

// Append into an E4M3 pool: each element is quantized as
// e4m3(float32(x) / float32(scale[head])), round to nearest even, saturating.
struct AppendFp8Args {
    const uint4* k;          // [T][row_vecs] 8 fp16 / bf16 elements per vector
    const uint4* v;
    uint2* key_cache;        // [num_blocks * block_size][row_vecs] 8 codes per vector
    uint2* value_cache;
    const int64_t* slots;
    const float* k_scale;    // [num_kv_heads]
    const float* v_scale;
    int64_t num_tokens;
    int64_t num_slots;
    int row_vecs;            // num_kv_heads * head_dim / 8
    int head_vecs;           // head_dim / 8
    int bf16;                // input elements: 0 = fp16, 1 = bf16
    unsigned* err;
};
cudaError_t launch_append_fp8(const AppendFp8Args& a, cudaStream_t s);

// Append with the position rotation (csrc/pkv_append_rotary.cu).
struct AppendRotaryArgs {
    void* q_out;             // rows of [num_heads][head_dim], a stride of elements apart
    const void* q;
    const void* k;           // rows of [num_kv_heads][head_dim]
    const void* v;
    void* key_cache;         // [num_blocks * block_size][num_kv_heads][head_dim] (16-bit elements, or codes)
    void* value_cache;
    const int64_t* slots;    // [num_tokens]
    const int32_t* positions;
    const float* cos_sin;    // [num_positions][rotary_dim]: cosines, then sines
    const float* k_scale;    // [num_kv_heads] (E4M3 pools only)
    const float* v_scale;
    int64_t num_tokens;
    int64_t num_slots;
    int64_t q_out_stride, q_stride, k_stride, v_stride;
    int num_positions;
    int num_heads;           // (0: no queries)
    int num_kv_heads;
    int head_dim;
    int rotary_dim;
    int interleaved;
    unsigned* err;
};
cudaError_t launch_append_rotary(const AppendRotaryArgs& a, bool bf16, bool kv8, cudaStream_t s);

// Block copies between two pools of the same block shape (the same pool for
// copy-on-write, a device pool and a pinned host pool for swapping).
struct CopyArgs {
    const uint4* src_key[kMaxCopyLayers];
    const uint4* src_value[kMaxCopyLayers];
    uint4* dst_key[kMaxCopyLayers];
    uint4* dst_value[kMaxCopyLayers];
    const int64_t* pairs;    // [num_pairs][2] (source block, destination block)
    int64_t num_pairs;
    int64_t src_num_blocks;
    int64_t dst_num_blocks;
    int num_layers;
    int block_vecs;          // block_size * num_kv_heads * head_dim * 2 / 16
    unsigned* err;
};
cudaError_t launch_copy_blocks(const CopyArgs& a, cudaStream_t s);

struct DecodeArgs {
    void* out;                       // [B][nq][Hq][D]
    const void* q;                   // [B][nq][Hq][D]
    const int32_t* block_tables;     // [B][max_blocks_per_seq]
    const int32_t* seq_lens;         // [B]
    int4* plan;                      // [plan_capacity][2] work list, written per call by the plan kernel
                                     // (nullptr: direct grid): (first sequence, partition, stream length,
                                     // partition tokens), then (unit members, shared prefix length, lengths of
                                     // the unit's first two sequences)
    unsigned* tickets;               // [B][num_kv_heads * head_groups] finished partitions (zeroed per call)
    float* ws_o;                     // [B][Hq*nq][max_parts][D] unnormalised partial outputs
    float2* ws_ml;                   // [B][Hq*nq][max_parts] (running max in log2 units, sum)
    unsigned* err;
    int64_t num_blocks;
    int max_blocks_per_seq;
    int num_seqs;
    int max_seq_len;
    int num_heads;
    int num_kv_heads;
    int group;                       // query rows per KV head: (num_heads / num_kv_heads) * num_queries
    int qgroup;                      // query heads per KV head: num_heads / num_kv_heads
    int num_queries;                 // query tokens per sequence (1 = decode; > 1 = verify, causal)
    int head_groups;                 // ceil(group / 8): groups of query rows per KV head
    int block_size;
    int part_tokens;                 // tokens per partition (multiple of 64); with a plan, the smallest the
                                     // plan kernel may use
    int part_auto;                   // with a plan: 1 = the plan kernel picks the partition size (>= part_tokens)
    int slots;                       // SMs x resident decode CTAs per SM (for the plan kernel's choice)
    int rule_weight;                 // the automatic partition rule's weight (twentieths; plan_rule_tokens)
    int max_parts;                   // partials per query row: ceil(max_seq_len / part_tokens), plus one when
                                     // shared-prefix units are possible (the partials' stride)
    int direct_parts;                // ceil(max_seq_len / part_tokens): the direct grid's partition extent
    int plan_capacity;               // entries of `plan` the grid covers (<= num_seqs * max_parts)
    int64_t sum_seq_lens;            // the caller's sum of seq_lens (0: not given); the plan checks it
    int units;                       // 1: the plan may serve adjacent sequences that share leading blocks
                                     // (forks of one prompt) as one unit (16-bit decode, <= 4 query heads
                                     // per KV head: the members' heads fill one CTA's 8 columns)
    float scale_log2;                // scale * log2(e)
    int kv8;                         // 1: the pools hold E4M3 codes (head_dim 128), scaled per KV head
    const float* k_scale;            // [num_kv_heads] (E4M3 pools only)
    const float* v_scale;
    // Fused slot write (decode only; nullptr k_new: none).  Before attending,
    // the CTA whose partition holds position seq_len - 1 of sequence s writes
    // that sequence's new token (k_new / v_new row s, quantized for an E4M3
    // pool) into slot_mapping[s], which must be that position's slot.
    const uint4* k_new = nullptr;    // [B][num_kv_heads][D] in the query dtype
    const uint4* v_new = nullptr;
    const int64_t* slot_mapping = nullptr;   // [B]
    void* key_cache = nullptr;       // the pools written by the fused slot write
    void* value_cache = nullptr;
    // 1: nothing still running before this launch writes the pools, block tables,
    // lengths or plan (the caller's PKV_INPUTS_READY): a CTA reads its work item,
    // stages its table and starts its first tile loads before waiting for the
    // preceding kernel, then waits before it reads q, the new rows or the slots
    // (and never loads early the chunk that receives the new token)
    int early = 0;
};

// Sequences a call plans (sorts and compacts) at most; larger batches run the
// direct grid (one CTA per (KV head group, partition, sequence)).
constexpr int kPlanMaxSeqs = 1024;

// Shared-prefix units.  Adjacent sequences whose block tables agree on a
// leading run of blocks (forks of one prompt, copy-on-write after the fork)
// hold the same K/V there.  The plan serves up to 8 / (query heads per KV
// head) of them as one unit: the unit's stream is the shared prefix once,
// then each member's own blocks from the end of the prefix, block-aligned;
// a member's query heads attend to the prefix and to its own segment only.
// A unit shares at least this many positions (shorter runs stay separate).
constexpr int kUnitMinShare = 256;
// Work-list entries are two int4 each.
constexpr int kPlanEntryInts = 2;

// Block-table entries a decode CTA stages (a partition spans at most this many blocks).
constexpr int kPlanTableEntries = 512;
// Automatic partition sizes are multiples of this many positions.
constexpr int kPlanGranule = 512;

// The plan kernel's automatic partition size from the lengths' sum alone:
// about w / 20 of the positions per resident CTA slot (sum * nh / slots),
// rounded to the nearest multiple of kPlanGranule, at least one granule.  The
// weight w (twentieths) is the kernel's: kRuleDecode for the 16-bit decode
// kernel (0.85), kRuleDecode8 for E4M3 pools (an E4M3 position is half the
// bytes of a 16-bit one, with the same arithmetic and per-CTA costs; measured
// best on the 8B-shaped batch: 3072 positions against 4096 at twice), and
// kRuleVerifyTc for the tensor-core verify kernel, whose items carry a longer
// start-up and epilogue.  The host uses the same rule to bound the work list
// the grid must cover.
constexpr int kRuleDecode = 17;
constexpr int kRuleDecode8 = 24;
constexpr int kRuleVerifyTc = 22;
__host__ __device__ inline long long plan_rule_tokens(long long sum_lens, long long nh, int weight, long long slots) {
    const long long target = (sum_lens * nh * weight) / (slots * 20);
    const long long p = ((target + kPlanGranule / 2) / kPlanGranule) * kPlanGranule;
    return p > kPlanGranule ? p : kPlanGranule;
}

// Query rows (mma columns) one decode CTA serves.
constexpr int dec_heads_per_cta() { return 8; }

// Workspace layout of one decode call:
//   [tickets | work list | partial outputs | (max, sum) pairs]
// each region 256-byte aligned.  Every call re-initialises what it uses.
struct DecodeWorkspace {
    size_t ticket_bytes;   // tickets, padded
    size_t plan_bytes;     // work list (16 bytes per entry), padded
    size_t o_bytes;        // partial outputs, padded (0 when max_parts == 1)
    size_t ml_bytes;       // (max, sum) pairs (0 when max_parts == 1)
    size_t total() const { return ticket_bytes + plan_bytes + o_bytes + ml_bytes; }
};
DecodeWorkspace decode_workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_parts);

// What one decode call launches: the plan kernel then the decode kernel; the
// plan alone; or the decode kernel alone over the plan already in the
// workspace (the merging CTA zeroes its ticket, so a plan serves any number
// of runs).
enum class DecodeMode { kPlanAndRun, kPlanOnly, kRunOnly };

// dtype: 0 = f16, 1 = bf16.  Runs one decode call on stream `s`: the plan
// kernel (work list + tickets) or, for a batch above kPlanMaxSeqs, a ticket
// memset; then the decode kernel, which merges split partitions in-kernel.
cudaError_t launch_decode(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int dtype,
                          int head_dim, cudaStream_t s, DecodeMode mode = DecodeMode::kPlanAndRun);
cudaError_t launch_decode_plan(const DecodeArgs& a, cudaStream_t s);

// More than kVerifyMinRows query rows per KV head (num_queries > 1, 16-bit pools):
// the verify kernel on the tensor cores; fewer, and E4M3 pools: the decode
// kernel's multi-query form, 8 rows per CTA.
constexpr int kVerifyMinRows = 16;

// The verify kernel on the fifth-generation tensor cores (tcgen05): up to
// kVerifyTcRows query rows per CTA (head_groups = ceil(rows / kVerifyTcRows));
// a KV head with at most 64 rows runs the M = 64 form.
constexpr int kVerifyTcRows = 128;
int verify_tc_rows_per_cta(int rows);
cudaError_t launch_verify_tc(const DecodeArgs& a, const CUtensorMap& tmk, const CUtensorMap& tmv, int dtype,
                             int head_dim, cudaStream_t s, DecodeMode mode = DecodeMode::kPlanAndRun);
int verify_tc_ctas_per_sm(int head_dim);

// CTAs of the decode kernel resident per SM on the current device (current
// configuration; kv8: the E4M3-pool kernel), or 0 if it cannot be queried.
int decode_ctas_per_sm(int head_dim, bool kv8 = false);

// ---------------------------------------------------------------- prefill (csrc/pkv_prefill.cu, pkv_prefill_plan.cu)
// A work item is kPrefillRows query rows of one KV head of one sequence over a run of
// kPrefillStep-position steps.  Row r of sequence s, KV head g is token r / group, query
// head g * group + r % group.
constexpr int kPrefillRows = 256;
constexpr int kPrefillSub = 128;                // rows of one of an item's two tiles (the MMA's M)
constexpr int kPrefillStep = 128;
constexpr int kTreeNodes = 64;                  // nodes of a drafted tree at most (a row's mask is one 64-bit word)
constexpr int kPrefillMaxParts = 152;           // parts one tile's positions are split into at most
constexpr int kPrefillMinPart = 2;              // steps of a part at least
// No tile is split in a batch of sequences of up to so many steps: what the parts save the planning and the merge cost.
// Tiles of 4 to 16 rows, one to four sequences: 6 steps 13.3 us whole, 13.7 to 17.6 split; 8 steps 15.8 and 14.0 to 16.8;
// 10 steps 18.4 and 14.2 to 17.6.
constexpr int kPrefillNoSplit = 8;
// The prefill kernel plans by itself up to this many sequences and tiles a KV head, and items (parts and all)
constexpr int kPrefillLocal = 512;
constexpr int kPrefillLocalItems = 1024;

// Division by a number the host knows: q = (hi(mul * n) + n) >> shift, exact for 0 <= n < 2^31 (Granlund and
// Montgomery's round-up method).
struct FastDiv {
    uint32_t mul;
    int shift;
};
inline FastDiv fast_div(int d) {
    int s = 0;
    while ((int64_t(1) << s) < d) ++s;
    return {static_cast<uint32_t>((((uint64_t(1) << s) - static_cast<uint64_t>(d)) << 32) / static_cast<uint64_t>(d) + 1), s};
}

struct PrefillArgs {
    void* out;                       // [num_tokens][num_heads][D]
    const void* q;
    const int32_t* block_tables;     // [B][max_blocks_per_seq]
    const int32_t* seq_lens;         // [B]
    const int32_t* query_starts;     // [B + 1]
    int* header;                     // [0] work items, [1] split tiles
    int4* items;                     // [capacity][2]: (sequence, tile, first step, end step),
                                     // (first query row of q, tokens, length, split: 0, or see prefill_split)
    int4* merges;                    // [part_cap / 2] split tiles: (split of part 0, tile, first query row, tokens)
    float2* part_ml;                 // [num_kv_heads][part_cap][part_rows] (reference maximum in log2 units, sum)
    float4* part_o;                  // [num_kv_heads][part_cap][D / 4][part_rows] unnormalised partial outputs
    unsigned* err;
    int64_t num_blocks;
    int64_t num_tokens;
    int max_blocks_per_seq;
    int num_seqs;
    int max_seq_len;
    int num_heads;
    int num_kv_heads;
    int group;                       // num_heads / num_kv_heads
    FastDiv by_group, by_kv_heads;
    int block_size;
    int block_shift;                 // log2(block_size)
    int capacity;                    // entries of `items`
    int part_cap;                    // partial slots per KV head
    int part_rows;                   // rows of a partial slot: min(256, num_tokens * group), a multiple of 32
    int slots;                       // CTAs the grid may hold at once
    int may_split;                   // 0: the plan splits no tile (no merge kernel follows)
    int direct;                      // 1: no plan: a CTA finds its item by itself (at most one each)
    int local;                       // 1: every CTA plans for itself (the same plan as the plan kernel's)
    int q_tma;                       // 1: a Q tile is one TMA box a column plane (the group divides 128)
    int negate_q;                    // scale < 0
    float scale_log2;                // |scale| * log2(e)
    const float* k_scale;            // [num_kv_heads] (E4M3 pools only, else nullptr)
    const float* v_scale;
    int lone_nodes;                  // the one-tile form takes trees of up to so many nodes (E4M3 pools; tree_lone_nodes)
    const unsigned long long* tree_mask;     // [num_tokens]: bit j, the token sees node j of its tree (nullptr: causal)
};

// A split tile's part: number of parts, this part, first partial slot.
__host__ __device__ inline int prefill_split(int nparts, int part, int base) { return base << 16 | part << 8 | nparts; }

// Workspace: [header | items | split tiles | (max, sum) pairs | partial outputs], each 256-byte aligned.
struct PrefillWorkspace {
    size_t items, merges, ml, o, total;            // offsets and size
    int capacity, part_cap, part_rows;
};
PrefillWorkspace prefill_workspace_layout(int num_seqs, int64_t num_tokens, int num_heads, int num_kv_heads,
                                          int head_dim, int slots);
// Whether the plan may split a tile of such a batch: long enough sequences, and not so many tiles that
// every SM has several anyway.
bool prefill_may_split(int64_t num_tokens, int max_seq_len, int num_heads, int num_kv_heads, int slots);
// A call so small that every item has a CTA of its own and none is split: no plan is made or read.
bool prefill_direct(int num_seqs, int64_t num_tokens, int max_seq_len, int num_heads, int num_kv_heads, int slots);
// A batch small enough for every CTA to plan it by itself, in its own shared memory, instead of a plan kernel.
bool prefill_local(int num_seqs, int64_t num_tokens, int num_heads, int num_kv_heads, int slots,
                   const PrefillWorkspace& w);
// Trees over an E4M3 pool take the form for tiles of 128 rows of a KV head where none has more, that is none more than so
// many nodes (from kTreeNodes on: none can, and the kernel does not look): 109 us against the two-tile form's 124 over 64
// sequences of 512 to 4096 positions with trees of 26 or of 20 to 32 nodes, 32 heads over 8.  A larger tree tile by tile
// would stream its sequence twice: that took 211 us against 154 with trees of 33, 211 against 155 with trees of 10 and 54 in
// turn, 343 against 275 over 128 trees of 1 to 24, 64 heads over 8, and 139 against 129 for two trees of 40 among 62 of 26.
inline int tree_lone_nodes(int64_t num_tokens, int group) {
    const int64_t most = num_tokens < kTreeNodes ? num_tokens : kTreeNodes;
    return most * group <= kPrefillSub ? kTreeNodes : kPrefillSub / group;
}
cudaError_t launch_prefill_plan(const PrefillArgs& a, cudaStream_t s);
cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& tmq, const CUtensorMap& tmk, const CUtensorMap& tmv,
                           int dtype, int head_dim, cudaStream_t s);

// ---------------------------------------------------------------- cache read-back (csrc/pkv_gather.cu)
struct GatherArgs {
    uint4* k_out;            // [num_rows][row_vecs] 8 elements a vector
    uint4* v_out;
    const void* key_cache;   // [num_blocks * block_size][row_vecs] (16-bit elements, or 8 codes a vector)
    const void* value_cache;
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* row_starts;       // [num_seqs + 1]
    const float* k_scale;    // [num_kv_heads] (E4M3 pools only, else nullptr)
    const float* v_scale;
    int64_t num_rows;
    int64_t num_blocks;
    int num_seqs;
    int max_blocks_per_seq;
    int block_size;
    int row_vecs;            // num_kv_heads * head_dim / 8
    int head_vecs;           // head_dim / 8
    int cta_rows;            // output rows a CTA (set by the launch)
    int bf16;                // the outputs' type over an E4M3 pool: 0 = fp16, 1 = bf16
    unsigned* err;
};
cudaError_t launch_gather(const GatherArgs& a, cudaStream_t s);

// ---------------------------------------------------------------- draft acceptance (csrc/pkv_accept.cu)
struct AcceptArgs {
    int64_t* tokens;                 // [num_seqs][max_drafts + 1]
    int32_t* num_accepted;           // [num_seqs]
    const int64_t* draft_tokens;     // [num_seqs][max_drafts]
    const int32_t* num_drafts;       // [num_seqs], or nullptr: max_drafts each
    const void* target_probs;        // [num_seqs][max_drafts + 1][vocab]
    const void* draft_probs;         // [num_seqs][max_drafts][vocab], or nullptr
    const float* uniform;            // [num_seqs][max_drafts + 1]
    int64_t vocab;
    int num_seqs;
    int max_drafts;
    unsigned* err;
};
cudaError_t launch_accept(const AcceptArgs& a, int dtype, cudaStream_t s);   // dtype 0: fp16, 1: bf16, 2: fp32

// ---------------------------------------------------------------- a drafted tree (csrc/pkv_accept_tree.cu, pkv_keep_path.cu)
struct AcceptTreeArgs {
    int64_t* tokens;                 // [num_seqs][width]
    int32_t* path;                   // [num_seqs][width]
    int32_t* num_accepted;           // [num_seqs]
    const int64_t* draft_tokens;     // [num_tokens]
    const int32_t* parents;          // [num_tokens]
    const int32_t* query_starts;     // [num_seqs + 1]
    const void* target_probs;        // [num_tokens][vocab]
    const float* uniform;            // [num_tokens]
    int64_t num_tokens;
    int64_t vocab;
    int num_seqs;
    int width;
    unsigned* err;
};
cudaError_t launch_accept_tree(const AcceptTreeArgs& a, int dtype, cudaStream_t s);   // dtype 0: fp16, 1: bf16, 2: fp32

struct KeepPathArgs {
    uint4* pools[2 * kMaxCopyLayers];        // every layer's K pool and V pool: [num_blocks * block_size][row_vecs]
    const int32_t* block_tables;
    const int32_t* seq_lens;
    const int32_t* query_starts;
    const int32_t* path;             // [num_seqs][width]
    const int32_t* num_accepted;     // [num_seqs]
    int64_t num_blocks;
    int num_seqs;
    int num_layers;
    int width;
    int max_blocks_per_seq;
    int block_size;
    int row_vecs;                    // 16-byte pieces of a row
    unsigned* err;
};
cudaError_t launch_keep_path(const KeepPathArgs& a, cudaStream_t s);

// Record `msg` as the calling thread's pkv_last_error() message and return `st`.
int set_error_message(int st, const char* msg);

}  // namespace pkv
