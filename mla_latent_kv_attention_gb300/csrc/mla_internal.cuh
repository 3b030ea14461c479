// mla_internal.cuh -- declarations shared by the translation units of libmla.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mla.h"

namespace mla {

constexpr int kD = MLA_D;
constexpr int kDV = MLA_DV;
constexpr int kKeyBlock = 128;     // keys per work block: the unit of split planning
// Split planning charges every sequence this many blocks' worth of time on top of its own
// blocks: a unit's epilogue and the refill of the pipeline after it. A CTA that takes a
// unit boundary gets correspondingly fewer blocks.
constexpr int kUnitCost = 5;
constexpr int kMaxRows = MLA_MAX_HEADS * MLA_MAX_NQ;  // query rows per sequence (64)

// Workspace header at offset 0 (256 bytes).
struct WsHeader {
  int num_ctas;      // CTAs of the last attention launch: status slots [0, num_ctas) are its
  int pad[63];
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Query rows one attention launch handles per unit (padded): 16, 32 or 48. More than 48
// rows per sequence run as two launches over halves of the heads.
inline int padded_rows(int rows_per_seq) {
  const int r = rows_per_seq > 48 ? (rows_per_seq + 1) / 2 : rows_per_seq;
  return r <= 16 ? 16 : (r <= 32 ? 32 : 48);
}

// One CTA's staged query image in global memory: the query operand of a later unit (two
// e4m3 terms of each padded row, in shared-memory layout) followed by the rows' score
// scales, copied into shared memory in one bulk copy when the unit starts.
inline size_t qimg_bytes(int rp) { return align_up((size_t)2 * rp * MLA_D + sizeof(float) * 48, 256); }

// Offsets of the workspace regions for one call.
//   status:   one word per CTA, written by that CTA at exit (0 or its first error)
//   qimg:     one staged query image per CTA (a tree's verify: per group of nodes)
//   part_*:   two partial slots per CTA (the first and the last unit of its block range
//             are the only ones that can hold part of a sequence), R rows each
struct WsLayout {
  size_t hdr, status, qimg, part_lse, part_out, total;
  size_t qimg_stride;
  int max_slots;
};

inline WsLayout ws_layout(int B, int rows_per_seq, int num_sms, int64_t images = 0) {
  WsLayout w;
  if (images == 0) images = num_sms;
  w.max_slots = 2 * num_sms;
  w.qimg_stride = qimg_bytes(padded_rows(rows_per_seq));
  size_t off = 0;
  w.hdr = off;
  off += sizeof(WsHeader);
  w.status = off = align_up(off, 256);
  off += sizeof(unsigned) * (size_t)num_sms;
  w.qimg = off = align_up(off, 256);
  off += w.qimg_stride * (size_t)images;
  w.part_lse = off = align_up(off, 256);
  off += sizeof(float) * (size_t)w.max_slots * rows_per_seq;
  w.part_out = off = align_up(off, 256);
  off += sizeof(float) * (size_t)w.max_slots * rows_per_seq * kDV;
  w.total = align_up(off, 256);
  return w;
}

// Tree verify: a sequence's n nodes run as groups of whole nodes, H rows each, of at most 48
// rows (what one unit of the attention kernel holds), as equal as they come. Every group reads
// all the sequence's keys, so teams of neighbouring CTAs take a group each of the same keys (a
// sequence's groups in `passes` passes of a team). The team divides the groups; of the divisors
// from four up (where the tensor cores, not HBM, set the pace of a team) or the whole the one
// that leaves the fewest SMs without a team (16 sequences of 12 heads: 64 nodes on 8K keys, 16
// groups, 224 us in teams of 4, 232 in teams of 16 on 144 of 152 SMs, 231 without teams; 24 nodes
// on 16K, 6 groups, 168 us in teams of 6, 171 to 174 of 3 and 2, 185 without).
struct TreePlan {
  int nodes;   // nodes of a group (the last may hold fewer)
  int team;    // CTAs of a team
  int passes;  // groups a sequence = team * passes
  // Query images to keep: every group's, staged by a kernel of its own beside the attention
  // kernel's prologue.
  int64_t images(int64_t B) const { return B * team * passes; }
};
// blocks: key blocks that a sequence can have at all (its page-table row's width; the lengths are
// on the device). Where even groups of 16 or 32 rows leave every CTA at most one block, the
// smaller group is the shorter wait (8 nodes of 12 heads on 1,024 keys in a table of 16 pages, rows
// of 12: 16.7 us; in one of 64 or 2,560 pages, rows of 48: 20.9 and 21.2 us); wider tables take the
// largest groups, which read the keys fewest times. The workspace is sized for the largest.
inline TreePlan tree_plan(int n, int H, int num_sms, int64_t B, int64_t blocks) {
  int most = 48 / H;
  for (int rows = 32; rows >= 16; rows -= 16)
    if (rows >= H && B * blocks * ((n + rows / H - 1) / (rows / H)) <= num_sms) most = rows / H;
  int groups = (n + most - 1) / most;
  const int nodes = (n + groups - 1) / groups;
  groups = (n + nodes - 1) / nodes;
  int team = groups <= num_sms ? groups : 1;
  for (int t = 4; t < groups; ++t)
    if (groups % t == 0 && num_sms / t * t > num_sms / team * team) team = t;
  return {nodes, team, groups / team};
}

// Prefill: the header, the per-CTA status words, the per-CTA query images (48 rows), and
// the partials of the units of the last round that are split in two along the keys: one
// slot per CTA, 48 rows each (float32 LSE, then float32 outputs).
inline size_t ws_prefill_status(int) { return align_up(sizeof(WsHeader), 256); }
inline size_t ws_prefill_qimg(int num_sms) {
  return align_up(ws_prefill_status(num_sms) + sizeof(unsigned) * (size_t)num_sms, 256);
}
inline size_t ws_prefill_part_lse(int num_sms) {
  return align_up(ws_prefill_qimg(num_sms) + qimg_bytes(48) * (size_t)num_sms, 256);
}
inline size_t ws_prefill_part_out(int num_sms) {
  return align_up(ws_prefill_part_lse(num_sms) + sizeof(float) * 48 * (size_t)num_sms, 256);
}
inline size_t ws_prefill_bytes(int num_sms) {
  return align_up(ws_prefill_part_out(num_sms) + sizeof(float) * 48 * kDV * (size_t)num_sms, 256);
}

// Everything an attention kernel needs for one call.
struct AttnParams {
  const uint8_t* pool;
  int64_t num_pages;
  int page_size;
  const int32_t* page_table;
  int64_t pt_stride;
  const int32_t* seq_lens;
  float kv_scale;
  float sm_scale;
  const uint16_t* q;  // [B][n_q][H][576]
  int B, n_q, H, R;   // R = n_q * H rows per sequence
  uint16_t* out;      // [B][n_q][H][512] bf16
  float* out_f32;     // when set, the output goes here as float32 instead of to `out`
  float* lse;         // [B][n_q][H] or null
  float* part_out;    // [slots][part_rows][512]
  float* part_lse;    // [slots][part_rows]
  int part_rows;      // rows of a partial slot: R (decode/verify), 48 (prefill)
  unsigned* status;   // [num_ctas]
  uint8_t* qimg;      // [num_ctas] staged query images, qimg_stride bytes apart
  int64_t qimg_stride;
  WsHeader* hdr;
  int num_ctas;
  int test_stall;     // test hook: the producer issues no loads, so every consumer's bounded
                      // wait runs out and the call reports MLA_ERR_TIMEOUT
  int mask_shift;     // key n visible to new position j iff n <= L - n_q + j + mask_shift
  // tree verify (null otherwise): which nodes each node sees. B then counts passes over
  // sequences (`passes` each), R the rows of a full group of group_nodes nodes, n_q all nodes.
  const uint64_t* tree_mask;  // [sequences][n_q]
  int group_nodes, team, passes;
  unsigned long long teams_inv, fewer_inv;  // ceil(2^64 / n), 0 for n = 1: n = teams, n = fewer_ranges
  unsigned long long* trace;  // profiling hook: kTraceWords globaltimer stamps per CTA, or null
  int trace_ctas;             // CTAs the trace buffer has room for
};

// Per-CTA stamps of the profiling hook (mla_set_trace_buffer), in nanoseconds of the GPU's
// global timer: entry, end of the wait on the previous kernel, end of the split plan (with
// the first tile loads issued), the first tile's scores read by the softmax, the last tile's
// probabilities written, the last values MMA done, end of the last epilogue, exit; the
// tiles and units the CTA processed; end of the first unit's epilogue and the second unit's
// first scores (CTAs with two units or more); decode/verify: end of the plan's scan, end of
// its L2 prefetches.
constexpr int kTraceWords = 16;
enum TraceSlot { kTrEntry = 0, kTrWaited, kTrPlanned, kTrFirstScores, kTrLastP, kTrLastPV,
                 kTrEpilogue, kTrExit, kTrCounts, kTrUnit1End, kTrUnit2Scores, kTrPlanScan,
                 kTrPlanPrefetch };

// The split plan's cost axis: all sequences laid end to end, each as kUnitCost units of
// fixed cost followed by its 128-key blocks (an empty sequence takes no room); CTA c owns
// the positions [c * total / n, (c + 1) * total / n). range_of(x): the CTA that holds
// position x, the largest c whose range starts at or before x.
__host__ __device__ __forceinline__ int64_t range_lo(int64_t c, int64_t total, int64_t n) {
  return c * total / n;
}
__host__ __device__ __forceinline__ int64_t range_of(int64_t x, int64_t total, int64_t n) {
  return ((x + 1) * n + total - 1) / total - 1;
}

// Ranges of a tree's cost axis: one a team, or two teams in three where that leaves a range less
// than kFewCost units: the merge then has fewer pieces, and starts on the SMs that are left. In us
// with all teams / two in three (12 heads): 8 nodes on 1,024 keys 19.0 / 16.8, 8 sequences of 8 on
// 2K keys 29.9 / 25.5, 12 of 4 on 6K (4.1 units a range) 36.2 / 32.8, 24 of 6 (8 heads) on 3K (4.6)
// 33.1 / 33.1; 17 of 20 on 0.2K to 0.8K (5.3) 31.0 / 32.3, 64 of 4 on 1.2K (6.3) 34.1 / 37.5.
constexpr int kFewCost = 5;
__host__ __device__ __forceinline__ int fewer_ranges(int teams) { return (2 * teams + 2) / 3; }
__host__ __device__ __forceinline__ int tree_ranges(int64_t total, int teams) {
  return total < (int64_t)kFewCost * teams ? fewer_ranges(teams) : teams;
}

// Up-projected 16-bit columns per head in kvup: bf16 form 128 key + 128 value columns;
// precise form 128 key (hi) + 128 key (lo) + 128 value columns.
inline __host__ __device__ int mha_up_width(bool precise) { return precise ? 384 : 256; }

// MHA-form prefill workspace: header, status words (one per attention CTA, then one for the
// dequantisation), the dequantised latent [L][512] bf16, the RoPE rows [L][64] bf16, the
// up-projected keys and values [L][H][384] 16-bit (room for the precise form's hi, lo and
// value columns; the bf16 form uses the first 256 columns' worth of each row), and the
// partials of units split along the key axis: one slot per pair of CTAs, each
// [2][128][128] float32 outputs and [2][128] float32 LSE.
struct MhaWsLayout {
  size_t status, latent, rope, kvup, part_out, part_lse, total;
};
inline MhaWsLayout mha_ws_layout(int64_t L, int H, int num_sms) {
  MhaWsLayout w;
  size_t off = align_up(sizeof(WsHeader), 256);
  w.status = off;
  off = align_up(off + sizeof(unsigned) * (size_t)(num_sms + 1), 256);
  w.latent = off;
  off = align_up(off + (size_t)L * kDV * 2, 256);
  w.rope = off;
  off = align_up(off + (size_t)L * 64 * 2, 256);
  w.kvup = off;
  off = align_up(off + (size_t)L * H * mha_up_width(true) * 2, 256);
  const size_t slots = (size_t)(num_sms / 2 + 1);
  w.part_out = off;
  off = align_up(off + slots * 2 * 128 * 128 * sizeof(float), 256);
  w.part_lse = off;
  off = align_up(off + slots * 2 * 128 * sizeof(float), 256);
  w.total = off;
  return w;
}

struct MhaArgs {
  const uint8_t* pool;
  int64_t num_pages;
  int page_size;
  const int32_t* page_table;
  float kv_scale;
  int L, T, H;
  float sm_scale;
  const void* q;      // [T][H][192] bf16
  const void* w_ukv;  // [512][H][256] bf16
  void* latent;
  void* rope;
  void* kvup;
  void* part_out;     // partials of split units (see MhaWsLayout)
  void* part_lse;
  uint16_t* out;      // [T][H][128] bf16
  float* lse;         // [T][H] or null
  unsigned* status;   // [num attention CTAs + 1]
  WsHeader* hdr;
  int device;
  int precise;        // 1: keys as bf16 hi + lo pairs, fp16 values and probabilities
  cudaEvent_t prof_start, prof_stop;  // recorded around the attention kernel when both set
};

// Launchers (each returns the CUDA error of its launch).
cudaError_t launch_merge(const AttnParams& p, cudaStream_t s);
cudaError_t launch_decode_tc(const AttnParams& p, int num_sms, cudaStream_t s, int* launches);
cudaError_t launch_tree_tc(const AttnParams& p, cudaStream_t s, int* launches);
cudaError_t launch_merge_tree(const AttnParams& p, int sequences, cudaStream_t s);
cudaError_t launch_prefill_tc(const AttnParams& p, int num_sms, cudaStream_t s, int* launches);
cudaError_t launch_merge_prefill(const AttnParams& p, int P, int split_units, cudaStream_t s);
cudaError_t launch_merge_standalone(const float* part_out, const float* part_lse, int S, int64_t R,
                                    uint16_t* out, float* lse, int num_sms, cudaStream_t s);
cudaError_t launch_cache_append(uint8_t* pool, int64_t pool_rows, const uint16_t* x,
                                const int64_t* slots, int64_t n, float inv, unsigned* status,
                                int num_sms, cudaStream_t s);
cudaError_t launch_rope(const mla_rope_t& rope, const uint16_t* x, int64_t x_token, int64_t x_head,
                        const int64_t* positions, int64_t n, int H, uint16_t* out, int64_t out_token,
                        int64_t out_head, int num_sms, cudaStream_t s);
struct AppendRopeArgs {
  uint8_t* pool;
  int64_t pool_rows;
  const uint16_t* x;       // [n] rows of 576 bf16, x_stride elements apart
  int64_t x_stride;
  const int64_t* slots;    // [n]
  int64_t n;
  float inv;               // 1 / kv_scale
  const uint16_t* weight;  // [512] bf16, or null: the latent is not normalised
  float eps;
  const int64_t* positions;  // [n], or null: no rotation
  unsigned* status;        // or null
};
cudaError_t launch_cache_append_rope(const AppendRopeArgs& a, const mla_rope_t& rope, int num_sms,
                                     cudaStream_t s);
cudaError_t launch_cache_gather(const mla_kv_t& kv, int B, const int32_t* starts,
                                const int64_t* cu_rows, int64_t n, void* out, int out_f32,
                                unsigned* status, cudaStream_t s);
struct AcceptArgs {
  const float* target;     // [B][n][V]
  const int32_t* tokens;   // [B][n]
  const int32_t* parents;  // [B][n], or null: a chain
  const float* draft;      // [B][n - 1][V], or null: drafts without probabilities
  const float* uniforms;   // [B][n + 1]
  int B, n, V;
  int32_t* out_tokens;     // [B][n]
  int32_t* path;           // [B][n]
  int32_t* num_accepted;   // [B]
};
cudaError_t launch_accept(const AcceptArgs& a, int num_sms, cudaStream_t s);
cudaError_t launch_mha_prefill(const MhaArgs& a, int num_sms, cudaStream_t s, int* launches);
cudaError_t launch_mha_projection(const void* latent, const void* w, void* kvup, int L, int H,
                                  float kv_scale, int precise, unsigned* status, cudaStream_t s);
cudaError_t launch_top_k_renorm(const float* probs, float* out, int B, int V, const int32_t* top_k,
                                int k_all, cudaStream_t s);

}  // namespace mla
