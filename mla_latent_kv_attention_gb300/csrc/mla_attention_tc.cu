// mla_attention_tc.cu -- MLA attention on tcgen05 tensor cores: split-KV decode, speculative
// verify and causal prefill over the paged FP8 latent cache.
//
// Work: one persistent CTA per SM walks the planner's units (keys [key_lo, key_hi) of one
// sequence, all of its query rows). Keys stream through shared memory 128 at a time
// (two 64-position pages, fetched by TMA straight from the paged pool) and every key is
// read from HBM exactly once per unit, whatever the head count or verify depth.
//
// Both contractions run on the FP8 cache bytes as they are, with no dequantisation pass:
//   scores  S^T[key][n] = sum_d code[key][d] * Qt[n][d]      tcgen05 kind::f8f6f4,
//           M = 128 keys, N = 2 x (padded rows), K = 576
//           The bf16 query row, scaled by the power of two that puts its largest
//           magnitude in (224, 448], is split into two e4m3 terms stacked along N: the
//           first is the entry rounded to e4m3, the second the residual times 16 rounded
//           to e4m3 (the residual is at most 16, so this never saturates), and the two
//           accumulators are summed as S1 + S2 / 16. The split is exact for every entry of
//           at least 2^-14.8 of the row's largest magnitude (bf16 has 8 significant bits,
//           e4m3 4, and the scaled residual is a multiple of e4m3's subnormal step there);
//           a smaller entry is carried to within 2^-21.8 of the row's largest magnitude.
//   values  O^T[dv][n]  += sum_key code[key][dv] * Pt[n][key] tcgen05 kind::f8f6f4,
//           M = 128 dv (x4 chunks), N = rows, K = keys; the same FP8 tile read MN-major
//           (A: e4m3 codes) against the probabilities as three e5m2 terms (B). A weight
//           p = 2^(x - m + 11) (at most 2^15) is rounded to fp16 and split by round to
//           nearest into e5m2 terms t0 + t1 + t2: each term takes the leading 3 bits of
//           what the previous ones left, so the sum carries p to about fp16's precision,
//           and e5m2's range (2^-16 .. 57344) keeps that precision for weights down to
//           about 2^-19 of the running maximum. Smaller weights lose bits gradually; the
//           smallest one kept is 2^-28 of the maximum. (An e4m3 split loses every weight
//           below about 2^-14 of the maximum: a long tail under a dominant key would then
//           vanish from the numerator but not from the row sum.)
// Keys sit on the MMA's M side ("swap A/B"): 8-16 heads x 1-4 positions are far below
// M = 128, so the few query rows take the narrow N side and nothing is padded in memory.
// Softmax is online over key tiles; one warpgroup owns one key per thread (its TMEM
// lane), so the running max per row needs a cross-warp reduction each tile.
//
// Roles: warp 0 issues TMA, warp 1 owns TMEM and issues the score MMAs, warp 3 issues the
// value MMAs, warp 2 stages query rows, and from warp 4 on two warpgroups (three with 48
// rows per unit: 384 or 512 threads) run the softmax and write the epilogue. Every wait is
// bounded.
//
// What bounds it: with 16 rows HBM (32 x 4K-16K keys: 28 us of the 44.7 that a call takes stream at
// 6.7 TB/s, the rest is start, epilogue and merge), with 48 the tile's chain. At 48 rows a tile's MMAs
// take about 2,700 cycles of the tensor pipe and the tile 3,400 to 3,600 (prefill 1.7 us, 8,192 on 32K
// 6.64 ms, 1.19 PFLOP/s, 0.63 of the measured bf16 rate): values - load - scores of a stage, two of
// them, sets the pace, so whatever issues on it was made shorter (Issuer), and the code smaller, which
// the tile loops and a call's start fetch through caches they overflow.
//
// Tree verify (PF = 3) is the same kernel over groups of a sequence's nodes, each node seeing the
// prefix and the nodes its 64-bit mask names: teams of CTAs walk the same keys, a group each; the
// query images come from a kernel of their own; a key's column of the masks is looked up only
// in tiles that reach the nodes. 32 x 32 nodes of 12 heads over 4K-16K keys: 270 us, 1.01
// PFLOP/s, 0.53 of the measured bf16 rate.
//
// Block scales (SC): key n's codes count times s_n, its block's scale. A softmax thread owns a key, so
// s_n is one number a thread and tile: with x_n the key's score in log2 units, its weight in the values
// MMA is 2^(x_n + log2 s_n - m) (the MMA then adds s_n v_n in units of the codes), its share of the row
// sum that weight over s_n, and m the running maximum of x_n + log2 s_n. That costs the tile loop one
// multiply-add a score and nothing in memory traffic but the scales, loaded a tile ahead (BlockScales);
// a rounded log2 acts on numerator and sum alike. The three e5m2 terms then keep their precision
// relative to the largest weight times scale, which is what the output's absolute error is about.
// One scale / scales of blocks, in us, the same codes: decode 32 x 4K-16K 44.7 / 45.5, 142,000 27.2 /
// 27.9, verify 8 x 4 on 32K 52.8 / 53.9, 8 x 16 nodes on 32K 126 / 133 (half of it from maxima that
// move more often where blocks differ), prefill 8,192 on 32K 6,640 / 6,690.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <math.h>
#include <stddef.h>

#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int kTileKeys = 128;
constexpr int kStages = 2;
constexpr int kChunkBytes = 16384;                     // 128 keys x 128 bytes, SW128
constexpr int kStageBytes = 4 * kChunkBytes + 2 * 4096;  // 73,728 bytes loaded per tile
// A stage is filled and freed in three parts: latent chunks 0-1, chunk 2, chunk 3 with the RoPE
// tail. The values MMA frees a part as soon as its own MMAs complete, so the next tile's keys begin
// to land while the rest of the stage is still being read. (Every tcgen05.commit costs the issuing
// warp time: draft trees, 32 x 32 nodes over 4K-16K, 291.7 us in two parts, 287.7 in three; four
// parts or 3 + 1 chunks ran slower.)
constexpr int kParts = 3;
__host__ __device__ constexpr int part_of_chunk(int c) { return c < 2 ? 0 : c - 1; }
constexpr int kTailPart = kParts - 1;
__host__ __device__ constexpr bool part_begins(int c) {
  return c == 0 || part_of_chunk(c) != part_of_chunk(c - 1);
}
__host__ __device__ constexpr bool part_ends(int c) {
  return c == 3 || part_of_chunk(c) != part_of_chunk(c + 1);
}
__host__ __device__ constexpr int part_bytes(int part) {
  int bytes = part == kTailPart ? 2 * 4096 : 0;
  for (int c = 0; c < 4; ++c) bytes += part_of_chunk(c) == part ? kChunkBytes : 0;
  return bytes;
}
static_assert(part_bytes(0) + part_bytes(1) + part_bytes(2) == kStageBytes, "the parts make up the stage");
constexpr int kMaxThreads = 512;  // producer, 2 MMA issuers, query stager, 2-3 softmax warpgroups
constexpr int kSoftmaxWarp0 = 4;
constexpr uint64_t kWaitLimitNs = 1000000000ull;        // 1 s
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPScale = 11.0f;     // P carried as 2^(x - m + 11): at most 2^15 while x <= m + 4
constexpr float kRescaleGap = 4.0f;  // the running max (log2 units) moves only past m + 4
// Tree verify and block scales use what e5m2 still holds above that (2^15.75 < 57,344 < 2^16): moving the max
// rescales O in tensor memory, and half as many tiles of N(0, 1) data do (a rescale costs its
// warpgroup about 1.5 us).
constexpr float kTreeGap = 4.75f;
constexpr float kQTerm2 = 16.0f;     // the second query term carries the residual times 16
constexpr float kNoMax = -1e30f;     // running max (less kPScale) of a row that has seen no key
constexpr int kPrefetchTiles = 1;    // tiles the producer pulls into L2 ahead of its TMA loads

// FINE: the probabilities as six e5m2 terms instead of three, in two sets of three side by side, both
// summed by the same accumulators: 18 bits, for float32 outputs under block scales, whose error falls
// from 1e-6 .. 1e-4 to 3e-7 .. 8e-7 (what a float32 computation of the formulas gives). In us, bfloat16
// out and three terms / float32 out and six: decode 32 x 4K-16K 45.5 / 50.0, verify 32 x 2 57.1 / 63.5; more
// than 32 rows of a sequence, which run as two halves of the heads, each reading the keys: 8 x 4 on 32K
// 54.2 / 98.0, of 16 heads (halved either way) 93.4 / 104.
template <int RP, bool FINE = false>
struct Cfg {
  static_assert(!FINE || RP <= 32, "six terms do not fit a 48-row unit's stages");
  static constexpr int kSets = FINE ? 2 : 1;
  // softmax warpgroups: three at 48 rows (16 rows per thread), else two
  static constexpr int kNWG = (RP == 48) ? 3 : 2;
  static constexpr int kThreads = 128 + 128 * kNWG;
  static constexpr int kRH = RP / kNWG;                // query rows per softmax thread
  static constexpr int kStageWarps = kThreads / 32 - 2;  // warps 2.. stage the first units
  static constexpr int NQK = 2 * RP;                    // two query terms per row
  // S^T buffers: two (the next tile's scores land while the softmax works on this one),
  // one at 48 rows, where TMEM is needed for stacked O chunks
  static constexpr int kSBuf = (RP == 48) ? 1 : 2;
  // O^T chunk c (128 dv lanes) holds the three P terms' products side by side ("stacked":
  // one N = 3 RP MMA per k-step, the V^T tile read once) or summed in one accumulator
  // (three N = RP MMAs per k-step, V^T read three times). Stacked everywhere up to 32
  // rows; at 48 rows TMEM holds two stacked chunks and two summed ones.
  static constexpr int kStackedChunks = (RP == 48) ? 2 : 4;
  static constexpr __host__ __device__ int oterms(int c) { return c < kStackedChunks ? 3 : 1; }
  static constexpr int kSCol = 0;                       // S^T buffers: [0, kSBuf NQK)
  static constexpr int kOCol = kSBuf * NQK;             // O^T chunks from here
  static constexpr __host__ __device__ int ocol(int c) {
    return kOCol + (c < kStackedChunks ? c * 3 * RP : kStackedChunks * 3 * RP + (c - kStackedChunks) * RP);
  }
  // all O^T columns are one run of kOParts pieces of RP columns (chunk by chunk, term by term)
  static constexpr int kOParts = kStackedChunks * 3 + (4 - kStackedChunks);
  static constexpr int kTmemUsed = ocol(3) + oterms(3) * RP;
  static constexpr int kTmemCols = kTmemUsed <= 256 ? 256 : 512;
  static constexpr int kQBytes = NQK * kD;
  // query operand buffers: two (the next unit is staged during this one) when they fit
  static constexpr int kQB = (RP == 16) ? 2 : 1;
  // A stage holds one key tile: dims 0..511 as four SW128 chunks of 128 keys x 128 bytes,
  // then dims 512..575 (the tail, SW64, 128 keys x 64 bytes). At 48 rows each stage also
  // holds its tile's probabilities (P^T, three e5m2 terms of 6 KB), so the softmax can
  // write the next tile's P while the values MMA still reads this one: terms 1 and 2 in
  // 12 KB between the chunks and the tail, term 0 over the first 6 KB of the tail, which
  // the scores no longer need by then. Otherwise one P buffer serves every tile.
  static constexpr bool kPInStage = (RP == 48);
  static constexpr int kPTerm = (RP / 16) * 2048;       // one term: RP/16 groups of 16 rows
  static constexpr int kTail = 4 * kChunkBytes + (kPInStage ? 2 * kPTerm : 0);
  static constexpr int kStageStride = kTail + 2 * 4096;
  static constexpr int kPBytes = kPInStage ? 0 : kSets * 3 * kPTerm;
  // offset of P term t from the P base (the stage's P area, or the shared buffer)
  static constexpr __host__ __device__ int pterm(int t) {
    return kPInStage ? ((t + 2) % 3) * kPTerm : t * kPTerm;
  }
  // shared memory layout (offsets from a 1024-aligned base)
  static constexpr int kOffStages = 0;
  static constexpr int kOffP = kStages * kStageStride;
  static constexpr int kOffQ = kOffP + ((kPBytes + 1023) / 1024) * 1024;
  static constexpr int kOffMisc = kOffQ + kQB * kQBytes;
  static_assert(kTmemUsed <= 512, "TMEM budget");
  static_assert(kOffMisc % 16 == 0 && kOffQ % 1024 == 0 && kOffP % 1024 == 0 &&
                    kQBytes % 1024 == 0, "alignment");
};

struct Misc {
  // float arrays first: they are read as float4 and must be 16-byte aligned
  alignas(16) float row_scale[2][48];  // by unit parity
  alignas(16) float red[2][48 * 4];  // per-tile warp maxima, [row][warp]
  alignas(16) float lred[4][48];
  alignas(16) float row_max[2][48];  // running maxima, by parity of the times they moved
  alignas(16) float alpha[48];       // this tile's rescale factors (each warp of a
                                     // warpgroup writes the same values for its rows)
  alignas(16) int row_j[48];         // new-position index j of each row (very negative for padding)
  alignas(16) int row_off[48];       // j * H + h: the row's index among its sequence's rows
  alignas(8) uint64_t kv_full[kStages][kParts];  // part landed (TMA transaction bytes)
  uint64_t kv_free[kStages][kParts];             // part no longer read by any MMA
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2];   // P of tile g is written: p_full[g % 2] (the softmax may run a tile
                        // ahead of the value MMAs when P lives in the stage)
  uint64_t q_full[2];   // query operand buffer holds its unit's terms
  uint64_t q_empty[2];  // the unit that used the buffer has finished its scores, and the softmax
                        // warps have read its row_scale
  uint64_t q0_done;     // the first unit's query rows are staged (by warps 2.. together)
  uint64_t q1_done;     // the second unit's rows are in this CTA's global query image
  uint64_t wg_bar[3];  // bounded barriers of the softmax warpgroups (128 arrivals)
  // decode/verify split plan of this CTA: positions [x0, x1) of the cost axis (all
  // sequences end to end, each as kUnitCost fixed units then its blocks); its first unit
  // is sequence b0 (length L0), whose first block sits at pre0
  long long plan_x0, plan_x1, plan_pre0;
  int plan_b0, plan_L0;
  int plan_seq0, plan_pass0, member;  // tree: b0 = seq0 * passes + pass0; this CTA's place in its team
  int scan[kMaxThreads / 32];
  uint32_t tmem_base;
  int abort;
  unsigned status;  // this CTA's first error
};
static_assert(offsetof(Misc, row_scale) % 16 == 0 && offsetof(Misc, red) % 16 == 0 &&
                  offsetof(Misc, lred) % 16 == 0 && offsetof(Misc, alpha) % 16 == 0 &&
                  offsetof(Misc, row_j) % 16 == 0,
              "vector-accessed arrays must be 16-byte aligned");
static_assert(offsetof(Misc, kv_full) % 8 == 0, "mbarriers must be 8-byte aligned");

template <int RP, bool FINE = false>
constexpr int smem_bytes() {
  return Cfg<RP, FINE>::kOffMisc + (int)sizeof(Misc) + 1024;
}
static_assert(smem_bytes<16, true>() <= 232448 && smem_bytes<32, true>() <= 232448 && smem_bytes<48>() <= 232448,
              "dynamic shared memory per CTA");

struct DecodeArgs {
  AttnParams p;
  int h0, Hs;  // heads [h0, h0 + Hs) handled by this launch
  int rows;    // rows per unit: n_q * Hs (decode/verify) or P * H (prefill), <= RP
  int prefill;    // 1: units are blocks of P new positions of one sequence (no split plan)
  int P;          // prefill: new positions per unit
  int num_units;  // prefill: ceil(n_q / P)
  int unit_end;   // prefill: this launch's units are [blockIdx.x, unit_end) in steps of the grid
  int split_base;  // prefill: units [split_base, num_units) run as two halves each
  int status_overwrite;  // 1: each CTA writes its status word even when clean (first launch)
};

// One unit of work as every role of the kernel sees it.
struct UnitInfo {
  int b, key_lo, key_hi;
  int L;          // cached positions of sequence b
  int qrow0;      // global row (of q, out, lse) of the unit's row 0
  int j0;         // new-position index of the unit's first position
  int rows;       // valid rows of the unit
  int final_out;  // 1: bf16 out + lse directly; 0: normalised partial for the merge
  int slot;       // partial slot (when final_out == 0)
  int image;      // tree: the unit's query image
};

// Position in this CTA's list of units. Decode/verify: the sequences whose blocks overlap
// the CTA's range, in order (b, the cost-axis position pre of its first block, its length
// L). Prefill: unit index u.
struct Cursor {
  int u;
  int b;
  long long pre;
  int L;
  int seq, pass;  // tree: b = seq * passes + pass
};

__device__ __forceinline__ int seq_len_of(const AttnParams& p, int b) {
  int L = p.seq_lens[b];
  const int64_t cap = p.pt_stride * (int64_t)p.page_size;
  if (L < 0) return 0;
  if ((int64_t)L > cap) return (int)cap;
  return L;
}

__device__ __forceinline__ int blocks_of(int L) { return (L + kKeyBlock - 1) / kKeyBlock; }

// A final output element: bf16, or float32 when the caller asked for it.
__device__ __forceinline__ void store_out(const AttnParams& p, int64_t idx, float v) {
  if (p.out_f32)
    p.out_f32[idx] = v;
  else
    p.out[idx] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// PF: 0 decode/verify (the split plan's units); 1 prefill (units are blocks of new
// positions, one a round per CTA); 2 prefill, the two halves along the keys of each unit of
// an incomplete last round (one half a CTA, a partial for the merge); 3 tree verify (the split
// plan over groups of a sequence's nodes). A compile-time parameter: each kernel carries only
// its own paths.
__host__ __device__ constexpr bool is_prefill(int pf) { return pf == 1 || pf == 2; }

// Tree verify: neighbouring CTAs form teams of p.team, and the plan cuts its cost axis into one
// range a team. What the plan calls a sequence is a pass over one, in which member m of the team
// takes group (pass * team + m) of its nodes: the members walk the same keys at the same time,
// so a tile comes from HBM once and from L2 for the others. Each group's query image is staged by
// a kernel of its own (stage_queries_kernel).
//
// The plan's indices b in order, with the sequence each stands for (a pass over it, in a tree;
// counted along, so that no index is divided).
template <int PF>
struct PlanIndex {
  int b, seq, pass;
  __device__ __forceinline__ PlanIndex(const AttnParams& p, int first) : b(first), seq(first), pass(0) {
    if constexpr (PF == 3) {
      seq = first / p.passes;
      pass = first % p.passes;
    }
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    ++b;
    if constexpr (PF == 3) {
      if (++pass == p.passes) {
        pass = 0;
        ++seq;
      }
    } else {
      ++seq;
    }
  }
};

template <int PF>
__device__ __forceinline__ Cursor first_unit(const DecodeArgs& a, const Misc* ms) {
  Cursor c;
  c.u = blockIdx.x;
  c.b = ms->plan_b0;
  c.pre = ms->plan_pre0;
  c.L = ms->plan_L0;
  if constexpr (PF == 3) {
    c.seq = ms->plan_seq0;
    c.pass = ms->plan_pass0;
  }
  return c;
}

template <int PF>
__device__ __forceinline__ bool has_unit(const DecodeArgs& a, const Misc* ms, const Cursor& c) {
  return is_prefill(PF) ? c.u < a.unit_end : (c.b < a.p.B && c.pre < ms->plan_x1);
}

// The next unit: the next sequence with at least one key (decode/verify), or the next
// unit index this CTA owns (prefill).
template <int PF>
__device__ __forceinline__ Cursor next_unit(const DecodeArgs& a, Cursor c) {
  if (is_prefill(PF)) {
    c.u += gridDim.x;
    return c;
  }
  c.pre += blocks_of(c.L);
  do {
    ++c.b;
    if constexpr (PF == 3) {
      if (++c.pass == a.p.passes) {
        c.pass = 0;
        ++c.seq;
      }
    }
    c.L = (c.b < a.p.B) ? seq_len_of(a.p, PF == 3 ? c.seq : c.b) : 0;
  } while (c.b < a.p.B && c.L == 0);
  c.pre += kUnitCost;  // the next sequence's fixed cost precedes its blocks
  return c;
}

template <int PF>
__device__ __forceinline__ UnitInfo unit_info(const DecodeArgs& a, const Misc* ms, const Cursor& c) {
  const AttnParams& p = a.p;
  UnitInfo x;
  if (!is_prefill(PF)) {
    const long long nb = blocks_of(c.L);
    const long long blo = max(ms->plan_x0, c.pre), bhi = min(ms->plan_x1, c.pre + nb);
    x.b = c.b;
    x.L = c.L;
    x.key_lo = (int)(blo - c.pre) * kKeyBlock;
    x.key_hi = (bhi > blo) ? min(c.L, (int)(bhi - c.pre) * kKeyBlock) : x.key_lo;
    x.qrow0 = c.b * p.R;
    x.j0 = 0;
    x.rows = a.rows;
    if constexpr (PF == 3) {  // this CTA's group of the sequence's nodes (the last may be short)
      const int group = c.pass * p.team + ms->member;
      x.b = c.seq;
      x.image = c.seq * (p.passes * p.team) + group;
      x.j0 = group * p.group_nodes;
      x.qrow0 = (c.seq * p.n_q + x.j0) * p.H;
      x.rows = min(p.group_nodes, p.n_q - x.j0) * p.H;
    }
    x.final_out = (blo == c.pre && bhi == c.pre + nb);
    // the CTA's first unit (nothing of an earlier sequence in its range) takes slot 2c
    x.slot = 2 * (int)blockIdx.x + (c.pre - kUnitCost <= ms->plan_x0 ? 0 : 1);
  } else {
    // the last positions see the most keys: hand those out first
    int v = c.u;
    if constexpr (PF == 2) v = a.split_base + c.u / 2;  // unit v, half c.u & 1
    const int pos0 = (a.num_units - 1 - v) * a.P;
    const int npos = min(a.P, p.n_q - pos0);
    const int L = seq_len_of(p, 0);
    x.b = 0;
    x.L = L;
    x.key_lo = 0;
    x.key_hi = max(0, min(L, L - p.n_q + pos0 + npos));  // last key the unit's last position sees, + 1
    x.qrow0 = pos0 * p.H;
    x.j0 = pos0;
    x.rows = npos * p.H;
    x.final_out = 1;
    x.slot = 0;
    if constexpr (PF == 2) {  // keys [0, mid) or [mid, key_hi), partial slot c.u
      const int mid = min(x.key_hi, ((x.key_hi + 2 * kTileKeys - 1) / (2 * kTileKeys)) * kTileKeys);
      if (c.u & 1)
        x.key_lo = mid;
      else
        x.key_hi = mid;
      x.final_out = 0;
      x.slot = c.u;
    }
  }
  return x;
}

__device__ __forceinline__ int tiles_in(const UnitInfo& x) {
  return (x.key_hi - x.key_lo + kTileKeys - 1) / kTileKeys;
}

// First error of this CTA wins; the CTA writes it to its status word at exit.
__device__ __forceinline__ void report(Misc* m, mla_status_t code) {
  atomicCAS(&m->status, 0u, (unsigned)code);
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Misc* m,
                                              const AttnParams& p) {
  if (mbar_wait(bar, parity, kWaitLimitNs)) return true;
  m->abort = 1;
  report(m, MLA_ERR_TIMEOUT);
  return false;
}

// A warp that runs whole leaves together: the outcome of a wait that any of its lanes gave up.
__device__ __forceinline__ bool warp_waited(bool ok) { return (bool)__all_sync(0xffffffffu, ok); }

__device__ __forceinline__ bool aborted(const Misc* m) {
  return *reinterpret_cast<const volatile int*>(&m->abort) != 0;
}

// fp8 e4m3 helpers (round to nearest even, saturating; and exact back-conversion)
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
  return (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
  __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// the same for e5m2, from float32 and back
__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E5M2);
}
__device__ __forceinline__ float2 from_e5m2x2(uint32_t v) {
  __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E5M2);
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// four e4m3 codes, NaN ones (0x7F, 0xFF) as zero
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// (lo, hi) -> f16x2 with lo in the low half
__device__ __forceinline__ uint32_t f32x2_to_f16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
__device__ __forceinline__ uint32_t e5m2x2_to_f16x2(uint32_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return h;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Byte offset of the 16-byte group `w16` (16 codes, dims 16*w16 .. +15) of term-row n
// inside the query operand (K-major: four SW128 chunks of 128 dims, then one SW64 chunk).
template <int NQK>
__device__ __forceinline__ int q_offset(int n, int w16) {
  if (w16 < 32) {
    const int c = w16 >> 3, w = w16 & 7;
    return c * (NQK * 128) + (n >> 3) * 1024 + (n & 7) * 128 + ((w ^ (n & 7)) << 4);
  }
  const int w = w16 - 32;
  return 4 * (NQK * 128) + (n >> 3) * 512 + (n & 7) * 64 + (((w ^ ((n & 7) >> 1)) & 3) << 4);
}

// Stage rows w, w + nw, ... (< RP) of one unit's queries into a query operand buffer as two
// e4m3 terms after a per-row power-of-two scale (the entry rounded, then 16 x the residual
// rounded: exact for entries down to 2^-14.8 of the row's largest magnitude, within
// 2^-21.8 of it below), and the rows' score scales into row_scale[]. Rows at or past R are
// written as zeros.
//
// INF: a row with an infinite entry, which saturates to 448, gets a NaN scale: its scores are then
// NaN, as its softmax is by the formula. (In the attention kernels themselves that one addition
// moved the 48-row code enough to cost verify 1 %: 69.3 -> 70.0 us.)
template <int RP, int NW, bool INF = false>
__device__ __forceinline__ void stage_rows(const AttnParams& p, int R, const int* row_off,
                                       const uint16_t* qseq, uint8_t* qdst, float* row_scale,
                                       int w0, int lane) {
  using C = Cfg<RP>;
  const float kv_scale = p.kv_scale;
  constexpr int nw = NW;  // warps staging together
  // Rows of one pass of a warp: two. Fewer are shorter code, fetched cold at a call's start, more hide a
  // lone warp's loads better (in us, one / two / three a pass: verify 8 x 4 on 32K 53.1 / 53.8 / 54.1, 300 x
  // 2 on 200 55.9 / 53.1 / 52.3, decode 512 x 100-300 53.1 / 50.1 / 50.3, prefill 2,048 178 / 155 / 160).
  constexpr int K2 = (RP + NW - 1) / NW < 2 ? (RP + NW - 1) / NW : 2;
  // rows r0, r0 + nw, ... of this warp: all loads first, then the arithmetic. A lane takes latent dims
  // 16 lane .. + 15 and RoPE dims 2 lane, 2 lane + 1 (a whole group of 16 RoPE dims a lane would have the
  // warp run the conversion a second time for four lanes).
  for (int r0 = w0; r0 < RP; r0 += K2 * nw) {
    uint4 ld[K2][2];
    uint32_t tl[K2];
#pragma unroll
    for (int k2 = 0; k2 < K2; ++k2) {
      const int r = r0 + nw * k2;
      ld[k2][0] = ld[k2][1] = make_uint4(0, 0, 0, 0);
      tl[k2] = 0;
      if (r < R) {
        const uint16_t* row = qseq + (int64_t)row_off[r] * kD;
        const uint4* s4 = reinterpret_cast<const uint4*>(row);
        ld[k2][0] = s4[2 * lane];
        ld[k2][1] = s4[2 * lane + 1];
        tl[k2] = reinterpret_cast<const uint32_t*>(row + kDV)[lane];
      }
    }
#pragma unroll
    for (int k2 = 0; k2 < K2; ++k2) {
      const int r = r0 + nw * k2;
      if (r >= RP) break;
      const bool real = r < R;
      float v[18];  // the latent entries, then the two of the RoPE part
      {
        const uint32_t w[9] = {ld[k2][0].x, ld[k2][0].y, ld[k2][0].z, ld[k2][0].w, ld[k2][1].x,
                               ld[k2][1].y, ld[k2][1].z, ld[k2][1].w, tl[k2]};
#pragma unroll
        for (int e = 0; e < 18; ++e) v[e] = __uint_as_float((w[e >> 1] >> ((e & 1) * 16)) << 16);
      }
      float amax = 0.f;
#pragma unroll
      for (int e = 0; e < 18; ++e) amax = fmaxf(amax, fabsf(v[e]));
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // scale 2^ex so that amax * 2^ex lies in (224, 448]; from the exponent field of
      // amax (normal floats: biased exponent E means amax in [2^(E-127), 2^(E-126)))
      int ex = 0;
      if (amax >= 1.17549435e-38f && amax <= 3.4e38f) {
        const int E = (__float_as_int(amax) >> 23) & 0xFF;
        ex = 135 - E;  // amax * 2^ex in [256, 512)
        if (amax * __int_as_float((127 + ex) << 23) > 448.f) ex -= 1;
        ex = max(-126, min(126, ex));  // both 2^ex and 2^-ex stay normal floats
      }
      const float up = __int_as_float((127 + ex) << 23);    // 2^ex, exact
      const float down = __int_as_float((127 - ex) << 23);  // 2^-ex, exact
      if (lane == 0) {
        float scale = real ? p.sm_scale * kv_scale * down * kLog2e : 0.f;
        if (INF) scale += amax - amax;  // 0, or NaN
        row_scale[r] = scale;
      }
      // two terms per value, two codes (one pair of values) a word's half
      uint32_t t1[9], t2[9];
#pragma unroll
      for (int e = 0; e < 9; ++e) {
        const float a0 = v[2 * e] * up, a1 = v[2 * e + 1] * up;
        t1[e] = to_e4m3x2(a0, a1);
        const float2 b1 = from_e4m3x2((uint16_t)t1[e]);
        t2[e] = to_e4m3x2((a0 - b1.x) * kQTerm2, (a1 - b1.y) * kQTerm2);
      }
      auto words = [](const uint32_t* t) {
        return make_uint4(t[0] | t[1] << 16, t[2] | t[3] << 16, t[4] | t[5] << 16, t[6] | t[7] << 16);
      };
      *reinterpret_cast<uint4*>(qdst + q_offset<C::NQK>(r, lane)) = words(t1);
      *reinterpret_cast<uint4*>(qdst + q_offset<C::NQK>(RP + r, lane)) = words(t2);
      const int w16 = 32 + (lane >> 3), in16 = (lane & 7) * 2;  // the RoPE pair's group, its place there
      *reinterpret_cast<uint16_t*>(qdst + q_offset<C::NQK>(r, w16) + in16) = (uint16_t)t1[8];
      *reinterpret_cast<uint16_t*>(qdst + q_offset<C::NQK>(RP + r, w16) + in16) = (uint16_t)t2[8];
    }
  }
}

// How the producer and the two issuing warps run: whole, an elected lane issuing. The control flow
// and the operands are then the same for every lane as far as the compiler can tell (votes and
// broadcasts say so), so it keeps them (of a descriptor only the low half moves) in the uniform
// registers that the MMA and the TMA read, instead of moving up to eight registers there for each
// one. All three lie on the chain of a key stage (values done, load, scores). In us, one thread
// each (and a stage in two parts) / this: draft trees, 32 x 32 nodes over 4K-16K, 315 / 291 for the
// MMAs, 281 / 270 for the loads; prefill 8,192 on 32K 8,787 / 6,777; verify 8 x 4 on 32K 69.2 / 57.1;
// decode 32 x 4K-16K 48.9 / 46.5, 142,000 30.8 / 28.7, 512 x 100-300 60.1 / 57.6.
struct Issuer {
  uint32_t leader;
  __device__ __forceinline__ Issuer() : leader(elect_one()) {}
  __device__ __forceinline__ bool same(bool v) const { return (bool)__all_sync(0xffffffffu, v); }
  __device__ __forceinline__ uint32_t same(uint32_t v) const { return __shfl_sync(0xffffffffu, v, 0); }
  // a tile's place within a descriptor's base, and the descriptor `off` (16-byte units) past it
  __device__ __forceinline__ uint32_t place(uint64_t base, uint32_t tile_off) const {
    return same((uint32_t)base + tile_off);
  }
  static __device__ __forceinline__ uint64_t at(uint64_t base, uint32_t place, uint32_t off) {
    return (base >> 32 << 32) | (place + off);
  }
  __device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                      uint32_t accumulate) const {
    mma_f8f6f4_by(leader, d, a, b, idesc, accumulate);
  }
  __device__ __forceinline__ void load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar,
                                       uint64_t policy) const {
    tma_load_2d_hint_by(leader, dst, map, x, y, bar, policy);
  }
  __device__ __forceinline__ void commit(uint64_t* bar) const {
    if (leader) mma_commit(bar);
  }
};

// A key's scale as the softmax uses it. A scale that is none gives NaN scores to the rows that see the
// key (those that do not see it are masked after the scores, and their weight 0 meets finite numbers).
// The approximate log2 (2^-22) enters weight and row sum alike, the reciprocal (2^-23) the sum; both
// are exact for powers of two.
struct KeyScale {
  float scale, log2, inv;
  __device__ __forceinline__ KeyScale() {}
  __device__ __forceinline__ explicit KeyScale(float s) {
    const bool good = is_scale(s);
    scale = good ? s : __int_as_float(0x7FC00000);
    const float t = good ? s : 1.f;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(log2) : "f"(t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(t));
  }
};

// One thread's walk over the scales of its keys, 128 positions a tile. Its keys are places of one
// 64-key half of every tile, which lies in one page; the page's place in the table is counted along.
// (Pool rows fit 32 bits: encode_pool_maps refuses more.)
struct BlockScales {
  const int32_t* table;  // the sequence's page-table entry of the half
  float next;            // the coming tile's scale (1 past the unit's keys)
  int page;              // the pool page of the tile after it, or -1
  int kk, off;           // this thread's key in that tile: position, offset in its page
  __device__ __forceinline__ void find(int key_hi) { page = kk < key_hi ? __ldg(table) : -1; }
  __device__ __forceinline__ void load(const AttnParams& p) {
    next = 1.f;
    if ((unsigned)page < (unsigned)p.num_pages)
      next = __ldg(p.scales + ((unsigned)(page * p.page_size + off) >> p.scale_shift));
  }
  __device__ __forceinline__ void advance(const AttnParams& p) {
    kk += kTileKeys;
    off += kTileKeys;
    while (off >= p.page_size) {
      off -= p.page_size;
      ++table;
    }
  }
  // key: this thread's in the unit's first tile
  __device__ __forceinline__ void begin(const AttnParams& p, int b, int key, int key_hi) {
    kk = key;
    table = p.page_table + (int64_t)b * p.pt_stride + kk / p.page_size;
    off = kk % p.page_size;
    find(key_hi);
    load(p);
    advance(p);
    find(key_hi);
  }
  // this tile's scale; the next one's load goes out
  __device__ __forceinline__ KeyScale take(const AttnParams& p, int key_hi) {
    const float s = next;
    load(p);
    advance(p);
    find(key_hi);
    return KeyScale(s);
  }
};

template <int RP, int PF, bool TR, bool SC, bool FINE>
__global__ void __launch_bounds__(Cfg<RP>::kThreads, 1)
    attn_tc_kernel(const __grid_constant__ DecodeArgs args,
                     const __grid_constant__ CUtensorMap map_main,
                     const __grid_constant__ CUtensorMap map_tail) {
  using C = Cfg<RP, FINE>;
  const AttnParams& p = args.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Misc* ms = reinterpret_cast<Misc*>(smem + C::kOffMisc);
  uint8_t* pbuf = smem + C::kOffP;
  uint8_t* qbuf = smem + C::kOffQ;
  const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  // profiling hook: this CTA's stamps, or null
  // (TR: a separate instantiation for traced calls, so the usual one carries no stamp code)
  unsigned long long* const trace = (TR && p.trace && (int)blockIdx.x < p.trace_ctas)
                                        ? p.trace + (size_t)blockIdx.x * kTraceWords
                                        : nullptr;
  if (trace && threadIdx.x == 0) trace[kTrEntry] = globaltimer_ns();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s)
      for (int c = 0; c < kParts; ++c) {
        mbar_init(&ms->kv_full[s][c], 1);
        mbar_init(&ms->kv_free[s][c], 1);
      }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->s_full[s], 1);
      mbar_init(&ms->s_empty[s], 4 * C::kNWG);  // one arrival per softmax warp
    }
    for (int w = 0; w < C::kNWG; ++w) mbar_init(&ms->wg_bar[w], 4);
    mbar_init(&ms->p_full[0], 4 * C::kNWG);
    mbar_init(&ms->p_full[1], 4 * C::kNWG);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ms->q_full[s], 1);
      mbar_init(&ms->q_empty[s], 1 + 4 * C::kNWG);
    }
    mbar_init(&ms->q0_done, 32 * C::kStageWarps);
    mbar_init(&ms->q1_done, 32 * C::kStageWarps);
    ms->abort = 0;
    ms->status = 0;
    ms->plan_b0 = args.p.B;  // no unit unless the plan finds one
    ms->plan_x0 = ms->plan_x1 = ms->plan_pre0 = 0;
    ms->plan_L0 = 0;
    if constexpr (PF == 3) {
      ms->plan_seq0 = ms->plan_pass0 = 0;
      ms->member = blockIdx.x % args.p.team;
    }
    fence_mbar_init();
    prefetch_tensormap(&map_main);
    prefetch_tensormap(&map_tail);
  }
  // the unit's row tables, one entry a thread (a single thread spent about 3 us on them,
  // integer divisions included, ahead of everything else)
  if (threadIdx.x < 48) {
    const int r = threadIdx.x;
    ms->row_j[r] = (r < args.rows) ? r / args.Hs : -(1 << 30);
    ms->row_off[r] = (r < args.rows) ? (r / args.Hs) * p.H + args.h0 + r % args.Hs : 0;
  }
  if (warp == 1) tmem_alloc(&ms->tmem_base, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  // Everything above may overlap the previous kernel in the stream (programmatic dependent
  // launch); inputs are read only after it has completed. The merge kernel, a programmatic
  // dependent of this one, may be scheduled from here on and waits for this grid itself. (Tree: the
  // kernel before is stage_queries_kernel, which began when everything before it had completed
  // and writes query images only; the warp that copies them waits for it.)
  if constexpr (PF != 3) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  if (trace && threadIdx.x == 0) trace[kTrWaited] = globaltimer_ns();

  if (!is_prefill(PF)) {
    // ---- split plan (decode/verify), computed by every CTA for itself. All sequences,
    // laid end to end on a cost axis (each as kUnitCost fixed units, then its 128-key
    // blocks), are cut into gridDim.x nearly equal contiguous ranges; this CTA owns
    // [x0, x1), one unit per sequence whose blocks the range overlaps. A long history thus
    // spreads over every SM ("Scaling Kimi K3 on AMD Instinct MI355X", section
    // "并行度必须适配真正的形状": hand the long history to more work groups), a batch of
    // short sequences stays one unit per sequence, a sequence is split only where a range
    // boundary falls inside it, and a CTA that crosses into another sequence takes fewer
    // blocks.
    const int B = p.B, tid = threadIdx.x;
    const int per = (B + C::kThreads - 1) / C::kThreads;  // sequences per thread, contiguous
    const int b_lo = min(B, tid * per), b_hi = min(B, b_lo + per);
    long long mine = 0;
#pragma unroll 1
    for (PlanIndex<PF> i(p, b_lo); i.b < b_hi; i.next(p)) {
      const int L = p.seq_lens[i.seq];
      const int64_t cap = p.pt_stride * (int64_t)p.page_size;
      if (L < 0 || (int64_t)L > cap) report(ms, MLA_ERR_BOUNDS);
      const int nb = blocks_of(seq_len_of(p, i.seq));
      mine += nb > 0 ? nb + kUnitCost : 0;
    }
    // exclusive prefix of the per-thread block counts over the CTA
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) ms->scan[warp] = (int)incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < C::kThreads / 32; ++w) {
      if (w < warp) before += ms->scan[w];
      total += ms->scan[w];
    }
    long long pre = before + incl - mine;
    long long x0, x1;
    {
      // range_lo's quotients by the reciprocal: exact, as c * total is below 2^64 / n (and less code
      // than 64-bit divisions, which a short call fetches cold; the same goes for the plan's loops not
      // being unrolled). A tree's ranges belong to teams of CTAs (tree_ranges).
      const unsigned c = PF == 3 ? blockIdx.x / p.team : blockIdx.x;
      const unsigned teams = PF == 3 ? gridDim.x / p.team : gridDim.x;
      const unsigned n = PF == 3 ? tree_ranges(total, teams) : teams;
      const unsigned long long inv = n == teams ? p.teams_inv : p.fewer_inv;
      x0 = (long long)__umul64hi(c * (unsigned long long)total, inv);
      x1 = inv ? (long long)__umul64hi((c + 1) * (unsigned long long)total, inv) : total;
      if (c >= n) x0 = x1 = total;  // a team without a range
    }
#pragma unroll 1
    for (PlanIndex<PF> i(p, b_lo); i.b < b_hi; i.next(p)) {
      const int nb = blocks_of(seq_len_of(p, i.seq));
      const long long first = pre + kUnitCost;  // the sequence's first block
      // the range's first unit: the sequence whose span holds x0, if the range reaches
      // one of its blocks
      if (nb > 0 && pre <= x0 && x0 < first + nb && first < x1 && x0 < x1) {
        ms->plan_b0 = i.b;
        ms->plan_pre0 = first;
        ms->plan_L0 = seq_len_of(p, i.seq);
        if constexpr (PF == 3) {
          ms->plan_seq0 = i.seq;
          ms->plan_pass0 = i.pass;
        }
      }
      if (nb > 0) pre = first + nb;
    }
    if (tid == 0) {
      ms->plan_x0 = x0;
      ms->plan_x1 = x1;
    }
    __syncthreads();
    if (trace && threadIdx.x == 0) trace[kTrPlanScan] = globaltimer_ns();
    // Ask L2 for the first unit's query rows and page-table entries before the first TMA
    // loads go out: behind the initial burst of key traffic they would arrive late, and
    // both are on the path to the first scores.
    if (warp >= 2 && ms->plan_b0 < B) {
      const int b0 = ms->plan_b0;
      if constexpr (PF != 3) {
        const int t = threadIdx.x - 64;
        const int qlines = args.rows * 9;  // 1,152 bytes per row
        if (t < qlines)
          prefetch_l2(reinterpret_cast<const uint8_t*>(
                          p.q + ((int64_t)b0 * p.R + ms->row_off[t / 9]) * kD) + (t % 9) * 128);
        // and the second unit's rows (its sequence follows b0) for the prologue's second pass
        const Cursor c1 = next_unit<PF>(args, first_unit<PF>(args, ms));
        if (t < qlines && has_unit<PF>(args, ms, c1))
          prefetch_l2(reinterpret_cast<const uint8_t*>(
                          p.q + ((int64_t)c1.b * p.R + ms->row_off[t / 9]) * kD) + (t % 9) * 128);
      }
      // four lines of 32 page-table entries, by the CTA's last four threads (past the
      // query lines: at most 48 rows x 9)
      const int64_t pg0 = (unsigned)(max(0ll, ms->plan_x0 - ms->plan_pre0) * kKeyBlock) / (unsigned)p.page_size;
      const int tp = (int)threadIdx.x - (C::kThreads - 4);
      const int64_t pg = pg0 + (int64_t)tp * 32;
      if (tp >= 0 && pg < p.pt_stride) prefetch_l2(p.page_table + (int64_t)(PF == 3 ? ms->plan_seq0 : b0) * p.pt_stride + pg);
    }
    __syncthreads();
    if (trace && threadIdx.x == 0) trace[kTrPlanPrefetch] = globaltimer_ns();
  }
  // Loads of one key tile into its stage (producer thread): the two 64-key halves' pool rows
  // from the page table, then the stage's parts, each once the MMAs of the tile that
  // held it have released it.
  const int64_t rows64 = p.num_pages * (int64_t)p.page_size;
  const int total_rows = rows64 > 0x7fffff00 ? 0x7fffff00 : (int)rows64;
  auto issue_tile = [&](const Issuer& by, const UnitInfo& un, int k0, uint32_t fill,
                        uint64_t policy) -> bool {
    const int s = fill % kStages;
    const uint32_t n = fill / kStages;
    uint8_t* st = smem + C::kOffStages + s * C::kStageStride;
    int y[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kk = k0 + 64 * h;
      y[h] = total_rows;  // fully out of range: TMA fills zeros
      if (kk < un.key_hi) {
        const int lp = kk / p.page_size;
        const int phys = p.page_table[(int64_t)un.b * p.pt_stride + lp];
        if (phys >= 0 && phys < p.num_pages)
          y[h] = phys * p.page_size + (kk % p.page_size);
        else
          report(ms, MLA_ERR_BOUNDS);
      }
      y[h] = (int)by.same((uint32_t)y[h]);
    }
#pragma unroll
    for (int c = 0; c < 5; ++c) {  // chunks 0..3, then the tail
      const int part = c < 4 ? part_of_chunk(c) : kTailPart;
      uint64_t* full = &ms->kv_full[s][part];
      if (c < 4 && part_begins(c)) {  // a part begins
        if (!by.same(wait_or_abort(&ms->kv_free[s][part], (n & 1) ^ 1, ms, p))) return false;
        if (by.leader) mbar_arrive_expect_tx(full, part_bytes(part));
      }
      if (c < 4) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          by.load(st + c * kChunkBytes + h * 8192, &map_main, c * 128, y[h], full, policy);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          by.load(st + C::kTail + h * 4096, &map_tail, 0, y[h], full, policy);
      }
    }
    return true;
  };
  // Decode reads each cached row once per launch: its lines should not push out of L2 what is
  // reused (code, query rows, page tables, the partials the merge reads next). (A call whose heads
  // run as two launches reads them twice, and marks them so in the first one too.) Prefill
  // re-reads the same rows for every unit and keeps the default policy, as a tree's verify does
  // for the groups of one sequence.
  const uint64_t read_once = (is_prefill(PF) || (PF == 3 && p.team * p.passes > 1)) ? l2_policy_evict_normal()
                                                                          : l2_policy_evict_first();
  if (trace && threadIdx.x == 0) trace[kTrPlanned] = globaltimer_ns();

  // The first unit's queries are on every CTA's critical path: warps 2.. stage them into
  // shared memory together (about two rows each). Later units' rows go to this CTA's query
  // image in global memory and reach shared memory in one bulk copy when their unit starts
  // (staging takes one warp far longer than a unit boundary may last): warps 2.. stage the
  // second unit there before the first key tile lands, the stager warp each later one while
  // the unit before it runs.
  if (PF != 3 && warp >= 2) {
    uint8_t* img = p.qimg + (int64_t)blockIdx.x * p.qimg_stride;
    Cursor cu = first_unit<PF>(args, ms);
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      while (has_unit<PF>(args, ms, cu) && tiles_in(unit_info<PF>(args, ms, cu)) == 0) cu = next_unit<PF>(args, cu);
      if (!has_unit<PF>(args, ms, cu)) break;
      const UnitInfo ui = unit_info<PF>(args, ms, cu);
      stage_rows<RP, C::kStageWarps>(p, ui.rows, ms->row_off, p.q + (int64_t)ui.qrow0 * kD, k == 0 ? qbuf : img,
                                     k == 0 ? ms->row_scale[0] : reinterpret_cast<float*>(img + C::kQBytes),
                                     warp - 2, lane);
      if (k == 0) {
        fence_proxy_async_smem();
        mbar_arrive(&ms->q0_done);
      } else {
        fence_proxy_async_global();
        mbar_arrive(&ms->q1_done);
      }
      cu = next_unit<PF>(args, cu);
    }
  }

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    const Issuer by;
    uint32_t fill = 0;  // tiles issued so far
    // L2 prefetch cursor: runs kPrefetchTiles tiles ahead of the TMA loads so that they
    // find their pages in L2 (deeper than the two shared-memory stages allow). The first
    // kStages tiles are the TMA loads' own: the cursor starts past them (no page-table
    // reads there: each is a round trip the second tile's load would wait behind).
    Cursor pf_c = first_unit<PF>(args, ms);
    UnitInfo pu = has_unit<PF>(args, ms, pf_c) ? unit_info<PF>(args, ms, pf_c) : UnitInfo{};
    int pf_k = pu.key_lo;
    uint32_t pf_tiles = 0;
    auto prefetch_upto = [&](uint32_t target, bool issue) {
      while (pf_tiles < target && has_unit<PF>(args, ms, pf_c)) {
        if (pf_k >= pu.key_hi) {  // unit done (or empty)
          pf_c = next_unit<PF>(args, pf_c);
          if (has_unit<PF>(args, ms, pf_c)) pu = unit_info<PF>(args, ms, pf_c);
          pf_k = pu.key_lo;
          continue;
        }
        for (int h = 0; h < 2 && issue; ++h) {
          const int kk = pf_k + 64 * h;
          if (kk < pu.key_hi) {
            const int phys = p.page_table[(int64_t)pu.b * p.pt_stride + kk / p.page_size];
            if (phys >= 0 && phys < p.num_pages) {
              const int rows = min(64, pu.key_hi - kk);
              if (by.leader) bulk_prefetch_l2(p.pool + ((int64_t)phys * p.page_size + kk % p.page_size) * kD,
                               (uint32_t)rows * kD);
            }
          }
        }
        ++pf_tiles;
        pf_k += kTileKeys;
      }
    };
    prefetch_upto(kStages, false);
    for (Cursor cu = first_unit<PF>(args, ms);
         by.same(has_unit<PF>(args, ms, cu) && !aborted(ms) && !p.test_stall);
         cu = next_unit<PF>(args, cu)) {
      const UnitInfo un = unit_info<PF>(args, ms, cu);
      const int key_hi = (int)by.same((uint32_t)un.key_hi);
      for (int k0 = (int)by.same((uint32_t)un.key_lo); k0 < key_hi; k0 += kTileKeys) {
        const bool ok = issue_tile(by, un, k0, fill, read_once);
        if (!ok) break;
        ++fill;
        prefetch_upto(fill + kPrefetchTiles, true);
      }
    }
    // Drain: wait (bounded) until the consumers released every part still holding a load.
    for (uint32_t f = (fill > kStages ? fill - kStages : 0); f < fill; ++f)
      for (int c = 0; c < kParts; ++c)
        mbar_wait(&ms->kv_free[f % kStages][c], (f / kStages) & 1, kWaitLimitNs);
  } else if (warp == 1) {
    // ------------------------------------------------------------------ scores issuer
    // QK of every tile, chunk by chunk as its KV stage fills, once its S^T buffer has been
    // read and its unit's query terms are staged. Values (PV) have their own issuing warp: a
    // single thread spends tens of cycles per tcgen05.mma, so one issuer would serialise the
    // two.
    const Issuer by;
    constexpr uint32_t idesc_qk = instr_desc(0, 0, 0, 0, 128, C::NQK);
    const uint64_t a_main0 = smem_desc(smem_addr(smem + C::kOffStages), 16, 1024, Swizzle::k128B);
    const uint64_t a_tail0 = smem_desc(smem_addr(smem + C::kOffStages + C::kTail), 16, 512, Swizzle::k64B);
    const uint64_t b_main0 = smem_desc(smem_addr(qbuf), 16, 1024, Swizzle::k128B);
    const uint64_t b_tail0 = smem_desc(smem_addr(qbuf + 4 * (C::NQK * 128)), 16, 512, Swizzle::k64B);
    uint32_t g = 0, units_done = 0;
    bool ok = true;
    for (Cursor cu = first_unit<PF>(args, ms); by.same(has_unit<PF>(args, ms, cu) && ok);
         cu = next_unit<PF>(args, cu)) {
      const int n = (int)by.same((uint32_t)tiles_in(unit_info<PF>(args, ms, cu)));
      if (n == 0) continue;
      const int qslot = units_done % C::kQB;
      if (!(ok = by.same(wait_or_abort(&ms->q_full[qslot], (units_done / C::kQB) & 1, ms, p)))) break;
      const uint32_t qoff = (uint32_t)(qslot * C::kQBytes) >> 4;
      for (int t = 0; t < n; ++t, ++g) {
        const int s = g % kStages, sb = g % C::kSBuf;
        const uint32_t ph = (g / kStages) & 1;
        if (!(ok = by.same(wait_or_abort(&ms->s_empty[sb], ((g / C::kSBuf) & 1) ^ 1, ms, p)))) break;
        const uint32_t soff = (uint32_t)(s * C::kStageStride) >> 4;
        const uint32_t d = by.same(tmem + C::kSCol + sb * C::NQK);
        const uint32_t am = by.place(a_main0, soff), at = by.place(a_tail0, soff);
        const uint32_t bm = by.place(b_main0, qoff), bt = by.place(b_tail0, qoff);
        // each latent chunk as soon as it has landed, then the RoPE tail
#pragma unroll
        for (int c = 0; c < 4 && ok; ++c) {
          if (part_begins(c)) {  // a part has landed
            if (!(ok = by.same(wait_or_abort(&ms->kv_full[s][part_of_chunk(c)], ph, ms, p)))) break;
            tc_fence_after();
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            by.mma(d, by.at(a_main0, am, (c * kChunkBytes + kk * 32) >> 4),
                   by.at(b_main0, bm, (c * (C::NQK * 128) + kk * 32) >> 4), idesc_qk, (c | kk) != 0);
        }
        if (!ok) break;  // the tail belongs to the last part, landed by now
#pragma unroll
        for (int kk = 0; kk < 2; ++kk)
          by.mma(d, by.at(a_tail0, at, (kk * 32) >> 4), by.at(b_tail0, bt, (kk * 32) >> 4), idesc_qk, 1);
        by.commit(&ms->s_full[sb]);
      }
      if (!ok) break;
      by.commit(&ms->q_empty[qslot]);  // that query buffer is free once these complete
      ++units_done;
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------------ values issuer
    // PV of every tile the moment its probabilities are in shared memory; completion hands
    // the KV stage back to the producer, part by part, and lets the softmax reuse P and
    // rescale O.
    const Issuer by;
    // A = V^T as e4m3 codes, B = P^T as e5m2 terms (kind::f8f6f4 takes each operand's
    // format from its own descriptor field), both MN-major
    constexpr uint32_t idesc_stacked = instr_desc(kFmtE4M3, kFmtE5M2, 1, 1, 128, 3 * RP);
    constexpr uint32_t idesc_term = instr_desc(kFmtE4M3, kFmtE5M2, 1, 1, 128, RP);
    const uint64_t a0 = smem_desc(smem_addr(smem + C::kOffStages), kChunkBytes, 1024, Swizzle::k128B);
    // P^T of stage 0's tile (at 48 rows; each stage has its own) or the shared buffer
    const uint64_t b0 = smem_desc(smem_addr(C::kPInStage ? smem + C::kOffStages + 4 * kChunkBytes : pbuf),
                                  128, 2048, Swizzle::kNone);
    uint32_t g = 0;
    bool ok = true;
    for (Cursor cu = first_unit<PF>(args, ms); by.same(has_unit<PF>(args, ms, cu) && ok);
         cu = next_unit<PF>(args, cu)) {
      const int n = (int)by.same((uint32_t)tiles_in(unit_info<PF>(args, ms, cu)));
      for (int t = 0; t < n; ++t, ++g) {
        if (!(ok = by.same(wait_or_abort(&ms->p_full[g & 1], (g >> 1) & 1, ms, p)))) break;
        tc_fence_after();
        const int s = g % kStages;
        const uint32_t soff = (uint32_t)(s * C::kStageStride) >> 4;
        const uint32_t poff = C::kPInStage ? soff : 0u;
        const uint32_t o = by.same(tmem), av = by.place(a0, soff), bp = by.place(b0, poff);
        // chunk by chunk (back-to-back MMAs into one accumulator cost no more than
        // alternating ones); each part of the stage is handed back once its MMAs complete.
        // The last part's release also stands for the whole tile's values being done
        // (P, which lives in the tail at 48 rows, and O for the softmax's rescale).
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t a = by.at(a0, av, (c * kChunkBytes + ks * 4096) >> 4);
            if (C::oterms(c) == 3) {  // stacked: one MMA over all three terms' rows (of a set)
#pragma unroll
              for (int set = 0; set < C::kSets; ++set)
                by.mma(o + C::ocol(c), a, by.at(b0, bp, (set * 3 * C::kPTerm + ks * 512) >> 4), idesc_stacked,
                       t > 0 || ks > 0 || set > 0);
            } else {  // summed: one MMA per term into the same accumulator
#pragma unroll
              for (int term = 0; term < 3; ++term)
                by.mma(o + C::ocol(c), a, by.at(b0, bp, (C::pterm(term) + ks * 512) >> 4), idesc_term,
                       t > 0 || ks > 0 || term > 0);
            }
          }
          if (part_ends(c)) by.commit(&ms->kv_free[s][part_of_chunk(c)]);
        }
      }
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------------ query stager
    // Each unit's query rows go into the query operand as two e4m3 terms with a per-row
    // power-of-two scale, as soon as the previous unit's scores stopped reading it; the
    // softmax warps meanwhile finish the previous unit.
    uint32_t k = 0;  // units with work, in order
    uint8_t* img = p.qimg + (int64_t)blockIdx.x * p.qimg_stride;
    constexpr uint32_t kImgBytes = C::kQBytes + 48 * sizeof(float);
    for (Cursor cu = first_unit<PF>(args, ms); has_unit<PF>(args, ms, cu); cu = next_unit<PF>(args, cu)) {
      const UnitInfo ui = unit_info<PF>(args, ms, cu);
      if (tiles_in(ui) == 0) continue;
      const int slot = k % C::kQB;
      const uint8_t* from = img;
      if constexpr (PF == 3) {  // staged by the kernel before: nothing but the copy
        from = p.qimg + (int64_t)ui.image * p.qimg_stride;
        if (k == 0) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          fence_proxy_async_global();
        }
      } else if (k == 0) {  // staged into shared memory by warps 2.. in the prologue
        if (!warp_waited(wait_or_abort(&ms->q0_done, 0, ms, p))) break;
        if (lane == 0) mbar_arrive(&ms->q_full[0]);
        ++k;
        continue;
      } else if (k == 1) {  // staged into the image by warps 2.. in the prologue
        if (!warp_waited(wait_or_abort(&ms->q1_done, 0, ms, p))) break;
      } else {
        // the image is free once the previous unit's copy out of it has landed
        const uint32_t pk = k - 1;
        if (!warp_waited(wait_or_abort(&ms->q_full[pk % C::kQB], (pk / C::kQB) & 1, ms, p))) break;
        stage_rows<RP, 1>(p, ui.rows, ms->row_off, p.q + (int64_t)ui.qrow0 * kD, img,
                          reinterpret_cast<float*>(img + C::kQBytes), 0, lane);
        fence_proxy_async_global();
        __syncwarp();
      }
      // The copy for unit k waits until the unit before in this buffer has its scores, and until the
      // softmax warps have seen that unit's copy and read its row scales: a unit of one tile may
      // have its scores done before its softmax has begun, and q_full would run two phases ahead of
      // those warps, which a parity cannot tell from none (and unit k or the one after it replaces
      // the scales). One barrier for both: a second one took verify 69.1 us to this one's 68.8.
      if (k >= (uint32_t)C::kQB && !warp_waited(wait_or_abort(&ms->q_empty[slot], ((k / C::kQB) - 1) & 1, ms, p)))
        break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&ms->q_full[slot], kImgBytes);
        bulk_g2s(qbuf + slot * C::kQBytes, from, C::kQBytes, &ms->q_full[slot]);
        bulk_g2s(ms->row_scale[k & 1], from + C::kQBytes, 48 * sizeof(float), &ms->q_full[slot]);
      }
      __syncwarp();
      ++k;
    }
  } else if (warp >= kSoftmaxWarp0) {
    // ------------------------------------------------------------------ softmax warpgroups
    // Two or three warpgroups, each owning an equal share of the query rows; thread i of a
    // warpgroup owns key i of the tile (its TMEM lane).
    constexpr int RH = C::kRH;
    constexpr float kHeadroom = kPScale + (PF == 3 || SC ? kTreeGap : kRescaleGap);
    const int wg = (warp - kSoftmaxWarp0) >> 2;
    const int rb = wg * RH;  // rows [rb, rb + RH)
    const int wq = warp & 3;  // TMEM lane quadrant
    const int i = wq * 32 + lane;
    const uint32_t lane_addr = (uint32_t)(wq * 32) << 16;
    const float kv_scale = p.kv_scale;
    uint32_t tile = 0, wg_phase = 0, k = 0;  // k: units with work, in order
    uint32_t moves = 0;  // times a running maximum of the warpgroup has moved
    // PV completions are confirmed in tile order, each before the PV two tiles later can
    // complete (that one needs this warpgroup's next P), so a phase parity names one tile
    // A wait that gives up does not make its lane leave on its own: `ok` collects the
    // outcome and the warp votes at fixed points (once a tile, before the epilogue), so a
    // timeout never splits a warp ahead of a warp-wide instruction (tcgen05.ld, __syncwarp).
    // After a failed wait the lanes run on to the vote on whatever they read; the call
    // reports MLA_ERR_TIMEOUT and its outputs are not to be used.
    // Arrivals are one per warp: the lanes meet at __syncwarp first (which also orders
    // their earlier memory accesses before lane 0's release).
    auto warp_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return wait_or_abort(bar, parity, ms, p);
    };
    auto warp_arrive = [&](uint64_t* bar) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    int pv_seen = -1;
    auto wait_pv_upto = [&](int target) -> bool {
      for (int g = pv_seen + 1; g <= target; ++g) {
        if (!warp_wait(&ms->kv_free[g % kStages][kTailPart], (g / kStages) & 1)) return false;
        pv_seen = g;
      }
      return true;
    };
    // Block scales: the scale of this thread's key of the next tile and the pool page of the one
    // after it are loaded while a tile is worked on.
    BlockScales bs;
    uint64_t* wg_bar = &ms->wg_bar[wg];
    // Bounded warpgroup barrier: every warp arrives, then waits for the phase.
    auto wg_sync = [&]() -> bool {
      warp_arrive(wg_bar);
      const bool good = warp_wait(wg_bar, wg_phase & 1);
      ++wg_phase;
      return good;
    };
    // Whether v holds for any thread of the warpgroup, by one hardware barrier instead of a vote
    // through shared memory and an mbarrier (draft trees: 4% of a call). It has no limit of its
    // own, and needs none: the warps of a warpgroup run the same units and tiles, every wait
    // between two of these barriers has a limit, and a warp whose wait gave up carries on to the
    // next barrier, from which all four leave together.
    auto wg_any = [&](bool v) -> bool {
      uint32_t any;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n"
          " barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(any)
          : "r"((uint32_t)v), "r"(1 + wg)
          : "memory");
      return any != 0;
    };
    bool ok = true;
    for (Cursor cu = first_unit<PF>(args, ms); has_unit<PF>(args, ms, cu) && ok; cu = next_unit<PF>(args, cu)) {
      const UnitInfo un = unit_info<PF>(args, ms, cu);
      const int R = un.rows;
      const int ntiles = tiles_in(un);
      const bool final_out = un.final_out != 0;
      if (ntiles == 0) {  // no visible key at all: out = 0, lse = -inf (or an empty partial)
        for (int r = rb; r < rb + RH && r < R; ++r) {
          if (final_out) {
            const int64_t row = (int64_t)un.qrow0 + ms->row_off[r];
            for (int dv = i; dv < kDV; dv += 128) store_out(p, row * kDV + dv, 0.f);
            if (i == 0 && p.lse) p.lse[row] = -INFINITY;
          } else if (i == 0) {
            p.part_lse[(int64_t)un.slot * p.part_rows + ms->row_off[r]] = -INFINITY;
          }
        }
        continue;
      }
      const int L = un.L;
      // last visible key of new position j is L - n_q + j + mask_shift (and the unit ends at
      // key_hi); mask_shift is 0 except for a shard that holds none of the new positions
      const int lim_cap = un.key_hi - 1;
      // (tree: the last key of the prefix, which every node sees; the nodes' own keys follow)
      const int lim0 = min(lim_cap, L - p.n_q + (PF == 3 ? -1 : un.j0 + p.mask_shift));
      if constexpr (SC) bs.begin(p, un.b, un.key_lo + i, un.key_hi);
      // this unit's row scales (staged with its query terms)
      ok &= warp_wait(&ms->q_full[k % C::kQB], (k / C::kQB) & 1);
      // mo: the row's running max less kPScale (p = 2^(x - mo)); kNoMax before its first key
      float rs[RH], mo[RH], l[RH];
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        rs[r] = ms->row_scale[k & 1][rb + r];
        mo[r] = kNoMax;
        l[r] = 0.f;
      }
      if (lane < RH) ms->row_max[moves & 1][rb + lane] = kNoMax;
      warp_arrive(&ms->q_empty[k % C::kQB]);
      for (int t = 0; t < ntiles; ++t, ++tile) {
        const int sb = tile % C::kSBuf;
        const int s = tile % kStages;
        const int k0 = un.key_lo + t * kTileKeys;
        const int kabs = k0 + i;
        KeyScale ks;
        if constexpr (SC) ks = bs.take(p, un.key_hi);
        ok &= warp_wait(&ms->s_full[sb], (tile / C::kSBuf) & 1);
        tc_fence_after();
        float x[RH];
        {
          const uint32_t base = tmem + lane_addr + C::kSCol + sb * C::NQK + rb;
          // every load of the tile first, one wait
          float a[RH], b2[RH];
#pragma unroll
          for (int c = 0; c < RH; c += 8) {
            tmem_ld8(base + c, *reinterpret_cast<float(*)[8]>(&a[c]));
            tmem_ld8(base + RP + c, *reinterpret_cast<float(*)[8]>(&b2[c]));
          }
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < RH; ++e) {
            x[e] = fmaf(b2[e], 1.0f / kQTerm2, a[e]);
            x[e] = SC ? fmaf(x[e] * ks.scale, rs[e], ks.log2) : x[e] * rs[e];
          }
        }
        tc_fence_before();
        warp_arrive(&ms->s_empty[sb]);
        if (trace && threadIdx.x == 32 * kSoftmaxWarp0 && t == 0) {
          if (tile == 0) trace[kTrFirstScores] = globaltimer_ns();
          if (k == 1) trace[kTrUnit2Scores] = globaltimer_ns();
        }
        // masking only on tiles that reach past the first new position's last visible key
        bool odd_key = false;  // tree: this thread's key may hold NaN codes, and not every row sees it
        if (k0 + kTileKeys - 1 > lim0) {
          if constexpr (PF == 3) {
            odd_key = x[0] != x[0];
            // this thread's key is node `node`'s: which of its rows see it, node by node of the
            // unit (a node is H neighbouring rows), from the half of each mask that holds its bit
            const int node = kabs - (L - p.n_q);
            uint32_t seen = node < 0 ? ~0u : 0u;
            if (node >= 0 && kabs < un.key_hi) {
              const uint32_t* half = reinterpret_cast<const uint32_t*>(p.tree_mask) +
                                     2 * ((int64_t)un.b * p.n_q + un.j0) + (node >> 5);
              const int end = min(rb + RH, R);
#pragma unroll 1
              for (int j = rb / p.H; j * p.H < end; ++j)
                if (half[2 * j] >> (node & 31) & 1u)
                  seen |= ((1u << min(RH, (j + 1) * p.H - rb)) - 1u) & (~0u << max(0, j * p.H - rb));
            }
#pragma unroll
            for (int r = 0; r < RH; ++r)
              if (!(seen >> r & 1u)) x[r] = -INFINITY;
          } else {
#pragma unroll
            for (int r = 0; r < RH; ++r) {
              const int lim = min(lim_cap, lim0 + ms->row_j[rb + r]);
              if (kabs > lim) x[r] = -INFINITY;
            }
          }
        }
        // The running max of a row moves only when some score exceeds it by more than the
        // headroom (in log2 units); only then is the exact tile max needed. The warps of the
        // warpgroup first agree whether that happens anywhere, and the common case skips the
        // exchange of per-row maxima.
        bool over = false;
#pragma unroll
        for (int r = 0; r < RH; ++r) over |= (x[r] > mo[r] + kHeadroom);
        bool need_rescale = false;
        if (wg_any(over || !ok)) {
          if (wg_any(!ok)) {  // the warpgroup's once-a-tile vote on its waits
            ok = false;
            break;
          }
          // The tile's maximum of each row: a warp's in hardware, then the four warps' through shared
          // memory, a lane a row. The running maxima are read from the side that the time before wrote
          // and written to the other (each warp of the warpgroup the same values).
          float* red = &ms->red[tile & 1][0];
          float v = 0.f;
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            const float w = warp_max(x[r]);
            if (lane == r) v = w;
          }
          if (lane < RH) red[(rb + lane) * 4 + wq] = v;
          ok &= wg_sync();
          bool moved = false;
          if (lane < RH) {
            const float4 t4 = *reinterpret_cast<const float4*>(&red[(rb + lane) * 4]);
            const float tm = fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
            float now = ms->row_max[moves & 1][rb + lane], al = 1.f;
            if (tm > now + kHeadroom) {  // lazy: the headroom absorbs small increases
              al = ex2(now + kPScale - tm);  // 0 before the first key (nothing accumulated yet)
              moved = now != kNoMax;
              now = tm - kPScale;
            }
            ms->row_max[(moves & 1) ^ 1][rb + lane] = now;
            ms->alpha[rb + lane] = al;
          }
          need_rescale = __any_sync(0xffffffffu, moved);
          __syncwarp();
          ++moves;
#pragma unroll
          for (int r = 0; r < RH; ++r) {
            mo[r] = ms->row_max[moves & 1][rb + r];
            l[r] *= ms->alpha[rb + r];
          }
        }
        // p = 2^(x - m + 11) <= 2^15 rounded to fp16, then three e5m2 terms, each the
        // nearest e5m2 value to what the terms before it left (the differences are exact
        // in fp16); the row sum takes the float32 p. FINE: six terms of the float32 p, each within 2^-3 of
        // what the terms before it left, so p to 2^-18 (and no closer than 2^-17, 2^-33 of the largest).
        uint32_t w1[RH / 4], w2[RH / 4], w3[RH / 4];
#pragma unroll
        for (int r = 0; r < RH; r += 2) {
          const float p0 = ex2(x[r] - mo[r]);  // masked (x = -inf) and keyless rows give 0
          const float p1 = ex2(x[r + 1] - mo[r + 1]);
          l[r] = SC ? fmaf(p0, ks.inv, l[r]) : l[r] + p0;
          l[r + 1] = SC ? fmaf(p1, ks.inv, l[r + 1]) : l[r + 1] + p1;
          if constexpr (FINE) {  // (its terms go out one by one, below)
            x[r] = p0;
            x[r + 1] = p1;
            continue;
          }
          const uint32_t h = f32x2_to_f16x2(p0, p1);
          const uint32_t c1 = f16x2_to_e5m2x2(h);
          const uint32_t r1 = hsub2(h, e5m2x2_to_f16x2(c1));
          const uint32_t c2 = f16x2_to_e5m2x2(r1);
          const uint32_t r2 = hsub2(r1, e5m2x2_to_f16x2(c2));
          const uint32_t c3 = f16x2_to_e5m2x2(r2);
          const int wi = r >> 2;
          if ((r & 2) == 0) {
            w1[wi] = c1;
            w2[wi] = c2;
            w3[wi] = c3;
          } else {
            w1[wi] |= c1 << 16;
            w2[wi] |= c2 << 16;
            w3[wi] |= c3 << 16;
          }
        }
        // The previous tile's PV must be done before O is rescaled, and before P is written
        // when one P buffer serves every tile. With P in the stage, PV(tile - 2) is known
        // done (this tile's keys replaced its stage) and is only confirmed here.
        {
          const int upto = (int)tile - ((C::kPInStage && !need_rescale) ? 2 : 1);
          ok &= wait_pv_upto(upto);
          tc_fence_after();
        }
        if (t > 0 && need_rescale) {
          // (one small loop over the pieces of O; its code is fetched cold when a short call first
          // needs it)
          __syncwarp();
          const float* al = &ms->alpha[rb];
#pragma unroll 1
          for (int part = 0; part < C::kOParts; ++part) {
            const uint32_t a = tmem + lane_addr + C::kOCol + part * RP + rb;
            float v[RH];
#pragma unroll
            for (int cc = 0; cc < RH; cc += 8) tmem_ld8(a + cc, *reinterpret_cast<float(*)[8]>(&v[cc]));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < RH; ++e) v[e] *= al[e];
#pragma unroll
            for (int cc = 0; cc < RH; cc += 8) tmem_st8(a + cc, *reinterpret_cast<float(*)[8]>(&v[cc]));
          }
          tmem_wait_st();
        }
        // keys past this unit's range: zero their V bytes so 0 * garbage cannot be NaN
        if (wg == 0 && kabs >= un.key_hi) {
          uint8_t* st = smem + C::kOffStages + s * C::kStageStride + (i >> 6) * 8192 + (i & 63) * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4*>(st + c * kChunkBytes)[e] = make_uint4(0, 0, 0, 0);
        } else if (PF == 3 && wg == 0 && odd_key) {
          // Tree: a node's key is hidden from some rows (P = 0) and seen by others. NaN codes among
          // its values would reach them all as 0 * NaN, so they are zeroed: a row that sees the key
          // has NaN from its score, whose product holds the same codes. That score is also how they
          // are found (NaN for every query, the unit's first one too).
          uint8_t* st = smem + C::kOffStages + s * C::kStageStride + (i >> 6) * 8192 + (i & 63) * 128;
#pragma unroll 1
          for (int e = 0; e < 32; ++e) {
            uint4* at = reinterpret_cast<uint4*>(st + (e >> 3) * kChunkBytes) + (e & 7);
            const uint4 v = *at;
            *at = make_uint4(without_nan(v.x), without_nan(v.y), without_nan(v.z), without_nan(v.w));
          }
        }
        // P^T: MN-major, 16 rows x 8 keys core matrices; term t, row group g at
        // pterm(t) + g * 2048, key i at (i / 8) * 128 + (i % 8) * 16, row r at byte r % 16.
        // A warpgroup with 16 rows (a whole row group) writes each key's 16 bytes at once: a
        // warp then stores 512 contiguous bytes, free of bank conflicts (8-byte halves at a
        // 16-byte stride took four shared-memory wavefronts a store where two suffice). With
        // 8 rows it writes its 8-byte half.
        uint8_t* pb = C::kPInStage ? smem + C::kOffStages + s * C::kStageStride + 4 * kChunkBytes : pbuf;
        const int off = (i >> 3) * 128 + (i & 7) * 16;
        if constexpr (FINE) {
          const int o = (rb >> 4) * 2048 + off + ((rb & 15) >> 3) * 8;
#pragma unroll 1
          for (int term = 0; term < 3 * C::kSets; ++term) {
            uint32_t w[RH / 4];
#pragma unroll
            for (int r = 0; r < RH; r += 2) {
              const uint32_t c = to_e5m2x2(x[r], x[r + 1]);
              const float2 b = from_e5m2x2(c);
              x[r] -= b.x;
              x[r + 1] -= b.y;
              w[r >> 2] = (r & 2) == 0 ? c : w[r >> 2] | c << 16;
            }
            if constexpr (RH == 16)
              *reinterpret_cast<uint4*>(pb + C::pterm(term) + o) = make_uint4(w[0], w[1], w[2], w[3]);
            else
              *reinterpret_cast<uint2*>(pb + C::pterm(term) + o) = make_uint2(w[0], w[1]);
          }
        } else if constexpr (RH % 16 == 0) {
#pragma unroll
          for (int blk = 0; blk < RH / 16; ++blk) {
            const int o = ((rb >> 4) + blk) * 2048 + off;
            *reinterpret_cast<uint4*>(pb + C::pterm(0) + o) =
                make_uint4(w1[4 * blk], w1[4 * blk + 1], w1[4 * blk + 2], w1[4 * blk + 3]);
            *reinterpret_cast<uint4*>(pb + C::pterm(1) + o) =
                make_uint4(w2[4 * blk], w2[4 * blk + 1], w2[4 * blk + 2], w2[4 * blk + 3]);
            *reinterpret_cast<uint4*>(pb + C::pterm(2) + o) =
                make_uint4(w3[4 * blk], w3[4 * blk + 1], w3[4 * blk + 2], w3[4 * blk + 3]);
          }
        } else {
#pragma unroll
          for (int blk = 0; blk < RH / 8; ++blk) {
            const int row0 = rb + 8 * blk;
            const int o = (row0 >> 4) * 2048 + off + ((row0 & 15) >> 3) * 8;
            *reinterpret_cast<uint2*>(pb + C::pterm(0) + o) = make_uint2(w1[2 * blk], w1[2 * blk + 1]);
            *reinterpret_cast<uint2*>(pb + C::pterm(1) + o) = make_uint2(w2[2 * blk], w2[2 * blk + 1]);
            *reinterpret_cast<uint2*>(pb + C::pterm(2) + o) = make_uint2(w3[2 * blk], w3[2 * blk + 1]);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&ms->p_full[tile & 1]);
      }
      if (trace && threadIdx.x == 32 * kSoftmaxWarp0) trace[kTrLastP] = globaltimer_ns();
      // ---- epilogue: row sums, then O / l
      if constexpr (PF == 3 || SC) {
        // all rows at once: each exchange halves the rows that a lane still adds up
        float s[RH];
#pragma unroll
        for (int r = 0; r < RH; ++r) s[r] = l[r];
        int row = 0, width = 16;
#pragma unroll
        for (int h = RH / 2; h > 0; h >>= 1, width >>= 1) {
          const bool up = lane & width;
#pragma unroll
          for (int r = 0; r < h; ++r) {
            const float give = up ? s[r] : s[r + h], keep = up ? s[r + h] : s[r];
            s[r] = keep + __shfl_xor_sync(0xffffffffu, give, width);
          }
          row += up ? h : 0;
        }
        for (; width > 0; width >>= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], width);
        ms->lred[wq][rb + row] = s[0];  // (two or four lanes the same)
      } else {
#pragma unroll
        for (int r = 0; r < RH; ++r) {
          float v = l[r];
          for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) ms->lred[wq][rb + r] = v;
        }
      }
      ok &= wg_sync();
      float inv[RH];
#pragma unroll
      for (int r = 0; r < RH; ++r) {
        const int rr = rb + r;
        const float lt = ms->lred[0][rr] + ms->lred[1][rr] + ms->lred[2][rr] + ms->lred[3][rr];
        l[r] = lt;
        inv[r] = lt == 0.f ? 0.f : kv_scale / lt;  // (a row that saw a NaN: its sum is NaN, so is it)
      }
      ok &= wait_pv_upto((int)tile - 1);
      if (wg_any(!ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (trace && threadIdx.x == 32 * kSoftmaxWarp0) trace[kTrLastPV] = globaltimer_ns();
      // One small loop (the rows' reciprocals in shared memory, not in registers that only unrolled
      // code can index): a short call fetches the epilogue's code cold. Two passes at once where a thread
      // has 16 rows (in us, one / two: verify 8 x 4 on 32K 52.9 / 51.9, 1 x 4 on 1K 17.5 / 17.0; with 8 rows
      // decode 512 x 100-300 50.2 / 50.8, trees 132.8 / 133.7).
      __syncwarp();
#pragma unroll
      for (int r = 0; r < RH; ++r)
        if (lane == 0) ms->alpha[rb + r] = inv[r];  // (every warp of the warpgroup the same)
      __syncwarp();
#pragma unroll(RP == 48 && PF != 3 ? 2 : 1)
      for (int u = 0; u < 4 * (RH / 8); ++u) {
        const int c = u / (RH / 8), row = rb + u % (RH / 8) * 8;
        if (row >= R) continue;
        const uint32_t a = tmem + lane_addr + C::ocol(c) + row;
        // The rows' output offsets go to registers before any of these stores: as far as the
        // compiler knows a store may alias the table, so a lookup between two stores would wait for
        // the first one to drain (about 60 ns a store when every SM writes).
        int roff[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) roff[e] = PF == 3 ? row + e : ms->row_off[row + e];
        float o[8];
        tmem_ld8(a, o);
        if (C::oterms(c) == 3) {
          float o1[8], o2[8];
          tmem_ld8(a + RP, o1);
          tmem_ld8(a + 2 * RP, o2);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = PF == 3 || SC ? o[e] + (o1[e] + o2[e]) : o[e] + o1[e] + o2[e];
        } else {
          tmem_wait_ld();
        }
        const int dv = c * 128 + i;
        const float* scale = &ms->alpha[row];
        if (final_out) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row + e < R) store_out(p, ((int64_t)un.qrow0 + roff[e]) * kDV + dv, o[e] * scale[e]);
        } else {
          float* dst = p.part_out + (int64_t)un.slot * p.part_rows * kDV + dv;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (row + e < R) dst[(int64_t)roff[e] * kDV] = o[e] * scale[e];
        }
      }
      tc_fence_before();
      if (i < RH && rb + i < R) {
        float lt = 0.f, mm = kNoMax;
#pragma unroll
        for (int r = 0; r < RH; ++r)
          if (r == i) {
            lt = l[r];
            mm = mo[r];
          }
        const float lse = (lt == 0.f) ? -INFINITY : 0.6931471805599453f * (mm + log2f(lt));
        const int roff = ms->row_off[rb + i];
        if (final_out) {
          if (p.lse) p.lse[(int64_t)un.qrow0 + roff] = lse;
        } else {
          p.part_lse[(int64_t)un.slot * p.part_rows + roff] = lse;
        }
      }
      ++k;
      if (trace && threadIdx.x == 32 * kSoftmaxWarp0) {
        trace[kTrEpilogue] = globaltimer_ns();
        trace[kTrCounts] = ((unsigned long long)tile << 32) | k;
        if (k == 1) trace[kTrUnit1End] = globaltimer_ns();
      }
    }
  }

  // (tree: a CTA without units has not waited yet, and this grid must not complete before the one
  // in front of it)
  if constexpr (PF == 3) asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
  if (trace && threadIdx.x == 0) trace[kTrExit] = globaltimer_ns();
  if (threadIdx.x == 0) {
    // this CTA's status word (a later launch of the same call only adds errors)
    if (args.status_overwrite || ms->status != 0) p.status[blockIdx.x] = ms->status;
    if (blockIdx.x == 0 && args.status_overwrite) p.hdr->num_ctas = gridDim.x;
  }
}

// Tree verify: every group's query image, one CTA a group. The attention kernel, a programmatic
// dependent, plans and loads its first keys meanwhile. (Staged by the attention kernel itself, as
// decode does: 77 KB of its code, fetched cold on the way to the first scores, and one warp for a
// CTA's later units, 28 us each: 64 sequences of 64 nodes of 16 heads on 100 to 130 keys took
// 305 us, 175 us this way; 8 nodes of 12 heads on 1,024 keys 22.1 and 20.3 us.)
// Bound: one round of loads and cold code (32 groups of 48 rows 6.9 us alone with cold caches,
// behind which the attention kernel's start hides most).
template <int RP>
__global__ void __launch_bounds__(512) stage_queries_kernel(const __grid_constant__ AttnParams p) {
  __shared__ int row_off[48];
  if (threadIdx.x < 48) row_off[threadIdx.x] = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;");
  __syncthreads();
  const int groups = p.team * p.passes;
  const int node0 = (int)(blockIdx.x % groups) * p.group_nodes;
  const int64_t row0 = ((int64_t)(blockIdx.x / groups) * p.n_q + node0) * p.H;
  uint8_t* img = p.qimg + (int64_t)blockIdx.x * p.qimg_stride;
  stage_rows<RP, 16, true>(p, min(p.group_nodes, p.n_q - node0) * p.H, row_off, p.q + row0 * kD, img,
                           reinterpret_cast<float*>(img + Cfg<RP>::kQBytes), threadIdx.x >> 5, threadIdx.x & 31);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, looked up through the runtime so the library needs no link-time
// dependency on the driver library.
EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
    else
      cudaGetLastError();
  }
  return fn;
}

bool encode_pool_maps(const AttnParams& p, CUtensorMap* main_map, CUtensorMap* tail_map) {
  const EncodeTiledFn encode = encode_fn();
  if (!encode) return false;
  const uint64_t rows = (uint64_t)p.num_pages * (uint64_t)p.page_size;
  if (rows == 0 || rows > 0x7fffff00ull) return false;
  cuuint64_t dims_main[2] = {512, rows};
  cuuint64_t dims_tail[2] = {64, rows};
  cuuint64_t strides[1] = {(cuuint64_t)kD};
  cuuint32_t box_main[2] = {128, 64};
  cuuint32_t box_tail[2] = {64, 64};
  cuuint32_t estr[2] = {1, 1};
  CUresult r1 = encode(main_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                                       const_cast<uint8_t*>(p.pool), dims_main, strides, box_main,
                                       estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                       CU_TENSOR_MAP_SWIZZLE_128B,
                                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  CUresult r2 = encode(tail_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                                       const_cast<uint8_t*>(p.pool + 512), dims_tail, strides,
                                       box_tail, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                       CU_TENSOR_MAP_SWIZZLE_64B,
                                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r1 == CUDA_SUCCESS && r2 == CUDA_SUCCESS;
}

template <int RP, int PF, bool TR, bool SC, bool FINE = false>
cudaError_t launch_rp_tr(const DecodeArgs& a, const CUtensorMap& mm, const CUtensorMap& mt,
                         int grid, cudaStream_t s) {
  constexpr int smem = smem_bytes<RP, FINE>();
  auto* kernel = attn_tc_kernel<RP, PF, TR, SC, FINE>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Cfg<RP>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, mm, mt);
}

template <int RP, int PF, bool SC, bool FINE = false>
cudaError_t launch_rp_sc(const DecodeArgs& a, const CUtensorMap& mm, const CUtensorMap& mt,
                         int grid, cudaStream_t s) {
  if constexpr (PF >= 2) {  // (never traced)
    return launch_rp_tr<RP, PF, false, SC, FINE>(a, mm, mt, grid, s);
  } else {
    return a.p.trace ? launch_rp_tr<RP, PF, true, SC, FINE>(a, mm, mt, grid, s)
                     : launch_rp_tr<RP, PF, false, SC, FINE>(a, mm, mt, grid, s);
  }
}

template <int RP, int PF>
cudaError_t launch_rp(const DecodeArgs& a, const CUtensorMap& mm, const CUtensorMap& mt,
                      int grid, cudaStream_t s) {
  return a.p.scales ? launch_rp_sc<RP, PF, true>(a, mm, mt, grid, s)
                    : launch_rp_sc<RP, PF, false>(a, mm, mt, grid, s);
}

}  // namespace

// Decode / verify attention for every unit of the plan. Rows per launch are limited to 48
// (three query terms of 48 rows fit TMEM); 16 heads x 4 positions run as two head halves.
cudaError_t launch_decode_tc(const AttnParams& p, int num_sms, cudaStream_t s, int* launches) {
  CUtensorMap mm, mt;
  if (!encode_pool_maps(p, &mm, &mt)) return cudaErrorInvalidValue;
  const int grid = p.num_ctas;  // the split plan cuts the blocks into this many ranges
  (void)num_sms;
  // A float32 output under block scales carries its probabilities in six terms (FINE), for which units
  // of 48 rows have no room.
  const bool fine = p.scales && p.out_f32;
  const int groups = (p.R > (fine ? 32 : 48)) ? 2 : 1;
  for (int gi = 0; gi < groups; ++gi) {
    DecodeArgs a;
    a.p = p;
    a.Hs = p.H / groups;
    a.h0 = gi * a.Hs;
    if (gi == groups - 1) a.Hs = p.H - a.h0;
    a.rows = p.n_q * a.Hs;
    a.prefill = 0;
    a.P = 0;
    a.num_units = 0;
    a.unit_end = 0;
    a.split_base = 0;
    a.status_overwrite = (gi == 0);
    cudaError_t e;
    if (fine)
      e = a.rows <= 16 ? launch_rp_sc<16, 0, true, true>(a, mm, mt, grid, s)
                       : launch_rp_sc<32, 0, true, true>(a, mm, mt, grid, s);
    else if (a.rows <= 16)
      e = launch_rp<16, 0>(a, mm, mt, grid, s);
    else if (a.rows <= 32)
      e = launch_rp<32, 0>(a, mm, mt, grid, s);
    else
      e = launch_rp<48, 0>(a, mm, mt, grid, s);
    if (e != cudaSuccess) return e;
    ++*launches;
  }
  return cudaSuccess;
}

// Tree verify: the split plan over the passes of every sequence's groups of nodes (p.B passes in
// all, groups of at most 48 rows; mla_internal.cuh, tree_plan).
cudaError_t launch_tree_tc(const AttnParams& p, cudaStream_t s, int* launches) {
  CUtensorMap mm, mt;
  if (!encode_pool_maps(p, &mm, &mt)) return cudaErrorInvalidValue;
  DecodeArgs a = {};
  a.p = p;
  a.Hs = p.H;
  a.rows = p.R;
  a.status_overwrite = 1;
  cudaError_t e;
  const unsigned units = (unsigned)(p.B * p.team);  // (passes x team groups a sequence)
  auto* stage = a.rows <= 16 ? stage_queries_kernel<16>
                             : (a.rows <= 32 ? stage_queries_kernel<32> : stage_queries_kernel<48>);
  stage<<<units, 512, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  ++*launches;
  if (a.rows <= 16)
    e = launch_rp<16, 3>(a, mm, mt, p.num_ctas, s);
  else if (a.rows <= 32)
    e = launch_rp<32, 3>(a, mm, mt, p.num_ctas, s);
  else
    e = launch_rp<48, 3>(a, mm, mt, p.num_ctas, s);
  if (e == cudaSuccess) ++*launches;
  return e;
}

// Causal prefill of one sequence: units are blocks of P = 48 / H new positions (all their
// heads, at most 48 rows) over every key they see, handed out longest first, one a round
// per CTA. A last round that would leave CTAs idle runs instead as a second launch over
// the halves of its units (keys split in two), and a merge kernel joins the halves.
cudaError_t launch_prefill_tc(const AttnParams& p, int num_sms, cudaStream_t s, int* launches) {
  CUtensorMap mm, mt;
  if (!encode_pool_maps(p, &mm, &mt)) return cudaErrorInvalidValue;
  DecodeArgs a;
  a.p = p;
  a.h0 = 0;
  a.Hs = p.H;
  a.P = 48 / p.H;
  a.rows = a.P * p.H;
  a.prefill = 1;
  a.status_overwrite = 1;
  a.num_units = (p.n_q + a.P - 1) / a.P;
  const int grid = min(num_sms, a.num_units);
  const int left = a.num_units % grid;  // units of an incomplete last round
  const bool split = left > 0 && 2 * left <= grid;
  a.split_base = a.num_units - left;
  a.unit_end = split ? a.split_base : a.num_units;
  cudaError_t e = launch_rp<48, 1>(a, mm, mt, grid, s);
  if (e != cudaSuccess) return e;
  ++*launches;
  if (!split) return cudaSuccess;
  DecodeArgs b = a;
  b.unit_end = 2 * left;  // halves: one a CTA
  b.status_overwrite = 0;
  b.p.trace = nullptr;    // the profiling hook traces the main launch
  if ((e = launch_rp<48, 2>(b, mm, mt, 2 * left, s)) != cudaSuccess) return e;
  ++*launches;
  if ((e = launch_merge_prefill(p, a.P, left, s)) != cudaSuccess) return e;
  ++*launches;
  return cudaSuccess;
}

}  // namespace mla
