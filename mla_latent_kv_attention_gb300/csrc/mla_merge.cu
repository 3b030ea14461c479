// mla_merge.cu -- the log-sum-exp merge of split-KV partial results.
//
// Per query row, lse = ln sum_s exp(lse_s) and out = sum_s exp(lse_s - lse) out_s, the
// "merge by normalisation statistics" of position-sharded attention ("Scaling Kimi K3 on
// AMD Instinct MI355X", section "缓存可复用，还要能一致地恢复").
//
// Where the partials come from: the attention kernel lays all sequences end to end on a
// cost axis (a fixed cost per sequence, then its 128-key blocks) and cuts it into one
// contiguous range per CTA; a sequence is split only where a range boundary falls inside
// its blocks, so its pieces sit on consecutive CTAs, and only the first and the last unit
// of a CTA's range can hold part of a sequence. Partial slot 2c is the piece that is CTA
// c's first unit, slot 2c + 1 the piece that ends its range after an earlier sequence.
#include <cuda_bf16.h>
#include <math.h>

#include "mla_internal.cuh"

namespace mla {

namespace {

constexpr int kMergeWarps = 8;
constexpr int kMergeThreads = 32 * kMergeWarps;


// Merge one dv chunk (32 * VEC values; lane l owns VEC consecutive ones) of one row from
// `count` partials; slot_of(i) gives the partial index of piece i, whose row sits at
// po[(slot * R + r) * 512] and pl[slot * R + r]. Latency sets the cost (the partials were
// written by the kernel just before), so everything is loaded in one round: each lane the
// lse values it reduces (every warp reduces them all, no barrier) and warp w's pieces
// w, w + 8, ..., with their own lse values for the weights; only pieces past the first
// batch, or lse values past 256, take further rounds. The warps' sums meet in shared memory.
__device__ __forceinline__ void store_val(uint16_t* p, float v) {
  *p = __bfloat16_as_ushort(__float2bfloat16_rn(v));
}
__device__ __forceinline__ void store_val(float* p, float v) { *p = v; }

// WPR: warps on one row (kMergeWarps / WPR rows a CTA, each its own group of warps with its
// own named barrier, so one group may leave early without the other).
template <int VEC, int WPR, typename OutT, typename SlotOf>
__device__ void merge_row_chunk(const float* __restrict__ po, const float* __restrict__ pl,
                                int count, SlotOf slot_of, int64_t r, int64_t R, int chunk,
                                OutT* __restrict__ out_row, float* lse_out) {
  constexpr int W = 32 * VEC;                             // dv per CTA
  constexpr int NB = VEC >= 16 ? 2 : (VEC >= 4 ? 8 : 24);  // pieces per batch and warp
  constexpr int kLse = 8;                                 // lse values per lane (256 pieces)
  constexpr int kGroupThreads = 32 * WPR;
  __shared__ __align__(16) float s_acc[kMergeWarps][W];
  const int lane = threadIdx.x & 31, gw = threadIdx.x >> 5;
  const int g = gw / WPR, warp = gw % WPR;  // row group, warp within it
  const int gt = threadIdx.x - g * kGroupThreads;
  if (count <= 0) {  // nothing to merge: out = 0, lse = -inf
    for (int x = gt; x < W; x += kGroupThreads) store_val(out_row + chunk * W + x, 0.f);
    if (gt == 0 && chunk == 0 && lse_out) *lse_out = -INFINITY;
    return;
  }
  // load the pieces i0 + k * WPR (k < NB) of this warp: weights' lse values and data. Lane k looks up
  // piece k's slot (a lookup may divide), the warp takes it from there; pieces past the end weigh 0 and
  // are not loaded.
  float v[NB][VEC];
  float w[NB];
  auto load_batch = [&](int i0) {
    const int slot = (int)slot_of(min(i0 + lane * WPR, count - 1));
    int64_t at[NB];
#pragma unroll
    for (int k = 0; k < NB; ++k) at[k] = __shfl_sync(0xffffffffu, slot, k) * R + r;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      w[k] = -INFINITY;
      if (i0 + k * WPR >= count) continue;
      w[k] = __ldg(pl + at[k]);
      const float* src = po + at[k] * kDV + chunk * W + lane * VEC;
      if constexpr (VEC % 4 == 0) {
#pragma unroll
        for (int e = 0; e < VEC; e += 4) {
          const float4 t = __ldg(reinterpret_cast<const float4*>(src + e));
          v[k][e] = t.x;
          v[k][e + 1] = t.y;
          v[k][e + 2] = t.z;
          v[k][e + 3] = t.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[k][e] = __ldg(src + e);
      }
    }
  };
  // round one: this lane's share of the lse values, and the warp's first batch
  float lv[kLse];
#pragma unroll
  for (int j = 0; j < kLse; ++j) {
    lv[j] = -INFINITY;
    if (32 * j < count) lv[j] = __ldg(pl + slot_of(min(lane + 32 * j, count - 1)) * R + r);
  }
  load_batch(warp);
  // lse = max + ln sum exp(lse_i - max)
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < kLse; ++j) {
    if (lane + 32 * j >= count) lv[j] = -INFINITY;
    m = fmaxf(m, lv[j]);
  }
  float sum = 0.f;
  for (int i = lane + 32 * kLse; i < count; i += 32) {  // online, past 256 pieces
    const float x = __ldg(pl + slot_of(i) * R + r);
    if (x == -INFINITY) continue;  // an empty partial adds nothing (and -inf - -inf is NaN)
    if (x > m) {
      sum = sum * expf(m - x);
      m = x;
    }
    sum += expf(x - m);
  }
  float mw = m;
  for (int o = 16; o > 0; o >>= 1) mw = fmaxf(mw, __shfl_xor_sync(0xffffffffu, mw, o));
  if (m != -INFINITY) sum *= expf(m - mw);  // (else 0, or NaN past 256 pieces)
#pragma unroll
  for (int j = 0; j < kLse; ++j)
    if (lv[j] != -INFINITY) sum += expf(lv[j] - mw);
  m = mw;
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  // a NaN piece, which the maxima pass over, makes the sum NaN, and so the row
  const bool none = m == -INFINITY && sum == 0.f;
  const float lse = none ? -INFINITY : m + logf(sum);
  float acc[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
  if (!none) {
    for (int i0 = warp;;) {
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        // an empty partial (lse = -inf) has weight 0; whatever its data holds is skipped
        if (w[k] == -INFINITY) continue;
        const float wk = expf(w[k] - lse);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] += wk * v[k][e];
      }
      i0 += NB * WPR;
      if (i0 >= count) break;
      load_batch(i0);
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) s_acc[gw][lane * VEC + e] = acc[e];
  // the row group's warps meet (barrier 1 + g, its threads only)
  asm volatile("bar.sync %0, %1;" ::"r"(1 + g), "r"(kGroupThreads) : "memory");
  // every thread finishes W / kGroupThreads (or one) of the chunk's outputs
  for (int x = gt; x < W; x += kGroupThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < WPR; ++k) t += s_acc[g * WPR + k][x];
    store_val(out_row + chunk * W + x, t);
  }
  if (gt == 0 && chunk == 0 && lse_out) *lse_out = lse;
}

// Blocks of sequence b on the split plan's cost axis: its length clamped to what its
// page-table row can address, as the attention kernel plans it (which also reports a
// length out of range).
__device__ __forceinline__ int plan_blocks(const AttnParams& p, int b) {
  int L = __ldg(p.seq_lens + b);
  const int64_t cap = p.pt_stride * (int64_t)p.page_size;
  if (L < 0) L = 0;
  if ((int64_t)L > cap) L = (int)cap;
  return (L + kKeyBlock - 1) / kKeyBlock;
}

// Rows of the decode/verify path whose sequence was split over several CTAs, and rows of
// sequences with no key at all (out = 0, lse = -inf). Launched as a programmatic dependent
// of the attention kernel. Before waiting for that grid it works out, from the lengths
// alone, where each of its rows' pieces sit: the lengths are inputs of the call, complete
// before the attention kernel passed its own wait on the kernels before it, and only then
// could this grid start. So after the wait the partials are loaded at once, and rows with
// nothing to merge (but the first CTA's) never wait. A following attention call launched the same way may be
// scheduled from the wait on (its prologue overlaps this kernel, its inputs are read only
// after this grid has completed).
// Minimum resident CTAs an SM (register budget) of each instantiation, measured: two rows
// a CTA want their registers (fewer, with spills, ran slower), one row with eight warps
// wants three CTAs an SM (384 CTAs for 384 rows), the narrow chunks of a few long rows run
// best with the compiler's own choice (0).
template <int VEC, int WPR>
constexpr int kMergeMinBlocks = (VEC == 16 && WPR == 4) ? 2 : ((VEC == 1) ? 0 : 3);

// TREE: the plan's sequences are passes over one, its ranges belong to teams of CTAs, and
// member m's slots are those of CTA range * team + m (mla_internal.cuh, tree_plan); rows are
// still numbered through all sequences' nodes.
struct PlanRow {
  int b;      // the plan's sequence
  int64_t r;  // row within its unit
  int member;
};
template <bool TREE>
__device__ __forceinline__ PlanRow plan_row(const AttnParams& p, int64_t row) {
  if constexpr (TREE) {
    const int per = p.n_q * p.H;
    const int in = (int)(row % per), group = in / p.R;
    return {(int)(row / per) * p.passes + group / p.team, in % p.R, group % p.team};
  } else {
    return {(int)(row / p.R), row % p.R, 0};
  }
}
template <bool TREE>
__device__ __forceinline__ int plan_seq(const AttnParams& p, int b) {
  return TREE ? b / p.passes : b;
}

template <int VEC, int WPR, typename OutT, bool TREE = false>
__global__ void __launch_bounds__(kMergeThreads, kMergeMinBlocks<VEC, WPR>)
    merge_split_kernel(AttnParams p) {
  constexpr int kRowsPerCta = kMergeWarps / WPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = warp / WPR, gt = threadIdx.x - g * 32 * WPR;
  const int64_t rows = TREE ? (int64_t)(p.B / p.passes) * p.n_q * p.H : (int64_t)p.B * p.R;
  const int64_t row0 = (int64_t)blockIdx.x * kRowsPerCta;
  // the cost axis: every sequence as kUnitCost units, then its blocks (none if empty);
  // its length, and the units before each row group's sequence
  int bg[kRowsPerCta];
  long long tot = 0, before[kRowsPerCta];
#pragma unroll
  for (int k = 0; k < kRowsPerCta; ++k) {
    bg[k] = plan_row<TREE>(p, min(row0 + k, rows - 1)).b;
    before[k] = 0;
  }
  for (int x = threadIdx.x; x < p.B; x += kMergeThreads) {
    const int nb = plan_blocks(p, plan_seq<TREE>(p, x));
    const long long cost = nb > 0 ? nb + kUnitCost : 0;
    tot += cost;
#pragma unroll
    for (int k = 0; k < kRowsPerCta; ++k)
      if (x < bg[k]) before[k] += cost;
  }
  __shared__ long long s_red[kMergeWarps][1 + kRowsPerCta];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
#pragma unroll
    for (int k = 0; k < kRowsPerCta; ++k) before[k] += __shfl_xor_sync(0xffffffffu, before[k], o);
  }
  if (lane == 0) {
    s_red[warp][0] = tot;
#pragma unroll
    for (int k = 0; k < kRowsPerCta; ++k) s_red[warp][1 + k] = before[k];
  }
  __syncthreads();
  long long total = 0, pre = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    total += s_red[w][0];
    pre += s_red[w][1 + g];
  }
  // The first CTA waits for the attention grid whatever it has to merge: this grid must not
  // complete before that one, for the sake of a programmatic dependent that waits for this one
  // (the next call's attention kernel, which may use the same workspace). Letting that dependent go
  // before the wait gains nothing (152 whole sequences, eight calls in a graph, 23.9 us a call
  // either way).
  if (blockIdx.x + blockIdx.y == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = row0 + g;  // b * R + r
  if (row >= rows) return;
  const int chunk = blockIdx.y;
  static_assert(kRowsPerCta <= 2, "row groups a CTA");
  const int b = (g == 0) ? bg[0] : bg[kRowsPerCta - 1];  // (no indexing of a local array)
  const PlanRow at = plan_row<TREE>(p, row);
  const int64_t r = at.r;
  const int num_blocks = plan_blocks(p, plan_seq<TREE>(p, b));
  OutT* out_row;
  if constexpr (sizeof(OutT) == 4)
    out_row = p.out_f32 + row * kDV;
  else
    out_row = p.out + row * kDV;
  float* lse_out = p.lse ? p.lse + row : nullptr;
  if (num_blocks == 0) {  // no unit of the attention kernel touches these rows
    for (int x = gt; x < 32 * VEC; x += 32 * WPR) store_val(out_row + chunk * 32 * VEC + x, 0.f);
    if (gt == 0 && chunk == 0 && lse_out) *lse_out = -INFINITY;
    return;
  }
  const int64_t n = TREE ? tree_ranges(total, p.num_ctas / p.team) : p.num_ctas;
  const int64_t first = pre + kUnitCost;  // the sequence's first block
  // pieces: one per CTA range the sequence's blocks overlap (with fewer blocks than CTAs
  // every range holds at most one block)
  const int64_t c0 = range_of(first, total, n);
  const int count = (total >= n) ? (int)(range_of(first + num_blocks - 1, total, n) - c0 + 1)
                                 : num_blocks;
  if (count == 1) return;  // the attention kernel writes this row itself
  // piece 0 takes the second slot of its CTA when that CTA's range began before this
  // sequence's span (in an earlier sequence); every later piece begins its CTA's range
  const int64_t first_odd = (range_lo(c0, total, n) < first - kUnitCost) ? 1 : 0;
  auto cta_of = [&](int64_t c) -> int64_t { return TREE ? c * p.team + at.member : c; };
  auto slot_of = [&](int i) -> int64_t {
    if (i == 0) return 2 * cta_of(c0) + first_odd;
    return 2 * cta_of((total >= n) ? c0 + i : range_of_few((int)first + i, (int)total, (int)n));
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  merge_row_chunk<VEC, WPR, OutT>(p.part_out, p.part_lse, count, slot_of, r, p.R, chunk, out_row,
                                  lse_out);
}

// Tree verify, when there are rows enough to fill the GPU: a CTA takes eight rows of one group of
// a sequence's nodes, a warp a row. The rows of a group share their pieces, so the plan is looked
// up once for the eight, and a warp moves whole 2 KB rows of partials (a lane 16 values).
// merge_split_kernel, two rows a CTA, looked it up four times as often: 73 us where this takes
// 12 us (12,288 rows, most of them in two or three pieces). Bound: one round of dependent L2
// loads a CTA, then the partials' bytes through L2.
constexpr int kTreeMergePieces = 2;  // pieces a warp loads at once
__global__ void __launch_bounds__(kMergeThreads, 3) merge_tree_kernel(AttnParams p, int chunks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int chunk = blockIdx.x % chunks;            // eight rows of the group
  const int group = blockIdx.x / chunks % (p.team * p.passes);
  const int seq = blockIdx.x / chunks / (p.team * p.passes);
  const int b = seq * p.passes + group / p.team, member = group % p.team;
  const int r = chunk * kMergeWarps + warp;         // row of the group
  long long tot = 0, before = 0;
  for (int x = threadIdx.x; x < p.B; x += kMergeThreads) {
    const int nb = plan_blocks(p, x / p.passes);
    const long long cost = nb > 0 ? nb + kUnitCost : 0;
    tot += cost;
    if (x < b) before += cost;
  }
  __shared__ long long s_red[kMergeWarps][2];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tot += __shfl_xor_sync(0xffffffffu, tot, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    s_red[warp][0] = tot;
    s_red[warp][1] = before;
  }
  __syncthreads();
  long long total = 0, pre = 0;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    total += s_red[w][0];
    pre += s_red[w][1];
  }
  // The first CTA waits for the attention grid whatever it has to merge: this grid must not
  // complete before that one, for the sake of a programmatic dependent that waits for this one.
  if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  const int node0 = group * p.group_nodes;
  if (r >= min(p.group_nodes, p.n_q - node0) * p.H) return;
  const int64_t row = ((int64_t)seq * p.n_q + node0) * p.H + r;
  uint4* out = reinterpret_cast<uint4*>(p.out + row * kDV + lane * 16);
  const int num_blocks = plan_blocks(p, seq);
  if (num_blocks == 0) {  // no unit of the attention kernel touches these rows
    out[0] = out[1] = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0 && p.lse) p.lse[row] = -INFINITY;
    return;
  }
  // the pieces and their slots, as in merge_split_kernel
  const int64_t n = tree_ranges(total, p.num_ctas / p.team);
  const int64_t first = pre + kUnitCost;
  const int64_t c0 = range_of(first, total, n);
  const int count = (total >= n) ? (int)(range_of(first + num_blocks - 1, total, n) - c0 + 1)
                                 : num_blocks;
  if (count == 1) return;  // the attention kernel writes this row itself
  const int64_t first_odd = (range_lo(c0, total, n) < first - kUnitCost) ? 1 : 0;
  auto at_of = [&](int i) -> int64_t {
    const int64_t c = (i == 0 || total >= n) ? c0 + i : range_of_few((int)first + i, (int)total, (int)n);
    return (2 * (c * p.team + member) + (i == 0 ? first_odd : 0)) * p.part_rows + r;
  };
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  float lse_of = lane < count ? p.part_lse[at_of(lane)] : -INFINITY;
  float4 v[kTreeMergePieces][4];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kTreeMergePieces; ++k)
      if (i0 + k < count) {
        const float4* src = reinterpret_cast<const float4*>(p.part_out + at_of(i0 + k) * kDV + lane * 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k][e] = src[e];
      }
  };
  load(0);
  float m = lse_of;
  for (int i = lane + 32; i < count; i += 32) m = fmaxf(m, p.part_lse[at_of(i)]);
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float sum = lse_of == -INFINITY ? 0.f : expf(lse_of - m);
  for (int i = lane + 32; i < count; i += 32) {
    const float l = p.part_lse[at_of(i)];
    if (l != -INFINITY) sum += expf(l - m);
  }
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (m == -INFINITY && sum == 0.f) {  // no piece saw a key (a NaN piece: the sum is NaN)
    out[0] = out[1] = make_uint4(0u, 0u, 0u, 0u);
    if (lane == 0 && p.lse) p.lse[row] = -INFINITY;
    return;
  }
  const float lse = m + logf(sum);
  float acc[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int i0 = 0;;) {
#pragma unroll
    for (int k = 0; k < kTreeMergePieces; ++k) {
      const int i = i0 + k;
      if (i >= count) break;
      const float l = i < 32 ? __shfl_sync(0xffffffffu, lse_of, i) : p.part_lse[at_of(i)];
      if (l == -INFINITY) continue;  // an empty piece's data was never written
      const float w = expf(l - lse);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[4 * e] += w * v[k][e].x;
        acc[4 * e + 1] += w * v[k][e].y;
        acc[4 * e + 2] += w * v[k][e].z;
        acc[4 * e + 3] += w * v[k][e].w;
      }
    }
    i0 += kTreeMergePieces;
    if (i0 >= count) break;
    load(i0);
  }
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(acc[2 * e], acc[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t*>(&t);
  }
  out[0] = make_uint4(w[0], w[1], w[2], w[3]);
  out[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (lane == 0 && p.lse) p.lse[row] = lse;
}

// Prefill units of an incomplete last round, each run as two halves along the keys: split
// unit v (v = 0 .. split_units - 1, the units handed out last, i.e. the first positions)
// covers positions [pos0, pos0 + npos) with rows j * H + h, and its halves sit in partial
// slots 2v and 2v + 1 of 48 rows. Two rows a CTA (four warps a row), 24 CTAs a unit.
template <typename OutT>
__global__ void __launch_bounds__(kMergeThreads, 2)
    merge_prefill_kernel(AttnParams p, int P, int split_units) {
  constexpr int WPR = 4;
  const int g = (threadIdx.x >> 5) / WPR;
  const int v = blockIdx.x / 24;
  const int r = (blockIdx.x % 24) * 2 + g;  // row of the unit
  const int pos0 = (split_units - 1 - v) * P;
  const int npos = min(P, p.n_q - pos0);
  if (r >= npos * p.H) return;
  const int64_t row = (int64_t)pos0 * p.H + r;
  OutT* out_row;
  if constexpr (sizeof(OutT) == 4)
    out_row = p.out_f32 + row * kDV;
  else
    out_row = p.out + row * kDV;
  float* lse_out = p.lse ? p.lse + row : nullptr;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  merge_row_chunk<16, WPR, OutT>(p.part_out, p.part_lse, 2,
                                 [v](int i) -> int64_t { return 2 * v + i; }, r, p.part_rows, 0,
                                 out_row, lse_out);
}

template <int VEC>
__global__ void __launch_bounds__(kMergeThreads)
    merge_standalone_kernel(const float* po, const float* pl, int S, int64_t R, uint16_t* out,
                            float* lse) {
  const int64_t row = blockIdx.x;
  merge_row_chunk<VEC, kMergeWarps, uint16_t>(po, pl, S, [](int i) -> int64_t { return i; }, row, R,
                                              blockIdx.y, out + row * kDV, lse ? lse + row : nullptr);
}

// Chunk width: whole 512-wide rows when there are rows enough to fill the GPU, narrower
// chunks (more CTAs per row) for the few rows of a long history split over every SM.
int merge_vec(int64_t rows, int num_sms) {
  if (rows >= num_sms) return 16;
  if (rows * 4 >= num_sms) return 4;
  return 1;
}

}  // namespace

cudaError_t launch_merge(const AttnParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.B * p.R;
  const int vec = merge_vec(rows, p.num_ctas);
  // Whole 512-wide rows split over few CTAs each (a batch of short sequences): two rows a
  // CTA, four warps a row (half the CTAs to launch: measured faster). Rows with many pieces
  // (a sequence over more than 8 CTAs) keep eight warps, which load twice the pieces a round.
  const bool two_rows = vec == 16 && p.num_ctas <= 8 * p.B;
  const int64_t per = two_rows ? 2 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((rows + per - 1) / per), kDV / (32 * vec));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.out_f32) {
    if (two_rows) return cudaLaunchKernelEx(&cfg, merge_split_kernel<16, 4, float>, p);
    if (vec == 16) return cudaLaunchKernelEx(&cfg, merge_split_kernel<16, kMergeWarps, float>, p);
    if (vec == 4) return cudaLaunchKernelEx(&cfg, merge_split_kernel<4, kMergeWarps, float>, p);
    return cudaLaunchKernelEx(&cfg, merge_split_kernel<1, kMergeWarps, float>, p);
  }
  if (two_rows) return cudaLaunchKernelEx(&cfg, merge_split_kernel<16, 4, uint16_t>, p);
  if (vec == 16) return cudaLaunchKernelEx(&cfg, merge_split_kernel<16, kMergeWarps, uint16_t>, p);
  if (vec == 4) return cudaLaunchKernelEx(&cfg, merge_split_kernel<4, kMergeWarps, uint16_t>, p);
  return cudaLaunchKernelEx(&cfg, merge_split_kernel<1, kMergeWarps, uint16_t>, p);
}

cudaError_t launch_merge_tree(const AttnParams& p, int sequences, cudaStream_t s) {
  const int64_t rows = (int64_t)sequences * p.n_q * p.H;
  // 512 or 128 values a CTA, as launch_merge; never 32 (24 rows in up to 64 pieces: 33 to 38 us a
  // call with 384 CTAs of 32 values, in two waves, 19 to 34 us with 96 of 128)
  const int vec = rows >= p.num_ctas ? 16 : 4;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  // (a warp a row takes its pieces two at a time: with more than a dozen of them, eight warps a
  // row. Whole calls in us, this / that: 9 pieces a row 32.6 / 35.1 and 24.6 / 30.8, 13 pieces, or
  // 9 of them where fewer_ranges applies, 39.4 / 38.2 and 30.5 / 34.0, 19 pieces 24.4 / 22.8 and 48.7
  // / 37.9)
  if (vec == 16 && p.num_ctas / p.team <= 13 * p.B) {
    const int chunks = (p.R + kMergeWarps - 1) / kMergeWarps;
    cfg.gridDim = dim3((unsigned)sequences * p.team * p.passes * chunks);
    return cudaLaunchKernelEx(&cfg, merge_tree_kernel, p, chunks);
  }
  cfg.gridDim = dim3((unsigned)rows, kDV / (32 * vec));
  if (vec == 16) return cudaLaunchKernelEx(&cfg, merge_split_kernel<16, kMergeWarps, uint16_t, true>, p);
  return cudaLaunchKernelEx(&cfg, merge_split_kernel<4, kMergeWarps, uint16_t, true>, p);
}

cudaError_t launch_merge_prefill(const AttnParams& p, int P, int split_units, cudaStream_t s) {
  if (split_units <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split_units * 24);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (p.out_f32) return cudaLaunchKernelEx(&cfg, merge_prefill_kernel<float>, p, P, split_units);
  return cudaLaunchKernelEx(&cfg, merge_prefill_kernel<uint16_t>, p, P, split_units);
}

cudaError_t launch_merge_standalone(const float* part_out, const float* part_lse, int S, int64_t R,
                                    uint16_t* out, float* lse, int num_sms, cudaStream_t s) {
  const int vec = merge_vec(R, num_sms);
  const dim3 grid((unsigned)R, kDV / (32 * vec));
  if (vec == 16)
    merge_standalone_kernel<16><<<grid, kMergeThreads, 0, s>>>(part_out, part_lse, S, R, out, lse);
  else if (vec == 4)
    merge_standalone_kernel<4><<<grid, kMergeThreads, 0, s>>>(part_out, part_lse, S, R, out, lse);
  else
    merge_standalone_kernel<1><<<grid, kMergeThreads, 0, s>>>(part_out, part_lse, S, R, out, lse);
  return cudaGetLastError();
}

}  // namespace mla
