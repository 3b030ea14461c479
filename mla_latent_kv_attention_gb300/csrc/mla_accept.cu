// mla_accept.cu -- acceptance of drafted tokens against the target's probabilities, and the draw
// of the token after them: the step behind a verify pass (speculative decoding's accept and
// resample, the sampler that "AMD MI355X推理Kimi K3：吞吐量超NVIDIA，首字优化显著", section
// "ROCm适配迎来突破，软件壁垒不再高不可攀", counts among what verification needs).
//
// The mathematics. A draft x drawn from q is kept with probability min(1, p(x) / q(x)), and
// after a refusal the next token is drawn from max(p - q, 0) / sum: together they emit exactly p.
// Drafts without probabilities (a tree's children) are intervals of [0, 1) as wide as p gives
// them, so one uniform number picks a child or none, and the draw after none is from p without
// the children: again p.
//
// Whole numbers. A weight is a multiple of 2^-43 (rounded to nearest; float32 values from 2^-19 up
// are such multiples), and every sum is a sum of 64-bit integers: exact, whatever order the
// threads add in, so the token drawn does not depend on the launch shape. At most 2^19 weights
// of at most 2^43 stay below 2^62. Tokens of probability below 2^-44 are never drawn, which
// together is less than 2^-25 of a row: a float32 uniform cannot tell. The threshold
// floor(u * total), u in steps of 2^-31, is a 64-bit high product.
//
// Arithmetic. A float32 weight w becomes its whole number in two float32 additions: w + 12
// rounds w to a multiple of 2^-20 (the unit of [8, 16)), whose count is the difference of the bit
// patterns, and what is left, at most 2^-21, added to 1.5 * 2^-20 is rounded to 2^-43 the same
// way. The pair of counts is the weight rounded to nearest even, because the first is a whole
// multiple of the second's unit. A conversion instruction to 64 bits runs at a small fraction of
// the rate (it took 14 us of the 32 us of 64 sequences of 129,280 tokens).
//
// Layout. A cluster of CTAs takes one sequence. Warp 0 of each CTA walks the nodes by itself (a
// lane two nodes, all nodes' entries fetched at once: two dependent loads in all), which names
// the row to draw from. Then warp w of CTA r sums the weights of its own contiguous span of the
// row, 128 a step; the CTAs exchange their totals through distributed shared memory (one cluster
// barrier), the CTA that holds the threshold finds the warp from its warps' totals, and that
// warp the step, the lane and the token. One pass over one row (two with draft probabilities) is
// all that is read of the vocabulary. Bound: latency (two loads to walk, one round over the row,
// one barrier: 8 sequences of 129,280 tokens 6.2 us, with 3 drafts and their probabilities), then
// HBM (64 sequences of 7 drafts: 66 MB in 16.9 us, 3.9 TB/s; 10.8 us when they lie in L2).
#include <cuda_runtime.h>

#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kAcThreads = 512;
constexpr int kAcWarps = kAcThreads / 32;
constexpr int kAcCluster = 8;
constexpr int kAcStep = 128;  // entries a warp takes a step
constexpr int kNone = -1;

struct AcSmem {
  int tok[MLA_MAX_TREE], par[MLA_MAX_TREE];  // par = kNone: node is no draft
  long long share[MLA_MAX_TREE];             // its width on [0, 1) (drafts without probabilities)
  int kid[MLA_MAX_TREE];                     // tokens of the last node's children, each once
  int kids;
  int last, count;                           // last node accepted, drafts accepted
  int more;                                  // 1: a draft after `last` was refused
  unsigned long long cta_sum[kAcCluster];    // every CTA's total (each CTA writes all copies)
  unsigned long long warp_sum[kAcWarps];
};

// A weight as whole multiples of 2^-20 (hi) and 2^-43 (lo, signed) that add up to it; NaN and
// negative weights are 0, larger ones than 1 are 1.
struct Weight {
  int hi, lo;
};
__device__ __forceinline__ Weight split_weight(float w) {
  w = fminf(fmaxf(w, 0.f), 1.f);
  const float coarse = __fadd_rn(w, 12.f);
  const float rest = __fsub_rn(w, __fsub_rn(coarse, 12.f));  // both exact
  const float fine = __fadd_rn(rest, 0x1.8p-20f);
  return {__float_as_int(coarse) - __float_as_int(12.f), __float_as_int(fine) - __float_as_int(0x1.8p-20f)};
}
__device__ __forceinline__ long long whole_weight(Weight w) { return ((long long)w.hi << 23) + w.lo; }

// A draft probability within [0, 1]; NaN is 1, which leaves nothing of the target's to draw.
// (A clamp by fminf, then fmaxf, says the same, but compiled to one whose NaN is 0.)
__device__ __forceinline__ float draft_weight(float q) { return q == q ? __saturatef(q) : 1.f; }

// A uniform number in steps of 2^-BITS, in [0, 2^BITS).
template <int BITS>
__device__ __forceinline__ long long uniform_of(float u) {
  const float scale = (float)(1ull << BITS);
  const long long v = __float2ll_rz(fminf(fmaxf(u, 0.f), 1.f) * scale);
  return v < (1ll << BITS) ? v : (1ll << BITS) - 1;
}

__device__ __forceinline__ unsigned long long warp_sum_u64(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The walk (one warp; lane l holds nodes l and l + 32): which drafts are accepted, what the draw
// starts from.
template <bool DRAFT>
__device__ void walk(const AcceptArgs& a, AcSmem& s, int b, bool write) {
  const int lane = threadIdx.x & 31, n = a.n;
  const float* target = a.target + (int64_t)b * n * a.V;
  const float* u = a.uniforms + (int64_t)b * (n + 1);
  int tok[2], par[2];
  float pt[2], qt[2], up[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = lane + 32 * h;
    tok[h] = par[h] = kNone;
    if (t >= 1 && t < n) {
      tok[h] = a.tokens[(int64_t)b * n + t];
      par[h] = a.parents ? a.parents[(int64_t)b * n + t] : t - 1;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int t = lane + 32 * h;
    if (tok[h] < 0 || tok[h] >= a.V || par[h] < 0 || par[h] >= t) par[h] = kNone;
    pt[h] = qt[h] = up[h] = 0.f;
    if (par[h] != kNone) {
      pt[h] = target[(int64_t)par[h] * a.V + tok[h]];
      if (DRAFT) qt[h] = a.draft[((int64_t)b * (n - 1) + t - 1) * a.V + tok[h]];
      up[h] = fminf(fmaxf(u[par[h]], 0.f), 0x1.fffffep-1f);  // in [0, 1), NaN as 0
    }
    s.tok[t] = tok[h];
    s.par[t] = par[h];
  }
  __syncwarp();
  bool first[2] = {par[0] != kNone, par[1] != kNone};  // no sibling before it has its token
  if (!DRAFT && a.parents) {
    for (int i = 1; i < n; ++i) {
      const int pi = s.par[i], ti = s.tok[i];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (i < lane + 32 * h && pi == par[h] && ti == tok[h]) first[h] = false;
    }
  }
  bool taken[2];
  if (DRAFT) {
#pragma unroll
    for (int h = 0; h < 2; ++h)  // (a NaN pt is 0: nothing is below it)
      taken[h] = par[h] != kNone && qt[h] == qt[h] && __fmul_rn(up[h], draft_weight(qt[h])) < __saturatef(pt[h]);
  } else {
    long long below[2] = {0, 0}, share[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      share[h] = first[h] ? whole_weight(split_weight(pt[h])) : 0;
      s.share[lane + 32 * h] = share[h];
    }
    __syncwarp();
    if (a.parents) {
      for (int i = 1; i < n; ++i) {
        const int pi = s.par[i];
        const long long si = s.share[i];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (i < lane + 32 * h && pi == par[h]) below[h] += si;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long mark = uniform_of<43>(up[h]);
      taken[h] = first[h] && mark >= below[h] && mark < below[h] + share[h];
    }
  }
  // a child's index is above its parent's, and of a node's children at most one is taken: one
  // pass upwards over the taken nodes follows the chain (every lane the same pass)
  unsigned long long bits = __ballot_sync(0xffffffffu, taken[0]) |
                            (unsigned long long)__ballot_sync(0xffffffffu, taken[1]) << 32;
  unsigned long long kept = 1;  // nodes of the chain
  int last = 0;
  while (bits) {
    const int j = __ffsll((long long)bits) - 1;
    bits &= bits - 1;
    if (s.par[j] == last) {
      last = j;
      kept |= 1ull << j;
    }
  }
  const int count = __popcll(kept) - 1;
  // the refused children's tokens, each once
  int at = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const bool kid = first[h] && par[h] == last;
    const unsigned m = __ballot_sync(0xffffffffu, kid);
    if (kid) s.kid[at + __popc(m & ((1u << lane) - 1))] = tok[h];
    at += __popc(m);
  }
  if (lane == 0) {
    s.kids = at;
    s.last = last;
    s.count = count;
    s.more = DRAFT && at > 0;
  }
  if (write) {
    // (the drawn token's own place is written by the CTA that draws it)
    int32_t* path = a.path + (int64_t)b * n;
    int32_t* out = a.out_tokens + (int64_t)b * n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = lane + 32 * h;
      if (t < n && (kept >> t & 1)) {  // its place on the chain
        const int k = __popcll(kept & ((1ull << t) - 1));
        path[k] = t;
        if (k > 0) out[k - 1] = tok[h];
      }
      if (t < n && t > count) path[t] = out[t] = -1;
    }
    if (lane == 0) a.num_accepted[b] = count;
  }
}

// DRAFT: drafts come with their probabilities (a chain). VEC: a lane's four entries of a step are
// one 16-byte vector (rows 16-byte aligned, V a multiple of four); otherwise they lie 32 apart, so
// that single loads stay coalesced.
template <bool DRAFT, bool VEC>
__global__ void __launch_bounds__(kAcThreads, 2) accept_kernel(const __grid_constant__ AcceptArgs a) {
  // steps in flight: 16-byte loads of one row or of two, eight a lane
  constexpr int kSteps = DRAFT ? 4 : 8;
  __shared__ AcSmem s;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const unsigned rank = sm100::cluster_ctarank();
  const int ctas = gridDim.x;  // CTAs of the cluster
  const int b = blockIdx.y, n = a.n, V = a.V;
  // the other CTAs' shared memory may be written once they all run: arrive here, wait below
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (warp == 0) walk<DRAFT>(a, s, b, rank == 0);
  __syncthreads();
  const float* prow = a.target + ((int64_t)b * n + s.last) * V;
  const float* qrow = nullptr;  // the refused draft's probabilities
  if (DRAFT && s.more) qrow = a.draft + ((int64_t)b * (n - 1) + s.last) * V;
  int32_t* drawn = a.out_tokens + (int64_t)b * n + s.count;

  const int span = (V + ctas * kAcWarps * kAcStep - 1) / (ctas * kAcWarps * kAcStep) * kAcStep;
  const int w0 = ((int)rank * kAcWarps + warp) * span;  // (below 2^19 + 2^18)
  const int w1 = min(V, w0 + span);
  auto load4 = [&](const float* row, int at, float (&v)[4]) {
    if constexpr (VEC) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (at + 4 * lane < w1) f = *reinterpret_cast<const float4*>(row + at + 4 * lane);
      v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = at + 32 * e + lane < w1 ? row[at + 32 * e + lane] : 0.f;
    }
  };
  // index of entry e of this lane in the step at `at`
  auto index_of = [&](int at, int e) { return VEC ? at + 4 * lane + e : at + 32 * e + lane; };
  // the weights of the steps that w [steps][4] has room for
  auto load = [&](int at, auto& w) {
    constexpr int K = sizeof(w) / sizeof(w[0]);
    float q[K][4];
#pragma unroll
    for (int k = 0; k < K; ++k) load4(prow, at + k * kAcStep, w[k]);
    if (DRAFT && qrow) {
#pragma unroll
      for (int k = 0; k < K; ++k) load4(qrow, at + k * kAcStep, q[k]);
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[k][e] = __saturatef(w[k][e]) - draft_weight(q[k][e]);
    }
  };
  // children's tokens in this warp's span: left out of the draw (a bit a child)
  unsigned long long out_of_span = 0;
  if (!DRAFT)
    for (int k = 0; k < s.kids; ++k)
      if (s.kid[k] >= w0 && s.kid[k] < w1) out_of_span |= 1ull << k;
  unsigned long long total = 0, mine = 0, before = 0;
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (int round = 0;; ++round) {
    long long sum = 0;
    for (int at = w0; at < w1; at += kSteps * kAcStep) {
      float w[kSteps][4];
      load(at, w);
      int hi = 0, lo = 0;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // (32 at most, each within 2^20 and 2^22)
          const Weight x = split_weight(w[k][e]);
          hi += x.hi;
          lo += x.lo;
        }
      sum += whole_weight({hi, lo});
    }
    if (lane == 0)
      for (unsigned long long m = out_of_span; m; m &= m - 1)
        sum -= whole_weight(split_weight(prow[s.kid[__ffsll((long long)m) - 1]]));
    mine = warp_sum_u64((unsigned long long)sum);
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    unsigned long long cta = lane < kAcWarps ? s.warp_sum[lane] : 0;
    before = warp_sum_u64(lane < warp ? cta : 0);
    cta = warp_sum_u64(cta);
    if (t < ctas) {
      unsigned* dst = reinterpret_cast<unsigned*>(&s.cta_sum[rank]);
      sm100::st_dsmem_u32(dst, (uint32_t)t, (unsigned)cta);
      sm100::st_dsmem_u32(dst + 1, (uint32_t)t, (unsigned)(cta >> 32));
    }
    __syncwarp();
    sm100::cluster_sync();  // every CTA holds every total
    total = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r < (int)rank) before += s.cta_sum[r];
      total += s.cta_sum[r];
    }
    if (total != 0 || round == 1) break;
    // nothing was left: a second round over the target row itself
    qrow = nullptr;
    out_of_span = 0;
    sm100::cluster_sync();  // the totals have been read before the second round writes them
  }
  if (total == 0) {
    if (rank == 0 && t == 0) *drawn = -1;
    return;
  }
  const float un = a.uniforms[(int64_t)b * (n + 1) + n];
  const unsigned long long mark = __umul64hi(total, (unsigned long long)uniform_of<31>(un) << 33);
  if (mark < before || mark >= before + mine) return;

  // ---- this warp's span holds the token: find the steps, then the step, then the entry
  constexpr int kFind = 4;
  unsigned long long left = mark - before;  // weight of the span before the token's end
  for (int at = w0; at < w1; at += kFind * kAcStep) {
    float w[kFind][4];
    load(at, w);
    unsigned long long own[kFind], step[kFind];
#pragma unroll
    for (int k = 0; k < kFind; ++k) {
      for (unsigned long long m = out_of_span; m; m &= m - 1) {
        const int token = s.kid[__ffsll((long long)m) - 1];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (index_of(at + k * kAcStep, e) == token) w[k][e] = 0.f;
      }
      long long x = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) x += whole_weight(split_weight(w[k][e]));
      own[k] = step[k] = (unsigned long long)x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < kFind; ++k) step[k] += __shfl_xor_sync(0xffffffffu, step[k], o);
    // the step that holds the token, and its entries
    int found = -1;
    unsigned long long mine_before = left, lane_sum = 0;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < kFind; ++k) {
      if (found < 0) {
        if (left < step[k]) {
          found = k;
          mine_before = left;
          lane_sum = own[k];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = w[k][e];
        } else {
          left -= step[k];
        }
      }
    }
    if (found < 0) continue;
    const int base = at + found * kAcStep;
    int token = 0x7fffffff;
    unsigned long long acc = 0;
    if constexpr (VEC) {  // entries in index order: lane by lane
      unsigned long long incl = lane_sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      acc = incl - lane_sum;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc += (unsigned long long)whole_weight(split_weight(x[e]));
        if (acc > mine_before) token = min(token, index_of(base, e));
      }
    } else {  // the lanes of entry 0, then of entry 1, ...
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        unsigned long long incl = (unsigned long long)whole_weight(split_weight(x[e]));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (acc + incl > mine_before) token = min(token, index_of(base, e));
        acc += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    token = __reduce_min_sync(0xffffffffu, token);
    if (lane == 0) *drawn = token;
    return;
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, int num_sms, cudaStream_t s) {
  // 16-byte loads where rows start on 16 bytes (64 x 129,280: 9.9 us, 10.1 an entry at a time)
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.target) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.draft) % 16 == 0;
  // CTAs a sequence: eight, halved where all sequences' would not run at once (two an SM: the walk
  // and the exchange are waited for once a wave) or where a warp would have no step of its own.
  // Single replays from HBM in us with 8 / 4 / 2 CTAs (129,280 tokens, draft probabilities): 25
  // sequences 15.6 / 17.5 / 23.7, 38 21.7 / 19.6 / 23.7, 39 22.7 / 19.6 / 23.7, 64 of seven drafts 27.8
  // / 25.7 / 29.8, 77 31.9 / 31.9 / 29.8, 152 42.1 / 40.1 / 38.0. The sizes between fill more places
  // and gain nothing (39: six 19.6, seven 22.7; 50: four 21.6, six 25.8), but for three at 77 (27.8).
  const int steps = (a.V + kAcStep - 1) / kAcStep;
  int ctas = kAcCluster;
  while (ctas > 1 && ((int64_t)a.B * ctas > 2 * num_sms || (ctas / 2) * kAcWarps >= steps)) ctas /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)a.B);
  cfg.blockDim = dim3(kAcThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ctas;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (a.draft)
    return vec ? cudaLaunchKernelEx(&cfg, accept_kernel<true, true>, a)
               : cudaLaunchKernelEx(&cfg, accept_kernel<true, false>, a);
  return vec ? cudaLaunchKernelEx(&cfg, accept_kernel<false, true>, a)
             : cudaLaunchKernelEx(&cfg, accept_kernel<false, false>, a);
}

}  // namespace mla
