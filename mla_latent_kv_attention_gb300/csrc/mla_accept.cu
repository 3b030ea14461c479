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
// Layout. A cluster of CTAs takes one sequence. Each CTA first walks the nodes by itself (all
// nodes' entries are fetched at once, one thread a node: two dependent loads in all), which
// names the row to draw from. Then warp w of CTA r sums the weights of its own contiguous span
// of the row, 128 a step; the CTAs exchange their totals through distributed shared memory (one
// cluster barrier), the CTA that holds the threshold finds the warp from its warps' totals, and
// that warp the step, the lane and the token. One pass over one row (two with draft
// probabilities) is all that is read of the vocabulary. Bound: latency (two loads to walk, one
// round over the row, one barrier), then HBM.
#include <cuda_runtime.h>

#include "mla_internal.cuh"
#include "sm100.cuh"

namespace mla {
namespace {

constexpr int kAcThreads = 512;
constexpr int kAcWarps = kAcThreads / 32;
constexpr int kAcCluster = 8;
constexpr int kAcStep = 128;  // entries a warp takes a step
constexpr int kAcUnroll = 8;  // steps in flight
constexpr int kNone = -1;

struct AcSmem {
  int tok[MLA_MAX_TREE], par[MLA_MAX_TREE];  // par = kNone: node is no draft
  long long share[MLA_MAX_TREE];             // its width on [0, 1) (drafts without probabilities)
  unsigned taken[2];                         // one bit a node: accepted if its parent is
  int path[MLA_MAX_TREE];
  int last, count;                           // last node accepted, drafts accepted
  unsigned long long cta_sum[kAcCluster];    // every CTA's total (each CTA writes all copies)
  unsigned long long warp_sum[kAcWarps];
};

// A weight as a whole multiple of 2^-43; NaN and negative weights are 0, larger ones than 1 are 1.
__device__ __forceinline__ long long weight_of(float w) {
  return __float2ll_rn(fminf(fmaxf(w, 0.f), 1.f) * 0x1p43f);
}
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

// VEC: a lane's four entries of a step are one 16-byte vector (rows 16-byte aligned, V a
// multiple of four); otherwise they lie 32 apart, so that single loads stay coalesced.
template <bool VEC>
__global__ void __launch_bounds__(kAcThreads, 2) accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ AcSmem s;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const unsigned rank = sm100::cluster_ctarank();
  const int ctas = gridDim.x;  // CTAs of the cluster
  const int b = blockIdx.y, n = a.n, V = a.V;
  const float* target = a.target + (int64_t)b * n * V;
  const float* draft = a.draft ? a.draft + (int64_t)b * (n - 1) * V : nullptr;
  const float* u = a.uniforms + (int64_t)b * (n + 1);
  // the other CTAs' shared memory may be written once they all run: arrive here, wait below
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");

  // ---- the walk
  bool drafted = false, taken = false;
  int par = kNone, tok = 0;
  float pt = 0.f, qt = 0.f, up = 0.f;
  if (t < MLA_MAX_TREE) {
    if (t >= 1 && t < n) {
      tok = a.tokens[(int64_t)b * n + t];
      par = a.parents ? a.parents[(int64_t)b * n + t] : t - 1;
      drafted = tok >= 0 && tok < V && par >= 0 && par < t;
    }
    if (drafted) {
      pt = target[(int64_t)par * V + tok];
      if (draft) qt = draft[(int64_t)(t - 1) * V + tok];
      up = u[par];
    } else {
      par = kNone;
    }
    s.tok[t] = tok;
    s.par[t] = par;
    s.share[t] = weight_of(pt);
  }
  __syncthreads();
  if (t < MLA_MAX_TREE) {
    if (!draft) {
      // a sibling before this one with the same token leaves it nothing
      for (int i = 1; i < t && drafted; ++i)
        if (s.par[i] == par && s.tok[i] == tok) drafted = false;
    }
  }
  __syncthreads();
  if (t < MLA_MAX_TREE && !draft && !drafted) s.share[t] = 0;
  __syncthreads();
  if (t < MLA_MAX_TREE) {
    if (drafted) {
      if (draft) {
        taken = __fmul_rn(up, qt) < pt;
      } else {
        long long below = 0;
        for (int i = 1; i < t; ++i)
          if (s.par[i] == par) below += s.share[i];
        const long long mark = uniform_of<43>(up);
        taken = mark >= below && mark < below + s.share[t];
      }
    }
    const unsigned bits = __ballot_sync(0xffffffffu, taken);
    if (lane == 0) s.taken[warp] = bits;
  }
  __syncthreads();
  if (t == 0) {
    // a child's index is above its parent's, and of a node's children at most one is taken:
    // one pass upwards over the taken nodes follows the chain
    unsigned long long bits = ((unsigned long long)s.taken[1] << 32) | s.taken[0];
    int at = 0, k = 0;
    s.path[0] = 0;
    while (bits) {
      const int j = __ffsll((long long)bits) - 1;
      bits &= bits - 1;
      if (s.par[j] == at) {
        at = j;
        s.path[++k] = j;
      }
    }
    s.last = at;
    s.count = k;
  }
  __syncthreads();
  const int last = s.last, count = s.count;
  if (rank == 0 && t < n) {
    // the drawn token's own place is written by the CTA that draws it
    const int64_t o = (int64_t)b * n + t;
    a.path[o] = t <= count ? s.path[t] : -1;
    if (t != count) a.out_tokens[o] = t < count ? s.tok[s.path[t + 1]] : -1;
    if (t == 0) a.num_accepted[b] = count;
  }

  // ---- the draw
  const float* prow = target + (int64_t)last * V;
  const float* qrow = nullptr;  // the refused draft's probabilities
  if (draft && last + 1 < n && s.par[last + 1] == last) qrow = draft + (int64_t)last * V;
  const int span = (V + ctas * kAcWarps * kAcStep - 1) / (ctas * kAcWarps * kAcStep) * kAcStep;
  const int w0 = ((int)rank * kAcWarps + warp) * span;  // (at most 2^19 + a span)
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
  bool whole = false;  // second round: nothing was left, draw from the target row itself
  unsigned long long total = 0, mine = 0, before = 0;
  // weights of the step at `at`, with the refused children's tokens left out
  auto weigh = [&](int at, const float (&p)[4], const float (&q)[4], long long (&w)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = weight_of(whole ? p[e] : p[e] - q[e]);
    if (!draft && !whole)
      for (int j = last + 1; j < n; ++j)
        if (s.par[j] == last) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (index_of(at, e) == s.tok[j]) w[e] = 0;
        }
  };
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  for (;;) {
    unsigned long long sum = 0;
    for (int at = w0; at < w1; at += kAcUnroll * kAcStep) {
      float p[kAcUnroll][4], q[kAcUnroll][4];
#pragma unroll
      for (int k = 0; k < kAcUnroll; ++k) {
        load4(prow, at + k * kAcStep, p[k]);
        if (qrow)
          load4(qrow, at + k * kAcStep, q[k]);
        else
          q[k][0] = q[k][1] = q[k][2] = q[k][3] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < kAcUnroll; ++k) {
        long long w[4];
        weigh(at + k * kAcStep, p[k], q[k], w);
        sum += (unsigned long long)(w[0] + w[1] + w[2] + w[3]);
      }
    }
    mine = warp_sum_u64(sum);
    if (lane == 0) s.warp_sum[warp] = mine;
    __syncthreads();
    unsigned long long cta = 0;
    before = 0;
    for (int w = 0; w < kAcWarps; ++w) {
      if (w < warp) before += s.warp_sum[w];
      cta += s.warp_sum[w];
    }
    if (t < ctas) {
      unsigned* dst = reinterpret_cast<unsigned*>(&s.cta_sum[rank]);
      sm100::st_dsmem_u32(dst, (uint32_t)t, (unsigned)cta);
      sm100::st_dsmem_u32(dst + 1, (uint32_t)t, (unsigned)(cta >> 32));
    }
    sm100::cluster_sync();  // every CTA holds every total
    total = 0;
    for (int r = 0; r < ctas; ++r) {
      if (r < (int)rank) before += s.cta_sum[r];
      total += s.cta_sum[r];
    }
    if (total != 0 || whole) break;
    whole = true;
    qrow = nullptr;
    sm100::cluster_sync();  // the totals have been read before the second round writes them
  }
  if (total == 0) {
    if (rank == 0 && t == 0) a.out_tokens[(int64_t)b * n + count] = -1;
    return;
  }
  const unsigned long long mark = __umul64hi(total, (unsigned long long)uniform_of<31>(u[n]) << 33);
  if (mark < before || mark >= before + mine) return;
  // this warp's span holds the token: find the step, then the entry
  unsigned long long left = mark - before;  // weight of the span before the token's end
  for (int at = w0; at < w1; at += kAcStep) {
    float p[4], q[4] = {0.f, 0.f, 0.f, 0.f};
    long long w[4];
    load4(prow, at, p);
    if (qrow) load4(qrow, at, q);
    weigh(at, p, q, w);
    const unsigned long long step = warp_sum_u64((unsigned long long)(w[0] + w[1] + w[2] + w[3]));
    if (left >= step) {
      left -= step;
      continue;
    }
    // entries in index order: lane by lane (VEC), or the lanes of entry 0, then of entry 1, ...
    unsigned long long acc = 0;
    int found = 0x7fffffff;
    if constexpr (VEC) {
      const unsigned long long own = (unsigned long long)(w[0] + w[1] + w[2] + w[3]);
      unsigned long long incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      acc = incl - own;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc += (unsigned long long)w[e];
        if (acc > left) found = min(found, index_of(at, e));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        unsigned long long incl = (unsigned long long)w[e];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned long long y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        if (acc + incl > left) found = min(found, index_of(at, e));
        acc += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    found = __reduce_min_sync(0xffffffffu, found);
    if (lane == 0) a.out_tokens[(int64_t)b * n + count] = found;
    return;
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, cudaStream_t s) {
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.target) % 16 == 0 &&
                   reinterpret_cast<uintptr_t>(a.draft) % 16 == 0;
  // CTAs a sequence: a warp has at least one step of its own
  const int steps = (a.V + kAcStep - 1) / kAcStep;
  const int ctas = min(kAcCluster, (steps + kAcWarps - 1) / kAcWarps);
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
  return vec ? cudaLaunchKernelEx(&cfg, accept_kernel<true>, a)
             : cudaLaunchKernelEx(&cfg, accept_kernel<false>, a);
}

}  // namespace mla
