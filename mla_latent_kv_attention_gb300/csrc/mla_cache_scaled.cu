// mla_cache_scaled.cu -- writing new latent rows to a cache with a scale for each block of positions.
//
// Rows are normalised and rotated as in cache_append_rope_kernel; the scale that a block needs is
// s = 2^ceil(log2(max |y| / 448)) over its new rows, at least the one it has while it holds earlier
// positions. A power of two costs e4m3, a floating format, nothing in precision, needs no division,
// and a block whose scale grows has its earlier codes moved by whole exponents, exactly (subnormals
// round): rows written one a step end up as if written once.
//
// A unit of work is a block of one sequence that new positions fall into. Sequence b's units begin
// at cu_rows[b] / G + 2 b: m rows touch at most m / G + 2 blocks of G, so no unit needs to know how
// many blocks the sequences before it touch, at the price of a few units that find nothing (G = 1:
// a unit a row, none wasted). Rows stay in registers, normalised, from the loads to the codes; the
// warps of a unit exchange their largest entries through shared memory.
//
// Rows a warp: two, four for blocks of 64 (whose unit would be a CTA of 1,024 threads otherwise). In
// us for 8,192 rows from HBM with one / two / four: G = 4 8.2 / 7.4 / 8.2, 16 8.9 / 7.4 / 8.1, 32 10.5 /
// 7.7 / 8.1, 64 - / 8.4 / 8.3; 32 sequences of one row, G = 16: 3.2 / 3.4 / 3.9.
// Bound: the launch and a chain of dependent steps (cu_rows, rows and page, the largest entry over the
// unit, codes), one round of CTAs each: 8,192 rows (14.2 MB) 5.8 us in L2, 7.4 us from HBM; 32
// sequences of one row 3.4 us in blocks of 16, of which about 0.7 us are the earlier positions' scale
// and codes, 2.7 us with a scale a position; 0.5 us more where every block grows (1 us in blocks of 64).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "mla_internal.cuh"
#include "mla_rope.cuh"

namespace mla {
namespace {

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | e4m3x2(c, d) << 16;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// A number about as large as v for a conversion that rounds: v itself, a float's rounding of a product or
// quotient, where it has no rest, else that cut off, with the last bit set, so that the conversion's rounding to
// nearest is the only one. rest: what v lacks, its sign at least.
__device__ __forceinline__ float cut_off(float v, float rest) {
  const int bits = __float_as_int(v);
  const int past = (__float_as_int(rest) ^ bits) < 0 ? 1 : 0;  // v is the larger one
  return rest == 0.f ? v : __int_as_float((bits - past) | 1);
}
// a * b (NaN where b is)
__device__ __forceinline__ float product(float a, float b) {
  const float v = a * b;
  return cut_off(v, fmaf(a, b, -v));
}
// y / s (infinite or NaN where y is); inv: about 1 / s
__device__ __forceinline__ float quotient(float y, float s, float inv) {
  float q = y * inv;
  const float rest = fmaf(-q, s, y);
  if (!(fabsf(rest) < INFINITY)) return q;
  q = fmaf(rest, inv, q);  // the nearest, or the one beside it
  return cut_off(q, fmaf(-q, s, y));
}
// four codes times a factor, rounded again; EXACT: the products are (a power of two)
template <bool EXACT>
__device__ __forceinline__ uint32_t rescaled(uint32_t four, float by) {
  const float2 a = from_e4m3x2(four & 0xFFFFu), b = from_e4m3x2(four >> 16);
  if (EXACT) return e4m3x4(a.x * by, a.y * by, b.x * by, b.y * by);
  return e4m3x4(product(a.x, by), product(a.y, by), product(b.x, by), product(b.y, by));
}

// The smallest power of two in [2^-60, 2^60] that brings `top` (finite, not negative) to 448 =
// 1.75 * 2^8 or less (2^60 where none does).
__device__ __forceinline__ float scale_for(float top) {
  const int bits = __float_as_int(top);
  const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return __int_as_float((127 + max(-60, min(60, e))) << 23);
}

template <int G>
struct ScaledCfg {
  static constexpr int kRows = G == 64 ? 4 : (G < 2 ? 1 : 2);  // rows a warp
  static constexpr int kUnitWarps = G / kRows;            // warps a unit
  static constexpr int kWarps = kUnitWarps > 8 ? kUnitWarps : 8;  // warps a CTA
  static constexpr int kUnits = kWarps / kUnitWarps;      // units a CTA
};

template <int G>
__host__ __device__ __forceinline__ int64_t first_unit_of(int64_t row, int64_t b) {
  return G == 1 ? row : row / G + 2 * b;
}

template <int G>
__global__ void __launch_bounds__(32 * ScaledCfg<G>::kWarps)
    cache_append_scaled_kernel(const __grid_constant__ AppendScaledArgs a,
                               const __grid_constant__ mla_rope_t rope) {
  using C = ScaledCfg<G>;
  __shared__ uint64_t s_turns[MLA_ROPE / 2];
  __shared__ unsigned s_top[C::kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int part = warp % C::kUnitWarps;  // this warp's place in its unit
  const int64_t unit = (int64_t)blockIdx.x * C::kUnits + warp / C::kUnitWarps;
  // the frequencies from the parameters, where lanes' different addresses are read one after another
  if (warp == 0) s_turns[lane] = rope.turns[lane];
  // (sequences whose rows all lie behind x's have no unit that could say so)
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.status && a.cu_rows[a.B] > a.n)
    atomicCAS(a.status, 0u, (unsigned)MLA_ERR_BOUNDS);

  // the last sequence whose units begin at or before this one: 32 candidates a round, of which the
  // last round's come with what the unit needs of them
  int64_t lo = 0, len = a.B, row0, row1;
  int L;
  bool found;
  while (true) {
    const int64_t step = (len + 31) / 32;
    const int64_t at = min(lo + lane * step, lo + len - 1);
    row0 = a.cu_rows[at];
    row1 = 0;
    L = 0;
    if (step == 1) {
      row1 = a.cu_rows[at + 1];
      L = a.kv.seq_lens[at];
    }
    const bool begun = lane * step < len && first_unit_of<G>(row0, at) <= unit;
    const int hits = __popc(__ballot_sync(0xffffffffu, begun));
    const int last = max(hits - 1, 0);
    found = hits > 0;  // (not found: rows before the first sequence)
    lo += last * step;
    len = min(step, len - last * step);
    if (step == 1) {
      row0 = __shfl_sync(0xffffffffu, row0, last);
      row1 = __shfl_sync(0xffffffffu, row1, last);
      L = __shfl_sync(0xffffffffu, L, last);
      break;
    }
  }
  const int64_t b = lo;
  const int64_t m = row1 - row0;
  // (the unit's place among its sequence's, and its block's first position)
  const int64_t nth = unit - first_unit_of<G>(row0, b);
  const int64_t p0 = L - m;
  // (nth < 0: the search was led astray by a cu_rows that decreases)
  bool write = found && m != 0;
  if (write && (m < 0 || nth < 0 || p0 < 0 || row0 < 0 || row1 > a.n ||
                L > a.kv.page_table_stride * a.kv.page_size)) {
    if (lane == 0 && a.status) atomicCAS(a.status, 0u, (unsigned)MLA_ERR_BOUNDS);
    write = false;
  }
  const int64_t start = write ? (p0 / G + nth) * G : 0;
  write = write && start < L;
  const int begin = write ? (int)start : 0;
  const int first = write ? max((int)p0 - begin, 0) : G;  // places below hold earlier positions
  const int end = write ? min(L - begin, G) : 0;          // and from here on none yet
  // every row of this warp's at once
  uint4 v0[C::kRows], v1[C::kRows];
  uint32_t pair[C::kRows];  // this lane's RoPE pair, the first entry in the low half
  int64_t position[C::kRows];
#pragma unroll
  for (int k = 0; k < C::kRows; ++k) {
    const int place = part * C::kRows + k;
    v0[k] = v1[k] = make_uint4(0, 0, 0, 0);
    pair[k] = 0;
    position[k] = 0;
    if (place >= first && place < end) {
      const int64_t i = row0 + (begin + place - p0);
      const uint16_t* row = a.x + i * a.x_stride;
      const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * lane;
      v0[k] = src[0], v1[k] = src[1];
      if (rope.interleaved)
        pair[k] = *reinterpret_cast<const uint32_t*>(row + kDV + 2 * lane);
      else
        pair[k] = row[kDV + lane] | (uint32_t)row[kDV + MLA_ROPE / 2 + lane] << 16;
      if (a.positions) position[k] = a.positions[a.axes.of(lane) * a.n + i];
    }
  }
  int64_t pool_row = 0;
  float old = 0.f;
  if (write) {
    const int64_t page = a.kv.page_table[b * a.kv.page_table_stride + (unsigned)begin / (unsigned)a.kv.page_size];
    write = page >= 0 && page < a.kv.num_pages;
    if (write) {
      pool_row = page * a.kv.page_size + (unsigned)begin % (unsigned)a.kv.page_size;
      if (first > 0) old = a.scale[pool_row / G];
    } else if (lane == 0 && part == 0 && a.status) {
      atomicCAS(a.status, 0u, (unsigned)MLA_ERR_BOUNDS);
    }
  }
  uint32_t g[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (a.weight) {
    const uint4* wp = reinterpret_cast<const uint4*>(a.weight) + 2 * lane;
    const uint4 g0 = __ldg(wp), g1 = __ldg(wp + 1);
    g[0] = g0.x, g[1] = g0.y, g[2] = g0.z, g[3] = g0.w;
    g[4] = g1.x, g[5] = g1.y, g[6] = g1.z, g[7] = g1.w;
  }
  __syncthreads();  // (the frequencies)
  float y[C::kRows][16];
  float2 pe[C::kRows];
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < C::kRows; ++k) {
    const uint32_t w[8] = {v0[k].x, v0[k].y, v0[k].z, v0[k].w, v1[k].x, v1[k].y, v1[k].z, v1[k].w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[k][2 * e] = __uint_as_float(w[e] << 16);
      y[k][2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    if (a.weight) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(y[k][e], y[k][e], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float norm = rsqrtf(ss * (1.0f / kDV) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[k][2 * e] = y[k][2 * e] * norm * __uint_as_float(g[e] << 16);
        y[k][2 * e + 1] = y[k][2 * e + 1] * norm * __uint_as_float(g[e] & 0xFFFF0000u);
      }
    }
    pe[k] = make_float2(__uint_as_float(pair[k] << 16), __uint_as_float(pair[k] & 0xFFFF0000u));
    if (a.positions)
      pe[k] = rope_turn(pe[k].x, pe[k].y, rope_cos_sin(s_turns[lane], position[k], rope.amplitude));
    // (fmaxf passes over NaN)
    top = fmaxf(top, fmaxf(fabsf(pe[k].x), fabsf(pe[k].y)));
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(y[k][e]));
  }
  if (top == INFINITY) {  // rare: the largest of the finite entries
    auto finite = [](float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.f; };
    top = 0.f;
#pragma unroll
    for (int k = 0; k < C::kRows; ++k) {
      top = fmaxf(top, fmaxf(finite(pe[k].x), finite(pe[k].y)));
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, finite(y[k][e]));
    }
  }
  // (bits of floats that are not negative order as they do)
  unsigned most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  if constexpr (C::kUnitWarps > 1) {
    if (lane == 0) s_top[warp] = most;
    __syncthreads();
    most = s_top[warp - part];
#pragma unroll
    for (int w = 1; w < C::kUnitWarps; ++w) most = max(most, s_top[warp - part + w]);
  }
  // (every warp of the unit has its `old` by now: it was read before the barrier, and the scale
  // is written after it)
  if (!write) return;
  float scale = scale_for(__uint_as_float(most));
  const bool was = is_scale(old);
  if (first > 0 && was) scale = fmaxf(scale, old);
  if (part == 0 && lane == 0) a.scale[pool_row / G] = scale;
  const float inv = 1.0f / scale;
  const bool power = (__float_as_int(scale) & 0x7FFFFF) == 0;  // (all but scales kept from elsewhere)
  uint8_t* dst0 = const_cast<uint8_t*>(a.kv.pool) + pool_row * kD;
#pragma unroll
  for (int k = 0; k < C::kRows; ++k) {
    const int place = part * C::kRows + k;
    uint8_t* dst = dst0 + place * kD;
    if (place < first) {
      if (scale != old) {  // earlier positions move to the block's new scale
        const float by = was ? old / scale : __int_as_float(0x7FC00000);
        uint4 c = reinterpret_cast<const uint4*>(dst)[lane];
        uint32_t t = *reinterpret_cast<const uint16_t*>(dst + kDV + 2 * lane);
        if ((__float_as_int(by) & 0x7FFFFF) == 0) {
          c = make_uint4(rescaled<true>(c.x, by), rescaled<true>(c.y, by), rescaled<true>(c.z, by), rescaled<true>(c.w, by));
          t = rescaled<true>(t, by);
        } else {
          c = make_uint4(rescaled<false>(c.x, by), rescaled<false>(c.y, by), rescaled<false>(c.z, by),
                         rescaled<false>(c.w, by));
          t = rescaled<false>(t, by);
        }
        reinterpret_cast<uint4*>(dst)[lane] = c;
        *reinterpret_cast<uint16_t*>(dst + kDV + 2 * lane) = (uint16_t)t;
      }
    } else if (place < end) {
      uint32_t code[4], pc;
      if (power) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          code[e] = e4m3x4(y[k][4 * e] * inv, y[k][4 * e + 1] * inv, y[k][4 * e + 2] * inv, y[k][4 * e + 3] * inv);
        pc = e4m3x2(pe[k].x * inv, pe[k].y * inv);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          code[e] = e4m3x4(quotient(y[k][4 * e], scale, inv), quotient(y[k][4 * e + 1], scale, inv),
                           quotient(y[k][4 * e + 2], scale, inv), quotient(y[k][4 * e + 3], scale, inv));
        pc = e4m3x2(quotient(pe[k].x, scale, inv), quotient(pe[k].y, scale, inv));
      }
      reinterpret_cast<uint4*>(dst)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
      if (!rope.interleaved) {
        // dims 2 l, 2 l + 1 of the row: first entries of two pairs (lanes below 16) or second ones
        const uint32_t q0 = __shfl_sync(0xffffffffu, pc, (2 * lane) & 31);
        const uint32_t q1 = __shfl_sync(0xffffffffu, pc, (2 * lane + 1) & 31);
        pc = lane < 16 ? (q0 & 0xFFu) | (q1 & 0xFFu) << 8 : (q0 >> 8) | (q1 & 0xFF00u);
      }
      *reinterpret_cast<uint16_t*>(dst + kDV + 2 * lane) = (uint16_t)pc;
    }
  }
}

template <int G>
cudaError_t launch_block(const AppendScaledArgs& a, const mla_rope_t& rope, cudaStream_t s) {
  using C = ScaledCfg<G>;
  const int64_t units = first_unit_of<G>(a.n, a.B);
  const int64_t grid = a.n == 0 ? 1 : (units + C::kUnits - 1) / C::kUnits;  // (no rows: the check of cu_rows alone)
  cache_append_scaled_kernel<G><<<(unsigned)grid, 32 * C::kWarps, 0, s>>>(a, rope);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append_scaled(const AppendScaledArgs& a, const mla_rope_t& rope, int block,
                                       cudaStream_t s) {
  switch (block) {
    case 1: return launch_block<1>(a, rope, s);
    case 2: return launch_block<2>(a, rope, s);
    case 4: return launch_block<4>(a, rope, s);
    case 8: return launch_block<8>(a, rope, s);
    case 16: return launch_block<16>(a, rope, s);
    case 32: return launch_block<32>(a, rope, s);
    case 64: return launch_block<64>(a, rope, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace mla
