// mla_rope.cu -- rotary positions of the 64 RoPE dims: the frequencies (host) and the rotation
// of the queries' RoPE parts.
//
// A thread takes a quarter of a token's 64 dims (eight pairs, two 16-byte vectors) and turns it
// in several heads: the eight angles belong to the token, so their cosines and sines are
// computed once for all the heads that the thread takes. Bound: 256 bytes a head through L2 and
// HBM when there are many tokens (8,192 of 12 heads, 25.2 MB: 6.5 us and 3.9 TB/s from HBM; in L2
// 4.5 us in the half layout, 5.4 us interleaved), the launch when there are few (32: 1.8 us).
#include <cuda_bf16.h>
#include <math.h>

#include "mla_internal.cuh"
#include "mla_rope.cuh"

namespace mla {
namespace {

constexpr int kRopeThreads = 128;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// HEADS: heads a thread turns (loads of all of them in flight together).
// AXES: positions [axes][n], each pair by its own axis' (its position is loaded where it is used:
// the quarter's eight pairs read at most four words, in flight with x; 8,192 tokens of 12 heads 6.5 us
// from HBM, 4.6 us in L2, half layout, 32 tokens 1.95 us: as with one axis, to 0.1 us).
template <bool INTERLEAVED, int HEADS, bool AXES>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ mla_rope_t rope, const PairAxes axes, const uint16_t* x,
                int64_t x_token, int64_t x_head, const int64_t* __restrict__ positions, int64_t n, int H,
                uint16_t* out, int64_t out_token, int64_t out_head) {
  const int parts = (H + HEADS - 1) / HEADS;
  const int64_t item = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 2;
  const int quarter = threadIdx.x & 3;
  const int64_t token = item / parts;
  if (token >= n) return;
  const int h0 = (int)(item % parts) * HEADS;
  // the thread's two vectors: neighbours (interleaved pairs), or 32 dims apart (half layout)
  const int d0 = INTERLEAVED ? 16 * quarter : 8 * quarter;
  const int d1 = INTERLEAVED ? d0 + 8 : d0 + 32;
  const uint16_t* src = x + token * x_token + h0 * x_head;
  uint16_t* dst = out + token * out_token + h0 * out_head;
  uint4 a[HEADS], b[HEADS];
#pragma unroll
  for (int h = 0; h < HEADS; ++h)
    if (h0 + h < H) {
      a[h] = *reinterpret_cast<const uint4*>(src + h * x_head + d0);
      b[h] = *reinterpret_cast<const uint4*>(src + h * x_head + d1);
    }
  float2 cs[8];
  if constexpr (AXES) {
    int64_t position[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) position[i] = positions[axes.of(8 * quarter + i) * n + token];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = rope_cos_sin(rope.turns[8 * quarter + i], position[i], rope.amplitude);
  } else {
    const int64_t position = positions[token];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = rope_cos_sin(rope.turns[8 * quarter + i], position, rope.amplitude);
  }
#pragma unroll
  for (int h = 0; h < HEADS; ++h) {
    if (h0 + h >= H) break;
    uint32_t u[4] = {a[h].x, a[h].y, a[h].z, a[h].w}, v[4] = {b[h].x, b[h].y, b[h].z, b[h].w};
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = rope_turn(bf16_lo(u[i]), bf16_hi(u[i]), cs[i]);
        const float2 q = rope_turn(bf16_lo(v[i]), bf16_hi(v[i]), cs[4 + i]);
        u[i] = pack_bf16(p.x, p.y);
        v[i] = pack_bf16(q.x, q.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = rope_turn(bf16_lo(u[i]), bf16_lo(v[i]), cs[2 * i]);
        const float2 q = rope_turn(bf16_hi(u[i]), bf16_hi(v[i]), cs[2 * i + 1]);
        u[i] = pack_bf16(p.x, q.x);
        v[i] = pack_bf16(p.y, q.y);
      }
    }
    *reinterpret_cast<uint4*>(dst + h * out_head + d0) = make_uint4(u[0], u[1], u[2], u[3]);
    *reinterpret_cast<uint4*>(dst + h * out_head + d1) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

}  // namespace

template <bool AXES>
static cudaError_t launch_rope_with(const mla_rope_t& rope, PairAxes axes, const uint16_t* x, int64_t x_token,
                                    int64_t x_head, const int64_t* positions, int64_t n, int H, uint16_t* out,
                                    int64_t out_token, int64_t out_head, int num_sms, cudaStream_t s) {
  // Four heads a thread share their angles. Where that would leave an SM with less than two
  // warps, one head a thread: more threads, each with a shorter wait. In us, one / four, at 12
  // heads, interleaved, in L2: 32 tokens 1.9 / 2.3, 512 2.2 / 2.3, 1,024 2.4 / 2.4, 4,096 4.3 / 3.8, 8,192 7.0 / 5.4;
  // 8 heads cross at 1,024 tokens too, 16 heads at 800.
  const bool many = n * ((H + 3) / 4) * 4 >= (int64_t)num_sms * 2 * 32;
  const int heads = many ? 4 : 1;
  const int64_t threads = n * ((H + heads - 1) / heads) * 4;
  const unsigned grid = (unsigned)((threads + kRopeThreads - 1) / kRopeThreads);
  auto go = [&](auto kernel) {
    kernel<<<grid, kRopeThreads, 0, s>>>(rope, axes, x, x_token, x_head, positions, n, H, out, out_token,
                                         out_head);
  };
  if (rope.interleaved) {
    if (many)
      go(rope_kernel<true, 4, AXES>);
    else
      go(rope_kernel<true, 1, AXES>);
  } else {
    if (many)
      go(rope_kernel<false, 4, AXES>);
    else
      go(rope_kernel<false, 1, AXES>);
  }
  return cudaGetLastError();
}

cudaError_t launch_rope(const mla_rope_t& rope, const PairAxes* axes, const uint16_t* x, int64_t x_token,
                        int64_t x_head, const int64_t* positions, int64_t n, int H, uint16_t* out,
                        int64_t out_token, int64_t out_head, int num_sms, cudaStream_t s) {
  if (axes)
    return launch_rope_with<true>(rope, *axes, x, x_token, x_head, positions, n, H, out, out_token, out_head,
                                  num_sms, s);
  return launch_rope_with<false>(rope, PairAxes{0}, x, x_token, x_head, positions, n, H, out, out_token,
                                 out_head, num_sms, s);
}

}  // namespace mla

extern "C" mla_status_t mla_rope_init(mla_rope_t* rope, double base, double factor,
                                      int original_positions, double beta_fast, double beta_slow,
                                      float amplitude, int interleaved) {
  constexpr double kPi = 3.14159265358979323846;
  constexpr int kPairs = MLA_ROPE / 2;
  if (!rope || !(base > 1.0) || !isfinite(base) || !(factor > 0.0) || !isfinite(factor) ||
      original_positions < 0 || !isfinite(amplitude))
    return MLA_ERR_INVALID_ARG;
  double low = 0.0, high = 0.0;
  if (original_positions > 0) {
    if (!(beta_slow > 0.0) || !(beta_fast > beta_slow) || !isfinite(beta_fast)) return MLA_ERR_INVALID_ARG;
    // the (fractional) pair that turns `r` times over the original positions:
    // original * base^(-2i / 64) / (2 pi) = r
    auto pair_of = [&](double r) {
      return MLA_ROPE * log(original_positions / (r * 2.0 * kPi)) / (2.0 * log(base));
    };
    low = fmax(floor(pair_of(beta_fast)), 0.0);
    high = fmin(ceil(pair_of(beta_slow)), (double)(MLA_ROPE - 1));
  }
  for (int i = 0; i < kPairs; ++i) {
    const double f = pow(base, -2.0 * i / MLA_ROPE);
    double stretched = 1.0;  // share of f / factor
    if (original_positions > 0) stretched = fmin(fmax((i - low) / fmax(high - low, 0.001), 0.0), 1.0);
    const double turn = (f / factor * stretched + f * (1.0 - stretched)) / (2.0 * kPi);
    if (!isfinite(turn)) return MLA_ERR_INVALID_ARG;  // f / factor is past float64
    // whole turns drop out (positions are whole); the rest lies in [0, 1) and is rounded to nearest
    // (from 2^-11 up it is a multiple of 2^-64 already)
    rope->turns[i] = (uint64_t)nearbyint(ldexp(turn - floor(turn), 64));
  }
  rope->amplitude = amplitude;
  rope->interleaved = interleaved != 0;
  return MLA_OK;
}

extern "C" mla_status_t mla_rope_axes_init(mla_rope_axes_t* axes, const int32_t* sections, int n_axes,
                                           int interleaved) {
  constexpr int kPairs = MLA_ROPE / 2;
  if (!axes || !sections || n_axes < 1 || n_axes > MLA_MAX_AXES) return MLA_ERR_INVALID_ARG;
  int left[MLA_MAX_AXES] = {0}, sum = 0;
  for (int a = 0; a < n_axes; ++a) {
    if (sections[a] < 0 || sections[a] > kPairs) return MLA_ERR_INVALID_ARG;
    left[a] = sections[a];
    sum += sections[a];
  }
  if (sum != kPairs) return MLA_ERR_INVALID_ARG;
  int a = interleaved ? n_axes - 1 : 0;  // the axis of the pair before
  for (int i = 0; i < kPairs; ++i) {
    if (interleaved) a = (a + 1) % n_axes;
    while (left[a] == 0) a = (a + 1) % n_axes;
    axes->axis[i] = (uint8_t)a;
    --left[a];
  }
  axes->n_axes = n_axes;
  return MLA_OK;
}
