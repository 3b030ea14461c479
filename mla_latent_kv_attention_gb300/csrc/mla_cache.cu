// mla_cache.cu -- writing new latent rows to the paged FP8 cache, and reading rows back.
//
// The step in front of decode, verify and prefill: the new positions' latent rows (576
// wide: 512 latent + 64 RoPE) are written into their cache slots as e4m3 codes under the
// cache's per-tensor scale, so that the attention kernels read them like every other
// cached row ("MI355X Kimi K2.5 vLLM AITER 7x speedup", section "PR #35850 修复了什么":
// the FP8 KV cache handled natively; "Scaling Kimi K3 on AMD Instinct MI355X", section
// "缓存可复用，还要能一致地恢复": 576 FP8 bytes per position).
//
// code = e4m3(x * inv_scale), both the reciprocal and the product rounded to binary32,
// the conversion rounding to nearest even and saturating at +-448. HBM-bound: 1,152 bytes
// read and 576 written per row, one warp per row, every access 16 bytes wide.
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

// bf16 pair (lo in the low half) scaled by inv -> two e4m3 codes (lo in the low byte)
__device__ __forceinline__ uint32_t quant2(uint32_t w, float inv) {
  const float lo = __uint_as_float(w << 16) * inv;
  const float hi = __uint_as_float(w & 0xFFFF0000u) * inv;
  return e4m3x2(lo, hi);
}

__global__ void __launch_bounds__(256) cache_append_kernel(uint8_t* __restrict__ pool,
                                                           int64_t pool_rows,
                                                           const uint16_t* __restrict__ x,
                                                           const int64_t* __restrict__ slots,
                                                           int64_t n, float inv,
                                                           unsigned* status) {
  const int lane = threadIdx.x & 31;
  const int64_t nwarps = ((int64_t)gridDim.x * blockDim.x) >> 5;
  for (int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5; i < n; i += nwarps) {
    const int64_t s = slots[i];
    if (s < 0) continue;  // padding: nothing to write
    if (s >= pool_rows) {
      if (lane == 0 && status) atomicCAS(status, 0u, (unsigned)MLA_ERR_BOUNDS);
      continue;
    }
    // 36 groups of 16 values: 32 bytes of bf16 in, 16 bytes of codes out
    const uint4* src = reinterpret_cast<const uint4*>(x + i * kD);
    uint4* dst = reinterpret_cast<uint4*>(pool + s * kD);
    for (int g = lane; g < kD / 16; g += 32) {
      const uint4 a = src[2 * g], b = src[2 * g + 1];
      uint4 c;
      c.x = quant2(a.x, inv) | (quant2(a.y, inv) << 16);
      c.y = quant2(a.z, inv) | (quant2(a.w, inv) << 16);
      c.z = quant2(b.x, inv) | (quant2(b.y, inv) << 16);
      c.w = quant2(b.z, inv) | (quant2(b.w, inv) << 16);
      dst[g] = c;
    }
  }
}

// Rows as the latent projection leaves them, one warp a row: lane l holds latent entries 16 l ..
// 16 l + 15 and RoPE pair l. y = c * rsqrt(mean(c^2) + eps) * w for the latent (the sum of
// squares of 512 float32 values over the lanes), the pair turned to its position, and
// e4m3(y * inv) for all 576, the only rounding: the values never pass through bf16, which a
// norm and a rotation run on their own would add.
//
// The frequencies lie in the parameters, where the 32 lanes' different addresses are read one
// after another: one warp of the CTA copies them to shared memory while every warp's row is on
// its way (8,192 rows 5.3 -> 4.3 us; copied before the loads 5.1). Bound: L2 or HBM for many rows
// (32,768, 56.6 MB: 10.9 us in L2, 14.2 us and 4.0 TB/s from HBM), the launch and two rounds of CTAs
// for fewer (8,192 rows are 1,024 CTAs, of which 608 run at once, each a chain of load, norm and
// write: 4.2 us in L2, 6.0 us from HBM), the launch alone for 32 (1.9 us). The half layout's two-byte
// loads and byte exchange add 0.4 to 0.6 us.
__global__ void __launch_bounds__(256, 4)  // (four: 8,192 rows 4.3 us; left open 4.85, six 4.9)
    cache_append_rope_kernel(const __grid_constant__ AppendRopeArgs a,
                             const __grid_constant__ mla_rope_t rope) {
  __shared__ uint64_t s_turns[MLA_ROPE / 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = blockDim.x >> 5;
  if (warp == 0) s_turns[lane] = rope.turns[lane];
  bool copied = false;  // s_turns seen by this warp (its CTA's warps turn alike through the loop)
  for (int64_t i0 = (int64_t)blockIdx.x * warps; i0 < a.n; i0 += (int64_t)gridDim.x * warps) {
    const int64_t i = i0 + warp;
    // every load of the row at once, its slot among them
    int64_t slot = -1, position = 0;
    uint4 v0 = make_uint4(0, 0, 0, 0), v1 = v0;
    uint32_t pair = 0;  // this lane's RoPE pair, the first entry in the low half
    if (i < a.n) {
      slot = a.slots[i];
      if (a.positions) position = a.positions[i];
      const uint16_t* row = a.x + i * a.x_stride;
      const uint4* src = reinterpret_cast<const uint4*>(row) + 2 * lane;
      v0 = src[0], v1 = src[1];
      if (rope.interleaved)
        pair = *reinterpret_cast<const uint32_t*>(row + kDV + 2 * lane);
      else
        pair = row[kDV + lane] | (uint32_t)row[kDV + MLA_ROPE / 2 + lane] << 16;
    }
    if (!copied) __syncthreads();
    copied = true;
    if (slot < 0) continue;  // padding: nothing to write
    if (slot >= a.pool_rows) {
      if (lane == 0 && a.status) atomicCAS(a.status, 0u, (unsigned)MLA_ERR_BOUNDS);
      continue;
    }
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    float c[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      c[2 * e] = __uint_as_float(w[e] << 16);
      c[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
    if (a.weight) {
      const uint4* wp = reinterpret_cast<const uint4*>(a.weight) + 2 * lane;
      const uint4 g0 = __ldg(wp), g1 = __ldg(wp + 1);
      const uint32_t g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) ss = fmaf(c[e], c[e], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = rsqrtf(ss * (1.0f / kDV) + a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[2 * e] = c[2 * e] * r * __uint_as_float(g[e] << 16);
        c[2 * e + 1] = c[2 * e + 1] * r * __uint_as_float(g[e] & 0xFFFF0000u);
      }
    }
    float2 pe = make_float2(__uint_as_float(pair << 16), __uint_as_float(pair & 0xFFFF0000u));
    if (a.positions)
      pe = rope_turn(pe.x, pe.y, rope_cos_sin(s_turns[lane], position, rope.amplitude));
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      code[e] = e4m3x2(c[4 * e] * a.inv, c[4 * e + 1] * a.inv) |
                e4m3x2(c[4 * e + 2] * a.inv, c[4 * e + 3] * a.inv) << 16;
    uint8_t* dst = a.pool + slot * kD;
    reinterpret_cast<uint4*>(dst)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
    uint32_t pc = e4m3x2(pe.x * a.inv, pe.y * a.inv);
    if (!rope.interleaved) {
      // dims 2 l, 2 l + 1 of the row: first entries of two pairs (lanes below 16) or second ones
      const uint32_t p0 = __shfl_sync(0xffffffffu, pc, (2 * lane) & 31);
      const uint32_t p1 = __shfl_sync(0xffffffffu, pc, (2 * lane + 1) & 31);
      pc = lane < 16 ? (p0 & 0xFFu) | (p1 & 0xFFu) << 8 : (p0 >> 8) | (p1 & 0xFF00u);
    }
    *reinterpret_cast<uint16_t*>(dst + kDV + 2 * lane) = (uint16_t)pc;
  }
}

// Cached rows back into a dense array. A CTA takes 32 consecutive output rows: first a thread a
// row finds its sequence (binary search in cu_rows), its page and the pool row, then the threads
// move the rows 16 bytes of output at a time (8 codes to bf16, four rows a round, or 4 codes to
// float32, two rows a round: a warp's stores are whole lines), every load of a thread in flight
// before its first store. HBM-bound: 576 bytes read and 1,152 (bf16) or 2,304 (float32) written a
// row: 8 x 32,768 rows to bf16 in 70 us (453 MB, 6.5 TB/s, 0.95 of the measured copy), 66,000 rows
// to float32 in 31.4 us (190 MB, 6.1 TB/s; with 8 codes a thread, two stores each, 44.2 us), 8 x
// 333 to bf16 in 4.1 us (the launch and three dependent loads).
constexpr int kGatherRows = 32;
constexpr int kGatherThreads = 288;
constexpr int64_t kRowSkip = -1, kRowBad = -2;

template <typename Out>
__global__ void __launch_bounds__(kGatherThreads)
    cache_gather_kernel(const __grid_constant__ mla_kv_t kv, int B, const int32_t* __restrict__ starts,
                        const int64_t* __restrict__ cu_rows, int64_t n, Out* __restrict__ out,
                        unsigned* status) {
  __shared__ int64_t s_row[kGatherRows];  // pool row, or kRowSkip / kRowBad
  const int64_t row0 = (int64_t)blockIdx.x * kGatherRows;
  if (threadIdx.x < kGatherRows) {
    const int64_t row = row0 + threadIdx.x;
    int64_t from = kRowSkip;
    if (row < n && row >= cu_rows[0] && row < cu_rows[B]) {
      int lo = 0, hi = B;  // cu_rows[lo] <= row < cu_rows[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_rows[mid] <= row)
          lo = mid;
        else
          hi = mid;
      }
      const int64_t pos = row - cu_rows[lo] + (starts ? starts[lo] : 0);
      from = kRowBad;
      if (pos >= 0 && pos < kv.seq_lens[lo] && pos / kv.page_size < kv.page_table_stride) {
        const int64_t page = kv.page_table[lo * kv.page_table_stride + pos / kv.page_size];
        if (page >= 0 && page < kv.num_pages) from = page * kv.page_size + pos % kv.page_size;
      }
      if (from == kRowBad && status) atomicCAS(status, 0u, (unsigned)MLA_ERR_BOUNDS);
    }
    s_row[threadIdx.x] = from;
  }
  __syncthreads();
  constexpr int kCodes = 16 / sizeof(Out);          // a thread's piece of a row
  constexpr int kPieces = kD / kCodes;
  constexpr int kAtOnce = kGatherThreads / kPieces;  // rows a round
  constexpr int kRounds = kGatherRows / kAtOnce;
  const int r = threadIdx.x / kPieces, piece = threadIdx.x % kPieces;
  uint32_t code[kRounds][kCodes / 4];
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    const int64_t from = s_row[kAtOnce * k + r];
#pragma unroll
    for (int e = 0; e < kCodes / 4; ++e) code[k][e] = 0u;
    if (from < 0) continue;
    const uint8_t* src = kv.pool + from * kD + kCodes * piece;
    if constexpr (kCodes == 8) {
      const uint2 c = __ldcs(reinterpret_cast<const uint2*>(src));
      code[k][0] = c.x;
      code[k][kCodes / 4 - 1] = c.y;
    } else {
      code[k][0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
    }
  }
#pragma unroll
  for (int k = 0; k < kRounds; ++k) {
    if (s_row[kAtOnce * k + r] == kRowSkip) continue;
    float2 v[kCodes / 2];
#pragma unroll
    for (int e = 0; e < kCodes / 2; ++e) {
      const uint32_t two = (e & 1) ? code[k][e / 2] >> 16 : code[k][e / 2] & 0xFFFFu;
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
      v[e] = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[e].x *= kv.kv_scale;
      v[e].y *= kv.kv_scale;
    }
    Out* dst = out + (row0 + kAtOnce * k + r) * kD + kCodes * piece;
    if constexpr (kCodes == 4) {
      __stcs(reinterpret_cast<float4*>(dst), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    } else {
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[e].x, v[e].y);
        o[e] = *reinterpret_cast<const uint32_t*>(&t);
      }
      __stcs(reinterpret_cast<uint4*>(dst), make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

}  // namespace

cudaError_t launch_cache_append_rope(const AppendRopeArgs& a, const mla_rope_t& rope, int num_sms,
                                     cudaStream_t s) {
  // one warp per row, at most 8 CTAs per SM (of which four run at once)
  const int64_t blocks = (a.n * 32 + 255) / 256;
  const int grid = (int)(blocks < (int64_t)num_sms * 8 ? blocks : (int64_t)num_sms * 8);
  cache_append_rope_kernel<<<grid, 256, 0, s>>>(a, rope);
  return cudaGetLastError();
}

cudaError_t launch_cache_gather(const mla_kv_t& kv, int B, const int32_t* starts,
                                const int64_t* cu_rows, int64_t n, void* out, int out_f32,
                                unsigned* status, cudaStream_t s) {
  const unsigned grid = (unsigned)((n + kGatherRows - 1) / kGatherRows);
  if (out_f32)
    cache_gather_kernel<float><<<grid, kGatherThreads, 0, s>>>(kv, B, starts, cu_rows, n,
                                                               static_cast<float*>(out), status);
  else
    cache_gather_kernel<uint16_t><<<grid, kGatherThreads, 0, s>>>(kv, B, starts, cu_rows, n,
                                                                  static_cast<uint16_t*>(out), status);
  return cudaGetLastError();
}

cudaError_t launch_cache_append(uint8_t* pool, int64_t pool_rows, const uint16_t* x,
                                const int64_t* slots, int64_t n, float inv, unsigned* status,
                                int num_sms, cudaStream_t s) {
  const int64_t blocks = (n * 32 + 255) / 256;  // one warp per row, at most 8 CTAs per SM
  const int grid = (int)(blocks < (int64_t)num_sms * 8 ? blocks : (int64_t)num_sms * 8);
  cache_append_kernel<<<grid, 256, 0, s>>>(pool, pool_rows, x, slots, n, inv, status);
  return cudaGetLastError();
}

}  // namespace mla
