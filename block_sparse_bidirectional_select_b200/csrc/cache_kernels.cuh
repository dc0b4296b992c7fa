// The 8-bit cache of keys and values: e4m3 values with one power-of-two scale
// for each block of 64 tokens and head, K and V apart.
//
//   cache value = e4m3 * 2^e,   e = the block's exponent, -117 <= e <= 119
//
// A power of two costs e4m3 nothing but range below its normal numbers (its
// relative step does not depend on the scale) and buys three things: scaling
// and unscaling are exact, a block whose scale grows keeps its older values
// bit for bit unless they leave the normal range, and attention can fold the
// scales into exponents. The bounds keep 448 * 2^e finite and the smallest
// step 2^-9 * 2^e normal in bf16 and fp32.
#pragma once

#include "ptx_sm100.cuh"
#include "rope_kernels.cuh"

namespace sparsed {

constexpr int kCacheBlock = 64;
constexpr int kCacheEMin = -117;
constexpr int kCacheEMax = 119;

// 2^e for -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// exponent of a scale, whatever the memory holds
__device__ __forceinline__ int scale_exponent(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 255u) - 127;
  return min(max(e, kCacheEMin), kCacheEMax);
}

// The smallest e with amax <= 448 * 2^e (448 = 1.75 * 2^8); amax a finite bf16
// in its 15 magnitude bits.
__device__ __forceinline__ int exponent_for(uint32_t amax15) {
  const int x = static_cast<int>(amax15 >> 7) - 127;       // amax = m * 2^x
  const int e = x - 8 + ((amax15 & 0x7Fu) > 0x60u ? 1 : 0);  // m > 1.75
  return min(max(e, kCacheEMin), kCacheEMax);
}

// Two fp32 to e4m3 (nearest even, beyond the range to +-448), `lo` in bits 0..7.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 to fp32 (exact).
__device__ __forceinline__ void unpack_e4m3x2(uint32_t v, float& lo, float& hi) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(v)));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h2));
}

struct AppendArgs {
  const uint16_t* x[2];          // new K, V
  size_t s_n[2], s_h[2], s_b[2];  // strides in elements
  uint8_t* x8[2];                // [N, H, C, d]
  float* scale[2];               // [N, H, C / 64]
  const int32_t* start;          // [N]
  const int32_t* count;          // [N], or null: B
  int N, H, B, C;
};

// One CTA per (touched block of 64 tokens, K or V, head, sequence): the
// block's new values stay in registers between the maximum and the rounding,
// so every input is read once and every output written once. Tokens of the
// block before `start` are rounded again only where the scale grew; bytes at
// and past the last new token are left as they are. VEC: 16-byte loads.
// Bound by memory: 2 bytes read and 1 written per element. Two prompts of 16384
// tokens and 32 heads (805 MB) take 127 us, 6.3 TB/s, 98% of a copy; with the
// maximum taken one value at a time the ALU was 77% busy and it took 133 us.
template <int D, bool VEC>
__global__ void __launch_bounds__(256) cache_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int TPR = D / 8;        // threads of a token's row, 8 elements each
  constexpr int ROWS = 256 / TPR;   // rows of a pass
  constexpr int NP = kCacheBlock / ROWS;
  __shared__ uint32_t s_max[8];
  const int which = blockIdx.x & 1;
  const int h = blockIdx.y, n = blockIdx.z;
  const int start = a.start[n];
  const int count = a.count ? a.count[n] : a.B;
  if (start < 0 || count < 0 || count > a.B || start > a.C - count) {
    if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) ptx::record_error(kErrBadPattern);
    return;
  }
  const int end = start + count;
  const int blk = start / kCacheBlock + (blockIdx.x >> 1);
  const int t0 = blk * kCacheBlock;
  if (t0 >= end || count == 0) return;
  const int row0 = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * 8;
  const uint16_t* src = a.x[which] + n * a.s_n[which] + h * a.s_h[which] + c0;
  uint8_t* dst = a.x8[which] + ((static_cast<long>(n) * a.H + h) * a.C + t0) * D + c0;
  float* scale = a.scale[which] + (static_cast<long>(n) * a.H + h) * (a.C / kCacheBlock) + blk;
  uint4 v[NP];
  uint32_t mx = 0;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int t = t0 + row0 + p * ROWS;
    v[p] = make_uint4(0, 0, 0, 0);
    if (t >= start && t < end) {
      const uint16_t* s = src + static_cast<long>(t - start) * a.s_b[which];
      if constexpr (VEC) {
        v[p] = *reinterpret_cast<const uint4*>(s);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = s[2 * e] | (static_cast<uint32_t>(s[2 * e + 1]) << 16);
        v[p] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  const float held = *scale;  // of a block that holds older tokens
  // magnitudes as 16-bit integers, two to a word (two operations for two values)
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) mx = __vmaxu2(mx, w[e] & 0x7FFF7FFFu);
  }
  mx = max(mx & 0xFFFFu, mx >> 16);
  if (mx >= 0x7F80u) {  // an infinity or NaN among them: the maximum of the finite ones
    mx = 0;
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7FFFu, hi = (w[e] >> 16) & 0x7FFFu;
        mx = max(mx, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
      }
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = mx;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) mx = max(mx, s_max[w]);
  int e = exponent_for(mx);
  const bool older = t0 < start;
  const int e_old = scale_exponent(held);
  if (older) e = max(e, e_old);
  const float inv = pow2i(-e);
  // older tokens, where the scale grew: a step of 2^-126 or less leaves nothing
  const bool regrade = older && e > e_old;
  const float step = e - e_old > 126 ? 0.f : pow2i(e_old - e);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = row0 + p * ROWS, t = t0 + r;
    uint2* out = reinterpret_cast<uint2*>(dst + static_cast<long>(r) * D);
    if (t >= start && t < end) {
      float f[8];
      bf16x8_to_f32(v[p], f);
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] *= inv;
      *out = make_uint2(pack_e4m3x2(f[0], f[1]) | (pack_e4m3x2(f[2], f[3]) << 16),
                        pack_e4m3x2(f[4], f[5]) | (pack_e4m3x2(f[6], f[7]) << 16));
    } else if (regrade && t < start) {
      const uint2 o = *out;
      uint32_t w[4] = {o.x & 0xFFFFu, o.x >> 16, o.y & 0xFFFFu, o.y >> 16};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float lo, hi;
        unpack_e4m3x2(w[u], lo, hi);
        w[u] = pack_e4m3x2(lo * step, hi * step);
      }
      *out = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    }
  }
  // every thread read the old scale before the barrier above
  if (threadIdx.x == 0) *scale = pow2i(e);
}

}  // namespace sparsed
