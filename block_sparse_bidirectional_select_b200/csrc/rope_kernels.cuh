// Rotary positions with several axes (time, height, width of a token), applied
// to the heads of a projection's output on their way to the [H, L, d] layout
// of the attention entry points.
//
// Pair j of a head (J pairs, 2J <= d) belongs to one axis and turns by
// t = position[axis][l] * inv_j:
//   a' = a cos t - b sin t,   b' = b cos t + a sin t
// with (a, b) = elements (j, J + j), or (2j, 2j + 1) when interleaved; the
// elements from 2J on are copied.
//
// The angle. inv_j / 2 pi is given as a 64-bit binary fraction of a turn, so
// position * fraction in 64-bit integers drops whole turns exactly. An fp32
// product would be off by position * 2^-24 (0.06 rad at a position of 10^6);
// this one is off by position * 2^-53 turns at most. The nearest quarter turn
// is taken off in integers too, before the rest becomes an fp32: so the sine
// and the cosine are right to a few fp32 roundings of themselves, also where
// they are nearly 0 (the hardware sine of the whole angle is off by 2^-21 of 1,
// more than a bf16 step of a result below 2^-12, for 2% less time).
#pragma once

#include "ptx_sm100.cuh"

namespace sparsed {

constexpr int kRopeMaxPairs = 128;
constexpr int kRopeMaxAxes = 8;
constexpr int kRopeThreads = 256;

struct RopeArgs {
  const uint16_t* x;
  uint16_t* y;
  const int32_t* pos;           // [n_axes, L]
  size_t xs_h, xs_l, ys_h, ys_l;  // strides in elements
  int H, L, d, J;
  int units;                    // work units of a token and head: rotated ones, then copied ones
  int rot_units;
  int heads_per_cta;
  int sign;                     // +1, or -1 for the inverse rotation
  uint64_t turn[kRopeMaxPairs];  // inv_j / 2 pi as a fraction of 2^64
  uint8_t axis[kRopeMaxPairs];
};

__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 f32_to_bf16x8(const float (&f)[8]) {
  return make_uint4(ptx::pack_bf16x2(f[0], f[1]), ptx::pack_bf16x2(f[2], f[3]), ptx::pack_bf16x2(f[4], f[5]),
                    ptx::pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  return static_cast<uint16_t>(ptx::pack_bf16x2(f, 0.f) & 0xFFFFu);
}

// Sine and cosine of turns / 2^64 turns: of the angle t left by the nearest
// quarter turn, |t| <= pi / 4, by their Taylor series up to t^9 and t^8, which
// end 2.5e-9 (of the sine) and 2.5e-8 from them.
__device__ __forceinline__ void turn_sincos(uint64_t turns, float& sn, float& cs) {
  const uint32_t quarter = static_cast<uint32_t>((turns + (1ull << 61)) >> 62);  // mod 4
  const int64_t rest = static_cast<int64_t>(turns - (static_cast<uint64_t>(quarter) << 62));
  const float t = static_cast<float>(rest) * (0x1p-64f * 6.283185307179586f), w = t * t;
  const float s = fmaf(fmaf(fmaf(fmaf(1.f / 362880, w, -1.f / 5040), w, 1.f / 120), w, -1.f / 6) * w, t, t);
  const float c = fmaf(fmaf(fmaf(fmaf(1.f / 40320, w, -1.f / 720), w, 1.f / 24), w, -0.5f), w, 1.f);
  sn = quarter & 1 ? c : s;
  cs = quarter & 1 ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cs = -cs;
}

// A thread owns one unit of eight pairs of one token: it takes their sines and
// cosines once and turns that unit of every head of its CTA's share. VEC: all
// addresses are 16-byte aligned and, with split halves, J is a multiple of 8,
// so a unit is two 16-byte loads and stores; otherwise element by element.
// Bound by memory: 2 bytes read and written per element. 32768 tokens of 32
// heads (537 MB) take 97 us, 5.5 TB/s, 86% of a copy (95 us with the hardware's
// sine and cosine); a CTA of few heads pays its sines again (16, 8, 4, 2 heads:
// 97, 99, 104, 141 us).
template <bool INTERLEAVED, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_axes_kernel(const __grid_constant__ RopeArgs a) {
  const int tokens = kRopeThreads / a.units;
  const int tok = threadIdx.x / a.units;
  const int unit = threadIdx.x - tok * a.units;
  const long l = static_cast<long>(blockIdx.x) * tokens + tok;
  if (tok >= tokens || l >= a.L) return;
  const int h0 = blockIdx.y * a.heads_per_cta;
  const int h1 = min(a.H, h0 + a.heads_per_cta);
  const uint16_t* x = a.x + l * a.xs_l;
  uint16_t* y = a.y + l * a.ys_l;
  if (unit >= a.rot_units) {
    const int e0 = 2 * a.J + (unit - a.rot_units) * 8;
    const int n = min(8, a.d - e0);
    for (int h = h0; h < h1; ++h)
      for (int e = 0; e < n; ++e) y[h * a.ys_h + e0 + e] = x[h * a.xs_h + e0 + e];
    return;
  }
  const int j0 = unit * 8;
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int j = min(j0 + e, a.J - 1);
    const long p = a.pos[static_cast<long>(a.axis[j]) * a.L + l] * static_cast<long>(a.sign);
    const uint64_t turns = static_cast<uint64_t>(p) * a.turn[j];
    turn_sincos(turns, sn[e], cs[e]);
  }
  if constexpr (VEC) {
    // the unit's two 16-byte parts
    const int o0 = INTERLEAVED ? 2 * j0 : j0;
    const int o1 = INTERLEAVED ? 2 * j0 + 8 : a.J + j0;
#pragma unroll 4
    for (int h = h0; h < h1; ++h) {
      const uint16_t* xh = x + h * a.xs_h;
      float u[8], v[8], p[8], q[8];
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(xh + o0), u);
      bf16x8_to_f32(*reinterpret_cast<const uint4*>(xh + o1), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (INTERLEAVED) {
          // pair e: elements 2e, 2e+1 of the 16 in (u, v)
          const float ea = e < 4 ? u[(2 * e) & 7] : v[(2 * e) & 7];
          const float eb = e < 4 ? u[(2 * e + 1) & 7] : v[(2 * e + 1) & 7];
          const float ra = ea * cs[e] - eb * sn[e], rb = eb * cs[e] + ea * sn[e];
          if (e < 4) p[(2 * e) & 7] = ra, p[(2 * e + 1) & 7] = rb;
          else q[(2 * e) & 7] = ra, q[(2 * e + 1) & 7] = rb;
        } else {
          p[e] = u[e] * cs[e] - v[e] * sn[e];
          q[e] = v[e] * cs[e] + u[e] * sn[e];
        }
      }
      uint16_t* yh = y + h * a.ys_h;
      *reinterpret_cast<uint4*>(yh + o0) = f32_to_bf16x8(p);
      *reinterpret_cast<uint4*>(yh + o1) = f32_to_bf16x8(q);
    }
  } else {
    for (int h = h0; h < h1; ++h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + e;
        if (j >= a.J) break;
        const int oa = INTERLEAVED ? 2 * j : j, ob = INTERLEAVED ? 2 * j + 1 : a.J + j;
        const float ea = bf16_to_f32(x[h * a.xs_h + oa]), eb = bf16_to_f32(x[h * a.xs_h + ob]);
        y[h * a.ys_h + oa] = f32_to_bf16(ea * cs[e] - eb * sn[e]);
        y[h * a.ys_h + ob] = f32_to_bf16(eb * cs[e] + ea * sn[e]);
      }
    }
  }
}

}  // namespace sparsed
