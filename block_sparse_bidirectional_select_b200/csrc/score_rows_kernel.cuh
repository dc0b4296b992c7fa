// Attention with modified scores, one query row per CTA on the CUDA cores: the
// simple form of scored_attn and cache_attn.
//   x = scale * <q, k_c>; capped: x = cap * tanh(x / cap); biased: x -= slope * |at - c|
#pragma once

#include "cache_kernels.cuh"

namespace sparsed {

struct ScoreMod {
  float scale;
  float softcap;        // 0: none
  const float* slopes;  // [Hq], or null
};

struct RowsArgs {
  const uint16_t* q;
  size_t qs_n, qs_h, qs_b;
  // bf16 keys and values (k8 == nullptr) ...
  const uint16_t *k, *v;
  size_t ks_h, ks_l, vs_h, vs_l;
  // ... or the 8-bit cache
  const uint8_t *k8, *v8;
  const float *k_scale, *v_scale;
  int N, Hq, Hkv, B, Lk;       // Lk: keys, or the cache's capacity
  const int32_t* lengths;      // [N] (cache)
  const int32_t* q_start;      // [N] or null
  int q_start0;
  const int32_t* ranges;       // [B, 2] or null
  ScoreMod mod;
  uint16_t* o;                 // [N, Hq, B, D]
  float* lse;                  // [N, Hq, B]
};

template <int D>
__global__ void __launch_bounds__(128) score_rows_kernel(const __grid_constant__ RowsArgs a) {
  __shared__ float s_q[D];
  __shared__ float s_p[128];
  __shared__ float s_red[4];
  __shared__ float s_o[D];
  const int b = blockIdx.x, h = blockIdx.y, n = blockIdx.z;
  const int tid = threadIdx.x;
  const int hk = h / (a.Hq / a.Hkv);
  const float ninf = -__int_as_float(0x7f800000);
  for (int e = tid; e < D; e += 128) s_q[e] = bf16_to_f32(a.q[n * a.qs_n + h * a.qs_h + b * a.qs_b + e]);
  int lo = 0, hi = a.Lk, at = a.q_start0 + b;
  if (a.lengths) {
    hi = min(max(a.lengths[n], 0), a.Lk);
    at = (a.q_start ? a.q_start[n] : hi - a.B) + b;
  }
  if (a.ranges) {
    lo = max(a.ranges[2 * b], 0);
    hi = min(a.ranges[2 * b + 1], a.Lk);
  }
  const float slope = a.mod.slopes ? a.mod.slopes[h] : 0.f;
  const long base = (static_cast<long>(n) * a.Hkv + hk) * a.Lk;
  const long sbase = (static_cast<long>(n) * a.Hkv + hk) * (a.Lk / kCacheBlock);
  float m = ninf, l = 0.f, acc = 0.f;  // acc: element tid of the row (tid < D)
  __syncthreads();
  for (int c0 = lo; c0 < hi; c0 += 128) {
    const int c = c0 + tid;
    float x = ninf;
    if (c < hi) {
      float dot = 0.f;
      if (a.k8) {
        const uint8_t* k = a.k8 + (base + c) * D;
        for (int e = 0; e < D; e += 2) {
          float f0, f1;
          unpack_e4m3x2(*reinterpret_cast<const uint16_t*>(k + e), f0, f1);
          dot += s_q[e] * f0 + s_q[e + 1] * f1;
        }
        dot *= pow2i(scale_exponent(a.k_scale[sbase + c / kCacheBlock]));
      } else {
        const uint16_t* k = a.k + hk * a.ks_h + c * a.ks_l;
        for (int e = 0; e < D; ++e) dot += s_q[e] * bf16_to_f32(k[e]);
      }
      x = dot * a.mod.scale;
      if (a.mod.softcap > 0.f) x = a.mod.softcap * tanhf(x / a.mod.softcap);
      if (a.mod.slopes) x -= slope * fabsf(static_cast<float>(at - c));
    }
    float mx = x;
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    if ((tid & 31) == 0) s_red[tid >> 5] = mx;
    __syncthreads();
    const float m_new = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float m_use = m_new == ninf ? 0.f : m_new;
    const float p = expf(x - m_use);
    const float alpha = expf(m - m_use);
    s_p[tid] = p;
    float ps = p;
    for (int off = 16; off > 0; off >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, off);
    __syncthreads();
    if ((tid & 31) == 0) s_red[tid >> 5] = ps;
    __syncthreads();
    l = l * alpha + ((s_red[0] + s_red[1]) + (s_red[2] + s_red[3]));
    m = m_new;
    acc *= alpha;
    if (tid < D) {
      for (int u = 0; u < 128 && c0 + u < hi; ++u) {
        const int cc = c0 + u;
        float vv;
        if (a.k8) {
          float f0, f1;
          unpack_e4m3x2(a.v8[(base + cc) * D + tid], f0, f1);
          vv = f0 * pow2i(scale_exponent(a.v_scale[sbase + cc / kCacheBlock]));
        } else {
          vv = bf16_to_f32(a.v[hk * a.vs_h + cc * a.vs_l + tid]);
        }
        acc += s_p[u] * vv;
      }
    }
    __syncthreads();
  }
  const long row = (static_cast<long>(n) * a.Hq + h) * a.B + b;
  if (tid < D) a.o[row * D + tid] = f32_to_bf16(l > 0.f ? acc / l : (l == 0.f ? 0.f : acc));
  if (tid == 0) a.lse[row] = l == 0.f ? ninf : m + logf(l);
  (void)s_o;
}

// Visible keys of every token of packed documents. starts [n_docs + 1]
// ascending; token r of document i (starts[i] <= r < starts[i+1]) sees its
// document's keys: all of them, or, with prefix [n_docs], the first prefix[i]
// and those up to its own. Tokens of no document see nothing.
__global__ void __launch_bounds__(256)
    document_ranges_kernel(const int32_t* starts, const int32_t* prefix, int n_docs, int L, int2* ranges) {
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r >= L) return;
  // the last document that starts at or before r
  int lo = 0, hi = n_docs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (starts[mid] <= r) lo = mid + 1;
    else hi = mid;
  }
  int2 out = make_int2(0, 0);
  if (lo > 0) {
    const int a = starts[lo - 1], b = min(starts[lo], L);
    if (r < b) {
      out = make_int2(max(a, 0), b);
      if (prefix) {
        const long p = static_cast<long>(a) + max(prefix[lo - 1], 0);
        out.y = static_cast<int>(min(static_cast<long>(b), max(p, static_cast<long>(r) + 1)));
      }
    }
  }
  ranges[r] = out;
}

}  // namespace sparsed
