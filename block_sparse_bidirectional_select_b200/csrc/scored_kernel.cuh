// Dense attention with modified scores for sm_100a: capped (tanh) scores, a
// distance bias, per-row key ranges (document and prefix masks) and key/value
// heads shared by several query heads. Two query tiles per CTA.
//
//   x = scale * <q_r, k_c>;  x = cap * tanh(x / cap);  x -= slope_h * |q_start + r - c|
//   O_r = sum over c in [lo_r, hi_r) of softmax(x)_c v_c
//
// The pipeline is that of attn_kernel.cuh: pairs of query tiles share the K/V
// tiles of one ring, each slot has its own S/P and O in TMEM, its softmax
// warpgroup and its MMA issuer, and PV is issued in two parts. What differs:
//   * the producer reads the ranges of a pair's rows and walks only the key
//     tiles between the smallest lo and the largest hi (publishing that span
//     with the pair); a pair whose rows see nothing has no tiles at all;
//   * each softmax thread holds one row and its range; a warp masks only tiles
//     that are not inside the ranges of all its 32 rows;
//   * the scores are modified in registers between the TMEM load and the
//     exponentials (below);
//   * with a distance bias the tiles are walked from the pair's own position
//     outwards, so that the row maxima are set at once (towards the position,
//     every tile would raise them and rescale O), and a warp whose scores all
//     lie where 2^x is exactly 0 stores zeros;
//   * with ranges, warp 11 clears the V rows of a tile that no row of the pair
//     sees, so that whatever padding holds (0 * NaN) stays out of O. It looks
//     closer only at tiles that no single row sees whole;
//   * when the pairs would leave SMs idle (`split`), a CTA takes one query tile, and
//     its two slots the even and the odd key tiles of it; slot 0 joins their
//     sums and outputs at the end.
//
// Capped scores. tanh(u) = u * P(u^2), P by a minimax fit (the coefficients are
// scaled on the host so that the polynomial takes the raw product and gives
// log2 units): of degree 2 for |u| <= 0.25 (off by 4e-7 of the score) and 3
// for |u| <= 0.5 (5.7e-7; a few roundings of a score). The narrow one
// costs four packed FP32 operations for two scores, one of which replaces the
// scaling of the plain path; a packed operation takes the FP32 pipe two clocks,
// which is what a capped pass pays for. A warp whose tile holds a larger score
// takes 1 - 2 / (1 + e^2u), two MUFU operations, off by 2^-22 of the cap: as
// good as the polynomial for scores of that size, and with a cap above 64 kept
// for those alone (kCapHigh). MUFU is what bounds that path (16 operations a
// clock and SM, three per score with the softmax's own).
//
// Measured, 32 heads of 8192 tokens, d = 128: 1002 us plain (attn_fwd_kernel:
// 995), 1010 to 1050 with a bias, 1300 capped, 1455 capped and biased. What bounds them
// is a slot's chain (S and P share columns, so S waits for PV) and the power cap.
#pragma once

#include <type_traits>

#include "attn_kernel.cuh"

namespace sparsed {

struct ScoredArgs {
  int H, group;             // query heads, query heads per kv head
  int L, Lk;                // query rows, keys
  int nqb, qpp;             // query tiles of 128 rows per head; tiles per turn (2, or 1: split, one turn per CTA)
  float scale_log2;         // scale * log2(e), above 0
  const float* slopes;      // [H] or null
  int q_start;
  const int2* ranges;       // [L] or null
  // capped scores: y = s * P(s^2) in log2 units while |s| <= cap_fast, with a
  // narrow P (cap_n) up to half of it, else cap_log2 * tanh(s * cap_in)
  float cap_c[4], cap_n[3];
  float cap_fast, cap_in, cap_log2;
  float* lse;               // [H, L]
  uint16_t* o;              // [H, L, D]
  uint64_t timeout_ns;
  int* sched;               // as AttnArgs
};

template <int D>
struct ScoredCfg {
  static constexpr int BK = 128;
  using A = AttnCfg<D, BK>;
  static constexpr int NST = A::NST;
  // Split: a slot waits for its own tiles only, every second K and V, so the
  // use of a stage before must be its own too. A wait can tell a phase from
  // the one before it, and no order of loads says that another slot's has landed.
  static constexpr int NST_SPLIT = NST & ~3;
  static constexpr int B_VOK = A::NUM_BARS;           // [NST] V tile cleared of unseen rows
  static constexpr int B_JOIN = B_VOK + NST;          // split: slot 1's sums are in shared memory, 4 warp arrivals
  static constexpr int NUM_BARS = B_JOIN + 1;
  static constexpr int N_WTAKERS = A::N_WTAKERS + 1;  // and warp 11
  static constexpr int OFF_MISC = A::OFF_BAR + NUM_BARS * 8;  // tmem slot, abort flag, 2 x (pair, first tile, tiles, near)
  static constexpr int OFF_JOIN = (OFF_MISC + 48 + 15) & ~15;  // split: (max, sum) of slot 1's rows
  static constexpr int SMEM_BYTES = OFF_JOIN + 128 * 8 + 1024;
  static_assert(SMEM_BYTES <= A::SMEM_LIMIT, "shared memory budget");
  static_assert(NST_SPLIT >= 4, "ring too shallow");
};

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R) : "memory");
}
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R) : "memory");
}

// tanh(u) = u * (c0 + c1 u^2 + c2 u^4 + c3 u^6) while |u| <= 0.5, off by 5.7e-7 of it.
constexpr double kTanhPoly[4] = {0.9999994765759067, -0.33326466944456906, 0.13191881871914507, -0.044444433804554644};

// tanh(u) for |u| > 0.5: 1 - 2 / (1 + 2^(2 u log2 e)); saturates to +-1.
__device__ __forceinline__ float tanh_wide(float u) {
  const float e = ptx::ex2(u * 2.885390081777926815f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return fmaf(-2.0f, r, 1.0f);
}
// c ? x : y without a branch around x.
__device__ __forceinline__ float select_f32(bool c, float x, float y) {
  float r;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tselp.f32 %0, %1, %2, p;\n\t}"
      : "=f"(r) : "f"(x), "f"(y), "r"(static_cast<uint32_t>(c)));
  return r;
}
// tanh(u) for any u, off by 2^-20 of itself at most; the wide form is off by
// 2^-22 (of 1), which a small u shows once a cap multiplies it. In single
// operations on constants: packed ones on registers spill.
__device__ __forceinline__ float tanh_any(float u) {
  constexpr float c0 = static_cast<float>(kTanhPoly[0]), c1 = static_cast<float>(kTanhPoly[1]),
                  c2 = static_cast<float>(kTanhPoly[2]), c3 = static_cast<float>(kTanhPoly[3]);
  const float w = u * u;
  const float p = u * fmaf(fmaf(fmaf(c3, w, c2), w, c1), w, c0);
  return select_f32(fabsf(u) > 0.5f, tanh_wide(u), p);
}
// How the kernel caps its scores: not at all, or by a cap of up to 64 or above.
// With a low cap the wide form serves every score of a warp that has a large
// one: it is off by 2^-16 at most, a 128th of a weight's rounding. 32 heads of
// 8192 tokens, cap 50, scores of deviation 8 take 2640 us with it, 2800 with
// tanh_any. A choice inside one kernel costs small scores 4% (1300 to 1355 us),
// so it is the kernel's.
constexpr int kCapNone = 0, kCapLow = 1, kCapHigh = 2;
constexpr float kCapLowMost = 64.0f;

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// P(s^2) for a pair of raw scores; the narrow one has a term less.
__device__ __forceinline__ uint64_t cap_poly_narrow(uint64_t s, const uint64_t (&c)[3]) {
  const uint64_t w = mul_f32x2(s, s);
  return ptx::fma_f32x2(ptx::fma_f32x2(c[2], w, c[1]), w, c[0]);
}
__device__ __forceinline__ uint64_t cap_poly(uint64_t s, const uint64_t (&c)[4]) {
  const uint64_t w = mul_f32x2(s, s);
  uint64_t p = ptx::fma_f32x2(c[3], w, c[2]);
  p = ptx::fma_f32x2(p, w, c[1]);
  return ptx::fma_f32x2(p, w, c[0]);
}

// s[0..N) = s * mul(s) - slope2 * |at - c| for the N consecutive keys c from c0
// on, in log2 units; mul: of a pair of scores, the scale or a cap polynomial.
// Distances are exact in fp32 up to 2^24; |at - c| is linear in the key where a
// warp's keys all lie on one side of each thread's row: then eight keys share
// a base and four pairs of offsets, two packed operations for two scores.
template <int N, typename Mul>
__device__ __forceinline__ void scale_and_bias(float (&s)[N], Mul mul, float slope2, int at, int c0) {
  const float d0 = static_cast<float>(at - c0);
  if (__any_sync(0xffffffffu, at > c0 && at < c0 + N - 1)) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const uint64_t v = ptx::f32x2(s[e], s[e + 1]);
      const uint64_t t = ptx::f32x2(-slope2 * fabsf(d0 - static_cast<float>(e)), -slope2 * fabsf(d0 - static_cast<float>(e + 1)));
      ptx::f32x2_split(ptx::fma_f32x2(v, mul(v), t), s[e], s[e + 1]);
    }
  } else {
    const float b1 = at > c0 ? slope2 : -slope2;  // per key: keys left of the row come nearer
    uint64_t off[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) off[u] = ptx::f32x2(b1 * (2 * u), b1 * (2 * u + 1));
    const float b0 = -slope2 * fabsf(d0);
#pragma unroll
    for (int q = 0; q < N / 8; ++q) {
      const float base = fmaf(b1, static_cast<float>(8 * q), b0);
      const uint64_t base2 = ptx::f32x2(base, base);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int e = 8 * q + 2 * u;
        const uint64_t v = ptx::f32x2(s[e], s[e + 1]);
        ptx::f32x2_split(ptx::fma_f32x2(v, mul(v), ptx::add_f32x2(base2, off[u])), s[e], s[e + 1]);
      }
    }
  }
}

// Three-input maximum that is NaN if an input is (one instruction).
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// The largest of a row's scores; NAN_TOO: NaN if one is, else NaNs are left out.
template <bool NAN_TOO = false, int N>
__device__ __forceinline__ float row_max(const float (&s)[N]) {
  auto max3 = [](float a, float b, float c) { return NAN_TOO ? max3_nan(a, b, c) : ptx::max3(a, b, c); };
  float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
#pragma unroll
  for (int c = 4; c < N; c += 8) {
    mx0 = max3(mx0, s[c], s[c + 1]);
    mx1 = max3(mx1, s[c + 2], s[c + 3]);
    if (c + 4 < N) {
      mx2 = max3(mx2, s[c + 4], s[c + 5]);
      mx3 = max3(mx3, s[c + 6], s[c + 7]);
    }
  }
  return NAN_TOO ? max3_nan(max3_nan(mx0, mx1, mx2), mx3, mx3) : fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
}
// Three-input minimum (one instruction).
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
template <int N>
__device__ __forceinline__ float row_min(const float (&s)[N]) {
  float mn0 = s[0], mn1 = s[1], mn2 = s[2], mn3 = s[3];
#pragma unroll
  for (int c = 4; c < N; c += 8) {
    mn0 = min3(mn0, s[c], s[c + 1]);
    mn1 = min3(mn1, s[c + 2], s[c + 3]);
    if (c + 4 < N) {
      mn2 = min3(mn2, s[c + 4], s[c + 5]);
      mn3 = min3(mn3, s[c + 6], s[c + 7]);
    }
  }
  return fminf(fminf(mn0, mn1), fminf(mn2, mn3));
}

// The exponentials of 32 scores of a row in log2 units: CAPPED takes raw
// scores through a polynomial on the way (1: the narrow one).
template <int CAPPED>
__device__ __forceinline__ void scored_exp32(const float* s, uint64_t mul2, uint64_t negm2, const uint64_t (&cap)[4],
                                             const uint64_t (&cap_n)[3],
                                             uint32_t (&pk)[16], uint64_t& acc0, uint64_t& acc1) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const uint64_t v = ptx::f32x2(s[2 * e], s[2 * e + 1]);
    uint64_t arg;
    if constexpr (CAPPED == 2) arg = ptx::fma_f32x2(v, cap_poly(v, cap), negm2);
    else if constexpr (CAPPED == 1) arg = ptx::fma_f32x2(v, cap_poly_narrow(v, cap_n), negm2);
    else arg = ptx::fma_f32x2(v, mul2, negm2);
    float x0, x1;
    ptx::f32x2_split(arg, x0, x1);
    const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
    if (e & 1) acc1 = ptx::add_f32x2(acc1, ptx::f32x2(p0, p1));
    else acc0 = ptx::add_f32x2(acc0, ptx::f32x2(p0, p1));
    pk[e] = ptx::pack_bf16x2(p0, p1);
  }
}

struct ScoredPair {
  int h, q0;
  bool has1;
};
// turn w: head w / nph; its later (under causal masks longer) tiles first
__device__ __forceinline__ ScoredPair scored_pair(const ScoredArgs& a, int w, int nph) {
  ScoredPair r;
  r.h = w / nph;
  r.q0 = (nph - 1 - (w - r.h * nph)) * a.qpp;
  r.has1 = a.qpp == 2 && r.q0 + 1 < a.nqb;
  return r;
}

// The walk's j-th tile: from tile `near` down to the first, then on upwards.
__device__ __forceinline__ int scored_tile(int j, int near) { return j <= near ? near - j : j; }

// [lo, hi) of row r with 0 <= lo and 0 <= hi <= Lk, so that differences from key
// positions fit; rows past the last see all keys when `outside_all`, else nothing.
__device__ __forceinline__ int2 scored_range(const ScoredArgs& a, int r, bool outside_all) {
  int2 v = make_int2(0, a.Lk);
  if (r >= a.L) return outside_all ? v : make_int2(0, 0);
  if (a.ranges) {
    v = a.ranges[r];
    v.x = max(v.x, 0);
    v.y = min(max(v.y, 0), a.Lk);
  }
  return v;
}

// Bits lo .. hi - 1 of a word (none if hi <= lo). A tile's mask goes by such
// words: with two comparisons a score 5 packed documents of 1000 tokens took
// 17.9 us instead of 15.2, prefixes of 8190 tokens with a bias 430 instead of 381.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const int f = min(max(lo, 0), 32), t = min(max(hi, 0), 32);
  return f < t ? (0xffffffffu >> (32 - (t - f))) << f : 0u;
}

template <int D, int CAP, bool BIAS, bool SPLIT>
__global__ void __launch_bounds__(384, 1)
    scored_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ ScoredArgs a) {
  using S = ScoredCfg<D>;
  using C = typename S::A;
  constexpr int BK = S::BK;
  constexpr int NST = SPLIT ? S::NST_SPLIT : S::NST;  // ring stages in use
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nph = (a.nqb + a.qpp - 1) / a.qpp;
  const int n_pairs = a.H * nph;
  constexpr bool split = SPLIT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::OFF_MISC + 4);
  // the producer publishes each turn here, double-buffered: pair, first key
  // tile, key tiles, and the tile that the walk starts from (scored_tile)
  volatile int* turn = reinterpret_cast<volatile int*>(smem + S::OFF_MISC + 8);
  auto bar = [&](int idx) -> uint32_t { return sb + C::OFF_BAR + 8 * idx; };

  // ---- setup
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(bar(C::B_WFULL + s), 1);
      ptx::mbar_init(bar(C::B_WEMPTY + s), S::N_WTAKERS);
      ptx::mbar_init(bar(C::B_QFULL + s), 1);
      ptx::mbar_init(bar(C::B_QEMPTY + s), 1);
      ptx::mbar_init(bar(C::B_SFULL + s), 1);
      for (int q = 0; q < C::NPV; ++q)
        ptx::mbar_init(bar(C::B_PFULL + s * C::NPV + q), 4);  // one arrival per softmax warp of the slot
      ptx::mbar_init(bar(C::B_PVDONE + s), 1);
      ptx::mbar_init(bar(C::B_DRAIN + s), 1);
    }
    for (int s = 0; s < NST; ++s) {
      ptx::mbar_init(bar(C::B_FULL + s), 1);
      ptx::mbar_init(bar(C::B_EMPTY + s), a.ranges ? 3 : 2);  // two commits per tile, and warp 11
      ptx::mbar_init(bar(S::B_VOK + s), 1);
    }
    ptx::mbar_init(bar(S::B_JOIN), 4);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TM_ALLOC);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    setmaxnreg_dec_56();
    const uint32_t leader = ptx::elect_one();
    auto wait = [&](int idx, int parity) -> bool {
      return ptx::mbar_wait_warp(bar(idx), parity & 1, abort_flag, a.timeout_ns, kErrTimeout);
    };
    if (warp == 8) {
      // ============================================================ producer
      if (leader) {
        ptx::tma_prefetch_desc(&tm_q);
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
      }
      int seq = 0;               // ring tiles issued
      int qn0 = 0, qn1 = 0;      // Q tiles issued per slot
      bool ok = true;
      int hk = 0, h = 0;
      auto load_tile = [&](const CUtensorMap* tm, int blk) -> bool {
        const int st = seq % NST;
        if (seq >= NST && !wait(C::B_EMPTY + st, (seq / NST) - 1)) return false;
        ptx::mbar_arrive_expect_tx_if(leader, bar(C::B_FULL + st), C::KV_BYTES);
#pragma unroll
        for (int c = 0; c < C::DCH; ++c)
          ptx::tma_load_3d_if(leader, sb + C::OFF_RING + st * C::KV_BYTES + c * C::KV_CHUNK, tm, bar(C::B_FULL + st),
                              c * 64, blk * BK, hk);
        ++seq;
        return true;
      };
      auto load_q = [&](int s, int qi) -> bool {
        const int qn = s ? qn1 : qn0;
        if (qn > 0 && !wait(C::B_QEMPTY + s, qn - 1)) return false;
        ptx::mbar_arrive_expect_tx_if(leader, bar(C::B_QFULL + s), C::Q_BYTES);
#pragma unroll
        for (int c = 0; c < C::DCH; ++c)
          ptx::tma_load_3d_if(leader, sb + (s ? C::OFF_Q1 : C::OFF_Q0) + c * C::Q_CHUNK, &tm_q, bar(C::B_QFULL + s),
                              c * 64, qi * 128, h);
        if (s) ++qn1;
        else ++qn0;
        return true;
      };
      int np = 0;  // turns published
      auto publish = [&](int w, int j0, int nj, int near) -> bool {
        const int b = np & 1;
        if (np >= 2 && !wait(C::B_WEMPTY + b, (np >> 1) - 1)) return false;
        if (leader) {
          turn[4 * b] = w;
          turn[4 * b + 1] = j0;
          turn[4 * b + 2] = nj;
          turn[4 * b + 3] = near;
          ptx::mbar_arrive(bar(C::B_WFULL + b));
        }
        __syncwarp();
        ++np;
        return true;
      };
      int w = blockIdx.x;
      while (ok) {
        if (w >= n_pairs) {
          publish(n_pairs, 0, 0, 0);
          break;
        }
        const ScoredPair pr = scored_pair(a, w, nph);
        h = pr.h;
        hk = h / a.group;
        // the key tiles between the smallest lo and the largest hi of the pair's rows
        int lo = 0, hi = a.Lk;
        if (a.ranges) {
          lo = a.Lk;
          hi = 0;
          const int rows = pr.has1 ? 256 : 128;
          for (int u = lane; u < rows; u += 32) {
            const int2 v = scored_range(a, pr.q0 * 128 + u, false);
            if (v.x < v.y) {
              lo = min(lo, v.x);
              hi = max(hi, v.y);
            }
          }
          lo = __reduce_min_sync(0xffffffffu, lo);
          hi = __reduce_max_sync(0xffffffffu, hi);
        }
        const int j0 = lo / BK;
        const int nj = hi > lo ? (hi + BK - 1) / BK - j0 : 0;
        // with a bias, the tile of the middle of the pair's rows
        const int near =
            BIAS ? min(max((a.q_start + pr.q0 * 128 + (pr.has1 ? 128 : 64)) / BK - j0, 0), max(nj - 1, 0)) : 0;
        ok = publish(w, j0, nj, near);
        if (!ok) break;
        // the CTA's next turn: the static stride, or a claim on the counter
        int w_next = w + static_cast<int>(gridDim.x);
        if (a.sched) {
          int claim = 0;
          if (leader) claim = atomicAdd(a.sched, 1);
          w_next = static_cast<int>(gridDim.x) + __reduce_max_sync(0xffffffffu, claim);
        }
        if (leader && w_next < n_pairs) {
          const ScoredPair pn = scored_pair(a, w_next, nph);
#pragma unroll
          for (int c = 0; c < C::DCH; ++c) {
            ptx::tma_prefetch_3d(&tm_q, c * 64, pn.q0 * 128, pn.h);
            if (pn.has1) ptx::tma_prefetch_3d(&tm_q, c * 64, (pn.q0 + 1) * 128, pn.h);
          }
        }
        // in the order the slots consume them: Q0, K_0, Q1, V_0, K_1, V_1, ...
        for (int j = 0; ok && j < nj; ++j) {
          if (j == 0) ok = load_q(0, pr.q0);
          const int blk = j0 + (BIAS ? scored_tile(j, near) : j);
          if (ok) ok = load_tile(&tm_k, blk);
          if (ok && j == 0 && (split ? nj > 1 : pr.has1)) ok = load_q(1, split ? pr.q0 : pr.q0 + 1);
          if (ok) ok = load_tile(&tm_v, blk);
        }
        // Slot 1 waits for no tile of a pair without a second query tile. All of
        // them have landed before the next turn is published, so that slot 1 can
        // tell the phase of its next waits.
        if (!split && !pr.has1)
          for (int u = seq > NST ? seq - NST : 0; ok && u < seq; ++u) ok = wait(C::B_FULL + u % NST, u / NST);
        w = w_next;
      }
      if (!ok) {
        // let the copies in flight land before the CTA's shared memory goes away
        const uint64_t short_ns = a.timeout_ns / 4;
        volatile int dummy = 0;
        if (qn0 > 0) ptx::mbar_wait(bar(C::B_QFULL + 0), (qn0 - 1) & 1, &dummy, short_ns, 0);
        if (qn1 > 0) ptx::mbar_wait(bar(C::B_QFULL + 1), (qn1 - 1) & 1, &dummy, short_ns, 0);
        for (int u = (seq > NST ? seq - NST : 0); u < seq; ++u)
          ptx::mbar_wait(bar(C::B_FULL + u % NST), (u / NST) & 1, &dummy, short_ns, 0);
        __syncwarp();
      }
    } else if (warp == 9 || warp == 10) {
      // ============================================================ MMA issuers (as attn_fwd_kernel)
      const int s = warp - 9;
      constexpr uint32_t HI = ptx::sdesc_sw128_hi(1024);
      const uint32_t q_lo = ptx::sdesc_sw128_lo(sb + (s ? C::OFF_Q1 : C::OFF_Q0), 16);
      const uint32_t k_lo = ptx::sdesc_sw128_lo(sb + C::OFF_RING, 16);
      const uint32_t v_lo = ptx::sdesc_sw128_lo(sb + C::OFF_RING, C::KV_CHUNK);
      const uint32_t s_tmem = tmem + (s ? C::TM_S1 : C::TM_S0);
      const uint32_t o_tmem = tmem + (s ? C::TM_O1 : C::TM_O0);
      constexpr int KPP = BK / 16 / C::NPV;  // PV MMAs per part of P
      int seq = 0;      // ring tiles (same numbering as the producer)
      int qn = 0;       // Q tiles consumed
      int tcnt = 0;     // tiles of this slot (PFULL phases)
      bool ok = true;
      auto commit = [&](int idx) { ptx::umma_commit_if(leader, bar(idx)); };
      for (int np = 0; ok; ++np) {
        if (!wait(C::B_WFULL + (np & 1), np >> 1)) {
          ok = false;
          break;
        }
        const int w = turn[4 * (np & 1)];
        const int nj = turn[4 * (np & 1) + 2];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_WEMPTY + (np & 1)));
        if (w >= n_pairs) break;
        const ScoredPair pr = scored_pair(a, w, nph);
        const bool sole = !pr.has1;       // a tile has one slot, which gives both commits
        const int first = split ? s : 0;  // my first tile
        for (int j = 0; j < nj; ++j) {
          const int sk = seq, sv = seq + 1;
          seq += 2;
          if (split ? (j & 1) != s : (s == 1 && !pr.has1)) continue;
          if ((j == first && !wait(C::B_QFULL + s, qn++)) || !wait(C::B_FULL + sk % NST, sk / NST)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            constexpr uint32_t QC = C::Q_CHUNK >> 4, KC = C::KV_CHUNK >> 4;
            const uint32_t ao = (kk >> 2) * QC + (kk & 3) * 2;
            const uint32_t bo = (kk >> 2) * KC + (kk & 3) * 2;
            ptx::umma_ss_lohi_if(leader, s_tmem, q_lo + ao,
                                 k_lo + static_cast<uint32_t>((sk % NST) * C::KV_BYTES >> 4) + bo, HI, C::IDESC_S,
                                 kk > 0 ? 1u : 0u);
          }
          commit(C::B_SFULL + s);
          commit(C::B_EMPTY + sk % NST);
          if (sole) commit(C::B_EMPTY + sk % NST);
          if (j + (split ? 2 : 1) >= nj) commit(C::B_QEMPTY + s);
          // with ranges, the V tile once warp 11 has passed it
          if (!wait(C::B_FULL + sv % NST, sv / NST) || (a.ranges && !wait(S::B_VOK + sv % NST, sv / NST))) {
            ok = false;
            break;
          }
          const uint32_t vb = v_lo + static_cast<uint32_t>((sv % NST) * C::KV_BYTES >> 4);
#pragma unroll
          for (int q = 0; q < C::NPV; ++q) {
            if (!wait(C::B_PFULL + s * C::NPV + q, tcnt)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
#pragma unroll
            for (int u = 0; u < KPP; ++u) {
              const int kk = q * KPP + u;
              ptx::umma_ts_lohi_if(leader, o_tmem, s_tmem + kk * 8, vb + kk * (2048 >> 4), HI, C::IDESC_PV,
                                   (j > first || kk > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          commit(C::B_PVDONE + s);
          commit(C::B_EMPTY + sv % NST);
          if (sole) commit(C::B_EMPTY + sv % NST);
          ++tcnt;
        }
        if (!ok) break;
      }
      if (!ok) {
        commit(C::B_DRAIN + s);
        volatile int dummy = 0;
        ptx::mbar_wait(bar(C::B_DRAIN + s), 0, &dummy, a.timeout_ns / 4, 0);
        __syncwarp();
      }
    } else {
      // ============================================================ warp 11: V rows that no row sees
      // B_VOK counts every use of a stage, K tiles included, so that its
      // parity is the stage's; its arrival comes before the one on B_EMPTY, so
      // a use's B_FULL implies that all earlier B_VOK phases are complete.
      int seq = 0;
      bool ok = true;
      for (int np = 0; ok; ++np) {
        if (!wait(C::B_WFULL + (np & 1), np >> 1)) break;
        const int w = turn[4 * (np & 1)], j0 = turn[4 * (np & 1) + 1], nj = turn[4 * (np & 1) + 2];
        const int near = turn[4 * (np & 1) + 3];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_WEMPTY + (np & 1)));
        if (w >= n_pairs) break;
        if (!a.ranges) continue;
        const ScoredPair pr = scored_pair(a, w, nph);
        int2 rg[8];  // the ranges of my eight rows of the pair
#pragma unroll
        for (int u = 0; u < 8; ++u)
          rg[u] = (u < 4 || pr.has1) ? scored_range(a, pr.q0 * 128 + u * 32 + lane, false) : make_int2(0, 0);
        for (int j = 0; j < nj; ++j, seq += 2) {
          const int st_k = seq % NST, st = (seq + 1) % NST;
          if (!wait(C::B_FULL + st_k, seq / NST)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            ptx::mbar_arrive(bar(S::B_VOK + st_k));
            ptx::mbar_arrive(bar(C::B_EMPTY + st_k));
          }
          if (!wait(C::B_FULL + st, (seq + 1) / NST)) {
            ok = false;
            break;
          }
          const int c0 = (j0 + (BIAS ? scored_tile(j, near) : j)) * BK;
          bool whole = false;
#pragma unroll
          for (int u = 0; u < 8; ++u) whole |= rg[u].x <= c0 && rg[u].y >= c0 + BK;
          if (!__any_sync(0xffffffffu, whole)) {
            uint32_t seen[4] = {0, 0, 0, 0};  // bit per key of the tile
#pragma unroll
            for (int u = 0; u < 8; ++u) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                seen[q] |= bit_range(rg[u].x - c0 - 32 * q, rg[u].y - c0 - 32 * q);
              }
            }
            bool cleared = false;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t all = __reduce_or_sync(0xffffffffu, seen[q]);
              if (!((all >> lane) & 1u)) {
                uint8_t* row = smem + C::OFF_RING + st * C::KV_BYTES + (32 * q + lane) * 128;
#pragma unroll
                for (int c = 0; c < C::DCH; ++c)
#pragma unroll
                  for (int x = 0; x < 8; ++x)
                    *reinterpret_cast<uint4*>(row + c * C::KV_CHUNK + x * 16) = make_uint4(0, 0, 0, 0);
                cleared = true;
              }
            }
            if (cleared) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          }
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(bar(S::B_VOK + st));
            ptx::mbar_arrive(bar(C::B_EMPTY + st));
          }
        }
      }
    }
  } else {
    // ================================================================ softmax
    setmaxnreg_inc_224();
    const int slot = warp >> 2;
    const int wq = warp & 3;
    const int r = wq * 32 + lane;  // row == TMEM lane
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t s_col = slot ? C::TM_S1 : C::TM_S0;
    const uint32_t o_col = slot ? C::TM_O1 : C::TM_O0;
    const float ninf = -__int_as_float(0x7f800000);
    const uint64_t scale2 = ptx::f32x2(a.scale_log2, a.scale_log2);
    const uint64_t one2 = ptx::f32x2(1.f, 1.f);
    uint64_t cap[4], cap_n[3];
    if constexpr (CAP != 0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) cap[u] = ptx::f32x2(a.cap_c[u], a.cap_c[u]);
#pragma unroll
      for (int u = 0; u < 3; ++u) cap_n[u] = ptx::f32x2(a.cap_n[u], a.cap_n[u]);
    }
    int tcount = 0;  // tiles of this slot so far (SFULL / PVDONE phases)
    bool ok = true;
    for (int np = 0; ok; ++np) {
      if (!ptx::mbar_wait_warp(bar(C::B_WFULL + (np & 1)), (np >> 1) & 1, abort_flag, a.timeout_ns, kErrTimeout)) {
        ok = false;
        break;
      }
      const int w = turn[4 * (np & 1)], j0 = turn[4 * (np & 1) + 1], nj = turn[4 * (np & 1) + 2];
      const int near = turn[4 * (np & 1) + 3];
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_WEMPTY + (np & 1)));
      if (w >= n_pairs) break;
      const ScoredPair pr = scored_pair(a, w, nph);
      const int h = pr.h;
      const int qi = split ? pr.q0 : pr.q0 + slot;
      if (slot == 1 && (split ? nj == 0 : !pr.has1)) continue;
      const int grow = qi * 128 + r;
      const bool row_valid = grow < a.L;
      uint4* o_dst = reinterpret_cast<uint4*>(a.o + (static_cast<long>(h) * a.L + grow) * D);
      float* lse_dst = a.lse + static_cast<long>(h) * a.L + grow;
      // my row's keys, and those that all 32 rows of the warp see
      const int2 rg = scored_range(a, grow, true);
      const int all_lo = __reduce_max_sync(0xffffffffu, rg.x), all_hi = __reduce_min_sync(0xffffffffu, rg.y);
      // A row that stands outside its keys is moved to the nearest of them: all
      // its distances shrink by the same amount, which is taken off its log-sum.
      // Else the differences between the keys would drown in the rounding of
      // large biases.
      float slope2 = 0.f, beyond = 0.f;
      int at = a.q_start + grow;
      if constexpr (BIAS) {
        slope2 = a.slopes[h] * 1.44269504088896340736f;
        const int in = rg.x < rg.y ? min(max(at, rg.x), rg.y - 1) : at;
        if (in != at) beyond = a.slopes[h] * static_cast<float>(abs(at - in));
        at = in;
      }
      float m = ninf;  // running row max, log2 units
      float l = 0.f;   // running row sum
      const int first = split ? slot : 0, step = split ? 2 : 1;  // my tiles
      for (int jj = first; jj < nj; jj += step, ++tcount) {
        const int c0 = (j0 + (BIAS ? scored_tile(jj, near) : jj)) * BK;
        if (!ptx::mbar_wait_warp(bar(C::B_SFULL + slot), tcount & 1, abort_flag, a.timeout_ns, kErrTimeout)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float s[BK];
        {
          uint32_t raw[BK / 32][32];
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) ptx::tmem_ld32(lane_base + s_col + c * 32, raw[c]);
          ptx::tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) {
            ptx::reg_fence32(raw[c]);
#pragma unroll
            for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(raw[c][e]);
          }
        }
        const bool masked = c0 < all_lo || c0 + BK > all_hi;  // warp-uniform
        // `raw_args`: s stays raw and the exp pass applies the scale or the
        // polynomial; otherwise s is brought to log2 units here
        bool raw_args = true, narrow = false;
        float mx;
        if constexpr (CAP != 0) {
          const float top = row_max(s), low = row_min(s);
          float far = fmaxf(top, -low);
          if (masked) {  // keys out of the row's range have no say in the path taken
            far = 0.f;
#pragma unroll
            for (int q = 0; q < BK / 32; ++q) {
              const uint32_t seen = bit_range(rg.x - c0 - 32 * q, rg.y - c0 - 32 * q);
#pragma unroll
              for (int e = 0; e < 32; ++e) far = fmaxf(far, (seen >> e) & 1u ? fabsf(s[32 * q + e]) : 0.f);
            }
          }
          const bool wide = __any_sync(0xffffffffu, far > a.cap_fast);
          narrow = !__any_sync(0xffffffffu, far > 0.5f * a.cap_fast);
          raw_args = !wide && !masked && !BIAS;
          if (raw_args) {
            float y0, y1;
            const uint64_t v = ptx::f32x2(top, top);
            ptx::f32x2_split(mul_f32x2(v, cap_poly(v, cap)), y0, y1);
            mx = y0;  // the polynomials rise with s and agree to their error
          } else if (wide) {
#pragma unroll
            for (int c = 0; c < BK; ++c)
              s[c] = a.cap_log2 * (CAP == kCapHigh ? tanh_any(s[c] * a.cap_in) : tanh_wide(s[c] * a.cap_in));
            if constexpr (BIAS) scale_and_bias(s, [&](uint64_t) { return one2; }, slope2, at, c0);
          } else if constexpr (BIAS) {
            if (narrow) scale_and_bias(s, [&](uint64_t v) { return cap_poly_narrow(v, cap_n); }, slope2, at, c0);
            else scale_and_bias(s, [&](uint64_t v) { return cap_poly(v, cap); }, slope2, at, c0);
          } else {
#pragma unroll
            for (int c = 0; c < BK; c += 2) {
              const uint64_t v = ptx::f32x2(s[c], s[c + 1]);
              ptx::f32x2_split(mul_f32x2(v, cap_poly(v, cap)), s[c], s[c + 1]);
            }
          }
        } else if constexpr (BIAS) {
          raw_args = false;
          scale_and_bias(s, [&](uint64_t) { return scale2; }, slope2, at, c0);
        }
        if (masked) {
#pragma unroll
          for (int q = 0; q < BK / 32; ++q) {
            const uint32_t seen = bit_range(rg.x - c0 - 32 * q, rg.y - c0 - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((seen >> e) & 1u)) s[32 * q + e] = ninf;
          }
        }
        // with a bias a NaN shows in mx, so that its tile does not pass for one of
        // zeros below; the running maximum leaves it out either way. Rows past the
        // last, which see padding too, have no say in the warp's votes.
        if constexpr (CAP != 0) {
          if (!raw_args) mx = row_max<BIAS>(s);
        } else {
          mx = row_max<BIAS>(s);
          if constexpr (!BIAS) mx *= a.scale_log2;  // scale_log2 > 0
        }
        if (BIAS && !row_valid) mx = ninf;
        const float m_new = fmaxf(m, mx);
        if (jj == first) {
          m = m_new;
        } else if (__any_sync(0xffffffffu, m_new > m + 8.0f)) {
          // O_s holds every earlier tile of this item: rescale my row (a row
          // that saw nothing yet has zeros)
          const float alpha = m_new == ninf ? 1.0f : ptx::ex2(m - m_new);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t raw[32];
            ptx::tmem_ld32(lane_base + o_col + c * 32, raw);
            ptx::tmem_wait_ld();
            ptx::reg_fence32(raw);
#pragma unroll
            for (int e = 0; e < 32; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * alpha);
            ptx::tmem_st32(lane_base + o_col + c * 32, raw);
          }
          l *= alpha;
          m = m_new;
        }
        const float mu = m == ninf ? 0.f : m;
        const uint64_t negm2 = ptx::f32x2(-mu, -mu);
        uint64_t acc0 = ptx::f32x2(0.f, 0.f), acc1 = acc0;
        constexpr int CPP = BK / 32 / C::NPV;  // 32-column chunks per part of P
        // with a steep bias whole tiles lie where 2^x is exactly 0
        const bool zero = BIAS && !__any_sync(0xffffffffu, !(mx - mu < -127.f));
        auto exp_pass = [&](auto capped, uint64_t mul2) {
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) {
            uint32_t pk[16];
            if (zero) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            } else {
              scored_exp32<decltype(capped)::value>(s + 32 * c, mul2, negm2, cap, cap_n, pk, acc0, acc1);
            }
            ptx::tmem_st32_16(lane_base + s_col + c * 16, pk);
            if ((c + 1) % CPP == 0 && c + 1 < BK / 32) {
              // this part of P is in TMEM: its PV MMAs may start
              ptx::tmem_wait_st();
              ptx::tc_fence_before();
              __syncwarp();
              if (lane == 0) ptx::mbar_arrive(bar(C::B_PFULL + slot * C::NPV + c / CPP));
            }
          }
        };
        using Plain = std::integral_constant<int, 0>;
        if constexpr (CAP != 0 && !BIAS) {
          if (raw_args && narrow) exp_pass(std::integral_constant<int, 1>{}, one2);
          else if (raw_args) exp_pass(std::integral_constant<int, 2>{}, one2);
          else exp_pass(Plain{}, one2);
        } else {
          exp_pass(Plain{}, BIAS ? one2 : scale2);
        }
        float a0, a1, b0, b1;
        ptx::f32x2_split(acc0, a0, a1);
        ptx::f32x2_split(acc1, b0, b1);
        l += (a0 + b0) + (a1 + b1);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_PFULL + slot * C::NPV + C::NPV - 1));
      }
      if (!ok) break;
      if (nj == 0) {
        if (row_valid) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) o_dst[c] = make_uint4(0, 0, 0, 0);
          *lse_dst = ninf;
        }
        continue;
      }
      // ---- epilogue: every PV of the item is done -> O / l -> bf16 -> global; LSE
      if (tcount > 0 && !ptx::mbar_wait_warp(bar(C::B_PVDONE + slot), (tcount - 1) & 1, abort_flag, a.timeout_ns,
                                             kErrTimeout)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      float own = 1.f, other = 0.f;  // split: weights of both slots' outputs
      if constexpr (split) {
        float2* ml = reinterpret_cast<float2*>(smem + S::OFF_JOIN);
        if (slot == 1) {
          ml[r] = make_float2(m, l);
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(S::B_JOIN));
          continue;
        }
        const int n1 = nj >> 1;  // slot 1's tiles
        if (!ptx::mbar_wait_warp(bar(S::B_JOIN), 0, abort_flag, a.timeout_ns, kErrTimeout) ||
            (n1 > 0 && !ptx::mbar_wait_warp(bar(C::B_PVDONE + 1), (n1 - 1) & 1, abort_flag, a.timeout_ns, kErrTimeout))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (n1 > 0) {
          const float2 x = ml[r];
          const float M = fmaxf(m, x.x);
          own = m == ninf && M != ninf ? 0.f : (m == M ? 1.f : ptx::ex2(m - M));
          other = x.x == M ? 1.f : (x.x == ninf ? 0.f : ptx::ex2(x.x - M));
          l = l * own + x.y * other;
          m = M;
        }
      }
      const bool empty = l == 0.f;  // the row saw nothing
      const float inv_l = empty ? 0.f : 1.0f / l;
      const bool two = split && __any_sync(0xffffffffu, other != 0.f);
      const float f0 = own * inv_l, f1 = other * inv_l;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t raw[32];
        ptx::tmem_ld32(lane_base + o_col + c * 32, raw);
        ptx::tmem_wait_ld();
        ptx::reg_fence32(raw);
        float v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = f0 == 0.f ? 0.f : __uint_as_float(raw[e]) * f0;
        if (two) {
          ptx::tmem_ld32(lane_base + C::TM_O1 + c * 32, raw);
          ptx::tmem_wait_ld();
          ptx::reg_fence32(raw);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] += f1 == 0.f ? 0.f : __uint_as_float(raw[e]) * f1;
        }
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = ptx::pack_bf16x2(v[2 * e], v[2 * e + 1]);
        if (row_valid) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            o_dst[c * 4 + u] = make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
        }
      }
      if (row_valid) *lse_dst = empty ? ninf : (m + ptx::lg2(l)) * 0.69314718055994530942f - beyond;
      // the next item's first PV overwrites O_s only after this warp's next
      // PFULL arrival, which follows the loads above (tcgen05.wait::ld)
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TM_ALLOC);
  }
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
