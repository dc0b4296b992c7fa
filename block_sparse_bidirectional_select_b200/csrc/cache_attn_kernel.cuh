// Attention over the 8-bit cache for sm_100a: the query tokens of each sequence
// (one token, or a block being denoised) against all its cached keys.
//
//   x = scale * <q, k>, k = e4m3 * 2^ek;  capped, biased as scored_attn
//   O = sum softmax(x)_c v_c,  v = e4m3 * 2^ev
//
// Rows. A kv head's query rows (its query heads times B tokens) are cut into
// row tiles of up to 128; an item is one row tile of one kv head of one
// sequence. Its keys are walked in tiles, last first (with a distance bias the
// keys near the queries then set the row maxima at once; ascending, O would be
// rescaled at every tile).
//
// Work split. All key tiles of all items, in order, are dealt out as one run
// of equal length per CTA, whatever the sequences' lengths, so every SM reads
// the same number of bytes. A CTA's run crosses item boundaries; an item cut by
// a run's end leaves partial results (O normalised, log2 of the sum) that
// cache_merge_kernel joins in the order of the runs: no atomics, the same bits
// every time. Beginning an item (its Q, the last one's epilogue) costs a CTA
// some 4 us, so each item counts `toll` tiles more than it has, ahead of its
// first (kTollFew, kTollMany below): a CTA among many short items gets fewer
// tiles.
//
// Exact operands. e4m3 has 4 significant bits and bf16 has 8, so a bf16 query
// is the sum of two e4m3 numbers: hi = e4m3(q 2^-e), lo = e4m3(q 2^-e - hi),
// with 2^e the row's own scale. lo is exact while the element is at least 2^-2
// of the row's scaled range (224..448 at its top); below, it is off by
// 2^-10, 2^-17.8 of the row's largest element. S = hi K^T + lo K^T runs on the
// fp8 tensor path straight from the cached bytes, at the cost of one bf16
// product. For P V that trick would lose the tail of a peaked row (a weight
// below 2^-10 of the largest has no bits left in e4m3), so V is widened to
// f16, exactly, and P is f16 with its top at 2^7 .. 2^15 (error 2^-11, or
// 2^-32 of the largest weight). Each V block is brought to the largest scale of
// the run's part of the item (a power of two: exact, or below 2^-24 of that
// scale), so O accumulates in one unit.
//
// Many rows (Q == 0, more than 64 rows of a kv head): tiles of 128 keys. All
// eight softmax warps work on every tile, each 16 lanes of the accumulators
// with 64 keys to a thread; P is written over the first half of its S.
//
// Few rows (Q == 1, 2, 4: at most 64, 32, 16 rows): what bounds the pass is then
// the chain load S - maximum - exponentials - store P of one tile, a fixed cost
// of several hundred clocks that does not shrink with the rows. So the rows are
// held 2 * Q times in the 128 lanes, each copy a softmax of its own over its
// part of the keys: lanes 0-15 of every quarter take the even tiles (warps 0-3),
// lanes 16-31 the odd ones (warps 4-7), so two tiles are in work at any time; and
// Q quarters that hold the same rows take a Q-th of a tile's keys each. A copy's
// P is zero for the keys of the others: P has columns of its own, which are
// cleared once and written only by their owners. With 64 keys to a tile, S, P
// and Q all fit twice, and S(g+2) starts when S(g) has been read. The copies
// are joined through shared memory when an item's part ends.
//
// Warp roles (512 threads):
//   warps 0-7   softmax: warp w covers the lanes 32*(w%4) + 16*(w/4) + 0..15, thread
//               t lane t%16 and half t/16 of its keys; they also bring each item's
//               Q into TMEM as hi and lo
//   warp 8      TMA producer: K and V tiles
//   warp 9      TMEM owner; issues S
//   warp 10     issues O += P V
//   warp 11     idle
//   warps 12-15 widen V tiles (e4m3 -> f16, rows past the length cleared)
// Every wait is bounded.
//
// Measured: 16 single tokens of 32 heads on 8 over 16384 keys (537 MB) 111 to
// 116 us, 4.6 to 4.8 TB/s with set-up, joins and launches, 5.2 TB/s in the
// steady state; a single token over 8192 keys 17 us, of which the tiles are 4;
// two 64-token blocks of 32 heads over 32768 keys with a bias 162 to 170 us. No
// unit is saturated (DRAM 44% busy for 4 single tokens, 29% for a block): what
// bounds both is the chain of a tile, and the ends of the parts.
#pragma once

#include "cache_kernels.cuh"
#include "scored_kernel.cuh"

namespace sparsed {

constexpr int kCacheMaxCtas = 160;
constexpr int kTollFew = 8, kTollMany = 3;
constexpr float kPShift = 7.0f;  // P's top is 2^7 when its row maximum is fresh

struct CacheArgs {
  const uint16_t* q;
  size_t qs_n, qs_h, qs_b;
  const float *k_scale, *v_scale;  // [N, Hkv, C/64]
  const int32_t* lengths;
  const int32_t* q_start;          // or null
  int N, Hkv, group, B, C;
  int R, RT;                       // rows of a kv head, row tiles
  int part_rows;                   // rows of a partial result's slot
  int tile;                        // keys of a tile
  int toll;                        // what beginning an item costs, in tiles
  float scale_log2;                // above 0
  const float* slopes;             // or null
  float cap_c[4];                  // as ScoredArgs
  float cap_fast, cap_in, cap_log2;
  uint16_t* o;                     // [N, Hkv * group, B, D]
  float* lse;
  float* o_part;                   // [2 * CTAs][part_rows][D]
  float* l_part;                   // [2 * CTAs][part_rows], log2 units
  uint64_t timeout_ns;
};

template <int D, int Q>
struct CacheCfg {
  static constexpr bool FEW = Q > 0;
  static constexpr int BK = FEW ? 64 : 128;      // keys of a tile
  static constexpr int COLS = FEW ? BK / Q : BK; // keys of a tile for one copy of the rows
  static constexpr int N = COLS / 2;             // ... for one thread
  static constexpr int T8 = BK * D;              // bytes of an e4m3 tile
  static constexpr int T16 = 2 * T8;
  static constexpr int VT = FEW ? 2 : 1;         // tiles of a V stage, widened together
  static constexpr int KS = D == 64 ? 8 : (FEW ? 6 : 4);  // ring stages of K
  static constexpr int VS = KS / VT;                      // ... of V
  static constexpr int ROWS = FEW ? 64 / Q : 128;        // rows of a row tile at most
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KS * T8;
  static constexpr int OFF_W = OFF_V + VS * VT * T8;  // widened V: two buffers of VT tiles
  static constexpr int OFF_J = OFF_W + 2 * VT * T16;  // joining copies: 128 lanes x 64 fp32, then (m, l) of each lane
  static constexpr int J_BYTES = FEW ? 128 * 64 * 4 : 0;
  static constexpr int OFF_Q = OFF_J + J_BYTES + (FEW ? 128 * 8 : 0);  // a part's Q: hi, lo, exponents
  static constexpr int OFF_BAR = OFF_Q + 2 * ROWS * D + ROWS * 4;
  static constexpr int B_KFULL = 0;
  static constexpr int B_KEMPTY = B_KFULL + KS;
  static constexpr int B_VFULL = B_KEMPTY + KS;
  static constexpr int B_VEMPTY = B_VFULL + VS;  // 4 converter-warp arrivals
  static constexpr int B_WFULL = B_VEMPTY + VS;  // [2] 4 converter-warp arrivals
  static constexpr int B_WEMPTY = B_WFULL + 2;   // [2]
  static constexpr int B_SFULL = B_WEMPTY + 2;   // [2]
  static constexpr int B_SREAD = B_SFULL + 2;    // [2] FEW: S read, its owners' 4 warp arrivals
  static constexpr int B_PFULL = B_SREAD + 2;    // [2] its owners' warp arrivals
  static constexpr int B_PVDONE = B_PFULL + 2;   // [2]
  static constexpr int B_DRAIN = B_PVDONE + 2;   // [2]
  static constexpr int B_QTFULL = B_DRAIN + 2;   // [2] 8 softmax-warp arrivals
  static constexpr int B_QTEMPTY = B_QTFULL + 2; // [2]
  static constexpr int B_JOIN = B_QTEMPTY + 2;   // 8 softmax-warp arrivals
  static constexpr int NUM_BARS = B_JOIN + 1;
  static constexpr int OWNERS = FEW ? 4 : 8;     // softmax warps that work on a tile
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;  // tmem slot, abort flag, run
  static constexpr int SMEM_BYTES = OFF_MISC + 48 + 1024;
  // TMEM columns: S0, S1, then P0, P1 (or P over the first half of S), O, Q0, Q1
  static constexpr int TM_S0 = 0;
  static constexpr int TM_S1 = BK;
  static constexpr int TM_P0 = FEW ? 2 * BK : TM_S0;
  static constexpr int TM_P1 = FEW ? 2 * BK + BK / 2 : TM_S1;
  static constexpr int TM_O = FEW ? 3 * BK : 2 * BK;
  static constexpr int TM_Q0 = TM_O + D;    // hi: D/4 columns of four e4m3, lo: D/4
  static constexpr int TM_Q1 = TM_Q0 + D / 2;
  static constexpr int TM_ALLOC = 512;
  // f32 accumulators; e4m3 x e4m3 (kind::f8f6f4) and f16 x f16 (kind::f16) are both format 0
  static constexpr uint32_t idesc(int n, int b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
  }
  static constexpr uint32_t IDESC_S = idesc(BK, 0);
  static constexpr uint32_t IDESC_PV = idesc(D, 1);
  // K rows of D bytes: one swizzle span of 128 or 64 bytes, 8 rows a group
  static constexpr uint32_t HI_K = ((8u * D) >> 4) | (1u << 14) | ((D == 128 ? 2u : 4u) << 29);
  static constexpr int THREADS = 512;
  static constexpr int REGS_SOFTMAX = 184, REGS_CONTROL = 56, REGS_WIDEN = 88;
  static constexpr int REGS_TOTAL = 256 * REGS_SOFTMAX + 128 * REGS_CONTROL + 128 * REGS_WIDEN;
  static_assert(TM_Q1 + D / 2 <= 512, "TMEM budget");
  static_assert(SMEM_BYTES <= 232448, "shared memory budget");
  static_assert(REGS_TOTAL <= 65536, "register budget");
};

namespace ptx {
__device__ __forceinline__ void umma_ts_f8_if(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                              uint32_t hi, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 db;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "setp.ne.b32 q, %6, 0;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], db, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tmem_st32_8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// "16x32bx2" accesses of 16, 8 and 4 columns per half (see tmem_ld16x2_32):
// register i to or from column col + (t / 16) * SPLIT + i.
template <int SPLIT>
__device__ __forceinline__ void tmem_ld16x2(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x32bx2.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16], %17;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr), "n"(SPLIT)
      : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16x2(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x32bx2.x16.b32 [%0], %17, {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "n"(SPLIT)
      : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16x2(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x8.b32 [%0], %9, {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "n"(SPLIT)
               : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16x2(uint32_t taddr, const uint32_t (&r)[32]) {
  tmem_st16x2_32<SPLIT>(taddr, r);
}
template <int SPLIT>
__device__ __forceinline__ void tmem_ld16x2(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x32bx2.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8], %9;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr), "n"(SPLIT)
               : "memory");
}
template <int SPLIT>
__device__ __forceinline__ void tmem_st16x2(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.16x32bx2.x4.b32 [%0], %5, {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "n"(SPLIT)
               : "memory");
}
__device__ __forceinline__ void reg_fence8(uint32_t (&r)[8]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
}
// Keeps uses of r below a preceding tmem_wait_ld (as reg_fence32).
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
               "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
}  // namespace ptx

__device__ __forceinline__ int cache_len(const CacheArgs& a, int n) { return min(max(a.lengths[n], 0), a.C); }
__device__ __forceinline__ int cache_tiles(const CacheArgs& a, int len) { return (len + a.tile - 1) / a.tile; }

// Position of query token b of sequence n, and the nearest cached one to it. A
// row's distances are taken from the latter (scored_attn does the same): they
// are all shorter by the same amount, which its log-sum loses at the end.
__device__ __forceinline__ int query_position(const CacheArgs& a, int n, int len, int b) {
  return (a.q_start ? min(max(a.q_start[n], -(1 << 29)), 1 << 29) : len - a.B) + b;
}
__device__ __forceinline__ int nearest_key(int at, int len) { return min(max(at, 0), len - 1); }
// What row rr of a kv head's rows loses (natural units).
__device__ __forceinline__ float beyond_keys(const CacheArgs& a, int n, int hk, int len, int rr) {
  if (!a.slopes) return 0.f;
  const int hg = rr / a.B;
  const int at = query_position(a, n, len, rr - hg * a.B), in = nearest_key(at, len);
  return at == in ? 0.f : a.slopes[hk * a.group + hg] * static_cast<float>(abs(at - in));
}

// An item's length in the runs' unit: its tiles and the toll.
__device__ __forceinline__ int item_units(const CacheArgs& a, int nt) { return nt > 0 ? nt + a.toll : 0; }

// Total units of the call, and those before sequence n_stop (one warp).
__device__ __forceinline__ long cache_total(const CacheArgs& a, int lane, int n_stop, long* before) {
  long t = 0, b = 0;
  for (int n = lane; n < a.N; n += 32) {
    const long x = static_cast<long>(item_units(a, cache_tiles(a, cache_len(a, n)))) * a.Hkv * a.RT;
    t += x;
    if (n < n_stop) b += x;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    t += __shfl_xor_sync(0xffffffffu, t, off);
    b += __shfl_xor_sync(0xffffffffu, b, off);
  }
  if (before) *before = b;
  return t;
}

// First unit of run c of G runs over T units.
__device__ __forceinline__ long run_begin(long T, int c, int G) {
  const long q = T / G;
  return q * c + static_cast<int>(T - q * G) * c / G;
}

// A run's parts: the tiles of one item that lie in it.
struct CachePart {
  int n, hk, rt;   // item
  int len;         // the sequence's length
  int nt;          // the item's tiles
  int t0, cnt;     // this part's tiles
};
struct CacheRun {
  int n, hk, rt, u;  // where the run stands: item, unit of it
  int len, nt;       // of sequence n
  int left;          // units to go
  __device__ __forceinline__ void load(const CacheArgs& a) {
    len = cache_len(a, n);
    nt = cache_tiles(a, len);
  }
  __device__ __forceinline__ bool next(const CacheArgs& a, CachePart& p) {
    while (left > 0) {
      if (u >= nt + a.toll) {  // the next item, past empty sequences
        u = 0;
        if (++rt >= a.RT) {
          rt = 0;
          if (++hk >= a.Hkv) {
            hk = 0;
            do {
              if (++n >= a.N) return false;
              load(a);
            } while (nt == 0);
          }
        }
      }
      const int step = min(nt + a.toll - u, left);
      const int t0 = max(u - a.toll, 0), t1 = max(u + step - a.toll, 0);
      u += step;
      left -= step;
      if (t1 > t0) {  // not the toll alone
        p.n = n;
        p.hk = hk;
        p.rt = rt;
        p.len = len;
        p.nt = nt;
        p.t0 = t0;
        p.cnt = t1 - t0;
        return true;
      }
    }
    return false;
  }
};

// The largest exponent among the part's V scales (one warp).
__device__ __forceinline__ int part_vref(const CacheArgs& a, const CachePart& p, int lane) {
  const float* vs = a.v_scale + (static_cast<long>(p.n) * a.Hkv + p.hk) * (a.C / kCacheBlock);
  const int per = a.tile / kCacheBlock;
  const int b0 = per * p.t0, b1 = min(per * (p.t0 + p.cnt), (p.len + kCacheBlock - 1) / kCacheBlock);
  int e = kCacheEMin;
  for (int b = b0 + lane; b < b1; b += 32) e = max(e, scale_exponent(vs[b]));
  return __reduce_max_sync(0xffffffffu, e);
}

// N scores of a thread (64, 32, 16 or 8) from its lane of S: N columns from
// `taddr` for half 0, N further on for half 1.
template <int N>
__device__ __forceinline__ void load_scores(uint32_t taddr, float (&s)[N]) {
  if constexpr (N == 8) {
    uint32_t raw[8];
    ptx::tmem_ld16x2<8>(taddr, raw);
    ptx::tmem_wait_ld();
    ptx::reg_fence8(raw);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = __uint_as_float(raw[e]);
  } else if constexpr (N == 16) {
    uint32_t raw[16];
    ptx::tmem_ld16x2<16>(taddr, raw);
    ptx::tmem_wait_ld();
    ptx::reg_fence16(raw);
#pragma unroll
    for (int e = 0; e < 16; ++e) s[e] = __uint_as_float(raw[e]);
  } else {
    uint32_t raw[N / 32][32];
#pragma unroll
    for (int c = 0; c < N / 32; ++c) ptx::tmem_ld16x2_32<N>(taddr + c * 32, raw[c]);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < N / 32; ++c) {
      ptx::reg_fence32(raw[c]);
#pragma unroll
      for (int e = 0; e < 32; ++e) s[c * 32 + e] = __uint_as_float(raw[c][e]);
    }
  }
}

// MODE: 0 plain scores, 1 with a distance bias, 2 capped (and biased, if slopes are given).
template <int D, int MODE, int Q>
__global__ void __launch_bounds__(CacheCfg<D, Q>::THREADS, 1)
    cache_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CacheArgs a) {
  using C = CacheCfg<D, Q>;
  constexpr bool FEW = C::FEW;
  constexpr int N = C::N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = ptx::smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  volatile int* run_s = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 8);  // sequence, item in it, unit, units
  auto bar = [&](int idx) -> uint32_t { return sb + C::OFF_BAR + 8 * idx; };

  // ---- setup
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::KS; ++s) {
      ptx::mbar_init(bar(C::B_KFULL + s), 1);
      ptx::mbar_init(bar(C::B_KEMPTY + s), 1);
    }
    for (int s = 0; s < C::VS; ++s) {
      ptx::mbar_init(bar(C::B_VFULL + s), 1);
      ptx::mbar_init(bar(C::B_VEMPTY + s), 4);
    }
    for (int b = 0; b < 2; ++b) {
        ptx::mbar_init(bar(C::B_SREAD + b), C::OWNERS);
      ptx::mbar_init(bar(C::B_WFULL + b), 4);
      ptx::mbar_init(bar(C::B_WEMPTY + b), 1);
      ptx::mbar_init(bar(C::B_SFULL + b), 1);
      ptx::mbar_init(bar(C::B_PFULL + b), C::OWNERS);
      ptx::mbar_init(bar(C::B_PVDONE + b), 1);
      ptx::mbar_init(bar(C::B_DRAIN + b), 1);
      ptx::mbar_init(bar(C::B_QTFULL + b), 8);
      ptx::mbar_init(bar(C::B_QTEMPTY + b), 1);
    }
    ptx::mbar_init(bar(C::B_JOIN), 8);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), C::TM_ALLOC);
    ptx::tmem_relinquish();
  }
  if (warp == 12) {
    // my run: its first unit's sequence, and the unit within the sequence
    const long T = cache_total(a, lane, 0, nullptr);
    const long begin = run_begin(T, blockIdx.x, gridDim.x), end = run_begin(T, blockIdx.x + 1, gridDim.x);
    long base = 0;
    int n0 = a.N;
    for (int nb = 0; nb < a.N && begin < end; nb += 32) {
      const int n = nb + lane;
      const long x = n < a.N ? static_cast<long>(item_units(a, cache_tiles(a, cache_len(a, n)))) * a.Hkv * a.RT : 0;
      long inc = x;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const long y = __shfl_up_sync(0xffffffffu, inc, off);
        if (lane >= off) inc += y;
      }
      const uint32_t hit = __ballot_sync(0xffffffffu, base + inc > begin);
      if (hit) {
        const int src = __ffs(hit) - 1;
        n0 = nb + src;
        base += __shfl_sync(0xffffffffu, inc - x, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      const bool some = n0 < a.N;
      const int units = some ? item_units(a, cache_tiles(a, cache_len(a, n0))) : 1;
      const long off = begin - base;
      run_s[0] = some ? n0 : 0;
      run_s[1] = some ? static_cast<int>(off / units) : 0;
      run_s[2] = some ? static_cast<int>(off % units) : 0;
      run_s[3] = some ? static_cast<int>(end - begin) : 0;
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  ptx::grid_dep_launch();
  const uint32_t tmem = *tmem_slot;
  if constexpr (FEW) {
    // P: all zero; from here on a copy writes its own keys only
    if (warp < 4) {
      uint32_t zero[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) zero[e] = 0u;
      ptx::tmem_st32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::TM_P0, zero);
      ptx::tmem_st32(tmem + (static_cast<uint32_t>(warp * 32) << 16) + C::TM_P1, zero);
      ptx::tmem_wait_st();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
  }
  CacheRun run;
  run.n = run_s[0];
  run.hk = run_s[1] / a.RT;
  run.rt = run_s[1] - run.hk * a.RT;
  run.u = run_s[2];
  run.left = run_s[3];
  if (run.left > 0) run.load(a);
  CachePart part;

  if (warp >= 12) {
    // ================================================================ widen V
    setmaxnreg_dec<C::REGS_WIDEN>();
    const int tid = threadIdx.x - 384;
    constexpr int TPR = D / 16;            // threads of a row, 16 values each
    constexpr int ROWS = 128 / TPR;        // rows of a pass
    constexpr int NP = C::BK / ROWS;       // passes of a tile
    constexpr int PER = C::BK / kCacheBlock;  // scale blocks of a tile
    const int j = tid % TPR, row0 = tid / TPR;
    const int chunk = j >> 2;
    // The two 16-byte units of a thread's f16 values. With 128 elements a row,
    // the threads of its second half write their second unit first, so that
    // eight threads of a row cover all banks.
    const bool sw = (chunk & 1) != 0;
    const int swz = row0 & 7;  // ROWS is a multiple of 8
    const uint32_t off_a = row0 * 128 + (((2 * (j & 3) + (sw ? 1 : 0)) ^ swz) << 4) + chunk * (C::BK * 128);
    const uint32_t off_b = row0 * 128 + (((2 * (j & 3) + (sw ? 0 : 1)) ^ swz) << 4) + chunk * (C::BK * 128);
    int pp = 0;  // V stages so far (VT tiles each, fewer at a part's end)
    bool ok = true;
    while (ok && run.next(a, part)) {
      const int vref = part_vref(a, part, lane);
      const float* vs = a.v_scale + (static_cast<long>(part.n) * a.Hkv + part.hk) * (a.C / kCacheBlock);
      const int last = a.C / kCacheBlock - 1;
      // a stage's scales are read a stage ahead
      constexpr int SB = C::VT * PER;  // scale blocks of a stage: tile t - x / PER, block x % PER
      const int t_last = part.t0 + part.cnt - 1;
      auto scale_at = [&](int t, int x) -> float {
        return vs[min(max(PER * (t - x / PER) + x % PER, 0), last)];
      };
      float sc[SB];
#pragma unroll
      for (int x = 0; x < SB; ++x) sc[x] = scale_at(t_last, x);
#pragma unroll 1
      for (int t = t_last; t >= part.t0; t -= C::VT, ++pp) {
        const int st = pp % C::VS, b = pp & 1;
        // 2^(ev - vref) as f16 pairs (0 below f16's range; a block past the
        // length may hold any scale: its rows are cleared)
        uint32_t mul[SB];
#pragma unroll
        for (int x = 0; x < SB; ++x) {
          const int dlt = min(scale_exponent(sc[x]) - vref, 0);
          const uint32_t hbits = dlt >= -14 ? static_cast<uint32_t>(dlt + 15) << 10
                                            : (dlt >= -24 ? 1u << (dlt + 24) : 0u);
          mul[x] = hbits | (hbits << 16);
          sc[x] = scale_at(t - C::VT, x);
        }
        if (!ptx::mbar_wait_warp(bar(C::B_VFULL + st), (pp / C::VS) & 1, abort_flag, a.timeout_ns, kErrTimeout)) {
          ok = false;
          break;
        }
        const uint8_t* src = smem + C::OFF_V + st * (C::VT * C::T8) + row0 * D + j * 16;
        uint8_t* dst = smem + C::OFF_W + b * (C::VT * C::T16);
        const int valid = part.len - t * C::BK;  // of the stage's first tile; a second one is whole
        uint4 x[C::VT * NP];
#pragma unroll
        for (int p = 0; p < C::VT * NP; ++p) x[p] = *reinterpret_cast<const uint4*>(src + p * (ROWS * D));
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_VEMPTY + st));
        if (valid < C::BK) {
#pragma unroll
          for (int p = 0; p < NP; ++p)
            if (row0 + p * ROWS >= valid) x[p] = make_uint4(0, 0, 0, 0);
        }
        if (pp >= 2 &&
            !ptx::mbar_wait_warp(bar(C::B_WEMPTY + b), ((pp >> 1) - 1) & 1, abort_flag, a.timeout_ns, kErrTimeout)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int p = 0; p < C::VT * NP; ++p) {
          const uint32_t m2 = mul[p * PER / NP];
          const uint32_t w[4] = {sw ? x[p].z : x[p].x, sw ? x[p].w : x[p].y, sw ? x[p].x : x[p].z, sw ? x[p].y : x[p].w};
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, u;\n\t}"
                : "=r"(h[2 * e]), "=r"(h[2 * e + 1])
                : "r"(w[e]));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[2 * e]) : "r"(m2));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[2 * e + 1]) : "r"(m2));
          }
          uint8_t* tile = dst + (p / NP) * C::T16 + (p % NP) * (ROWS * 128);
          *reinterpret_cast<uint4*>(tile + off_a) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(tile + off_b) = make_uint4(h[4], h[5], h[6], h[7]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_WFULL + b));
      }
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<C::REGS_CONTROL>();
    const uint32_t leader = ptx::elect_one();
    auto wait = [&](int idx, int parity) -> bool {
      return ptx::mbar_wait_warp(bar(idx), parity & 1, abort_flag, a.timeout_ns, kErrTimeout);
    };
    if (warp == 8) {
      // ============================================================ producer
      if (leader) {
        ptx::tma_prefetch_desc(&tm_k);
        ptx::tma_prefetch_desc(&tm_v);
      }
      int g = 0, pp = 0;  // K tiles, V stages issued
      bool ok = true;
      while (ok && run.next(a, part)) {
        const int z = part.n * a.Hkv + part.hk;
        for (int jj = 0; jj < part.cnt; ++jj, ++g) {
          const int t = part.t0 + part.cnt - 1 - jj;
          const int st = g % C::KS;
          if (g >= C::KS && !wait(C::B_KEMPTY + st, g / C::KS - 1)) {
            ok = false;
            break;
          }
          ptx::mbar_arrive_expect_tx_if(leader, bar(C::B_KFULL + st), C::T8);
          ptx::tma_load_3d_if(leader, sb + C::OFF_K + st * C::T8, &tm_k, bar(C::B_KFULL + st), 0, t * C::BK, z);
          if (jj % C::VT != 0) continue;
          // the V stage that begins with this tile
          const int sv = pp % C::VS;
          if (pp >= C::VS && !wait(C::B_VEMPTY + sv, pp / C::VS - 1)) {
            ++g;
            ok = false;
            break;
          }
          const int tiles = min(C::VT, part.cnt - jj);
          ptx::mbar_arrive_expect_tx_if(leader, bar(C::B_VFULL + sv), tiles * C::T8);
          for (int x = 0; x < tiles; ++x)
            ptx::tma_load_3d_if(leader, sb + C::OFF_V + (sv * C::VT + x) * C::T8, &tm_v, bar(C::B_VFULL + sv), 0,
                                (t - x) * C::BK, z);
          ++pp;
        }
      }
      if (!ok) {
        // let the copies in flight land before the CTA's shared memory goes away
        const uint64_t short_ns = a.timeout_ns / 4;
        volatile int dummy = 0;
        for (int u = (g > C::KS ? g - C::KS : 0); u < g; ++u)
          ptx::mbar_wait(bar(C::B_KFULL + u % C::KS), (u / C::KS) & 1, &dummy, short_ns, 0);
        for (int u = (pp > C::VS ? pp - C::VS : 0); u < pp; ++u)
          ptx::mbar_wait(bar(C::B_VFULL + u % C::VS), (u / C::VS) & 1, &dummy, short_ns, 0);
        __syncwarp();
      }
    } else if (warp == 9) {
      // ============================================================ S issuer
      const uint32_t klo = ptx::sdesc_sw128_lo(sb + C::OFF_K, 16);
      int g = 0, iq = 0;
      bool ok = true;
      while (ok && run.next(a, part)) {
        const int qc = iq & 1;
        if (!wait(C::B_QTFULL + qc, iq >> 1)) {
          ok = false;
          break;
        }
        const uint32_t q_tmem = tmem + (qc ? C::TM_Q1 : C::TM_Q0);
        for (int t = 0; t < part.cnt; ++t, ++g) {
          const int b = g & 1, st = g % C::KS;
          // S_b is free once it has been read (few rows), or PV has read the P over it
          if (!wait(C::B_KFULL + st, g / C::KS) ||
              (g >= 2 && !wait((FEW ? C::B_SREAD : C::B_PVDONE) + b, (g - 2) >> 1))) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t b0 = klo + static_cast<uint32_t>(st * C::T8 >> 4);
          const uint32_t s_tmem = tmem + (b ? C::TM_S1 : C::TM_S0);
#pragma unroll
          for (int part2 = 0; part2 < 2; ++part2)
#pragma unroll
            for (int kk = 0; kk < D / 32; ++kk)
              ptx::umma_ts_f8_if(leader, s_tmem, q_tmem + part2 * (D / 4) + kk * 8, b0 + kk * 2, C::HI_K, C::IDESC_S,
                                 (part2 > 0 || kk > 0) ? 1u : 0u);
          ptx::umma_commit_if(leader, bar(C::B_SFULL + b));
          ptx::umma_commit_if(leader, bar(C::B_KEMPTY + st));
        }
        if (!ok) break;
        ptx::umma_commit_if(leader, bar(C::B_QTEMPTY + qc));
        ++iq;
      }
      if (!ok) {
        ptx::umma_commit_if(leader, bar(C::B_DRAIN));
        volatile int dummy = 0;
        ptx::mbar_wait(bar(C::B_DRAIN), 0, &dummy, a.timeout_ns / 4, 0);
        __syncwarp();
      }
    } else if (warp == 10) {
      // ============================================================ PV issuer
      constexpr uint32_t HI = ptx::sdesc_sw128_hi(1024);
      const uint32_t vlo = ptx::sdesc_sw128_lo(sb + C::OFF_W, C::BK * 128);
      int g = 0, pp = 0;
      bool ok = true;
      while (ok && run.next(a, part)) {
        for (int t = 0; t < part.cnt; ++t, ++g) {
          const int b = g & 1, x = t % C::VT, wb = pp & 1;
          if ((x == 0 && !wait(C::B_WFULL + wb, pp >> 1)) || !wait(C::B_PFULL + b, g >> 1)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t b0 = vlo + static_cast<uint32_t>((wb * C::VT + x) * C::T16 >> 4);
          const uint32_t p_tmem = tmem + (b ? C::TM_P1 : C::TM_P0);
#pragma unroll
          for (int kk = 0; kk < C::BK / 16; ++kk)
            ptx::umma_ts_lohi_if(leader, tmem + C::TM_O, p_tmem + kk * 8, b0 + kk * (2048 >> 4), HI, C::IDESC_PV,
                                 (t > 0 || kk > 0) ? 1u : 0u);
          ptx::umma_commit_if(leader, bar(C::B_PVDONE + b));
          if (x == C::VT - 1 || t == part.cnt - 1) {
            ptx::umma_commit_if(leader, bar(C::B_WEMPTY + wb));
            ++pp;
          }
        }
      }
      if (!ok) {
        ptx::umma_commit_if(leader, bar(C::B_DRAIN + 1));
        volatile int dummy = 0;
        ptx::mbar_wait(bar(C::B_DRAIN + 1), 0, &dummy, a.timeout_ns / 4, 0);
        __syncwarp();
      }
    }
  } else {
    // ================================================================ softmax
    setmaxnreg_inc<C::REGS_SOFTMAX>();
    const int half = lane >> 4;
    const int quad = warp & 3, hw = warp >> 2;
    // lanes 16*hw.. of quarter `quad` hold the 16 rows of block rb, for the
    // tiles of parity hw and part `copy` of their keys (few rows)
    const int rb = Q == 0 ? 2 * quad + hw : (Q == 1 ? quad : (Q == 2 ? (quad & 1) : 0));
    const int copy = Q <= 1 ? 0 : (Q == 2 ? quad >> 1 : quad);
    const int r = rb * 16 + (lane & 15);           // my row
    const int key0 = copy * C::COLS + half * N;    // my first key of a tile
    const int sblk = key0 / kCacheBlock;           // ... its scale block in the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32 + hw * 16) << 16);
    const float ninf = -__int_as_float(0x7f800000);
    uint64_t cap[4];
    if constexpr (MODE == 2) {
#pragma unroll
      for (int u = 0; u < 4; ++u) cap[u] = ptx::f32x2(a.cap_c[u], a.cap_c[u]);
    }
    int g = 0;
    int joins = 0;  // phases of B_JOIN
    bool ok = true;
    // every softmax warp has come here (the copies exchange through shared memory)
    auto join = [&]() -> bool {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_JOIN));
      return ptx::mbar_wait_warp(bar(C::B_JOIN), joins++ & 1, abort_flag, a.timeout_ns, kErrTimeout);
    };
    // Few rows: PV of the last tile before g in the same buffers (of my last one
    // before it, where g is mine) is complete.
    auto pv_before = [&](int g, int b) -> bool {
      return !FEW || g < 2 ||
             ptx::mbar_wait_warp(bar(C::B_PVDONE + b), ((g - 2) >> 1) & 1, abort_flag, a.timeout_ns, kErrTimeout);
    };
    int cq = 0;      // Q copies so far
    int eq_new = 0;  // the last copy's exponent of my row
    // Q of a part into TMEM Q_{cq&1}, hi and lo. First each row by D/8 threads of
    // eight elements: its largest exponent, hi and lo, into shared memory (16-byte
    // units permuted by the row). Then warp w takes the half w/4 of the rows in
    // lanes 32*(w%4) + lane. Rows past the last are zero.
    auto copy_q = [&](const CachePart& p) -> bool {
      constexpr int TPR = D / 8, RPP = 256 / TPR, NP = (C::ROWS + RPP - 1) / RPP, UNITS = D / 16;
      const int c = cq & 1;
      const int rows = min(128, a.R - p.rt * 128);
      const int ch = threadIdx.x % TPR, row0 = threadIdx.x / TPR;
      uint8_t* stage = smem + C::OFF_Q;
      int* eqs = reinterpret_cast<int*>(stage + 2 * C::ROWS * D);
      const uint16_t* qn = a.q + p.n * a.qs_n + static_cast<size_t>(p.hk) * a.group * a.qs_h + ch * 8;
      uint4 x[NP < 4 ? NP : 4];
      bool joined = false;
#pragma unroll 1
      for (int base = 0; base < NP; base += 4) {
#pragma unroll
        for (int u = 0; u < (NP < 4 ? NP : 4); ++u) {
          const int row = row0 + (base + u) * RPP, rr = p.rt * 128 + row;
          const int hg = rr / a.B;
          x[u] = row < rows ? *reinterpret_cast<const uint4*>(qn + hg * a.qs_h + (rr - hg * a.B) * a.qs_b)
                            : make_uint4(0, 0, 0, 0);
        }
        if (!joined) {  // the last copy has been read
          if (!join()) return false;
          joined = true;
        }
#pragma unroll
        for (int u = 0; u < (NP < 4 ? NP : 4); ++u) {
          const int row = row0 + (base + u) * RPP;
          const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          uint32_t mx = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) mx = max(mx, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
          for (int off = TPR / 2; off > 0; off >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          // a row with an infinity or NaN becomes NaN whatever its exponent
          const int e = exponent_for(min(mx, 0x7F7Fu));
          const float inv = pow2i(-e);
          float f[8];
          bf16x8_to_f32(x[u], f);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float f0 = f[2 * k] * inv, f1 = f[2 * k + 1] * inv;
            // infinity has no e4m3
            if (fabsf(f0) == __int_as_float(0x7f800000)) f0 = __int_as_float(0x7fffffff);
            if (fabsf(f1) == __int_as_float(0x7f800000)) f1 = __int_as_float(0x7fffffff);
            hi[k] = pack_e4m3x2(f0, f1);
            float g0, g1;
            unpack_e4m3x2(hi[k], g0, g1);
            lo[k] = pack_e4m3x2(f0 - g0, f1 - g1);
          }
          if (row < C::ROWS) {
            uint8_t* dst = stage + row * D + (((ch >> 1) ^ (row & (UNITS - 1))) << 4) + (ch & 1) * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | (hi[1] << 16), hi[2] | (hi[3] << 16));
            *reinterpret_cast<uint2*>(dst + C::ROWS * D) = make_uint2(lo[0] | (lo[1] << 16), lo[2] | (lo[3] << 16));
            if (ch == 0) eqs[row] = e;
          }
        }
      }
      if (!join()) return false;
      if (cq >= 2 &&
          !ptx::mbar_wait_warp(bar(C::B_QTEMPTY + c), ((cq >> 1) - 1) & 1, abort_flag, a.timeout_ns, kErrTimeout))
        return false;
      ptx::tc_fence_after();
      const int qr = Q == 0 ? quad * 32 + lane : rb * 16 + (lane & 15);
      const uint32_t qa = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (c ? C::TM_Q1 : C::TM_Q0) + hw * (D / 8);
#pragma unroll
      for (int part2 = 0; part2 < 2; ++part2) {  // hi, lo
        uint32_t v[D / 8];
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          const uint4 y = *reinterpret_cast<const uint4*>(stage + part2 * C::ROWS * D + qr * D +
                                                          (((hw * (D / 32) + u) ^ (qr & (UNITS - 1))) << 4));
          v[4 * u] = y.x;
          v[4 * u + 1] = y.y;
          v[4 * u + 2] = y.z;
          v[4 * u + 3] = y.w;
        }
        if constexpr (D == 128) ptx::tmem_st32_16(qa + part2 * (D / 4), v);
        else ptx::tmem_st32_8(qa + part2 * (D / 4), v);
      }
      eq_new = eqs[r];
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(C::B_QTFULL + c));
      ++cq;
      return true;
    };
    // One turn: the next part's Q goes into TMEM, so that its S MMAs start while
    // the last part is written out; then that part's epilogue, then the tiles.
    CachePart nextp;
    bool have = false;  // a part's tiles are done and wait for their epilogue
    int rows = 0, vref = 0;
    bool warp_on = false;
    float m = ninf, l = 0.f;
    while (ok) {
      const bool more = run.next(a, nextp);
      if (more && !copy_q(nextp)) {
        ok = false;
        break;
      }
      if (have) {
        // ---- epilogue. PV(g-1) is the part's last. Few rows: a warp whose own
        // last tile is g-2 knows of no PV after g-4, and the bit of PV(g-1)'s
        // phase may still be that of PV(g-3): PV(g-2) first, which follows it.
        if (!pv_before(g, g & 1) ||
            !ptx::mbar_wait_warp(bar(C::B_PVDONE + ((g - 1) & 1)), ((g - 1) >> 1) & 1, abort_flag, a.timeout_ns,
                                 kErrTimeout)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const bool row_valid = r < rows;
        const float lt = l + __shfl_xor_sync(0xffffffffu, l, 16);
        const bool whole = part.cnt == part.nt;
        const long grow0 = (static_cast<long>(part.n) * a.Hkv + part.hk) * a.R + part.rt * 128;
        const long prow0 = static_cast<long>(2 * blockIdx.x + (part.t0 == 0 ? 1 : 0)) * a.part_rows;
        // sums of my row over all copies, of which mine is number cc
        constexpr int K = FEW ? 2 * Q : 1, RB = FEW ? 4 / Q : 8;  // copies, row blocks
        const int cc = hw * Q + copy;
        float M = m, L = lt;
        if constexpr (FEW) {
          float2* ml = reinterpret_cast<float2*>(smem + C::OFF_J + C::J_BYTES);  // [copy][row]
          if (half == 0) ml[(cc * RB + rb) * 16 + (lane & 15)] = make_float2(m, lt);
          if (!join()) {
            ok = false;
            break;
          }
          M = ninf;
          L = 0.f;
          if (warp_on) {
#pragma unroll
            for (int o = 0; o < K; ++o) M = fmaxf(M, ml[(o * RB + rb) * 16 + (lane & 15)].x);
#pragma unroll
            for (int o = 0; o < K; ++o) {
              const float2 x = ml[(o * RB + rb) * 16 + (lane & 15)];
              L += x.y == 0.f ? 0.f : x.y * ptx::ex2(x.x - M);
            }
          }
        }
        const bool empty = L == 0.f;
        // a copy that saw no key left m at -inf and its O at zero
        const float share = !FEW || m == M ? 1.f : (m == ninf ? 0.f : ptx::ex2(m - M));
        const float f = (empty ? 0.f : share / L) * pow2i(vref);
        if (row_valid && half == 0 && (!FEW || cc == 0)) {
          const float lse2 = empty ? ninf : M - kPShift + ptx::lg2(L);
          if (whole)
            a.lse[grow0 + r] = lse2 * 0.69314718055994530942f -
                               (MODE != 0 ? beyond_keys(a, part.n, part.hk, part.len, part.rt * 128 + r) : 0.f);
          else a.l_part[prow0 + r] = lse2;
        }
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          float v[32];
          if (warp_on) {
            uint32_t raw[32];
            ptx::tmem_ld16x2_32<D / 2>(lane_base + C::TM_O + c * 32, raw);
            ptx::tmem_wait_ld();
            ptx::reg_fence32(raw);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = f == 0.f ? 0.f : __uint_as_float(raw[e]) * f;
          }
          if constexpr (!FEW) {
            if (row_valid) {
              uint4* o_dst = reinterpret_cast<uint4*>(a.o + (grow0 + r) * D) + half * (D / 16) + c * 4;
              float4* p_dst = reinterpret_cast<float4*>(a.o_part + (prow0 + r) * D) + half * (D / 8) + c * 8;
              if (whole) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  o_dst[u] = make_uint4(ptx::pack_bf16x2(v[8 * u], v[8 * u + 1]), ptx::pack_bf16x2(v[8 * u + 2], v[8 * u + 3]),
                                        ptx::pack_bf16x2(v[8 * u + 4], v[8 * u + 5]), ptx::pack_bf16x2(v[8 * u + 6], v[8 * u + 7]));
              } else {
#pragma unroll
                for (int u = 0; u < 8; ++u) p_dst[u] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
              }
            }
          } else {
            // [copy][row][16 float4], the float4 of a row permuted by the row
            float4* jb = reinterpret_cast<float4*>(smem + C::OFF_J);
            if (c > 0 && !join()) {  // the previous columns have been read
              ok = false;
              break;
            }
            if (warp_on) {
              float4* dst = jb + ((cc * RB + rb) * 16 + (lane & 15)) * 16;
#pragma unroll
              for (int u = 0; u < 8; ++u)
                dst[(half * 8 + u) ^ (lane & 15)] = make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
            }
            if (!join()) {
              ok = false;
              break;
            }
            const int tid = threadIdx.x;  // 0..255
            for (int x = tid; x < rows * 16; x += 256) {
              const int row = x >> 4, u = x & 15;
              float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int o = 0; o < K; ++o) {
                const float4 y = jb[(o * RB * 16 + row) * 16 + (u ^ (row & 15))];
                sum.x += y.x;
                sum.y += y.y;
                sum.z += y.z;
                sum.w += y.w;
              }
              // element: half u/8 of the row, 32 columns of this pass
              const int e = (u >> 3) * (D / 2) + c * 32 + (u & 7) * 4;
              if (whole)
                *reinterpret_cast<uint2*>(a.o + (grow0 + row) * D + e) =
                    make_uint2(ptx::pack_bf16x2(sum.x, sum.y), ptx::pack_bf16x2(sum.z, sum.w));
              else
                *reinterpret_cast<float4*>(a.o_part + (prow0 + row) * D + e) = sum;
            }
          }
        }
        if (!ok) break;
        // the next part's first PV overwrites O only after this warp's next PFULL
        // arrival (few rows: after the last join), which follows the loads above
      }
      if (!more) break;
      part = nextp;
      have = true;
      rows = min(128, a.R - part.rt * 128);
      warp_on = rb * 16 < rows;
      const long sbase = (static_cast<long>(part.n) * a.Hkv + part.hk) * (a.C / kCacheBlock);
      const float qmul = pow2i(eq_new);
      float slope2 = 0.f;
      int at = 0;
      if constexpr (MODE != 0) {
        const int rr = min(part.rt * 128 + r, a.R - 1);
        const int hg = rr / a.B;
        if (a.slopes) slope2 = a.slopes[part.hk * a.group + hg] * 1.44269504088896340736f;
        at = nearest_key(query_position(a, part.n, part.len, rr - hg * a.B), part.len);
      }
      m = ninf;
      l = 0.f;
      // <q, k> from the scaled operands; the factor stays finite
      auto scale_of = [&](int t) -> float {
        const int blk = min(t * (C::BK / kCacheBlock) + sblk, a.C / kCacheBlock - 1);
        return warp_on ? a.k_scale[sbase + blk] : 1.f;
      };
      // my tiles: all, or those of parity hw; a tile's scale is read a tile ahead
      const int t_last = part.t0 + part.cnt - 1;
      const int skip = FEW ? ((g ^ hw) & 1) : 0;
      constexpr int STEP = FEW ? 2 : 1;
      const int g_part = g;
      float ks_next = scale_of(max(t_last - skip, 0));
      bool fresh = true;  // no tile of this part yet
      vref = part_vref(a, part, lane);
      for (int jj = skip; jj < part.cnt; jj += STEP) {
        g = g_part + jj;
        const int t = t_last - jj, b = g & 1;
        const float f2 = fminf(qmul * pow2i(scale_exponent(ks_next)), 1e37f);
        if (t >= part.t0 + STEP) ks_next = scale_of(t - STEP);
        if (!ptx::mbar_wait_warp(bar(C::B_SFULL + b), (g >> 1) & 1, abort_flag, a.timeout_ns, kErrTimeout)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float s[N];
        if (warp_on) load_scores<N>(lane_base + (b ? C::TM_S1 : C::TM_S0) + copy * C::COLS, s);
        if constexpr (FEW) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar(C::B_SREAD + b));
        }
        if (warp_on) {
          float f = fminf(fmaxf(f2 * a.scale_log2, 1.17549435e-38f), 1e37f);  // 0 would turn a masked -inf into NaN
          // keys past the length, in an item's last tile only
          const int valid = part.len - t * C::BK - key0;
          const bool ragged = t == part.nt - 1;
          if constexpr (MODE == 2) {
            if (ragged) {  // ... have no say in the path taken
#pragma unroll
              for (int c = 0; c < N; ++c)
                if (c >= valid) s[c] = 0.f;
            }
            const uint64_t f22 = ptx::f32x2(f2, f2);
#pragma unroll
            for (int c = 0; c < N; c += 2)
              ptx::f32x2_split(mul_f32x2(ptx::f32x2(s[c], s[c + 1]), f22), s[c], s[c + 1]);
            // the polynomial while the warp's vote on it is under way
            float y[N];
#pragma unroll
            for (int c = 0; c < N; c += 2) {
              const uint64_t v = ptx::f32x2(s[c], s[c + 1]);
              ptx::f32x2_split(mul_f32x2(v, cap_poly(v, cap)), y[c], y[c + 1]);
            }
            if (__any_sync(0xffffffffu, fmaxf(row_max(s), -row_min(s)) > a.cap_fast)) {
#pragma unroll
              for (int c = 0; c < N; ++c) {  // for large scores only: it is off by 2^-22 of the cap
                const float wide = a.cap_log2 * tanh_wide(s[c] * a.cap_in);
                y[c] = select_f32(fabsf(s[c]) > a.cap_fast, wide, y[c]);
              }
            }
#pragma unroll
            for (int c = 0; c < N; ++c) s[c] = y[c];
            f = 1.f;
            if (a.slopes) scale_and_bias(s, [](uint64_t) { return ptx::f32x2(1.f, 1.f); }, slope2, at, t * C::BK + key0);
          }
          if constexpr (MODE == 1) {
            const uint64_t ff = ptx::f32x2(f, f);
            scale_and_bias(s, [&](uint64_t) { return ff; }, slope2, at, t * C::BK + key0);
            f = 1.f;
          }
          if (ragged) {
#pragma unroll
            for (int c = 0; c < N; ++c)
              if (c >= valid) s[c] = ninf;
          }
          float mx = row_max(s) * f;
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float m_new = fmaxf(m, mx);
          if (fresh) {
            m = m_new;
            fresh = false;
          } else if (__any_sync(0xffffffffu, m_new > m + 8.0f)) {
            // every PV before this tile's is complete, and this one's waits for me.
            // Few rows: S(g) may be there before PV(g-3) is done, when the bit of
            // PV(g-1)'s phase still says the one before it; PV(g-2) follows PV(g-3).
            if (!pv_before(g, b) ||
                !ptx::mbar_wait_warp(bar(C::B_PVDONE + ((g - 1) & 1)), ((g - 1) >> 1) & 1, abort_flag, a.timeout_ns,
                                     kErrTimeout)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
            const float alpha = m_new == ninf ? 1.0f : ptx::ex2(m - m_new);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              uint32_t raw[32];
              ptx::tmem_ld16x2_32<D / 2>(lane_base + C::TM_O + c * 32, raw);
              ptx::tmem_wait_ld();
              ptx::reg_fence32(raw);
#pragma unroll
              for (int e = 0; e < 32; ++e) raw[e] = __float_as_uint(__uint_as_float(raw[e]) * alpha);
              ptx::tmem_st16x2_32<D / 2>(lane_base + C::TM_O + c * 32, raw);
            }
            ptx::tmem_wait_st();
            l *= alpha;
            m = m_new;
          }
          const float neg = (m == ninf ? 0.f : -m) + kPShift;
          const uint64_t f2x = ptx::f32x2(f, f), neg2 = ptx::f32x2(neg, neg);
          uint64_t acc0 = ptx::f32x2(0.f, 0.f), acc1 = acc0;
          uint32_t pk[N / 2];
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            float x0, x1;
            ptx::f32x2_split(ptx::fma_f32x2(ptx::f32x2(s[2 * e], s[2 * e + 1]), f2x, neg2), x0, x1);
            const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
            if (e & 1) acc1 = ptx::add_f32x2(acc1, ptx::f32x2(p0, p1));
            else acc0 = ptx::add_f32x2(acc0, ptx::f32x2(p0, p1));
            pk[e] = ptx::pack_f16x2(p0, p1);
          }
          float a0, a1, b0, b1;
          ptx::f32x2_split(acc0, a0, a1);
          ptx::f32x2_split(acc1, b0, b1);
          l += (a0 + b0) + (a1 + b1);
          if constexpr (FEW) {  // the last P of these columns has been read
            if (!pv_before(g, b)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
          }
          ptx::tmem_st16x2<N / 2>(lane_base + (b ? C::TM_P1 : C::TM_P0) + copy * (C::COLS / 2), pk);
          ptx::tmem_wait_st();
        } else if (!pv_before(g, b)) {
          // a warp without rows keeps the others' pace: two arrivals of it in one
          // phase of PFULL would let PV begin before a slower warp's P is there
          ok = false;
          break;
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bar(C::B_PFULL + b));
      }
      if (!ok) break;
      g = g_part + part.cnt;
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TM_ALLOC);
  }
}

// Joins the partial results of items cut by the ends of runs:
//   O = sum_i 2^(l_i - L) O_i,  L = log2 sum_i 2^(l_i)
// in the order of the runs, and writes the rows of empty sequences.
// blockIdx: item of the sequence (kv head and row tile), sequence, group of
// kMergeRows rows. Thread c looks whether run c holds part of the item; a warp
// then takes whole rows. `runs`: the CTAs of the attention kernel. Launched as
// its programmatic dependent: only the part after grid_dep_wait reads its
// results. Every CTA waits before it ends, also one that has nothing to join:
// what follows on the stream is ordered behind this grid alone, which must not
// end before the attention kernel's last rows are written.
// BIAS: with slopes, a row loses what beyond_keys says (as code that a call
// without them does not run it takes 0.6 us of a single token's 17).
constexpr int kMergeRows = 10;
template <int D, bool BIAS>
__global__ void __launch_bounds__(kCacheMaxCtas) cache_merge_kernel(const __grid_constant__ CacheArgs a, int runs) {
  constexpr int V = D / 32;  // elements of a lane
  constexpr int WARPS = kCacheMaxCtas / 32;
  __shared__ int s_slot[kCacheMaxCtas];     // the item's slots in the order of the runs
  __shared__ int s_count[WARPS];
  __shared__ float s_w[WARPS][kCacheMaxCtas];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float ninf = -__int_as_float(0x7f800000);
  const int n = blockIdx.y, item = blockIdx.x;
  const int hk = item / a.RT, rt = item - hk * a.RT;
  const int r0 = blockIdx.z * kMergeRows;
  const int r1 = min(min(128, a.R - rt * 128), r0 + kMergeRows);
  if (r0 >= r1) {
    ptx::grid_dep_wait();
    return;
  }
  const long grow0 = (static_cast<long>(n) * a.Hkv + hk) * a.R + rt * 128;
  const int len = cache_len(a, n), nt = cache_tiles(a, len);
  if (nt == 0) {
    ptx::grid_dep_wait();  // O and LSE may still be read by what ran before the attention kernel
    for (int r = r0 + warp; r < r1; r += WARPS) {
      for (int e = lane; e < D; e += 32) a.o[(grow0 + r) * D + e] = 0;
      if (lane == 0) a.lse[grow0 + r] = ninf;
    }
    return;
  }
  long before;
  const long T = cache_total(a, lane, n, &before);
  const long x0 = before + static_cast<long>(item) * item_units(a, nt) + a.toll, x1 = x0 + nt;  // the item's tiles
  const int c = threadIdx.x;
  const long b0 = run_begin(T, c, runs), b1 = c < runs ? run_begin(T, c + 1, runs) : b0;
  const bool holds = b0 < b1 && b0 < x1 && b1 > x0;
  const uint32_t vote = __ballot_sync(0xffffffffu, holds);
  if (lane == 0) s_count[warp] = __popc(vote);
  __syncthreads();
  int at = 0, count = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    at += w < warp ? s_count[w] : 0;
    count += s_count[w];
  }
  if (holds) s_slot[at + __popc(vote & ((1u << lane) - 1u))] = 2 * c + (b0 <= x0 ? 1 : 0);
  __syncthreads();
  ptx::grid_dep_wait();
  if (count == 1) return;  // whole in one run: written there
  using Vec = typename std::conditional<V == 4, float4, float2>::type;
  constexpr int BATCH = 8;  // slots whose loads are in flight together
  const long slot_stride = static_cast<long>(a.part_rows) * D;
  for (int r = r0 + warp; r < r1; r += WARPS) {
    const float* base_o = a.o_part + static_cast<long>(r) * D + lane * V;
    float L = ninf, l[WARPS];
#pragma unroll
    for (int u = 0; u < WARPS; ++u) {
      const int i = u * 32 + lane;
      l[u] = i < count ? a.l_part[static_cast<long>(s_slot[i]) * a.part_rows + r] : ninf;
    }
    Vec x[BATCH];
#pragma unroll
    for (int u = 0; u < BATCH; ++u)
      x[u] = *reinterpret_cast<const Vec*>(base_o + s_slot[min(u, count - 1)] * slot_stride);
#pragma unroll
    for (int u = 0; u < WARPS; ++u) L = fmaxf(L, l[u]);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L = fmaxf(L, __shfl_xor_sync(0xffffffffu, L, off));
    const float base = L == ninf ? 0.f : L;
#pragma unroll
    for (int u = 0; u < WARPS; ++u) s_w[warp][u * 32 + lane] = ptx::ex2(l[u] - base);
    __syncwarp();
    float sum = 0.f, acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll 1
    for (int i = 0; i < count; i += BATCH) {
#pragma unroll
      for (int u = 0; u < BATCH; ++u) {
        const float w = i + u < count ? s_w[warp][i + u] : 0.f;
        const float* y = reinterpret_cast<const float*>(&x[u]);
        sum += w;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += i + u < count ? w * y[e] : 0.f;
      }
      if (i + BATCH < count) {
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
          x[u] = *reinterpret_cast<const Vec*>(base_o + s_slot[min(i + BATCH + u, count - 1)] * slot_stride);
      }
    }
    __syncwarp();
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + (grow0 + r) * D) + lane * (V / 2);
#pragma unroll
    for (int e = 0; e < V / 2; ++e) dst[e] = ptx::pack_bf16x2(acc[2 * e] * inv, acc[2 * e + 1] * inv);
    if (lane == 0)
      a.lse[grow0 + r] = sum == 0.f ? ninf
                                    : (base + ptx::lg2(sum)) * 0.69314718055994530942f -
                                          (BIAS ? beyond_keys(a, n, hk, len, rt * 128 + r) : 0.f);
  }
}

}  // namespace sparsed
