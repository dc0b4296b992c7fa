// Host side of the rotary, 8-bit cache and modified-score entry points
// (include/sparsed.h); part of the translation unit of sparsed_api.cu, whose
// helpers it uses.

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// What the launches need of the current device, looked up once per device
// (kernel attributes are per device too). Each entry is written whole before
// `ready` is set; two threads that race write the same values.
constexpr int kMaxDevices = 64;
struct DeviceInfo {
  std::atomic<int> ready{0};
  int sms = 0;
};
DeviceInfo g_device_info[kMaxDevices];

// The current device, which must be sm_100, and its SM count.
int current_device(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess && *dev < kMaxDevices && g_device_info[*dev].ready.load(std::memory_order_acquire)) {
    *sms = g_device_info[*dev].sms;
    return SPARSED_OK;
  }
  SP_TRY(require_sm100());
  SP_TRY(sm_count(sms));
  if (*dev < kMaxDevices) {
    g_device_info[*dev].sms = *sms;
    g_device_info[*dev].ready.store(1, std::memory_order_release);
  }
  return SPARSED_OK;
}

// Raises a kernel's dynamic shared memory limit on the current device and
// checks that its launch funds its register split (as launch_attn_t), once per
// device and kernel (`done`: one bit per device, a static of the launcher).
template <typename Kern>
int prepare_kernel(Kern kern, int dev, int smem, int regs_needed, int threads, std::atomic<uint64_t>* done) {
  const uint64_t bit = dev < kMaxDevices ? 1ull << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return SPARSED_OK;
  cudaFuncAttributes fa;
  SP_CUDA(cudaFuncGetAttributes(&fa, kern));
  if (fa.numRegs * threads < regs_needed) return SPARSED_ERR_UNSUPPORTED;
  SP_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  done->fetch_or(bit, std::memory_order_release);
  return SPARSED_OK;
}

// fraction of 2^64 of x turns (x >= 0; whole turns dropped)
uint64_t turn_fraction(double x) {
  x -= std::floor(x);
  return static_cast<uint64_t>(std::ldexp(x, 64) < 18446744073709549568.0 ? std::ldexp(x, 64) : 18446744073709549568.0);
}

// Whether two of the H x L rows of d elements at h * sh + l * sl share one.
bool rows_overlap(long H, size_t sh, long L, size_t sl, size_t d) {
  if (H > L) return rows_overlap(L, sl, H, sh, d);
  // the usual layouts: the rows of one dimension side by side, those of the other past them
  if (sl >= d && (H == 1 || sh >= sl * static_cast<size_t>(L - 1) + d)) return false;
  if (sh >= d && (L == 1 || sl >= sh * static_cast<size_t>(H - 1) + d)) return false;
  if (L > 1 && sl < d) return true;
  for (long h = 1; h < H; ++h) {  // the rows l of head 0 next to row 0 of head h
    const size_t at = static_cast<size_t>(h) * sh;
    const size_t l = L > 1 ? at / sl : 0;
    if (l < static_cast<size_t>(L) && at - l * sl < d) return true;
    if (l + 1 < static_cast<size_t>(L) && (l + 1) * sl - at < d) return true;
  }
  return false;
}

template <bool I, bool V>
int launch_rope(const RopeArgs& a, dim3 grid, cudaStream_t st) {
  rope_axes_kernel<I, V><<<grid, kRopeThreads, 0, st>>>(a);
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

template <int D>
int launch_append(const AppendArgs& a, bool vec, dim3 grid, cudaStream_t st) {
  if (vec) cache_append_kernel<D, true><<<grid, 256, 0, st>>>(a);
  else cache_append_kernel<D, false><<<grid, 256, 0, st>>>(a);
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

// Scores' options shared by scored_attn and cache_attn. A negative scale would
// turn row maxima into minima and is refused.
int check_mod(float scale, float softcap, const float* slopes) {
  if (!std::isfinite(scale) || scale < 0.f) return SPARSED_ERR_INVALID_ARG;
  if (!std::isfinite(softcap) || softcap < 0.f) return SPARSED_ERR_INVALID_ARG;
  if (!aligned4(slopes)) return SPARSED_ERR_INVALID_ARG;
  return SPARSED_OK;
}

// [H, L, d] bf16 with strides (in elements) as a 3-D tensor map, boxes of 64
// columns x rows.
int make_map_strided(CUtensorMap* m, const void* ptr, int H, int L, int d, size_t stride_h, size_t stride_l,
                     int box_rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(L), static_cast<cuuint64_t>(H)};
  // the stride of a dimension of one says nothing
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(L > 1 ? stride_l : d) * 2,
                           static_cast<cuuint64_t>(H > 1 ? stride_h : d) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail_cuda(cudaErrorInvalidValue);
  return SPARSED_OK;
}

// A strided [H, L, d] operand that a tensor map can describe: strides of 16
// bytes' multiples, not 0 (a broadcast head is fewer kv heads instead).
int check_map_strides(int H, int L, size_t stride_h, size_t stride_l) {
  if (((stride_h | stride_l) & 7u) != 0) return SPARSED_ERR_INVALID_ARG;
  if ((H > 1 && stride_h == 0) || (L > 1 && stride_l == 0)) return SPARSED_ERR_INVALID_ARG;
  if (stride_h >= (1ull << 38) || stride_l >= (1ull << 38)) return SPARSED_ERR_UNSUPPORTED;
  return SPARSED_OK;
}

struct ScoredMaps {
  CUtensorMap q, k, v;
};

template <int D, int CAP, bool BIAS, bool SPLIT>
int launch_scored_t(const ScoredMaps& t, const ScoredArgs& a, int dev, int grid, cudaStream_t st) {
  using C = AttnCfg<D, 128>;
  auto kern = scored_attn_kernel<D, CAP, BIAS, SPLIT>;
  static std::atomic<uint64_t> done{0};
  SP_TRY(prepare_kernel(kern, dev, ScoredCfg<D>::SMEM_BYTES,
                        C::REGS_SOFTMAX * 256 + C::REGS_OTHER * (C::THREADS - 256), C::THREADS, &done));
  kern<<<grid, C::THREADS, ScoredCfg<D>::SMEM_BYTES, st>>>(t.q, t.k, t.v, a);
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

template <int D, int CAP, bool BIAS>
int launch_scored_s(const ScoredMaps& t, const ScoredArgs& a, int dev, int grid, cudaStream_t st) {
  return a.qpp == 1 ? launch_scored_t<D, CAP, BIAS, true>(t, a, dev, grid, st)
                    : launch_scored_t<D, CAP, BIAS, false>(t, a, dev, grid, st);
}
template <int D, int CAP>
int launch_scored_b(const ScoredMaps& t, const ScoredArgs& a, int dev, int grid, cudaStream_t st) {
  return a.slopes ? launch_scored_s<D, CAP, true>(t, a, dev, grid, st) : launch_scored_s<D, CAP, false>(t, a, dev, grid, st);
}
template <int D>
int launch_scored(const ScoredMaps& t, const ScoredArgs& a, float softcap, int dev, int grid, cudaStream_t st) {
  if (softcap > kCapLowMost) return launch_scored_b<D, kCapHigh>(t, a, dev, grid, st);
  if (softcap > 0.f) return launch_scored_b<D, kCapLow>(t, a, dev, grid, st);
  return launch_scored_b<D, kCapNone>(t, a, dev, grid, st);
}

// Capped scores in log2 units: y = s * P(s^2) while |s| * scale / cap <= 0.5,
// with tanh(u) = u * (c0 + c1 u^2 + c2 u^4 + c3 u^6) to 5.7e-7 of it there, and
// (scored_attn alone) with u * (n0 + n1 u^2 + n2 u^4) to 4e-7 of it while it is
// at most 0.25. The fits are minimax in the relative error: a fit of the
// absolute one is off by 1.4e-6 to 2.3e-6 of a score far below the cap, which a
// row of few keys shows in its log-sum.
template <typename Args>
void cap_coefficients(float scale, float softcap, Args* a) {
  constexpr const double (&kC)[4] = kTanhPoly;
  constexpr double kN[3] = {0.999999608340289, -0.3332195994712142, 0.12842442158716916};
  const double u = static_cast<double>(scale) / softcap, cl = softcap * 1.4426950408889634;
  double f = cl * u;
  bool finite = true;
  for (int i = 0; i < 4; ++i, f *= u * u) {
    a->cap_c[i] = static_cast<float>(kC[i] * f);
    if constexpr (std::is_same<Args, ScoredArgs>::value)
      if (i < 3) a->cap_n[i] = static_cast<float>(kN[i] * f);
    finite = finite && std::isfinite(a->cap_c[i]);
  }
  a->cap_in = u < 3e38 ? static_cast<float>(u) : 3e38f;
  a->cap_log2 = static_cast<float>(cl);
  // above this the wide form; everywhere if the polynomial does not fit fp32
  a->cap_fast = !finite ? -1.f : (u > 0 && 0.5 / u < 1e18 ? static_cast<float>(0.5 / u) : 1e18f);
}

// Partial results of cache_attn: two slots per CTA.
struct CachePartLayout {
  int rows;
  size_t lse, total;
};
CachePartLayout cache_part_layout(int B, int group, int d) {
  CachePartLayout w;
  const long rows = static_cast<long>(B) * group;
  w.rows = static_cast<int>(rows < 1 ? 1 : (rows < 128 ? rows : 128));
  w.lse = align256(static_cast<size_t>(2 * kCacheMaxCtas) * w.rows * d * sizeof(float));
  w.total = w.lse + align256(static_cast<size_t>(2 * kCacheMaxCtas) * w.rows * sizeof(float));
  return w;
}

// e4m3 [H, C, d] as a 3-D tensor map, boxes of whole rows.
int make_map_cache(CUtensorMap* m, const uint8_t* ptr, long H, int C, int d, int rows, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(C), static_cast<cuuint64_t>(H)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(C) * d};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(rows), 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(ptr), dims, strides, box, es,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail_cuda(cudaErrorInvalidValue);
  return SPARSED_OK;
}

// The merge kernel asks for the attention kernel's split of an SM's memory: its
// CTAs can then sit beside the last runs, and no SM changes its split.
template <int D, bool BIAS>
int launch_cache_merge(const CacheArgs& a, int dev, unsigned items, int runs, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = dev < kMaxDevices ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_acquire) & bit)) {
    SP_CUDA(cudaFuncSetAttribute(cache_merge_kernel<D, BIAS>, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared));
    done.fetch_or(bit, std::memory_order_release);
  }
  const unsigned row_groups = static_cast<unsigned>(cdiv(a.R < 128 ? a.R : 128, kMergeRows));
  return launch_k(cache_merge_kernel<D, BIAS>, dim3(items, static_cast<unsigned>(a.N), row_groups),
                  dim3(kCacheMaxCtas), 0, st, runs > 0, a, runs > 0 ? runs : 1);
}

template <int D, int MODE, int Q>
int launch_cache_attn(const uint8_t* k8, const uint8_t* v8, CacheArgs& a, int dev, int sms, cudaStream_t st) {
  using C = CacheCfg<D, Q>;
  a.tile = C::BK;
  a.toll = C::FEW ? kTollFew : kTollMany;
  const unsigned items = static_cast<unsigned>(a.Hkv) * static_cast<unsigned>(a.RT);
  if (sms > kCacheMaxCtas) sms = kCacheMaxCtas;
  // no more runs than there can be key tiles
  const long most = static_cast<long>(a.N) * items * cdiv(a.C, C::BK);
  if (static_cast<long>(a.N) * items * (cdiv(a.C, C::BK) + a.toll) / sms >= (1l << 30)) return SPARSED_ERR_UNSUPPORTED;
  const int runs = static_cast<int>(most < sms ? most : sms);
  if (runs > 0) {
    auto kern = cache_attn_kernel<D, MODE, Q>;
    static std::atomic<uint64_t> done{0};
    SP_TRY(prepare_kernel(kern, dev, C::SMEM_BYTES,
                          C::REGS_TOTAL, C::THREADS, &done));
    CUtensorMap tk, tv;
    const long H = static_cast<long>(a.N) * a.Hkv;
    SP_TRY(make_map_cache(&tk, k8, H, a.C, D, C::BK, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B));
    SP_TRY(make_map_cache(&tv, v8, H, a.C, D, C::BK, CU_TENSOR_MAP_SWIZZLE_NONE));
    kern<<<runs, C::THREADS, C::SMEM_BYTES, st>>>(tk, tv, a);
    SP_CUDA(cudaGetLastError());
  }
  return a.slopes ? launch_cache_merge<D, true>(a, dev, items, runs, st)
                  : launch_cache_merge<D, false>(a, dev, items, runs, st);
}

}  // namespace

extern "C" {

int sparsed_rope_axes(const uint16_t* X, size_t x_stride_h, size_t x_stride_l, const int32_t* positions, int n_axes,
                      const int* sections, int H, int L, int d, float theta, int interleaved, int shared_ladder,
                      int inverse, uint16_t* Y, size_t y_stride_h, size_t y_stride_l, void* stream) {
  if (H < 0 || L < 0 || n_axes < 1 || !sections) return SPARSED_ERR_INVALID_ARG;
  if (!std::isfinite(theta) || theta < 1.f) return SPARSED_ERR_INVALID_ARG;
  if (d < 8 || d > 512 || d % 8 != 0 || n_axes > kRopeMaxAxes) return SPARSED_ERR_UNSUPPORTED;
  long J = 0;
  for (int s = 0; s < n_axes; ++s) {
    if (sections[s] < 0) return SPARSED_ERR_INVALID_ARG;
    J += sections[s];
  }
  if (J < 1 || 2 * J > d) return SPARSED_ERR_INVALID_ARG;
  if (J > kRopeMaxPairs) return SPARSED_ERR_UNSUPPORTED;
  if (H == 0 || L == 0) return SPARSED_OK;
  if (!X || !Y || !positions || !aligned2(X) || !aligned2(Y) || !aligned4(positions)) return SPARSED_ERR_INVALID_ARG;
  if (rows_overlap(H, y_stride_h, L, y_stride_l, static_cast<size_t>(d))) return SPARSED_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  SP_TRY(current_device(&dev, &sms));
  RopeArgs a;
  a.x = X;
  a.y = Y;
  a.pos = positions;
  a.xs_h = x_stride_h;
  a.xs_l = x_stride_l;
  a.ys_h = y_stride_h;
  a.ys_l = y_stride_l;
  a.H = H;
  a.L = L;
  a.d = d;
  a.J = static_cast<int>(J);
  a.sign = inverse ? -1 : 1;
  // the ladder of frequencies, kept from the thread's last call with the same
  // axes (J powers cost more than the launch)
  struct Ladder {
    float theta = 0.f;
    int shared = -1, n_axes = 0, sections[kRopeMaxAxes];
    uint64_t turn[kRopeMaxPairs];
    uint8_t axis[kRopeMaxPairs];
  };
  static thread_local Ladder ladder;
  const int shared = shared_ladder != 0;
  if (ladder.theta != theta || ladder.shared != shared || ladder.n_axes != n_axes ||
      std::memcmp(ladder.sections, sections, n_axes * sizeof(int)) != 0) {
    ladder.theta = theta;
    ladder.shared = shared;
    ladder.n_axes = n_axes;
    std::memcpy(ladder.sections, sections, n_axes * sizeof(int));
    int j = 0;
    for (int s = 0; s < n_axes; ++s)
      for (int i = 0; i < sections[s]; ++i, ++j) {
        const double ex = shared ? static_cast<double>(j) / static_cast<double>(J)
                                 : static_cast<double>(i) / sections[s];
        ladder.turn[j] = turn_fraction(std::pow(static_cast<double>(theta), -ex) * 0.15915494309189533577);
        ladder.axis[j] = static_cast<uint8_t>(s);
      }
  }
  std::memcpy(a.turn, ladder.turn, J * sizeof(uint64_t));
  std::memcpy(a.axis, ladder.axis, J);
  a.rot_units = static_cast<int>(cdiv(J, 8));
  a.units = a.rot_units + static_cast<int>(cdiv(d - 2 * J, 8));
  const bool vec = J % 8 == 0 && aligned16(X) && aligned16(Y) &&
                   ((x_stride_h | x_stride_l | y_stride_h | y_stride_l) & 7u) == 0;
  const long gx = cdiv(L, kRopeThreads / a.units);
  // as many heads per CTA as leave about four CTAs per SM: a CTA takes its
  // sines and cosines once for all its heads
  long share = gx * H / (4l * sms);
  share = share < 1 ? 1 : (share > 16 ? 16 : share);
  a.heads_per_cta = static_cast<int>(share < H ? share : H);
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(cdiv(H, a.heads_per_cta)));
  if (grid.y > 65535u) return SPARSED_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (interleaved) return vec ? launch_rope<true, true>(a, grid, st) : launch_rope<true, false>(a, grid, st);
  return vec ? launch_rope<false, true>(a, grid, st) : launch_rope<false, false>(a, grid, st);
}

int sparsed_cache_append(const uint16_t* K, size_t k_stride_n, size_t k_stride_h, size_t k_stride_b,
                         const uint16_t* V, size_t v_stride_n, size_t v_stride_h, size_t v_stride_b,
                         int N, int H, int B, int C, int d, const int32_t* start, const int32_t* count,
                         uint8_t* k8, uint8_t* v8, float* k_scale, float* v_scale, void* stream) {
  if (N < 0 || H < 0 || B < 0 || C < 0) return SPARSED_ERR_INVALID_ARG;
  if (C % kCacheBlock != 0) return SPARSED_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SPARSED_ERR_UNSUPPORTED;
  if (N > 65535 || H > 65535 || C > (1 << 30)) return SPARSED_ERR_UNSUPPORTED;
  if (N == 0 || H == 0 || B == 0) return SPARSED_OK;
  if (B > C) return SPARSED_ERR_INVALID_ARG;
  if (!K || !V || !start || !k8 || !v8 || !k_scale || !v_scale) return SPARSED_ERR_INVALID_ARG;
  if (!aligned2(K) || !aligned2(V) || !aligned16(k8) || !aligned16(v8) || !aligned4(k_scale) || !aligned4(v_scale) ||
      !aligned4(start) || !aligned4(count))
    return SPARSED_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  SP_TRY(current_device(&dev, &sms));
  AppendArgs a;
  a.x[0] = K;
  a.x[1] = V;
  a.s_n[0] = k_stride_n;
  a.s_h[0] = k_stride_h;
  a.s_b[0] = k_stride_b;
  a.s_n[1] = v_stride_n;
  a.s_h[1] = v_stride_h;
  a.s_b[1] = v_stride_b;
  a.x8[0] = k8;
  a.x8[1] = v8;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.start = start;
  a.count = count;
  a.N = N;
  a.H = H;
  a.B = B;
  a.C = C;
  const bool vec = aligned16(K) && aligned16(V) &&
                   ((k_stride_n | k_stride_h | k_stride_b | v_stride_n | v_stride_h | v_stride_b) & 7u) == 0;
  // blocks that B tokens can touch, wherever the first one lies in its block
  const unsigned blocks = static_cast<unsigned>((B + 2 * kCacheBlock - 2) / kCacheBlock);
  const dim3 grid(2 * blocks, static_cast<unsigned>(H), static_cast<unsigned>(N));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d == 64 ? launch_append<64>(a, vec, grid, st) : launch_append<128>(a, vec, grid, st);
}

int sparsed_cache_attn_workspace_bytes(int N, int Hq, int Hkv, int B, int d, size_t* bytes) {
  if (!bytes || N < 0 || Hq < 0 || Hkv < 0 || B < 0) return SPARSED_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SPARSED_ERR_UNSUPPORTED;
  *bytes = cache_part_layout(B, Hkv > 0 ? Hq / Hkv : 0, d).total;
  return SPARSED_OK;
}

int sparsed_cache_attn(const uint16_t* Q, size_t q_stride_n, size_t q_stride_h, size_t q_stride_b,
                       const uint8_t* k8, const uint8_t* v8, const float* k_scale, const float* v_scale,
                       int N, int Hq, int Hkv, int B, int C, int d, const int32_t* lengths, const int32_t* q_start,
                       float scale, float softcap, const float* slopes, uint16_t* O, float* LSE,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (N < 0 || Hq < 0 || Hkv < 0 || B < 0 || C < 0) return SPARSED_ERR_INVALID_ARG;
  SP_TRY(check_mod(scale, softcap, slopes));
  if (C % kCacheBlock != 0) return SPARSED_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return SPARSED_ERR_UNSUPPORTED;
  if (N == 0 || Hq == 0 || B == 0) return SPARSED_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return SPARSED_ERR_INVALID_ARG;
  if (N > 16384 || Hq > 65535 || C > (1 << 29) || B > (1 << 24)) return SPARSED_ERR_UNSUPPORTED;
  if (!Q || !O || !LSE || !lengths || (C > 0 && (!k8 || !v8 || !k_scale || !v_scale))) return SPARSED_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k8) || !aligned16(v8) || !aligned16(O) || !aligned4(LSE) || !aligned4(lengths) ||
      !aligned4(q_start) || !aligned4(k_scale) || !aligned4(v_scale))
    return SPARSED_ERR_INVALID_ARG;
  if (((q_stride_n | q_stride_h | q_stride_b) & 7u) != 0) return SPARSED_ERR_INVALID_ARG;
  const CachePartLayout w = cache_part_layout(B, Hq / Hkv, d);
  if (!workspace || workspace_bytes < w.total || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPARSED_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  SP_TRY(current_device(&dev, &sms));
  SP_TRY(get_encoder());
  CacheArgs a = {};
  a.q = Q;
  a.qs_n = q_stride_n;
  a.qs_h = q_stride_h;
  a.qs_b = q_stride_b;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.lengths = lengths;
  a.q_start = q_start;
  a.N = N;
  a.Hkv = Hkv;
  a.group = Hq / Hkv;
  a.B = B;
  a.C = C;
  const long R = static_cast<long>(a.group) * B;
  if (R >= (1l << 30)) return SPARSED_ERR_UNSUPPORTED;
  a.R = static_cast<int>(R);
  a.RT = static_cast<int>(cdiv(R, 128));
  a.part_rows = w.rows;
  a.scale_log2 = scale * 1.44269504088896340736f;
  if (a.scale_log2 < 1.17549435e-38f) a.scale_log2 = 1.17549435e-38f;  // as scored_attn
  a.slopes = slopes;
  const int mode = softcap > 0.f ? 2 : (slopes ? 1 : 0);
  if (mode == 2) cap_coefficients(scale, softcap, &a);
  a.o = O;
  a.lse = LSE;
  a.o_part = static_cast<float*>(workspace);
  a.l_part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + w.lse);
  a.timeout_ns = kWaitTimeoutNs;
  const long items = static_cast<long>(Hkv) * a.RT;
  if (items >= (1l << 31)) return SPARSED_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // the few-rows form as far as its lanes reach, with the most copies of the rows
  const int form = R <= 16 ? 4 : (R <= 32 ? 2 : (R <= 64 ? 1 : 0));
#define SP_CACHE(D_, MODE_)                                                                      \
  if (d == D_ && mode == MODE_) {                                                                \
    if (form == 4) return launch_cache_attn<D_, MODE_, 4>(k8, v8, a, dev, sms, st);              \
    if (form == 2) return launch_cache_attn<D_, MODE_, 2>(k8, v8, a, dev, sms, st);              \
    if (form == 1) return launch_cache_attn<D_, MODE_, 1>(k8, v8, a, dev, sms, st);              \
    return launch_cache_attn<D_, MODE_, 0>(k8, v8, a, dev, sms, st);                             \
  }
  SP_CACHE(64, 0)
  SP_CACHE(64, 1)
  SP_CACHE(64, 2)
  SP_CACHE(128, 0)
  SP_CACHE(128, 1)
  SP_CACHE(128, 2)
#undef SP_CACHE
  return SPARSED_ERR_UNSUPPORTED;
}

int sparsed_document_ranges(const int32_t* starts, const int32_t* prefix, int n_docs, int L, int32_t* ranges,
                            void* stream) {
  if (n_docs < 0 || L < 0) return SPARSED_ERR_INVALID_ARG;
  if (L == 0) return SPARSED_OK;
  if (!starts || !ranges || !aligned4(starts) || !aligned4(prefix) || (reinterpret_cast<uintptr_t>(ranges) & 7u))
    return SPARSED_ERR_INVALID_ARG;
  int dev = 0, sms = 0;
  SP_TRY(current_device(&dev, &sms));
  document_ranges_kernel<<<static_cast<unsigned>(cdiv(L, 256)), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      starts, prefix, n_docs, L, reinterpret_cast<int2*>(ranges));
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

int sparsed_scored_attn_workspace_bytes(int Hq, int Lq, size_t* bytes) {
  if (!bytes || Hq < 0 || Lq < 0) return SPARSED_ERR_INVALID_ARG;
  *bytes = 256;
  return SPARSED_OK;
}

int sparsed_scored_attn(const uint16_t* Q, size_t q_stride_h, size_t q_stride_l,
                        const uint16_t* K, size_t k_stride_h, size_t k_stride_l,
                        const uint16_t* V, size_t v_stride_h, size_t v_stride_l,
                        int Hq, int Hkv, int Lq, int Lk, int d, float scale, float softcap, const float* slopes,
                        int q_start, const int32_t* ranges, uint16_t* O, float* LSE,
                        void* workspace, size_t workspace_bytes, void* stream) {
  if (Hq < 0 || Hkv < 0 || Lq < 0 || Lk < 0) return SPARSED_ERR_INVALID_ARG;
  SP_TRY(check_mod(scale, softcap, slopes));
  if (d != 64 && d != 128) return SPARSED_ERR_UNSUPPORTED;
  if (Hq == 0 || Lq == 0) return SPARSED_OK;
  if (Hkv == 0 || Hq % Hkv != 0) return SPARSED_ERR_INVALID_ARG;
  if (Hq > 65535 || Lq > (1 << 29) || Lk > (1 << 29) || q_start > (1 << 29) || q_start < -(1 << 29))
    return SPARSED_ERR_UNSUPPORTED;
  if (!Q || !O || !LSE || (Lk > 0 && (!K || !V))) return SPARSED_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned4(LSE) ||
      (reinterpret_cast<uintptr_t>(ranges) & 7u))
    return SPARSED_ERR_INVALID_ARG;
  SP_TRY(check_map_strides(Hq, Lq, q_stride_h, q_stride_l));
  SP_TRY(check_map_strides(Hkv, Lk, k_stride_h, k_stride_l));
  SP_TRY(check_map_strides(Hkv, Lk, v_stride_h, v_stride_l));
  size_t need = 0;
  SP_TRY(sparsed_scored_attn_workspace_bytes(Hq, Lq, &need));
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPARSED_ERR_WORKSPACE;
  int dev = 0, sms = 0;
  SP_TRY(current_device(&dev, &sms));
  SP_TRY(get_encoder());
  ScoredMaps t;
  SP_TRY(make_map_strided(&t.q, Q, Hq, Lq, d, q_stride_h, q_stride_l, 128));
  if (Lk > 0) {
    SP_TRY(make_map_strided(&t.k, K, Hkv, Lk, d, k_stride_h, k_stride_l, 128));
    SP_TRY(make_map_strided(&t.v, V, Hkv, Lk, d, v_stride_h, v_stride_l, 128));
  } else {
    t.k = t.v = t.q;  // no key, no tile is read
  }
  ScoredArgs a = {};
  a.H = Hq;
  a.group = Hq / Hkv;
  a.L = Lq;
  a.Lk = Lk;
  a.nqb = static_cast<int>(cdiv(Lq, 128));
  // tiles in pairs share K/V tiles; single ones, their keys split over the two
  // slots, while each can have its own SM (8 heads of 1000 tokens: 21 to 18 us)
  a.qpp = static_cast<long>(Hq) * a.nqb <= sms ? 1 : 2;
  const long turns = static_cast<long>(Hq) * cdiv(a.nqb, a.qpp);
  if (turns >= (1l << 31) - sms) return SPARSED_ERR_UNSUPPORTED;
  a.scale_log2 = scale * 1.44269504088896340736f;
  if (a.scale_log2 < 1.17549435e-38f) a.scale_log2 = 1.17549435e-38f;  // 0 would turn a masked -inf into NaN
  a.slopes = slopes;
  a.q_start = q_start;
  a.ranges = reinterpret_cast<const int2*>(ranges);
  if (softcap > 0.f) cap_coefficients(scale, softcap, &a);
  a.lse = LSE;
  a.o = O;
  a.timeout_ns = kWaitTimeoutNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // more turns than CTAs: later ones are claimed from a counter
  if (turns > sms) {
    a.sched = static_cast<int*>(workspace);
    SP_CUDA(cudaMemsetAsync(a.sched, 0, sizeof(int), st));
  }
  const int grid = static_cast<int>(turns < sms ? turns : sms);
  return d == 64 ? launch_scored<64>(t, a, softcap, dev, grid, st) : launch_scored<128>(t, a, softcap, dev, grid, st);
}

}  // extern "C"
