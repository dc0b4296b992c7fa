// Host side of the rotary, 8-bit cache and modified-score entry points
// (include/sparsed.h); part of the translation unit of sparsed_api.cu, whose
// helpers it uses.

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

// fraction of 2^64 of x turns (x >= 0; whole turns dropped)
uint64_t turn_fraction(double x) {
  x -= std::floor(x);
  return static_cast<uint64_t>(std::ldexp(x, 64) < 18446744073709549568.0 ? std::ldexp(x, 64) : 18446744073709549568.0);
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
  SP_TRY(require_sm100());
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
  int j = 0;
  for (int s = 0; s < n_axes; ++s)
    for (int i = 0; i < sections[s]; ++i, ++j) {
      const double ex = shared_ladder ? static_cast<double>(j) / static_cast<double>(J)
                                      : static_cast<double>(i) / sections[s];
      a.turn[j] = turn_fraction(std::pow(static_cast<double>(theta), -ex) * 0.15915494309189533577);
      a.axis[j] = static_cast<uint8_t>(s);
    }
  a.rot_units = static_cast<int>(cdiv(J, 8));
  a.units = a.rot_units + static_cast<int>(cdiv(d - 2 * J, 8));
  const bool vec = J % 8 == 0 && aligned16(X) && aligned16(Y) &&
                   ((x_stride_h | x_stride_l | y_stride_h | y_stride_l) & 7u) == 0;
  const long gx = cdiv(L, kRopeThreads / a.units);
  // as many heads per CTA as leave about four CTAs per SM: a CTA takes its
  // sines and cosines once for all its heads
  int sms = 0;
  SP_TRY(sm_count(&sms));
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
  SP_TRY(require_sm100());
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
  *bytes = 256;
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
  if (N > 65535 || Hq > 65535 || C > (1 << 30)) return SPARSED_ERR_UNSUPPORTED;
  if (!Q || !k8 || !v8 || !k_scale || !v_scale || !lengths || !O || !LSE) return SPARSED_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k8) || !aligned16(v8) || !aligned16(O) || !aligned4(LSE) || !aligned4(lengths) ||
      !aligned4(q_start) || !aligned4(k_scale) || !aligned4(v_scale))
    return SPARSED_ERR_INVALID_ARG;
  if (((q_stride_n | q_stride_h | q_stride_b) & 7u) != 0) return SPARSED_ERR_INVALID_ARG;
  size_t need = 0;
  SP_TRY(sparsed_cache_attn_workspace_bytes(N, Hq, Hkv, B, d, &need));
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPARSED_ERR_WORKSPACE;
  SP_TRY(require_sm100());
  RowsArgs a = {};
  a.q = Q;
  a.qs_n = q_stride_n;
  a.qs_h = q_stride_h;
  a.qs_b = q_stride_b;
  a.k8 = k8;
  a.v8 = v8;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.B = B;
  a.Lk = C;
  a.lengths = lengths;
  a.q_start = q_start;
  a.mod = ScoreMod{scale, softcap, slopes};
  a.o = O;
  a.lse = LSE;
  const dim3 grid(B, Hq, N);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 64) score_rows_kernel<64><<<grid, 128, 0, st>>>(a);
  else score_rows_kernel<128><<<grid, 128, 0, st>>>(a);
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

int sparsed_document_ranges(const int32_t* starts, const int32_t* prefix, int n_docs, int L, int32_t* ranges,
                            void* stream) {
  if (n_docs < 0 || L < 0) return SPARSED_ERR_INVALID_ARG;
  if (L == 0) return SPARSED_OK;
  if (!starts || !ranges || !aligned4(starts) || !aligned4(prefix) || (reinterpret_cast<uintptr_t>(ranges) & 7u))
    return SPARSED_ERR_INVALID_ARG;
  SP_TRY(require_sm100());
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
  if (Hq > 65535 || Lq > (1 << 30) || Lk > (1 << 30) || q_start > (1 << 30) || q_start < -(1 << 30))
    return SPARSED_ERR_UNSUPPORTED;
  if (!Q || !O || !LSE || (Lk > 0 && (!K || !V))) return SPARSED_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned4(LSE) ||
      (reinterpret_cast<uintptr_t>(ranges) & 7u))
    return SPARSED_ERR_INVALID_ARG;
  if (((q_stride_h | q_stride_l | k_stride_h | k_stride_l | v_stride_h | v_stride_l) & 7u) != 0)
    return SPARSED_ERR_INVALID_ARG;
  size_t need = 0;
  SP_TRY(sparsed_scored_attn_workspace_bytes(Hq, Lq, &need));
  if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return SPARSED_ERR_WORKSPACE;
  SP_TRY(require_sm100());
  RowsArgs a = {};
  a.q = Q;
  a.qs_h = q_stride_h;
  a.qs_b = q_stride_l;
  a.k = K;
  a.v = V;
  a.ks_h = k_stride_h;
  a.ks_l = k_stride_l;
  a.vs_h = v_stride_h;
  a.vs_l = v_stride_l;
  a.N = 1;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.B = Lq;
  a.Lk = Lk;
  a.q_start0 = q_start;
  a.ranges = ranges;
  a.mod = ScoreMod{scale, softcap, slopes};
  a.o = O;
  a.lse = LSE;
  const dim3 grid(Lq, Hq, 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 64) score_rows_kernel<64><<<grid, 128, 0, st>>>(a);
  else score_rows_kernel<128><<<grid, 128, 0, st>>>(a);
  SP_CUDA(cudaGetLastError());
  return SPARSED_OK;
}

}  // extern "C"
