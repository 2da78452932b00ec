// Host side of the adapter entry points.  Included by segquant.cu behind its
// helpers and api_group_norm.cuh.
#pragma once

namespace {

sq_status check_adapters(const sq_adapters* ad, const int32_t* bounds, const int32_t* index, int32_t requests,
                         int64_t M) {
  if (ad == nullptr || ad->L <= 0 || ad->R <= 0 || ad->K <= 0 || ad->N <= 0) return SQ_ERR_INVALID_ARG;
  if (M < 0 || requests < 0) return SQ_ERR_INVALID_ARG;
  if (ad->a == nullptr || ad->b == nullptr) return SQ_ERR_INVALID_ARG;
  if (ad->R % 8 != 0 || ad->R > sq::kAdapterMaxRank || ad->K % 16 != 0 || ad->N % 16 != 0) return SQ_ERR_UNSUPPORTED;
  if (ad->K > SQ_MAX_K || ad->N > SQ_MAX_K || M > (1 << 30) || requests > (1 << 24) ||
      (int64_t)ad->L * std::max(ad->K, ad->N) > (int64_t)INT32_MAX - 256)
    return SQ_ERR_RANGE;
  if (!aligned16(ad->a) || !aligned16(ad->b)) return SQ_ERR_ALIGNMENT;
  if (bounds == nullptr || (requests > 0 && index == nullptr)) return SQ_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(bounds) & 3u) || (reinterpret_cast<uintptr_t>(index) & 3u) ||
      (reinterpret_cast<uintptr_t>(ad->scale) & 3u))
    return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

sq_status check_matrix(const void* p, sq_dtype t, int64_t cols, int64_t ld) {
  if (!dtype_ok(t) || ld < cols || p == nullptr) return SQ_ERR_INVALID_ARG;
  if (!aligned16(p) || (ld * elt_size(t)) % 16 != 0) return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

sq::AdapterArgs adapter_args(const sq_adapters* ad, const int32_t* bounds, const int32_t* index, int32_t requests,
                             int64_t M) {
  sq::AdapterArgs a = {};
  a.a = static_cast<const __nv_bfloat16*>(ad->a);
  a.b = static_cast<const __nv_bfloat16*>(ad->b);
  a.scale = ad->scale;
  a.bounds = bounds;
  a.index = index;
  a.M = (int32_t)M;
  a.K = (int32_t)ad->K;
  a.N = (int32_t)ad->N;
  a.L = ad->L;
  a.R = ad->R;
  a.Q = requests;
  return a;
}

template <bool BWD>
sq_status launch_few_rows(const sq::AdapterArgs& a, sq_dtype xt, sq_dtype yt, cudaStream_t s) {
  const int64_t slots = (int64_t)a.M / sq::kFewRows + a.Q + 3;
  // enough CTAs for one wave over the SMs, no slice shorter than a warp's loads
  int cs = 1;
  while (cs < 8 && slots * cs * 2 <= 3 * (int64_t)num_sms() && std::min(a.K, a.N) >= 512 * cs) cs *= 2;
  const dim3 grid((unsigned)(slots * cs));
  if (xt == SQ_BF16)
    return yt == SQ_BF16
               ? launch_grid<sq::adapter_few_rows_kernel<__nv_bfloat16, __nv_bfloat16, BWD>>(grid, sq::kFewThreads, 0, cs, false, s, a, cs)
               : launch_grid<sq::adapter_few_rows_kernel<__nv_bfloat16, float, BWD>>(grid, sq::kFewThreads, 0, cs, false, s, a, cs);
  return yt == SQ_BF16
             ? launch_grid<sq::adapter_few_rows_kernel<float, __nv_bfloat16, BWD>>(grid, sq::kFewThreads, 0, cs, false, s, a, cs)
             : launch_grid<sq::adapter_few_rows_kernel<float, float, BWD>>(grid, sq::kFewThreads, 0, cs, false, s, a, cs);
}

template <bool TRANS>
sq_status launch_adapter_grad(const sq::AdapterGradArgs& g, sq_dtype gt, cudaStream_t s) {
  const dim3 grid((unsigned)((g.C + sq::kGradCols - 1) / sq::kGradCols), (unsigned)g.L);
  if (gt == SQ_BF16)
    return launch_grid<sq::adapter_grad_kernel<__nv_bfloat16, TRANS>>(grid, sq::kGradThreads, 0, 1, false, s, g);
  return launch_grid<sq::adapter_grad_kernel<float, TRANS>>(grid, sq::kGradThreads, 0, 1, false, s, g);
}

}  // namespace

extern "C" {

sq_status sq_adapter_add(const void* x, sq_dtype xt, int64_t M, int64_t ldx, const sq_adapters* adapters,
                         const int32_t* bounds, const int32_t* index, int32_t requests, void* y, sq_dtype yt,
                         int64_t ldy, float* hidden, sq_stream_t stream) {
  sq_status st = check_adapters(adapters, bounds, index, requests, M);
  if (st != SQ_OK) return st;
  if (!dtype_ok(xt) || !dtype_ok(yt)) return SQ_ERR_INVALID_ARG;
  if (M == 0 || (requests == 0 && hidden == nullptr)) return SQ_OK;
  if ((st = check_matrix(x, xt, adapters->K, ldx)) != SQ_OK) return st;
  if ((st = check_matrix(y, yt, adapters->N, ldy)) != SQ_OK) return st;
  if (hidden != nullptr && !aligned16(hidden)) return SQ_ERR_ALIGNMENT;
  sq::AdapterArgs a = adapter_args(adapters, bounds, index, requests, M);
  a.x = x; a.ldx = ldx; a.y = y; a.ldy = ldy; a.h = hidden;
  return launch_few_rows<false>(a, xt, yt, reinterpret_cast<cudaStream_t>(stream));
}

sq_status sq_adapter_backward_workspace_size(int64_t M, int32_t R, size_t* bytes) {
  if (bytes == nullptr || M < 0 || R <= 0) return SQ_ERR_INVALID_ARG;
  *bytes = sizeof(float) * (size_t)M * (size_t)R;
  return SQ_OK;
}

sq_status sq_adapter_backward(const void* dy, sq_dtype dyt, int64_t M, int64_t lddy, const void* x, sq_dtype xt,
                              int64_t ldx, const float* hidden, const sq_adapters* adapters, const int32_t* bounds,
                              const int32_t* index, int32_t requests, void* dx, int64_t lddx, float* da, float* db,
                              void* workspace, size_t workspace_bytes, sq_stream_t stream) {
  sq_status st = check_adapters(adapters, bounds, index, requests, M);
  if (st != SQ_OK) return st;
  if (!dtype_ok(xt) || !dtype_ok(dyt) || da == nullptr || db == nullptr) return SQ_ERR_INVALID_ARG;
  if (!aligned16(da) || !aligned16(db)) return SQ_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M > 0) {
    if ((st = check_matrix(dy, dyt, adapters->N, lddy)) != SQ_OK) return st;
    if ((st = check_matrix(x, xt, adapters->K, ldx)) != SQ_OK) return st;
    if ((st = check_matrix(dx, xt, adapters->K, lddx)) != SQ_OK) return st;
    if (hidden == nullptr || workspace == nullptr || workspace_bytes < sizeof(float) * (size_t)M * adapters->R)
      return SQ_ERR_INVALID_ARG;
    if (!aligned16(hidden) || !aligned16(workspace)) return SQ_ERR_ALIGNMENT;
    sq::AdapterArgs a = adapter_args(adapters, bounds, index, requests, M);
    a.x = dy; a.ldx = lddy; a.y = dx; a.ldy = lddx; a.h = static_cast<float*>(workspace);
    if ((st = launch_few_rows<true>(a, dyt, xt, s)) != SQ_OK) return st;
  }
  sq::AdapterGradArgs g = {};
  g.bounds = bounds; g.index = index; g.M = (int32_t)M; g.R = adapters->R; g.L = adapters->L;
  g.Q = M > 0 ? requests : 0;
  g.f = static_cast<const float*>(workspace); g.g = x; g.ldg = ldx; g.C = (int32_t)adapters->K; g.out = da;
  if ((st = launch_adapter_grad<false>(g, xt, s)) != SQ_OK) return st;
  g.f = hidden; g.g = dy; g.ldg = lddy; g.C = (int32_t)adapters->N; g.out = db; g.scale = adapters->scale;
  return launch_adapter_grad<true>(g, dyt, s);
}

}  // extern "C"
