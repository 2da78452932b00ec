// Host side of the group norm entry points: argument checks, the choice of
// tiles, and launches.  Included by segquant.cu behind its helpers.
#pragma once

namespace {

constexpr int kNormSmem = 227 * 1024;

// How a [B, S, C] map is cut.  cluster = true: a cluster of cs CTAs holds the
// slab of an image and channel block in shared memory, nv vectors per thread.
struct NormPlan {
  sq::NormTile t;
  int cs, nv, tiles;
  int threads;        // of the two-pass form
  bool cluster;
};

int gcd_i(int a, int b) { return b == 0 ? a : gcd_i(b, a % b); }

// Shared memory of a cluster CTA: `tensors` slabs of nv vectors per thread, and the
// reductions.
int norm_cluster_smem(const sq::NormTile& t, int nv, int vn, int tensors) {
  return nv * sq::kNormThreads * 16 * tensors + 4 * sq::norm_smem_floats(sq::kNormThreads, t.vx, vn, t.nb);
}

// Chooses the tiles of `tensors` read (1 forward: x; 2 backward: x and dy).
sq_status norm_plan_for(int64_t B, int64_t S, int64_t C, int32_t groups, int es, int tensors, NormPlan* out) {
  const int vn = 16 / es;
  const int cpg = (int)(C / groups);
  const int unit = vn / gcd_i(vn, cpg);                 // groups in whole vectors
  const int64_t unit_vec = (int64_t)unit * cpg / vn;
  if (unit_vec > sq::kNormThreadsMax) return SQ_ERR_UNSUPPORTED;
  const int blocks_all = groups / unit;                 // C is a multiple of the vector
  const int sms = num_sms();
  NormPlan best = {};
  double best_us = 1e30;
  for (int m = 1; m <= blocks_all; ++m) {
    if (blocks_all % m != 0) continue;
    const int64_t vx = unit_vec * m;
    if (vx > sq::kNormThreads) break;
    const int ty = (int)(sq::kNormThreads / vx);
    for (int cs = 1; cs <= 8; cs *= 2) {
      const int64_t rows = (S + cs - 1) / cs;
      const int64_t nv = (rows + ty - 1) / ty;
      if (cs > 1 && (int64_t)(cs - 1) * rows >= S) continue;   // a CTA without rows
      if (nv > 64) continue;
      const sq::NormTile t{(int32_t)S, (int32_t)C, groups, cpg, unit * m, (int32_t)vx, ty, (int32_t)rows};
      const int smem = norm_cluster_smem(t, (int)nv, vn, tensors) + 1024;
      if (smem > kNormSmem) continue;
      // Estimated time: waves of resident CTAs, each the latency of its loads, reductions
      // and stores and of the cluster barriers, its arithmetic (an SM's 16 warps or more
      // take 0.022 us a KB, fewer in proportion longer), and its traffic at an SM's share of
      // the copy rate (44 KB/us); fitted to all choices at eight sizes.
      const int res = std::min(tensors == 1 ? 3 : 2, kNormSmem / smem);
      const int64_t ctas = B * (blocks_all / m) * cs;
      const int64_t waves = (ctas + (int64_t)sms * res - 1) / ((int64_t)sms * res);
      const double on_sm = (double)std::min<int64_t>(res, (ctas + sms - 1) / sms);
      const int chunk = (int)vx * 16;
      const double waste = chunk % 32 == 0 || chunk >= C * es ? 1.0 : (double)((chunk + 31) / 32 * 32 + 16) / chunk;
      const double slab = (double)rows * chunk / 1024.0;
      const double busy = std::max(1.0, 16.0 / (on_sm * sq::kNormThreads / 32.0));
      const double us = (double)waves * (2.0 + 0.7 * (cs > 1) + 0.15 * (cs - 1) +
                                         on_sm * slab * (0.022 * tensors * busy + waste * (tensors + 1) / 44.0));
      if (us < best_us) {
        best_us = us;
        best.t = t;
        best.cs = cs;
        best.nv = (int)nv;
        best.tiles = 1;
        best.cluster = true;
      }
    }
  }
  // Two passes read the inputs twice, the second time mostly from L2, in two
  // launches.
  const double total_kb = (double)B * S * C * es / 1024.0;
  const double two_us = 8.0 + total_kb * (2 * tensors + 1) / (44.0 * sms);
  if (best_us <= two_us) {
    *out = best;
    return SQ_OK;
  }
  NormPlan p = {};
  p.threads = unit_vec <= sq::kNormThreads ? sq::kNormThreads : sq::kNormThreadsMax;
  int m = 1;
  for (int k = 1; k <= blocks_all; ++k)
    if (blocks_all % k == 0 && unit_vec * k <= p.threads) m = k;
  const int vx = (int)(unit_vec * m), ty = p.threads / vx;
  const int64_t cols = (int64_t)B * (blocks_all / m);
  // one wave of resident CTAs, each a whole number of thread rows
  const int smem = sq::norm_ring_bytes(p.threads, tensors == 1 ? sq::kNormU1 : sq::kNormU2, tensors) +
                   4 * sq::norm_smem_floats(p.threads, vx, vn, unit * m) + 1024;
  const int64_t resident =
      (int64_t)sms * std::min(p.threads != sq::kNormThreads ? 1 : tensors == 1 ? 3 : 2, kNormSmem / smem);
  int64_t tiles = std::max<int64_t>(1, resident / cols);
  int64_t rows = (S + tiles - 1) / tiles;
  rows = (rows + ty - 1) / ty * ty;
  tiles = (S + rows - 1) / rows;
  p.t = sq::NormTile{(int32_t)S, (int32_t)C, groups, cpg, unit * m, vx, ty, (int32_t)rows};
  p.tiles = (int)tiles;
  p.cs = 1;
  p.cluster = false;
  *out = p;
  return SQ_OK;
}

// The thread's last plan serves a call of the same sizes (the choice costs as much host
// time as an argument check of the whole call).
sq_status norm_plan(int64_t B, int64_t S, int64_t C, int32_t groups, int es, int tensors, NormPlan* out) {
  thread_local int64_t key[7] = {};
  thread_local NormPlan last;
  const int64_t k[7] = {B, S, C, groups, es, tensors, num_sms()};
  if (std::memcmp(k, key, sizeof(k)) != 0) {
    NormPlan p;
    const sq_status st = norm_plan_for(B, S, C, groups, es, tensors, &p);
    if (st != SQ_OK) return st;
    last = p;
    std::memcpy(key, k, sizeof(k));
  }
  *out = last;
  return SQ_OK;
}

sq_status norm_sizes(int64_t B, int64_t S, int64_t C, int32_t groups, sq_dtype xt) {
  if (!dtype_ok(xt) || B < 0 || S < 0 || C <= 0 || groups <= 0 || C % groups != 0) return SQ_ERR_INVALID_ARG;
  if (C % 8 != 0) return SQ_ERR_UNSUPPORTED;
  if (C > SQ_MAX_K || B > 65535 || S > (1 << 30)) return SQ_ERR_RANGE;
  return SQ_OK;
}

// A channels-last map: positions ld apart, images bs apart (read maps may repeat an image),
// 16-byte vectors.
sq_status norm_map(const void* p, int es, int64_t B, int64_t C, int64_t ld, int64_t bs, bool written) {
  if (p == nullptr || ld < C || (B > 1 && bs < (written ? C : 0))) return SQ_ERR_INVALID_ARG;
  if (!aligned16(p) || (ld * es) % 16 != 0 || (B > 1 && (bs * es) % 16 != 0)) return SQ_ERR_ALIGNMENT;
  return SQ_OK;
}

// Whether fp32 arrays (or null) lie on multiples of `bytes`.
template <typename... P>
bool aligned_f32(uintptr_t bytes, P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & (bytes - 1)) == 0;
}

template <auto KERN, typename... Args>
sq_status launch_grid(dim3 grid, int threads, int smem, int cluster, bool dependent, cudaStream_t stream,
                      Args... args) {
  if (smem > 48 * 1024) {
    cudaError_t e = smem_limit<KERN>(227 * 1024);
    if (e != cudaSuccess) return cuda_status(e);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (dependent) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cuda_status(cudaLaunchKernelEx(&cfg, KERN, args...));
}

template <typename XT, int NT>
sq_status norm_forward_two(const NormPlan& pl, int64_t B, const sq::NormArgs& a, cudaStream_t s) {
  const int ring = sq::norm_ring_bytes(NT, sq::kNormU1, 1);
  const int smem = ring + 4 * sq::norm_smem_floats(NT, pl.t.vx, sq::Vec<XT>::n, pl.t.nb);
  const dim3 grid((unsigned)pl.tiles, (unsigned)(pl.t.G / pl.t.nb), (unsigned)B);
  sq_status st = launch_grid<sq::group_norm_stats_kernel<XT, NT>>(grid, NT, smem, 1, true, s, a);
  if (st != SQ_OK) return st;
  return launch_grid<sq::group_norm_apply_kernel<XT, NT>>(grid, NT, ring + 8 * pl.t.nb, 1, true, s, a);
}

template <typename XT>
sq_status norm_forward(const NormPlan& pl, int64_t B, sq::NormArgs& a, cudaStream_t s) {
  a.t = pl.t;
  a.tiles = pl.tiles;
  if (!pl.cluster)
    return pl.threads == sq::kNormThreads ? norm_forward_two<XT, sq::kNormThreads>(pl, B, a, s)
                                          : norm_forward_two<XT, sq::kNormThreadsMax>(pl, B, a, s);
  const dim3 grid((unsigned)(pl.t.G / pl.t.nb * pl.cs), (unsigned)B);
  return launch_grid<sq::group_norm_cluster_kernel<XT>>(grid, sq::kNormThreads,
                                                        norm_cluster_smem(pl.t, pl.nv, sq::Vec<XT>::n, 1), pl.cs,
                                                        true, s, a, pl.cs, pl.nv);
}

template <typename XT, int NT>
sq_status norm_backward_two(const NormPlan& pl, int64_t B, const sq::NormBwdArgs& a, cudaStream_t s) {
  constexpr int vn = sq::Vec<XT>::n;
  const dim3 grid((unsigned)pl.tiles, (unsigned)(pl.t.G / pl.t.nb), (unsigned)B);
  const int ring = sq::norm_ring_bytes(NT, sq::kNormU2, 2);
  const int smem = ring + 4 * sq::norm_smem_floats(NT, pl.t.vx, vn, pl.t.nb);
  sq_status st = launch_grid<sq::group_norm_bwd_sums_kernel<XT, NT>>(grid, NT, smem, 1, true, s, a);
  if (st != SQ_OK) return st;
  st = launch_grid<sq::group_norm_bwd_totals_kernel>(dim3((unsigned)((a.t.C + 31) / 32), (unsigned)B),
                                                     32 * sq::kParamWarps, 0, 1, true, s, a);
  if (st != SQ_OK) return st;
  return launch_grid<sq::group_norm_bwd_apply_kernel<XT, NT>>(grid, NT, ring + 8 * (pl.t.vx * vn + pl.t.nb), 1, true, s,
                                                              a);
}

template <typename XT>
sq_status norm_backward(const NormPlan& pl, int64_t B, sq::NormBwdArgs& a, cudaStream_t s) {
  a.t = pl.t;
  a.tiles = pl.tiles;
  a.B = (int32_t)B;
  if (!pl.cluster)
    return pl.threads == sq::kNormThreads
               ? norm_backward_two<XT, sq::kNormThreads>(pl, B, a, s)
               : norm_backward_two<XT, sq::kNormThreadsMax>(pl, B, a, s);
  const dim3 grid((unsigned)(pl.t.G / pl.t.nb * pl.cs), (unsigned)B);
  const sq_status st = launch_grid<sq::group_norm_bwd_cluster_kernel<XT>>(
      grid, sq::kNormThreads, norm_cluster_smem(pl.t, pl.nv, sq::Vec<XT>::n, 2), pl.cs, true, s, a, pl.cs, pl.nv);
  if (st != SQ_OK || (a.dgamma == nullptr && a.dbeta == nullptr)) return st;
  return launch_grid<sq::group_norm_bwd_params_kernel>(dim3((unsigned)((a.t.C + 31) / 32)), 32 * sq::kParamWarps, 0, 1,
                                                       true, s, a);
}

// Bytes of a backward call's workspace: the images' sums, then the tiles' (none when
// an image is one tile).
size_t norm_bwd_bytes(const NormPlan& pl, int64_t B, int64_t C) {
  return sizeof(float) * 2 * (size_t)B * (size_t)C * (pl.cluster ? 1 : 1 + (size_t)pl.tiles);
}

sq_status group_norm_forward(const void* x, sq_dtype xt, int64_t B, int64_t S, int64_t C, int64_t ldx, int64_t xbs,
                             int32_t groups, const float* gamma, const float* beta, float eps, int act, void* y,
                             sq_dtype yt, int64_t ldy, int64_t ybs, const sq_segments* kseg, const float* s_pos,
                             const float* s_neg, int8_t* q_pos, int8_t* q_neg, int64_t ldq, float* stats, void* workspace,
                             size_t workspace_bytes, sq_stream_t stream) {
  sq_status st = norm_sizes(B, S, C, groups, xt);
  if (st != SQ_OK) return st;
  if (act < 0 || act > 2 || !(eps >= 0.0f)) return SQ_ERR_INVALID_ARG;
  sq::NormArgs a = {};
  if (q_pos != nullptr) {
    if (s_pos == nullptr || s_neg == nullptr || ldq < C) return SQ_ERR_INVALID_ARG;
    st = check_segments(kseg, C, SQ_MAX_SEGMENTS, 128, &a.kseg);
    if (st != SQ_OK) return st;
    if (C % 16 != 0) return SQ_ERR_UNSUPPORTED;
    if (!aligned16(q_pos) || !aligned16(q_neg) || ldq % 16 != 0) return SQ_ERR_ALIGNMENT;
  }
  if (y != nullptr && !dtype_ok(yt)) return SQ_ERR_INVALID_ARG;
  NormPlan pl;
  st = norm_plan(std::max<int64_t>(B, 1), std::max<int64_t>(S, 1), C, groups, elt_size(xt), 1, &pl);
  if (st != SQ_OK) return st;
  if (B == 0 || S == 0) return SQ_OK;
  if (!aligned_f32(4, gamma, beta, s_pos, s_neg, stats)) return SQ_ERR_ALIGNMENT;
  st = norm_map(x, elt_size(xt), B, C, ldx, xbs, false);
  if (st != SQ_OK) return st;
  if (y != nullptr) {
    st = norm_map(y, elt_size(yt), B, C, ldy, ybs, true);
    if (st != SQ_OK) return st;
  }
  if (!pl.cluster) {
    if (workspace == nullptr || workspace_bytes < sizeof(float2) * (size_t)B * pl.tiles * groups)
      return SQ_ERR_INVALID_ARG;
    if (!aligned16(workspace)) return SQ_ERR_ALIGNMENT;
  }
  a.x = x; a.ldx = ldx; a.xbs = B > 1 ? xbs : 0;
  a.y = y; a.ldy = ldy; a.ybs = B > 1 ? ybs : 0; a.y_bf16 = yt == SQ_BF16;
  a.q_pos = q_pos; a.q_neg = q_neg; a.ldq = ldq; a.s_pos = s_pos; a.s_neg = s_neg;
  a.gamma = gamma; a.beta = beta; a.eps = eps; a.act = act; a.stats = stats;
  a.part = static_cast<float2*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return xt == SQ_BF16 ? norm_forward<__nv_bfloat16>(pl, B, a, s) : norm_forward<float>(pl, B, a, s);
}

}  // namespace

extern "C" {

sq_status sq_group_norm_workspace_size(int64_t B, int64_t S, int64_t C, int32_t groups, sq_dtype xt,
                                       int32_t backward, size_t* bytes) {
  if (bytes == nullptr) return SQ_ERR_INVALID_ARG;
  *bytes = 0;
  sq_status st = norm_sizes(B, S, C, groups, xt);
  if (st != SQ_OK) return st;
  NormPlan pl;
  st = norm_plan(std::max<int64_t>(B, 1), std::max<int64_t>(S, 1), C, groups, elt_size(xt), backward ? 2 : 1, &pl);
  if (st != SQ_OK || B == 0 || S == 0) return st;
  if (backward) *bytes = norm_bwd_bytes(pl, B, C);
  else if (!pl.cluster) *bytes = sizeof(float2) * (size_t)B * pl.tiles * (size_t)groups;
  return SQ_OK;
}

sq_status sq_group_norm_act(const void* x, sq_dtype xt, int64_t B, int64_t S, int64_t C, int64_t ldx, int64_t xbs,
                            int32_t groups, const float* gamma, const float* beta, float eps, int32_t act, void* y,
                            sq_dtype yt, int64_t ldy, int64_t ybs, float* stats, void* workspace,
                            size_t workspace_bytes, sq_stream_t stream) {
  if (y == nullptr && B > 0 && S > 0) return SQ_ERR_INVALID_ARG;
  if (!dtype_ok(yt)) return SQ_ERR_INVALID_ARG;
  return group_norm_forward(x, xt, B, S, C, ldx, xbs, groups, gamma, beta, eps, act, y, yt, ldy, ybs, nullptr,
                            nullptr, nullptr, nullptr, nullptr, 0, stats, workspace, workspace_bytes, stream);
}

sq_status sq_quantize_activations_norm(const void* x, sq_dtype xt, int64_t B, int64_t S, int64_t C,
                                                int64_t ldx, int64_t xbs, int32_t groups, const float* gamma,
                                                const float* beta, float eps, int32_t act, const sq_segments* kseg,
                                                const float* s_pos, const float* s_neg, int8_t* q_pos, int8_t* q_neg,
                                                int64_t ldq,
                                                void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                                                sq_stream_t stream) {
  if (q_pos == nullptr || q_neg == nullptr) return SQ_ERR_INVALID_ARG;
  return group_norm_forward(x, xt, B, S, C, ldx, xbs, groups, gamma, beta, eps, act, y, SQ_BF16, ldy, S * ldy, kseg,
                            s_pos, s_neg, q_pos, q_neg, ldq, nullptr, workspace, workspace_bytes, stream);
}

sq_status sq_group_norm_act_backward(const void* dy, int64_t lddy, int64_t dybs, const void* x, sq_dtype xt,
                                     int64_t B, int64_t S, int64_t C, int64_t ldx, int64_t xbs, int32_t groups,
                                     const float* stats, const float* gamma, const float* beta, int32_t act,
                                     void* dx, int64_t lddx, int64_t dxbs, float* dgamma, float* dbeta,
                                     void* workspace, size_t workspace_bytes, sq_stream_t stream) {
  sq_status st = norm_sizes(B, S, C, groups, xt);
  if (st != SQ_OK) return st;
  if (act < 0 || act > 2) return SQ_ERR_INVALID_ARG;
  // the statistics are read in pairs
  if (!aligned_f32(8, stats) || !aligned_f32(4, gamma, beta, dgamma, dbeta)) return SQ_ERR_ALIGNMENT;
  NormPlan pl;
  const int es = elt_size(xt);
  st = norm_plan(std::max<int64_t>(B, 1), std::max<int64_t>(S, 1), C, groups, es, 2, &pl);
  if (st != SQ_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || S == 0) {   // sums over nothing
    if (dgamma != nullptr && (st = cuda_status(cudaMemsetAsync(dgamma, 0, sizeof(float) * (size_t)C, s))) != SQ_OK)
      return st;
    return dbeta == nullptr ? SQ_OK : cuda_status(cudaMemsetAsync(dbeta, 0, sizeof(float) * (size_t)C, s));
  }
  if (stats == nullptr) return SQ_ERR_INVALID_ARG;
  if ((st = norm_map(x, es, B, C, ldx, xbs, false)) != SQ_OK) return st;
  if ((st = norm_map(dy, es, B, C, lddy, dybs, false)) != SQ_OK) return st;
  if ((st = norm_map(dx, es, B, C, lddx, dxbs, true)) != SQ_OK) return st;
  if (workspace == nullptr || workspace_bytes < norm_bwd_bytes(pl, B, C))
    return SQ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return SQ_ERR_ALIGNMENT;
  sq::NormBwdArgs a = {};
  a.x = x; a.ldx = ldx; a.xbs = B > 1 ? xbs : 0;
  a.dy = dy; a.lddy = lddy; a.dybs = B > 1 ? dybs : 0;
  a.dx = dx; a.lddx = lddx; a.dxbs = B > 1 ? dxbs : 0;
  a.gamma = gamma; a.beta = beta; a.stats = stats; a.act = act;
  a.dgamma = dgamma; a.dbeta = dbeta;
  a.total = static_cast<float*>(workspace);
  a.part = a.total + 2 * (size_t)B * (size_t)C;
  return xt == SQ_BF16 ? norm_backward<__nv_bfloat16>(pl, B, a, s)
                       : norm_backward<float>(pl, B, a, s);
}

}  // extern "C"
