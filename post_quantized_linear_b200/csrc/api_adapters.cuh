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
  if (ad->K > SQ_MAX_K || ad->N > SQ_MAX_K || M > (1 << 30) || requests > (1 << 24) || ad->L > 65535)
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

template <int T, typename XT, bool BWD>
sq_status launch_few_rows_x(const sq::AdapterArgs& a, sq_dtype yt, cudaStream_t s) {
  const int64_t slots = sq::adapter_slots(a.M, a.Q, T);
  const int D = BWD ? a.N : a.K;
  // as many CTAs per piece as the SMs hold at once, each with a warp's load of the long axis
  const int64_t room = (int64_t)num_sms() * (T == 1 ? 4 : 2);
  int cs = 1;
  while (cs < 8 && slots * cs * 2 <= room && D >= 256 * cs) cs *= 2;
  const dim3 grid((unsigned)(slots * cs));
  using bf16 = __nv_bfloat16;
  constexpr int n = sq::kFewThreads;
  if constexpr (!BWD)
    if (a.out != nullptr)
      return launch_grid<sq::adapter_few_rows_kernel<T, XT, float, bf16, false>>(grid, n, 0, cs, true, s, a, cs);
  return yt == SQ_BF16 ? launch_grid<sq::adapter_few_rows_kernel<T, XT, bf16, bf16, BWD>>(grid, n, 0, cs, true, s, a, cs)
                       : launch_grid<sq::adapter_few_rows_kernel<T, XT, float, float, BWD>>(grid, n, 0, cs, true, s, a, cs);
}
template <int T, bool BWD>
sq_status launch_few_rows_t(const sq::AdapterArgs& a, sq_dtype xt, sq_dtype yt, cudaStream_t s) {
  return xt == SQ_BF16 ? launch_few_rows_x<T, __nv_bfloat16, BWD>(a, yt, s) : launch_few_rows_x<T, float, BWD>(a, yt, s);
}

// Pieces of one row where requests have up to two on average, of eight elsewhere: 64
// requests of one, two, four, eight rows, 2304 -> 2304, rank 32, take 10.7, 13.0, 18.2, 29.4 us
// in pieces of one and 16.7, 17.4, 18.9, 22.0 us in pieces of eight, which read an
// adapter once for eight rows.
template <bool BWD>
sq_status launch_few_rows(const sq::AdapterArgs& a, sq_dtype xt, sq_dtype yt, cudaStream_t s) {
  return a.M <= 2 * (int64_t)a.Q ? launch_few_rows_t<1, BWD>(a, xt, yt, s)
                    : launch_few_rows_t<sq::kFewRows, BWD>(a, xt, yt, s);
}

constexpr int kGradCtas = 3;      // of adapter_grad_kernel on an SM, by its registers

sq_status launch_adapter_grad(sq::AdapterGradArgs& g, sq_dtype xt, sq_dtype dyt, cudaStream_t s) {
  g.tiles0 = (g.C[0] + sq::kGradCols - 1) / sq::kGradCols;
  const int tiles = g.tiles0 + (g.C[1] + sq::kGradCols - 1) / sq::kGradCols;
  // The cluster shares an adapter's pieces: the number of CTAs that takes the least time,
  // all of them over the resident ones and the last one behind them, each about two
  // pieces' time to begin and end (8000 rows of ten uneven requests, 2304 -> 2304, rank 64: 406 us
  // where one CTA has an adapter's pieces 500).
  const int used = std::max(1, std::min(g.L, g.Q));
  const int64_t per = std::max<int64_t>(1, (int64_t)g.M / sq::kGradPiece / used);
  const double over = (double)tiles * used / (num_sms() * kGradCtas);
  int cs = 1;
  double least = 1e30;
  for (int k = 1; k <= 8 && k <= per; ++k) {
    const double t = (std::max(1.0, over * k) + 1.0) * (2.0 + (double)per / k);
    if (t < least) { least = t; cs = k; }
  }
  g.cs = cs;
  const dim3 grid((unsigned)(tiles * cs), (unsigned)g.L);
  using bf16 = __nv_bfloat16;
  constexpr int n = sq::kGradThreads;
  if (xt == SQ_BF16)
    return dyt == SQ_BF16 ? launch_grid<sq::adapter_grad_kernel<bf16, bf16>>(grid, n, 0, cs, true, s, g)
                          : launch_grid<sq::adapter_grad_kernel<bf16, float>>(grid, n, 0, cs, true, s, g);
  return dyt == SQ_BF16 ? launch_grid<sq::adapter_grad_kernel<float, bf16>>(grid, n, 0, cs, true, s, g)
                        : launch_grid<sq::adapter_grad_kernel<float, float>>(grid, n, 0, cs, true, s, g);
}

// A tiled map of rank 2 or 3, boxes with 128-byte swizzled rows; strides in bytes
// for dimensions 1, 2.
sq_status make_adapter_map(CUtensorMap* map, sq_dtype t, const void* base, int rank, uint64_t d0, uint64_t d1,
                           uint64_t d2, uint64_t s1, uint64_t s2, uint32_t b0, uint32_t b1) {
  auto fn = encode_fn();
  if (fn == nullptr) return SQ_ERR_CUDA;
  cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1, s2};
  cuuint32_t box[3] = {b0, b1, 1}, estr[3] = {1, 1, 1};
  CUresult r = fn(map, t == SQ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                  (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? SQ_OK : SQ_ERR_CUDA;
}

constexpr int kSmemPerSm = 227 * 1024;

// How many clusters of cs CTAs of a kernel the device holds at once with one CTA on an
// SM (which is what the query counts for clusters), asked once per device and size of
// shared memory (per kernel, the last one asked for).
template <auto KERN>
int resident_clusters(int cs, int threads, int smem) {
  static std::atomic<uint64_t> known[kMaxDevices][9] = {};   // smem << 32 | clusters + 1
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices || cs > 8) return 0;
  const uint64_t v = known[dev][cs].load(std::memory_order_relaxed);
  if (v != 0 && (int)(v >> 32) == smem) return (int)(v & 0xFFFFFFFFu) - 1;
  if (smem_limit<KERN>(kSmemPerSm) != cudaSuccess) return 0;
  // the answer, and what the device really holds, go by the kernel's carve-out
  if (cudaFuncSetAttribute(KERN, cudaFuncAttributePreferredSharedMemoryCarveout, 100) != cudaSuccess)
    (void)cudaGetLastError();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(cs * 1024));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, KERN, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    n = num_sms() / cs;
  }
  known[dev][cs].store((uint64_t)smem << 32 | (uint64_t)(n + 1), std::memory_order_relaxed);
  return n;
}

template <int RB, typename YT, typename OT, bool BWD>
sq_status launch_tile_rb(sq::AdapterTileArgs t, const CUtensorMap& tx, const CUtensorMap& tw1,
                         const CUtensorMap& tw2, const CUtensorMap& ty, cudaStream_t s) {
  constexpr auto kern = sq::adapter_tile_kernel<RB, YT, OT, BWD>;
  const sq::AdapterArgs& a = t.p;
  const int D = BWD ? a.N : a.K, E = BWD ? a.K : a.N;
  const int rp = (a.R + 15) / 16 * 16;
  t.parts = sizeof(OT) == 2 ? 2 : 3;
  t.wide = reinterpret_cast<uintptr_t>(a.out != nullptr ? a.out : a.y) % 32 == 0 &&
           (a.out != nullptr ? a.ldo : a.ldy) * (int64_t)sizeof(OT) % 32 == 0;
  t.slot_bytes = sq::kTileX + (RB == 64 ? 8192 : 16384);
  t.wait_budget = g_wait_budget;
  t.starve = g_debug_starve;
  const int rest = sq::adapter_h_bytes(rp, t.parts) + sq::kTileBars + 1024;
  // Pieces expected: the batch cut into 128 rows, or one per request.  The largest
  // cluster whose pieces are all resident at once: a second wave of a few clusters
  // costs a whole pass.  Two CTAs on an SM overlap one another's steps; where that would
  // make clusters of more than four, one CTA with a deep ring and a smaller exchange is
  // faster (32 pieces of 4608 -> 4608, rank 64: 39.1 us, not 45.1; all gradients of 64 pieces,
  // 8192 x 1152 -> 4608: 95.4 us, not 91.2, so not below that).
  const int64_t pieces = std::max<int64_t>((a.M + sq::kTileRows - 1) / sq::kTileRows, std::min<int64_t>(a.Q, a.M));
  const int most = std::max(1, std::min({8, (D + 63) / 64, (E + 128 / (int)sizeof(YT) - 1) / (128 / (int)sizeof(YT))}));
  auto choose = [&](bool two, int* stages) {
    const int room = two ? kSmemPerSm / 2 - 1024 : kSmemPerSm;
    *stages = std::min(sq::kTileStages, (room - rest) / t.slot_bytes);
    const int smem = *stages * t.slot_bytes + rest;
    int cs = most;
    while (cs > 1 && pieces > (two ? 2 : 1) * resident_clusters<kern>(cs, sq::kTileThreads, smem)) --cs;
    return cs;
  };
  bool two = RB == 64 && 3 * t.slot_bytes + rest <= kSmemPerSm / 2 - 1024;
  int cs = choose(two, &t.stages);
  if (two && cs > 4) cs = choose(two = false, &t.stages);
  const int smem = t.stages * t.slot_bytes + rest;
  t.cs = cs;
  cudaError_t e = smem_limit<kern>(kSmemPerSm);
  if (e != cudaSuccess) return cuda_status(e);
  const int64_t slots = sq::adapter_slots(a.M, a.Q, sq::kTileRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(slots * cs));
  cfg.blockDim = dim3(sq::kTileThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, tx, tw1, tw2, ty, t));
}

template <bool BWD>
sq_status launch_tile(const sq::AdapterTileArgs& t, sq_dtype yt, cudaStream_t s) {
  const sq::AdapterArgs& a = t.p;
  const uint64_t K = a.K, N = a.N, R = a.R, L = a.L, M = a.M;
  const uint32_t rp = (uint32_t)((R + 15) / 16 * 16), bn = yt == SQ_BF16 ? 64 : 32;
  CUtensorMap tx, tw1, tw2, ty;
  sq_status st = make_adapter_map(&tx, SQ_BF16, a.x, 2, BWD ? N : K, M, 1, a.ldx * 2, 0, 64, 32);
  if (st != SQ_OK) return st;
  if (BWD) {
    if ((st = make_adapter_map(&tw1, SQ_BF16, a.b, 3, R, N, L, R * 2, N * R * 2, 64, 64)) != SQ_OK) return st;
    if ((st = make_adapter_map(&tw2, SQ_BF16, a.a, 3, K, R, L, K * 2, K * R * 2, 64, rp)) != SQ_OK) return st;
    if ((st = make_adapter_map(&ty, yt, a.y, 2, K, M, 1, a.ldy * elt_size(yt), 0, bn, 32)) != SQ_OK) return st;
  } else {
    if ((st = make_adapter_map(&tw1, SQ_BF16, a.a, 3, K, R, L, K * 2, K * R * 2, 64, (uint32_t)R)) != SQ_OK) return st;
    if ((st = make_adapter_map(&tw2, SQ_BF16, a.b, 3, R, N, L, R * 2, N * R * 2, 64, bn)) != SQ_OK) return st;
    if ((st = make_adapter_map(&ty, yt, a.y, 2, N, M, 1, a.ldy * elt_size(yt), 0, bn, 32)) != SQ_OK) return st;
  }
  using bf16 = __nv_bfloat16;
  if constexpr (BWD) {
    return R <= 64 ? launch_tile_rb<64, bf16, bf16, true>(t, tx, tw1, tw2, ty, s)
                   : launch_tile_rb<128, bf16, bf16, true>(t, tx, tw1, tw2, ty, s);
  } else {
    if (a.out != nullptr)
      return R <= 64 ? launch_tile_rb<64, float, bf16, false>(t, tx, tw1, tw2, ty, s)
                     : launch_tile_rb<128, float, bf16, false>(t, tx, tw1, tw2, ty, s);
    if (R <= 64)
      return yt == SQ_BF16 ? launch_tile_rb<64, bf16, bf16, false>(t, tx, tw1, tw2, ty, s)
                           : launch_tile_rb<64, float, float, false>(t, tx, tw1, tw2, ty, s);
    return yt == SQ_BF16 ? launch_tile_rb<128, bf16, bf16, false>(t, tx, tw1, tw2, ty, s)
                         : launch_tile_rb<128, float, float, false>(t, tx, tw1, tw2, ty, s);
  }
}

// The first product in bf16 tiles of 128 rows pays where requests have rows to fill
// them; with a few rows each, and for fp32 rows, the few-rows form is taken (64 requests of
// 4, 8, 16, 32 rows, 2304 -> 2304, rank 32: 23.5, 23.9, 23.9, 24.4 us in tiles, 19.0, 22.0, 35.6,
// 53.9 us in few rows; all gradients 52, 50, 50, 48 us and 32, 37, 55, 88 us).
bool use_tiles(const sq::AdapterArgs& a, sq_dtype xt) {
  return xt == SQ_BF16 && (int64_t)a.M > (int64_t)sq::kFewRows * std::max(a.Q, 1);
}

template <int RB>
sq_status launch_grad_tile_rb(sq::AdapterGradTileArgs g, const CUtensorMap (&t)[4], int tiles, cudaStream_t s) {
  constexpr auto kern = sq::adapter_grad_tile_kernel<RB>;
  const int rp = (g.R + 15) / 16 * 16;
  const int slot = sq::kTileX + sq::adapter_grad_atoms(rp) * 8192;
  constexpr int on_sm = sq::adapter_grad_ctas(RB);
  const int room = kSmemPerSm / on_sm - 1024 - sq::kTileBars - 1024;
  g.stages = std::min(4, room / slot);
  // The cluster shares an adapter's pieces: the number of CTAs that takes the least time by
  // waves of resident CTAs, each about ten pieces' time to begin and end.
  const int64_t per = std::max<int64_t>(1, (int64_t)g.M / sq::kGradPiece / std::max(1, std::min(g.L, g.Q)));
  const int64_t ctas = (int64_t)tiles * std::max(1, std::min(g.L, g.Q));
  const int64_t resident = (int64_t)num_sms() * on_sm;
  int cs = 1;
  int64_t least = INT64_MAX;
  for (int k = 1; k <= 8 && k <= per; ++k) {
    const int64_t t = (ctas * k + resident - 1) / resident * (10 + (per + k - 1) / k);
    if (t < least) { least = t; cs = k; }
  }
  g.cs = cs;
  // At least the share of shared memory that the CTA has of TMEM (a quarter, half, or
  // all): a CTA that is resident never waits for TMEM of another cluster's.
  const int smem = std::max(std::max(g.stages * slot, cs > 1 ? 128 * rp * 4 : 0) + sq::kTileBars + 1024,
                            kSmemPerSm / (RB == 32 ? 4 : on_sm) - 4096);
  cudaError_t e = smem_limit<kern>(kSmemPerSm);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * cs), (unsigned)g.L);
  cfg.blockDim = dim3(sq::kTileThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, t[0], t[1], t[2], t[3], g));
}

// Both gradients on the tensor cores, from the parts of u and h that launch_tile<true> wrote.
sq_status launch_grad_tiles(const sq::AdapterTileArgs& t, const void* x, int64_t ldx, const void* dy, int64_t lddy,
                            float* da, float* db, cudaStream_t s) {
  const sq::AdapterArgs& a = t.p;
  const uint64_t cols = 3 * (uint64_t)((a.R + 15) / 16 * 16);
  CUtensorMap maps[4];
  sq_status st;
  if ((st = make_adapter_map(&maps[0], SQ_BF16, x, 2, a.K, a.M, 1, ldx * 2, 0, 64, sq::kGradPiece)) != SQ_OK) return st;
  if ((st = make_adapter_map(&maps[1], SQ_BF16, dy, 2, a.N, a.M, 1, lddy * 2, 0, 64, sq::kGradPiece)) != SQ_OK) return st;
  if ((st = make_adapter_map(&maps[2], SQ_BF16, t.f_u, 2, cols, a.M, 1, cols * 2, 0, 64, sq::kGradPiece)) != SQ_OK) return st;
  if ((st = make_adapter_map(&maps[3], SQ_BF16, t.f_h, 2, cols, a.M, 1, cols * 2, 0, 64, sq::kGradPiece)) != SQ_OK) return st;
  sq::AdapterGradTileArgs g = {};
  g.out[0] = da; g.out[1] = db;
  g.scale = a.scale; g.bounds = a.bounds; g.index = a.index;
  g.C[0] = a.K; g.C[1] = a.N;
  g.tiles0 = (a.K + 127) / 128;
  g.M = a.M; g.R = a.R; g.L = a.L; g.Q = a.Q;
  g.wait_budget = g_wait_budget;
  g.starve = g_debug_starve;
  const int tiles = g.tiles0 + (a.N + 127) / 128;
  return a.R <= 32   ? launch_grad_tile_rb<32>(g, maps, tiles, s)
         : a.R <= 64 ? launch_grad_tile_rb<64>(g, maps, tiles, s)
                     : launch_grad_tile_rb<128>(g, maps, tiles, s);
}

// Bytes of a backward call's workspace: u in fp32, or u and h as three bf16 parts.
size_t adapter_bwd_bytes(int64_t M, int32_t R) {
  return (size_t)M * (size_t)((R + 15) / 16 * 16) * 3 * sizeof(__nv_bfloat16) * 2;
}

// y += the term, or out = y + the term where out is given (y fp32, out bf16).
sq_status adapter_forward(const void* x, sq_dtype xt, int64_t M, int64_t ldx, const sq_adapters* adapters,
                          const int32_t* bounds, const int32_t* index, int32_t requests, void* y, sq_dtype yt,
                          int64_t ldy, void* out, int64_t ldo, float* hidden, sq_stream_t stream) {
  sq_status st = check_adapters(adapters, bounds, index, requests, M);
  if (st != SQ_OK) return st;
  if (!dtype_ok(xt) || !dtype_ok(yt)) return SQ_ERR_INVALID_ARG;
  if (M == 0 || (requests == 0 && hidden == nullptr && out == nullptr)) return SQ_OK;
  if ((st = check_matrix(x, xt, adapters->K, ldx)) != SQ_OK) return st;
  if ((st = check_matrix(y, yt, adapters->N, ldy)) != SQ_OK) return st;
  if (out != nullptr && (st = check_matrix(out, SQ_BF16, adapters->N, ldo)) != SQ_OK) return st;
  if (hidden != nullptr && !aligned16(hidden)) return SQ_ERR_ALIGNMENT;
  sq::AdapterArgs a = adapter_args(adapters, bounds, index, requests, M);
  a.x = x; a.ldx = ldx; a.y = y; a.ldy = ldy; a.out = out; a.ldo = ldo; a.h = hidden;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!use_tiles(a, xt)) return launch_few_rows<false>(a, xt, yt, s);
  sq::AdapterTileArgs t = {};
  t.p = a;
  return launch_tile<false>(t, yt, s);
}

}  // namespace

extern "C" {

sq_status sq_adapter_add(const void* x, sq_dtype xt, int64_t M, int64_t ldx, const sq_adapters* adapters,
                         const int32_t* bounds, const int32_t* index, int32_t requests, void* y, sq_dtype yt,
                         int64_t ldy, float* hidden, sq_stream_t stream) {
  return adapter_forward(x, xt, M, ldx, adapters, bounds, index, requests, y, yt, ldy, nullptr, 0, hidden, stream);
}

sq_status sq_adapter_add_to(const void* x, sq_dtype xt, int64_t M, int64_t ldx, const sq_adapters* adapters,
                            const int32_t* bounds, const int32_t* index, int32_t requests, const float* y,
                            int64_t ldy, void* out, int64_t ldo, float* hidden, sq_stream_t stream) {
  if (out == nullptr && M > 0) return SQ_ERR_INVALID_ARG;
  return adapter_forward(x, xt, M, ldx, adapters, bounds, index, requests, const_cast<float*>(y), SQ_F32, ldy, out,
                         ldo, hidden, stream);
}

sq_status sq_adapter_backward_workspace_size(int64_t M, int32_t R, size_t* bytes) {
  if (bytes == nullptr || M < 0 || R <= 0) return SQ_ERR_INVALID_ARG;
  *bytes = adapter_bwd_bytes(M, R);
  return SQ_OK;
}

sq_status sq_adapter_backward(const void* dy, sq_dtype dyt, int64_t M, int64_t lddy, const void* x, sq_dtype xt,
                              int64_t ldx, const float* hidden, const sq_adapters* adapters, const int32_t* bounds,
                              const int32_t* index, int32_t requests, void* dx, int64_t lddx, float* da, float* db,
                              void* workspace, size_t workspace_bytes, sq_stream_t stream) {
  sq_status st = check_adapters(adapters, bounds, index, requests, M);
  if (st != SQ_OK) return st;
  if (!dtype_ok(xt) || !dtype_ok(dyt) || da == nullptr || db == nullptr) return SQ_ERR_INVALID_ARG;
  // Each CTA of the gradients walks all requests, 32 at a time, about 0.5 us each, for its
  // adapter (2^20 requests of 8 adapters, 4096 rows of 128 columns: 18 ms; 2^16 requests of one row, 1152 ->
  // 1152: 13 ms).  Beyond these numbers a call could hold the GPU for minutes.
  if (requests > (1 << 20) || (int64_t)requests * adapters->L > (1 << 26)) return SQ_ERR_RANGE;
  if (!aligned16(da) || !aligned16(db)) return SQ_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  sq::AdapterArgs a = adapter_args(adapters, bounds, index, requests, M);
  if (M > 0) {
    if ((st = check_matrix(dy, dyt, adapters->N, lddy)) != SQ_OK) return st;
    if ((st = check_matrix(x, xt, adapters->K, ldx)) != SQ_OK) return st;
    if ((st = check_matrix(dx, xt, adapters->K, lddx)) != SQ_OK) return st;
    if (hidden == nullptr || workspace == nullptr || workspace_bytes < adapter_bwd_bytes(M, adapters->R))
      return SQ_ERR_INVALID_ARG;
    if (!aligned16(hidden) || !aligned16(workspace)) return SQ_ERR_ALIGNMENT;
    a.x = dy; a.ldx = lddy; a.y = dx; a.ldy = lddx;
    if (use_tiles(a, dyt) && xt == SQ_BF16) {
      sq::AdapterTileArgs t = {};
      t.p = a;
      t.hidden = hidden;
      t.f_u = static_cast<__nv_bfloat16*>(workspace);
      t.f_h = t.f_u + (size_t)M * (size_t)((a.R + 15) / 16 * 16) * 3;
      if ((st = launch_tile<true>(t, xt, s)) != SQ_OK) return st;
      return launch_grad_tiles(t, x, ldx, dy, lddy, da, db, s);
    }
    a.h = static_cast<float*>(workspace);
    if ((st = launch_few_rows<true>(a, dyt, xt, s)) != SQ_OK) return st;
  }
  sq::AdapterGradArgs g = {};
  g.bounds = bounds; g.index = index; g.M = (int32_t)M; g.R = adapters->R; g.L = adapters->L;
  g.Q = M > 0 ? requests : 0;
  g.f[0] = static_cast<const float*>(workspace); g.g[0] = x; g.ldg[0] = ldx; g.C[0] = (int32_t)adapters->K; g.out[0] = da;
  g.f[1] = hidden; g.g[1] = dy; g.ldg[1] = lddy; g.C[1] = (int32_t)adapters->N; g.out[1] = db;
  g.scale = adapters->scale;
  return launch_adapter_grad(g, xt, dyt, s);
}

}  // extern "C"
