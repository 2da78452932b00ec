// Low-rank adapters of many requests beside a shared projection.
//
// Rows bounds[q] .. bounds[q+1] of the batch belong to request q, which uses
// adapter l = index[q] (A_l [R, K], B_l [N, R] in bf16, scale_l; -1: none):
//   forward   h = x A_l^T,   y += scale_l h B_l^T
//   backward  u = scale_l dy B_l,  dx = u A_l,  dA_l = sum u^T x,
//             dB_l = scale_l sum dy^T h, over all rows of all requests that use l
// Bounds and indices stay on the device: a captured call replays with new ones.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "common.cuh"
#include "group_norm.cuh"
#include "ptx.cuh"
#include "quant_kernels.cuh"

namespace sq {

constexpr int kAdapterMaxRank = 128;

struct AdapterArgs {
  const void* x;                 // forward: x [M, K]; backward: dy [M, N]
  int64_t ldx;
  void* y;                       // forward: y [M, N], added to; backward: dx [M, K], written
  int64_t ldy;
  void* out;                     // forward into an output of its own: bf16 [M, N] = y + the term, else null
  int64_t ldo;
  const __nv_bfloat16* a;        // [L, R, K]
  const __nv_bfloat16* b;        // [L, N, R]
  const float* scale;            // [L]
  const int32_t* bounds;         // [Q + 1]
  const int32_t* index;          // [Q]
  float* h;                      // forward: h [M, R] or null; backward: u [M, R]
  int32_t M, K, N, L, R, Q;
};

// A piece of one request: rows row .. row + n of the batch, adapter l (-1: none).
struct AdapterItem {
  int32_t row, n, l;
};

// Item `slot` when requests are cut into pieces of T rows.  The rows before the
// first request and behind the last count as two more requests, without an
// adapter.  Up to kExactRequests: a warp counts the pieces of all of them and sums the
// counts, so the items come without gaps.  More: request r's pieces begin at slot
// floor(start_r / T) + r, which leaves room for a request of any length before the
// next one's, so its own bounds alone place them and a 32-way search finds the
// request of a slot.  adapter_slots() slots hold every piece in both.
// The bounds are cut to the batch, so no read or write leaves the tensors.  A request that
// request_counts() leaves out keeps its rows in the batch, without an adapter;
// check_requests raises the range status for it.
constexpr int kLaneRequests = 8, kExactRequests = 32 * kLaneRequests - 2;
__host__ __device__ inline int64_t adapter_slots(int M, int Q, int T) {
  // pieces: every T rows of the batch end at most one, and so does every request's end
  return T == 1 && Q <= kExactRequests ? M : (int64_t)M / T + Q + 3;
}
// Whether a request with the bounds s, e and the adapter l counts: not with bounds outside
// the batch or an unknown adapter.  The kernels of a call have to agree on it: what the
// gradients' kernel sums over a request's rows, the one before it has written.
__device__ __forceinline__ bool request_counts(int s, int e, int l, int M, int L) {
  return s >= 0 && e <= M && l < L;
}
__device__ __forceinline__ AdapterItem adapter_item(const AdapterArgs& p, int slot, int T) {
  const int lane = threadIdx.x & 31;
  const int count = p.Q + 2;
  auto start = [&](int r) {
    return r == 0 ? 0 : r <= p.Q + 1 ? min(max(__ldg(p.bounds + r - 1), 0), p.M) : p.M;
  };
  AdapterItem it;
  it.row = it.n = 0;
  it.l = -1;
  int lo, piece;
  if (count <= 32 * kLaneRequests) {
    // a lane: `per` requests side by side
    const int per = (count + 31) >> 5, r0 = lane * per;
    int n[kLaneRequests], sum = 0;
    int from = r0 < count ? start(r0) : p.M;
#pragma unroll
    for (int i = 0; i < kLaneRequests; ++i) {
      n[i] = 0;
      if (i < per && r0 + i < count) {
        const int to = start(r0 + i + 1);
        n[i] = max(0, to - from + T - 1) / T;
        from = to;
      }
      sum += n[i];
    }
    const int own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned m = __ballot_sync(0xffffffffu, sum > slot);
    if (m == 0) return it;
    int left = slot - (sum - own), k = 0;       // within this lane's requests
#pragma unroll
    for (int i = 0; i < kLaneRequests - 1; ++i)
      if (k == i && left >= n[i]) { left -= n[i]; k = i + 1; }
    const int src = __ffs(m) - 1;
    lo = __shfl_sync(0xffffffffu, r0 + k, src);
    piece = __shfl_sync(0xffffffffu, left, src);
  } else {
    lo = 0;
    int span = count;
    while (span > 1) {
      const int step = (span + 31) >> 5;
      const int r = lo + lane * step;
      const bool le = lane * step < span && start(r) / T + r <= slot;
      const unsigned m = __ballot_sync(0xffffffffu, le) | 1u;
      const int k = 31 - __clz(m);
      span = min(step, span - k * step);
      lo += k * step;
    }
    piece = slot - (start(lo) / T + lo);
  }
  if (lo >= count) return it;
  const bool request = lo > 0 && lo <= p.Q;
  const int from = lo > 0 ? __ldg(p.bounds + lo - 1) : 0, to = lo <= p.Q ? __ldg(p.bounds + lo) : p.M;
  const int l = request ? __ldg(p.index + lo - 1) : -1;
  const int s = min(max(from, 0), p.M), e = min(max(to, 0), p.M);
  // (of falling bounds the search may bring any piece)
  if (e < s || piece < 0 || piece > (e - s) / T) return it;
  if (request && request_counts(from, to, l, p.M, p.L)) it.l = l;
  it.row = s + piece * T;
  it.n = min(T, e - it.row);
  return it;
}

// Raises the range status for bounds outside the batch, falling bounds (which
// hide other requests from the search, too) and unknown adapters.  One CTA of a
// launch calls it, with all its threads.
__device__ __forceinline__ void check_requests(const AdapterArgs& p, int threads) {
  bool bad = threadIdx.x == 0 && (__ldg(p.bounds) < 0 || __ldg(p.bounds + p.Q) > p.M);
  for (int q = threadIdx.x; q < p.Q; q += threads)
    bad |= __ldg(p.bounds + q) > __ldg(p.bounds + q + 1) || __ldg(p.index + q) >= p.L;
  if (bad) raise_status(SQ_STATUS_RANGE);
}

// ------------------------------------------------------- few rows, fp32 rows
// One cluster of CTAs per piece of one or eight rows: each CTA contracts its
// slice of the long axis on the fp32 lanes, the partial h (or u) are added
// through distributed shared memory in rank order, and each CTA then writes its
// slice of the columns.  This is the form for batches of requests of a few rows
// (one conditioning vector each), which are bound by launch and load latency
// and by the adapters' bytes, and for fp32 rows, bound by the fp32 lanes when there are many.
// 64 requests of one row, 1152 -> 3456, rank 16: 9.0 us; 777 fp32 rows, 1152 -> 2304, rank 8:
// 14.8 us.
constexpr int kFewRows = 8;
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewChunk = 1016;  // elements of the long axis staged at a time

template <typename T>
__device__ __forceinline__ float ld_elem(const T* p) { return to_f32(*p); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// Eight consecutive elements widened to fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
  if constexpr (Vec<T>::n == 8) {
    Vec<T>::load(p, v);
  } else {
    float a[4], b[4];
    Vec<T>::load(p, a);
    Vec<T>::load(p + 4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  }
}
// Vectors from, from + step, .. below `to` of eight elements, fp32 -> bf16, of a row without an adapter.
template <typename YT, typename OT>
__device__ __forceinline__ void copy_row(const YT* y, OT* out, int from, int to, int step) {
  for (int i = from; i < to; i += step) {
    float v[8];
    load8(y + i * 8, v);
    store_vec<8>(out, (int64_t)i * 8, sizeof(OT) == 2, v);
  }
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Slice k of n elements cut into cs slices of whole 8-element vectors.
__device__ __forceinline__ void long_slice(int n, int cs, int k, int& from, int& to) {
  const int per = ((n + 8 * cs - 1) / (8 * cs)) * 8;
  from = min(n, k * per);
  to = min(n, from + per);
}

// Sums over the threads that share a vector of 8 ranks, M rows at a time: thread
// tid holds v[m][] for ranks 8 * (tid % rv) .., out[r * pitch + m] receives the totals.
// red: kFewThreads * 8 * M floats.
template <int M>
__device__ __forceinline__ void reduce_rank_vectors(const float (&v)[M][8], bool active, int rv, float* red, float* out,
                                                    int pitch) {
  const int tid = threadIdx.x, outs = 8 * M * rv, lanes = kFewThreads / rv;
  __syncthreads();
  if (active) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      *reinterpret_cast<float4*>(red + (tid * M + m) * 8) = make_float4(v[m][0], v[m][1], v[m][2], v[m][3]);
      *reinterpret_cast<float4*>(red + (tid * M + m) * 8 + 4) = make_float4(v[m][4], v[m][5], v[m][6], v[m][7]);
    }
  }
  __syncthreads();
  // a total o = ((rank vector * M) + m) * 8 + i; `ways` threads share it, then one adds theirs
  const int ways = max(1, min(lanes, kFewThreads / outs));
  auto put = [&](int o, float t) { out[((o / (8 * M)) * 8 + o % 8) * pitch + o / 8 % M] = t; };
  if (ways == 1) {
    for (int o = tid; o < outs; o += kFewThreads) {
      float t = 0.0f;
#pragma unroll 4
      for (int j = 0; j < lanes; ++j) t += red[j * outs + o];
      put(o, t);
    }
    return;
  }
  const int o = tid % outs, wy = tid / outs;
  float t = 0.0f;
  if (wy < ways) {
#pragma unroll 4
    for (int j = wy; j < lanes; j += ways) t += red[j * outs + o];
  }
  __syncthreads();
  if (wy < ways) red[wy * outs + o] = t;
  __syncthreads();
  if (tid < outs) {
    float a = 0.0f;
    for (int j = 0; j < ways; ++j) a += red[j * outs + tid];
    put(tid, a);
  }
}

// T rows (1 or 8).  BWD = false: x A^T, then y += scale h B^T (OT other than YT: out = y + ..,
// rounded once).  BWD = true: scale dy B, then dx = u A.
template <int T, typename XT, typename YT, typename OT, bool BWD>
__global__ void __launch_bounds__(kFewThreads, T == 1 ? 4 : 2)
    adapter_few_rows_kernel(const AdapterArgs p, int cs) {
  constexpr bool APART = !std::is_same<YT, OT>::value;
  constexpr int XP = kFewChunk + 4;                                   // row pitch: shifts the banks
  constexpr int MR = T == 1 ? 1 : 4;                                  // rows reduced at a time
  // rows [row][k] while they are contracted, then the threads' sums
  __shared__ __align__(16) float xs[kFewThreads * 8 * MR];
  static_assert(T == 1 || T * XP <= kFewThreads * 8 * MR, "");
  __shared__ __align__(16) float part[T * kAdapterMaxRank];           // [r][row], this CTA's share
  __shared__ __align__(16) float full[T * kAdapterMaxRank];           // [r][row], times scale
  __shared__ __align__(16) float red[BWD ? 4 : T * kAdapterMaxRank];  // forward: the warps' sums
  const int rank = blockIdx.x % cs;
  const int tid = threadIdx.x;
  grid_dep_wait();
  if (blockIdx.x == 0) check_requests(p, kFewThreads);
  const AdapterItem it = adapter_item(p, blockIdx.x / cs, T);
  const int D = BWD ? p.N : p.K, E = BWD ? p.K : p.N, R = p.R;   // contracted, written
  int e0, e1;
  long_slice(E, cs, rank, e0, e1);
  if (it.n == 0 || it.l < 0) {       // the same for every CTA of the cluster
    if (BWD) {
      YT* y = static_cast<YT*>(p.y);
      for (int m = 0; m < it.n; ++m)
        for (int c = e0 + tid; c < e1; c += kFewThreads) st_elem(y + (int64_t)(it.row + m) * p.ldy + c, 0.0f);
      return;
    }
    if (p.h != nullptr && rank == 0)
      for (int i = tid; i < it.n * R; i += kFewThreads) p.h[(int64_t)it.row * R + i] = 0.0f;
    if (APART)
      for (int m = 0; m < it.n; ++m)
        copy_row(static_cast<const YT*>(p.y) + (int64_t)(it.row + m) * p.ldy,
                 static_cast<OT*>(p.out) + (int64_t)(it.row + m) * p.ldo, e0 / 8 + tid, e1 / 8, kFewThreads);
    return;
  }
  const XT* x = static_cast<const XT*>(p.x) + (int64_t)it.row * p.ldx;
  YT* y = static_cast<YT*>(p.y) + (int64_t)it.row * p.ldy;
  OT* out = APART ? static_cast<OT*>(p.out) + (int64_t)it.row * p.ldo : reinterpret_cast<OT*>(y);
  const int64_t ldo = APART ? p.ldo : p.ldy;
  const __nv_bfloat16* wa = p.a + (int64_t)it.l * R * p.K;
  const __nv_bfloat16* wb = p.b + (int64_t)it.l * p.N * R;
  int d0, d1;
  long_slice(D, cs, rank, d0, d1);
  // what the second product reads, on its way to L2 while the first one runs
  if (!BWD) {
    for (int64_t i = (int64_t)e0 * R + tid * 64; i < (int64_t)e1 * R; i += kFewThreads * 64) prefetch_l2(wb + i);
    if (T == 1)
      for (int c = e0 + tid * (128 / (int)sizeof(YT)); c < e1; c += kFewThreads * (128 / (int)sizeof(YT)))
        prefetch_l2(y + c);
  } else {
    for (int i = tid; i < R * ((e1 - e0 + 63) / 64); i += kFewThreads)
      prefetch_l2(wa + (int64_t)(i % R) * p.K + e0 + i / R * 64);
  }
  const int RV = R / 8;
  const int warp = tid >> 5, lane = tid & 31;
  // BWD: thread = (vector of 8 ranks, one of `nl` lanes over n), 8 x T sums.
  // Forward: warp = (four ranks, one of `kg` groups over k), 4 x T sums a lane.
  const int rv = tid % RV, nl_i = tid / RV, nl = kFewThreads / RV;

  if constexpr (BWD) {
    float acc[T][8];
#pragma unroll
    for (int m = 0; m < T; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[m][i] = 0.0f;
    for (int c0 = d0; c0 < d1; c0 += kFewChunk) {
      const int len = min(kFewChunk, d1 - c0);
      if constexpr (T > 1) {
        __syncthreads();
        if (warp < it.n)
          for (int k = lane * 8; k < len; k += 256) {
            float v[8];
            load8(x + (int64_t)warp * p.ldx + c0 + k, v);
            *reinterpret_cast<float4*>(xs + warp * XP + k) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(xs + warp * XP + k + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        else if (warp < T)
          for (int k = lane; k < len; k += 32) xs[warp * XP + k] = 0.0f;
        __syncthreads();
      }
      if (nl_i < nl) {
#pragma unroll 2
        for (int k = nl_i; k < len; k += nl) {
          float w[8];
          Vec<__nv_bfloat16>::load(wb + (int64_t)(c0 + k) * R + rv * 8, w);
#pragma unroll
          for (int m = 0; m < T; ++m) {
            const float v = T == 1 ? ld_elem(x + c0 + k) : xs[m * XP + k];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[m][i] = fmaf(w[i], v, acc[m][i]);
          }
        }
      }
    }
#pragma unroll
    for (int m0 = 0; m0 < T; m0 += MR) {
      float v[MR][8];
#pragma unroll
      for (int m = 0; m < MR; ++m)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[m][i] = acc[m0 + m][i];
      if (m0 < it.n) reduce_rank_vectors<MR>(v, nl_i < nl, RV, xs, part + m0, T);
    }
  } else {
    const int quads = (R + 3) / 4, kg = max(1, kFewWarps / quads);
    for (int i = tid; i < T * R; i += kFewThreads) part[i] = 0.0f;
    for (int c0 = d0; c0 < d1; c0 += kFewChunk) {
      const int len = min(kFewChunk, d1 - c0);
      if constexpr (T > 1) {
        __syncthreads();
        if (warp < it.n)
          for (int k = lane * 8; k < len; k += 256) {
            float v[8];
            load8(x + (int64_t)warp * p.ldx + c0 + k, v);
            *reinterpret_cast<float4*>(xs + warp * XP + k) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(xs + warp * XP + k + 4) = make_float4(v[4], v[5], v[6], v[7]);
          }
        else if (warp < T)
          for (int k = lane; k < len; k += 32) xs[warp * XP + k] = 0.0f;
        __syncthreads();
      }
      // quads beyond the warps go round again; kg > 1 only when they all fit
      for (int q = kg > 1 ? warp % quads : warp; q < quads; q += (kg > 1 ? quads : kFewWarps)) {
        const int g = kg > 1 ? warp / quads : 0;
        float s[4 * T];
#pragma unroll
        for (int i = 0; i < 4 * T; ++i) s[i] = 0.0f;
        if (g < kg) {
          for (int k = (g * 32 + lane) * 8; k < len; k += kg * 256) {
            uint4 raw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              raw[i] = make_uint4(0u, 0u, 0u, 0u);
              if (q * 4 + i < R)
                raw[i] = __ldg(reinterpret_cast<const uint4*>(wa + (int64_t)(q * 4 + i) * p.K + c0 + k));
            }
#pragma unroll
            for (int m = 0; m < T; ++m) {
              float v[8];
              if constexpr (T == 1) {
                load8(x + c0 + k, v);
              } else {
                const float4 v0 = *reinterpret_cast<const float4*>(xs + m * XP + k);
                const float4 v1 = *reinterpret_cast<const float4*>(xs + m * XP + k + 4);
                v[0] = v0.x; v[1] = v0.y; v[2] = v0.z; v[3] = v0.w;
                v[4] = v1.x; v[5] = v1.y; v[6] = v1.z; v[7] = v1.w;
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float w[8];
                Vec<__nv_bfloat16>::load_raw(raw[i], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) s[i * T + m] = fmaf(w[j], v[j], s[i * T + m]);
              }
            }
          }
        }
        if constexpr (T == 8) {
          // fold 32 sums over 32 lanes: lane i ends with the total of sum i
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (i < o) {
                const float give = (lane & o) ? s[i] : s[i + o];
                const float keep = (lane & o) ? s[i + o] : s[i];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              }
            }
          }
          if (g < kg) red[(g * quads + q) * 32 + lane] = s[0];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = warp_sum(s[i]);
          if (g < kg && lane < 4) red[(g * quads + q) * 4 + lane] = lane == 0 ? s[0] : lane == 1 ? s[1] : lane == 2 ? s[2] : s[3];
        }
      }
      __syncthreads();
      for (int i = tid; i < R * T; i += kFewThreads) {
        float t = part[i];
        for (int g = 0; g < kg; ++g) t += red[g * quads * 4 * T + i];
        part[i] = t;
      }
      if (T == 1) __syncthreads();
    }
  }
  __syncthreads();
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  const float scale = p.scale != nullptr ? __ldg(p.scale + it.l) : 1.0f;
  for (int i = tid; i < T * R; i += kFewThreads) {
    const int m = i % T;
    float t = 0.0f;
    if (m < it.n) {
      t = cs > 1 ? dsmem_sum(part + i, cs) : part[i];
    }
    full[i] = t * scale;
    if (p.h != nullptr && rank == 0 && m < it.n)
      p.h[(int64_t)(it.row + m) * R + i / T] = BWD ? t * scale : t;
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();
  if constexpr (BWD && T == 1) {
    // two columns a thread: whole lines of A's rows per warp (4 fp32 rows, 2304 -> 2304, rank 128,
    // with the gradients: 16.1 us, not 18.1)
    for (int c = e0 + 2 * tid; c < e1; c += 2 * kFewThreads) {
      float o0 = 0.0f, o1 = 0.0f;
#pragma unroll 2
      for (int r = 0; r < R; r += 8) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t*>(wa + (int64_t)(r + i) * p.K + c));
        const float4 v0 = *reinterpret_cast<const float4*>(full + r);
        const float4 v1 = *reinterpret_cast<const float4*>(full + r + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o0 = fmaf(__uint_as_float(w[i] << 16), v[i], o0);
          o1 = fmaf(__uint_as_float(w[i] & 0xFFFF0000u), v[i], o1);
        }
      }
      if constexpr (sizeof(YT) == 2) *reinterpret_cast<uint32_t*>(y + c) = pack_bf16(o0, o1);
      else *reinterpret_cast<float2*>(y + c) = make_float2(o0, o1);
    }
    __syncwarp();
    if (cs > 1) cluster_wait();
    return;
  }
  for (int c = e0 + tid; c < e1; c += kFewThreads) {
    float o[T];
#pragma unroll
    for (int m = 0; m < T; ++m) o[m] = 0.0f;
    for (int r = 0; r < R; r += 8) {
      float w[8];
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = to_f32(wa[(int64_t)(r + i) * p.K + c]);
      } else {
        Vec<__nv_bfloat16>::load(wb + (int64_t)c * R + r, w);
      }
      if constexpr (T == 1) {
        const float4 v0 = *reinterpret_cast<const float4*>(full + r);
        const float4 v1 = *reinterpret_cast<const float4*>(full + r + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) o[0] = fmaf(w[i], v[i], o[0]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 v0 = *reinterpret_cast<const float4*>(full + (r + i) * T);
          const float4 v1 = *reinterpret_cast<const float4*>(full + (r + i) * T + 4);
          const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int m = 0; m < T; ++m) o[m] = fmaf(w[i], v[m], o[m]);
        }
      }
    }
#pragma unroll
    for (int m = 0; m < T; ++m)
      if (m < it.n) {
        const YT* d = y + (int64_t)m * p.ldy + c;
        st_elem(out + (int64_t)m * ldo + c, BWD ? o[m] : to_f32(*d) + o[m]);
      }
  }
  __syncwarp();
  if (cs > 1) cluster_wait();
}

// ------------------------------------------------- gradients of the adapters
constexpr int kGradPiece = 64;

// The pieces of kGradPiece rows of adapter l's requests, found by a warp together, 32
// requests at a time; the CTAs of a cluster take them in turn.
struct GradPieces {
  const int32_t* bounds;
  const int32_t* index;
  int M, L, Q, l, rank, cs;
  int base = -32, pos = 0, end = 0, s = 0, e = 0, turn = 0;
  unsigned mask = 0;
  __device__ __forceinline__ bool next(int& m0, int& n) {
    const int lane = threadIdx.x & 31;
    while (pos >= end) {
      while (mask == 0) {
        base += 32;
        if (base >= Q) return false;
        const int q = base + lane;
        bool hit = false;
        if (q < Q && __ldg(index + q) == l) {
          s = __ldg(bounds + q);
          e = __ldg(bounds + q + 1);
          hit = s < e && request_counts(s, e, l, M, L);
        }
        mask = __ballot_sync(0xffffffffu, hit);
      }
      const int src = __ffs(mask) - 1;
      mask &= mask - 1;
      pos = __shfl_sync(0xffffffffu, s, src);
      end = __shfl_sync(0xffffffffu, e, src);
    }
    m0 = pos;
    n = min(kGradPiece, end - pos);
    pos += kGradPiece;
    return true;
  }
  __device__ __forceinline__ bool mine(int& m0, int& n) {
    while (next(m0, n)) {
      const bool is = turn == rank;
      turn = turn + 1 == cs ? 0 : turn + 1;
      if (is) return true;
    }
    return false;
  }
};

// fp32 rows, and requests of few: both gradients in one launch,
//   out[0][l][r][c] = sum over the rows of requests that use l of f[0][m][r] * g[0][m][c] (dA: u, x),
//   out[1][l][c][r] = scale_l times the same of f[1] and g[1]                              (dB: h, dy).
// One cluster per (64 columns, adapter): its CTAs share the pieces and add their sums in
// rank order, so they repeat bit for bit.  With the backward's first kernel, 777 fp32 rows,
// 1152 -> 2304, rank 8: 27 us (34.5 in a launch for each gradient), bound by the latency of the
// two kernels' loads and sums.
struct AdapterGradArgs {
  const float* f[2];             // [M, R]
  const void* g[2];              // [M, C]
  int64_t ldg[2];
  float* out[2];
  const float* scale;            // of the second, or null
  const int32_t* bounds;
  const int32_t* index;
  int32_t C[2];
  int32_t tiles0;                // column tiles of the first
  int32_t M, R, L, Q, cs;
};
constexpr int kGradCols = 64, kGradThreads = 256;

__device__ __forceinline__ float4 dsmem_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// Eight consecutive values at p summed over the cluster's CTAs in rank order, four
// CTAs' reads in flight together.
__device__ __forceinline__ void dsmem_sum8(const float* p, int cs, float (&v)[8]) {
  const uint32_t at = smem_u32(p);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  for (int q = 0; q < cs; q += 4) {
    float4 a[4], b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      a[k] = b[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (q + k < cs) {
        const uint32_t from = mapa_shared(at, q + k);
        a[k] = dsmem_f32x4(from);
        b[k] = dsmem_f32x4(from + 16);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[0] += a[k].x; v[1] += a[k].y; v[2] += a[k].z; v[3] += a[k].w;
      v[4] += b[k].x; v[5] += b[k].y; v[6] += b[k].z; v[7] += b[k].w;
    }
  }
}

template <typename GT, int WHICH>
__device__ __forceinline__ void adapter_grad_tile(const AdapterGradArgs& p, int tile, float* sh) {
  constexpr bool TRANS = WHICH == 1;
  const int C = p.C[WHICH];
  // rows of f and g, a whole piece of them where the ranks leave room; then the sums
  // [rank][column]
  const int step = p.R <= 64 ? kGradPiece : kGradPiece / 2;
  float* fs = sh;                                           // [row][rank]
  float* gs = sh + kAdapterMaxRank * kGradCols / 2;         // [row][column]
  const int tid = threadIdx.x, l = blockIdx.y, rank = blockIdx.x % p.cs, c0 = tile * kGradCols;
  // a thread: four ranks (r0 ..), the columns cx .. cx + 3 and 32 + cx .. , and every
  // `groups`-th row; the groups' sums are added at the end
  const int quads = p.R / 4, cx = (tid % 8) * 4, r0 = tid / 8 % quads * 4, group = tid / 8 / quads;
  const int groups = kGradThreads / 8 / quads;
  const bool active = group < groups;
  float acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  GradPieces pieces{p.bounds, p.index, p.M, p.L, p.Q, l, rank, p.cs};
  const int R4 = p.R / 4;
  int first, count;
  bool more = pieces.mine(first, count);
  while (more) {
    // rows of as many pieces as there is room for: requests of a row or two share a step (64
    // requests of one row, 6 adapters of rank 64, 4608 -> 1152: 29.3 us for all gradients, not 42.7)
    __syncthreads();
    int n = 0;
    while (more && n < step) {
      const int to = n + min(count, step - n);
      // the threads go by the rows' places, so pieces meet different warps
      for (int i = n * R4 + ((tid - n * R4) & (kGradThreads - 1)); i < to * R4; i += kGradThreads) {
        const int m = i / R4, r = i % R4 * 4;
        *reinterpret_cast<float4*>(fs + m * p.R + r) =
            __ldg(reinterpret_cast<const float4*>(p.f[WHICH] + (int64_t)(first + m - n) * p.R + r));
      }
      // C is a multiple of 16
      constexpr int G8 = kGradCols / 8;
      for (int i = n * G8 + ((tid - n * G8) & (kGradThreads - 1)); i < to * G8; i += kGradThreads) {
        const int m = i / G8, c = i % G8 * 8;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (c0 + c < C)
          load8(static_cast<const GT*>(p.g[WHICH]) + (int64_t)(first + m - n) * p.ldg[WHICH] + c0 + c, v);
        *reinterpret_cast<float4*>(gs + m * kGradCols + c) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(gs + m * kGradCols + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
      }
      first += to - n;
      count -= to - n;
      n = to;
      if (count == 0) more = pieces.mine(first, count);
    }
    __syncthreads();
    if (active) {
#pragma unroll 2
      for (int m = group; m < n; m += groups) {
        const float4 w = *reinterpret_cast<const float4*>(fs + m * p.R + r0);
        const float4 v0 = *reinterpret_cast<const float4*>(gs + m * kGradCols + cx);
        const float4 v1 = *reinterpret_cast<const float4*>(gs + m * kGradCols + cx + 32);
        const float wv[4] = {w.x, w.y, w.z, w.w};
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(wv[i], v[j], acc[i][j]);
      }
    }
  }
  // the groups' sums [group][rank][column] (groups * R <= 128), then this CTA's in the first
  const int outs = p.R * kGradCols;
  __syncthreads();
  if (active) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float* d = sh + group * outs + (r0 + i) * kGradCols + cx;
      *reinterpret_cast<float4*>(d) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
      *reinterpret_cast<float4*>(d + 32) = make_float4(acc[i][4], acc[i][5], acc[i][6], acc[i][7]);
    }
  }
  __syncthreads();
  for (int o = tid * 4; o < outs; o += kGradThreads * 4) {
    float4 t = *reinterpret_cast<const float4*>(sh + o);
    for (int k = 1; k < groups; ++k) {
      const float4 v = *reinterpret_cast<const float4*>(sh + k * outs + o);
      t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    *reinterpret_cast<float4*>(sh + o) = t;
  }
  if (p.cs > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  const float scale = TRANS && p.scale != nullptr ? __ldg(p.scale + l) : 1.0f;
  // the CTAs of the cluster write eight columns of a rank in turn
  for (int u = tid; u < outs / 8; u += kGradThreads) {
    if (p.cs > 1 && u % p.cs != rank) continue;
    const int r = u / (kGradCols / 8), c = c0 + u % (kGradCols / 8) * 8;
    if (c >= C) continue;
    float v[8];
    dsmem_sum8(sh + u * 8, p.cs, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    if (TRANS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p.out[1][((int64_t)l * C + c + j) * p.R + r] = v[j];
    } else {
      store_vec<8>(p.out[0], ((int64_t)l * p.R + r) * C + c, false, v);
    }
  }
  __syncwarp();
  if (p.cs > 1) { cluster_arrive(); cluster_wait(); }
}

template <typename XT, typename DT>
__global__ void __launch_bounds__(kGradThreads, 3) adapter_grad_kernel(const AdapterGradArgs p) {
  __shared__ __align__(16) float sh[kAdapterMaxRank * kGradCols];
  const int tile = blockIdx.x / p.cs;
  grid_dep_wait();
  if (tile < p.tiles0) adapter_grad_tile<XT, 0>(p, tile, sh);
  else adapter_grad_tile<DT, 1>(p, tile - p.tiles0, sh);
}

}  // namespace sq
