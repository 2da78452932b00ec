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
// adapter.  Up to 62 requests: a warp counts the pieces of all of them and sums the
// counts, so the items come without gaps.  More: request r's pieces begin at slot
// floor(start_r / T) + r, which leaves room for a request of any length before the
// next one's, so its own bounds alone place them and a 32-way search finds the
// request of a slot.  M / T + Q + 3 slots hold every piece in both.
// Pieces of a request with bounds outside the batch or an index beyond the adapters
// are left out, so no read or write leaves the tensors; check_requests raises the
// range status for them.
__device__ __forceinline__ AdapterItem adapter_item(const AdapterArgs& p, int slot, int T) {
  const int lane = threadIdx.x & 31;
  const int count = p.Q + 2;
  auto start = [&](int r) { return r == 0 ? 0 : r <= p.Q + 1 ? __ldg(p.bounds + r - 1) : p.M; };
  AdapterItem it;
  int s, e, piece, lo;
  if (count <= 64) {
    // lane: requests 2 lane and 2 lane + 1
    const int r = 2 * lane;
    const int b0 = r < count ? start(r) : p.M, b1 = r < count ? start(r + 1) : p.M,
              b2 = r + 1 < count ? start(r + 2) : p.M;
    const int l0 = r >= 1 && r <= p.Q ? __ldg(p.index + r - 1) : -1, l1 = r + 1 <= p.Q ? __ldg(p.index + r) : -1;
    const int n0 = max(0, b1 - b0 + T - 1) / T, n1 = max(0, b2 - b1 + T - 1) / T;
    int sum = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned m = __ballot_sync(0xffffffffu, sum > slot);
    it.row = it.n = 0;
    it.l = -1;
    if (m == 0) return it;
    const int src = __ffs(m) - 1;
    const int first = slot - (sum - n0 - n1);              // within the lane's two requests
    const bool second = first >= n0;
    s = __shfl_sync(0xffffffffu, second ? b1 : b0, src);
    e = __shfl_sync(0xffffffffu, second ? b2 : b1, src);
    it.l = __shfl_sync(0xffffffffu, second ? l1 : l0, src);
    piece = __shfl_sync(0xffffffffu, second ? first - n0 : first, src);
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
    s = start(lo);
    e = start(lo + 1);
    it.l = (lo == 0 || lo == p.Q + 1) ? -1 : __ldg(p.index + lo - 1);
    piece = slot - (s / T + lo);
  }
  it.row = s + piece * T;
  it.n = min(T, e - it.row);
  if (s < 0 || e > p.M || it.l >= p.L || piece < 0 || it.n < 0) it.n = 0;
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
// One cluster of CTAs per piece of up to eight rows: each CTA contracts its
// slice of the long axis on the fp32 lanes, the partial h (or u) are added
// through distributed shared memory in rank order, and each CTA then writes its
// slice of the columns.  This is the form for batches of requests of a few rows
// (one conditioning vector each), which are bound by launch and load latency
// and by the adapters' bytes, and for fp32 rows.
constexpr int kFewRows = 8;
constexpr int kFewThreads = 512;
constexpr int kFewChunk = 512;   // elements of the long axis staged at a time

template <typename T>
__device__ __forceinline__ float ld_elem(const T* p) { return to_f32(*p); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Slice k of n elements cut into cs slices of whole 8-element vectors.
__device__ __forceinline__ void long_slice(int n, int cs, int k, int& from, int& to) {
  const int per = ((n + 8 * cs - 1) / (8 * cs)) * 8;
  from = min(n, k * per);
  to = min(n, from + per);
}

// BWD = false: x A^T, then y += scale h B^T.  BWD = true: scale dy B, then dx = u A.
template <typename XT, typename YT, bool BWD>
__global__ void __launch_bounds__(kFewThreads, 1)
    adapter_few_rows_kernel(const AdapterArgs p, int cs) {
  __shared__ __align__(16) float xs[kFewChunk * kFewRows];            // [k][row]
  __shared__ float part[kFewRows * kAdapterMaxRank];                  // [r][row], this CTA's share
  __shared__ __align__(16) float full[kFewRows * kAdapterMaxRank];    // [r][row], times scale
  __shared__ __align__(16) float red[kFewThreads * kFewRows];
  const int rank = blockIdx.x % cs;
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) check_requests(p, kFewThreads);
  const AdapterItem it = adapter_item(p, blockIdx.x / cs, kFewRows);
  const int D = BWD ? p.N : p.K, E = BWD ? p.K : p.N, R = p.R;   // contracted, written
  int e0, e1;
  long_slice(E, cs, rank, e0, e1);
  if (it.n == 0 || it.l < 0) {       // the same for every CTA of the cluster
    if (BWD) {
      YT* y = static_cast<YT*>(p.y);
      for (int m = 0; m < it.n; ++m)
        for (int c = e0 + tid; c < e1; c += kFewThreads) st_elem(y + (int64_t)(it.row + m) * p.ldy + c, 0.0f);
    } else if (p.h != nullptr && rank == 0) {
      for (int i = tid; i < it.n * R; i += kFewThreads) p.h[(int64_t)it.row * R + i] = 0.0f;
    }
    return;
  }
  const XT* x = static_cast<const XT*>(p.x) + (int64_t)it.row * p.ldx;
  const __nv_bfloat16* wa = p.a + (int64_t)it.l * R * p.K;
  const __nv_bfloat16* wb = p.b + (int64_t)it.l * p.N * R;
  int d0, d1;
  long_slice(D, cs, rank, d0, d1);
  const int RV = R / 8;
  const int warp = tid >> 5, lane = tid & 31;

  // BWD: thread = (vector of 8 ranks, one of `nl` lanes over n), 8 x 8 sums.
  // Forward: warp = (four ranks, one of `kg` groups over k), 4 x 8 sums a lane.
  const int rv = tid % RV, nl_i = tid / RV, nl = kFewThreads / RV;
  const int quads = (R + 3) / 4, kg = max(1, (kFewThreads / 32) / quads);
  float acc[BWD ? 64 : 32];
  if (BWD) {
#pragma unroll
    for (int i = 0; i < (BWD ? 64 : 32); ++i) acc[i] = 0.0f;
  }
  for (int i = tid; i < kFewRows * R; i += kFewThreads) part[i] = 0.0f;
  for (int c0 = d0; c0 < d1; c0 += kFewChunk) {
    const int len = min(kFewChunk, d1 - c0);
    __syncthreads();
    for (int i = tid; i < len * kFewRows; i += kFewThreads) {
      const int m = i / len, k = i % len;
      xs[k * kFewRows + m] = m < it.n ? ld_elem(x + (int64_t)m * p.ldx + c0 + k) : 0.0f;
    }
    __syncthreads();
    if constexpr (BWD) {
      if (nl_i < nl) {
        for (int k = nl_i; k < len; k += nl) {
          float w[8];
          Vec<__nv_bfloat16>::load(wb + (int64_t)(c0 + k) * R + rv * 8, w);
          const float4 v0 = *reinterpret_cast<const float4*>(xs + k * kFewRows);
          const float4 v1 = *reinterpret_cast<const float4*>(xs + k * kFewRows + 4);
          const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int m = 0; m < 8; ++m) acc[i * 8 + m] = fmaf(w[i], v[m], acc[i * 8 + m]);
        }
      }
    } else {
      // quads beyond the warps go round again; kg > 1 only when they all fit
      for (int q = kg > 1 ? warp % quads : warp; q < quads; q += (kg > 1 ? quads : kFewThreads / 32)) {
        const int g = kg > 1 ? warp / quads : 0;
        float s[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = 0.0f;
        if (g < kg) {
          for (int k = (g * 32 + lane) * 8; k < len; k += kg * 256) {
            float w[4][8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (q * 4 + i < R) Vec<__nv_bfloat16>::load(wa + (int64_t)(q * 4 + i) * p.K + c0 + k, w[i]);
              else
#pragma unroll
                for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float4 v0 = *reinterpret_cast<const float4*>(xs + (k + j) * kFewRows);
              const float4 v1 = *reinterpret_cast<const float4*>(xs + (k + j) * kFewRows + 4);
              const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int m = 0; m < 8; ++m) s[i * 8 + m] = fmaf(w[i][j], v[m], s[i * 8 + m]);
            }
          }
        }
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
      }
      __syncthreads();
      for (int i = tid; i < R * kFewRows; i += kFewThreads) {
        float t = part[i];
        for (int g = 0; g < kg; ++g) t += red[(g * quads + i / 32) * 32 + i % 32];
        part[i] = t;
      }
    }
  }
  if constexpr (BWD) {
    // add the nl lanes' sums, one rank of each vector at a time
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      __syncthreads();
      if (nl_i < nl) {
#pragma unroll
        for (int m = 0; m < 8; ++m) red[tid * 8 + m] = acc[i * 8 + m];
      }
      __syncthreads();
      // 8 * RV totals; `ways` threads share each, then one adds theirs
      const int outs = 8 * RV;
      const int ways = min(nl, kFewThreads / outs);
      const int o = tid % outs, wy = tid / outs;
      float t = 0.0f;
      if (wy < ways)
        for (int j = wy; j < nl; j += ways) t += red[j * outs + o];
      __syncthreads();
      if (wy < ways) red[wy * outs + o] = t;
      __syncthreads();
      if (tid < outs) {
        float a = 0.0f;
        for (int j = 0; j < ways; ++j) a += red[j * outs + tid];
        part[(tid / 8 * 8 + i) * kFewRows + tid % 8] = a;
      }
    }
  }
  __syncthreads();
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  const float scale = p.scale != nullptr ? p.scale[it.l] : 1.0f;
  for (int i = tid; i < kFewRows * R; i += kFewThreads) {
    float t = 0.0f;
    if (cs > 1) {
      for (int k = 0; k < cs; ++k) t += dsmem_f32(part + i, k);
    } else {
      t = part[i];
    }
    full[i] = t * scale;
    const int m = i % kFewRows;
    if (p.h != nullptr && rank == 0 && m < it.n)
      p.h[(int64_t)(it.row + m) * R + i / kFewRows] = BWD ? t * scale : t;
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();
  YT* y = static_cast<YT*>(p.y) + (int64_t)it.row * p.ldy;
  for (int c = e0 + tid; c < e1; c += kFewThreads) {
    float o[kFewRows];
#pragma unroll
    for (int m = 0; m < kFewRows; ++m) o[m] = 0.0f;
    for (int r = 0; r < R; r += 8) {
      float w[8];
      if constexpr (BWD) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = to_f32(wa[(int64_t)(r + i) * p.K + c]);
      } else {
        Vec<__nv_bfloat16>::load(wb + (int64_t)c * R + r, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 v0 = *reinterpret_cast<const float4*>(full + (r + i) * kFewRows);
        const float4 v1 = *reinterpret_cast<const float4*>(full + (r + i) * kFewRows + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int m = 0; m < 8; ++m) o[m] = fmaf(w[i], v[m], o[m]);
      }
    }
#pragma unroll
    for (int m = 0; m < kFewRows; ++m)
      if (m < it.n) {
        YT* d = y + (int64_t)m * p.ldy + c;
        st_elem(d, BWD ? o[m] : to_f32(*d) + o[m]);
      }
  }
  __syncwarp();
  if (cs > 1) cluster_wait();
}

// ------------------------------------------------- gradients of the adapters
// out[l][r][c] = sum over the rows of requests that use l of f[m][r] * g[m][c]
// (TRANS: written as out[l][c][r]), times scale_l when asked.  One CTA per
// (64 columns, adapter): rows in order, so the sums repeat bit for bit.
struct AdapterGradArgs {
  const float* f;                // [M, R]
  const void* g;                 // [M, C]
  int64_t ldg;
  const float* scale;            // or null
  const int32_t* bounds;
  const int32_t* index;
  float* out;
  int32_t M, C, R, L, Q;
};
constexpr int kGradCols = 64, kGradRows = 32, kGradThreads = 256;

template <typename GT, bool TRANS>
__global__ void __launch_bounds__(kGradThreads) adapter_grad_kernel(const AdapterGradArgs p) {
  __shared__ __align__(16) float fs[kGradRows][kAdapterMaxRank];
  __shared__ __align__(16) float gs[kGradRows][kGradCols];
  const int tid = threadIdx.x, l = blockIdx.y, c0 = blockIdx.x * kGradCols;
  // thread: 8 columns (cx) and the ranks ry, ry + 32, ...
  const int cx = (tid % 8) * 8, ry = tid / 8;
  float acc[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = 0.0f;
  for (int q = 0; q < p.Q; ++q) {
    if (p.index[q] != l) continue;
    const int s = max(0, p.bounds[q]), e = min(p.M, p.bounds[q + 1]);
    for (int m0 = s; m0 < e; m0 += kGradRows) {
      const int n = min(kGradRows, e - m0);
      __syncthreads();
      for (int i = tid; i < kGradRows * p.R; i += kGradThreads) {
        const int m = i / p.R, r = i % p.R;
        fs[m][r] = m < n ? p.f[(int64_t)(m0 + m) * p.R + r] : 0.0f;
      }
      for (int i = tid; i < kGradRows * kGradCols; i += kGradThreads) {
        const int m = i / kGradCols, c = i % kGradCols;
        gs[m][c] = m < n && c0 + c < p.C
                       ? ld_elem(static_cast<const GT*>(p.g) + (int64_t)(m0 + m) * p.ldg + c0 + c)
                       : 0.0f;
      }
      __syncthreads();
      for (int m = 0; m < n; ++m) {
        const float4 v0 = *reinterpret_cast<const float4*>(&gs[m][cx]);
        const float4 v1 = *reinterpret_cast<const float4*>(&gs[m][cx + 4]);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (ry + 32 * i < p.R) {
            const float w = fs[m][ry + 32 * i];
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(w, v[j], acc[i][j]);
          }
        }
      }
    }
  }
  const float scale = p.scale != nullptr ? p.scale[l] : 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = ry + 32 * i;
    if (r < p.R) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = c0 + cx + j;
        if (c < p.C)
          p.out[TRANS ? ((int64_t)l * p.C + c) * p.R + r : ((int64_t)l * p.R + r) * p.C + c] = acc[i][j] * scale;
      }
    }
  }
}

}  // namespace sq
