// Group norm with an activation on channels-last maps x [B, S, C] (S = H*W
// positions, unit channel stride): forward, gradients, and the norm fused into
// the producer of the DualScale codes.
//
//   mean_g, var_g over the S positions and the C/G channels of group g
//   xhat = (x - mean_g) * rstd_g,  rstd_g = 1 / sqrt(var_g + eps)
//   z = xhat * gamma_c + beta_c,   y = act(z)
//   dz = dy * act'(z), dbeta_c = sum dz, dgamma_c = sum dz * xhat
//   dx = rstd_g * (dz gamma_c - m1 - xhat m2), with m1, m2 the group's means
//   of dz gamma_c and dz gamma_c xhat
//
// Everything here is bound by memory: an element costs about ten instructions.
// Where the slab of one image and one block of groups fits the registers of a
// cluster of CTAs, it is read once, the cluster exchanges the group's sums
// through distributed shared memory and writes the result from registers (one
// launch, no workspace).  Larger maps take two passes, the second reading what
// the first left in L2.  Every sum has a fixed order: results repeat bit for bit.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "quant_kernels.cuh"

namespace sq {

constexpr int kNormThreads = 512;    // of the cluster form
constexpr int kNormThreads2 = 256;   // of the two-pass form (512 for groups wider than 256 vectors)
constexpr int ACT_NONE = 0;

// One block of channels (whole groups, a multiple of 16 bytes wide) and how a
// CTA's threads lie over it: vx 16-byte vectors across, ty positions down.
struct NormTile {
  int32_t S, C, G, cpg;   // positions, channels, groups, channels per group
  int32_t nb;             // groups per channel block
  int32_t vx, ty;         // vx * ty <= threads of the CTA
  int32_t rows;           // positions per CTA
};

struct NormArgs {
  const void* x;
  int64_t ldx, xbs;              // element strides of positions and images
  void* y;                       // fp32 or bf16, may be null when codes are written
  int64_t ldy, ybs;
  int8_t* q_pos;                 // DualScale codes [B*S, C], or null
  int8_t* q_neg;
  int64_t ldq;
  const float* gamma;            // [C] or null (1)
  const float* beta;             // [C] or null (0)
  const float* s_pos;
  const float* s_neg;
  float* stats;                  // [B][G][2] mean, rstd; or null
  float2* part;                  // two passes: [B][tiles][G] mean, M2 of each tile
  SegBounds kseg;
  NormTile t;
  int32_t tiles;
  int32_t act;
  int32_t y_bf16;
  float eps;
};

struct NormBwdArgs {
  const void* x;
  int64_t ldx, xbs;
  const void* dy;
  int64_t lddy, dybs;
  void* dx;
  int64_t lddx, dxbs;
  const float* gamma;
  const float* beta;
  const float* stats;            // [B][G][2] mean, rstd of the forward pass
  float* part;                   // [B][tiles][2][C]: sums of dz and of dz * (x - mean)
  float* total;                  // [B][2][C]: the same over all positions of an image
  NormTile t;
  int32_t tiles;                 // per image; 0: total is written by the clusters
  int32_t act;
};

// ------------------------------------------------------------ vector access
template <typename T>
__device__ __forceinline__ uint4 load_stream(const T* p) {
  return __ldcs(reinterpret_cast<const uint4*>(p));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// VN consecutive fp32 values (4 or 8) stored as bf16 or fp32.
template <int VN>
__device__ __forceinline__ void store_vec(void* y, int64_t at, bool bf16, const float (&v)[VN]) {
  if (bf16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(y) + at;
    if constexpr (VN == 8) {
      const uint4 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                       pack_bf16(v[6], v[7])};
      *reinterpret_cast<uint4*>(p) = u;
    } else {
      const uint2 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
      *reinterpret_cast<uint2*>(p) = u;
    }
  } else {
    float* p = static_cast<float*>(y) + at;
#pragma unroll
    for (int i = 0; i < VN; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

// -------------------------------------------------------------- activations
// exp and the quotient by CUDA's fast forms (relative error about 2^-21): the
// result is stored in bf16, or in fp32 within 1e-6 of its scale.
template <int ACT>
__device__ __forceinline__ float norm_act(float z) {
  if constexpr (ACT == ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
  else if constexpr (ACT == ACT_GELU) return 0.5f * z * (1.0f + erff(z * 0.70710678f));
  else return z;
}
template <int ACT>
__device__ __forceinline__ float norm_act_slope(float z) {
  if constexpr (ACT == ACT_SILU) {
    const float p = __fdividef(1.0f, 1.0f + __expf(-z));
    return p * fmaf(z, 1.0f - p, 1.0f);
  } else if constexpr (ACT == ACT_GELU) {
    return fmaf(z * 0.39894228f, __expf(-0.5f * z * z), fmaf(0.5f, erff(z * 0.70710678f), 0.5f));
  } else {
    return 1.0f;
  }
}
// The activation is a launch argument: one uniform branch outside the loops.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else f(std::integral_constant<int, ACT_NONE>{});
}

// --------------------------------------------------------------- reductions
// Per-thread, per-channel values v[VN] of all rows of threads -> per-channel
// totals ch[0 .. vx*VN) in shared memory.  `scratch` holds NT * VN
// floats.  Begins and ends with every thread past a barrier.
template <int NT, int VN>
__device__ __forceinline__ void reduce_channels(const float (&v)[VN], bool active, int tx, int r,
                                                const NormTile& t, float* scratch, float* ch) {
  const int W = t.vx * VN;
  __syncthreads();
  if (active) {
#pragma unroll
    for (int i = 0; i < VN; i += 4)
      *reinterpret_cast<float4*>(scratch + r * W + tx * VN + i) =
          make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
  __syncthreads();
  const int nseg = W < NT ? NT / W : 1;
  if (nseg == 1) {
    for (int c = threadIdx.x; c < W; c += NT) {
      float s = 0.0f;
      for (int k = 0; k < t.ty; ++k) s += scratch[k * W + c];
      ch[c] = s;
    }
    __syncthreads();
    return;
  }
  const int c = threadIdx.x % W, sg = threadIdx.x / W;
  float s = 0.0f;
  if (sg < nseg)
    for (int k = sg; k < t.ty; k += nseg) s += scratch[k * W + c];
  __syncthreads();
  if (sg < nseg) scratch[sg * W + c] = s;
  __syncthreads();
  if (threadIdx.x < W) {
    float a = 0.0f;
    for (int k = 0; k < nseg; ++k) a += scratch[k * W + threadIdx.x];
    ch[threadIdx.x] = a;
  }
  __syncthreads();
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Group totals grp[0 .. nb) of the per-thread, per-channel values.
template <int NT, int VN>
__device__ __forceinline__ void reduce_groups(const float (&v)[VN], bool active, int tx, int r,
                                              const NormTile& t, float* scratch, float* ch,
                                              float* grp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (t.cpg % VN == 0) {
    // a vector lies in one group: one value per thread
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VN; ++i) s += v[i];
    if (t.nb == 1) {
      s = warp_sum(active ? s : 0.0f);
      __syncthreads();
      if (lane == 0) scratch[warp] = s;
      __syncthreads();
      s = warp_sum(lane < (NT / 32) ? scratch[lane] : 0.0f);
      if (threadIdx.x == 0) grp[0] = s;
      __syncthreads();
      return;
    }
    __syncthreads();
    const int vg = t.cpg / VN;                       // vectors across a group
    const int per = vg * t.ty;
    if (active) scratch[(tx / vg) * per + r * vg + tx % vg] = s;
    __syncthreads();
    for (int g = warp; g < t.nb; g += (NT / 32)) {
      float a = 0.0f;
      for (int k = lane; k < per; k += 32) a += scratch[g * per + k];
      a = warp_sum(a);
      if (lane == 0) grp[g] = a;
    }
    __syncthreads();
    return;
  }
  reduce_channels<NT, VN>(v, active, tx, r, t, scratch, ch);
  for (int g = warp; g < t.nb; g += (NT / 32)) {
    float a = 0.0f;
    for (int k = lane; k < t.cpg; k += 32) a += ch[g * t.cpg + k];
    a = warp_sum(a);
    if (lane == 0) grp[g] = a;
  }
  __syncthreads();
}

// (n, mean, M2) of a union of two sets (Chan et al., "Updating Formulae and a
// Pairwise Algorithm for Computing Sample Variances").
__device__ __forceinline__ void chan_merge(float& n, float& mean, float& m2, float nb, float meanb,
                                           float m2b) {
  if (nb == 0.0f) return;
  const float nn = n + nb, d = meanb - mean, f = nb / nn;
  mean = fmaf(d, f, mean);
  m2 += m2b + d * d * n * f;
  n = nn;
}

__device__ __forceinline__ float dsmem_f32(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// --------------------------------------------------------- per-thread apply
// The channel constants of one thread's vector and what it writes: z = x a + b
// with b = beta - mean a, off by 2^-24 of |mean a| like the mean itself.
template <int VN>
struct NormOut {
  float a[VN], b[VN], rp, rn;
  __device__ __forceinline__ void init(const NormArgs& p, int c0, int lc, const float* mean_g,
                                       const float* rstd_g) {
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int g = (lc + i) / p.t.cpg, c = c0 + lc + i;
      a[i] = rstd_g[g] * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      b[i] = fmaf(-mean_g[g], a[i], p.beta ? __ldg(p.beta + c) : 0.0f);
    }
    rp = rn = 0.0f;
    if (p.q_pos != nullptr) {
      const int j = p.kseg.segment_of(c0 + lc);   // bounds are multiples of 128
      const float sp = p.s_pos[j], sn = p.s_neg[j];
      rp = sp > 0.0f ? __frcp_rn(sp) : 0.0f;
      rn = sn > 0.0f ? __frcp_rn(sn) : 0.0f;
    }
  }
  template <int ACT>
  __device__ __forceinline__ void put(const NormArgs& p, int img, int row, int c, const float (&x)[VN]) {
    float v[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] = norm_act<ACT>(fmaf(x[i], a[i], b[i]));
    if (p.q_pos != nullptr) {
      // the codes are those of the bf16 values that y holds
      uint32_t q[VN], n[VN];
#pragma unroll
      for (int i = 0; i < VN; ++i) {
        v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
        q[i] = code_pos(v[i], rp);
        n[i] = code_neg(v[i], rn);
      }
      const int64_t at = ((int64_t)img * p.t.S + row) * p.ldq + c;
      if constexpr (VN == 8) {
        *reinterpret_cast<uint2*>(p.q_pos + at) =
            make_uint2(pack4_low(q[0], q[1], q[2], q[3]), pack4_low(q[4], q[5], q[6], q[7]));
        *reinterpret_cast<uint2*>(p.q_neg + at) =
            make_uint2(pack4_low(n[0], n[1], n[2], n[3]), pack4_low(n[4], n[5], n[6], n[7]));
      } else {
        *reinterpret_cast<uint32_t*>(p.q_pos + at) = pack4_low(q[0], q[1], q[2], q[3]);
        *reinterpret_cast<uint32_t*>(p.q_neg + at) = pack4_low(n[0], n[1], n[2], n[3]);
      }
    }
    if (p.y != nullptr)
      store_vec<VN>(p.y, (int64_t)img * p.ybs + (int64_t)row * p.ldy + c, p.y_bf16 != 0, v);
  }
};

// Shared memory of the norm kernels, in floats: scratch (reductions, then the
// cluster's totals), two totals per channel and four values per group.
__host__ __device__ inline int norm_smem_floats(int threads, int vx, int vn, int nb) {
  const int w2 = 2 * vx * vn;
  return (threads * vn > w2 ? threads * vn : w2) + w2 + 4 * nb;
}

// ------------------------------------------------- forward, slab in registers
// Cluster of `cs` CTAs per (image, channel block); CTA rank k holds positions
// k*rows .. of it, NV 16-byte vectors per thread, all requested at once.
template <typename XT, int NV>
__global__ void __launch_bounds__(kNormThreads, NV <= 4 ? 2 : 1)
    group_norm_cluster_kernel(const NormArgs p, int cs) {
  constexpr int VN = Vec<XT>::n;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = sm;
  float* ch = scratch + max(kNormThreads * VN, 2 * W);
  float* pub_mean = ch + 2 * W;
  float* pub_m2 = pub_mean + t.nb;
  float* fin_mean = pub_m2 + t.nb;
  float* fin_rstd = fin_mean + t.nb;

  const int rank = blockIdx.x % cs, cb = blockIdx.x / cs, img = blockIdx.y;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = rank * t.rows, r1 = min(t.S, r0 + t.rows);
  const int n_rows = max(0, r1 - r0);
  const XT* base = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;

  uint4 raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int row = r0 + r + i * t.ty;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (active && row < r1) raw[i] = load_stream(base + (int64_t)row * p.ldx);
  }
  float s[VN];
#pragma unroll
  for (int k = 0; k < VN; ++k) s[k] = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[VN];
    Vec<XT>::load_raw(raw[i], v);
#pragma unroll
    for (int k = 0; k < VN; ++k) s[k] += v[k];   // absent rows are zeros
  }
  reduce_groups<kNormThreads, VN>(s, active, tx, r, t, scratch, ch, pub_mean);
  const float n_loc = (float)n_rows * (float)t.cpg;
  for (int g = threadIdx.x; g < t.nb; g += kNormThreads)
    pub_mean[g] = n_loc > 0.0f ? pub_mean[g] / n_loc : 0.0f;
  __syncthreads();
  float m[VN];
#pragma unroll
  for (int k = 0; k < VN; ++k) { m[k] = active ? pub_mean[(lc + k) / t.cpg] : 0.0f; s[k] = 0.0f; }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float v[VN];
    Vec<XT>::load_raw(raw[i], v);
    if (r0 + r + i * t.ty < r1) {
#pragma unroll
      for (int k = 0; k < VN; ++k) { const float d = v[k] - m[k]; s[k] = fmaf(d, d, s[k]); }
    }
  }
  reduce_groups<kNormThreads, VN>(s, active, tx, r, t, scratch, ch, pub_m2);
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  for (int g = threadIdx.x; g < t.nb; g += kNormThreads) {
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    if (cs > 1) {
      for (int k = 0; k < cs; ++k) {
        const float nk = (float)max(0, min(t.S, (k + 1) * t.rows) - k * t.rows) * (float)t.cpg;
        chan_merge(n, mean, m2, nk, dsmem_f32(pub_mean + g, k), dsmem_f32(pub_m2 + g, k));
      }
    } else {
      n = n_loc; mean = pub_mean[g]; m2 = pub_m2[g];
    }
    const float rstd = 1.0f / sqrtf(m2 / n + p.eps);
    fin_mean[g] = mean;
    fin_rstd[g] = rstd;
    if (p.stats != nullptr && rank == 0) {
      float* d = p.stats + ((int64_t)img * t.G + cb * t.nb + g) * 2;
      d[0] = mean;
      d[1] = rstd;
    }
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();   // this CTA has read its peers' shared memory
  if (active) {
    NormOut<VN> o;
    o.init(p, c0, lc, fin_mean, fin_rstd);
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = r0 + r + i * t.ty;
        float v[VN];
        Vec<XT>::load_raw(raw[i], v);
        if (row < r1) o.template put<decltype(act)::value>(p, img, row, c0 + lc, v);
      }
    });
  }
  __syncwarp();
  if (cs > 1) cluster_wait();     // the peers have read this CTA's
}

// ------------------------------------------------------- forward, two passes
// Pass 1: one CTA per (tile of positions, channel block, image) writes mean and
// M2 of each of its groups.  A thread takes a few rows at a time: their mean
// and squared deviations per channel, merged into its running ones.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 1) group_norm_stats_kernel(const NormArgs p) {
  constexpr int VN = Vec<XT>::n, U = 32 / VN;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = sm;
  float* ch = scratch + max(NT * VN, 2 * W);
  float* g_mean = ch + 2 * W;
  float* g_m2 = g_mean + t.nb;
  grid_dep_launch();
  const int tile = blockIdx.x, cb = blockIdx.y, img = blockIdx.z;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = tile * t.rows, r1 = min(t.S, r0 + t.rows);
  const XT* base = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;
  float n = 0.0f, mean[VN], m2[VN];
#pragma unroll
  for (int k = 0; k < VN; ++k) mean[k] = m2[k] = 0.0f;
  if (active) {
    uint4 raw[U], ahead[U];
    auto fetch = [&](uint4 (&to)[U], int row) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        to[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row + i * t.ty < r1)
          to[i] = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)(row + i * t.ty) * p.ldx));
      }
    };
    fetch(ahead, r0 + r);
    for (int row = r0 + r; row < r1; row += U * t.ty) {
#pragma unroll
      for (int i = 0; i < U; ++i) raw[i] = ahead[i];
      fetch(ahead, row + U * t.ty);      // in flight while this chunk is summed
      const int cnt = min(U, (r1 - row + t.ty - 1) / t.ty);
      float s[VN];
#pragma unroll
      for (int k = 0; k < VN; ++k) s[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[VN];
        Vec<XT>::load_raw(raw[i], v);
#pragma unroll
        for (int k = 0; k < VN; ++k) s[k] += v[k];
      }
      const float nc = (float)cnt, inv = 1.0f / nc, nn = n + nc, f = nc / nn;
      float q[VN];
#pragma unroll
      for (int k = 0; k < VN; ++k) { s[k] *= inv; q[k] = 0.0f; }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[VN];
        Vec<XT>::load_raw(raw[i], v);
        if (i < cnt) {
#pragma unroll
          for (int k = 0; k < VN; ++k) { const float d = v[k] - s[k]; q[k] = fmaf(d, d, q[k]); }
        }
      }
#pragma unroll
      for (int k = 0; k < VN; ++k) {
        const float d = s[k] - mean[k];
        mean[k] = fmaf(d, f, mean[k]);
        m2[k] += fmaf(d * d, n * f, q[k]);
      }
      n = nn;
    }
  }
  float s[VN];
#pragma unroll
  for (int k = 0; k < VN; ++k) s[k] = n * mean[k];
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, g_mean);
  const float n_tile = (float)(r1 - r0) * (float)t.cpg;
  for (int g = threadIdx.x; g < t.nb; g += NT) g_mean[g] /= n_tile;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < VN; ++k) {
    const float d = active ? mean[k] - g_mean[(lc + k) / t.cpg] : 0.0f;
    s[k] = fmaf(n * d, d, m2[k]);
  }
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, g_m2);
  for (int g = threadIdx.x; g < t.nb; g += NT)
    p.part[((int64_t)img * p.tiles + tile) * t.G + cb * t.nb + g] = make_float2(g_mean[g], g_m2[g]);
}

// Pass 2: the same tiles in the opposite order (the last ones read are the
// likeliest in L2); each CTA merges its groups' tiles first, a warp per group.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 1) group_norm_apply_kernel(const NormArgs p) {
  constexpr int VN = Vec<XT>::n, U = 4;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  float* fin_mean = sm;
  float* fin_rstd = sm + t.nb;
  const int tile = gridDim.x - 1 - blockIdx.x, cb = gridDim.y - 1 - blockIdx.y,
            img = gridDim.z - 1 - blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = cb * t.nb * t.cpg;
  grid_dep_wait();
  for (int g = warp; g < t.nb; g += (NT / 32)) {
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    for (int k = lane; k < p.tiles; k += 32) {
      const float2 v = p.part[((int64_t)img * p.tiles + k) * t.G + cb * t.nb + g];
      const float nk = (float)(min(t.S, (k + 1) * t.rows) - k * t.rows) * (float)t.cpg;
      chan_merge(n, mean, m2, nk, v.x, v.y);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float n2 = __shfl_down_sync(0xffffffffu, n, o), mean2 = __shfl_down_sync(0xffffffffu, mean, o),
                  m22 = __shfl_down_sync(0xffffffffu, m2, o);
      if (lane < o) chan_merge(n, mean, m2, n2, mean2, m22);
    }
    if (lane == 0) {
      const float rstd = 1.0f / sqrtf(m2 / n + p.eps);
      fin_mean[g] = mean;
      fin_rstd[g] = rstd;
      if (p.stats != nullptr && tile == 0) {
        float* d = p.stats + ((int64_t)img * t.G + cb * t.nb + g) * 2;
        d[0] = mean;
        d[1] = rstd;
      }
    }
  }
  __syncthreads();
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  if (r >= t.ty) return;
  const int lc = tx * VN;
  const int r0 = tile * t.rows, r1 = min(t.S, r0 + t.rows);
  const XT* base = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;
  NormOut<VN> o;
  o.init(p, c0, lc, fin_mean, fin_rstd);
  with_act(p.act, [&](auto act) {
    uint4 raw[U], ahead[U];
    auto fetch = [&](int row) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (row + i * t.ty < r1) ahead[i] = load_stream(base + (int64_t)(row + i * t.ty) * p.ldx);
    };
    fetch(r0 + r);
    for (int row = r0 + r; row < r1; row += U * t.ty) {
#pragma unroll
      for (int i = 0; i < U; ++i) raw[i] = ahead[i];
      fetch(row + U * t.ty);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        float v[VN];
        Vec<XT>::load_raw(raw[i], v);
        if (row + i * t.ty < r1) o.template put<decltype(act)::value>(p, img, row + i * t.ty, c0 + lc, v);
      }
    }
  });
}

// ------------------------------------------------------------------ gradients
// The sums run over d = x - mean: dz = dy act'(d a + beta), a = rstd gamma,
// s1 = sum dz, s2 = sum dz d = (sum dz xhat) / rstd.  With the group's m1, m2
//   dx = a dz + d p + q,  p = -rstd^2 m2,  q = -rstd m1,
// and with the constants of x itself (b = beta - mean a, q' = q - mean p), as the
// forward has them, dx = a dz + (x p + q').
template <int VN>
struct NormGrad {
  float mean[VN], a[VN], be[VN];
  __device__ __forceinline__ void init(const NormBwdArgs& p, int img, int c0, int lc) {
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int c = c0 + lc + i;
      const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + (int64_t)img * p.t.G + c / p.t.cpg);
      mean[i] = st.x;
      a[i] = st.y * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      be[i] = p.beta ? __ldg(p.beta + c) : 0.0f;
    }
  }
  template <int ACT, typename XT>
  __device__ __forceinline__ void sums(const uint4& xr, const uint4& gr, float (&s1)[VN], float (&s2)[VN]) const {
    float x[VN], g[VN];
    Vec<XT>::load_raw(xr, x);
    Vec<XT>::load_raw(gr, g);
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const float d = x[i] - mean[i], dz = g[i] * norm_act_slope<ACT>(fmaf(d, a[i], be[i]));
      s1[i] += dz;
      s2[i] = fmaf(dz, d, s2[i]);
    }
  }
};

template <int VN>
struct NormGradOut {
  float a[VN], b[VN], pp[VN], q[VN];
  // g1, g2: m1 and m2 of the block's groups
  __device__ __forceinline__ void init(const NormBwdArgs& p, int img, int c0, int lc, const float* g1,
                                       const float* g2) {
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int c = c0 + lc + i, g = (lc + i) / p.t.cpg;
      const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + (int64_t)img * p.t.G + c / p.t.cpg);
      a[i] = st.y * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      b[i] = fmaf(-st.x, a[i], p.beta ? __ldg(p.beta + c) : 0.0f);
      pp[i] = -st.y * st.y * g2[g];
      q[i] = -fmaf(st.x, pp[i], st.y * g1[g]);
    }
  }
  template <int ACT, typename XT>
  __device__ __forceinline__ void put(void* dx, int64_t at, const uint4& xr, const uint4& gr) const {
    float x[VN], g[VN], o[VN];
    Vec<XT>::load_raw(xr, x);
    Vec<XT>::load_raw(gr, g);
#pragma unroll
    for (int i = 0; i < VN; ++i)
      o[i] = fmaf(g[i] * norm_act_slope<ACT>(fmaf(x[i], a[i], b[i])), a[i], fmaf(x[i], pp[i], q[i]));
    store_vec<VN>(dx, at, VN == 8, o);
  }
};

// m1 and m2 of the block's groups from its channels' sums tot[2][W].
template <int NT>
__device__ __forceinline__ void grad_group_means(const NormBwdArgs& p, int img, int c0, int W, const float* tot,
                                                 float* g1, float* g2) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float inv = 1.0f / ((float)p.t.S * (float)p.t.cpg);
  for (int g = warp; g < p.t.nb; g += NT / 32) {
    float a = 0.0f, b = 0.0f;
    for (int k = lane; k < p.t.cpg; k += 32) {
      const int c = g * p.t.cpg + k;
      const float ga = p.gamma ? __ldg(p.gamma + c0 + c) : 1.0f;
      a = fmaf(ga, tot[c], a);
      b = fmaf(ga, tot[W + c], b);
    }
    a = warp_sum(a);
    b = warp_sum(b);
    // rstd turns the sum over d into the one over xhat
    if (lane == 0) {
      g1[g] = a * inv;
      g2[g] = b * inv * p.stats[((int64_t)img * p.t.G + c0 / p.t.cpg + g) * 2 + 1];
    }
  }
  __syncthreads();
}

// Slab of x and dy in the registers of a cluster; total[img] receives the
// image's sums for dgamma and dbeta.
template <typename XT, int NV>
__global__ void __launch_bounds__(kNormThreads, 1)
    group_norm_bwd_cluster_kernel(const NormBwdArgs p, int cs) {
  constexpr int VN = Vec<XT>::n;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = sm;                           // later the cluster's totals [2][W]
  float* ch = scratch + max(kNormThreads * VN, 2 * W);   // this CTA's totals [2][W]
  float* g1 = ch + 2 * W;
  float* g2 = g1 + t.nb;
  const int rank = blockIdx.x % cs, cb = blockIdx.x / cs, img = blockIdx.y;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = rank * t.rows, r1 = min(t.S, r0 + t.rows);
  const XT* xb = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;
  const XT* gb = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + c0 + lc;
  grid_dep_launch();
  uint4 xr[NV], gr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int row = r0 + r + i * t.ty;
    xr[i] = gr[i] = make_uint4(0u, 0u, 0u, 0u);
    if (active && row < r1) {
      xr[i] = load_stream(xb + (int64_t)row * p.ldx);
      gr[i] = load_stream(gb + (int64_t)row * p.lddy);
    }
  }
  float s1[VN], s2[VN];
#pragma unroll
  for (int i = 0; i < VN; ++i) s1[i] = s2[i] = 0.0f;
  if (active) {
    NormGrad<VN> k;
    k.init(p, img, c0, lc);
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (r0 + r + i * t.ty < r1) k.template sums<decltype(act)::value, XT>(xr[i], gr[i], s1, s2);
    });
  }
  reduce_channels<kNormThreads, VN>(s1, active, tx, r, t, scratch, ch);
  reduce_channels<kNormThreads, VN>(s2, active, tx, r, t, scratch, ch + W);
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  for (int c = threadIdx.x; c < 2 * W; c += kNormThreads) {
    float a = 0.0f;
    if (cs > 1) {
      for (int q = 0; q < cs; ++q) a += dsmem_f32(ch + c, q);
    } else {
      a = ch[c];
    }
    scratch[c] = a;
    if (rank == 0)
      p.total[(int64_t)img * 2 * t.C + (c < W ? c0 + c : t.C + c0 + c - W)] = a;
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();
  grad_group_means<kNormThreads>(p, img, c0, W, scratch, g1, g2);
  if (active) {
    NormGradOut<VN> o;
    o.init(p, img, c0, lc, g1, g2);
    with_act(p.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int row = r0 + r + i * t.ty;
        if (row < r1)
          o.template put<decltype(act)::value, XT>(
              p.dx, (int64_t)img * p.dxbs + (int64_t)row * p.lddx + c0 + lc, xr[i], gr[i]);
      }
    });
  }
  __syncwarp();
  if (cs > 1) cluster_wait();
}

// Two passes: the tiles' per-channel sums, the images' (group_norm_bwd_params_kernel),
// then dx.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) group_norm_bwd_sums_kernel(const NormBwdArgs p) {
  constexpr int VN = Vec<XT>::n, U = 4;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = sm;
  float* ch = scratch + max(NT * VN, 2 * W);
  grid_dep_launch();
  const int tile = blockIdx.x, cb = blockIdx.y, img = blockIdx.z;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = tile * t.rows, r1 = min(t.S, r0 + t.rows);
  const XT* xb = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;
  const XT* gb = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + c0 + lc;
  float s1[VN], s2[VN];
#pragma unroll
  for (int i = 0; i < VN; ++i) s1[i] = s2[i] = 0.0f;
  if (active) {
    uint4 xr[U], gr[U], xa[U], ga[U];
    auto fetch = [&](int row) {
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (row + i * t.ty < r1) {
          xa[i] = __ldg(reinterpret_cast<const uint4*>(xb + (int64_t)(row + i * t.ty) * p.ldx));
          ga[i] = __ldg(reinterpret_cast<const uint4*>(gb + (int64_t)(row + i * t.ty) * p.lddy));
        }
    };
    fetch(r0 + r);
    NormGrad<VN> k;
    k.init(p, img, c0, lc);
    with_act(p.act, [&](auto act) {
      for (int row = r0 + r; row < r1; row += U * t.ty) {
#pragma unroll
        for (int i = 0; i < U; ++i) { xr[i] = xa[i]; gr[i] = ga[i]; }
        fetch(row + U * t.ty);
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (row + i * t.ty < r1) k.template sums<decltype(act)::value, XT>(xr[i], gr[i], s1, s2);
      }
    });
  }
  reduce_channels<NT, VN>(s1, active, tx, r, t, scratch, ch);
  reduce_channels<NT, VN>(s2, active, tx, r, t, scratch, ch + W);
  float* d = p.part + ((int64_t)img * p.tiles + tile) * 2 * t.C + c0;
  for (int c = threadIdx.x; c < W; c += NT) {
    d[c] = ch[c];
    d[t.C + c] = ch[W + c];
  }
}

template <typename XT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) group_norm_bwd_apply_kernel(const NormBwdArgs p) {
  constexpr int VN = Vec<XT>::n, U = 2;
  extern __shared__ __align__(16) float sm[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* tot = sm;
  float* g1 = sm + 2 * W;
  float* g2 = g1 + t.nb;
  const int tile = gridDim.x - 1 - blockIdx.x, cb = gridDim.y - 1 - blockIdx.y,
            img = gridDim.z - 1 - blockIdx.z;
  const int c0 = cb * t.nb * t.cpg;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int lc = tx * VN;
  const int r0 = tile * t.rows, r1 = min(t.S, r0 + t.rows);
  const XT* xb = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + c0 + lc;
  const XT* gb = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + c0 + lc;
  grid_dep_wait();
  uint4 xr[U], gr[U], xa[U], ga[U];
  auto fetch = [&](int row) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (active && row + i * t.ty < r1) {
        xa[i] = load_stream(xb + (int64_t)(row + i * t.ty) * p.ldx);
        ga[i] = load_stream(gb + (int64_t)(row + i * t.ty) * p.lddy);
      }
  };
  fetch(r0 + r);
  for (int c = threadIdx.x; c < 2 * W; c += NT)
    tot[c] = p.total[(int64_t)img * 2 * t.C + (c < W ? c0 + c : t.C + c0 + c - W)];
  __syncthreads();
  grad_group_means<NT>(p, img, c0, W, tot, g1, g2);
  if (!active) return;
  NormGradOut<VN> o;
  o.init(p, img, c0, lc, g1, g2);
  with_act(p.act, [&](auto act) {
    for (int row = r0 + r; row < r1; row += U * t.ty) {
#pragma unroll
      for (int i = 0; i < U; ++i) { xr[i] = xa[i]; gr[i] = ga[i]; }
      fetch(row + U * t.ty);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (row + i * t.ty < r1)
          o.template put<decltype(act)::value, XT>(
              p.dx, (int64_t)img * p.dxbs + (int64_t)(row + i * t.ty) * p.lddx + c0 + lc, xr[i], gr[i]);
    }
  });
}

// dbeta and dgamma, and (two passes) each image's sums over its tiles.  A block
// has 32 channels; its warps share the tiles of an image and their sums are added in
// order, so every result repeats bit for bit.
constexpr int kParamWarps = 16;
__global__ void __launch_bounds__(32 * kParamWarps) group_norm_bwd_params_kernel(const NormBwdArgs p, int32_t B,
                                                                                 float* __restrict__ dgamma,
                                                                                 float* __restrict__ dbeta) {
  __shared__ float sh[2][kParamWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = p.t.C, c = blockIdx.x * 32 + lane;
  grid_dep_launch();
  grid_dep_wait();
  float sum1 = 0.0f, sum2 = 0.0f;                // this warp's images
  const float* stat = p.stats + (int64_t)(min(c, C - 1) / p.t.cpg) * 2 + 1;
  if (p.tiles > 0) {
    for (int b = 0; b < B; ++b) {
      float a1 = 0.0f, a2 = 0.0f;
      if (c < C) {
        const float* d = p.part + (int64_t)b * p.tiles * 2 * C + c;
#pragma unroll 4
        for (int k = warp; k < p.tiles; k += kParamWarps) {
          a1 += d[(int64_t)k * 2 * C];
          a2 += d[(int64_t)k * 2 * C + C];
        }
      }
      sh[0][warp][lane] = a1;
      sh[1][warp][lane] = a2;
      __syncthreads();
      if (warp < 2 && c < C) {
        float a = 0.0f;
#pragma unroll
        for (int k = 0; k < kParamWarps; ++k) a += sh[warp][k][lane];
        p.total[((int64_t)b * 2 + warp) * C + c] = a;
        sum1 += warp == 0 ? a : a * stat[(int64_t)b * p.t.G * 2];
      }
      __syncthreads();
    }
    if (warp < 2) sh[warp][0][lane] = sum1;
    __syncthreads();
    if (warp == 0 && c < C) {
      if (dbeta != nullptr) dbeta[c] = sh[0][0][lane];
      if (dgamma != nullptr) dgamma[c] = sh[1][0][lane];
    }
    return;
  }
  if (c < C) {
#pragma unroll 2
    for (int b = warp; b < B; b += kParamWarps) {
      sum1 += p.total[(int64_t)b * 2 * C + c];
      sum2 = fmaf(p.total[((int64_t)b * 2 + 1) * C + c], stat[(int64_t)b * p.t.G * 2], sum2);
    }
  }
  sh[0][warp][lane] = sum1;
  sh[1][warp][lane] = sum2;
  __syncthreads();
  if (warp < 2 && c < C) {
    float a = 0.0f;
#pragma unroll
    for (int k = 0; k < kParamWarps; ++k) a += sh[warp][k][lane];
    float* out = warp == 0 ? dbeta : dgamma;
    if (out != nullptr) out[c] = a;
  }
}

}  // namespace sq
