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
// An element is read and written once for about ten instructions and, with an activation, one
// and a half special-function ones: large maps are bound by memory, with the issue
// slots half busy; maps of some MB by the latency of a wave (loads, two reductions, stores).
// Where the slab of one image and one block of groups fits the shared memory of a
// cluster of CTAs, it is read once, the cluster exchanges the group's sums
// through distributed shared memory and writes the result from the slab (one
// launch, no workspace).  Larger maps take two passes, the second reading what
// the first left in L2.  Every sum has a fixed order: results repeat bit for bit.
//
// Data moves with 16-byte cp.async copies whose words only the copying thread reads:
// no barrier, no registers held, loops that stay small (the slab in registers, fully
// unrolled, spent most of its time fetching instructions: 18.0 us instead of 10.0 on
// 3 x 1023 x 1152 fp32).
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>

#include "common.cuh"
#include "ptx.cuh"
#include "quant_kernels.cuh"

namespace sq {

constexpr int kNormThreads = 256;     // 512 in two passes over groups wider than 256 vectors
constexpr int kNormThreadsMax = 512;
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
  float2* part;                  // two passes: [B][G][tiles] mean, M2 of each tile
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
  float* dgamma;                 // [C] or null
  float* dbeta;
  int32_t B;
  NormTile t;
  int32_t tiles;                 // two passes: per image
  int32_t act;
};

// ------------------------------------------------------------ vector access
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// A 16-byte vector as pairs of fp32 values.
template <typename XT>
__device__ __forceinline__ void load_pairs(const uint4& u, uint64_t (&v)[Vec<XT>::n / 2]) {
  if constexpr (Vec<XT>::n == 8) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  } else {
    v[0] = f2_pack(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = f2_pack(__uint_as_float(u.z), __uint_as_float(u.w));
  }
}
template <int VN>
__device__ __forceinline__ void unpack_pairs(const uint64_t (&v)[VN / 2], float (&o)[VN]) {
#pragma unroll
  for (int i = 0; i < VN / 2; ++i) f2_unpack(v[i], o[2 * i], o[2 * i + 1]);
}
// Waits until at most N groups of this thread's copies are in flight.
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
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
// Pairs of fp32 values in 64 bits (one packed instruction for both).
__device__ __forceinline__ uint64_t f2_both(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// min and max that give NaN where an operand is NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// For both values w = min(|z|, 14.5) (beyond that all terms are below the fp32 range),
// e = exp(-w^2 / 2) and c = -erfc(w / sqrt 2) / 2 = e t P(t) with t = 1 / (1 + w / 3.75): P is the
// polynomial of degree 8 of least relative error (1.5e-8) for c / (e t) over that range, fitted
// by iteratively weighted least squares; its coefficients are nearly all of one sign, so
// little cancels.  c is off by 2^-20 + z^2 2^-23 of itself at most (the exponent's roundings).
__device__ __forceinline__ void erfc_pair(uint64_t z2, uint64_t& w2, uint64_t& e2, uint64_t& c2) {
  float a, b;
  f2_unpack(z2, a, b);
  w2 = f2_pack(min_nan(fabsf(a), 14.5f), min_nan(fabsf(b), 14.5f));
  f2_unpack(f2_mul(f2_mul(w2, w2), f2_both(-0.5f * kLog2e)), a, b);
  e2 = f2_pack(ex2_ftz(a), ex2_ftz(b));
  f2_unpack(f2_fma(w2, f2_both(0.26666667f), f2_both(1.0f)), a, b);
  const uint64_t t = f2_pack(rcp_ftz(a), rcp_ftz(b));
  uint64_t p = f2_both(-0.030272834f);
  p = f2_fma(p, t, f2_both(0.138486668f));
  p = f2_fma(p, t, f2_both(-0.20164223f));
  p = f2_fma(p, t, f2_both(0.100022197f));
  p = f2_fma(p, t, f2_both(-0.127300635f));
  p = f2_fma(p, t, f2_both(-0.0645551905f));
  p = f2_fma(p, t, f2_both(-0.102310821f));
  p = f2_fma(p, t, f2_both(-0.106026821f));
  p = f2_fma(p, t, f2_both(-0.106400318f));
  c2 = f2_mul(f2_mul(p, t), e2);
}

// 1 / (1 + exp(-z)) of both values with one reciprocal, r = 1 / (a b): the special
// function unit (four lanes a clock) bounds these loops.  a and b are the denominators
// times 2^-63, so a b and r stay in the normal range down to z = -87.3; beyond, the
// exponential is held just above 2^126, whose reciprocal counts as zero.
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z2) {
  constexpr float scale = 1.0842022e-19f;      // 2^-63
  float a, b;
  f2_unpack(f2_mul(z2, f2_both(-kLog2e)), a, b);
  const uint64_t d = f2_fma(f2_pack(ex2_ftz(fminf(a, 126.001f)), ex2_ftz(fminf(b, 126.001f))), f2_both(scale),
                            f2_both(scale));
  f2_unpack(d, a, b);
  const float r = rcp_ftz(a * b);
  return f2_mul_ftz(f2_pack(r * b, r * a), f2_both(scale));
}

// act(z) and act'(z), with the hardware's exponential and reciprocal (relative error about
// 2^-22 each).  SiLU is off by (|z| + 4) 2^-22 of itself at most, GELU by 2^-20 + z^2 2^-23: the
// rounding to bf16 moves about one value in a thousand to its neighbour.
template <int ACT>
__device__ __forceinline__ uint64_t norm_act(uint64_t z2) {
  float z0, z1;
  if constexpr (ACT == ACT_SILU) {               // z / (1 + exp(-z))
    return f2_mul(z2, sigmoid2(z2));
  } else if constexpr (ACT == ACT_GELU) {        // max(z, 0) - |z| erfc(|z| / sqrt 2) / 2
    uint64_t w, e, c;
    erfc_pair(z2, w, e, c);
    f2_unpack(z2, z0, z1);
    return f2_fma(w, c, f2_pack(max_nan(z0, 0.0f), max_nan(z1, 0.0f)));
  } else {
    return z2;
  }
}
template <int ACT>
__device__ __forceinline__ uint64_t norm_act_slope(uint64_t z2) {
  if constexpr (ACT == ACT_SILU) {               // p (1 + z (1 - p))
    const uint64_t one = f2_both(1.0f), p = sigmoid2(z2);
    return f2_mul(p, f2_fma(z2, f2_fma(p, f2_both(-1.0f), one), one));
  } else if constexpr (ACT == ACT_GELU) {        // the normal distribution plus z times its density
    uint64_t w, e, c;
    erfc_pair(z2, w, e, c);
    float z0, z1, c0, c1, w0, w1;
    f2_unpack(z2, z0, z1);
    f2_unpack(c, c0, c1);
    f2_unpack(w, w0, w1);
    return f2_fma(f2_mul(f2_pack(copysignf(w0, z0), copysignf(w1, z1)), f2_both(0.39894228f)), e,
                  f2_pack(z0 >= 0.0f ? 1.0f + c0 : -c0, z1 >= 0.0f ? 1.0f + c1 : -c1));
  } else {
    return f2_both(1.0f);
  }
}
// The activation is a launch argument: one uniform branch outside the loops.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else f(std::integral_constant<int, ACT_NONE>{});
}
// So is what the forward writes.
constexpr int OUT_BF16 = 0, OUT_F32 = 1, OUT_CODES = 2, OUT_CODES_BF16 = 3;
template <typename F>
__device__ __forceinline__ void with_act_out(const NormArgs& p, F&& f) {
  with_act(p.act, [&](auto act) {
    if (p.q_pos == nullptr) {
      if (p.y_bf16) f(act, std::integral_constant<int, OUT_BF16>{});
      else f(act, std::integral_constant<int, OUT_F32>{});
    } else {
      if (p.y == nullptr) f(act, std::integral_constant<int, OUT_CODES>{});
      else f(act, std::integral_constant<int, OUT_CODES_BF16>{});
    }
  });
}

// --------------------------------------------------------------- reductions
// Per-thread, per-channel values v[m][VN] (M arrays) of all rows of threads ->
// per-channel totals ch[m * W + 0 .. W), W = vx * VN, in shared memory.  `scratch` holds
// NT * VN * M floats.  Begins and ends with every thread past a barrier.
template <int NT, int VN, int M>
__device__ __forceinline__ void reduce_channels(const float (&v)[M][VN], bool active, int tx, int r,
                                                const NormTile& t, float* scratch, float* ch) {
  const int W = t.vx * VN, W2 = M * W;
  __syncthreads();
  if (active) {
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < VN; i += 4)
        *reinterpret_cast<float4*>(scratch + r * W2 + m * W + tx * VN + i) =
            make_float4(v[m][i], v[m][i + 1], v[m][i + 2], v[m][i + 3]);
  }
  __syncthreads();
  const int nseg = W2 < NT ? NT / W2 : 1;
  if (nseg == 1) {
    for (int c = threadIdx.x; c < W2; c += NT) {
      float s = 0.0f;
#pragma unroll 4
      for (int k = 0; k < t.ty; ++k) s += scratch[k * W2 + c];
      ch[c] = s;
    }
    __syncthreads();
    return;
  }
  const int c = threadIdx.x % W2, sg = threadIdx.x / W2;
  float s = 0.0f;
  if (sg < nseg) {
#pragma unroll 4
    for (int k = sg; k < t.ty; k += nseg) s += scratch[k * W2 + c];
  }
  __syncthreads();
  if (sg < nseg) scratch[sg * W2 + c] = s;
  __syncthreads();
  if (threadIdx.x < W2) {
    float a = 0.0f;
    for (int k = 0; k < nseg; ++k) a += scratch[k * W2 + threadIdx.x];
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
  if (t.cpg > VN) {
    // a vector meets at most two groups: its first's share and the next one's, in two
    // columns of ty values; a group's are those of the vectors that begin in it, and the
    // second share of the one before them
    const int lc = tx * VN, split = (lc / t.cpg + 1) * t.cpg - lc;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      if (i < split) lo += v[i];
      else hi += v[i];
    }
    __syncthreads();
    if (active) {
      scratch[tx * t.ty + r] = lo;
      scratch[NT + tx * t.ty + r] = hi;
    }
    __syncthreads();
    for (int g = warp; g < t.nb; g += NT / 32) {
      const int first = (g * t.cpg + VN - 1) / VN, last = ((g + 1) * t.cpg - 1) / VN;
      float a = 0.0f;
      for (int k = first * t.ty + lane; k < (last + 1) * t.ty; k += 32) a += scratch[k];
      if (first * VN != g * t.cpg)
        for (int k = lane; k < t.ty; k += 32) a += scratch[NT + (first - 1) * t.ty + k];
      a = warp_sum(a);
      if (lane == 0) grp[g] = a;
    }
    __syncthreads();
    return;
  }
  float one[1][VN];
#pragma unroll
  for (int i = 0; i < VN; ++i) one[0][i] = v[i];
  reduce_channels<NT, VN, 1>(one, active, tx, r, t, scratch, ch);
  for (int g = warp; g < t.nb; g += (NT / 32)) {
    float a = 0.0f;
    for (int k = lane; k < t.cpg; k += 32) a += ch[g * t.cpg + k];
    a = warp_sum(a);
    if (lane == 0) grp[g] = a;
  }
  __syncthreads();
}

__device__ __forceinline__ float dsmem_f32(const float* p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), rank)) : "memory");
  return v;
}
// The values at p of the cluster's CTAs 0 .. cs - 1 (cs <= 8), all reads in flight together.
__device__ __forceinline__ void dsmem_gather(const float* p, int cs, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    v[k] = 0.0f;
    if (k < cs) v[k] = dsmem_f32(p, k);
  }
}
// Their sum, in rank order.
__device__ __forceinline__ float dsmem_sum(const float* p, int cs) {
  float v[8], a = 0.0f;
  dsmem_gather(p, cs, v);
#pragma unroll
  for (int k = 0; k < 8; ++k) a += v[k];
  return a;
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
  uint64_t a[VN / 2], b[VN / 2];
  float rp, rn;
  uint8_t* y;              // this thread's next vector, and the bytes from one to the next
  int64_t y_step;
  int64_t q_at, q_step;
  // row, ty: the thread's first position and the distance of its positions
  __device__ __forceinline__ void init(const NormArgs& p, int img, int row, int ty, int c0, int lc,
                                       const float* mean_g, const float* rstd_g) {
    float av[VN], bv[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int g = (lc + i) / p.t.cpg, c = c0 + lc + i;
      av[i] = rstd_g[g] * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      bv[i] = fmaf(-mean_g[g], av[i], p.beta ? __ldg(p.beta + c) : 0.0f);
    }
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      a[i] = f2_pack(av[2 * i], av[2 * i + 1]);
      b[i] = f2_pack(bv[2 * i], bv[2 * i + 1]);
    }
    const int es = p.y_bf16 ? 2 : 4;
    y = static_cast<uint8_t*>(p.y) + ((int64_t)img * p.ybs + (int64_t)row * p.ldy + c0 + lc) * es;
    y_step = (int64_t)ty * p.ldy * es;
    rp = rn = 0.0f;
    q_at = q_step = 0;
    if (p.q_pos != nullptr) {
      const int j = p.kseg.segment_of(c0 + lc);   // bounds are multiples of 128
      const float sp = p.s_pos[j], sn = p.s_neg[j];
      rp = sp > 0.0f ? __frcp_rn(sp) : 0.0f;
      rn = sn > 0.0f ? __frcp_rn(sn) : 0.0f;
      q_at = ((int64_t)img * p.t.S + row) * p.ldq + c0 + lc;
      q_step = (int64_t)ty * p.ldq;
    }
  }
  template <int ACT, int OUT, typename XT>
  __device__ __forceinline__ void put(const NormArgs& p, const uint4& raw) {
    uint64_t x[VN / 2];
    load_pairs<XT>(raw, x);
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) x[i] = norm_act<ACT>(f2_fma(x[i], a[i], b[i]));
    float v[VN];
    unpack_pairs<VN>(x, v);
    if constexpr (OUT == OUT_CODES || OUT == OUT_CODES_BF16) {
      // The codes are those of the bf16 values that y holds, by the quantizer's own functions:
      // the same codes for values that are not finite, too.
      uint32_t w[VN / 2], qp[VN / 4], qn[VN / 4];
#pragma unroll
      for (int i = 0; i < VN / 2; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < VN / 4; ++i) {
        uint32_t a[4], b[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t h = w[2 * i + k / 2];
          const float x1 = __uint_as_float(k & 1 ? h & 0xFFFF0000u : h << 16);
          a[k] = code_pos(x1, rp);
          b[k] = code_neg(x1, rn);
        }
        qp[i] = pack4_low(a[0], a[1], a[2], a[3]);
        qn[i] = pack4_low(b[0], b[1], b[2], b[3]);
      }
      if constexpr (VN == 8) {
        *reinterpret_cast<uint2*>(p.q_pos + q_at) = make_uint2(qp[0], qp[1]);
        *reinterpret_cast<uint2*>(p.q_neg + q_at) = make_uint2(qn[0], qn[1]);
      } else {
        *reinterpret_cast<uint32_t*>(p.q_pos + q_at) = qp[0];
        *reinterpret_cast<uint32_t*>(p.q_neg + q_at) = qn[0];
      }
      q_at += q_step;
      if constexpr (OUT == OUT_CODES_BF16) {
        if constexpr (VN == 8) *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
        y += y_step;
      }
    } else {
      store_vec<VN>(y, 0, OUT != OUT_F32, v);
      y += y_step;
    }
  }
};

// Shared memory of the norm kernels behind the slab, in floats: scratch (reductions,
// then the cluster's totals), two totals per channel and four values per group.
__host__ __device__ inline int norm_scratch_floats(int threads, int vn) { return 2 * threads * vn; }
__host__ __device__ inline int norm_smem_floats(int threads, int vx, int vn, int nb) {
  return norm_scratch_floats(threads, vn) + 2 * vx * vn + 4 * nb;
}
constexpr int kNormBatches = 4;   // groups of copies that a slab's sums wait for one after the other

// Waits for batch b of kNormBatches.
__device__ __forceinline__ void slab_wait(int b) {
  if (b == 0) cp_async_wait<3>();
  else if (b == 1) cp_async_wait<2>();
  else if (b == 2) cp_async_wait<1>();
  else cp_async_wait<0>();
}

// Running mean and squared deviations of a thread's rows, per channel: four rows at a
// time (their mean, the deviations from it, merged by the formula of Chan, Golub and
// LeVeque, "Updating Formulae and a Pairwise Algorithm for Computing Sample Variances"),
// so nothing is lost to a large mean or to rows far off the rest.
template <int VN>
struct RowStats {
  uint64_t mean[VN / 2], m2[VN / 2];
  float n;
  __device__ __forceinline__ void clear() {
    n = 0.0f;
#pragma unroll
    for (int k = 0; k < VN / 2; ++k) mean[k] = m2[k] = 0;
  }
  template <int U>
  __device__ __forceinline__ void add(const uint64_t (&v)[U][VN / 2]) {
    const float f = __fdividef((float)U, n + (float)U);   // the new rows' share of all
    const uint64_t inv = f2_both(-1.0f / (float)U), f2 = f2_both(-f), nf = f2_both(n * f);
#pragma unroll
    for (int c = 0; c < VN / 2; ++c) {
      uint64_t sum = v[0][c], q = 0;
#pragma unroll
      for (int i = 1; i < U; ++i) sum = f2_add(sum, v[i][c]);
      sum = f2_mul(sum, inv);                       // minus the rows' mean
      if (U > 1) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const uint64_t d = f2_add(v[i][c], sum);
          q = f2_fma(d, d, q);
        }
      }
      const uint64_t d = f2_add(sum, mean[c]);      // running mean minus the rows' mean
      mean[c] = f2_fma(d, f2, mean[c]);
      m2[c] = f2_add(m2[c], f2_fma(f2_mul(d, d), nf, q));
    }
    n += (float)U;
  }
};

// ------------------------------------------------------ forward, slab on chip
// Cluster of `cs` CTAs per (image, channel block); CTA rank k holds positions
// k*rows .. of it, nv 16-byte vectors per thread.  The statistics are taken as the rows
// arrive.  3 x 1023 x 1152 fp32 (28 MB): 9.2 us, 3.1 TB/s; 2 x 64 x 1280 bf16: 5.0 us, of which
// the launch, one load, two reductions and a store are all.  (512 threads per CTA, for slabs
// that have an SM to themselves, gained nothing: 11.9 us, not 11.2, on 8 x 1024 x 640 bf16.)
template <typename XT>
__global__ void __launch_bounds__(kNormThreads, 3) group_norm_cluster_kernel(const NormArgs p, int cs, int nv) {
  constexpr int VN = Vec<XT>::n, NT = kNormThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = reinterpret_cast<float*>(smem + (size_t)nv * NT * 16);
  float* ch = scratch + norm_scratch_floats(NT, VN);
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
  const XT* base = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  const int64_t step = (int64_t)t.ty * p.ldx;
  // this thread's vectors: rows r, r + ty, .. of the CTA's
  const int mine = active && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  const int batch = (nv + kNormBatches - 1) / kNormBatches;
  const uint32_t slab = smem_u32(smem) + threadIdx.x * 16;
  grid_dep_wait();
  for (int b = 0; b < kNormBatches; ++b) {
    for (int i = b * batch; i < min(mine, (b + 1) * batch); ++i) {
      cp_async16(slab + i * NT * 16, base, 16);
      base += step;
    }
    cp_async_commit();
  }
  RowStats<VN> st;
  st.clear();
  for (int b = 0; b < kNormBatches; ++b) {
    slab_wait(b);
    int i = b * batch;
    const int end = min(mine, (b + 1) * batch);
#pragma unroll 1
    for (; i + 4 <= end; i += 4) {
      uint64_t v[4][VN / 2];
#pragma unroll
      for (int j = 0; j < 4; ++j) load_pairs<XT>(lds128(slab + (i + j) * NT * 16), v[j]);
      st.add(v);
    }
#pragma unroll 1
    for (; i < end; ++i) {
      uint64_t v[1][VN / 2];
      load_pairs<XT>(lds128(slab + i * NT * 16), v[0]);
      st.add(v);
    }
  }
  // the CTA's means and deviations: of the threads' means, then their own and those from
  // the CTA's mean
  float mv[VN], qv[VN], s[VN];
  unpack_pairs<VN>(st.mean, mv);
  unpack_pairs<VN>(st.m2, qv);
#pragma unroll
  for (int k = 0; k < VN; ++k) s[k] = st.n * mv[k];
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, pub_mean);
  const float n_loc = (float)n_rows * (float)t.cpg;
  for (int g = threadIdx.x; g < t.nb; g += NT) pub_mean[g] = n_loc > 0.0f ? pub_mean[g] / n_loc : 0.0f;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < VN; ++k) {
    const float d = active ? mv[k] - pub_mean[(lc + k) / t.cpg] : 0.0f;
    s[k] = fmaf(st.n * d, d, qv[k]);
  }
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, pub_m2);
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  for (int g = threadIdx.x; g < t.nb; g += NT) {
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    if (cs > 1) {
      float mk[8], qk[8];
      dsmem_gather(pub_mean + g, cs, mk);
      dsmem_gather(pub_m2 + g, cs, qk);
      const float full = (float)t.rows * (float)t.cpg;
      n = (float)t.S * (float)t.cpg;
      const float last = n - full * (float)(cs - 1);
#pragma unroll
      for (int k = 0; k < 8; ++k) mean = fmaf(mk[k], k < cs - 1 ? full : k == cs - 1 ? last : 0.0f, mean);
      mean /= n;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float d = mk[k] - mean;
        m2 += fmaf(d * d, k < cs - 1 ? full : k == cs - 1 ? last : 0.0f, qk[k]);
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
  if (mine > 0) {
    NormOut<VN> o;
    o.init(p, img, r0 + r, t.ty, c0, lc, fin_mean, fin_rstd);
    with_act_out(p, [&](auto act, auto out) {
#pragma unroll 2
      for (int i = 0; i < mine; ++i)
        o.template put<decltype(act)::value, decltype(out)::value, XT>(p, lds128(slab + i * NT * 16));
    });
  }
  __syncwarp();
  if (cs > 1) cluster_wait();     // the peers have read this CTA's
}

// ------------------------------------------------------------------ two passes
// A thread's rows of a tile, streamed through a ring of its own in shared memory:
// U rows per step, kNormRing steps in flight.  N tensors of the same shape.
constexpr int kNormRing = 4;
template <typename XT, int NT, int U, int N>
struct NormStream {
  const XT* at[N];
  int64_t step[N];
  uint32_t ring;
  int left;              // rows not yet asked for
  __device__ __forceinline__ void begin(uint8_t* smem, int rows) {
    ring = smem_u32(smem) + threadIdx.x * 16;
    left = rows;
#pragma unroll
    for (int k = 0; k < kNormRing - 1; ++k) issue(k);
  }
  __device__ __forceinline__ uint32_t step_at(int k) const { return ring + (k & (kNormRing - 1)) * (U * N * NT * 16); }
  // the vector of tensor n and row i of a step at `base`
  __device__ __forceinline__ static uint4 get(uint32_t base, int i, int n) {
    return lds128(base + (i * N + n) * (NT * 16));
  }
  __device__ __forceinline__ void issue(int k) {
    const uint32_t base = step_at(k);
    if (left >= U) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          cp_async16(base + (i * N + n) * (NT * 16), at[n], 16);
          at[n] += step[n];
        }
    } else {
#pragma unroll 1
      for (int i = 0; i < left; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) {
          cp_async16(base + (i * N + n) * (NT * 16), at[n], 16);
          at[n] += step[n];
        }
    }
    left -= U;
    cp_async_commit();
  }
  // where step k has landed; the one behind the ring is on its way
  __device__ __forceinline__ uint32_t wait(int k) {
    cp_async_wait<kNormRing - 2>();
    issue(k + kNormRing - 1);
    return step_at(k);
  }
};
__host__ __device__ inline int norm_ring_bytes(int threads, int u, int tensors) {
  return kNormRing * u * tensors * threads * 16;
}
constexpr int kNormU1 = 4, kNormU2 = 2;    // rows per step: one tensor, two

// Pass 1: one CTA per (tile of positions, channel block, image) writes mean and
// M2 of each of its groups.  A thread takes a few rows at a time: their mean
// and squared deviations per channel, merged into its running ones.
// Both passes over 2 x 65536 x 256 bf16 (67 MB in, 67 MB out): 43.0 us.  Back to back the second
// reads 29 of its 67 MB from DRAM and finds the rest in L2, so a call moves 161 MB, 24.6 us at
// the copy rate (the bytes once: 20.5 us); the rest is the kernels' own beginnings and ends and
// the issue slots, half busy.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 1) group_norm_stats_kernel(const NormArgs p) {
  constexpr int VN = Vec<XT>::n, U = kNormU1;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = reinterpret_cast<float*>(smem + norm_ring_bytes(NT, U, 1));
  float* ch = scratch + norm_scratch_floats(NT, VN);
  float* g_mean = ch + 2 * W;
  float* g_m2 = g_mean + t.nb;
  const int tile = blockIdx.x, cb = blockIdx.y, img = blockIdx.z;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = tile * t.rows, n_rows = min(t.S, r0 + t.rows) - r0;
  const int mine = active && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  NormStream<XT, NT, U, 1> in;
  in.at[0] = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  in.step[0] = (int64_t)t.ty * p.ldx;
  grid_dep_wait();
  in.begin(smem, mine);
  RowStats<VN> st;
  st.clear();
  int k = 0;
  for (; (k + 1) * U <= mine; ++k) {
    const uint32_t at = in.wait(k);
    uint64_t v[U][VN / 2];
#pragma unroll
    for (int i = 0; i < U; ++i) load_pairs<XT>(in.get(at, i, 0), v[i]);
    st.add(v);
  }
  if (k * U < mine) {
    const uint32_t at = in.wait(k);
#pragma unroll 1
    for (int i = 0; k * U + i < mine; ++i) {
      uint64_t v[1][VN / 2];
      load_pairs<XT>(in.get(at, i, 0), v[0]);
      st.add(v);
    }
  }
  cp_async_wait<0>();
  float mv[VN], qv[VN], s[VN];
  unpack_pairs<VN>(st.mean, mv);
  unpack_pairs<VN>(st.m2, qv);
  const float n = st.n;
#pragma unroll
  for (int k = 0; k < VN; ++k) s[k] = n * mv[k];
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, g_mean);
  const float n_tile = (float)n_rows * (float)t.cpg;
  for (int g = threadIdx.x; g < t.nb; g += NT) g_mean[g] /= n_tile;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < VN; ++k) {
    const float d = active ? mv[k] - g_mean[(lc + k) / t.cpg] : 0.0f;
    s[k] = fmaf(n * d, d, qv[k]);
  }
  reduce_groups<NT, VN>(s, active, tx, r, t, scratch, ch, g_m2);
  for (int g = threadIdx.x; g < t.nb; g += NT)
    p.part[((int64_t)img * t.G + cb * t.nb + g) * p.tiles + tile] = make_float2(g_mean[g], g_m2[g]);
}

// Pass 2: the same tiles in the opposite order (the last ones read are the
// likeliest in L2); each CTA merges its groups' tiles first, a warp per group.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, NT == 256 ? 3 : 1) group_norm_apply_kernel(const NormArgs p) {
  constexpr int VN = Vec<XT>::n, U = kNormU1;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  float* fin_mean = reinterpret_cast<float*>(smem + norm_ring_bytes(NT, U, 1));
  float* fin_rstd = fin_mean + t.nb;
  const int tile = gridDim.x - 1 - blockIdx.x, cb = gridDim.y - 1 - blockIdx.y,
            img = gridDim.z - 1 - blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = cb * t.nb * t.cpg;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const int lc = tx * VN;
  const int r0 = tile * t.rows, n_rows = min(t.S, r0 + t.rows) - r0;
  const int mine = r < t.ty && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  grid_dep_wait();
  NormStream<XT, NT, U, 1> in;
  in.at[0] = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  in.step[0] = (int64_t)t.ty * p.ldx;
  in.begin(smem, mine);
  // mean and M2 of the whole image from the tiles' (all but the last have t.rows positions)
  const float n_tile = (float)t.rows * (float)t.cpg;
  const float n_last = (float)(t.S - (p.tiles - 1) * t.rows) * (float)t.cpg;
  const float n_all = (float)t.S * (float)t.cpg;
  for (int g = warp; g < t.nb; g += NT / 32) {
    const float2* d = p.part + ((int64_t)img * t.G + cb * t.nb + g) * p.tiles;
    float mean = 0.0f, m2 = 0.0f;
#pragma unroll 4
    for (int k = lane; k < p.tiles; k += 32)
      mean = fmaf(d[k].x, k == p.tiles - 1 ? n_last : n_tile, mean);
    mean = warp_sum(mean) / n_all;
#pragma unroll 4
    for (int k = lane; k < p.tiles; k += 32) {
      const float2 v = d[k];
      const float e = v.x - mean;
      m2 += fmaf(e * e, k == p.tiles - 1 ? n_last : n_tile, v.y);
    }
    m2 = warp_sum(m2);
    if (lane == 0) {
      const float rstd = 1.0f / sqrtf(m2 / n_all + p.eps);
      fin_mean[g] = mean;
      fin_rstd[g] = rstd;
      if (p.stats != nullptr && tile == 0) {
        float* st = p.stats + ((int64_t)img * t.G + cb * t.nb + g) * 2;
        st[0] = mean;
        st[1] = rstd;
      }
    }
  }
  __syncthreads();
  if (mine > 0) {
    NormOut<VN> o;
    o.init(p, img, r0 + r, t.ty, c0, lc, fin_mean, fin_rstd);
    with_act_out(p, [&](auto act, auto out) {
      constexpr int A = decltype(act)::value, O = decltype(out)::value;
      int k = 0;
      for (; (k + 1) * U <= mine; ++k) {
        const uint32_t at = in.wait(k);
#pragma unroll
        for (int i = 0; i < U; ++i) o.template put<A, O, XT>(p, in.get(at, i, 0));
      }
      if (k * U < mine) {
        const uint32_t at = in.wait(k);
#pragma unroll 1
        for (int i = 0; k * U + i < mine; ++i) o.template put<A, O, XT>(p, in.get(at, i, 0));
      }
    });
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ gradients
// The sums run over d = x - mean: dz = dy act'(d a + beta), a = rstd gamma,
// s1 = sum dz, s2 = sum dz d = (sum dz xhat) / rstd.  With the group's m1, m2
//   dx = a dz + d p + q,  p = -rstd^2 m2,  q = -rstd m1,
// and with the constants of x itself (b = beta - mean a, q' = q - mean p), as the
// forward has them, dx = a dz + (x p + q').
template <int VN>
struct NormGrad {
  uint64_t mean[VN / 2], a[VN / 2], be[VN / 2];   // mean: its negative
  __device__ __forceinline__ void init(const NormBwdArgs& p, int img, int c0, int lc) {
    float m[VN], av[VN], bv[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int c = c0 + lc + i;
      const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + (int64_t)img * p.t.G + c / p.t.cpg);
      m[i] = -st.x;
      av[i] = st.y * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      bv[i] = p.beta ? __ldg(p.beta + c) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      mean[i] = f2_pack(m[2 * i], m[2 * i + 1]);
      a[i] = f2_pack(av[2 * i], av[2 * i + 1]);
      be[i] = f2_pack(bv[2 * i], bv[2 * i + 1]);
    }
  }
  template <int ACT, typename XT>
  __device__ __forceinline__ void sums(const uint4& xr, const uint4& gr, uint64_t (&s1)[VN / 2],
                                       uint64_t (&s2)[VN / 2]) const {
    uint64_t x[VN / 2], g[VN / 2];
    load_pairs<XT>(xr, x);
    load_pairs<XT>(gr, g);
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      const uint64_t d = f2_add(x[i], mean[i]);
      uint64_t dz = g[i];
      if constexpr (ACT != ACT_NONE) dz = f2_mul(dz, norm_act_slope<ACT>(f2_fma(d, a[i], be[i])));
      s1[i] = f2_add(s1[i], dz);
      s2[i] = f2_fma(dz, d, s2[i]);
    }
  }
};

template <int VN>
struct NormGradOut {
  uint64_t a[VN / 2], b[VN / 2], pp[VN / 2], q[VN / 2];
  uint8_t* dx;             // this thread's next vector, and the bytes from one to the next
  int64_t step;
  // g1, g2: m1 and m2 of the block's groups
  __device__ __forceinline__ void init(const NormBwdArgs& p, int img, int row, int ty, int c0, int lc,
                                       const float* g1, const float* g2) {
    constexpr int ES = 16 / VN;
    float av[VN], bv[VN], pv[VN], qv[VN];
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      const int c = c0 + lc + i, g = (lc + i) / p.t.cpg;
      const float2 st = __ldg(reinterpret_cast<const float2*>(p.stats) + (int64_t)img * p.t.G + c / p.t.cpg);
      av[i] = st.y * (p.gamma ? __ldg(p.gamma + c) : 1.0f);
      bv[i] = fmaf(-st.x, av[i], p.beta ? __ldg(p.beta + c) : 0.0f);
      pv[i] = -st.y * st.y * g2[g];
      qv[i] = -fmaf(st.x, pv[i], st.y * g1[g]);
    }
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      a[i] = f2_pack(av[2 * i], av[2 * i + 1]);
      b[i] = f2_pack(bv[2 * i], bv[2 * i + 1]);
      pp[i] = f2_pack(pv[2 * i], pv[2 * i + 1]);
      q[i] = f2_pack(qv[2 * i], qv[2 * i + 1]);
    }
    dx = static_cast<uint8_t*>(p.dx) + ((int64_t)img * p.dxbs + (int64_t)row * p.lddx + c0 + lc) * ES;
    step = (int64_t)ty * p.lddx * ES;
  }
  template <int ACT, typename XT>
  __device__ __forceinline__ void put(const uint4& xr, const uint4& gr) {
    uint64_t x[VN / 2], g[VN / 2];
    load_pairs<XT>(xr, x);
    load_pairs<XT>(gr, g);
#pragma unroll
    for (int i = 0; i < VN / 2; ++i) {
      uint64_t dz = g[i];
      if constexpr (ACT != ACT_NONE) dz = f2_mul(dz, norm_act_slope<ACT>(f2_fma(x[i], a[i], b[i])));
      x[i] = f2_fma(dz, a[i], f2_fma(x[i], pp[i], q[i]));
    }
    float o[VN];
    unpack_pairs<VN>(x, o);
    store_vec<VN>(dx, 0, VN == 8, o);
    dx += step;
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

// Slabs of x and dy in the shared memory of a cluster; total[img] receives the
// image's sums for dgamma and dbeta, which a second launch adds (a cluster that holds all
// images and adds them itself was slower: 12.4 us, not 11.2, on 2 x 1024 x 640 bf16).
// 8 x 1024 x 640 bf16 (31 MB): 16.7 us, 1.9 TB/s: one wave of CTAs, half its issue slots
// busy, whose loads, reductions and stores follow one another.
template <typename XT>
__global__ void __launch_bounds__(kNormThreads, 2)
    group_norm_bwd_cluster_kernel(const NormBwdArgs p, int cs, int nv) {
  constexpr int VN = Vec<XT>::n, NT = kNormThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = reinterpret_cast<float*>(smem + (size_t)nv * NT * 32);   // later the cluster's totals [2][W]
  float* ch = scratch + norm_scratch_floats(NT, VN);                               // this CTA's totals [2][W]
  float* g1 = ch + 2 * W;
  float* g2 = g1 + t.nb;
  const int rank = blockIdx.x % cs, cb = blockIdx.x / cs, img = blockIdx.y;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = rank * t.rows, n_rows = max(0, min(t.S, r0 + t.rows) - r0);
  const int mine = active && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  const XT* xb = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  const XT* gb = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + (int64_t)(r0 + r) * p.lddy + c0 + lc;
  const int batch = (nv + kNormBatches - 1) / kNormBatches;
  const uint32_t slab = smem_u32(smem) + threadIdx.x * 16;
  grid_dep_wait();
  for (int b = 0; b < kNormBatches; ++b) {
    for (int i = b * batch; i < min(mine, (b + 1) * batch); ++i) {
      cp_async16(slab + 2 * i * NT * 16, xb, 16);
      cp_async16(slab + (2 * i + 1) * NT * 16, gb, 16);
      xb += (int64_t)t.ty * p.ldx;
      gb += (int64_t)t.ty * p.lddy;
    }
    cp_async_commit();
  }
  uint64_t t1[VN / 2], t2[VN / 2];
#pragma unroll
  for (int i = 0; i < VN / 2; ++i) t1[i] = t2[i] = 0;
  if (mine > 0) {
    NormGrad<VN> k;
    k.init(p, img, c0, lc);
    with_act(p.act, [&](auto act) {
      for (int b = 0; b < kNormBatches; ++b) {
        slab_wait(b);
#pragma unroll 1
        for (int i = b * batch; i < min(mine, (b + 1) * batch); ++i)
          k.template sums<decltype(act)::value, XT>(lds128(slab + 2 * i * NT * 16),
                                                    lds128(slab + (2 * i + 1) * NT * 16), t1, t2);
      }
    });
  }
  float both[2][VN];
  unpack_pairs<VN>(t1, both[0]);
  unpack_pairs<VN>(t2, both[1]);
  reduce_channels<NT, VN, 2>(both, active, tx, r, t, scratch, ch);
  if (cs > 1) { cluster_arrive(); cluster_wait(); }
  for (int c = threadIdx.x; c < 2 * W; c += NT) {
    float a = 0.0f;
    if (cs > 1) {
      a = dsmem_sum(ch + c, cs);
    } else {
      a = ch[c];
    }
    scratch[c] = a;
    if (rank == 0)
      p.total[(int64_t)img * 2 * t.C + (c < W ? c0 + c : t.C + c0 + c - W)] = a;
  }
  __syncthreads();
  if (cs > 1) cluster_arrive();
  grad_group_means<NT>(p, img, c0, W, scratch, g1, g2);
  if (mine > 0) {
    NormGradOut<VN> o;
    o.init(p, img, r0 + r, t.ty, c0, lc, g1, g2);
    with_act(p.act, [&](auto act) {
#pragma unroll 1
      for (int i = 0; i < mine; ++i)
        o.template put<decltype(act)::value, XT>(lds128(slab + 2 * i * NT * 16), lds128(slab + (2 * i + 1) * NT * 16));
    });
  }
  __syncwarp();
  if (cs > 1) cluster_wait();
}

// Two passes: the tiles' per-channel sums, the images' (group_norm_bwd_totals_kernel),
// then dx and the parameters' gradients.  3 x 16129 x 320 bf16 (31 MB each of x, dy, dx): 36.3 us
// for all three, the derivative of the activation, taken twice, above all.
template <typename XT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) group_norm_bwd_sums_kernel(const NormBwdArgs p) {
  constexpr int VN = Vec<XT>::n, U = kNormU2;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* scratch = reinterpret_cast<float*>(smem + norm_ring_bytes(NT, U, 2));
  float* ch = scratch + norm_scratch_floats(NT, VN);
  const int tile = blockIdx.x, cb = blockIdx.y, img = blockIdx.z;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const bool active = r < t.ty;
  const int c0 = cb * t.nb * t.cpg, lc = tx * VN;
  const int r0 = tile * t.rows, n_rows = min(t.S, r0 + t.rows) - r0;
  const int mine = active && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  NormStream<XT, NT, U, 2> in;
  in.at[0] = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  in.at[1] = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + (int64_t)(r0 + r) * p.lddy + c0 + lc;
  in.step[0] = (int64_t)t.ty * p.ldx;
  in.step[1] = (int64_t)t.ty * p.lddy;
  grid_dep_wait();
  in.begin(smem, mine);
  uint64_t t1[VN / 2], t2[VN / 2];
#pragma unroll
  for (int i = 0; i < VN / 2; ++i) t1[i] = t2[i] = 0;
  if (mine > 0) {
    NormGrad<VN> g;
    g.init(p, img, c0, lc);
    with_act(p.act, [&](auto act) {
      int k = 0;
      for (; (k + 1) * U <= mine; ++k) {
        const uint32_t at = in.wait(k);
#pragma unroll
        for (int i = 0; i < U; ++i)
          g.template sums<decltype(act)::value, XT>(in.get(at, i, 0), in.get(at, i, 1), t1, t2);
      }
      if (k * U < mine) {
        const uint32_t at = in.wait(k);
#pragma unroll 1
        for (int i = 0; k * U + i < mine; ++i)
          g.template sums<decltype(act)::value, XT>(in.get(at, i, 0), in.get(at, i, 1), t1, t2);
      }
    });
  }
  cp_async_wait<0>();
  float both[2][VN];
  unpack_pairs<VN>(t1, both[0]);
  unpack_pairs<VN>(t2, both[1]);
  reduce_channels<NT, VN, 2>(both, active, tx, r, t, scratch, ch);
  float* d = p.part + ((int64_t)img * p.tiles + tile) * 2 * t.C + c0;
  for (int c = threadIdx.x; c < W; c += NT) {
    d[c] = ch[c];
    d[t.C + c] = ch[W + c];
  }
}

template <typename XT, int NT>
__global__ void __launch_bounds__(NT, 512 / NT) group_norm_bwd_apply_kernel(const NormBwdArgs p) {
  constexpr int VN = Vec<XT>::n, U = kNormU2;
  extern __shared__ __align__(16) uint8_t smem[];
  const NormTile& t = p.t;
  const int W = t.vx * VN;
  float* tot = reinterpret_cast<float*>(smem + norm_ring_bytes(NT, U, 2));
  float* g1 = tot + 2 * W;
  float* g2 = g1 + t.nb;
  const int tile = gridDim.x - 1 - blockIdx.x, cb = gridDim.y - 1 - blockIdx.y,
            img = gridDim.z - 1 - blockIdx.z;
  const int c0 = cb * t.nb * t.cpg;
  const int tx = threadIdx.x % t.vx, r = threadIdx.x / t.vx;
  const int lc = tx * VN;
  const int r0 = tile * t.rows, n_rows = min(t.S, r0 + t.rows) - r0;
  const int mine = r < t.ty && r < n_rows ? (n_rows - r + t.ty - 1) / t.ty : 0;
  grid_dep_wait();
  NormStream<XT, NT, U, 2> in;
  in.at[0] = static_cast<const XT*>(p.x) + (int64_t)img * p.xbs + (int64_t)(r0 + r) * p.ldx + c0 + lc;
  in.at[1] = static_cast<const XT*>(p.dy) + (int64_t)img * p.dybs + (int64_t)(r0 + r) * p.lddy + c0 + lc;
  in.step[0] = (int64_t)t.ty * p.ldx;
  in.step[1] = (int64_t)t.ty * p.lddy;
  in.begin(smem, mine);
  for (int c = threadIdx.x; c < 2 * W; c += NT)
    tot[c] = p.total[(int64_t)img * 2 * t.C + (c < W ? c0 + c : t.C + c0 + c - W)];
  if (tile == 0 && img == 0) {
    // one CTA of each channel block adds the images for dbeta and dgamma, in order
    for (int c = threadIdx.x; c < 2 * W; c += NT) {
      const int ch = c < W ? c0 + c : c0 + c - W;
      float* out = c < W ? p.dbeta : p.dgamma;
      float a = 0.0f;
      for (int b = 0; b < p.B; ++b)
        a = fmaf(p.total[((int64_t)b * 2 + (c < W ? 0 : 1)) * t.C + ch],
                 c < W ? 1.0f : p.stats[((int64_t)b * t.G + ch / t.cpg) * 2 + 1], a);
      if (out != nullptr) out[ch] = a;
    }
  }
  __syncthreads();
  grad_group_means<NT>(p, img, c0, W, tot, g1, g2);
  if (mine > 0) {
    NormGradOut<VN> o;
    o.init(p, img, r0 + r, t.ty, c0, lc, g1, g2);
    with_act(p.act, [&](auto act) {
      int k = 0;
      for (; (k + 1) * U <= mine; ++k) {
        const uint32_t at = in.wait(k);
#pragma unroll
        for (int i = 0; i < U; ++i) o.template put<decltype(act)::value, XT>(in.get(at, i, 0), in.get(at, i, 1));
      }
      if (k * U < mine) {
        const uint32_t at = in.wait(k);
#pragma unroll 1
        for (int i = 0; k * U + i < mine; ++i)
          o.template put<decltype(act)::value, XT>(in.get(at, i, 0), in.get(at, i, 1));
      }
    });
  }
  cp_async_wait<0>();
}

// Two passes: each image's sums over its tiles.  A block has 32 channels of an image; its
// warps share the tiles and their sums are added in order, so results repeat bit for bit.
constexpr int kParamWarps = 16;
__global__ void __launch_bounds__(32 * kParamWarps) group_norm_bwd_totals_kernel(const NormBwdArgs p) {
  __shared__ float sh[2][kParamWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = p.t.C, c = blockIdx.x * 32 + lane, b = blockIdx.y;
  grid_dep_wait();
  float a1 = 0.0f, a2 = 0.0f;
  if (c < C) {
    const float* d = p.part + (int64_t)b * p.tiles * 2 * C + c;
#pragma unroll 8
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
  }
}

// dbeta and dgamma from the images' sums, in order.
__global__ void __launch_bounds__(32 * kParamWarps) group_norm_bwd_params_kernel(const NormBwdArgs p) {
  __shared__ float sh[2][kParamWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int C = p.t.C, c = blockIdx.x * 32 + lane;
  grid_dep_wait();
  float sum1 = 0.0f, sum2 = 0.0f;                // this warp's images
  if (c < C) {
    const float* stat = p.stats + (int64_t)(c / p.t.cpg) * 2 + 1;
#pragma unroll 4
    for (int b = warp; b < p.B; b += kParamWarps) {
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
    float* out = warp == 0 ? p.dbeta : p.dgamma;
    if (out != nullptr) out[c] = a;
  }
}

}  // namespace sq
