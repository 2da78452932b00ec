// Tensor-core forms of the adapter kernels (adapters.cuh has the formulas, the
// pieces of requests and the forms for few rows): 128 rows of a request per
// cluster of CTAs, bf16 operands, both products of the low-rank term in one
// kernel, and the adapters' gradients.
//
// The terms are bound by memory: x is read once and y read and written once,
// R/2 multiply-adds per byte.  So every byte moves by TMA through one ring that
// runs from the first product's tiles into the second's without a break, and h
// (or u) never leaves the chip between them.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "adapters.cuh"
#include "common.cuh"
#include "gemm_dualscale.cuh"
#include "ptx.cuh"

namespace sq {

// Shared-memory matrix descriptor of an MN-major operand in the 128-byte
// swizzle layout: atoms of 64 elements along M or N (128 bytes) by 8 along K,
// 1024 bytes from one group of 8 along K to the next, `lbo` bytes from one
// atom along M or N to the next.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescAMn = 1u << 15, kIdescBMn = 1u << 16;   // operand is MN-major

__device__ __forceinline__ void dsmem_store_u32x4(uint32_t addr, const uint32_t (&w)[4]) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3])
               : "memory");
}
// Orders this thread's generic-proxy accesses, to any CTA of the cluster, with the
// async proxy's.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void store_u32x8(void* p, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&w)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
               : "memory");
}
// The two epilogue warps of a TMEM lane quarter.
__device__ __forceinline__ void quarter_sync(int quad) {
  asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
}
// The same, and whether both came with `ok`.  Of two warps that wait for one mbarrier, one
// may see its phase and the other only the abort flag: both have to take the same way, or
// one of them waits for the other at the quarter's next barrier without a limit.
__device__ __forceinline__ bool quarter_agree(int quad, bool ok) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "bar.red.and.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q; }"
      : "=r"(r)
      : "r"(1 + quad), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
// Cuts 8 fp32 values into their nearest bf16 (packed into w) and the rest (left in v).
__device__ __forceinline__ void split_bf16(float (&v)[8], uint32_t (&w)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    w[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    v[2 * j] -= __uint_as_float(w[j] << 16);
    v[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
  }
}

constexpr int kTileRows = 128;
constexpr int kTileThreads = 320;          // TMA warp, MMA warp, eight epilogue warps
constexpr int kTileEpiWarps = 8;
constexpr int kTileX = kTileRows * 128;    // bytes of a 128-row, 128-byte-wide tile
constexpr int kTileBars = 512;             // bytes of barriers and flags
constexpr int kTileStages = 8;             // most slots of the ring
// The tensor core cuts its fp32 sums towards zero at every step, a bias that grows with the
// chain (1.4e-6 of the sum after 16 blocks of 64, where fp32 additions have 5e-7): after
// kChain blocks along the contracted axis the sums move to registers and are added there,
// while the next chain runs in a second accumulator.  h and u, which carry on into the second
// product and the gradients, move after kHChain blocks: their rms error is then that of fp32
// additions (1.3e-7 of h over 2048 or 4608 terms; 4.5e-7 in chains of eight), at the same time,
// since the reading warps have nothing else to do.
constexpr int kChain = 8, kHChain = 2;

struct AdapterTileArgs {
  AdapterArgs p;
  int32_t cs;          // CTAs per cluster
  int32_t stages;      // ring slots
  int32_t slot_bytes;  // kTileX + the weight tile
  int32_t parts;       // bf16 parts that h is multiplied as
  int32_t wide;        // the output's rows take 32-byte stores
  const float* hidden;         // backward: h of the forward pass [M, R], and
  __nv_bfloat16* f_u;          // u and h as three bf16 parts side by side, [M][3][rank padded to 16],
  __nv_bfloat16* f_h;          // the operands of the adapters' gradients
  long long wait_budget;
  int32_t starve;      // test hook: 0, or one more than the copies that the producer issues
};

// Shared memory between the two products: this CTA's partial h in fp32 (rows padded
// by 16 bytes against bank conflicts), then h as `parts` bf16 operand tiles.
__host__ __device__ inline int adapter_h_bytes(int rp, int parts) {
  const int op = parts * kTileX * ((rp + 63) / 64);
  const int ex = kTileRows * (rp + 4) * 4;
  return ((op > ex ? op : ex) + 1023) / 1024 * 1024;
}

// Forward (BWD = false): h = x A^T over this CTA's share of K; the shares are
// added over the cluster in rank order; y += scale h B^T over this CTA's share
// of the columns, in tiles 128 bytes wide.  Backward: u = scale dy B, dx = u A, the
// same steps with both weights MN-major.  RB: the largest rank (64 or 128).
//
// h is summed in TMEM in chains of kHChain blocks, which meet in fp32 registers; as an operand
// it is the sum of `parts` bf16 values (two for bf16 outputs: off by 2^-17 of h, against
// the output's own 2^-8; three for fp32 outputs: exact to 2^-24), which costs R/2 more
// multiply-adds per output and no bytes.
//
// 8192 x 4608 -> 1152, rank 64 (119 MB): 40.2 us, 2.97 TB/s; 16384 x 2304 -> 3456, rank 32, 23
// ragged requests (248 MB): 62.8 us, 3.95 TB/s.  A cluster's exchange between the products
// (about 9 us, in which it asks for no more than the ring holds) and the search and launch
// (3 us) bound them; the tensor cores are busy for 9 %.
// OT other than YT: y + the term goes to out, rounded once, and so do the rows without an adapter.
template <int RB, typename YT, typename OT, bool BWD>
__global__ void __launch_bounds__(kTileThreads, RB == 64 ? 2 : 1)
    adapter_tile_kernel(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap tw1,
                        const __grid_constant__ CUtensorMap tw2, const __grid_constant__ CUtensorMap ty,
                        const __grid_constant__ AdapterTileArgs args) {
  constexpr int ES = sizeof(YT);
  constexpr bool APART = !std::is_same<YT, OT>::value;
  constexpr int BN = 128 / ES;             // columns of an output tile
  constexpr int D2 = RB;                   // TMEM column of the second accumulator of h, and of the outputs,
  constexpr int ND = RB == 64 ? 3 : 2;     // and how many tiles of them there are room for
  const AdapterArgs& p = args.p;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int cs = args.cs, NS = args.stages;
  const int rank = blockIdx.x % cs;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dep_wait();
  if (blockIdx.x == 0) check_requests(p, kTileThreads);
  const AdapterItem it = adapter_item(p, blockIdx.x / cs, kTileRows);
  const int D = BWD ? p.N : p.K, E = BWD ? p.K : p.N, R = p.R;
  const int etiles = (E + BN - 1) / BN;
  const int t0 = (int)((int64_t)rank * etiles / cs), t1 = (int)((int64_t)(rank + 1) * etiles / cs);
  if (it.n == 0 || it.l < 0) {             // the same for every CTA of the cluster
    if (BWD) {
      const int c0 = t0 * BN, w = (min(E, t1 * BN) - c0) * ES / 16;
      for (int m = warp; m < it.n; m += kTileThreads / 32) {
        uint4* d = reinterpret_cast<uint4*>(static_cast<YT*>(p.y) + (int64_t)(it.row + m) * p.ldy + c0);
        for (int i = lane; i < w; i += 32) d[i] = make_uint4(0u, 0u, 0u, 0u);
      }
      return;
    }
    if (p.h != nullptr && rank == 0)
      for (int i = threadIdx.x; i < it.n * R; i += kTileThreads) p.h[(int64_t)it.row * R + i] = 0.0f;
    if (APART)
      for (int m = warp; m < it.n; m += kTileThreads / 32)
        copy_row(static_cast<const YT*>(p.y) + (int64_t)(it.row + m) * p.ldy,
                 static_cast<OT*>(p.out) + (int64_t)(it.row + m) * p.ldo, t0 * BN / 8 + lane, min(E, t1 * BN) / 8, 32);
    return;
  }
  const int RP = (R + 15) & ~15, rt = (RP + 63) / 64;
  uint8_t* hbuf = smem + NS * args.slot_bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(hbuf + adapter_h_bytes(RP, args.parts));
  uint64_t* full = bars;                       // [kTileStages]
  uint64_t* empty1 = full + kTileStages;       // [kTileStages] slot free: its products are done
  uint64_t* empty3 = empty1 + kTileStages;     // [kTileStages] forward, second product: its tile of y is read
  uint64_t* d_full = empty3 + kTileStages;     // [3]
  uint64_t* d_empty = d_full + 3;    // [3]
  uint64_t* h_full = d_empty + 3;    // [2] a chain of h is complete
  uint64_t* h_free = h_full + 2;     // [2] and read
  uint64_t* h_ready = h_free + 2;
  uint64_t* p_full = h_ready + 1;    // every CTA's partial h is written
  uint64_t* p_free = p_full + 1;     // every CTA has read this one's
  uint64_t* drain_bar = p_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const long long budget = args.wait_budget;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty1 + i), 1);
      mbar_init(smem_u32(empty3 + i), kTileEpiWarps);
    }
    for (int i = 0; i < ND; ++i) {
      mbar_init(smem_u32(d_full + i), 1);
      mbar_init(smem_u32(d_empty + i), kTileEpiWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(h_full + i), 1);
      mbar_init(smem_u32(h_free + i), kTileEpiWarps);
    }
    mbar_init(smem_u32(h_ready), kTileEpiWarps * cs);
    mbar_init(smem_u32(p_full), kTileEpiWarps * cs);
    mbar_init(smem_u32(p_free), kTileEpiWarps * cs);
    mbar_init(smem_u32(drain_bar), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (cs > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int nkb = (D + 63) / 64;
  const int kb0 = (int)((int64_t)rank * nkb / cs), kb1 = (int)((int64_t)(rank + 1) * nkb / cs);
  const int nk = kb1 - kb0, nt = t1 - t0;
  const int boxes = (it.n + 31) / 32;      // 32-row boxes that hold rows of the piece

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tx);
      tma_prefetch_desc(&tw1);
      tma_prefetch_desc(&tw2);
      if (!BWD) tma_prefetch_desc(&ty);
      bool ok = true;
      const int copies = args.starve == 0 ? nk + nt : min(nk + nt, args.starve - 1);
      int i = 0;
      for (; i < copies; ++i) {
        const int s = i % NS, prev = i - NS;
        if (prev >= 0) {
          if (BWD || prev < nk) {
            ok = wait1(smem_u32(empty1 + s), (prev / NS) & 1, abort_flag, budget);
          } else {
            const int first = nk + ((s - nk % NS) + NS) % NS;   // first tile of the second product in slot s
            ok = wait1(smem_u32(empty3 + s), ((prev - first) / NS) & 1, abort_flag, budget);
          }
          if (!ok) break;
        }
        const uint32_t st = smem_u32(smem + s * args.slot_bytes), wt = st + kTileX, bar = smem_u32(full + s);
        if (i < nk) {
          const int k = (kb0 + i) * 64;
          mbar_arrive_expect_tx(bar, boxes * 4096 + (BWD ? rt * 8192 : R * 128));
          for (int b = 0; b < boxes; ++b) tma_load_2d(st + b * 4096, &tx, bar, k, it.row + 32 * b);
          if (BWD) {
            for (int t = 0; t < rt; ++t) tma_load_3d(wt + t * 8192, &tw1, bar, 64 * t, k, it.l);
          } else {
            tma_load_3d(wt, &tw1, bar, k, 0, it.l);
          }
        } else {
          const int c = (t0 + i - nk) * BN;
          mbar_arrive_expect_tx(bar, BWD ? RP * 128 : boxes * 4096 + rt * BN * 128);
          if (BWD) {
            tma_load_3d(wt, &tw2, bar, c, 0, it.l);
          } else {
            for (int t = 0; t < rt; ++t) tma_load_3d(wt + t * BN * 128, &tw2, bar, 64 * t, c, it.l);
            for (int b = 0; b < boxes; ++b) tma_load_2d(st + b * 4096, &ty, bar, c, it.row + 32 * b);
          }
        }
      }
      drain_ring(full, NS, i, kDrainBudget);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      bool ok = true;
      const uint32_t id1 = idesc_bf16(kTileRows, RP) | (BWD ? kIdescBMn : 0u);
      // a slot of the ring and its phase are carried along: this thread's own steps bound it
      int s = 0;
      uint32_t phase = 0;
      for (int i = 0, b = 0, freed = 1; i < nk && ok; i += kHChain) {      // a chain
        if (i >= 2 * kHChain) {
          if (!(ok = wait1(smem_u32(h_free + b), (uint32_t)freed, abort_flag, budget))) break;
          tc_fence_after();
        }
        const int end = min(nk, i + kHChain);
        uint32_t acc = 0;
        for (int k = i; k < end; ++k) {
          if (!(ok = wait1(smem_u32(full + s), phase, abort_flag, budget))) break;
          const uint32_t st = smem_u32(smem + s * args.slot_bytes), wt = st + kTileX;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_bf16(tmem + b * D2, smem_desc_k_sw128(st + ks * 32),
                      BWD ? smem_desc_mn_sw128(wt + ks * 2048, 8192) : smem_desc_k_sw128(wt + ks * 32), id1,
                      ks > 0 ? 1u : acc);
          acc = 1;
          umma_commit(smem_u32(empty1 + s));
          if (++s == NS) { s = 0; phase ^= 1; }
        }
        if (ok) umma_commit(smem_u32(h_full + b));
        b ^= 1;
        freed ^= b == 0;           // the phase of h_free that the next two chains wait for
      }
      if (ok) {
        ok = wait1s<true>(smem_u32(h_ready), 0, abort_flag, budget);
        fence_proxy_async_all();
        tc_fence_after();
      }
      const uint32_t id2 = idesc_bf16(kTileRows, BN) | (BWD ? kIdescBMn : 0u);
      const uint32_t hb = smem_u32(hbuf);
      for (int j = 0; j < nt && ok; ++j) {
        const int b = j % ND;
        if (j >= ND && !(ok = wait1(smem_u32(d_empty + b), (j / ND - 1) & 1, abort_flag, budget))) break;
        if (!(ok = wait1(smem_u32(full + s), phase, abort_flag, budget))) break;
        tc_fence_after();
        const uint32_t wt = smem_u32(smem + s * args.slot_bytes) + kTileX;
        uint32_t acc = 0;
        for (int part = args.parts - 1; part >= 0; --part)       // the small terms first: little is cut off them
          for (int ks = 0; ks < RP / 16; ++ks) {
            const uint32_t a = hb + (part * rt + (ks >> 2)) * kTileX + (ks & 3) * 32;
            umma_bf16(tmem + D2 + b * BN, smem_desc_k_sw128(a),
                      BWD ? smem_desc_mn_sw128(wt + ks * 2048, 8192)
                          : smem_desc_k_sw128(wt + (ks >> 2) * BN * 128 + (ks & 3) * 32),
                      id2, acc);
            acc = 1;
          }
        if (BWD) umma_commit(smem_u32(empty1 + s));   // the slot held the weight tile alone
        umma_commit(smem_u32(d_full + b));
        if (++s == NS) { s = 0; phase ^= 1; }
      }
      umma_commit(smem_u32(drain_bar));
      wait_drain(smem_u32(drain_bar), 0, kDrainBudget);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const int row = quad * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    const int hc = RP / 2, c0 = half * hc;    // this thread's columns of the partial h
    // 1. this CTA's share of h: its chains added up, into its own shared memory
    float t[RB / 2];
#pragma unroll
    for (int c = 0; c < RB / 2; ++c) t[c] = 0.0f;
    bool ok = true;
    for (int chain = 0; chain * kHChain < nk; ++chain) {
      const int b = chain & 1;
      if (!(ok = wait_warp(smem_u32(h_full + b), (chain / 2) & 1, abort_flag, budget))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < RB / 2; c += 8) {
        if (c < hc) {
          uint32_t u[8];
          tmem_ld8(t_lane + b * D2 + c0 + c, u);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k) t[c + k] += __uint_as_float(u[k]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(h_free + b));
    }
    if (ok) {
      float* mine = reinterpret_cast<float*>(hbuf) + row * (RP + 4) + c0;
#pragma unroll
      for (int c = 0; c < RB / 2; c += 4)
        if (c < hc) *reinterpret_cast<float4*>(mine + c) = make_float4(t[c], t[c + 1], t[c + 2], t[c + 3]);
      __syncwarp();
      if (lane < cs) mbar_arrive_remote(mapa_shared(smem_u32(p_full), lane));
      ok = wait_warp<true>(smem_u32(p_full), 0, abort_flag, budget);
    }
    if (ok) {
      // 2. each CTA adds its share of the rows over the cluster, in rank order: units of
      // eight columns of a row, whole rows side by side, so that a warp reads long runs
      // of a peer's memory
      const int et = threadIdx.x - 64, octs = RP / 8;
      const int units = it.n * octs;
      const int u0 = (int)((int64_t)rank * units / cs), u1 = (int)((int64_t)(rank + 1) * units / cs);
      constexpr int MAXU = kTileRows * (RB / 8) / 256;
      float v[MAXU][8];
#pragma unroll
      for (int k = 0; k < MAXU; ++k) {
        const int u = u0 + et + 256 * k;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
        if (u < u1) {
          const float* at = reinterpret_cast<const float*>(hbuf) + (u / octs) * (RP + 4) + (u % octs) * 8;
          dsmem_sum8(at, cs, v[k]);
          // The values have to be here before this warp says so: a store of the sums (into the
          // unit's own place, which no other thread reads) depends on them, and the arrival
          // comes behind it.
          const uint32_t a = smem_u32(at);
          const uint32_t lo[4] = {__float_as_uint(v[k][0]), __float_as_uint(v[k][1]), __float_as_uint(v[k][2]),
                                  __float_as_uint(v[k][3])};
          const uint32_t hi[4] = {__float_as_uint(v[k][4]), __float_as_uint(v[k][5]), __float_as_uint(v[k][6]),
                                  __float_as_uint(v[k][7])};
          sts128(a, lo);
          sts128(a + 16, hi);
        }
      }
      __syncwarp();
      if (lane < cs) mbar_arrive_remote(mapa_shared(smem_u32(p_free), lane));
      const float scale = p.scale != nullptr ? __ldg(p.scale + it.l) : 1.0f;
      ok = wait_warp<true>(smem_u32(p_free), 0, abort_flag, budget);
      if (ok) {
        // 3. the sums, scaled and cut into bf16 parts, into every CTA's operand
#pragma unroll
        for (int k = 0; k < MAXU; ++k) {
          const int u = u0 + et + 256 * k;
          if (u < u1) {
            const int hr = u / octs, col = (u % octs) * 8;
            const int64_t gr = it.row + hr;
            if (!BWD && p.h != nullptr && col < R) store_vec<8>(p.h, gr * R + col, false, v[k]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = col < R ? v[k][j] * scale : 0.0f;   // the padding is an operand, too
            const uint32_t d = smem_u32(hbuf) + (col >> 6) * kTileX + hr * 128 + ((((col & 63) >> 3) ^ (hr & 7)) << 4);
            for (int part = 0; part < (BWD ? 3 : args.parts); ++part) {
              uint32_t w[4];
              split_bf16(v[k], w);
              if (part < args.parts)
                for (int q = 0; q < cs; ++q) dsmem_store_u32x4(mapa_shared(d + part * rt * kTileX, q), w);
              if (BWD)
                *reinterpret_cast<uint4*>(args.f_u + (gr * 3 + part) * RP + col) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            if (BWD && col < R) {
              float hv[8];
              load8(args.hidden + gr * R + col, hv);
              for (int part = 0; part < 3; ++part) {
                uint32_t w[4];
                split_bf16(hv, w);
                *reinterpret_cast<uint4*>(args.f_h + (gr * 3 + part) * RP + col) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        fence_proxy_async_all();
        __syncwarp();
        if (lane < cs) mbar_arrive_remote(mapa_shared(smem_u32(h_ready), lane));
      }
    }
    // Output tiles; a thread has 64 bytes of its row.  Forward: they are added to y's, read
    // from the ring, and stored in whole 32-byte sectors: that
    // costs the load/store unit a line per row, but held the ring's slots shorter than TMA
    // stores from them (62 us instead of 67 on the ragged batch of 16384 x 2304 -> 3456).
    // Backward: no ring to hold up; tiles are put together in the first product's room (the
    // slots' x tiles), and a quarter's 32 rows go out in one TMA store where the piece has
    // them all, else row by row (69 us instead of 73 for all gradients of 8192 x 4608 -> 1152).
    const int rows = min(32, it.n - quad * 32);     // rows of the piece in this quarter (may be < 1)
    const bool issuer = half == 0 && lane == 0;     // of the quarter's stores
    OT* out = APART ? static_cast<OT*>(p.out) + (int64_t)(it.row + row) * p.ldo
                    : static_cast<OT*>(p.y) + (int64_t)(it.row + row) * p.ldy;
    for (int j = 0; j < nt && ok; ++j) {
      const int i = nk + j, s = i % NS, b = j % ND;
      if (!BWD && !(ok = wait_warp(smem_u32(full + s), (i / NS) & 1, abort_flag, budget))) break;
      ok = wait_warp(smem_u32(d_full + b), (j / ND) & 1, abort_flag, budget);
      if (BWD && rows > 0) ok = quarter_agree(quad, ok);   // the quarter's warps meet below
      if (!ok) break;
      tc_fence_after();
      if (rows > 0) {
        const uint32_t tile = smem_u32(smem + s * args.slot_bytes + quad * 4096), mine = tile + lane * 128;
        const uint32_t acc = t_lane + D2 + b * BN + half * (BN / 2);
        uint32_t u[BN / 2];
#pragma unroll
        for (int g = 0; g < BN / 2; g += 16) tmem_ld16(acc + g, *reinterpret_cast<uint32_t(*)[16]>(u + g));
        uint4 y[4];
        if constexpr (!BWD) {
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = lds128(mine + (((half * 4 + q) ^ (lane & 7)) << 4));
        } else {
          // this room's last store has been read: NS >= 3 rooms, two younger ones may be under way
          if (issuer && j >= NS) bulk_wait_read<2>();
          quarter_sync(quad);
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(d_empty + b));
        uint32_t w[16];                              // 8 of them where fp32 becomes bf16
#pragma unroll
        for (int q = 0; q < 4; ++q) {                // 16-byte chunks
          constexpr int PER = 16 / ES;
          float o[PER];
          if constexpr (!BWD) {
            Vec<YT>::load_raw(y[q], o);
          } else {
#pragma unroll
            for (int k = 0; k < PER; ++k) o[k] = 0.0f;
          }
#pragma unroll
          for (int k = 0; k < PER; ++k) o[k] += __uint_as_float(u[q * PER + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (ES == 2) w[4 * q + k] = pack_bf16(o[2 * k], o[2 * k + 1]);
            else if constexpr (!APART) w[4 * q + k] = __float_as_uint(o[k]);
            else if (k < 2) w[2 * q + k] = pack_bf16(o[2 * k], o[2 * k + 1]);
          }
        }
        const int c0t = (t0 + j) * BN;
        if constexpr (!BWD) {
          const int c = c0t + half * (BN / 2);
          if (lane < rows) {
            // the columns come in multiples of 16
            if (c < E) store_u32x8(out + c, *reinterpret_cast<const uint32_t(*)[8]>(w), args.wide != 0);
            if (!APART && c + 32 / ES < E)
              store_u32x8(out + c + 32 / ES, *reinterpret_cast<const uint32_t(*)[8]>(w + 8), args.wide != 0);
          }
          // behind the stores, which depend on what was read of the slot: an arrival right after
          // the loads let the ring overwrite rows that were still on their way to registers
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(empty3 + s));
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            sts128(mine + (((half * 4 + q) ^ (lane & 7)) << 4), *reinterpret_cast<const uint32_t(*)[4]>(w + 4 * q));
          if (rows == 32) {
            fence_proxy_async_smem();
            quarter_sync(quad);
            if (issuer) {
              tma_store_2d(&ty, tile, c0t, it.row + quad * 32);
              bulk_commit_group();
            }
          } else {
            quarter_sync(quad);
            const int c = c0t + half * (BN / 2) + (lane & 3) * (16 / ES);
            if (c < E) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int r = k * 8 + (lane >> 2);
                if (r < rows)
                  *reinterpret_cast<uint4*>(static_cast<YT*>(p.y) + (int64_t)(it.row + quad * 32 + r) * p.ldy + c) =
                      lds128(tile + r * 128 + (((half * 4 + (lane & 3)) ^ (r & 7)) << 4));
              }
            }
          }
        }
      } else if (lane == 0) {
        mbar_arrive(smem_u32(d_empty + b));
        if (!BWD) mbar_arrive(smem_u32(empty3 + s));
      }
    }
    if (BWD && issuer) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (cs > 1) cluster_sync();      // no peer still reads this CTA's memory or signals its barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// -------------------------------------------- gradients of the adapters, bf16
// dA_l = sum u^T x and dB_l = scale sum dy^T h: 128 columns of the long axis by
// the rank per cluster and adapter, contracted over the rows of all its requests
// in pieces of 64, which the CTAs of the cluster take in turn; their sums are
// added through distributed shared memory in rank order.
// f (u or h) comes as three bf16 parts side by side along the rank axis (exact to
// 2^-24, since the sums are fp32 results), g (x or dy) as it is; both operands are
// MN-major, so TMA brings them as they lie in memory.
// The sums move to registers after chains of kChain pieces.
// 8192 rows, 4608 and 1152 columns, rank 16, 4 adapters (96 MB): 26 us, 3.7 TB/s, bound by the
// one thread that issues a CTA's products, 0.7 us a piece.
struct AdapterGradTileArgs {
  float* out[2];                 // da, db
  const float* scale;            // of the second, or null
  const int32_t* bounds;
  const int32_t* index;
  int32_t C[2];                  // K, N
  int32_t tiles0;                // tiles of the first
  int32_t M, R, L, Q;
  int32_t cs, stages;
  long long wait_budget;
  int32_t starve;
};
__host__ __device__ inline int adapter_grad_atoms(int rp) { return (3 * rp + 63) / 64; }   // 64 ranks wide

// RB: the largest rank (32, 64, 128); CTAs per SM 3, 2, 1, by their sums' registers and
// TMEM columns (an SM needs several issuing threads: two CTAs at rank 16 took 2.8 us longer).
__host__ __device__ constexpr int adapter_grad_ctas(int rb) { return rb == 32 ? 3 : rb == 64 ? 2 : 1; }
template <int RB>
__global__ void __launch_bounds__(kTileThreads, adapter_grad_ctas(RB))
    adapter_grad_tile_kernel(const __grid_constant__ CUtensorMap tg0, const __grid_constant__ CUtensorMap tg1,
                             const __grid_constant__ CUtensorMap tf0, const __grid_constant__ CUtensorMap tf1,
                             const __grid_constant__ AdapterGradTileArgs p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr int TM = RB == 32 ? 128 : RB == 64 ? 256 : 512;
  const int cs = p.cs, NS = p.stages, R = p.R, RP = (R + 15) & ~15;
  const int rank = blockIdx.x % cs, l = blockIdx.y;
  int tile = blockIdx.x / cs;
  const int which = tile < p.tiles0 ? 0 : 1;
  if (which) tile -= p.tiles0;
  const int C = p.C[which], c0 = tile * 128;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int atoms = adapter_grad_atoms(RP), slot_bytes = kTileX + atoms * 8192;
  const int cols = 3 * RP, buf = (cols + 31) & ~31, NB = 2 * buf <= TM ? 2 : 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + max(NS * slot_bytes, cs > 1 ? 128 * RP * 4 : 0));
  uint64_t* full = bars;           // [4] f and g have landed
  uint64_t* empty = full + 4;      // [4]
  uint64_t* d_full = empty + 4;    // [2] a chain's sums are complete
  uint64_t* d_empty = d_full + 2;  // [2] and read
  uint64_t* brief = d_empty + 2;   // a short piece has landed: the rows behind it are to be cleared
  uint64_t* ready = brief + 1;     // and they are
  uint64_t* p_full = ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(p_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* note = abort_flag + 1;   // [4] what the slot holds: 1 the last piece, 2 a short one, 4 nothing
  const long long budget = p.wait_budget;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(full + i), 1);
      mbar_init(smem_u32(empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(d_full + i), 1);
      mbar_init(smem_u32(d_empty + i), kTileEpiWarps);
    }
    mbar_init(smem_u32(brief), 1);
    mbar_init(smem_u32(ready), kTileEpiWarps);
    mbar_init(smem_u32(p_full), kTileEpiWarps * cs);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  if (cs > 1) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  grid_dep_wait();
  GradPieces pieces{p.bounds, p.index, p.M, p.L, p.Q, l, rank, cs};
  int m0, n, i = 0;
  bool ok = true;
  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    const CUtensorMap* tg = which ? &tg1 : &tg0;
    const CUtensorMap* tf = which ? &tf1 : &tf0;
    if (lane == 0) {
      tma_prefetch_desc(tg);
      tma_prefetch_desc(tf);
    }
    ok = p.starve == 0;
    bool more = pieces.mine(m0, n);
    if (!more && lane == 0) {      // no rows: the MMA thread hears of it through the first slot
      note[0] = 4;
      mbar_arrive(smem_u32(full));
    }
    while (ok && more) {
      const int s = i % NS, at = m0, cnt = n;
      more = pieces.mine(m0, n);
      if (i >= NS && !(ok = wait_warp(smem_u32(empty + s), (i / NS - 1) & 1, abort_flag, budget))) break;
      if (lane == 0) {
        const uint32_t st = smem_u32(smem + s * slot_bytes), bar = smem_u32(full + s);
        note[s] = (more ? 0 : 1) | (cnt < kGradPiece ? 2 : 0);
        mbar_arrive_expect_tx(bar, slot_bytes);
        tma_load_2d(st, tg, bar, c0, at);
        tma_load_2d(st + 8192, tg, bar, c0 + 64, at);
        for (int a = 0; a < atoms; ++a) tma_load_2d(st + kTileX + a * 8192, tf, bar, a * 64, at);
      }
      ++i;
    }
    if (lane == 0) drain_ring(full, NS, i, kDrainBudget);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // One thread, kept lean: the producer leaves a note with each slot.
    if (lane == 0) {
      const int n1 = cols > 256 ? 192 : cols, n2 = cols - n1;
      const uint32_t id1 = idesc_bf16(128, n1) | kIdescAMn | kIdescBMn;
      const uint32_t id2 = idesc_bf16(128, n2 > 0 ? n2 : 16) | kIdescAMn | kIdescBMn;
      int chain = 0, shorts = 0, s = 0, b = 0;
      uint32_t phase = 0;
      bool last = false;
      while (!last) {
        const bool first = i % kChain == 0;
        if (first && chain >= NB && !(ok = wait1(smem_u32(d_empty + b), (chain / NB - 1) & 1, abort_flag, budget))) break;
        if (!(ok = wait1(smem_u32(full + s), phase, abort_flag, budget))) break;
        const int what = note[s];
        if (what == 4) break;
        last = what & 1;
        if (what & 2) {
          mbar_arrive(smem_u32(brief));
          if (!(ok = wait1(smem_u32(ready), shorts & 1, abort_flag, budget))) break;
          ++shorts;
        }
        tc_fence_after();
        const uint32_t st = smem_u32(smem + s * slot_bytes), d = tmem + b * buf;
        const uint64_t da = smem_desc_mn_sw128(st, 8192), df = smem_desc_mn_sw128(st + kTileX, 8192);
        // 16 rows on: 2048 bytes, 128 units of a descriptor's address
#pragma unroll
        for (int ks = 0; ks < kGradPiece / 16; ++ks) {
          const uint32_t acc = !first || ks > 0 ? 1u : 0u;
          umma_bf16(d, da + ks * 128, df + ks * 128, id1, acc);
          if (n2 > 0) umma_bf16(d + n1, da + ks * 128, df + 3 * 512 + ks * 128, id2, acc);
        }
        ++i;
        umma_commit(smem_u32(empty + s));
        if (last || i % kChain == 0) umma_commit(smem_u32(d_full + b));
        if (++s == NS) { s = 0; phase ^= 1; }
        if (i % kChain == 0) { ++chain; b = chain % NB; }
      }
      if (i > 0)                   // every product has landed when the last commit has
        wait_drain(smem_u32(empty + (i - 1) % NS), ((i - 1) / NS) & 1, kDrainBudget);
    }
    __syncwarp();
  } else {
    // ----------------------- short pieces cleared, the chains' sums added up
    const int tid = threadIdx.x - 64;
    const int quad = warp & 3, half = (warp - 2) >> 2, row = quad * 32 + lane;
    const int hc = RP / 2, r0 = half * hc;
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    float t[RB / 2];
#pragma unroll
    for (int c = 0; c < RB / 2; ++c) t[c] = 0.0f;
    int chain = 0, shorts = 0;
    bool more = pieces.mine(m0, n);
    while (more) {
      const int s = i % NS, cnt = n;
      if (cnt < kGradPiece) {
        // rows behind the piece belong to other requests: cleared, whatever they hold
        if (!(ok = wait_warp(smem_u32(brief), shorts & 1, abort_flag, budget))) break;
        ++shorts;
        uint8_t* st = smem + s * slot_bytes;
        const int per = 8 * (2 + atoms);               // 16-byte words of a row
        for (int u = tid; u < (kGradPiece - cnt) * per; u += 256)
          *reinterpret_cast<uint4*>(st + (u % per >> 3) * 8192 + (cnt + u / per) * 128 + (u & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(ready));
      }
      more = pieces.mine(m0, n);
      ++i;
      if (!more || i % kChain == 0) {
        const int b = chain % NB;
        if (!(ok = wait_warp(smem_u32(d_full + b), (chain / NB) & 1, abort_flag, budget))) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < RB / 2; c += 8) {
          if (c < hc) {
            uint32_t a[8], bb[8], d[8];
            tmem_ld8(t_lane + b * buf + r0 + c, a);
            tmem_ld8(t_lane + b * buf + RP + r0 + c, bb);
            tmem_ld8(t_lane + b * buf + 2 * RP + r0 + c, d);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              t[c + k] += __uint_as_float(a[k]) + (__uint_as_float(bb[k]) + __uint_as_float(d[k]));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(d_empty + b));
        ++chain;
      }
    }
    const bool mine = cs == 1 || (quad * 2 + half) % cs == rank;
    if (cs > 1) {
      // the ring is idle: all copies have landed and all products are done
      float4* own = reinterpret_cast<float4*>(smem) + (r0 / 4) * 128 + row;
      if (ok) {
#pragma unroll
        for (int c = 0; c < RB / 2; c += 4)
          if (c < hc) own[(c / 4) * 128] = make_float4(t[c], t[c + 1], t[c + 2], t[c + 3]);
        __syncwarp();
        if (lane < cs) mbar_arrive_remote(mapa_shared(smem_u32(p_full), lane));
        ok = wait_warp<true>(smem_u32(p_full), 0, abort_flag, budget);
      }
      if (ok && mine) {
#pragma unroll
        for (int c = 0; c < RB / 2; ++c) t[c] = 0.0f;
        for (int k = 0; k < cs; ++k) {
          const uint32_t from = mapa_shared(smem_u32(own), k);
#pragma unroll
          for (int c = 0; c < RB / 2; c += 4)
            if (c < hc) {
              const float4 o = dsmem_f32x4(from + (c / 4) * 128 * 16);
              t[c] += o.x; t[c + 1] += o.y; t[c + 2] += o.z; t[c + 3] += o.w;
            }
        }
      }
    }
    if (ok && mine && c0 + row < C) {
      const float scale = which && p.scale != nullptr ? __ldg(p.scale + l) : 1.0f;
#pragma unroll
      for (int c = 0; c < RB / 2; c += 8) {
        if (c < hc && r0 + c < R) {
          if (which) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = t[c + k] * scale;
            store_vec<8>(p.out[1], ((int64_t)l * C + c0 + row) * R + r0 + c, false, o);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) p.out[0][((int64_t)l * R + r0 + c + k) * C + c0 + row] = t[c + k];
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (cs > 1) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM);
  }
}

}  // namespace sq
