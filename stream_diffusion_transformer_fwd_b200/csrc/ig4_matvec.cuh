// ig4_matvec.cuh - 1 to 8 bf16 rows times NVFP4 weights (E2M1 codes, an E4M3
// scale per 16 weights, an fp32 scale per output), alone or as the gated pair
// of a feed-forward layer: u = silu(x Wg^T) * (x Wu^T).
//
// Each weight is used M <= 8 times, so the weight bytes (4.5 bits per weight)
// bound it, as long as turning codes into operands keeps up: a few instructions
// per weight would not.  The products therefore run on mma.sync m16n8k16 with
// the weights as the 16-row operand and the M rows as its 8 columns: tcgen05
// would want the operands staged in shared memory and a 128-row accumulator to
// drain, while here a lane's 16 loaded bytes become its own operand registers.
// The order of the contraction is free: lane (g, t) of a warp takes 32
// consecutive codes of weight rows g and g + 8 (one 16-byte load each) and the
// same 32 elements of x row g, four per MMA.
//
// Exactness: code times group scale has at most 6 significant bits between
// 2^-10 and 2688, so the fp16 product of the two is exact; x (8 significant
// bits) is multiplied by a power of two per row and warp that brings its
// largest element into [2^14, 2^15) before it becomes fp16: exact down to
// 2^-28 of that element, rounded at 2^-39 of it below.  Sums are fp32.
//
// A warp keeps its slice of x in registers for all the weight rows it meets; a
// CTA's 8 warps split K, and for long K (or few rows) the CTAs of a cluster
// split it further and exchange partial sums through distributed shared
// memory.  16-row tiles take rows {4j .. 4j+3} + {0, 32, 64, 96} of a 128-row
// block: their 16 scale words of a k-block are then 64 consecutive bytes in the
// packed order.
#pragma once

#include <cuda_fp16.h>

#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int MATVEC_WARPS = 8;
constexpr int MATVEC_THREADS = 32 * MATVEC_WARPS;
constexpr int MATVEC_CHUNK = 128;    // k elements of a warp step: 4 lanes x 32
constexpr int MATVEC_MAX_CHUNKS = 3; // per warp
constexpr int MATVEC_MAX_CLUSTER = 8;
constexpr int MATVEC_BATCH = 8;      // row tiles per exchange between the CTAs of a cluster

struct MatvecWeights {
  const uint8_t *codes;
  const uint8_t *sf;
  const float *scale;
};

__device__ __forceinline__ uint4 ldg_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Two E2M1 codes (byte `i` of w, low nibble first) as an fp16 pair
template <int i>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (i == 0)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (i == 1)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (i == 2)
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// C: 128-element chunks of K per warp.  DUAL: w[0] gate, w[1] up.
template <int C, bool DUAL, typename OT>
__global__ void __launch_bounds__(MATVEC_THREADS, 2)
    nvfp4_matvec_kernel(const __nv_bfloat16 *x, MatvecWeights w0, MatvecWeights w1,
                        const float *bias, OT *out, int M, int N, int K, int n_tiles, int cluster) {
  constexpr int MATS = DUAL ? 2 : 1;
  __shared__ float red[2][MATVEC_WARPS][128];
  __shared__ float psum[2][MATVEC_BATCH][MATS][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cl = blockIdx.x / cluster, n_cl = gridDim.x / cluster;
  pdl_wait();
  pdl_trigger();

  // this warp's run of chunks
  const int nc = (K + MATVEC_CHUNK - 1) / MATVEC_CHUNK;
  const int slots = cluster * MATVEC_WARPS, slot = rank * MATVEC_WARPS + warp;
  const int c0 = nc * slot / slots, c1 = nc * (slot + 1) / slots;  // at most C chunks

  // x slice: 16 fp16 pairs per chunk, scaled by 2^sh; inv0, inv1 undo it for
  // the accumulator's columns (tokens 2t, 2t + 1)
  uint32_t xb[C][16];
  float inv0, inv1;
  {
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = (c0 + c) * MATVEC_CHUNK + 32 * t;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c0 + c < c1 && k < K && g < M)
          v = __ldg(reinterpret_cast<const uint4 *>(x + static_cast<long>(g) * K + k) + i);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          xb[c][4 * i + e] = u[e];
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(u[e] << 16)),
                                   fabsf(__uint_as_float(u[e] & 0xFFFF0000u))));
        }
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // -127 for zero
    const int sh = min(14 - ex, 126);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - sh) << 23);
    inv0 = __shfl_sync(0xffffffffu, inv, 8 * t);
    inv1 = __shfl_sync(0xffffffffu, inv, 8 * t + 4);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const __half2 h = __floats2half2_rn(__uint_as_float(xb[c][i] << 16) * up,
                                            __uint_as_float(xb[c][i] & 0xFFFF0000u) * up);
        xb[c][i] = *reinterpret_cast<const uint32_t *>(&h);
      }
  }

  // items of this cluster: its row tiles, gate then up for DUAL
  const int local_tiles = (n_tiles - cl + n_cl - 1) / n_cl;
  const int items = local_tiles * MATS;
  struct Tile {
    uint4 q[C][2];
    uint32_t s[C][2];  // two scale bytes each
  };
  auto fetch = [&](int it, Tile &a) {
    const MatvecWeights &w = (DUAL && (it & 1)) ? w1 : w0;
    const int tile = cl + (it / MATS) * n_cl;
    const int base = (tile >> 3) * 128, j4 = 4 * (tile & 7) + (g & 3);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int k = (c0 + c) * MATVEC_CHUNK + 32 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int quarter = (g >> 2) + 2 * h;
        const int row = base + 32 * quarter + j4;
        a.q[c][h] = make_uint4(0, 0, 0, 0);
        a.s[c][h] = 0;
        if (c0 + c < c1 && k < K && row < N) {
          a.q[c][h] = ldg_stream(w.codes + static_cast<long>(row) * (K / 2) + k / 2);
          const uint8_t *sp = w.sf + 512 * (static_cast<long>(tile >> 3) * (K / 64) + k / 64) +
                              16 * j4 + 4 * quarter + 2 * (t & 1);
          a.s[c][h] = __ldg(reinterpret_cast<const unsigned short *>(sp));
        }
      }
    }
  };

  Tile cur, nxt;
  if (items > 0) fetch(0, cur);
  float gate = 0.0f;
  for (int it = 0; it < items; ++it) {
    if (it + 1 < items) fetch(it + 1, nxt);
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      uint32_t s[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(static_cast<uint16_t>(cur.s[c][h])));
        s[h][0] = __byte_perm(f, 0, 0x1010);
        s[h][1] = __byte_perm(f, 0, 0x3232);
      }
      const uint32_t qa[4] = {cur.q[c][0].x, cur.q[c][0].y, cur.q[c][0].z, cur.q[c][0].w};
      const uint32_t qb[4] = {cur.q[c][1].x, cur.q[c][1].y, cur.q[c][1].z, cur.q[c][1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // 8 codes: two MMAs; words 0, 1 are group 0, 2, 3 group 1
        const uint32_t sa = s[0][i >> 1], sb = s[1][i >> 1];
        mma_f16(acc, hmul2_u(e2m1x2_to_f16x2<0>(qa[i]), sa), hmul2_u(e2m1x2_to_f16x2<0>(qb[i]), sb),
                hmul2_u(e2m1x2_to_f16x2<1>(qa[i]), sa), hmul2_u(e2m1x2_to_f16x2<1>(qb[i]), sb),
                xb[c][4 * i], xb[c][4 * i + 1]);
        mma_f16(acc, hmul2_u(e2m1x2_to_f16x2<2>(qa[i]), sa), hmul2_u(e2m1x2_to_f16x2<2>(qb[i]), sb),
                hmul2_u(e2m1x2_to_f16x2<3>(qa[i]), sa), hmul2_u(e2m1x2_to_f16x2<3>(qb[i]), sb),
                xb[c][4 * i + 2], xb[c][4 * i + 3]);
      }
    }
    cur = nxt;
    float *rw = red[it & 1][warp];
    *reinterpret_cast<float2 *>(rw + 8 * g + 2 * t) = make_float2(acc[0] * inv0, acc[1] * inv1);
    *reinterpret_cast<float2 *>(rw + 8 * (g + 8) + 2 * t) =
        make_float2(acc[2] * inv0, acc[3] * inv1);
    __syncthreads();
    const int o = threadIdx.x;  // tile row o / 8, token o % 8
    const int mat = DUAL ? it & 1 : 0;
    const int lt = it / MATS;  // local tile
    auto finish = [&](int tl, float v0, float v1) {
      const int tile = cl + tl * n_cl, rho = o >> 3, m = o & 7;
      const int row = (tile >> 3) * 128 + 32 * (rho >> 2) + 4 * (tile & 7) + (rho & 3);
      if (row >= N || m >= M) return;
      float v;
      if constexpr (DUAL)
        v = silu_f(v0 * __ldg(w0.scale + row)) * (v1 * __ldg(w1.scale + row));
      else
        v = fmaf(v0, __ldg(w0.scale + row), bias != nullptr ? __ldg(bias + row) : 0.0f);
      OT *op = out + static_cast<long>(m) * N + row;
      if constexpr (sizeof(OT) == 4)
        *op = v;
      else
        *op = __float2bfloat16_rn(v);
    };
    if (o < 128) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < MATVEC_WARPS; ++w) v += red[it & 1][w][o];
      if (cluster > 1)
        psum[(lt / MATVEC_BATCH) & 1][lt % MATVEC_BATCH][mat][o] = v;
      else if (DUAL && mat == 0)
        gate = v;
      else
        DUAL ? finish(lt, gate, v) : finish(lt, v, 0.0f);
    }
    // the cluster's CTAs add up a batch of tiles, each every `cluster`th one; a
    // buffer is written again two batches later, after the next batch's barrier
    if (cluster > 1 && mat == MATS - 1 &&
        (lt % MATVEC_BATCH == MATVEC_BATCH - 1 || lt == local_tiles - 1)) {
      cluster_sync_all();
      if (o < 128) {
        const int b = lt / MATVEC_BATCH;
        for (int i = rank; i <= lt % MATVEC_BATCH; i += cluster) {
          float v[2] = {0.0f, 0.0f};
          for (int q = 0; q < cluster; ++q)
#pragma unroll
            for (int m = 0; m < MATS; ++m)
              v[m] += ld_cluster_f32(map_shared_to_rank(&psum[b & 1][i][m][o], q));
          finish(b * MATVEC_BATCH + i, v[0], v[1]);
        }
      }
      __syncwarp();
    }
  }
  if (cluster > 1) cluster_sync_all();  // shared memory stays until the last remote read
}

}  // namespace ig4
