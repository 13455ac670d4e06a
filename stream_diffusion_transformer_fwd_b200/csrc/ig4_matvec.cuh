// ig4_matvec.cuh - 1 to 8 bf16 rows times NVFP4 weights (E2M1 codes, an E4M3
// scale per 16 weights, an fp32 scale per output), alone or as the gated pair
// of a feed-forward layer: u = silu(x Wg^T) * (x Wu^T).
//
// Each weight is used M <= 8 times, so the weight bytes (4.5 bits per weight)
// would bound it, 41 weights a clock and SM; what does is the products' rate.
// They run on mma.sync m16n8k16, the weights as the 16-row operand and the M
// rows as its 8 columns: a lane's 16 loaded bytes become its own operand
// registers, with nothing staged between decoding and product.  That instruction
// takes 32 clocks of a quarter SM here: 32 weights a clock and SM, 21 reached
// (16384 x 12288 weights: 35 us; 4608 x 12288: 13.1 us).  Decoding into tensor
// memory for tcgen05.mma instead, which has no such limit, took 25 us for the
// latter: its hand-shakes per 64 elements and a CTA's start cost more than they
// gain at these sizes.
//
// The order of the contraction is free: lane (g, t) of a warp takes 32
// consecutive codes of weight rows g and g + 8 (one 16-byte load each) and the
// same 32 elements of x row g, four per MMA, paired as its codes come out.
//
// Codes become fp16 pairs two ways.  cvt.f16x2.e2m1x2 takes two codes per
// instruction, but at 16 lanes per clock and SM: with it alone that pipe was 80%
// busy and bounded the kernel.  Or in the integer pipe: a nibble s|ee|m moved to
// bits 15 and 11..9 is the fp16 number +-code * 2^-14 (the exponent field ee and
// one mantissa bit; ee = 0 is an fp16 subnormal, as it should be), two masks and
// two shifts for a pair.  MATVEC_CVT_WORDS of a lane's four 8-code words take the
// first way, which keeps both pipes below the weights' time.
//
// Exactness: code times group scale has at most 6 significant bits between
// 2^-10 and 2688; both ways form it times 2^-9 in fp16, between 2^-19 and 5.25:
// exact.  x (8 significant bits) is multiplied by a power of two per row and
// warp that brings its largest element into [2^14, 2^15) before it becomes fp16:
// exact down to 2^-28 of that element, rounded at 2^-39 of it below.  Sums are
// fp32.
//
// Weights arrive by cp.async in a ring of shared-memory stages; a lane copies
// what it will read itself, so the ring needs no barrier, and the first stages
// are on their way before x is read.  (With one tile prefetched into registers
// 4608 x 12288 weights took 18 us.)  A warp keeps its slice of x in registers for
// all the weight rows it meets (read from shared memory per use, x of 8 rows made
// the gated pair at full width take 33 us instead of 28); a CTA's 8 to 16 warps
// split K, and for long K (or few rows) the CTAs of a cluster split it further and
// exchange partial sums through distributed shared memory.  16-row tiles take rows
// {4j .. 4j+3} + {0, 32, 64, 96} of a 128-row block: their 16 scale words of a
// k-block are then 64 consecutive bytes in the packed order.
#pragma once

#include <cuda_fp16.h>

#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int MATVEC_MIN_WARPS = 8;  // two CTAs of these fit an SM, one of more warps
constexpr int MATVEC_MAX_WARPS = 16;
constexpr int MATVEC_CHUNK = 128;    // k elements of a warp step: 4 lanes x 32
constexpr int MATVEC_MAX_CHUNKS = 3; // per warp
constexpr int MATVEC_MAX_CLUSTER = 8;
constexpr int MATVEC_MAX_K = 24576;  // what the widest clusters of the fewest warps hold
constexpr int MATVEC_BATCH = 4;      // row tiles per exchange between the CTAs of a cluster
constexpr int MATVEC_CVT_WORDS = 3;  // of a lane's four code words
constexpr int MATVEC_STAGES = 3;
// a stage: per warp, chunk and row half 32 x 16 code bytes, then 32 x 4 scale bytes
constexpr int MATVEC_UNIT_BYTES = 32 * 16 + 32 * 4;
__host__ __device__ constexpr int matvec_stage_bytes(int chunks, int warps) {
  return warps * chunks * 2 * MATVEC_UNIT_BYTES;
}
// the ring, then the warps' sums of two items, twice
__host__ __device__ constexpr int matvec_smem(int chunks, int warps) {
  return MATVEC_STAGES * matvec_stage_bytes(chunks, warps) + 2 * 2 * warps * 128 * 4;
}

struct MatvecWeights {
  const uint8_t *codes;
  const uint8_t *sf;
  const float *scale;
};

__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// Codes J and J + 4 of a word (nibble 0 lowest) times 2^-14 as an fp16 pair
template <int J>
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w) {
  const uint32_t mag = J < 3 ? w << (J < 3 ? 9 - 4 * J : 0) : w >> 3;
  const uint32_t sign = w << (12 - 4 * J);
  return (mag & 0x0E000E00u) | (sign & 0x80008000u);
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
__global__ void __launch_bounds__(32 * MATVEC_MAX_WARPS, 1)
    nvfp4_matvec_kernel(const __nv_bfloat16 *x, MatvecWeights w0, MatvecWeights w1,
                        const float *bias, OT *out, int M, int N, int K, int n_tiles, int cluster) {
  constexpr int MATS = DUAL ? 2 : 1;
  constexpr int BATCH = MATVEC_BATCH / MATS;
  extern __shared__ uint4 ring[];
  const int warps = blockDim.x >> 5;
  const int STAGE = matvec_stage_bytes(C, warps);
  // [parity][item][warp][128]
  float *red = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(ring) + MATVEC_STAGES * STAGE);
  __shared__ float psum[2][BATCH][MATS][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cl = blockIdx.x / cluster, n_cl = gridDim.x / cluster;
  pdl_wait();
  pdl_trigger();

  // this warp's run of chunks
  const int nc = (K + MATVEC_CHUNK - 1) / MATVEC_CHUNK;
  const int slots = cluster * warps, slot = rank * warps + warp;
  const int c0 = nc * slot / slots, c1 = nc * (slot + 1) / slots;  // at most C chunks

  const int nch = c1 - c0;

  // items of this cluster: its row tiles, gate then up for DUAL
  const int local_tiles = (n_tiles - cl + n_cl - 1) / n_cl;
  const int items = local_tiles * MATS;
  // A lane's unit of stage s, chunk c, row half h (weight rows g and g + 8 of the
  // tile, two 32-row quarters apart).  Rows past N read row N - 1 and are not
  // stored; the lanes whose half of the last chunk is past K read the other half
  // and have zero x.
  uint8_t *wring = reinterpret_cast<uint8_t *>(ring) + warp * (C * 2 * MATVEC_UNIT_BYTES);
  const int past = K % MATVEC_CHUNK != 0 && c1 == nc && t >= 2 ? 64 : 0;  // of chunk nch - 1
  auto fetch = [&](int it) {
    if (it < items) {
      const MatvecWeights &w = (DUAL && (it & 1)) ? w1 : w0;
      const int tile = cl + (it / MATS) * n_cl;
      const int j4 = 4 * (tile & 7) + (g & 3);
      uint8_t *st = wring + (it % MATVEC_STAGES) * STAGE;
      const uint8_t *sp = w.sf + 512 * (static_cast<long>(tile >> 3) * (K / 64) + 2 * c0 + (t >> 1)) +
                          16 * j4 + 4 * (g >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = min((tile >> 3) * 128 + 32 * (g >> 2) + 64 * h + j4, N - 1);
        const uint8_t *cp = w.codes + static_cast<long>(row) * (K / 2) + c0 * 64 + 16 * t;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (c >= nch) break;
          uint8_t *u = st + (c * 2 + h) * MATVEC_UNIT_BYTES;
          const int back = c == nch - 1 ? past : 0;
          cp_async16(u + 16 * lane, cp + c * 64 - back / 2);
          cp_async4(u + 512 + 4 * lane, sp + c * 1024 + 8 * h - back * 8);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < MATVEC_STAGES - 1; ++i) fetch(i);

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
    const float inv = __uint_as_float(static_cast<uint32_t>(127 + 9 - sh) << 23);
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
    // the integer way yields codes (0, 4), (1, 5), (2, 6), (3, 7) of a word
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 4 * MATVEC_CVT_WORDS; i < 16; i += 4) {
        const uint32_t p0 = xb[c][i], p1 = xb[c][i + 1], p2 = xb[c][i + 2], p3 = xb[c][i + 3];
        xb[c][i] = __byte_perm(p0, p2, 0x5410);
        xb[c][i + 1] = __byte_perm(p0, p2, 0x7632);
        xb[c][i + 2] = __byte_perm(p1, p3, 0x5410);
        xb[c][i + 3] = __byte_perm(p1, p3, 0x7632);
      }
  }

  const int o = threadIdx.x & 127;  // output of a tile: row o / 8, token o % 8
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
  // two items per step: gate and up of a tile, or two tiles
  for (int i0 = 0; i0 < items; i0 += 2) {
    const int par = (i0 >> 1) & 1;
#pragma unroll 1
    for (int it = i0; it < i0 + 2 && it < items; ++it) {
      cp_async_wait<MATVEC_STAGES - 2>();
      fetch(it + MATVEC_STAGES - 1);
      const uint8_t *st = wring + (it % MATVEC_STAGES) * STAGE;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (c >= nch) break;
        uint32_t s[2][2];  // row half, group
        uint4 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *u = st + (c * 2 + h) * MATVEC_UNIT_BYTES;
          q[h] = *reinterpret_cast<const uint4 *>(u + 16 * lane);
          const uint16_t two = *reinterpret_cast<const uint16_t *>(u + 512 + 4 * lane + 2 * (t & 1));
          uint32_t f;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(two));
          s[h][0] = __byte_perm(f, 0, 0x1010);
          s[h][1] = __byte_perm(f, 0, 0x3232);
        }
        const uint32_t qa[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
        const uint32_t qb[4] = {q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // words 0, 1 are group 0, words 2, 3 group 1
          const bool cvt = i < MATVEC_CVT_WORDS;
          const uint32_t f = cvt ? 0x18001800u : 0x50005000u;  // 2^-9 or 2^5
          const uint32_t sa = hmul2_u(s[0][i >> 1], f), sb = hmul2_u(s[1][i >> 1], f);
          uint32_t a[4], b[4];
          if (cvt) {
            a[0] = e2m1x2_to_f16x2<0>(qa[i]);
            a[1] = e2m1x2_to_f16x2<1>(qa[i]);
            a[2] = e2m1x2_to_f16x2<2>(qa[i]);
            a[3] = e2m1x2_to_f16x2<3>(qa[i]);
            b[0] = e2m1x2_to_f16x2<0>(qb[i]);
            b[1] = e2m1x2_to_f16x2<1>(qb[i]);
            b[2] = e2m1x2_to_f16x2<2>(qb[i]);
            b[3] = e2m1x2_to_f16x2<3>(qb[i]);
          } else {
            a[0] = e2m1_pair<0>(qa[i]);
            a[1] = e2m1_pair<1>(qa[i]);
            a[2] = e2m1_pair<2>(qa[i]);
            a[3] = e2m1_pair<3>(qa[i]);
            b[0] = e2m1_pair<0>(qb[i]);
            b[1] = e2m1_pair<1>(qb[i]);
            b[2] = e2m1_pair<2>(qb[i]);
            b[3] = e2m1_pair<3>(qb[i]);
          }
          mma_f16(acc, hmul2_u(a[0], sa), hmul2_u(b[0], sb), hmul2_u(a[1], sa), hmul2_u(b[1], sb),
                  xb[c][4 * i], xb[c][4 * i + 1]);
          mma_f16(acc, hmul2_u(a[2], sa), hmul2_u(b[2], sb), hmul2_u(a[3], sa), hmul2_u(b[3], sb),
                  xb[c][4 * i + 2], xb[c][4 * i + 3]);
        }
      }
      float *rw = red + ((2 * par + (it & 1)) * warps + warp) * 128;
      *reinterpret_cast<float2 *>(rw + 8 * g + 2 * t) = make_float2(acc[0] * inv0, acc[1] * inv1);
      *reinterpret_cast<float2 *>(rw + 8 * (g + 8) + 2 * t) =
          make_float2(acc[2] * inv0, acc[3] * inv1);
    }
    __syncthreads();
    // thread (half, o) sums output o of item i0 + half over the warps; for DUAL
    // the first half takes both
    const int half = threadIdx.x >> 7;  // (threads from 256 on have none)
    float v[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      v[m] = 0.0f;
      const float *rs = red + (2 * par + (DUAL ? m : half & 1)) * warps * 128 + o;
#pragma unroll 8
      for (int w = 0; w < warps; ++w) v[m] += rs[w * 128];
    }
    const int lt = DUAL ? i0 >> 1 : i0 + half;  // local tile
    if (lt < local_tiles && half < (DUAL ? 1 : 2)) {
      if (cluster == 1) {
        finish(lt, v[0], v[MATS - 1]);
      } else {
#pragma unroll
        for (int m = 0; m < MATS; ++m) psum[(lt / BATCH) & 1][lt % BATCH][m][o] = v[m];
      }
    }
    // the cluster's CTAs add up a batch of tiles, each every `cluster`th one; a
    // buffer is written again two batches later, after the next batch's barrier
    const int done = DUAL ? (i0 >> 1) + 1 : min(i0 + 2, local_tiles);
    if (cluster > 1 && (done % BATCH == 0 || done == local_tiles)) {
      cluster_sync_all();
      const int b = (done - 1) / BATCH;
      for (int i = 2 * rank + half; half < 2 && i <= (done - 1) % BATCH; i += 2 * cluster) {
        float z[2] = {0.0f, 0.0f};
        for (int q = 0; q < cluster; ++q)
#pragma unroll
          for (int m = 0; m < MATS; ++m)
            z[m] += ld_cluster_f32(map_shared_to_rank(&psum[b & 1][i][m][o], q));
        finish(b * BATCH + i, z[0], z[MATS - 1]);
      }
      __syncwarp();
    }
  }
  if (cluster > 1) cluster_sync_all();  // shared memory stays until the last remote read
}

}  // namespace ig4
