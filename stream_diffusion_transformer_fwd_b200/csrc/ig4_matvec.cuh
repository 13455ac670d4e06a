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
// exact.  x (8 significant bits) is multiplied by a power of two per row and 128
// elements that brings their largest into [2^14, 2^15) before it becomes fp16:
// exact down to 2^-28 of that element, rounded at 2^-39 of it below.  Sums are
// fp32.
//
// The 8 warps of a CTA split K in runs of 128-element chunks and add their sums
// per 16-row tile; for large x (M K) or few weight rows the CTAs of a cluster
// split K further and exchange partial sums through distributed shared memory.
// x is converted once per CTA into shared memory in the order the MMAs take it
// (with x slices in registers instead, 126 registers a thread left 16 warps on an
// SM and the issue slots half empty).  Weights arrive by cp.async in a ring of
// shared-memory stages of one chunk per warp; a lane copies what it will read
// itself, so the ring needs no barrier, and the first stages are on their way
// before x is read.  16-row tiles take rows {4j .. 4j+3} + {0, 32, 64, 96} of a
// 128-row block: their 16 scale words of a k-block are then 64 consecutive bytes
// in the packed order.
#pragma once

#include <cuda_fp16.h>

#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int MATVEC_WARPS = 8;
constexpr int MATVEC_THREADS = 32 * MATVEC_WARPS;
constexpr int MATVEC_CHUNK = 128;    // k elements of a warp step: 4 lanes x 32
constexpr int MATVEC_MAX_CLUSTER = 8;
constexpr int MATVEC_BATCH = 4;      // items per exchange between the CTAs of a cluster
constexpr int MATVEC_CVT_WORDS = 3;  // of a lane's four code words
constexpr int MATVEC_CTAS = 2;       // on an SM
constexpr int MATVEC_STAGES = 4;
// a stage: per warp and row half 32 x 16 code bytes, then 32 x 4 scale bytes
constexpr int MATVEC_UNIT_BYTES = 32 * 16 + 32 * 4;
constexpr int MATVEC_RING_BYTES = MATVEC_STAGES * MATVEC_WARPS * 2 * MATVEC_UNIT_BYTES;
// x of one CTA: per chunk and row 256 bytes of fp16 and the fp32 that undoes its scale
__host__ __device__ constexpr int matvec_x_bytes(int chunks, int M) { return chunks * M * 260; }
constexpr int MATVEC_MAX_X_BYTES = 50 << 10;
constexpr int MATVEC_MAX_K = 24576;  // 8 rows of it over the largest cluster stay under that
constexpr int MATVEC_SM_SMEM = 227 << 10;
constexpr int MATVEC_STATIC_SMEM = (21 << 10);  // partial sums, and what the system reserves

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

// DUAL: w0 gate, w1 up.
template <bool DUAL, typename OT>
__global__ void __launch_bounds__(MATVEC_THREADS, MATVEC_CTAS)
    nvfp4_matvec_kernel(const __nv_bfloat16 *x, MatvecWeights w0, MatvecWeights w1,
                        const float *bias, OT *out, int M, int N, int K, int n_tiles, int cluster) {
  constexpr int MATS = DUAL ? 2 : 1;
  constexpr int BATCH = MATVEC_BATCH / MATS;
  extern __shared__ uint4 mv_smem[];  // ring, x fragments, x scales
  __shared__ float red[2][2][MATVEC_WARPS][128];
  __shared__ float psum[2][BATCH][MATS][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cl = blockIdx.x / cluster, n_cl = gridDim.x / cluster;
  pdl_wait();
  pdl_trigger();

  // this CTA's chunks, and this warp's run [c0, c0 + nch) of them
  const int nc = (K + MATVEC_CHUNK - 1) / MATVEC_CHUNK;
  const int cta0 = nc * rank / cluster, cta_nc = nc * (rank + 1) / cluster - cta0;
  const int r0 = cta_nc * warp / MATVEC_WARPS;
  const int nch = cta_nc * (warp + 1) / MATVEC_WARPS - r0;
  const int c0 = cta0 + r0;

  // items of this cluster: its row tiles, gate then up for DUAL
  const int local_tiles = (n_tiles - cl + n_cl - 1) / n_cl;
  const int items = local_tiles * MATS;

  // The copies run MATVEC_STAGES - 1 steps (chunks) ahead of the products.  A
  // lane's unit: row half h holds weight rows g and g + 8 of the tile, two
  // 32-row quarters apart.  Rows past N read row N - 1 and are not stored; lanes
  // whose half of the last chunk is past K read the other half and have zero x.
  uint8_t *wring = reinterpret_cast<uint8_t *>(mv_smem) + warp * 2 * MATVEC_UNIT_BYTES;
  constexpr int STAGE = MATVEC_WARPS * 2 * MATVEC_UNIT_BYTES;
  const bool past = K % MATVEC_CHUNK != 0 && c0 + nch == nc && t >= 2;  // in chunk nch - 1
  const uint8_t *cp0 = nullptr, *cp1 = nullptr, *sp = nullptr;
  int f_item = 0, f_chunk = 0, f_stage = 0;
  auto fetch = [&]() {
    if (f_item < items && nch > 0) {
      if (f_chunk == 0) {
        const MatvecWeights &w = (DUAL && (f_item & 1)) ? w1 : w0;
        const int tile = cl + (f_item / MATS) * n_cl;
        const int j4 = 4 * (tile & 7) + (g & 3);
        const int row = (tile >> 3) * 128 + 32 * (g >> 2) + j4;
        const uint8_t *base = w.codes + c0 * 64 + 16 * t;
        cp0 = base + static_cast<long>(min(row, N - 1)) * (K / 2);
        cp1 = base + static_cast<long>(min(row + 64, N - 1)) * (K / 2);
        sp = w.sf + 512 * (static_cast<long>(tile >> 3) * (K / 64) + 2 * c0 + (t >> 1)) + 16 * j4 +
             4 * (g >> 2);
      }
      uint8_t *u = wring + f_stage * STAGE;
      const int back = past && f_chunk == nch - 1 ? 32 : 0;
      cp_async16(u + 16 * lane, cp0 - back);
      cp_async16(u + MATVEC_UNIT_BYTES + 16 * lane, cp1 - back);
      cp_async4(u + 512 + 4 * lane, sp - 16 * back);
      cp_async4(u + MATVEC_UNIT_BYTES + 512 + 4 * lane, sp - 16 * back + 8);
      cp0 += 64;
      cp1 += 64;
      sp += 1024;
      if (++f_chunk == nch) {
        f_chunk = 0;
        ++f_item;
      }
      if (++f_stage == MATVEC_STAGES) f_stage = 0;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < MATVEC_STAGES - 1; ++i) fetch();

  // x into shared memory: 8 elements (what a code word multiplies) of row m are
  // one uint4 at [chunk][word][m][lane t], 16 threads a chunk of a row
  uint4 *xs = reinterpret_cast<uint4 *>(reinterpret_cast<uint8_t *>(mv_smem) + MATVEC_RING_BYTES);
  float *xinv = reinterpret_cast<float *>(xs + cta_nc * M * 16);
  for (int base = 0; base < cta_nc * M * 16; base += MATVEC_THREADS) {
    const int i = base + threadIdx.x;
    const int c = i / (16 * M), m = (i >> 4) - c * M, e = i & 15;
    const int k = (cta0 + c) * MATVEC_CHUNK + 8 * e;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (i < cta_nc * M * 16 && k < K)
      v = __ldg(reinterpret_cast<const uint4 *>(x + static_cast<long>(m) * K + k));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    float amax = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      amax = fmax3(amax, fabsf(__uint_as_float(u[q] << 16)),
                   fabsf(__uint_as_float(u[q] & 0xFFFF0000u)));
#pragma unroll
    for (int q = 1; q < 16; q *= 2) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, q));
    const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;  // -127 for zero
    const int sh = min(14 - ex, 126);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
    uint32_t p[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __half2 h = __floats2half2_rn(__uint_as_float(u[q] << 16) * up,
                                          __uint_as_float(u[q] & 0xFFFF0000u) * up);
      p[q] = *reinterpret_cast<const uint32_t *>(&h);
    }
    const int word = e & 3;
    // the integer way yields codes (0, 4), (1, 5), (2, 6), (3, 7) of a word
    v = word < MATVEC_CVT_WORDS
            ? make_uint4(p[0], p[1], p[2], p[3])
            : make_uint4(__byte_perm(p[0], p[2], 0x5410), __byte_perm(p[0], p[2], 0x7632),
                         __byte_perm(p[1], p[3], 0x5410), __byte_perm(p[1], p[3], 0x7632));
    if (i < cta_nc * M * 16) {
      xs[((c * 4 + word) * M + m) * 4 + (e >> 2)] = v;
      // undoes 2^sh and the weights' 2^-9
      if (e == 0) xinv[c * M + m] = __uint_as_float(static_cast<uint32_t>(127 + 9 - sh) << 23);
    }
  }
  __syncthreads();

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
  // fragments of x row g (zero past M), scales of the accumulator's columns
  const uint4 *xw = xs + (r0 * 4 * M + g) * 4 + t;
  const float *xi = xinv + r0 * M;
  int stage = 0;
  // two items per step: gate and up of a tile, or two tiles
  for (int i0 = 0; i0 < items; i0 += 2) {
    const int par = (i0 >> 1) & 1;
#pragma unroll 1
    for (int it = i0; it < i0 + 2 && it < items; ++it) {
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (int c = 0; c < nch; ++c) {
        cp_async_wait<MATVEC_STAGES - 2>();
        fetch();
        const uint8_t *st = wring + stage * STAGE;
        if (++stage == MATVEC_STAGES) stage = 0;
        uint32_t s[2][2];  // row half, group
        uint4 q[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint8_t *u = st + h * MATVEC_UNIT_BYTES;
          q[h] = *reinterpret_cast<const uint4 *>(u + 16 * lane);
          const uint16_t two = *reinterpret_cast<const uint16_t *>(u + 512 + 4 * lane + 2 * (t & 1));
          uint32_t f;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"(two));
          s[h][0] = __byte_perm(f, 0, 0x1010);
          s[h][1] = __byte_perm(f, 0, 0x3232);
        }
        const uint32_t qa[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
        const uint32_t qb[4] = {q[1].x, q[1].y, q[1].z, q[1].w};
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // words 0, 1 are group 0, words 2, 3 group 1
          const bool cvt = i < MATVEC_CVT_WORDS;
          const uint32_t f = cvt ? 0x18001800u : 0x50005000u;  // 2^-9 or 2^5
          const uint32_t sa = hmul2_u(s[0][i >> 1], f), sb = hmul2_u(s[1][i >> 1], f);
          const uint4 xv = g < M ? xw[(c * 4 + i) * M * 4] : make_uint4(0, 0, 0, 0);
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
                  xv.x, xv.y);
          mma_f16(acc, hmul2_u(a[2], sa), hmul2_u(b[2], sb), hmul2_u(a[3], sa), hmul2_u(b[3], sb),
                  xv.z, xv.w);
        }
        // columns 2t, 2t + 1 (their products are zero past M)
        const float v0 = 2 * t < M ? xi[c * M + 2 * t] : 0.0f;
        const float v1 = 2 * t + 1 < M ? xi[c * M + 2 * t + 1] : 0.0f;
        sum[0] = fmaf(acc[0], v0, sum[0]);
        sum[1] = fmaf(acc[1], v1, sum[1]);
        sum[2] = fmaf(acc[2], v0, sum[2]);
        sum[3] = fmaf(acc[3], v1, sum[3]);
      }
      float *rw = red[par][it & 1][warp];
      *reinterpret_cast<float2 *>(rw + 8 * g + 2 * t) = make_float2(sum[0], sum[1]);
      *reinterpret_cast<float2 *>(rw + 8 * (g + 8) + 2 * t) = make_float2(sum[2], sum[3]);
    }
    __syncthreads();
    // thread (half, o) sums output o of item i0 + half over the warps; for DUAL
    // the first half takes both
    const int half = threadIdx.x >> 7;
    float v[MATS];
#pragma unroll
    for (int m = 0; m < MATS; ++m) {
      v[m] = 0.0f;
#pragma unroll
      for (int w = 0; w < MATVEC_WARPS; ++w) v[m] += red[par][DUAL ? m : half][w][o];
    }
    const int lt = DUAL ? i0 >> 1 : i0 + half;  // local tile
    if (lt < local_tiles && (!DUAL || half == 0)) {
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
      for (int i = 2 * rank + half; i <= (done - 1) % BATCH; i += 2 * cluster) {
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
