// ig4_addnorm.cuh - residual addition + RMSNorm with bf16, fp32 or FP8 output,
// and its gradients.
//
//   t = x + r;  s = RN(t);  y = t * rsqrt(mean(t^2) + eps) * g
//   dx = rstd (dy g - n mean(dy g n)) + ds,  n = s rstd;   dg = sum_rows dy n
//
// Both directions move a few bytes per multiply, so HBM bandwidth bounds them
// (latency for a handful of rows).  Every row is read once and stays in
// registers between its reduction and its output: 8-element vectors, NV per
// thread, a warp per row up to D = 512 and a CTA per row above.  A CTA walks
// rows with a grid stride and issues the next row's loads before it reduces
// the current one, so loads stay in flight across the block reduction; the
// weight g is loaded into registers once per CTA.
#pragma once

#include "ig4_mx8.cuh"
#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int ADDNORM_WARP_D = 512;       // up to this width a warp takes a row
constexpr int ADDNORM_WARPS = 4;          // warps (rows) per CTA in that form
constexpr int ADDNORM_MAX_THREADS = 512;  // CTA-per-row form: D <= 8192 with NV = 2
constexpr int ADDNORM_NV = 2;

enum AddNormOut { ADDNORM_BF16 = 0, ADDNORM_F32 = 1, ADDNORM_ROW8 = 2, ADDNORM_MX8 = 3 };

// 8 consecutive elements as loaded
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    q = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8_e4m3(uint8_t *p, const float (&v)[8]) {
  uint2 w;
  w.x = static_cast<uint32_t>(pack_e4m3x2(v[0], v[1])) |
        (static_cast<uint32_t>(pack_e4m3x2(v[2], v[3])) << 16);
  w.y = static_cast<uint32_t>(pack_e4m3x2(v[4], v[5])) |
        (static_cast<uint32_t>(pack_e4m3x2(v[6], v[7])) << 16);
  *reinterpret_cast<uint2 *>(p) = w;
}

// Weight of vector vi (1 without a weight)
__device__ __forceinline__ void load_g8(const float *g, int vi, float (&v)[8]) {
  if (g == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 1.0f;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4 *>(g) + 2 * vi);
  const float4 b = __ldg(reinterpret_cast<const float4 *>(g) + 2 * vi + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// Reductions over the threads of a row.  In the CTA form each call takes its
// own slots of `red` (callers alternate two sets, so one __syncthreads per
// reduction is enough); every thread adds the warps' values in the same order.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float *red) {
  v = warp_sum(v);
  if constexpr (!WARP) {
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < nw; ++w) v += red[w];
  }
  return v;
}
template <bool WARP>
__device__ __forceinline__ float row_max(float v, float *red) {
  v = warp_max(v);
  if constexpr (!WARP) {
    const int nw = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < nw; ++w) v = fmaxf(v, red[w]);
  }
  return v;
}

template <typename XT, int OUT, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ADDNORM_WARPS : ADDNORM_MAX_THREADS)
    add_rms_norm_kernel(const XT *x, const XT *r, const float *g, float eps, XT *s_out, void *y_out,
                        float *y_scale, uint8_t *y_sf, int M, int D) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[4][ADDNORM_MAX_THREADS / 32];
  const int T = WARP ? 32 : static_cast<int>(blockDim.x);
  const int tid = WARP ? (threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int nvec = D / 8;
  const long step = static_cast<long>(gridDim.x) * (WARP ? ADDNORM_WARPS : 1);
  long row = WARP ? static_cast<long>(blockIdx.x) * ADDNORM_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  float gv[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + T * i < nvec) load_g8(g, tid + T * i, gv[i]);
  Raw8<XT> cx[NV], cr[NV], nx[NV], nr[NV];
  auto fetch = [&](long rw, Raw8<XT>(&a)[NV], Raw8<XT>(&b)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      a[i].zero();
      b[i].zero();
      if (vi < nvec) {
        a[i].load(x + rw * D + 8 * vi);
        if (r != nullptr) b[i].load(r + rw * D + 8 * vi);
      }
    }
  };
  if (row < M) fetch(row, cx, cr);
  int par = 0;
  for (; row < M; row += step, par ^= 1) {
    if (row + step < M) fetch(row + step, nx, nr);
    float t[NV][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float b[8];
      cx[i].get(t[i]);
      cr[i].get(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[i][e] += b[e];
        ss = fmaf(t[i][e], t[i][e], ss);
      }
    }
    if (s_out != nullptr) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + T * i < nvec) store8(s_out + row * D + 8 * (tid + T * i), t[i]);
    }
    ss = row_sum<WARP>(ss, red[par]);
    const float rstd = rsqrtf(ss / static_cast<float>(D) + eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) t[i][e] = tid + T * i < nvec ? t[i][e] * rstd * gv[i][e] : 0.0f;
    if constexpr (OUT == ADDNORM_BF16 || OUT == ADDNORM_F32) {
      using YT = typename std::conditional<OUT == ADDNORM_BF16, __nv_bfloat16, float>::type;
      YT *yr = static_cast<YT *>(y_out) + row * D;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (tid + T * i < nvec) store8(yr + 8 * (tid + T * i), t[i]);
    } else if constexpr (OUT == ADDNORM_ROW8) {
      // scale = max|y| / 448 (1 for a zero row), codes of the fp32 y
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(t[i][e]));
      amax = row_max<WARP>(amax, red[2 + par]);
      const float qs = amax > 0.0f ? amax / 448.0f : 1.0f;
      const float inv = 1.0f / qs;
      uint8_t *yr = static_cast<uint8_t *>(y_out) + row * D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (tid + T * i < nvec) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[i][e] *= inv;
          store8_e4m3(yr + 8 * (tid + T * i), t[i]);
        }
      }
      if (tid == 0) y_scale[row] = qs;
    } else {
      // 32-element blocks: four neighbouring lanes; 16 lanes make the 4 scale
      // bytes of one 128-element k-block, stored as one word
      uint8_t *yr = static_cast<uint8_t *>(y_out) + row * D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vi = tid + T * i;
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          t[i][e] = bf16_round(t[i][e]);
          amax = fmaxf(amax, fabsf(t[i][e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int ex = mx8_exponent(amax);
        const float inv = mx8_inv_scale(ex);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[i][e] *= inv;
        uint32_t w = static_cast<uint32_t>(ex + 127) << (8 * ((threadIdx.x >> 2) & 3));
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        w |= __shfl_xor_sync(0xffffffffu, w, 8);
        if (vi < nvec) {
          store8_e4m3(yr + 8 * vi, t[i]);
          if ((threadIdx.x & 15) == 0)
            *reinterpret_cast<uint32_t *>(y_sf + mx8_sf_offset(static_cast<int>(row), vi / 4, D)) = w;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      cx[i] = nx[i];
      cr[i] = nr[i];
    }
  }
}

// Gradients.  A thread keeps the same columns for every row it sees, so dg
// accumulates in its registers; each CTA then writes one partial row of dg,
// and add_rms_norm_dg_kernel adds the partial rows in a fixed order (no
// atomics: the same inputs give the same bits).
template <typename XT, typename YT, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * ADDNORM_WARPS : ADDNORM_MAX_THREADS)
    add_rms_norm_grad_kernel(const XT *s, const float *g, float eps, const YT *dy, const XT *ds,
                             XT *dx, float *dg_part, int M, int D) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[4][ADDNORM_MAX_THREADS / 32];
  __shared__ float acc_s[WARP ? ADDNORM_WARPS * ADDNORM_WARP_D : 1];
  const int T = WARP ? 32 : static_cast<int>(blockDim.x);
  const int tid = WARP ? (threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int nvec = D / 8;
  const long step = static_cast<long>(gridDim.x) * (WARP ? ADDNORM_WARPS : 1);
  long row = WARP ? static_cast<long>(blockIdx.x) * ADDNORM_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  float gv[NV][8], acc[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = gv[i][e] = 0.0f;
    if (tid + T * i < nvec) load_g8(g, tid + T * i, gv[i]);
  }
  Raw8<XT> cs[NV], cd[NV], ns[NV], nd[NV];
  Raw8<YT> cy[NV], ny[NV];
  auto fetch = [&](long rw, Raw8<XT>(&a)[NV], Raw8<YT>(&b)[NV], Raw8<XT>(&c)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      a[i].zero();
      b[i].zero();
      c[i].zero();
      if (vi < nvec) {
        a[i].load(s + rw * D + 8 * vi);
        b[i].load(dy + rw * D + 8 * vi);
        if (ds != nullptr) c[i].load(ds + rw * D + 8 * vi);
      }
    }
  };
  if (row < M) fetch(row, cs, cy, cd);
  int par = 0;
  for (; row < M; row += step, par ^= 1) {
    if (row + step < M) fetch(row + step, ns, ny, nd);
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8];
      cs[i].get(a);
      cy[i].get(b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ss = fmaf(a[e], a[e], ss);
        dot = fmaf(b[e] * gv[i][e], a[e], dot);
      }
    }
    ss = warp_sum(ss);
    dot = warp_sum(dot);
    if constexpr (!WARP) {
      const int nw = blockDim.x >> 5;
      if ((threadIdx.x & 31) == 0) {
        red[par][threadIdx.x >> 5] = ss;
        red[2 + par][threadIdx.x >> 5] = dot;
      }
      __syncthreads();
      ss = dot = 0.0f;
      for (int w = 0; w < nw; ++w) {
        ss += red[par][w];
        dot += red[2 + par][w];
      }
    }
    const float rstd = rsqrtf(ss / static_cast<float>(D) + eps);
    const float m = dot * rstd / static_cast<float>(D);  // mean(dy g n)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float a[8], b[8], c[8];
      cs[i].get(a);
      cy[i].get(b);
      cd[i].get(c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = a[e] * rstd;
        acc[i][e] = fmaf(b[e], n, acc[i][e]);
        c[e] = fmaf(rstd, fmaf(b[e], gv[i][e], -n * m), c[e]);
      }
      if (tid + T * i < nvec) store8(dx + row * D + 8 * (tid + T * i), c);
      cs[i] = ns[i];
      cy[i] = ny[i];
      cd[i] = nd[i];
    }
  }
  if (dg_part == nullptr) return;
  float *part = dg_part + static_cast<long>(blockIdx.x) * D;
  if constexpr (WARP) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (tid + T * i < nvec) store8(acc_s + (threadIdx.x >> 5) * D + 8 * (tid + T * i), acc[i]);
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 32 * ADDNORM_WARPS) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < ADDNORM_WARPS; ++w) v += acc_s[w * D + c];
      part[c] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (tid + T * i < nvec) store8(part + 8 * (tid + T * i), acc[i]);
  }
}

// dg[c] = sum over the P partial rows: a CTA takes 32 columns, its 8 warps
// every eighth partial row (128-byte reads), then the 8 sums are added.
constexpr int ADDNORM_DG_THREADS = 256;
__global__ void __launch_bounds__(ADDNORM_DG_THREADS)
    add_rms_norm_dg_kernel(const float *part, int P, int D, float *dg) {
  pdl_wait();
  pdl_trigger();
  __shared__ float red[ADDNORM_DG_THREADS / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < D)
    for (int p = warp; p < P; p += ADDNORM_DG_THREADS / 32) v += part[static_cast<long>(p) * D + c];
  red[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < D) {
#pragma unroll
    for (int w = 1; w < ADDNORM_DG_THREADS / 32; ++w) v += red[w][lane];
    dg[c] = v;
  }
}

}  // namespace ig4
