// ig4_addnorm.cuh - residual addition + RMSNorm with bf16, fp32 or FP8 output,
// and its gradients.
//
//   t = x + r;  s = RN(t);  y = t * rsqrt(mean(t^2) + eps) * g
//   dx = rstd (dy g - n mean(dy g n)) + ds,  n = s rstd;   dg = sum_rows dy n
//
// Both directions move a few bytes per multiply, so HBM bandwidth bounds them
// (latency for a handful of rows).  Every row is read once and stays on chip
// between its reduction and its output.
//
// D > 512: a CTA per row at a time, two 8-element vectors per thread; rows
// arrive in a ring of shared-memory slots by bulk copies (cp.async.bulk), so
// the bytes in flight do not cost registers or depend on how far the threads
// are: with rows prefetched into registers instead, 18 KB per CTA and one row
// ahead, 9216 rows of 4608 reached 4.6 TB/s.  The reduction's barrier doubles
// as the hand-back of the slot: after it every thread has its part of the row
// in registers, and thread 0 issues the row S further on.
// D <= 512: a warp per row, the next row prefetched into registers.
//
// 9216 rows of 4608 bf16, sum and per-row E4M3 out: 53 to 57 us for 297 MB, 5.2 to
// 5.6 TB/s (a plain copy 6.6); issue slots 65% busy.  2047 rows to MX8: 16.2 us, 3 of
// them launch and ramp.  Gradients of 4608 rows with dg: 31 us for the rows (170 MB,
// 5.5 TB/s) and 4 to 5 us for the sum of the partial rows.  18000 rows of 512: 13.2 us.
// One row: 2.3 us.
#pragma once

#include <type_traits>

#include "ig4_mx8.cuh"
#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int ADDNORM_WARP_D = 512;       // up to this width a warp takes a row
constexpr int ADDNORM_WARPS = 4;          // warps (rows) per CTA in that form
constexpr int ADDNORM_NV = 2;             // vectors per thread
constexpr int ADDNORM_MAX_THREADS = 512;  // CTA-per-row form: D <= 8192
constexpr int ADDNORM_MAX_SLOTS = 8;
// Threads whose CTAs the grid counts for an SM.  The gradients' all fit: their register
// limit follows from it (96 a thread, at which the fp32 forms spill 80 bytes).  The
// forward's do not: at 54 to 64 registers 4 of the 5 CTAs at D = 4608 are resident, 3 for
// MX8, and 4 to 6 of the warp form's 12 (77 to 110 registers); the others start as those
// end.  Grids of the resident ones alone, with rings cut for them: 17.6 instead of 16.5 us
// for 2047 rows of 4608 to MX8, 53 as before for 9216, E4M3 rows 14.0 instead of 14.9 and
// 56.7 instead of 53 to 57, 18000 rows of 512 13.4 instead of 13.1.
constexpr int ADDNORM_FWD_THREADS_PER_SM = 1536;
constexpr int ADDNORM_BWD_THREADS_PER_SM = 640;

enum AddNormOut { ADDNORM_BF16 = 0, ADDNORM_F32 = 1, ADDNORM_ROW8 = 2, ADDNORM_MX8 = 3 };

// 8 consecutive elements as loaded; get(): as four packed pairs of floats (the
// arithmetic below is fp32 two at a time: these kernels are close to the issue
// limit, 30 instructions per element without it)
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) {
    q = *reinterpret_cast<const uint4 *>(p);
  }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    v[0] = bf16x2_to_f2(q.x);
    v[1] = bf16x2_to_f2(q.y);
    v[2] = bf16x2_to_f2(q.z);
    v[3] = bf16x2_to_f2(q.w);
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
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    v[0] = f2_pack(a.x, a.y);
    v[1] = f2_pack(a.z, a.w);
    v[2] = f2_pack(b.x, b.y);
    v[3] = f2_pack(b.z, b.w);
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const uint64_t (&v)[4]) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(pack_bf16x2(f2_lo(v[0]), f2_hi(v[0])), pack_bf16x2(f2_lo(v[1]), f2_hi(v[1])),
                 pack_bf16x2(f2_lo(v[2]), f2_hi(v[2])), pack_bf16x2(f2_lo(v[3]), f2_hi(v[3])));
}
__device__ __forceinline__ void store8(float *p, const uint64_t (&v)[4]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
  reinterpret_cast<float4 *>(p)[1] = make_float4(f2_lo(v[2]), f2_hi(v[2]), f2_lo(v[3]), f2_hi(v[3]));
}
// E4M3 codes of v * mul
__device__ __forceinline__ void store8_e4m3(uint8_t *p, const uint64_t (&v)[4], float mul) {
  const uint64_t m = f2_pack(mul, mul);
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t t = fmul2(v[e], m);
    c[e] = pack_e4m3x2(f2_lo(t), f2_hi(t));
  }
  *reinterpret_cast<uint2 *>(p) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ float max8(const uint64_t (&v)[4], float m) {
#pragma unroll
  for (int e = 0; e < 4; ++e) m = fmax3(m, fabsf(f2_lo(v[e])), fabsf(f2_hi(v[e])));
  return m;
}
__device__ __forceinline__ float sum2(uint64_t v) { return f2_lo(v) + f2_hi(v); }

// 1 / sqrt(v) to half a step: rsqrtf (2 steps) and one Newton correction with the
// residual 1 - v r^2 in two parts.  An error here is common to a whole row, and
// moves that many more of its values across a rounding border.
__device__ __forceinline__ float norm_rsqrt(float v) {
  const float r = rsqrtf(v);
  const float t = v * r;
  const float e = fmaf(-fmaf(v, r, -t), r, fmaf(-t, r, 1.0f));
  return v < INFINITY ? fmaf(0.5f * r, e, r) : r;
}

// Weight of vector vi (1 without a weight)
__device__ __forceinline__ void load_g8(const float *g, int vi, uint64_t (&v)[4]) {
  Raw8<float> w;
  if (g != nullptr)
    w.load(g + 8 * vi);
  else
    w.a = w.b = make_float4(1.f, 1.f, 1.f, 1.f);
  w.get(v);
}

// Reductions over the warps of a CTA through one word per warp in shared memory
// (the words past the last warp hold 0, which is neutral for the sum and for a
// maximum of absolute values); all threads combine them in the same order.
__device__ __forceinline__ void cta_put(float v, float *red) {
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
}
__device__ __forceinline__ float cta_sum(const float *red, int quads) {
  float v = 0.0f;
  for (int i = 0; i < quads; ++i) {
    const float4 a = reinterpret_cast<const float4 *>(red)[i];
    v += (a.x + a.y) + (a.z + a.w);
  }
  return v;
}
__device__ __forceinline__ float cta_max(const float *red, int quads) {
  float v = 0.0f;
  for (int i = 0; i < quads; ++i) {
    const float4 a = reinterpret_cast<const float4 *>(red)[i];
    v = fmax3(fmax3(a.x, a.y, a.z), a.w, v);
  }
  return v;
}

// y of one 8-element vector in MX8: blocks of 32 are four neighbouring lanes,
// and 16 lanes make the 4 scale bytes of one 128-element k-block, stored as one
// word.  All lanes of the warp take part; `in`: the vector exists.
__device__ __forceinline__ void store_mx8(const uint64_t (&t)[4], bool in, int vi, long row, int D,
                                          uint8_t *y, uint8_t *y_sf) {
  uint64_t b[4];  // the bf16 activation
#pragma unroll
  for (int e = 0; e < 4; ++e) b[e] = bf16x2_to_f2(pack_bf16x2(f2_lo(t[e]), f2_hi(t[e])));
  float amax = max8(b, 0.0f);
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int ex = mx8_exponent(amax);
  uint32_t w = static_cast<uint32_t>(ex + 127) << (8 * ((threadIdx.x >> 2) & 3));
  w |= __shfl_xor_sync(0xffffffffu, w, 4);
  w |= __shfl_xor_sync(0xffffffffu, w, 8);
  if (in) {
    store8_e4m3(y + row * D + 8 * vi, b, mx8_inv_scale(ex));
    if ((threadIdx.x & 15) == 0)
      *reinterpret_cast<uint32_t *>(y_sf + mx8_sf_offset(static_cast<int>(row), vi / 4, D)) = w;
  }
}

// scale = max|y| / 448 (1 for a zero row), codes of the fp32 y; at least 2^-126, whose
// reciprocal is finite
__device__ __forceinline__ float row8_scale(float amax) {
  return amax > 0.0f ? fmaxf(amax / 448.0f, 0x1p-126f) : 1.0f;
}

template <int OUT>
using AddNormY = typename std::conditional<OUT == ADDNORM_F32, float, __nv_bfloat16>::type;

// ------------------------------------------------------------ warp per row

template <typename XT, int OUT>
__global__ void __launch_bounds__(32 * ADDNORM_WARPS)
    add_rms_norm_warp_kernel(const XT *x, const XT *r, const float *g, float eps, XT *s_out,
                             void *y_out, float *y_scale, uint8_t *y_sf, int M, int D) {
  constexpr int NV = ADDNORM_NV;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int nvec = D / 8;
  const float inv_d = 1.0f / static_cast<float>(D);
  const long step = static_cast<long>(gridDim.x) * ADDNORM_WARPS;
  long row = static_cast<long>(blockIdx.x) * ADDNORM_WARPS + (threadIdx.x >> 5);
  uint64_t gv[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < nvec) load_g8(g, lane + 32 * i, gv[i]);
  Raw8<XT> cx[NV], cr[NV], nx[NV], nr[NV];
  auto fetch = [&](long rw, Raw8<XT>(&a)[NV], Raw8<XT>(&b)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = lane + 32 * i;
      a[i].zero();
      b[i].zero();
      if (vi < nvec) {
        a[i].load(x + rw * D + 8 * vi);
        if (r != nullptr) b[i].load(r + rw * D + 8 * vi);
      }
    }
  };
  if (row < M) fetch(row, cx, cr);
  for (; row < M; row += step) {
    if (row + step < M) fetch(row + step, nx, nr);
    uint64_t t[NV][4];
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t b[4];
      cx[i].get(t[i]);
      cr[i].get(b);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        t[i][e] = fadd2(t[i][e], b[e]);
        ss = ffma2(t[i][e], t[i][e], ss);
      }
      if (s_out != nullptr && lane + 32 * i < nvec)
        store8(s_out + row * D + 8 * (lane + 32 * i), t[i]);
      cx[i] = nx[i];
      cr[i] = nr[i];
    }
    const float rstd = norm_rsqrt(fmaf(warp_sum(sum2(ss)), inv_d, eps));
    const uint64_t rstd2 = f2_pack(rstd, rstd);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (lane + 32 * i >= nvec) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) t[i][e] = fmul2(fmul2(t[i][e], rstd2), gv[i][e]);
      if (OUT == ADDNORM_ROW8) amax = max8(t[i], amax);
    }
    float inv = 1.0f;
    if constexpr (OUT == ADDNORM_ROW8) {
      const float qs = row8_scale(warp_max(amax));
      inv = 1.0f / qs;
      if (lane == 0) y_scale[row] = qs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = lane + 32 * i;
      if constexpr (OUT == ADDNORM_MX8) {
        store_mx8(t[i], vi < nvec, vi, row, D, static_cast<uint8_t *>(y_out), y_sf);
      } else if (vi < nvec) {
        if constexpr (OUT == ADDNORM_ROW8)
          store8_e4m3(static_cast<uint8_t *>(y_out) + row * D + 8 * vi, t[i], inv);
        else
          store8(static_cast<AddNormY<OUT> *>(y_out) + row * D + 8 * vi, t[i]);
      }
    }
  }
}

// Gradients.  A thread keeps the same columns for every row it sees, so dg
// accumulates in its registers; each CTA then writes one partial row of dg,
// and add_rms_norm_dg_kernel adds the partial rows in a fixed order (no
// atomics: the same inputs give the same bits).
//   dx = rstd (dy g - n m) + ds,  m = mean(dy g n) = dot rstd / D,  dot = sum dy g s

// One vector's share of the two row sums
__device__ __forceinline__ void grad_sums(const uint64_t (&s)[4], const uint64_t (&dy)[4],
                                          const uint64_t (&g)[4], uint64_t &ss, uint64_t &dot) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    ss = ffma2(s[e], s[e], ss);
    dot = ffma2(fmul2(dy[e], g[e]), s[e], dot);
  }
}
// One vector's dx (into ds) and its part of dg; negm = -m
__device__ __forceinline__ void grad_apply(const uint64_t (&s)[4], const uint64_t (&dy)[4],
                                           const uint64_t (&g)[4], float rstd, float negm,
                                           uint64_t (&ds)[4], uint64_t (&acc)[4]) {
  const uint64_t r2 = f2_pack(rstd, rstd), m2 = f2_pack(negm, negm);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t n = fmul2(s[e], r2);
    acc[e] = ffma2(dy[e], n, acc[e]);
    ds[e] = ffma2(r2, ffma2(dy[e], g[e], fmul2(n, m2)), ds[e]);
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(32 * ADDNORM_WARPS)
    add_rms_norm_grad_warp_kernel(const XT *s, const float *g, float eps, const YT *dy,
                                  const XT *ds, XT *dx, float *dg_part, int M, int D) {
  constexpr int NV = ADDNORM_NV;
  pdl_wait();
  pdl_trigger();
  __shared__ alignas(16) float acc_s[ADDNORM_WARPS * ADDNORM_WARP_D];
  const int lane = threadIdx.x & 31;
  const int nvec = D / 8;
  const float inv_d = 1.0f / static_cast<float>(D);
  const long step = static_cast<long>(gridDim.x) * ADDNORM_WARPS;
  long row = static_cast<long>(blockIdx.x) * ADDNORM_WARPS + (threadIdx.x >> 5);
  uint64_t gv[NV][4], acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = gv[i][e] = 0;
    if (lane + 32 * i < nvec) load_g8(g, lane + 32 * i, gv[i]);
  }
  Raw8<XT> cs[NV], cd[NV], ns[NV], nd[NV];
  Raw8<YT> cy[NV], ny[NV];
  auto fetch = [&](long rw, Raw8<XT>(&a)[NV], Raw8<YT>(&b)[NV], Raw8<XT>(&c)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = lane + 32 * i;
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
  for (; row < M; row += step) {
    if (row + step < M) fetch(row + step, ns, ny, nd);
    uint64_t ss = 0, dot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t a[4], b[4];
      cs[i].get(a);
      cy[i].get(b);
      grad_sums(a, b, gv[i], ss, dot);
    }
    const float rstd = norm_rsqrt(fmaf(warp_sum(sum2(ss)), inv_d, eps));
    const float negm = -warp_sum(sum2(dot)) * rstd * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      uint64_t a[4], b[4], c[4];
      cs[i].get(a);
      cy[i].get(b);
      cd[i].get(c);
      grad_apply(a, b, gv[i], rstd, negm, c, acc[i]);
      if (lane + 32 * i < nvec) store8(dx + row * D + 8 * (lane + 32 * i), c);
      cs[i] = ns[i];
      cy[i] = ny[i];
      cd[i] = nd[i];
    }
  }
  if (dg_part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (lane + 32 * i < nvec) store8(acc_s + (threadIdx.x >> 5) * D + 8 * (lane + 32 * i), acc[i]);
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += 32 * ADDNORM_WARPS) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < ADDNORM_WARPS; ++w) v += acc_s[w * D + c];
    dg_part[static_cast<long>(blockIdx.x) * D + c] = v;
  }
}

// ------------------------------------------------------------- CTA per row
// Shared memory of a launch: `slots` of one row of each input, then the
// reduction words (4 sets of 16) and the slots' barriers.
__host__ __device__ constexpr size_t addnorm_smem(size_t slot_bytes, int slots) {
  return slot_bytes * slots + 4 * 16 * 4 + ADDNORM_MAX_SLOTS * 8 + 16;
}

// The ring: rows first, first + step, .. in slots 0 .. S-1, 0, ..
struct AddNormRing {
  uint8_t *base;
  float *red;
  uint64_t *full;
  volatile int *abort_flag;
  int slots;
  uint32_t slot_bytes;
  int in_slot = 0, out_slot = 0;  // next slot to fill (thread 0), to read
  uint32_t phase = 0;             // of out_slot
  bool alive = true;

  __device__ __forceinline__ AddNormRing(uint8_t *smem, int slots_, uint32_t bytes)
      : base(smem), slots(slots_), slot_bytes(bytes) {
    red = reinterpret_cast<float *>(smem + static_cast<size_t>(slots) * bytes);
    full = reinterpret_cast<uint64_t *>(red + 4 * 16);
    int *flag = reinterpret_cast<int *>(full + ADDNORM_MAX_SLOTS);
    abort_flag = flag;
    for (int i = threadIdx.x; i < 4 * 16; i += blockDim.x) red[i] = 0.0f;
    if (threadIdx.x == 0) {
      for (int i = 0; i < slots; ++i) mbar_init(&full[i], 1);
      *flag = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  // The next slot to fill, its barrier expecting a row
  __device__ __forceinline__ uint8_t *open(uint64_t **bar) {
    const int s = in_slot;
    if (++in_slot == slots) in_slot = 0;
    *bar = &full[s];
    mbar_arrive_expect_tx(*bar, slot_bytes);
    return base + s * slot_bytes;
  }
  // Waits for the next row.  A wait that runs out (the device error word is
  // set) is not repeated, and the threads go on in step to the end.
  __device__ __forceinline__ const uint8_t *wait() {
    const int s = out_slot;
    if (alive) alive = mbar_wait(&full[s], phase, abort_flag);
    if (++out_slot == slots) {
      out_slot = 0;
      phase ^= 1;
    }
    return base + s * slot_bytes;
  }
};

template <typename XT, int OUT>
__global__ void __launch_bounds__(ADDNORM_MAX_THREADS)
    add_rms_norm_kernel(const XT *x, const XT *r, const float *g, float eps, XT *s_out, void *y_out,
                        float *y_scale, uint8_t *y_sf, int M, int D, int slots) {
  constexpr int NV = ADDNORM_NV;
  extern __shared__ float4 norm_smem[];
  const uint32_t row_bytes = static_cast<uint32_t>(D) * sizeof(XT);
  AddNormRing ring(reinterpret_cast<uint8_t *>(norm_smem), slots,
                   r != nullptr ? 2 * row_bytes : row_bytes);
  pdl_wait();
  pdl_trigger();
  const int T = blockDim.x, tid = threadIdx.x;
  const int nvec = D / 8;
  const int quads = (T + 127) / 128;
  const float inv_d = 1.0f / static_cast<float>(D);
  const long step = gridDim.x;
  long ahead = blockIdx.x;  // the next row to fetch (thread 0)
  auto issue = [&]() {
    if (ahead >= M) return;
    uint64_t *bar;
    uint8_t *dst = ring.open(&bar);
    bulk_load(dst, x + ahead * D, row_bytes, bar);
    if (r != nullptr) bulk_load(dst + row_bytes, r + ahead * D, row_bytes, bar);
    ahead += step;
  };
  if (tid == 0)
    for (int i = 0; i < slots; ++i) issue();
  uint64_t gv[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + T * i < nvec) load_g8(g, tid + T * i, gv[i]);
  float *rd = ring.red, *rd_next = ring.red + 32;
  for (long row = blockIdx.x; row < M; row += step) {
    const XT *sx = reinterpret_cast<const XT *>(ring.wait());
    uint64_t t[NV][4];
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      if (vi < nvec) {
        Raw8<XT> a;
        a.load(sx + 8 * vi);
        a.get(t[i]);
        if (r != nullptr) {
          uint64_t b[4];
          a.load(sx + D + 8 * vi);
          a.get(b);
#pragma unroll
          for (int e = 0; e < 4; ++e) t[i][e] = fadd2(t[i][e], b[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = ffma2(t[i][e], t[i][e], ss);
      }
    }
    cta_put(warp_sum(sum2(ss)), rd);
    __syncthreads();
    if (tid == 0) issue();  // every thread has read its part of the slot
    const float rstd = norm_rsqrt(fmaf(cta_sum(rd, quads), inv_d, eps));
    const uint64_t rstd2 = f2_pack(rstd, rstd);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      if (vi < nvec) {
        if (s_out != nullptr) store8(s_out + row * D + 8 * vi, t[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) t[i][e] = fmul2(fmul2(t[i][e], rstd2), gv[i][e]);
        if (OUT == ADDNORM_ROW8) amax = max8(t[i], amax);
        if constexpr (OUT == ADDNORM_BF16 || OUT == ADDNORM_F32)
          store8(static_cast<AddNormY<OUT> *>(y_out) + row * D + 8 * vi, t[i]);
      }
      if constexpr (OUT == ADDNORM_MX8)
        store_mx8(t[i], vi < nvec, vi, row, D, static_cast<uint8_t *>(y_out), y_sf);
    }
    if constexpr (OUT == ADDNORM_ROW8) {
      cta_put(warp_max(amax), rd + 16);
      __syncthreads();
      const float qs = row8_scale(cta_max(rd + 16, quads));
      const float inv = 1.0f / qs;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int vi = tid + T * i;
        if (vi < nvec) store8_e4m3(static_cast<uint8_t *>(y_out) + row * D + 8 * vi, t[i], inv);
      }
      if (tid == 0) y_scale[row] = qs;
    }
    float *sw = rd;
    rd = rd_next;
    rd_next = sw;
  }
  if (!ring.alive && tid == 0) sleep_ns(20000);  // let the copies already issued land
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(ADDNORM_BWD_THREADS_PER_SM)
    add_rms_norm_grad_kernel(const XT *s, const float *g, float eps, const YT *dy, const XT *ds,
                             XT *dx, float *dg_part, int M, int D, int slots) {
  constexpr int NV = ADDNORM_NV;
  extern __shared__ float4 norm_smem[];
  const uint32_t xb = static_cast<uint32_t>(D) * sizeof(XT), yb = static_cast<uint32_t>(D) * sizeof(YT);
  AddNormRing ring(reinterpret_cast<uint8_t *>(norm_smem), slots, xb + yb + (ds != nullptr ? xb : 0));
  pdl_wait();
  pdl_trigger();
  const int T = blockDim.x, tid = threadIdx.x;
  const int nvec = D / 8;
  const int quads = (T + 127) / 128;
  const float inv_d = 1.0f / static_cast<float>(D);
  const long step = gridDim.x;
  long ahead = blockIdx.x;  // the next row to fetch (thread 0)
  auto issue = [&]() {
    if (ahead >= M) return;
    uint64_t *bar;
    uint8_t *dst = ring.open(&bar);
    bulk_load(dst, s + ahead * D, xb, bar);
    bulk_load(dst + xb, dy + ahead * D, yb, bar);
    if (ds != nullptr) bulk_load(dst + xb + yb, ds + ahead * D, xb, bar);
    ahead += step;
  };
  if (tid == 0)
    for (int i = 0; i < slots; ++i) issue();
  uint64_t gv[NV][4], acc[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = gv[i][e] = 0;
    if (tid + T * i < nvec) load_g8(g, tid + T * i, gv[i]);
  }
  float *rd = ring.red, *rd_next = ring.red + 32;
  for (long row = blockIdx.x; row < M; row += step) {
    const uint8_t *slot = ring.wait();
    uint64_t a[NV][4], b[NV][4];
    Raw8<XT> cd[NV];
    uint64_t ss = 0, dot = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      if (vi < nvec) {
        Raw8<XT> ra;
        Raw8<YT> rb;
        ra.load(reinterpret_cast<const XT *>(slot) + 8 * vi);
        rb.load(reinterpret_cast<const YT *>(slot + xb) + 8 * vi);
        cd[i].zero();
        if (ds != nullptr) cd[i].load(reinterpret_cast<const XT *>(slot + xb + yb) + 8 * vi);
        ra.get(a[i]);
        rb.get(b[i]);
        grad_sums(a[i], b[i], gv[i], ss, dot);
      }
    }
    cta_put(warp_sum(sum2(ss)), rd);
    cta_put(warp_sum(sum2(dot)), rd + 16);
    __syncthreads();
    if (tid == 0) issue();  // every thread has read its part of the slot
    const float rstd = norm_rsqrt(fmaf(cta_sum(rd, quads), inv_d, eps));
    const float negm = -cta_sum(rd + 16, quads) * rstd * inv_d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int vi = tid + T * i;
      if (vi < nvec) {
        uint64_t c[4];
        cd[i].get(c);
        grad_apply(a[i], b[i], gv[i], rstd, negm, c, acc[i]);
        store8(dx + row * D + 8 * vi, c);
      }
    }
    float *sw = rd;
    rd = rd_next;
    rd_next = sw;
  }
  if (!ring.alive && tid == 0) sleep_ns(20000);  // let the copies already issued land
  if (dg_part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (tid + T * i < nvec)
      store8(dg_part + static_cast<long>(blockIdx.x) * D + 8 * (tid + T * i), acc[i]);
}

// dg[c] = sum over the P partial rows: a CTA takes 8 columns (one 32-byte sector
// of each partial row), its 64 row lanes every 64th row, four in flight; then
// the lanes' sums are added in a fixed order.  (32 columns and 32 row lanes left
// most SMs idle at small D and took 5 us more at D = 1032.)
constexpr int ADDNORM_DG_THREADS = 512;
constexpr int ADDNORM_DG_COLS = 8;
__global__ void __launch_bounds__(ADDNORM_DG_THREADS)
    add_rms_norm_dg_kernel(const float *part, int P, int D, float *dg) {
  constexpr int ROWS = ADDNORM_DG_THREADS / ADDNORM_DG_COLS, W = ADDNORM_DG_THREADS / 32;
  __shared__ float red[W][ADDNORM_DG_COLS];
  pdl_wait();
  pdl_trigger();
  const int c = threadIdx.x % ADDNORM_DG_COLS;
  const float *col = part + blockIdx.x * ADDNORM_DG_COLS + c;  // D % 8 == 0
  float v = 0.0f;
  for (int p = threadIdx.x / ADDNORM_DG_COLS; p < P; p += 4 * ROWS) {
    float a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = p + i * ROWS < P ? col[static_cast<long>(p + i * ROWS) * D] : 0.0f;
    v += (a[0] + a[1]) + (a[2] + a[3]);
  }
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if ((threadIdx.x & 31) < ADDNORM_DG_COLS) red[threadIdx.x >> 5][c] = v;
  __syncthreads();
  if (threadIdx.x < ADDNORM_DG_COLS) {
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[w][c];
    dg[blockIdx.x * ADDNORM_DG_COLS + c] = v;
  }
}

}  // namespace ig4
