// ig4_rotate.cuh - rotary positions with several axes (t, h, w) applied to
// strided q and k heads, and the inverse rotation (its gradient).
//
// Pair j of a token turns by pos[axis(j)] * theta^(-2j/R).  The angle is
// formed in turns in fp64 and reduced to half a turn either way before it is
// rounded to fp32 (a far position times a frequency would lose its fraction in
// fp32); fp32 sincospi then gives cos and sin to fp32 accuracy.
//
// HBM bounds it: two bytes moved per element and pass, three multiplies.  A
// CTA takes TT tokens (and a share of the heads when there are few tokens),
// computes their cos/sin once into shared memory, and streams all its heads
// through registers with vector accesses; q and k share one launch and one
// table.
#pragma once

#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int ROTATE_THREADS = 256;
constexpr int ROTATE_MAX_PAIRS = 256;
constexpr int ROTATE_TABLE = 1024;  // table entries (cos, sin) of a CTA
constexpr int ROTATE_BATCH = 4;     // vectors in flight per thread

struct RotateHeads {
  const void *in;
  void *out;
  int H;
  long in_b, in_l, in_h, out_b, out_l, out_h;  // strides in elements
};

struct RotateArgs {
  RotateHeads t[2];  // q, k (H = 0: absent)
  const int32_t *pos;
  long pos_b;
  int B, L, d, R;
  int tt;        // tokens per CTA
  int hs;        // head shares (gridDim.y)
  double log2_theta;
  float sin_sign;
  uint32_t axis[ROTATE_MAX_PAIRS / 16];  // 2 bits per pair
};

// V consecutive elements
template <typename T, int V>
struct alignas(sizeof(T) * V) RotVec {
  T v[V];
};
__device__ __forceinline__ float rot_to_f(float x) { return x; }
__device__ __forceinline__ float rot_to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void rot_from_f(float x, float *o) { *o = x; }
__device__ __forceinline__ void rot_from_f(float x, __nv_bfloat16 *o) { *o = __float2bfloat16_rn(x); }

// Position of an item (token, head, unit) that a thread walks in steps of the
// CTA's thread count, without divisions in the loop.
struct RotWalk {
  int tok, h, u;
  int U, H;
  int dtok, dh, du;
  __device__ __forceinline__ RotWalk(int first, int stride, int U_, int H_) : U(U_), H(H_) {
    u = first % U;
    const int a = first / U;
    h = a % H;
    tok = a / H;
    du = stride % U;
    const int s = stride / U;
    dh = s % H;
    dtok = s / H;
  }
  __device__ __forceinline__ void next() {
    u += du;
    h += dh;
    tok += dtok;
    if (u >= U) {
      u -= U;
      ++h;
    }
    if (h >= H) {
      h -= H;
      ++tok;
    }
  }
};

// ADJ: pairs are neighbouring elements (2j, 2j+1); else (j, j + R/2).
template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(ROTATE_THREADS)
    mrope_rotate_kernel(const __grid_constant__ RotateArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ float2 tbl[ROTATE_TABLE];  // [token][pair in unit][unit]
  // pairs of one unit, and units of one head: half layout, V pairs from two
  // vectors; adjacent layout, V / 2 pairs from one (a pair for V = 1)
  constexpr int PU = ADJ ? (V >= 2 ? V / 2 : 1) : V;
  using Vec = RotVec<T, V>;
  const int P = a.R / 2;
  const int UP = P / PU;
  const long ntok = static_cast<long>(a.B) * a.L;
  const long tok0 = static_cast<long>(blockIdx.x) * a.tt;
  const int nt = static_cast<int>(min(static_cast<long>(a.tt), ntok - tok0));
  for (int i = threadIdx.x; i < nt * P; i += ROTATE_THREADS) {
    const int tk = i / P, j = i - tk * P;
    const long n = tok0 + tk;
    const long b = n / a.L, l = n - b * a.L;
    const int ax = (a.axis[j >> 4] >> (2 * (j & 15))) & 3;
    const double turns = exp2(-a.log2_theta * static_cast<double>(j) / static_cast<double>(P)) *
                         0.15915494309189533577 *
                         static_cast<double>(a.pos[b * a.pos_b + static_cast<long>(ax) * a.L + l]);
    const float f = static_cast<float>(2.0 * (turns - rint(turns)));
    float sn, cs;
    sincospif(f, &sn, &cs);
    tbl[(tk * PU + j % PU) * UP + j / PU] = make_float2(cs, a.sin_sign * sn);
  }
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const RotateHeads &t = a.t[w];
    // this CTA's share of the heads
    const int h0 = static_cast<int>(static_cast<long>(t.H) * blockIdx.y / a.hs);
    const int nh = static_cast<int>(static_cast<long>(t.H) * (blockIdx.y + 1) / a.hs) - h0;
    if (nh <= 0) continue;
    const T *in = static_cast<const T *>(t.in);
    T *out = static_cast<T *>(t.out);
    auto offsets = [&](const RotWalk &k, long *oi, long *oo) {
      const long n = tok0 + k.tok;
      const long b = a.B == 1 ? 0 : n / a.L;
      const long l = n - b * a.L;
      const int h = h0 + k.h;
      *oi = b * t.in_b + l * t.in_l + h * t.in_h;
      *oo = b * t.out_b + l * t.out_l + h * t.out_h;
    };
    {
      RotWalk k(threadIdx.x, ROTATE_THREADS, UP, nh);
      while (k.tok < nt) {
        Vec lo[ROTATE_BATCH], hi[ROTATE_BATCH];
        long oo[ROTATE_BATCH];
        int ti[ROTATE_BATCH];
#pragma unroll
        for (int i = 0; i < ROTATE_BATCH; ++i) {
          ti[i] = -1;
          if (k.tok < nt) {
            long oi;
            offsets(k, &oi, &oo[i]);
            ti[i] = k.tok * PU * UP + k.u;
            if constexpr (ADJ && V >= 2) {
              oi += V * k.u;
              oo[i] += V * k.u;
              lo[i] = *reinterpret_cast<const Vec *>(in + oi);
            } else if constexpr (ADJ) {
              oi += 2 * k.u;
              oo[i] += 2 * k.u;
              lo[i].v[0] = in[oi];
              hi[i].v[0] = in[oi + 1];
            } else {
              oi += V * k.u;
              oo[i] += V * k.u;
              lo[i] = *reinterpret_cast<const Vec *>(in + oi);
              hi[i] = *reinterpret_cast<const Vec *>(in + oi + P);
            }
            k.next();
          }
        }
#pragma unroll
        for (int i = 0; i < ROTATE_BATCH; ++i) {
          if (ti[i] < 0) continue;
#pragma unroll
          for (int e = 0; e < PU; ++e) {
            const float2 cs = tbl[ti[i] + e * UP];
            T *pa, *pb;
            if constexpr (ADJ && V >= 2) {
              pa = &lo[i].v[2 * e];
              pb = &lo[i].v[2 * e + 1];
            } else {
              pa = &lo[i].v[e];
              pb = &hi[i].v[e];
            }
            const float x = rot_to_f(*pa), z = rot_to_f(*pb);
            rot_from_f(x * cs.x - z * cs.y, pa);
            rot_from_f(z * cs.x + x * cs.y, pb);
          }
          if constexpr (ADJ && V >= 2) {
            *reinterpret_cast<Vec *>(out + oo[i]) = lo[i];
          } else if constexpr (ADJ) {
            out[oo[i]] = lo[i].v[0];
            out[oo[i] + 1] = hi[i].v[0];
          } else {
            *reinterpret_cast<Vec *>(out + oo[i]) = lo[i];
            *reinterpret_cast<Vec *>(out + oo[i] + P) = hi[i];
          }
        }
      }
    }
    // elements past the rotary ones are copied (already there in place)
    const int UC = (a.d - a.R) / V;
    if (UC > 0 && t.in != t.out) {
      RotWalk k(threadIdx.x, ROTATE_THREADS, UC, nh);
      while (k.tok < nt) {
        Vec x[ROTATE_BATCH];
        long oo[ROTATE_BATCH];
        int n = 0;
#pragma unroll
        for (int i = 0; i < ROTATE_BATCH; ++i) {
          if (k.tok < nt) {
            long oi;
            offsets(k, &oi, &oo[i]);
            oi += a.R + V * k.u;
            oo[i] += a.R + V * k.u;
            x[i] = *reinterpret_cast<const Vec *>(in + oi);
            n = i + 1;
            k.next();
          }
        }
#pragma unroll
        for (int i = 0; i < ROTATE_BATCH; ++i)
          if (i < n) *reinterpret_cast<Vec *>(out + oo[i]) = x[i];
      }
    }
  }
}

}  // namespace ig4
