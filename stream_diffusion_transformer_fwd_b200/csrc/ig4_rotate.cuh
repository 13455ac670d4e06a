// ig4_rotate.cuh - rotary positions with several axes (t, h, w) applied to
// strided q and k heads, and the inverse rotation (its gradient).
//
// Pair j of a token turns by pos[axis(j)] * theta^(-2j/R).  The angle is
// formed in turns in fp64 and reduced to half a turn either way before it is
// rounded to fp32 (a far position times a frequency would lose its fraction in
// fp32); fp32 sincospi then gives cos and sin to fp32 accuracy.
//
// HBM bounds it: each element is read and written once for three multiplies.  A
// CTA takes a few tokens (and a share of the heads when there are few tokens),
// computes their cos/sin and the addresses of their rows once into shared
// memory, and streams all its heads through registers.  A thread keeps one unit
// (a vector of V elements of each half of a head, or one vector of whole pairs
// in the adjacent layout) and walks tokens and heads: its cos/sin stay in
// registers over the heads, and a step costs two pointer additions.  q and k
// share one launch and one table.  Elements past the rotary ones are copied in a
// walk of their own, so that no warp holds both kinds of work.
//
// 2 x 4608 tokens, 18 + 18 bf16 heads of 256 (64 pairs), strided in and out: 63 us for
// 340 MB, 5.4 TB/s, 82% of a plain copy.  8 single tokens of as many heads: 4.8 us.
// 2032 tokens of 16 + 4 fp32 heads of 128, adjacent pairs: 10.9 us, 3.8 TB/s (508 CTAs,
// fewer than the SMs hold, and none's loads start before its table is done).
#pragma once

#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int ROTATE_THREADS = 256;
constexpr int ROTATE_MAX_PAIRS = 256;
constexpr int ROTATE_CTAS = 4;         // on an SM (64 registers a thread)
constexpr int ROTATE_MAX_TOKENS = 8;  // of a CTA
constexpr int ROTATE_TABLE = 1024;    // pairs in a CTA's table, all tokens
// Heads whose loads a thread has in flight: wide vectors fill the 64 registers
// with two (28 bytes spill for halves of bf16 heads; four take twice the time),
// narrow ones need more loads for the same bytes (three: 32 bytes spill at 8-byte
// vectors of bf16, 24 of fp32).
__host__ __device__ constexpr int rotate_batch(int bytes) { return bytes == 16 ? 2 : 3; }

// Threads of a walk: thread i takes unit i % U, of heads i / U % HG, + HG, ..
// and tokens i / (U HG), + TG, ..; mu and mh divide by U and HG ((i * m) >> 16 is
// exact while i * divisor < 65536).
struct RotateWalk {
  int U, HG, TG, mu, mh;
};

struct RotateHeads {
  const void *in;
  void *out;
  int H;
  long in_b, in_l, in_h, out_b, out_l, out_h;  // strides in elements
  RotateWalk turn, copy;
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

// BYTES (2, 4, 8 or 16) consecutive bytes as 32-bit words
template <int BYTES>
struct RotRaw {
  static constexpr int W = BYTES >= 4 ? BYTES / 4 : 1;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void *p) {
    if constexpr (BYTES == 16) {
      const uint4 v = *static_cast<const uint4 *>(p);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (BYTES == 8) {
      const uint2 v = *static_cast<const uint2 *>(p);
      w[0] = v.x;
      w[1] = v.y;
    } else if constexpr (BYTES == 4) {
      w[0] = *static_cast<const uint32_t *>(p);
    } else {
      w[0] = *static_cast<const unsigned short *>(p);
    }
  }
  __device__ __forceinline__ void store(void *p) const {
    if constexpr (BYTES == 16)
      *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (BYTES == 8)
      *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    else if constexpr (BYTES == 4)
      *static_cast<uint32_t *>(p) = w[0];
    else
      *static_cast<unsigned short *>(p) = static_cast<unsigned short>(w[0]);
  }
};

// (x, z) -> (x c - z s, z c + x s)
__device__ __forceinline__ void rot_pair(float &x, float &z, float c, float s) {
  const float a = x * c - z * s;
  z = z * c + x * s;
  x = a;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// What a thread's step loads: V elements of each half of a head, or V adjacent
// ones (a pair for V = 1); PU pairs, their cos/sin read from the table Q at a time.
template <typename T, int V, bool ADJ>
struct RotStep {
  static constexpr int PU = ADJ ? (V >= 2 ? V / 2 : 1) : V;
  static constexpr int Q = PU < 4 ? PU : 4;
  static constexpr bool TWO = !ADJ || V == 1;  // two vectors
  using Raw = RotRaw<V * static_cast<int>(sizeof(T))>;
  Raw lo, hi;
  __device__ __forceinline__ void load(const T *p, int far) {
    lo.load(p);
    if constexpr (TWO) hi.load(p + far);
  }
  __device__ __forceinline__ void store(T *p, int far) const {
    lo.store(p);
    if constexpr (TWO) hi.store(p + far);
  }
  __device__ __forceinline__ void turn(const float (&c)[PU], const float (&s)[PU]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < PU; ++e) {
        uint32_t &wa = TWO ? lo.w[e] : lo.w[2 * e];
        uint32_t &wb = TWO ? hi.w[e] : lo.w[2 * e + 1];
        float x = __uint_as_float(wa), z = __uint_as_float(wb);
        rot_pair(x, z, c[e], s[e]);
        wa = __float_as_uint(x);
        wb = __float_as_uint(z);
      }
    } else if constexpr (!TWO) {  // a bf16 pair in each word
#pragma unroll
      for (int e = 0; e < PU; ++e) {
        float x = bf16_lo(lo.w[e]), z = bf16_hi(lo.w[e]);
        rot_pair(x, z, c[e], s[e]);
        lo.w[e] = pack_bf16x2(x, z);
      }
    } else if constexpr (V == 1) {
      float x = bf16_lo(lo.w[0]), z = bf16_lo(hi.w[0]);
      rot_pair(x, z, c[0], s[0]);
      lo.w[0] = pack_bf16x2(x, 0.0f);
      hi.w[0] = pack_bf16x2(z, 0.0f);
    } else {  // two pairs across a word of each half
#pragma unroll
      for (int i = 0; i < PU / 2; ++i) {
        float x0 = bf16_lo(lo.w[i]), x1 = bf16_hi(lo.w[i]);
        float z0 = bf16_lo(hi.w[i]), z1 = bf16_hi(hi.w[i]);
        rot_pair(x0, z0, c[2 * i], s[2 * i]);
        rot_pair(x1, z1, c[2 * i + 1], s[2 * i + 1]);
        lo.w[i] = pack_bf16x2(x0, x1);
        hi.w[i] = pack_bf16x2(z0, z1);
      }
    }
  }
};

// Visits every (token < nt, head < nh) of the thread's unit, if that is below `units`:
// begin(token, unit) once per token, then load(value, address) of NB heads before finish(value,
// address) of the first (an output may be its input, so the compiler cannot move loads
// above stores by itself).
template <int NB, typename Raw, typename T, typename Begin, typename Load, typename Finish>
__device__ __forceinline__ void rotate_walk(const RotateWalk &k, const T *in, T *out,
                                            const long *base_in, const long *base_out, long in_h,
                                            long out_h, int unit_size, int units, int nt, int nh,
                                            Begin begin, Load load, Finish finish) {
  const int q = (static_cast<int>(threadIdx.x) * k.mu) >> 16;
  const int tk0 = (q * k.mh) >> 16;
  const int u = threadIdx.x - q * k.U, h0 = q - tk0 * k.HG;
  if (tk0 >= k.TG || u >= units) return;
  const long din = k.HG * in_h, dout = k.HG * out_h;
  for (int tk = tk0; tk < nt; tk += k.TG) {
    begin(tk, u);
    const T *ip = in + (base_in[tk] + h0 * in_h + u * unit_size);
    T *op = out + (base_out[tk] + h0 * out_h + u * unit_size);
    for (int h = h0; h < nh; h += NB * k.HG) {
      Raw v[NB];
#pragma unroll
      for (int i = 0; i < NB; ++i, ip += din)
        if (h + i * k.HG < nh) load(v[i], ip);
#pragma unroll
      for (int i = 0; i < NB; ++i, op += dout)
        if (h + i * k.HG < nh) finish(v[i], op);
    }
  }
}

// ADJ: pairs are neighbouring elements (2j, 2j+1); else (j, j + R/2).
template <typename T, int V, bool ADJ>
__global__ void __launch_bounds__(ROTATE_THREADS, ROTATE_CTAS)
    mrope_rotate_kernel(const __grid_constant__ RotateArgs a) {
  using Step = RotStep<T, V, ADJ>;
  constexpr int PU = Step::PU, Q = Step::Q;
  using Vec = typename Step::Raw;
  using Tab = RotRaw<4 * Q>;
  // table: per token a cos and a sin plane, each [PU / Q][unit][Q], so that the
  // lanes of a warp (neighbouring units) read consecutive words
  __shared__ alignas(16) float tbl[2 * ROTATE_TABLE];
  __shared__ long base_in[2][ROTATE_MAX_TOKENS], base_out[2][ROTATE_MAX_TOKENS];
  pdl_wait();
  pdl_trigger();
  const int P = a.R / 2;
  const int UP = P / PU;
  const long ntok = static_cast<long>(a.B) * a.L;
  const long tok0 = static_cast<long>(blockIdx.x) * a.tt;
  const int nt = static_cast<int>(min(static_cast<long>(a.tt), ntok - tok0));
  for (int i = threadIdx.x; i < nt * P; i += ROTATE_THREADS) {
    const int tk = i / P, j = i - tk * P;
    const int n = static_cast<int>(tok0) + tk;  // B L < 2^31
    const int b = n / a.L, l = n - b * a.L;
    const int ax = (a.axis[j >> 4] >> (2 * (j & 15))) & 3;
    const double turns = exp2(-a.log2_theta * static_cast<double>(j) / static_cast<double>(P)) *
                         0.15915494309189533577 *
                         static_cast<double>(a.pos[b * a.pos_b + static_cast<long>(ax) * a.L + l]);
    const float f = static_cast<float>(2.0 * (turns - rint(turns)));
    float sn, cs;
    sincospif(f, &sn, &cs);
    const int u = j / PU, e = j % PU;
    float *tp = tbl + 2 * tk * P + (e / Q * UP + u) * Q + e % Q;
    tp[0] = cs;
    tp[P] = a.sin_sign * sn;
    if (j < 4) {
      const RotateHeads &t = a.t[j & 1];
      if (j < 2)
        base_in[j][tk] = b * t.in_b + l * t.in_l;
      else
        base_out[j - 2][tk] = b * t.out_b + l * t.out_l;
    }
  }
  // (a table of fewer than four pairs does not cover the addresses)
  if (P < 4 && threadIdx.x < static_cast<unsigned>(nt)) {
    const int n = static_cast<int>(tok0) + threadIdx.x;
    const int b = n / a.L, l = n - b * a.L;
    for (int w = 0; w < 2; ++w) {
      base_in[w][threadIdx.x] = b * a.t[w].in_b + l * a.t[w].in_l;
      base_out[w][threadIdx.x] = b * a.t[w].out_b + l * a.t[w].out_l;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const RotateHeads &t = a.t[w];
    // this CTA's share of the heads
    const int h0 = static_cast<int>(static_cast<long>(t.H) * blockIdx.y / a.hs);
    const int nh = static_cast<int>(static_cast<long>(t.H) * (blockIdx.y + 1) / a.hs) - h0;
    if (nh <= 0) continue;
    const T *in = static_cast<const T *>(t.in) + h0 * t.in_h;
    T *out = static_cast<T *>(t.out) + h0 * t.out_h;
    float cs[PU], sn[PU];
    rotate_walk<rotate_batch(sizeof(Vec)), Step>(
        t.turn, in, out, base_in[w], base_out[w], t.in_h, t.out_h, ADJ && V == 1 ? 2 : V,
        ROTATE_THREADS, nt, nh,
        [&](int tk, int u) {
#pragma unroll
          for (int c = 0; c < PU / Q; ++c) {
            const float *tp = tbl + 2 * tk * P + (c * UP + u) * Q;
            Tab x, y;
            x.load(tp);
            y.load(tp + P);
#pragma unroll
            for (int e = 0; e < Q; ++e) {
              cs[c * Q + e] = __uint_as_float(x.w[e]);
              sn[c * Q + e] = __uint_as_float(y.w[e]);
            }
          }
        },
        [&](Step &v, const T *ip) { v.load(ip, ADJ ? 1 : P); },
        [&](Step &v, T *op) {
          v.turn(cs, sn);
          v.store(op, ADJ ? 1 : P);
        });
    // elements past the rotary ones are copied (already there in place); the last run may
    // be shorter
    if (t.copy.U > 0)
      for (int first = a.R; first < a.d; first += t.copy.U * V)
        rotate_walk<2 * rotate_batch(sizeof(Vec)), Vec>(
            t.copy, in + first, out + first, base_in[w], base_out[w], t.in_h, t.out_h, V,
            (a.d - first) / V, nt, nh,
            [](int, int) {}, [](Vec &v, const T *ip) { v.load(ip); },
            [](const Vec &v, T *op) { v.store(op); });
  }
}

}  // namespace ig4
