// ig4_matvec.cuh - 1 to 8 bf16 rows times NVFP4 weights (E2M1 codes, an E4M3
// scale per 16 weights, an fp32 scale per output), alone or as the gated pair
// of a feed-forward layer: u = silu(x Wg^T) * (x Wu^T).
//
// Each weight is used M <= 8 times, so the weight bytes (4.5 bits per weight)
// bound it, as long as nothing touches the weights one by one: decoded into
// registers for mma.sync they came at 21 weights a clock and SM, where HBM delivers
// 41.  So the weights stay as they are: a tile of 128 rows is the A operand of
// block-scaled FP4 MMAs (kind::mxf4nvf4), codes by TMA, scales by bulk copy and
// tcgen05.cp.  It is x that is brought into the form of the B operand (below).
// Measured, mma.sync form -> this one: one row, 16384 x 12288 weights 35.5 -> 25.4 us
// (4.5 TB/s), gated pair at 12288 x 4608 26.2 -> 17.3 us (3.7 TB/s), of 8 rows 26.5 ->
// 22.5, one row by 4608 x 12288 13.9 -> 12.0, 8 rows 15.0 -> 16.8.  About 4 us of each
// are launch, digits, the first loads' latency and the exchange of sums; the digits of 8
// rows take 2.5 us of the pair's and 4 of the single product's.
//
// A bf16 number is eight bits and a place, so a row's slice of x becomes integers that
// lose nothing: x = v 2^(E - 160), |v| < 2^34, E the exponent field of the slice's
// largest finite element, for every element down to 2^-26 of it.  v is written with
// twelve digits d_p in -4 .. 3 to the base 8, v = sum_p d_p 8^p.  E2M1 holds d / 2
// exactly (0, 1/2, 1, 3/2, 2), so the digits are rows of B (the lower four of two rows of
// x in one 8-row atom, the upper eight of either in another), their block scales 1, and
//   sum_k x W = 2^(E - 159) sum_p 8^p (sum_k (d_p / 2) W):
// the tensor cores' products are exact and summed in fp32, the twelve planes' sums are
// added in fp32.  The MMA's columns are free: with 8, 64 or 256 of them a k-block takes
// the same time, that of issuing its MMAs.
//
// What lies outside those 26 places (elements more than 2^26 times smaller than one of
// their slice, next to an outlier; infinities and NaN) has no digits: the epilogue's
// threads multiply these strays by their weights one by one, in fp32.  12288 normal
// numbers with one of 1e4 in each row, by 4608 weight rows: 12.5 us for one row as
// without it, 25.5 instead of 17.8 for 8; with one of 1e6 23 and 93; of 1e9, where the
// rest of its slice are strays, 0.2 and 1.6 ms.
// (Eight planes, rounded at 2^-22 of the slice's largest element, made 20.7 us of the
// pair's 22.5 at 8 rows and 14.8 of the single product's 16.8, but next to one element of
// 1e6 the outputs that do not see it were off by 3%.)
//
// A cluster's CTAs split K, each keeps the digits of its slice in shared memory
// for all row tiles it meets, and they add up their sums through distributed
// shared memory, each CTA a share of the rows.
#pragma once

#include "ig4_gemm.cuh"
#include "ig4_ptx.cuh"

namespace ig4 {

constexpr int MATVEC_THREADS = 512;  // warps 0-3 epilogue, 4 loads, 5-8 MMAs; all but 4 make digits
constexpr int MATVEC_DIGIT_WARPS = 15;
constexpr int MATVEC_MAX_ITEMS = 10;  // (row, 256-element k-block) pairs per warp
constexpr int MATVEC_MIN_STAGES = 4;  // where shared memory has them; never fewer than issuers
constexpr int MATVEC_MAX_CLUSTER = 8;
constexpr int MATVEC_MAX_K = 24576;
constexpr int MATVEC_STAGE_BYTES = 16384 + 2048;  // codes, scales of 128 rows x 256 elements
constexpr int MATVEC_MAX_STAGES = 10;
constexpr int MATVEC_SMEM = 224 << 10;  // dynamic
constexpr int MATVEC_PLACES = 26;  // v = mantissa << place, the largest element's at this place
// 8-row atoms of B, and with them the columns of an accumulator
__host__ __device__ constexpr int matvec_atoms(int M) { return M + (M + 1) / 2; }
__host__ __device__ constexpr int matvec_width(int M) { return (8 * matvec_atoms(M) + 15) / 16 * 16; }
// Issuing warps, at most; even: one of the gated pair's meets one matrix only
__host__ __device__ constexpr int matvec_slots(int M) { return M > 2 ? 2 : 4; }
// TMEM: two sets of accumulators, the stages' scales (16 columns each), the ones
__host__ __device__ constexpr int matvec_sf_col(int M) { return 2 * matvec_slots(M) * matvec_width(M); }
__host__ __device__ constexpr int matvec_max_stages(int M) {
  const int n = (512 - matvec_sf_col(M) - 4 * matvec_slots(M)) / 16;
  return n < MATVEC_MAX_STAGES ? n : MATVEC_MAX_STAGES;
}
static_assert(matvec_max_stages(1) >= 4 && matvec_max_stages(2) >= 4 && matvec_max_stages(5) >= 4 &&
                  matvec_max_stages(6) >= 4 && matvec_max_stages(8) >= 4, "stages for the issuers");

struct MatvecWeights {
  const uint8_t *codes;
  const uint8_t *sf;
  const float *scale;
};

struct MatvecArgs {
  const __nv_bfloat16 *x;
  const uint8_t *codes[2], *sf[2];
  const float *scale[2];
  const float *bias;
  void *out;
  int M, N, K;
  int tiles, cluster, clusters, stages;
  int kbs;        // k-blocks of a CTA, at most
  int rows_each;  // of a tile's 128 rows, added up by one CTA of the cluster
  // dividers by M, cluster and rows_each: (i * m) >> 16 (an integer division takes about
  // 100 clocks, and there were 30 in front of the first product)
  int div_m, div_cluster, div_rows;
};
constexpr int MATVEC_DIV = 65536;
__host__ __device__ constexpr int matvec_divider(int n) { return (MATVEC_DIV + n - 1) / n; }
__host__ __device__ constexpr int matvec_digit_bytes(int M, int kblocks) {
  return matvec_atoms(M) * kblocks * 1024;
}
__host__ __device__ constexpr int matvec_sum_bytes(int M, int mats, int cluster, int rows_each) {
  return cluster > 1 ? 2 * cluster * mats * M * rows_each * 4 : 0;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// All threads of the cluster meet, without ordering their memory accesses (which would
// wait for the outputs' stores)
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// A bf16 element (in the upper half of w): its mantissa with the leading bit, and the
// place of that mantissa in v for a slice whose largest finite element has exponent field
// emax >= 1.  Negative for what has no digits.
__device__ __forceinline__ int matvec_place(uint32_t w, int emax, uint32_t *mant) {
  const int e = (w >> 23) & 255;
  *mant = ((w >> 16) & 0x7Fu) | (e ? 0x80u : 0u);
  return e == 255 ? -1 : (*mant ? max(e, 1) - emax + MATVEC_PLACES : 0);
}

// Sum over one item's strays (a row of x in a k-block; `lanes`: which eight elements hold
// any) times weight row `row`, for each matrix.  The next eight are on their way while
// these are multiplied.
template <int MATS>
__device__ __forceinline__ void matvec_strays(const MatvecArgs &a, uint32_t lanes, const __nv_bfloat16 *x,
                                              int emax, int k0, int row, float (&sum)[MATS]) {
  struct Eight {
    uint4 x;
    uint32_t code[MATS];
    uint8_t sf[MATS];
  };
  const long code0 = static_cast<long>(row) * (a.K / 2);
  const long sf0 = static_cast<long>(row / 128) * (a.K / 64) * 512 + 16 * (row % 32) + 4 * (row % 128 / 32);
  auto fetch = [&](uint32_t l) {
    const int k = k0 + 8 * (__ffs(l) - 1);
    Eight n;
    n.x = __ldg(reinterpret_cast<const uint4 *>(x + k));
#pragma unroll
    for (int mat = 0; mat < MATS; ++mat) {
      n.code[mat] = __ldg(reinterpret_cast<const uint32_t *>(a.codes[mat] + code0 + k / 2));
      n.sf[mat] = __ldg(a.sf[mat] + sf0 + static_cast<long>(k / 64) * 512 + k / 16 % 4);
    }
    return n;
  };
  Eight next = fetch(lanes);
#pragma unroll 1
  while (lanes != 0) {
    const Eight n = next;
    lanes &= lanes - 1;
    if (lanes != 0) next = fetch(lanes);
    const uint32_t q[4] = {n.x.x, n.x.y, n.x.z, n.x.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w = e & 1 ? q[e / 2] & 0xFFFF0000u : q[e / 2] << 16;
      uint32_t mant;
      if (matvec_place(w, emax, &mant) >= 0) continue;
#pragma unroll
      for (int mat = 0; mat < MATS; ++mat) {
        __nv_fp8_e4m3 sf;
        sf.__x = n.sf[mat];
        const uint32_t code = n.code[mat] >> (4 * e);
        // twice E2M1's values, one in a nibble
        const float two = static_cast<float>((0xC8643210u >> (4 * (code & 7))) & 15u);
        sum[mat] = fmaf(__uint_as_float(w), (code & 8 ? -two : two) * (0.5f * static_cast<float>(sf)),
                        sum[mat]);
      }
    }
  }
}

// Digits of u = v + 04444 4444 (octal: 4 in every digit): octal digit p of u in
// nibble p, less 4, as an E2M1 code of half its value.  (Bits above a digit's
// three may be set in between; the masks of the last step drop them.)
__device__ __forceinline__ uint32_t octal_codes(uint32_t u) {
  u = (u & 0x0000FFFFu) | ((u << 4) & 0xFFFF0000u);
  u = (u & 0x00FF00FFu) | ((u << 2) & 0xFF00FF00u);
  u = (u & 0x0F0F0F0Fu) | ((u << 1) & 0xF0F0F0F0u);
  const uint32_t neg = (~u & 0x44444444u) >> 2;           // 1 in every digit below 4
  return (((u & 0x33333333u) ^ (3 * neg)) + neg) | (neg << 3);  // 4 - d = (3 - d) + 1, sign
}

// Nibbles of neighbouring bytes and words change places: the last two steps of the
// transpositions below
__device__ __forceinline__ void transpose_4x4(uint32_t *w) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t a = w[i], b = w[i + 2];
    w[i] = __byte_perm(a, b, 0x6240);
    w[i + 2] = __byte_perm(a, b, 0x7351);
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
    w[i + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}
// 8 x 8 nibbles transposed: nibble i of w[p] and nibble p of w[i] change places
__device__ __forceinline__ void transpose_nibbles(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
  transpose_4x4(w);
  transpose_4x4(w + 4);
}

// DUAL: tm0, sf[0], scale[0] gate, tm1, .. up.
template <bool DUAL, typename OT>
__global__ void __launch_bounds__(MATVEC_THREADS, 1)
    nvfp4_matvec_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                        const __grid_constant__ MatvecArgs a) {
  constexpr int MATS = DUAL ? 2 : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  __shared__ uint64_t full[MATVEC_MAX_STAGES], empty[MATVEC_MAX_STAGES], tfull[2], tempty[2];
  __shared__ uint64_t sum_full[2], sum_empty[2], drain;
  __shared__ uint32_t tmem_slot, amax[8];
  __shared__ uint32_t stray[MATVEC_MAX_ITEMS * MATVEC_DIGIT_WARPS];  // per item: lanes with strays
  constexpr int STRAY_WORDS = (MATVEC_MAX_ITEMS * MATVEC_DIGIT_WARPS + 31) / 32;
  __shared__ uint32_t stray_items[STRAY_WORDS];  // items with strays
  __shared__ int any_stray;
  __shared__ float inv[2][8];
  __shared__ int abort_word;
  __shared__ alignas(128) uint32_t ones[128];
  volatile int *abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cluster = a.cluster;
  const int rank = cluster > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cl = (static_cast<int>(blockIdx.x) * a.div_cluster) >> 16, n_cl = a.clusters;
  const int nkb = (a.K + 255) / 256;
  const int kb0 = (nkb * rank * a.div_cluster) >> 16, kb1 = (nkb * (rank + 1) * a.div_cluster) >> 16;
  const int M = a.M, N = a.N, K = a.K;
  // [k-block][atom][8 rows][128 bytes], 128-byte swizzle.  Two rows of x make three atoms:
  // their digits 0 to 3, digits 4 to 11 of the first, of the second.
  uint8_t *sB = smem;
  const int atoms = matvec_atoms(M);
  uint8_t *sA = sB + matvec_digit_bytes(M, a.kbs);
  float *sums = reinterpret_cast<float *>(sA + a.stages * MATVEC_STAGE_BYTES);
  // What streams is stages: the k-blocks of a tile, gate and up in turn for DUAL.  A
  // thread takes 930 clocks to issue a stage's four copies and four MMAs, more than
  // HBM needs to bring it (800), so `issuers` warps take the stages in turn, each with
  // an accumulator of its own, and that twice, so that a tile's sums are read while the
  // next tile's grow.  (One accumulator for each of four issuers instead, at M > 4: 16384 x
  // 12288 weights 35 us instead of 32.)
  const int per_tile = (kb1 - kb0) * MATS;
  const int width = matvec_width(M), slots = matvec_slots(M);
  const int issuers = min(slots, per_tile);
  // A stage always has the same issuer: loads may land out of order, and a parity wait
  // cannot tell a stage's use from the one two before, so who waits for a use must
  // have seen the one before it.
  const int stages = issuers == 3 ? a.stages / 3 * 3 : a.stages & -issuers;
  // 64-element steps of a k-block (the last may be short)
  auto steps = [&](int kb) { return min(4, K / 64 - 4 * kb); };

  // The thread that loads prepares the barriers itself, so that weights and x are on
  // their way while the CTA (and its peers) set up the rest.
  if (warp == 4 && lane == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], issuers);
      mbar_init(&tempty[b], 128);
      mbar_init(&sum_full[b], 4 * cluster);
      mbar_init(&sum_empty[b], 4 * cluster);
    }
    mbar_init(&drain, issuers);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm0);
    if constexpr (DUAL) tma_prefetch_desc(&tm1);
  }
  if (threadIdx.x < 128) ones[threadIdx.x] = 0x38383838u;  // E4M3 1
  if (threadIdx.x < 8) amax[threadIdx.x] = 0;
  if (threadIdx.x < STRAY_WORDS) stray_items[threadIdx.x] = 0;
  if (threadIdx.x == 8) any_stray = 0;
  pdl_wait();
  pdl_trigger();

  // ---------------- loads, in the order of the MMAs: tiles, k-blocks, matrices.
  // One thread's instructions are the limit here and at the MMAs (about 5 clocks
  // each): addresses advance by additions.
  int ld_row = cl * 128, ld_c0 = kb0 * 128, ld_s = 0, ld_mat = 0;
  uint32_t ld_ph = 0, ld_sf_bytes = steps(kb0) * 512;
  const long sf_first = (static_cast<long>(cl) * (K / 64) + 4 * kb0) * 512;
  const long sf_tile = static_cast<long>(n_cl) * (K / 64) * 512;
  const uint8_t *sf0 = a.sf[0] + sf_first, *sf1 = a.sf[1] + sf_first;  // of this tile
  const int ld_rows = a.tiles * 128, c0_end = kb1 * 128;
  long ld_off = 0;  // of this k-block in the tile's scales
  uint8_t *ld_st = sA;
  auto issue = [&]() {
    uint64_t *bar = &full[ld_s];
    mbar_arrive_expect_tx(bar, 16384 + ld_sf_bytes);
    if (DUAL && ld_mat) {
      tma_load_2d(ld_st, &tm1, bar, ld_c0, ld_row);
      bulk_load(ld_st + 16384, sf1 + ld_off, ld_sf_bytes, bar);
    } else {
      tma_load_2d(ld_st, &tm0, bar, ld_c0, ld_row);
      bulk_load(ld_st + 16384, sf0 + ld_off, ld_sf_bytes, bar);
    }
    ld_st += MATVEC_STAGE_BYTES;
    if (++ld_s == stages) {
      ld_s = 0;
      ld_st = sA;
      ld_ph ^= 1;
    }
    if (DUAL && (ld_mat ^= 1)) return;
    ld_c0 += 128;
    ld_off += 2048;
    if (ld_c0 == c0_end) {
      ld_c0 = kb0 * 128;
      ld_off = 0;
      ld_row += n_cl * 128;
      sf0 += sf_tile;
      sf1 += sf_tile;
    }
    ld_sf_bytes = min(2048, 8 * K - 16 * ld_c0);  // 8 bytes per element of K
  };
  if (warp == 4 && lane == 0)
    for (int i = 0; i < stages && ld_row < ld_rows; ++i) issue();
  // x: an item (k-block, row) per warp and step
  const int items = (kb1 - kb0) * M, w0 = warp - (warp > 4);
  uint4 v[MATVEC_MAX_ITEMS];
#pragma unroll
  for (int t = 0; t < MATVEC_MAX_ITEMS; ++t) {
    const int i = w0 + MATVEC_DIGIT_WARPS * t;
    v[t] = make_uint4(0, 0, 0, 0);
    if (warp != 4 && i < items) {
      const int b = (i * a.div_m) >> 16, m = i - b * M;
      const int k = (kb0 + b) * 256 + 8 * lane;
      if (k < K) v[t] = __ldg(reinterpret_cast<const uint4 *>(a.x + m * K + k));
    }
  }
  if (warp == 5) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  if (cluster > 1)
    cluster_sync_all();  // peers' barriers are set up
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  if (warp == 4) {
    __syncthreads();
  } else {
    // ---------------- digits of x
#pragma unroll
    for (int t = 0; t < MATVEC_MAX_ITEMS; ++t) {
      const int i = w0 + MATVEC_DIGIT_WARPS * t;
      if (i >= items) break;
      const uint32_t q[4] = {v[t].x, v[t].y, v[t].z, v[t].w};
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t w = (e & 1 ? q[e / 2] : q[e / 2] << 16) & 0x7FFF0000u;
        m = max(m, w < 0x7F800000u ? w : 0u);  // the finite ones
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) atomicMax(&amax[i - ((i * a.div_m) >> 16) * M], m);
    }
    asm volatile("bar.sync 1, 480;" ::: "memory");
    if (threadIdx.x < 8) {
      // 2^(E - 159) in two factors
      const int ex = static_cast<int>(max(amax[threadIdx.x] >> 23, 1u)) - 159, h = ex >> 1;
      inv[0][threadIdx.x] = __uint_as_float(static_cast<uint32_t>(127 + h) << 23);
      inv[1][threadIdx.x] = __uint_as_float(static_cast<uint32_t>(127 + ex - h) << 23);
    }
    // (a loop, its x read again from the cache: ten copies of this code took 1.5 us longer
    // for one row, fetching instructions)
    auto item_x = [&](int i) {
      const int b = (i * a.div_m) >> 16, m = i - b * M, k = (kb0 + b) * 256 + 8 * lane;
      return i < items && k < K ? __ldg(reinterpret_cast<const uint4 *>(a.x + m * K + k))
                                : make_uint4(0, 0, 0, 0);
    };
    uint4 next = v[0];
#pragma unroll 1
    for (int i = w0; i < items; i += MATVEC_DIGIT_WARPS) {
      const int b = (i * a.div_m) >> 16, m = i - b * M;
      const int emax = static_cast<int>(max(amax[m] >> 23, 1u));
      const uint32_t q[4] = {next.x, next.y, next.z, next.w};
      next = item_x(i + MATVEC_DIGIT_WARPS);
      // least (below zero comes last) and largest magnitude of the lane's elements
      uint32_t least = 0xFFFFFFFFu, most = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t n = (e & 1 ? q[e / 2] : q[e / 2] << 16) & 0x7FFF0000u;
        least = min(least, n - 1);
        most = max(most, n);
      }
      // v = (w - 04444 4444) 2^12 + what the lower digits, in z, hold
      uint32_t w[8], z[4] = {0, 0, 0, 0}, lanes = 0;
      const bool flat = least >= (static_cast<uint32_t>(max(emax - MATVEC_PLACES + 12, 1)) << 23) - 1 &&
                        most < 0x7F800000u;
      if (__all_sync(0xffffffffu, flat)) {  // no lower digits: v 2^-12 = x 2^sh by fp32
        const int sh = 148 - emax, h = sh / 2;
        const float s0 = __uint_as_float(static_cast<uint32_t>(127 + h) << 23);
        const float s1 = __uint_as_float(static_cast<uint32_t>(127 + sh - h) << 23);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = __uint_as_float(e & 1 ? q[e / 2] & 0xFFFF0000u : q[e / 2] << 16);
          // 1.5 * 2^23 + v 2^-12: an integer in the low bits of the float
          w[e] = __float_as_uint(fmaf(x * s0, s1, 12582912.0f)) - 0x4B400000u + 044444444u;
        }
      } else {
        bool lost = false;
        uint32_t low[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = e & 1 ? q[e / 2] & 0xFFFF0000u : q[e / 2] << 16;
          uint32_t n;
          const int s = matvec_place(x, emax, &n);
          lost |= s < 0;
          const uint32_t hi = s >= 12 ? n << (s - 12) : 0u, lo = s >= 0 && s < 12 ? n << s : 0u;
          const uint32_t neg = static_cast<uint32_t>(static_cast<int>(x) >> 31);
          const uint32_t u = (lo ^ neg) - neg + 04444u;
          w[e] = (hi ^ neg) - neg + static_cast<uint32_t>(static_cast<int>(u) >> 12) + 044444444u;
          low[e] = u & 0xFFFu;
        }
        lanes = __ballot_sync(0xffffffffu, lost);
        if (lane == 0 && lanes != 0) {
          any_stray = 1;
          atomicOr(&stray_items[i >> 5], 1u << (i & 31));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = octal_codes(low[e] | (low[e + 4] << 12));
        transpose_4x4(z);
      }
      if (lane == 0) stray[i] = lanes;
      uint8_t *low_atom = sB + (b * atoms + 3 * (m >> 1)) * 1024 + 4 * (lane & 3);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int r = 4 * (m & 1) + p;
        *reinterpret_cast<uint32_t *>(low_atom + 128 * r + 16 * ((lane >> 2) ^ r)) = z[p];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = octal_codes(w[e]);
      transpose_nibbles(w);
      uint8_t *atom = low_atom + (1 + (m & 1)) * 1024;
#pragma unroll
      for (int p = 0; p < 8; ++p)
        *reinterpret_cast<uint32_t *>(atom + 128 * p + 16 * ((lane >> 2) ^ p)) = w[p];
    }
    fence_proxy_async_smem();
    __syncthreads();
  }

  if (warp == 4) {
    if (lane == 0) {
      bool ok = true;
      while (ld_row < ld_rows) {
        // (the first `stages` loads are past; the wait is for the stage's last use)
        if (!mbar_wait(&empty[ld_s], ld_ph ^ 1, abort_flag)) {
          ok = false;
          break;
        }
        issue();
      }
      if (!ok) sleep_ns(50000);  // let the loads already issued land
    }
  } else if (warp >= 5 && warp < 5 + issuers) {
    if (lane == 0) {
      const int me = warp - 5;
      const uint32_t idesc = idesc_nvf4(128, 8 * atoms);
      const uint32_t sf_col = tmem + matvec_sf_col(M), sfb = sf_col + 16 * a.stages + 4 * me;
      tmem_cp_sf(sfb, sdesc_kmajor_none(smem_u32(ones), 128));
      // descriptors: address / 16 in the low bits
      const uint64_t ad0 = sdesc_kmajor_sw128(smem_u32(sA)), bd0 = sdesc_kmajor_sw128(smem_u32(sB));
      const uint64_t sd0 = sdesc_kmajor_none(smem_u32(sA) + 16384, 128);
      int local = 0;
      bool ok = true;
      for (int tile = cl; tile < a.tiles && ok; tile += n_cl, ++local) {
        const int buf = local & 1;
        if (!mbar_wait(&tempty[buf], ((local >> 1) & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem + (buf * slots + me) * width;
        // of the CTA's stages this tile's are g0 .. g0 + per_tile - 1, mine the ones that
        // are `me` modulo `issuers`
        int first = me, s = me;
        uint32_t ph = 0;
        if (local > 0) {
          const uint32_t g0 = static_cast<uint32_t>(local) * per_tile;
          first = (me + issuers - static_cast<int>(g0 % issuers)) % issuers;
          s = static_cast<int>((g0 + first) % stages);
          ph = ((g0 + first) / stages) & 1;
        }
        for (int i = first; i < per_tile; i += issuers) {
          if (!mbar_wait(&full[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int kb = static_cast<unsigned>(i) / MATS, n = steps(kb0 + kb);
          const uint64_t ad = ad0 + s * (MATVEC_STAGE_BYTES / 16), sd = sd0 + s * (MATVEC_STAGE_BYTES / 16);
          const uint64_t bd = bd0 + kb * (64 * atoms);
          const uint32_t sfa = sf_col + 16 * s;
          if (n == 4) {
#pragma unroll
            for (int j = 0; j < 4; ++j) tmem_cp_sf(sfa + 4 * j, sd + 32 * j);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              umma_nvf4(d, ad + 2 * j, bd + 2 * j, idesc, sfa + 4 * j, sfb, i != first || j != 0);
          } else {
            for (int j = 0; j < n; ++j) {
              tmem_cp_sf(sfa + 4 * j, sd + 32 * j);
              umma_nvf4(d, ad + 2 * j, bd + 2 * j, idesc, sfa + 4 * j, sfb, i != first || j != 0);
            }
          }
          umma_commit(&empty[s]);
          s += issuers;
          if (s >= stages) {
            s -= stages;
            ph ^= 1;
          }
        }
        if (ok) umma_commit(&tfull[buf]);
      }
      umma_commit(&drain);
      mbar_wait(&drain, 0, nullptr, WAIT_LIMIT_NS / 4);
    }
  } else if (warp < 4) {
    const int r = threadIdx.x;  // row of the tile
    const int re = a.rows_each;
    OT *out = static_cast<OT *>(a.out);
    // the row of a tile whose outputs this thread writes, for all rows of x or every
    // `groups`th: its own without a cluster, else one of the CTA's share
    const int groups = (128 * a.div_rows) >> 16;  // 1 without a cluster
    const int group = (r * a.div_rows) >> 16, rl = r - group * re;
    const int my_row = cluster > 1 ? rank * re + rl : r;
    float sc0 = 0.0f, sc1 = 0.0f, bias = 0.0f;
    auto finish = [&](int m, int row, float v0, float v1) {
      float v;
      if constexpr (DUAL)
        v = silu_f(v0 * sc0) * (v1 * sc1);
      else
        v = fmaf(v0, sc0, bias);
      OT *op = out + static_cast<long>(m) * N + row;
      if constexpr (sizeof(OT) == 4)
        *op = v;
      else
        *op = __float2bfloat16_rn(v);
    };
    int local = 0;
    for (int tile = cl; tile < a.tiles; tile += n_cl, ++local) {
      const int buf = local & 1;
      const uint32_t use = static_cast<uint32_t>(local >> 1) & 1;
      const int row = tile * 128 + my_row;
      const bool mine = row < N && my_row < 128 && group < groups;
      if (mine) {  // on their way while the sums grow
        sc0 = __ldg(a.scale[0] + row);
        if constexpr (DUAL) sc1 = __ldg(a.scale[1] + row);
        if (!DUAL && a.bias != nullptr) bias = __ldg(a.bias + row);
      }
      if (!mbar_wait_warp(&tfull[buf], use, abort_flag)) break;
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(warp * 32) << 16) + buf * slots * width;
      float y[MATS][8];
#pragma unroll
      for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
          if (c >= M) continue;
          // 24 columns of two rows (the rest is not used); two issuers' sums at a time
          const uint32_t at = acc + mat * width + 12 * c;
          float d[32], f[32];
          tmem_ld32(at, d);
          if (mat + MATS < issuers) tmem_ld32(at + MATS * width, f);
          tmem_ld_wait();
          if (mat + MATS < issuers) {
#pragma unroll
            for (int i = 0; i < 24; ++i) d[i] += f[i];
          }
          for (int h = mat + 2 * MATS; h < issuers; h += MATS) {
            tmem_ld32(at + (h - mat) * width, f);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 24; ++i) d[i] += f[i];
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float h = d[8 * i + 15];
#pragma unroll
            for (int p = 6; p >= 0; --p) h = fmaf(h, 8.0f, d[8 * i + 8 + p]);
#pragma unroll
            for (int p = 3; p >= 0; --p) h = fmaf(h, 8.0f, d[4 * i + p]);
            y[mat][c + i] = h * inv[0][c + i] * inv[1][c + i];
          }
        }
      tc_fence_before();
      mbar_arrive(&tempty[buf]);
      if (any_stray) {
#pragma unroll 1
        for (int w = 0; 32 * w < items; ++w)
#pragma unroll 1
          for (uint32_t left = stray_items[w]; left != 0; left &= left - 1) {
            const int i = 32 * w + __ffs(left) - 1, b = (i * a.div_m) >> 16, m = i - b * M;
            float z[MATS] = {};
            matvec_strays<MATS>(a, stray[i], a.x + m * K, static_cast<int>(max(amax[m] >> 23, 1u)),
                                (kb0 + b) * 256, min(tile * 128 + r, N - 1), z);
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (c == m) y[mat][c] += z[mat];
          }
      }
      if (cluster == 1) {
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (m < M && mine) finish(m, row, y[0][m], y[MATS - 1][m]);
        continue;
      }
      // every CTA's sums of rows q * rows_each + .. to CTA q:
      // sums [buffer][from][matrix][row of x][row]
      if (!mbar_wait_cluster_warp(&sum_empty[buf], use ^ 1, abort_flag)) break;
      const int base = (buf * cluster + rank) * MATS * M * re + rl;
      const uint32_t dst = map_shared_to_rank(sums + base, group);
#pragma unroll
      for (int mat = 0; mat < MATS; ++mat)
#pragma unroll
        for (int m = 0; m < 8; ++m)
          if (m < M) st_cluster_f32(dst + 4 * (mat * M + m) * re, y[mat][m]);
      __syncwarp();
      if (lane < cluster) mbar_arrive_cluster(map_shared_to_rank(&sum_full[buf], lane));
      if (!mbar_wait_cluster_warp(&sum_full[buf], use, abort_flag)) break;
      if (mine) {
        for (int m = group; m < M; m += groups) {
          float z[2] = {0.0f, 0.0f};
          const float *p = sums + buf * cluster * MATS * M * re + m * re + rl;
          for (int f = 0; f < cluster; ++f)
#pragma unroll
            for (int mat = 0; mat < MATS; ++mat) z[mat] += p[(f * MATS + mat) * M * re];
          finish(m, row, z[0], z[MATS - 1]);
        }
      }
      if (tile + 2 * n_cl >= a.tiles) continue;  // (nobody writes this buffer again)
      __syncwarp();
      if (lane < cluster) mbar_arrive_cluster(map_shared_to_rank(&sum_empty[buf], lane));
    }
  }

  __syncwarp();
  tc_fence_before();
  if (cluster > 1)
    cluster_meet();  // shared memory stays until the last remote store
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, 512);
}

}  // namespace ig4
