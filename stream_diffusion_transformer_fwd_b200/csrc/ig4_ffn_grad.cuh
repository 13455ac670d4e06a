// ig4_ffn_grad.cuh - gradients of the SwiGLU hidden state
// u = silu(G) * U, G = h Wg^T, U = h Wu^T, for sm_100a.
//
//   dU = du G sig(G),  dG = du U sig(G) (1 + G (1 - sig(G)))
//   dh = dG Wg + dU Wu,   dWg = dG^T h,   dWu = dU^T h
//
// Three tensor-core GEMMs of 4 M I K flops each.  The first recomputes G and U
// (the forward keeps neither: 4 M I bytes saved per layer) on the forward's
// dual-B tiles; its epilogue turns the two fp32 accumulators and du into dG
// and dU and stores them side by side as P [M][2I] in bf16, the type the next
// two GEMMs' tensor-core operands have (one rounding of 2^-9 relative per
// factor, as the forward rounds u).  dh contracts P with [Wg; Wu] over 2I in
// one fp32 accumulator; dW contracts P with h over the tokens.
//
// Both later GEMMs contract over a dimension that is not contiguous in
// memory: the rows of W for dh, the tokens for dW.  tcgen05 reads such
// operands directly in MN-major form (64 contiguous elements by 8 contraction
// rows per 128-byte-swizzled 1 KB atom), so nothing is transposed in memory.
// Tokens past M read as zero from the TMA loads and add nothing.
//
// 12288 x 4608 weights: 4608 tokens (3131 GFLOP) 2.40 to 2.54 ms, 1.23 to 1.30 PFLOP/s
// at the power-capped clock, where cuBLAS sustains 1.39; 1152 tokens 0.61 to 0.72 ms,
// depending on the GPU (recomputation, dh and dW 190 to 205 us each, tensor pipe 85, 89
// and 78% of active cycles); 17 tokens, dh only, 79 to 82 us.
#pragma once

#include "ig4_gemm.cuh"
#include "ig4_ptx.cuh"

namespace ig4 {

// Shared-memory descriptor of an MN-major operand in the 128-byte-swizzle
// layout: slabs of 64 MN-elements (128 bytes) by 64 contraction rows, 8 KB
// apart (leading offset), 8-row groups 1 KB apart (stride offset).  One K = 16
// step starts 16 rows (2 KB) further on.
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192u >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// idesc_bf16 with A and / or B MN-major (bits 15, 16)
__host__ __device__ constexpr uint32_t idesc_bf16_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u);
}

// dG and dU of one element
__device__ __forceinline__ void swiglu_grad(float g, float u, float du, float *dg, float *dup) {
  const float sig = 1.0f / (1.0f + __expf(-g));
  const float a = du * sig;
  *dg = a * u * fmaf(g, 1.0f - sig, 1.0f);
  *dup = a * g;
}

// Epilogue of the recomputation: accumulator columns [0,128) hold G, [128,256)
// hold U of output columns n .. n + 127; writes dG to p[row][n..] and dU to
// p[row][I + n..].
struct EpiSwiGLUGrad {
  const __nv_bfloat16 *du;
  __nv_bfloat16 *p;
  int I, M;

  __device__ __forceinline__ void operator()(int m0, int n0, uint32_t tacc, int r) const {
    const int row = m0 + r;
    const bool valid = row < M;
    const int n = n0 / 2;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      float g[32], up[32];
      tmem_ld32(tacc + c, g);
      tmem_ld32(tacc + 128 + c, up);
      tmem_ld_wait();
      if (valid) {
        float d[32];
        load32_bf16(du + static_cast<long>(row) * I + n + c, d);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          swiglu_grad(g[i], up[i], d[i], &g[i], &up[i]);
        }
        __nv_bfloat16 *dst = p + static_cast<long>(row) * 2 * I + n + c;
        store32_bf16(dst, g);
        store32_bf16(dst + I, up);
      }
      __syncwarp();  // tmem_ld32 takes the whole warp: rows past M wait here
    }
  }
};

// Tiled TMA store of a box in shared memory (clipped at the tensor's ends)
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int c0, int c1) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(m)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the latest N of this thread's bulk stores have read their source
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Work of a gradient GEMM.  Tiles 0 .. full - 1, a multiple of the pairs, are
// whole items.  The rest would leave most pairs idle for a whole tile's time,
// so each is cut along the contraction into `shares` items whose fp32 sums go to
// part [tile - full][share][256][256] and are added by grad_reduce_kernel.
struct GradPlan {
  int m_tiles, n_tiles, group_m;
  int full, shares, items;
  int kblocks, kb0;  // the contraction runs over B0 for kb0 k-blocks, then over B1
  int rows, N;       // of the output; rows from split_row on go to the second map
  int split_row;
  float *part;
};
struct GradItem {
  int mt, nt, share, b0, nkb;  // tile, contraction share (-1: whole), first k-block, k-blocks
};
__device__ __forceinline__ GradItem grad_item(const GradPlan &p, int t) {
  GradItem i;
  int tile = t;
  i.share = -1;
  i.b0 = 0;
  i.nkb = p.kblocks;
  if (t >= p.full) {
    const int e = t - p.full;
    tile = p.full + e / p.shares;
    if (p.shares > 1) {
      i.share = e % p.shares;
      i.b0 = static_cast<int>(static_cast<long>(p.kblocks) * i.share / p.shares);
      i.nkb = static_cast<int>(static_cast<long>(p.kblocks) * (i.share + 1) / p.shares) - i.b0;
    }
  }
  tile_coords(tile, p.m_tiles, p.n_tiles, p.group_m, &i.mt, &i.nt);
  return i;
}

// C = A B on CTA pairs, B MN-major, A K-major (dh) or MN-major (dW).
// A K-major: tmA maps A [rows][contraction] in boxes of 128 rows x 64; MN-major
// operands: 3-D maps {64 elements, contraction rows, slabs of 64 elements} in
// boxes {64, 64, 2}.  Roles, barriers and the two TMEM accumulators are those of
// gemm_pair_kernel.
//
// The results leave through shared memory by TMA stores, 64 columns at a time:
// a lane holds a row of the accumulator, and storing its 64 bytes directly, row
// after row 2 N bytes apart, took 13,000 cycles a tile, more than the MMAs of a
// tile take below 1600 tokens.
constexpr int GRAD_STAGES = 6;
constexpr int GRAD_STAGE_BYTES = 2 * 16384;
constexpr int GRAD_OUT_BYTES = 32 * 128;  // 32 rows x 64 columns
constexpr int GRAD_OUT_SLOTS = 2;         // per epilogue warp
constexpr int GRAD_SMEM_BYTES =
    GRAD_STAGES * GRAD_STAGE_BYTES + 4 * GRAD_OUT_SLOTS * GRAD_OUT_BYTES + 1024 + 256;

template <bool A_MN>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    grad_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
                     const __grid_constant__ CUtensorMap tmB1, const __grid_constant__ CUtensorMap tmO0,
                     const __grid_constant__ CUtensorMap tmO1, const GradPlan p) {
  constexpr uint32_t IDESC = idesc_bf16_major(2 * GEMM_BM, 256, A_MN, true);
  constexpr uint32_t TMEM_COLS = 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  uint8_t *sA = smem;
  uint8_t *sB = smem + GRAD_STAGES * 16384;
  uint8_t *sO = smem + GRAD_STAGES * GRAD_STAGE_BYTES;
  uint64_t *full = reinterpret_cast<uint64_t *>(sO + 4 * GRAD_OUT_SLOTS * GRAD_OUT_BYTES);
  uint64_t *empty = full + GRAD_STAGES;
  uint64_t *tfull = empty + GRAD_STAGES;
  uint64_t *tempty = tfull + 2;
  uint64_t *drain = tempty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  const int n_pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < GRAD_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB0);
    tma_prefetch_desc(&tmB1);
    tma_prefetch_desc(&tmO0);
    tma_prefetch_desc(&tmO1);
  }
  if (warp == 5) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 4) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      int local = 0;
      for (int t = pair; t < p.items && ok; t += n_pairs, ++local) {
        const GradItem w = grad_item(p, t);
        for (int it = 0; it < w.nkb; ++it) {
          const int kb = w.b0 + ((local & 1) ? w.nkb - 1 - it : it);  // K-snake
          if (!mbar_wait_cluster(&empty[s], ph ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * GRAD_STAGE_BYTES);
          const uint32_t bar = map_shared_to_rank(&full[s], 0);
          const int am = w.mt * 2 * GEMM_BM + static_cast<int>(rank) * GEMM_BM;
          if constexpr (A_MN)
            tma_load_3d_pair(sA + s * 16384, &tmA, bar, 0, kb * 64, am / 64);
          else
            tma_load_2d_pair(sA + s * 16384, &tmA, bar, kb * 64, am);
          const int bn = (w.nt * 256 + static_cast<int>(rank) * 128) / 64;
          if (kb < p.kb0)
            tma_load_3d_pair(sB + s * 16384, &tmB0, bar, 0, kb * 64, bn);
          else
            tma_load_3d_pair(sB + s * 16384, &tmB1, bar, 0, (kb - p.kb0) * 64, bn);
          if (++s == GRAD_STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) sleep_ns(50000);  // let the loads already issued land
    }
  } else if (warp == 5) {
    if (lane == 0 && rank == 0) {
      int s = 0;
      uint32_t ph = 0;
      int local = 0;
      bool ok = true;
      for (int t = pair; t < p.items && ok; t += n_pairs, ++local) {
        const int buf = local & 1;
        const uint32_t use = static_cast<uint32_t>(local >> 1);
        if (!mbar_wait_cluster(&tempty[buf], (use & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + buf * 256;
        const int nkb = grad_item(p, t).nkb;
        for (int it = 0; it < nkb; ++it) {
          if (!mbar_wait_cluster(&full[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(sA + s * 16384);
          const uint32_t b_base = smem_u32(sB + s * 16384);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t ad = A_MN ? sdesc_mnmajor_sw128(a_base + kk * 2048)
                                     : sdesc_kmajor_sw128(a_base + kk * 32);
            const uint64_t bd = sdesc_mnmajor_sw128(b_base + kk * 2048);
            umma_bf16_pair(d_tmem, ad, bd, IDESC, (it | kk) != 0);
          }
          umma_commit_pair_both(&empty[s]);
          if (++s == GRAD_STAGES) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) umma_commit_pair_both(&tfull[buf]);
      }
      umma_commit_pair_both(drain);
      mbar_wait_cluster(drain, 0, nullptr, WAIT_LIMIT_NS / 4);
    }
  } else {
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t tempty_leader0 = map_shared_to_rank(&tempty[0], 0);
    const uint32_t tempty_leader1 = map_shared_to_rank(&tempty[1], 0);
    uint8_t *out = sO + warp * GRAD_OUT_SLOTS * GRAD_OUT_BYTES;  // 1024-byte aligned: the swizzle's period
    int local = 0, slot = 0;
    for (int t = pair; t < p.items; t += n_pairs, ++local) {
      const int buf = local & 1;
      const uint32_t use = static_cast<uint32_t>(local >> 1);
      const bool ok = mbar_wait_cluster(&tfull[buf], use & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const GradItem w = grad_item(p, t);
      const uint32_t tacc = tmem_base + lane_base + buf * 256;
      const int n0 = w.nt * 256;
      const int row0 = w.mt * 2 * GEMM_BM + static_cast<int>(rank) * GEMM_BM + warp * 32;
      if (w.share >= 0) {
        const int tile = (t - p.full) / p.shares;
        float *dst = p.part + ((static_cast<long>(tile) * p.shares + w.share) * 256 +
                               rank * GEMM_BM + warp * 32 + lane) * 256;
#pragma unroll 1
        for (int c = 0; c < 256; c += 32) {
          float v[32];
          tmem_ld32(tacc + c, v);
          tmem_ld_wait();
          if (row0 + lane < p.rows && n0 + c < p.N) store32_f32(dst + c, v);
          __syncwarp();  // tmem_ld32 takes the whole warp
        }
      } else {
#pragma unroll 1
        for (int c = 0; c < 256; c += 64) {
          float v[32], u[32];
          tmem_ld32(tacc + c, v);
          tmem_ld32(tacc + c + 32, u);
          tmem_ld_wait();
          if (n0 + c >= p.N || row0 >= p.rows) continue;  // (uniform in the warp)
          uint8_t *o = out + slot * GRAD_OUT_BYTES;
          if (lane == 0) bulk_wait_read<GRAD_OUT_SLOTS - 1>();  // this slot's last store has read it
          __syncwarp();
          // row `lane`, 16-byte chunk q at q ^ (row % 8): the 128-byte swizzle
          uint8_t *orow = o + lane * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            *reinterpret_cast<uint4 *>(orow + ((q ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                           pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                           pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
            *reinterpret_cast<uint4 *>(orow + (((q + 4) ^ (lane & 7)) << 4)) =
                make_uint4(pack_bf16x2(u[8 * q], u[8 * q + 1]), pack_bf16x2(u[8 * q + 2], u[8 * q + 3]),
                           pack_bf16x2(u[8 * q + 4], u[8 * q + 5]),
                           pack_bf16x2(u[8 * q + 6], u[8 * q + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < p.split_row)
              tma_store_2d(&tmO0, o, n0 + c, row0);
            else
              tma_store_2d(&tmO1, o, n0 + c, row0 - p.split_row);
            bulk_commit();
          }
          if (++slot == GRAD_OUT_SLOTS) slot = 0;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(buf ? tempty_leader1 : tempty_leader0);
    }
    if (lane == 0) bulk_wait_all();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 5) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// The split tiles' sums: out = bf16 of the sum of a tile's partials, in share
// order.  Grid (split tiles, 32): a CTA takes 8 rows of a tile, a thread 8
// columns of one row.
__global__ void __launch_bounds__(256) grad_reduce_kernel(const GradPlan p, __nv_bfloat16 *out) {
  pdl_wait();
  pdl_trigger();
  int mt, nt;
  tile_coords(p.full + blockIdx.x, p.m_tiles, p.n_tiles, p.group_m, &mt, &nt);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5), c = (threadIdx.x & 31) * 8;
  const int row = mt * 256 + r, col = nt * 256 + c;
  if (row >= p.rows || col >= p.N) return;
  const float *src = p.part + (static_cast<long>(blockIdx.x) * p.shares * 256 + r) * 256 + c;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  for (int z = 0; z < p.shares; ++z) {
    const float4 u = *reinterpret_cast<const float4 *>(src + static_cast<long>(z) * 65536);
    const float4 v = *reinterpret_cast<const float4 *>(src + static_cast<long>(z) * 65536 + 4);
    a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
    b.x += v.x; b.y += v.y; b.z += v.z; b.w += v.w;
  }
  *reinterpret_cast<uint4 *>(out + static_cast<long>(row) * p.N + col) =
      make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                 pack_bf16x2(b.z, b.w));
}

// ------------------------------------------------------- up to 128 tokens
// With few tokens the weights' bytes bound the first two products.  Tokens as the
// MMA's 128 or 256 rows would spend most of it on empty rows (26 us of MMAs for 17
// tokens at full width, as much as the bytes take), so here the weights are the
// 128-row operand and the tokens, rounded up to 16, its columns.
//   G^T, U^T (DH false): a CTA takes R rows of both weights, R chosen so that the
//     CTAs cover all SMs evenly; the MMA's rows past R compute on what the stage
//     holds there, and nothing reads them.
//   dh^T (DH true): A is W MN-major, 128 of its columns; the contraction over 2I
//     is cut into shares, whose fp32 sums [share][M][K] grad_rows_reduce_kernel
//     adds (none with one share).
// 17 tokens at 12288 x 4608: 47 us for G, U (227 MB, 4.9 TB/s) and 41 us for dh (5.5 TB/s)
// by themselves with a cold L2, 79 to 82 us together; 1 token 78, 64 90, 128 105.  The
// weights (226 MB) are read by both products and do not fit L2 (126 MB) between them.
struct GradRowsPlan {
  int tiles, R;      // output tiles; weight rows (DH: columns, 128) of each
  int nt;            // tokens rounded up to 16
  int shares, items;
  int kblocks, kb0;  // as in GradPlan
  int stages;
  int M, I, K;
};
constexpr int GRAD_ROWS_SMEM = 220 << 10;
__host__ __device__ constexpr int grad_rows_stage_bytes(bool dh, int nt) {
  return (dh ? 16384 : 32768) + nt * 128;
}

template <bool DH>
__global__ void __launch_bounds__(GEMM_THREADS, 1)
    grad_rows_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                     const __grid_constant__ CUtensorMap tmB, const GradRowsPlan p,
                     const __nv_bfloat16 *du, __nv_bfloat16 *out, float *part) {
  constexpr uint32_t TMEM_COLS = DH ? 128 : 256;
  constexpr int B_OFF = DH ? 16384 : 32768;
  constexpr int MAX_STAGES = 13;  // 220 KB / (16 KB + 16 tokens)
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = align1024(smem_raw);
  const int stage_bytes = grad_rows_stage_bytes(DH, p.nt);
  __shared__ uint64_t full[MAX_STAGES], empty[MAX_STAGES], tfull, tempty, drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int *abort_flag = &abort_word;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&tfull, 1);
    mbar_init(&tempty, 128);
    mbar_init(&drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 && lane == 0) {
    tma_prefetch_desc(&tmA0);
    tma_prefetch_desc(&tmA1);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 5) {
    tmem_alloc(&tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = tmem_slot;
  pdl_wait();
  pdl_trigger();

  // item t: tile t / shares, k-blocks [first, last) of share t % shares
  auto first_kb = [&](int z) { return static_cast<int>(static_cast<long>(p.kblocks) * z / p.shares); };

  if (warp == 4) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      long issued = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.items && ok; t += gridDim.x) {
        const int tile = t / p.shares, z = t % p.shares;
        for (int kb = first_kb(z); kb < first_kb(z + 1); ++kb) {
          if (!mbar_wait(&empty[s], ph ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t *st = smem + s * stage_bytes;
          if constexpr (DH) {
            mbar_arrive_expect_tx(&full[s], stage_bytes);
            if (kb < p.kb0)
              tma_load_3d(st, &tmA0, &full[s], 0, kb * 64, tile * 2);
            else
              tma_load_3d(st, &tmA1, &full[s], 0, (kb - p.kb0) * 64, tile * 2);
          } else {
            mbar_arrive_expect_tx(&full[s], (2 * p.R + p.nt) * 128);
            tma_load_2d(st, &tmA0, &full[s], kb * 64, tile * p.R);
            tma_load_2d(st + 16384, &tmA1, &full[s], kb * 64, tile * p.R);
          }
          tma_load_2d(st + B_OFF, &tmB, &full[s], kb * 64, 0);
          ++issued;
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
      if (!ok) {
        // Let the loads already issued land before the CTA's shared memory goes away.
        for (long i = (issued > p.stages ? issued - p.stages : 0); i < issued; ++i)
          mbar_wait(&full[i % p.stages], static_cast<uint32_t>((i / p.stages) & 1), nullptr,
                    WAIT_LIMIT_NS / 4);
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16_major(128, p.nt, DH, false);
      int s = 0;
      uint32_t ph = 0;
      uint32_t local = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < p.items && ok; t += gridDim.x, ++local) {
        const int z = t % p.shares;
        if (!mbar_wait(&tempty, (local & 1) ^ 1, abort_flag)) break;
        tc_fence_after();
        const int b0 = first_kb(z), nkb = first_kb(z + 1) - b0;
        for (int it = 0; it < nkb; ++it) {
          if (!mbar_wait(&full[s], ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(smem + s * stage_bytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t bd = sdesc_kmajor_sw128(a_base + B_OFF + kk * 32);
            if constexpr (DH) {
              umma_bf16(tmem_base, sdesc_mnmajor_sw128(a_base + kk * 2048), bd, idesc, (it | kk) != 0);
            } else {
              umma_bf16(tmem_base, sdesc_kmajor_sw128(a_base + kk * 32), bd, idesc, (it | kk) != 0);
              umma_bf16(tmem_base + 128, sdesc_kmajor_sw128(a_base + 16384 + kk * 32), bd, idesc,
                        (it | kk) != 0);
            }
          }
          umma_commit(&empty[s]);
          if (++s == p.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        if (ok) umma_commit(&tfull);
      }
      // Every MMA issued above has finished once `drain` completes.
      umma_commit(&drain);
      mbar_wait(&drain, 0, nullptr, WAIT_LIMIT_NS / 4);
    }
  } else {
    const int r = warp * 32 + lane;
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    uint32_t local = 0;
    for (int t = blockIdx.x; t < p.items; t += gridDim.x, ++local) {
      const int tile = t / p.shares, z = t % p.shares;
      const int n = tile * p.R + r;  // weight row (DH: column) of this lane
      const bool valid = r < p.R && n < (DH ? p.K : p.I);
      __nv_bfloat16 d[32];
      auto load_du = [&](int c) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (valid && c + i < p.M) d[i] = du[static_cast<long>(c + i) * p.I + n];
      };
      if constexpr (!DH) load_du(0);  // on its way while the sums grow
      if (!mbar_wait_warp(&tfull, local & 1, abort_flag)) break;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < p.nt; c += 32) {  // tokens c .. c + 31
        float g[32];
        tmem_ld32(tacc + c, g);
        if constexpr (DH) {
          tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c + i >= p.M) break;
              if (p.shares > 1)
                part[(static_cast<long>(z) * p.M + c + i) * p.K + n] = g[i];
              else
                out[static_cast<long>(c + i) * p.K + n] = __float2bfloat16_rn(g[i]);
            }
          }
        } else {
          float up[32];
          tmem_ld32(tacc + 128 + c, up);
          tmem_ld_wait();
          if (valid) {
            if (c > 0) load_du(c);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c + i >= p.M) break;
              float dg, dup;
              swiglu_grad(g[i], up[i], __bfloat162float(d[i]), &dg, &dup);
              __nv_bfloat16 *dst = out + static_cast<long>(c + i) * 2 * p.I + n;
              dst[0] = __float2bfloat16_rn(dg);
              dst[p.I] = __float2bfloat16_rn(dup);
            }
          }
        }
        __syncwarp();  // tmem_ld32 takes the whole warp: lanes past the tile's rows wait here
      }
      tc_fence_before();
      mbar_arrive(&tempty);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem_base, TMEM_COLS);
}

// out[i] = bf16 of the sum of `shares` fp32 partials, in share order; n8 vectors of 8
__global__ void __launch_bounds__(256)
    grad_rows_reduce_kernel(const float4 *part, int shares, long n8, uint4 *out) {
  pdl_wait();
  pdl_trigger();
  for (long i = blockIdx.x * static_cast<long>(blockDim.x) + threadIdx.x; i < n8;
       i += static_cast<long>(gridDim.x) * blockDim.x) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    for (int z = 0; z < shares; ++z) {
      const float4 p = part[(z * n8 + i) * 2], q = part[(z * n8 + i) * 2 + 1];
      a.x += p.x; a.y += p.y; a.z += p.z; a.w += p.w;
      b.x += q.x; b.y += q.y; b.z += q.z; b.w += q.w;
    }
    out[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y),
                        pack_bf16x2(b.z, b.w));
  }
}

}  // namespace ig4
