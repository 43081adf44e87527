// Product of INT8 codes with a scale for each row of either side:
//   out[m, n] = (sum_k a[m, k] b[n, k]) * a_scale[m] * b_scale[n] + bias[n].
// The sum is exact in s32 (K < 2^17 keeps |sum| <= 2^14 K below 2^31); it is then rounded to
// f32 and scaled in f32, by a_scale first, with the second product and the bias in one fused
// multiply-add, and rounded once to the output's type.
#pragma once

#include <cstdint>
#include <cstring>
#include <cuda.h>

#include "norm_quant.cuh"
#include "ptx_sm100.cuh"

namespace qbsa {

constexpr int kMatmulMaxK = 131071;  // 2^14 K < 2^31


// f32 from the exact sum, by the rule above.
__device__ __forceinline__ float scale_acc(uint32_t acc, float sa, float sb, float bias) {
  return __fmaf_rn(__fmul_rn(__int2float_rn(static_cast<int32_t>(acc)), sa), sb, bias);
}

template <typename O>
__device__ __forceinline__ uint32_t pack_out2(float lo, float hi) {
  O v[2] = {from_f32<O>(lo), from_f32<O>(hi)};
  uint32_t r;
  memcpy(&r, v, 4);
  return r;
}

// -------------------------------------------------------------------------------------
// Many tokens: a pair of CTAs per 256 x BN tile
// -------------------------------------------------------------------------------------
//
// Two CTAs of a cluster share one tile (tcgen05 cta_group::2): each holds 128 of its 256 token
// rows and half of its BN channels in shared memory, and the tensor cores of both read both
// halves, so a byte of B fetched once serves 256 rows.  The grid stays resident and each pair
// walks the tiles; sums alternate between two TMEM buffers, so that one tile is scaled and
// stored while the next is multiplied.
//
// CTA = 8 warps: 0 TMA producer (A rows and B rows of this CTA; the bytes of both CTAs complete
// on the even CTA's barrier), 1 MMA issuer (even CTA only), 2 TMEM owner, 4-7 epilogue, one
// TMEM lane quarter each: scale, round, stage 32 rows x 128 bytes, TMA store.

struct MatmulPairParams {
  CUtensorMap tm_a;    // {K, M} bytes, box {128, 128}, SW128
  CUtensorMap tm_b;    // {K, N} bytes, box {128, BN / 2}, SW128
  CUtensorMap tm_out;  // {N, M}, box {128 bytes, 32}, SW128 (out_tma)
  const float* a_scale;
  const float* b_scale;
  const float* bias;  // or nullptr
  void* out;
  int64_t o_stride;
  int M, N, slabs;  // slabs of 128 bytes of K
  int BN;
  int tiles_m, tiles_n;
  int out_tma;  // rows of out on 16-byte boundaries
};

struct MatmulPairCfg {
  static constexpr int kThreads = 256;
  static constexpr int kStages = 6;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kStageBytes = 2 * kABytes;  // B: at most 128 rows
  static constexpr int kOutOff = kStages * kStageBytes;
  static constexpr int kOutBytes = 32 * 128;  // per epilogue warp
  static constexpr int kColOff = kOutOff + 4 * kOutBytes;
  static constexpr int kColBytes = 2 * 256 * 4;  // b_scale and bias of a tile, per epilogue warp
  static constexpr int kBarOff = kColOff + 4 * kColBytes;
  static constexpr int kBarFull = 0;
  static constexpr int kBarEmpty = kBarFull + kStages;
  static constexpr int kBarAccFull = kBarEmpty + kStages;
  static constexpr int kBarAccEmpty = kBarAccFull + 2;
  static constexpr int kBarDrain = kBarAccEmpty + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  static constexpr int kGroupM = 8;  // tile rows walked together, for L2
};
static_assert(MatmulPairCfg::kSmemBytes <= 232448, "shared memory above the 227 KB opt-in limit");

// 32 rows x 128 bytes of scaled sums: from `acc` (this lane's row) to the staging tile, swizzled
// as the output's tensor map reads it.  col: b_scale and, 256 further on, bias of the columns.
template <typename O, int kCols>
__device__ __forceinline__ void stage_out(uint32_t stage, int lane, const uint32_t (&acc)[kCols], float sa,
                                          const float* col) {
  constexpr int kPer = 16 / sizeof(O);  // values of 16 bytes
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    float f[kPer];
#pragma unroll
    for (int y = 0; y < kPer; y += 4) {
      const float4 sb = *reinterpret_cast<const float4*>(col + x * kPer + y);
      const float4 bi = *reinterpret_cast<const float4*>(col + 256 + x * kPer + y);
      const uint32_t* v = acc + x * kPer + y;
      f[y] = scale_acc(v[0], sa, sb.x, bi.x);
      f[y + 1] = scale_acc(v[1], sa, sb.y, bi.y);
      f[y + 2] = scale_acc(v[2], sa, sb.z, bi.z);
      f[y + 3] = scale_acc(v[3], sa, sb.w, bi.w);
    }
    uint32_t w[4];
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if constexpr (sizeof(O) == 4) w[y] = __float_as_uint(f[y]);
      else w[y] = pack_out2<O>(f[2 * y], f[2 * y + 1]);
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((x ^ (lane & 7)) << 4)),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
  }
}

template <typename O>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MatmulPairCfg::kThreads, 1)
    matmul_i8_pair_kernel(const __grid_constant__ MatmulPairParams p) {
  using C = MatmulPairCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  auto bar = [&](int i) -> uint32_t { return base + C::kBarOff + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOff + 4);

  if (warp == 0) {
    if (lane == 0) {
      *abort_flag = 0;
      for (int s = 0; s < C::kStages; ++s) {
        mbar_init(bar(C::kBarFull + s), 1);
        mbar_init(bar(C::kBarEmpty + s), 1);
      }
      for (int t = 0; t < 2; ++t) {
        mbar_init(bar(C::kBarAccFull + t), 1);
        mbar_init(bar(C::kBarAccEmpty + t), 8);  // the epilogue warps of both CTAs
      }
      mbar_init(bar(C::kBarDrain), 1);
      fence_mbar_init();
      tma_prefetch_desc(&p.tm_a);
      tma_prefetch_desc(&p.tm_b);
      if (p.out_tma) tma_prefetch_desc(&p.tm_out);
    }
  } else if (warp == 2) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int tiles = p.tiles_m * p.tiles_n;
  const int per_group = C::kGroupM * p.tiles_n;
  // token and channel of tile t's first element: groups of kGroupM tile rows, channels outermost
  auto tile_at = [&](int t, int& m0, int& n0) {
    const int g = t / per_group, r = t - g * per_group;
    const int rows = min(C::kGroupM, p.tiles_m - g * C::kGroupM);
    m0 = (g * C::kGroupM + r % rows) * 256;
    n0 = r / rows * p.BN;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t full0 = cluster_map(bar(C::kBarFull), 0);  // the even CTA's barriers
      const uint32_t bytes = 2u * (C::kABytes + static_cast<uint32_t>(p.BN / 2) * 128u);
      const uint64_t pol_a = l2_policy_evict_first(), pol_b = l2_policy_evict_last();
      int it = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int m0, n0;
        tile_at(t, m0, n0);
        for (int k = 0; k < p.slabs; ++k, ++it) {
          const int s = it % C::kStages;
          if (it >= C::kStages &&
              !mbar_wait<true>(bar(C::kBarEmpty + s), (static_cast<uint32_t>(it / C::kStages) & 1) ^ 1, abort_flag)) {
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(bar(C::kBarFull + s), bytes);
          const uint32_t dst = base + s * C::kStageBytes, full = full0 + 8u * s;
          tma_load_2d_pair(dst, &p.tm_a, full, k * 128, m0 + static_cast<int>(rank) * 128, pol_a);
          tma_load_2d_pair(dst + C::kABytes, &p.tm_b, full, k * 128, n0 + static_cast<int>(rank) * (p.BN / 2), pol_b);
        }
      }
      // let the copies still in flight land before the pair can exit (matters only after an
      // abort): the even CTA's barriers count the bytes of both
      if (rank == 0)
        for (int q = max(0, it - C::kStages); q < it; ++q)
          mbar_wait_drain(bar(C::kBarFull + q % C::kStages), static_cast<uint32_t>(q / C::kStages) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_s8(256, p.BN);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs, ++n) {
        const int acc = n & 1;
        if (n >= 2 && !mbar_wait<true>(bar(C::kBarAccEmpty + acc), (static_cast<uint32_t>(n / 2) & 1) ^ 1, abort_flag))
          break;
        tc_fence_after();
        for (int k = 0; k < p.slabs; ++k, ++it) {
          const int s = it % C::kStages;
          if (!mbar_wait<true>(bar(C::kBarFull + s), static_cast<uint32_t>(it / C::kStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a = base + s * C::kStageBytes, b = a + C::kABytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_i8_ss_pair(tmem + acc * 256, sdesc_sw128(a + kk * 32, 16, 1024), sdesc_sw128(b + kk * 32, 16, 1024),
                           idesc, (k | kk) != 0 ? 1u : 0u);
          mma_commit_pair(bar(C::kBarEmpty + s));
        }
        if (ok) mma_commit_pair(bar(C::kBarAccFull + acc));
      }
      mma_commit_pair(bar(C::kBarDrain));
    }
    // every MMA has retired, and every arrival that a commit sends to this CTA has come, before
    // TMEM is released and either CTA exits
    if (lane == 0) mbar_wait_drain(bar(C::kBarDrain), 0);
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    constexpr int kCols = 128 / sizeof(O);  // columns of a staged piece
    const int quarter = warp & 3;
    const uint32_t stage = base + C::kOutOff + quarter * C::kOutBytes;
    float* col = reinterpret_cast<float*>(smem + C::kColOff + quarter * C::kColBytes);
    const uint32_t empty0 = cluster_map(bar(C::kBarAccEmpty), 0);
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      int m0, n0;
      tile_at(t, m0, n0);
      const int acc = n & 1;
      const int m_warp = m0 + static_cast<int>(rank) * 128 + quarter * 32, m = m_warp + lane;
      for (int c = lane; c < p.BN; c += 32) {
        const bool in = n0 + c < p.N;
        col[c] = in ? p.b_scale[n0 + c] : 0.f;
        col[256 + c] = in && p.bias ? p.bias[n0 + c] : 0.f;
      }
      const float sa = m < p.M ? p.a_scale[m] : 0.f;
      __syncwarp();
      if (!warp_wait(bar(C::kBarAccFull + acc), static_cast<uint32_t>(n / 2) & 1, abort_flag)) break;
      tc_fence_after();
      const uint32_t src = tmem + acc * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int c = 0; c < p.BN; c += kCols) {
        uint32_t r[kCols];
        if constexpr (kCols == 64) tmem_ld64_wait(src + c, r);
        else tmem_ld32_wait(src + c, r);
        if (c + kCols >= p.BN) {  // the sums are out of TMEM: the next tile but one may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(empty0 + 8u * acc);
        }
        if (m_warp >= p.M || n0 + c >= p.N) continue;
        if (lane == 0) bulk_wait_read_all();  // the staging tile's previous store
        __syncwarp();
        stage_out<O, kCols>(stage, lane, r, sa, col + c);
        if (p.out_tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&p.tm_out, stage, n0 + c, m_warp);
            bulk_commit_group();
          }
        } else {
          // rows of out at any alignment: a warp writes a row's piece at a time
          __syncwarp();
          const int rows = min(32, p.M - m_warp), cols = min(kCols, p.N - n0 - c);
          for (int i = 0; i < rows; ++i) {
            O* dst = static_cast<O*>(p.out) + (m_warp + i) * p.o_stride + n0 + c;
#pragma unroll
            for (int j = lane; j < kCols; j += 32) {
              const int at = j * static_cast<int>(sizeof(O));
              if (j < cols)
                dst[j] = *reinterpret_cast<const O*>(smem + C::kOutOff + quarter * C::kOutBytes + i * 128 +
                                                     (((at >> 4) ^ (i & 7)) << 4) + (at & 15));
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) bulk_wait_read_all();  // shared memory must outlive the stores' reads
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// -------------------------------------------------------------------------------------
// Few tokens: 128 channels x up to 256 tokens per CTA, K split over a cluster
// -------------------------------------------------------------------------------------
//
// With few tokens the time is the weight's way from HBM, so every SM has to stream.  The
// weight's rows take the MMA's 128 lanes and the tokens its columns (16 at least), and K is
// split over the CTAs of a cluster, whose s32 sums are joined through distributed shared
// memory: exact in any order, with no scratch memory and no second launch.
//
// CTA = 6 warps: 0-3 epilogue (TMEM lane quarters), 4 TMA producer, 5 TMEM owner and MMA issuer.

struct MatmulSplitParams {
  CUtensorMap tm_a;  // tokens {K, M} bytes, box {128, T}, SW128
  CUtensorMap tm_b;  // weight {K, N} bytes, box {128, 128}, SW128
  const float* a_scale;
  const float* b_scale;
  const float* bias;  // or nullptr
  void* out;
  int64_t o_stride;
  int M, N, slabs, slabs_per;  // slabs of 128 bytes of K, in all and per CTA of the cluster
  int T;       // tokens of a tile: a multiple of 16 up to 256
  int stages, stage_bytes;
  int tmem_cols;
  int vec;  // four neighbouring outputs lie on a boundary of their own size
};

struct MatmulSplitCfg {
  static constexpr int kThreads = 192;
  static constexpr int kMaxStages = 8;
  static constexpr int kWBytes = 128 * 128;
  static constexpr int kBarFull = 0;
  static constexpr int kBarEmpty = kBarFull + kMaxStages;
  static constexpr int kBarAccFull = kBarEmpty + kMaxStages;
  static constexpr int kNumBars = kBarAccFull + 1;
  static constexpr int kTailBytes = kNumBars * 8 + 16;  // barriers, TMEM address, abort flag
};

template <typename O>
__global__ void __launch_bounds__(MatmulSplitCfg::kThreads)
    matmul_i8_split_kernel(const __grid_constant__ MatmulSplitParams p) {
  using C = MatmulSplitCfg;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  const uint32_t base = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw_base);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tail = static_cast<uint32_t>(p.stages * p.stage_bytes);
  auto bar = [&](int i) -> uint32_t { return base + tail + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + tail + C::kNumBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int rank = static_cast<int>(blockIdx.x), splits = static_cast<int>(gridDim.x);  // cluster = gridDim.x CTAs
  const int n0 = blockIdx.y * 128, m0 = blockIdx.z * p.T;
  const int k0 = rank * p.slabs_per, slabs = min(p.slabs_per, p.slabs - k0);

  // this lane's channels and this warp's first token: fetched while the sums are made
  const int n = n0 + 4 * lane, tokens = min(p.T, p.M - m0);
  float sb[4], bi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sb[i] = n + i < p.N ? p.b_scale[n + i] : 0.f;
    bi[i] = n + i < p.N && p.bias ? p.bias[n + i] : 0.f;
  }
  float sa = rank + splits * warp < tokens ? p.a_scale[m0 + rank + splits * warp] : 0.f;
  bool acc_ok = false;

  const uint64_t pol_w = l2_policy_evict_first(), pol_t = l2_policy_evict_last();
  auto load = [&](int it) {  // slab `it` of this CTA into its stage
    const int s = it % p.stages;
    mbar_arrive_expect_tx(bar(C::kBarFull + s), p.stage_bytes);
    const uint32_t dst = base + s * p.stage_bytes;
    tma_load_2d(dst, &p.tm_b, bar(C::kBarFull + s), (k0 + it) * 128, n0, pol_w);
    tma_load_2d(dst + C::kWBytes, &p.tm_a, bar(C::kBarFull + s), (k0 + it) * 128, m0, pol_t);
  };
  if (warp == 4 && lane == 0) {
    *abort_flag = 0;
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(bar(C::kBarFull + s), 1);
      mbar_init(bar(C::kBarEmpty + s), 1);
    }
    mbar_init(bar(C::kBarAccFull), 1);
    fence_mbar_init();
    for (int it = 0; it < min(p.stages, slabs); ++it) load(it);  // under way while TMEM is allocated
  } else if (warp == 5) {
    tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int it = min(p.stages, slabs);
      for (; it < slabs; ++it) {
        if (!mbar_wait(bar(C::kBarEmpty + it % p.stages), (static_cast<uint32_t>(it / p.stages) & 1) ^ 1, abort_flag))
          break;
        load(it);
      }
      // let the copies still in flight land before the CTA can exit (matters only after an abort)
      for (int q = max(0, it - p.stages); q < it; ++q)
        mbar_wait_drain(bar(C::kBarFull + q % p.stages), static_cast<uint32_t>(q / p.stages) & 1);
    }
  } else if (warp == 5) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      const uint32_t idesc = idesc_s8(128, p.T);
      for (int it = 0; it < slabs; ++it) {
        const int s = it % p.stages;
        if (!mbar_wait(bar(C::kBarFull + s), static_cast<uint32_t>(it / p.stages) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t w = base + s * p.stage_bytes, x = w + C::kWBytes;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_i8_ss(tmem, sdesc_sw128(w + kk * 32, 16, 1024), sdesc_sw128(x + kk * 32, 16, 1024), idesc,
                    (it | kk) != 0 ? 1u : 0u);
        mma_commit(bar(C::kBarEmpty + s));
      }
      // every MMA issued above has retired before TMEM can be released
      mma_commit(bar(C::kBarAccFull));
      mbar_wait_drain(bar(C::kBarAccFull), 0);
    }
  } else {
    acc_ok = warp_wait(bar(C::kBarAccFull), 0, abort_flag);
    tc_fence_after();
  }
  __syncwarp();
  cluster_sync();  // every MMA of the cluster has read its stages: their memory takes the sums

  // ------------------------------------------------------------------ sums to their owners
  // Token t belongs to CTA t % splits, which gets [splits][per][128] sums.  Stores to the other
  // CTAs, so that no warp waits for a remote load (each CTA reading its share from the others took
  // 21.6 us at 256 x 5120 x 5120, this 18.3).
  const int per = (p.T + splits - 1) / splits;
  if (warp < 4 && acc_ok) {
    int owner = 0, idx = 0;
    const uint32_t mine = base + static_cast<uint32_t>(rank * per * 128 + warp * 32 + lane) * 4u;
    for (int t = 0; t < p.T; t += 16) {
      uint32_t r[16];
      tmem_ld16_wait(tmem + t + (static_cast<uint32_t>(warp * 32) << 16), r);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        st_cluster_b32(cluster_map(mine + static_cast<uint32_t>(idx) * 512u, owner), r[i]);
        if (++owner == splits) {
          owner = 0;
          ++idx;
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();

  // ------------------------------------------------------------------ joined, scaled and stored
  // a warp takes a token, a lane four channels
  for (int idx = warp; rank + splits * idx < tokens; idx += C::kThreads / 32) {
    const int m = m0 + rank + splits * idx;
    if (idx != warp) sa = p.a_scale[m];
    int4 v = make_int4(0, 0, 0, 0);
    for (int c = 0; c < splits; ++c) {
      const uint4 u = lds128(base + static_cast<uint32_t>((c * per + idx) * 512 + 16 * lane));
      v.x += static_cast<int>(u.x);
      v.y += static_cast<int>(u.y);
      v.z += static_cast<int>(u.z);
      v.w += static_cast<int>(u.w);
    }
    const float f[4] = {scale_acc(v.x, sa, sb[0], bi[0]), scale_acc(v.y, sa, sb[1], bi[1]),
                        scale_acc(v.z, sa, sb[2], bi[2]), scale_acc(v.w, sa, sb[3], bi[3])};
    O* dst = static_cast<O*>(p.out) + m * p.o_stride + n;
    if (p.vec && n + 4 <= p.N) {
      if constexpr (sizeof(O) == 4) *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
      else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_out2<O>(f[0], f[1]), pack_out2<O>(f[2], f[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < p.N) dst[i] = from_f32<O>(f[i]);
    }
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// -------------------------------------------------------------------------------------
// Up to 8 tokens: the weight straight from HBM into the registers of warp-level MMAs
// -------------------------------------------------------------------------------------
//
// One token's product reads the weight once and does next to nothing else, and at its few
// microseconds every hand-over counts (TMA descriptors, TMEM, clusters).  Here a CTA takes 16
// channels and its warps every kWarps-th 64-byte piece of K.  The sum does not care for the order
// of k, so a lane loads 16 neighbouring bytes of a row and takes them for the four words that
// m16n8k32 wants at other places of k, with the tokens' bytes in the same order: no shared memory
// and no shuffles before the warps' sums are joined.  (With a second tile of 8 tokens the registers
// allow too few loads in flight: 11 us at 16 x 6144 x 4096, the split kernel 9.7.)

struct MatmulRowsParams {
  const int8_t* a;
  const int8_t* b;
  const float* a_scale;
  const float* b_scale;
  const float* bias;  // or nullptr
  void* out;
  int64_t a_stride, b_stride, o_stride;
  int M, N, K;
};

__device__ __forceinline__ void mma_m16n8k32_s8(int32_t (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes of a row from byte k on, zeros from K on.
__device__ __forceinline__ uint4 load_codes16(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return ld_stream_v4(reinterpret_cast<const uint4*>(row + k));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (k + i < K) w[i >> 2] |= static_cast<uint32_t>(static_cast<uint8_t>(row[k + i])) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename O, int kWarps>
__global__ void __launch_bounds__(kWarps * 32) matmul_i8_rows_kernel(const __grid_constant__ MatmulRowsParams p) {
  constexpr int kUnroll = 4;
  __shared__ int32_t part[kWarps][8][17];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int n0 = blockIdx.x * 16;
  // thread i of the first 16 M scales and stores token i / 16, channel i % 16 (8 x 16 <= 4 warps)
  const int m = threadIdx.x >> 4, n = n0 + (threadIdx.x & 15);
  const bool mine = m < p.M && n < p.N;
  const float sa = mine ? p.a_scale[m] : 0.f, sb = mine ? p.b_scale[n] : 0.f, bias = mine && p.bias ? p.bias[n] : 0.f;
  // rows past the end repeat the last one; their sums are not stored
  const int8_t* w0 = p.b + min(n0 + g, p.N - 1) * p.b_stride;
  const int8_t* w1 = p.b + min(n0 + g + 8, p.N - 1) * p.b_stride;
  const int8_t* token = p.a + min(g, p.M - 1) * p.a_stride;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  int32_t acc[4] = {};
  for (int k0 = warp * 64; k0 < p.K; k0 += kUnroll * kWarps * 64) {
    uint4 a0[kUnroll], a1[kUnroll], x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * kWarps * 64 + tig * 16;
      const bool in = k < p.K;
      a0[u] = in ? load_codes16(w0, k, p.K) : zero;
      a1[u] = in ? load_codes16(w1, k, p.K) : zero;
      x[u] = in && g < p.M ? load_codes16(token, k, p.K) : zero;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      mma_m16n8k32_s8(acc, a0[u].x, a1[u].x, a0[u].y, a1[u].y, x[u].x, x[u].y);
      mma_m16n8k32_s8(acc, a0[u].z, a1[u].z, a0[u].w, a1[u].w, x[u].z, x[u].w);
    }
  }
  // lane (g, tig) holds channels g, g + 8 of tokens 2 tig, 2 tig + 1
  part[warp][2 * tig][g] = acc[0];
  part[warp][2 * tig + 1][g] = acc[1];
  part[warp][2 * tig][g + 8] = acc[2];
  part[warp][2 * tig + 1][g + 8] = acc[3];
  __syncthreads();
  if (!mine) return;
  int32_t sum = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += part[w][m][threadIdx.x & 15];
  static_cast<O*>(p.out)[m * p.o_stride + n] = from_f32<O>(scale_acc(sum, sa, sb, bias));
}

}  // namespace qbsa
