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
#include "ptx_cluster.cuh"

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
// Many tokens: a pair of CTAs per 256 x W tile
// -------------------------------------------------------------------------------------
//
// Two CTAs of a cluster share one tile (tcgen05 cta_group::2): each holds 128 of its 256 token
// rows and half of its W <= 256 channels in shared memory, and the tensor cores of both read both
// halves, so a byte of B fetched once serves 256 rows.  The grid stays resident and each pair
// walks the tiles; sums alternate between two TMEM accumulators, so that one tile is scaled and
// stored while the next is multiplied.
//
// An MMA of 256 x N x 32 takes 128 cycles at N = 256, but 113 at 192 and 107 at 128 (timed without
// the loads), so narrow tiles are for small products only.  A tile of 512 channels in both
// accumulators, with a quarter fewer bytes from L2, lost more where the accumulators change hands
// than it gained (568 us against 546 at 32768 x 5120 x 5120).
//
// CTA = 8 or 12 warps: 0 TMA producer (A rows and B rows of this CTA; the bytes of both CTAs
// complete on the even CTA's barrier), 1 MMA issuer (even CTA only), 2 TMEM owner, 4 and up
// epilogue, one or two per TMEM lane quarter: scale, round, turn 32 rows x 128 bytes through shared
// memory, store whole lines.  kEpi = 8 takes a stage of the ring from kEpi = 4
// (4096 x 6144 x 4096: 70.4 us with six stages, 74.5 with five).

struct MatmulPairParams {
  CUtensorMap tm_a;    // {K, M} bytes, box {128, 128}, SW128
  CUtensorMap tm_b;    // {K, N} bytes, box {128, W / 2}, SW128
  const float* a_scale;
  const float* b_scale;
  const float* bias;  // or nullptr
  void* out;
  int64_t o_stride;
  int M, N, slabs;  // slabs of 128 bytes of K
  int W;
  int tiles_m, tiles_n;
  int stages, stage_bytes;
  int out_vec;  // rows of out on 16-byte boundaries
};

template <int kEpi>  // epilogue warps
struct MatmulPairCfg {
  static constexpr int kThreads = 128 + 32 * kEpi;
  static constexpr int kMaxStages = 8;
  static constexpr int kABytes = 128 * 128;
  static constexpr int kRingBytes = (kEpi == 4 ? 6 : 5) * 2 * kABytes;
  static constexpr int kOutOff = kRingBytes;
  static constexpr int kOutBytes = 32 * 128;  // per epilogue warp
  static constexpr int kColOff = kOutOff + kEpi * kOutBytes;
  static constexpr int kColBytes = 2 * 256 * 4;  // b_scale and bias of a tile, per epilogue warp
  static constexpr int kBarOff = kColOff + kEpi * kColBytes;
  static constexpr int kBarFull = 0;
  static constexpr int kBarEmpty = kBarFull + kMaxStages;
  static constexpr int kBarAccFull = kBarEmpty + kMaxStages;
  static constexpr int kBarAccEmpty = kBarAccFull + 2;
  static constexpr int kBarDrain = kBarAccEmpty + 2;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  static constexpr int kGroupM = 8;  // tile rows walked together, for L2
  static_assert(kSmemBytes <= 232448, "shared memory above the 227 KB opt-in limit");
};

// 128 bytes of scaled and rounded sums from `acc` (this lane's row).  col: b_scale and, 256 further
// on, bias of the columns.
template <typename O, int kCols>
__device__ __forceinline__ void round_out(uint32_t (&w)[32], const uint32_t (&acc)[kCols], float sa, const float* col) {
  const float2 sa2 = make_float2(sa, sa);
#pragma unroll
  for (int x = 0; x < kCols; x += 4) {
    const float4 sb = *reinterpret_cast<const float4*>(col + x);
    const float4 bi = *reinterpret_cast<const float4*>(col + 256 + x);
    float2 f[2];  // scale_acc, two at a time
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      f[y] = make_float2(__int2float_rn(static_cast<int32_t>(acc[x + 2 * y])),
                         __int2float_rn(static_cast<int32_t>(acc[x + 2 * y + 1])));
      f[y] = mul2(f[y], sa2);
    }
    f[0] = fma2(f[0], make_float2(sb.x, sb.y), make_float2(bi.x, bi.y));
    f[1] = fma2(f[1], make_float2(sb.z, sb.w), make_float2(bi.z, bi.w));
    if constexpr (sizeof(O) == 4) {
      w[x] = __float_as_uint(f[0].x), w[x + 1] = __float_as_uint(f[0].y);
      w[x + 2] = __float_as_uint(f[1].x), w[x + 3] = __float_as_uint(f[1].y);
    } else {
      w[x / 2] = pack2<O>(f[0]);
      w[x / 2 + 1] = pack2<O>(f[1]);
    }
  }
}

template <typename O, int kEpi>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(MatmulPairCfg<kEpi>::kThreads, 1)
    matmul_i8_pair_kernel(const __grid_constant__ MatmulPairParams p) {
  using C = MatmulPairCfg<kEpi>;
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
      for (int s = 0; s < p.stages; ++s) {
        mbar_init(bar(C::kBarFull + s), 1);
        mbar_init(bar(C::kBarEmpty + s), 1);
      }
      for (int t = 0; t < 2; ++t) {
        mbar_init(bar(C::kBarAccFull + t), 1);
        mbar_init(bar(C::kBarAccEmpty + t), 2 * kEpi);  // the epilogue warps of both CTAs
      }
      mbar_init(bar(C::kBarDrain), 1);
      fence_mbar_init();
      tma_prefetch_desc(&p.tm_a);
      tma_prefetch_desc(&p.tm_b);
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
    n0 = r / rows * p.W;
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t full0 = cluster_map(bar(C::kBarFull), 0);  // the even CTA's barriers
      // B is read again by every group of tile rows; with one group it is A that is read again
      const bool one_group = p.tiles_m <= C::kGroupM;
      const uint64_t pol_a = one_group ? l2_policy_evict_last() : l2_policy_evict_first();
      const uint64_t pol_b = one_group ? l2_policy_evict_first() : l2_policy_evict_last();
      const uint32_t bytes = 2u * static_cast<uint32_t>(p.stage_bytes);
      const int slabs = p.slabs, stages = p.stages;
      int it = 0, s = 0;
      uint32_t phase = 1;  // parity of the phase that a stage's reader completed last: none yet
      uint32_t dst = base, full = full0, own = bar(C::kBarFull);
      constexpr uint32_t kToEmpty = 8u * (C::kBarEmpty - C::kBarFull);
      bool ok = true;
      for (int t = pair; ok && t < tiles; t += pairs) {
        int m0, n0;
        tile_at(t, m0, n0);
        m0 += static_cast<int>(rank) * 128;
        n0 += static_cast<int>(rank) * (p.W / 2);
#pragma unroll 2
        for (int k = 0; k < slabs; ++k, ++it) {
          if (!(ok = mbar_wait_hot(own + kToEmpty, phase, abort_flag))) break;
          if (rank == 0) mbar_arrive_expect_tx(own, bytes);
          tma_load_2d_pair(dst, &p.tm_a, full, k * 128, m0, pol_a);
          tma_load_2d_pair(dst + C::kABytes, &p.tm_b, full, k * 128, n0, pol_b);
          const bool wrap = ++s == stages;
          s = wrap ? 0 : s;
          phase ^= wrap ? 1u : 0u;
          dst = wrap ? base : dst + p.stage_bytes;
          full = wrap ? full0 : full + 8u;
          own = wrap ? bar(C::kBarFull) : own + 8u;
        }
      }
      // let the copies still in flight land before the pair can exit (matters only after an
      // abort): the even CTA's barriers count the bytes of both
      if (rank == 0)
        for (int q = max(0, it - p.stages); q < it; ++q)
          mbar_wait_drain(bar(C::kBarFull + q % p.stages), static_cast<uint32_t>(q / p.stages) & 1);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && rank == 0) {
      // One thread issues everything, each instruction some cycles after the one before it, so what
      // it does per slab is kept short: stage addresses and descriptors are stepped, not computed
      // (with the address arithmetic in the loop a slab took 850 cycles at any width).
      const uint32_t idesc = idesc_s8(256, p.W);
      const uint64_t desc0 = sdesc_sw128(base, 16, 1024);
      const uint32_t desc_hi = static_cast<uint32_t>(desc0 >> 32), desc_lo0 = static_cast<uint32_t>(desc0);
      const uint32_t step = static_cast<uint32_t>(p.stage_bytes) >> 4;
      constexpr uint32_t b_off = C::kABytes >> 4;
      const uint32_t full_0 = bar(C::kBarFull), full_end = bar(C::kBarFull + p.stages);
      constexpr uint32_t kToEmpty = 8u * (C::kBarEmpty - C::kBarFull);
      const int slabs = p.slabs;
      struct Stage {
        uint32_t full, desc, phase;  // its full barrier, lower descriptor word and parity
      } st = {full_0, desc_lo0, 0u};
      auto advance = [&](Stage& x) {
        const bool wrap = x.full + 8u == full_end;
        x.full = wrap ? full_0 : x.full + 8u;
        x.desc = wrap ? desc_lo0 : x.desc + step;
        x.phase ^= wrap ? 1u : 0u;
      };
      bool ok = true;
      int unit = 0;  // tiles begun
      for (int t = pair; ok && t < tiles; t += pairs, ++unit) {
        const int acc = unit & 1;
        if (unit >= 2 &&
            !mbar_wait_hot<true>(bar(C::kBarAccEmpty + acc), (static_cast<uint32_t>(unit / 2) & 1) ^ 1, abort_flag))
          break;
        tc_fence_after();
        const uint32_t d = tmem + acc * 256;
#pragma unroll 4
        for (int k = 0; k < slabs; ++k) {
          if (!(ok = mbar_wait_hot(st.full, st.phase, abort_flag))) break;
          tc_fence_after();
          mma_i8_ss_pair_x4(d, st.desc, st.desc + b_off, desc_hi, idesc, static_cast<uint32_t>(k));
          mma_commit_pair(st.full + kToEmpty);
          advance(st);
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
    constexpr int kTurns = kEpi / 4;        // the warps of a quarter take a tile's pieces in turn
    const int quarter = warp & 3, own = warp - 4, first = own / 4 * kCols;
    const uint32_t stage = base + C::kOutOff + own * C::kOutBytes;
    float* col = reinterpret_cast<float*>(smem + C::kColOff + own * C::kColBytes);
    const uint32_t empty0 = cluster_map(bar(C::kBarAccEmpty), 0);
    // b_scale and bias of a tile's channels, a_scale of this lane's row: the next tile's are on
    // their way while a tile is stored
    float sb[8], bi[8], sa_next = 0.f;
    auto prefetch = [&](int t) {
      int m0, n0;
      tile_at(t, m0, n0);
      const int m = m0 + static_cast<int>(rank) * 128 + quarter * 32 + lane;
      sa_next = m < p.M ? p.a_scale[m] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 32 * i + lane, n = n0 + c;
        const bool in = c < p.W && n < p.N;
        sb[i] = in ? p.b_scale[n] : 0.f;
        bi[i] = in && p.bias ? p.bias[n] : 0.f;
      }
    };
    if (pair < tiles) prefetch(pair);
    int unit = 0;
    for (int t = pair; t < tiles; t += pairs, ++unit) {
      int m0, n0;
      tile_at(t, m0, n0);
      const int m_warp = m0 + static_cast<int>(rank) * 128 + quarter * 32;
      const float sa = sa_next;
      const int acc = unit & 1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        col[32 * i + lane] = sb[i];
        col[256 + 32 * i + lane] = bi[i];
      }
      __syncwarp();
      if (t + pairs < tiles) prefetch(t + pairs);
      const bool ok =
          lane != 0 || mbar_wait_hot(bar(C::kBarAccFull + acc), static_cast<uint32_t>(unit / 2) & 1, abort_flag);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      const uint32_t src = tmem + acc * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
      for (int c = first; c < p.W; c += kTurns * kCols) {
        uint32_t r[kCols], w[32];
        if constexpr (kCols == 64) tmem_ld64_wait(src + c, r);
        else tmem_ld32_wait(src + c, r);
        if (c + kTurns * kCols >= p.W) {  // this warp's sums are out of TMEM: the next tile but one may have it
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(empty0 + 8u * acc);
        }
        if (m_warp >= p.M || n0 + c >= p.N) continue;
        round_out<O, kCols>(w, r, sa, col + c);
        // 16-byte chunk x of row r lies at chunk x ^ (r % 8): conflict-free both ways
#pragma unroll
        for (int x = 0; x < 8; ++x)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((x ^ (lane & 7)) << 4)),
                       "r"(w[4 * x]), "r"(w[4 * x + 1]), "r"(w[4 * x + 2]), "r"(w[4 * x + 3])
                       : "memory");
        __syncwarp();
        const int rows = min(32, p.M - m_warp), cols = min(kCols, p.N - n0 - c);
        O* const dst = static_cast<O*>(p.out) + m_warp * p.o_stride + n0 + c;
        if (p.out_vec && cols == kCols) {
          const int x = lane & 7;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            const uint4 v = lds128(stage + row * 128 + ((x ^ (row & 7)) << 4));
            if (row < rows)
              *reinterpret_cast<uint4*>(dst + row * p.o_stride + x * (16 / static_cast<int>(sizeof(O)))) = v;
          }
        } else if (cols == kCols) {
          // rows at any alignment: eight lanes store a row's whole 16-byte units, each cut out of two
          // chunks, and the 16 bytes left over at its two ends value by value (77 us for all of it
          // value by value at 27520 x 1348 x 83 fp16, 53 so)
          const int x = lane & 7;
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const int row = 4 * i + (lane >> 3);
            uint8_t* const d = reinterpret_cast<uint8_t*>(dst + row * p.o_stride);
            const uint32_t lead = (0u - static_cast<uint32_t>(reinterpret_cast<uint64_t>(d))) & 15u;
            const uint32_t src = stage + row * 128;
            const uint4 u = lds128(src + ((x ^ (row & 7)) << 4)), v = lds128(src + ((min(x + 1, 7) ^ (row & 7)) << 4));
            const bool hi8 = (lead & 8u) != 0u, hi4 = (lead & 4u) != 0u;
            const uint32_t w0 = hi8 ? u.z : u.x, w1 = hi8 ? u.w : u.y, w2 = hi8 ? v.x : u.z, w3 = hi8 ? v.y : u.w,
                           w4 = hi8 ? v.z : v.x, w5 = hi8 ? v.w : v.y;
            const uint32_t y0 = hi4 ? w1 : w0, y1 = hi4 ? w2 : w1, y2 = hi4 ? w3 : w2, y3 = hi4 ? w4 : w3,
                           y4 = hi4 ? w5 : w4, shift = (lead & 3u) * 8u;
            const uint32_t edge = static_cast<uint32_t>(x * static_cast<int>(sizeof(O)));
            const uint32_t at = edge < lead ? edge : 112u + edge;  // byte of the row's piece
            const uint32_t value = lds_value<sizeof(O)>(src + (((at >> 4) ^ (row & 7)) << 4) + (at & 15u));
            if (row < rows) {
              if (lead == 0u || x < 7)
                *reinterpret_cast<uint4*>(d + lead + 16 * x) =
                    make_uint4(__funnelshift_r(y0, y1, shift), __funnelshift_r(y1, y2, shift),
                               __funnelshift_r(y2, y3, shift), __funnelshift_r(y3, y4, shift));
              if (lead != 0u && edge < 16u) *reinterpret_cast<O*>(d + at) = value_of<O>(value);
            }
          }
        } else {  // the last columns, the loads of eight rows ahead of their stores
#pragma unroll 1
          for (int i0 = 0; i0 < rows; i0 += 8) {
            uint32_t v[8][kCols / 32];
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < kCols / 32; ++j) {
                const int at = (32 * j + lane) * static_cast<int>(sizeof(O));
                v[i][j] = lds_value<sizeof(O)>(stage + (i0 + i) * 128 + (((at >> 4) ^ i) << 4) + (at & 15));
              }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int j = 0; j < kCols / 32; ++j)
                if (i0 + i < rows && 32 * j + lane < cols) dst[(i0 + i) * p.o_stride + 32 * j + lane] = value_of<O>(v[i][j]);
          }
        }
        __syncwarp();
      }
      if (first >= p.W) {  // a narrow tile: no piece for this warp
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(empty0 + 8u * acc);
      }
      __syncwarp();  // col is read
    }
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
  static constexpr int kScalesOff = kNumBars * 8 + 24;       // after barriers, TMEM address, abort flag
  static constexpr int kTailBytes = kScalesOff + 256 * 4;  // a_scale of the tile's tokens
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

  // scales of this lane's channels and of the tile's tokens: fetched while the sums are made
  const int n = n0 + 4 * lane, tokens = min(p.T, p.M - m0);
  float sb[4], bi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sb[i] = n + i < p.N ? p.b_scale[n + i] : 0.f;
    bi[i] = n + i < p.N && p.bias ? p.bias[n + i] : 0.f;
  }
  float* a_scales = reinterpret_cast<float*>(smem + tail + C::kScalesOff);
  for (int t = threadIdx.x; t < tokens; t += C::kThreads) a_scales[t] = p.a_scale[m0 + t];
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
        if (!mbar_wait_hot(bar(C::kBarEmpty + it % p.stages), (static_cast<uint32_t>(it / p.stages) & 1) ^ 1, abort_flag))
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
        if (!mbar_wait_hot(bar(C::kBarFull + s), static_cast<uint32_t>(it / p.stages) & 1, abort_flag)) break;
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
    acc_ok = lane != 0 || mbar_wait_hot(bar(C::kBarAccFull), 0, abort_flag);
    acc_ok = __all_sync(0xffffffffu, acc_ok);
    tc_fence_after();
  }
  __syncwarp();
  cluster_sync();  // every MMA of the cluster has read its stages: their memory takes the sums

  // ------------------------------------------------------------------ sums to their owners
  // Token t belongs to CTA t % splits, which gets [splits][per][128] sums.  Stores to the other
  // CTAs, so that no warp waits for a remote load (each CTA reading its share from the others took
  // 21.6 us at 256 x 5120 x 5120, this 18.0), of 128 neighbouring bytes per warp (16 bytes a lane,
  // four tokens of a channel: 18.1 there, and 10.4 against 9.6 at 16 x 6144 x 4096).
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
    const int t = rank + splits * idx;
    const float sa = a_scales[t];
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
    O* dst = static_cast<O*>(p.out) + (m0 + t) * p.o_stride + n;
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
