// dx_pair.cuh -- input gradient of the fused layers on two SMs at a time:
//   dX[m][k] = sum_n dZ[m][n] Weff[k][n]     (Weff: backward.cuh)
//
// The channel factor is split c'_n = m_n p_n, p_n a power of two.  dZ arrives
// as dZ m_n 2^(e_m) in fp16 (dact.cuh), and the weights are widened once per
// call to fp16 operand blocks of Weff / m_n: p_n B, which is exact, and the
// blended outlier rows (p_n B + (s - 1) W_O / m_n) / s, rounded once.  So
// the roundings are those of dZ, of the outlier rows and of dX.
//
// Up to 128 tokens, which would leave half of a tile's rows empty, dZ arrives in
// two fp16 terms instead: rows 2m and 2m + 1 of the product are token m's value
// and what its rounding left, and the epilogue adds the two lanes.  With few
// tokens the gradient has few numbers, and the rounding of dZ alone took its
// error to as much as twice that of one rounding of dX (1.42 times at the
// median); with two terms the last rounding is all that counts.
//
// Widening once (dx_widen_kernel, bound by HBM: 2 K N bytes written) and
// reading fp16 blocks by TMA leaves the tensor cores of both kernels' tiles
// to the product.  Converting inside the product, one code block per 256
// tokens, keeps them waiting: measured 2540 to 3100 cycles a 256 x 256 x 64
// step against the 1024 that the products take.
//
// dx_pair_kernel: a pair of CTAs (cta_group::2) computes 256 tokens x 256
// inputs, reducing over the channels 64 at a time.  Each CTA loads its own
// 128 token rows of dZ and its own 128 inputs of the operand per step (32 KB
// against 64 KB for one CTA alone); the even CTA issues the pair products.
// The accumulators are double-buffered in tensor memory, so a tile's output
// leaves under the next tile's products.  Calls with fewer tiles than pairs
// split the reduction into S ranges whose fp32 partial sums dx_reduce_kernel
// adds in order: no CTA waits for another.  2048 tokens x 4096 inputs: 127 us
// over 11008 channels, 242 over 22016 (1450 and 1530 TFLOP/s).
#pragma once

#include "backward.cuh"
#include "norm.cuh"

namespace qlin {

// p_n and m_n of a channel factor c'_n = m_n p_n: p_n = 2^k with k in
// [-14, 8], which keeps p_n and 127 p_n inside fp16's normal range; m_n is in
// [1, 2) unless c'_n lies outside [2^-14, 2^9).
__device__ __forceinline__ float chan_pow2(float c) {
  const int e = static_cast<int>((__float_as_uint(c) >> 23) & 0xFFu);
  const int k = e < 113 ? 113 : (e > 135 ? 135 : e);
  return __uint_as_float(static_cast<uint32_t>(k) << 23);
}
__device__ __forceinline__ float chan_mant(float c) {  // exact
  const uint32_t k = __float_as_uint(chan_pow2(c)) >> 23;
  return __fmul_rn(c, __uint_as_float((254u - k) << 23));
}

// m_n in [1, 2): the fraction field of c'_n.
__device__ __forceinline__ bool chan_mant_is_fraction(float c) {
  const uint32_t e = (__float_as_uint(c) >> 23) & 0xFFu;
  return e >= 113u && e <= 135u;
}

// c'_n of the forward's INT8 operand: c_n / 16 for per-channel INT4 (16 q), else c_n.
template <int FMT>
__device__ __forceinline__ float bwd_chan(float c) {
  return FMT == kFmtW4PC ? __fmul_rn(c, 0.0625f) : c;
}

struct DxWidenArgs {
  const uint8_t* codes;
  const uint16_t* rfold;
  const uint16_t* wot;
  const float* cscale;
  const int32_t* oidx;
  const float* s;
  uint8_t* out;  // operand blocks [ceil(K / 128)][nst] of 16 KiB
  int N, nO, kb, nst, nib;
  // the CTAs behind the blocks sum the bias gradient's partial rows (null: none)
  const float* part;
  float* dbias;
  int blocks, G;
};

// One CTA per packed block of 128 channels x 128 inputs, two operand blocks
// of 64 channels x 128 inputs out: channel groups of 8 (2 KiB), in them two
// atoms of 64 inputs (1 KiB), in them a 128-byte row per channel with the
// tensor core's 128-byte swizzle (inputs contiguous: the packed rows'
// direction, so nothing is transposed).  The blocks are put together in
// shared memory, eight threads a row, the outlier inputs are blended there
// by two threads a row, and one bulk copy each takes them out.  The column
// sums of the bias's gradient ride along in CTAs of their own: alone they are
// a launch that waits for a few loads.  4096 x 11008 INT8: 33 us, 4.1 TB/s of
// codes and operand; 4096 x 22016 g128: 49 us, 4.6 TB/s.  A warp waits for
// its codes two fifths of the time: a CTA loads, converts and stores in turn, and
// five of them on an SM do not cover it.
template <int FMT>
__global__ void __launch_bounds__(256) dx_widen_kernel(const __grid_constant__ DxWidenArgs g) {
  __shared__ __align__(128) unsigned char blk[32768];
  __shared__ int first, count;  // the block's outliers: consecutive entries of the sorted list
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= g.blocks) {
    griddep_wait();
    column_sum<8>(g.part, g.G, g.N, static_cast<int>(blockIdx.x) - g.blocks, g.dbias);
    return;
  }
  const int tn = static_cast<int>(blockIdx.x) / g.kb;
  const int kb = static_cast<int>(blockIdx.x) - tn * g.kb;
  const uint8_t* src = g.codes + static_cast<size_t>(blockIdx.x) * (FMT == kFmtW8 ? 16384 : 8192);
  constexpr int U = 8;  // chunks of 8 inputs per thread
  uint32_t w0[U], w1[U];
  float c[U];
  uint16_t rb[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = threadIdx.x + i * 256;
    const int row = u >> 4, kl = (u & 15) * 8;
    if (FMT == kFmtW8) {
      const uint2 t = __ldg(reinterpret_cast<const uint2*>(src + row * 128 + (((kl >> 4) ^ (row & 7)) << 4) + (kl & 15)));
      w0[i] = t.x;
      w1[i] = t.y;
    } else {
      w0[i] = __ldg(reinterpret_cast<const uint32_t*>(src + row * 64 + (((kl >> 5) ^ ((row >> 1) & 3)) << 4) + ((kl & 31) >> 1)));
      w1[i] = 0u;
    }
    const int n = tn * 128 + row;
    c[i] = n < g.N ? bwd_chan<FMT>(__ldg(g.cscale + n)) : 0.f;
    rb[i] = (FMT == kFmtW4G128 && n < g.N) ? __ldg(g.rfold + static_cast<size_t>(kb) * g.N + n) : uint16_t(0);
  }
  if (g.nO > 0) {
    // which entries: the whole list read at once (a binary search is a chain
    // of dependent loads)
    if (threadIdx.x == 0) {
      first = g.nO;
      count = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < g.nO; i += 256) {
      const int k = __ldg(g.oidx + i) - kb * 128;
      if (k >= 0 && k < 128) {
        atomicMin(&first, i);
        atomicAdd(&count, 1);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int u = threadIdx.x + i * 256;
    const int row = u >> 4, cc = u & 15;
    uint32_t q0, q1;
    if (FMT == kFmtW8) {
      q0 = w0[i];
      q1 = w1[i];
    } else if (FMT == kFmtW4PC) {
      q0 = (w0[i] << 4) & 0xF0F0F0F0u;
      q1 = w0[i] & 0xF0F0F0F0u;
    } else {
      const __half2 r1 = __half2half2(__ushort_as_half(rb[i]));
      const __half2 r16 = __hmul2(r1, __half2half2(__ushort_as_half(static_cast<unsigned short>(0x2C00))));  // * 1/16
      const uint2 a = requant_g128(w0[i], r1, r16);
      q0 = a.x;
      q1 = a.y;
    }
    const __half2 p2 = __float2half2_rn(chan_pow2(c[i]));
    uint4 h;
    i8x4_scale_h2(q0, p2, h.x, h.y);
    i8x4_scale_h2(q1, p2, h.z, h.w);
    *reinterpret_cast<uint4*>(blk + (row >> 3) * 2048 + (cc >> 3) * 1024 + (row & 7) * 128 + (((cc & 7) ^ (row & 7)) << 4)) = h;
  }
  griddep_wait();  // s comes from the forward; the workspace may still be read
  __syncthreads();
  if (g.nO > 0 && count > 0) {
    const int row = threadIdx.x >> 1;
    const int n = tn * 128 + row;
    const float m = n < g.N ? chan_mant(bwd_chan<FMT>(__ldg(g.cscale + n))) : 0.f;
    const float rm = m > 0.f ? __fdiv_rn(1.f, m) : 0.f;  // a channel without a scale has only zero weights
    for (int e = threadIdx.x & 1; e < count; e += 2) {
      const int o = first + e;
      const int k = __ldg(g.oidx + o) - kb * 128;
      const float sv = g.s[o];
      const float w = __half2float(__ushort_as_half(__ldg(g.wot + wot_tile_index(n, o, g.nib))));
      __half* p = reinterpret_cast<__half*>(blk + (row >> 3) * 2048 + (k >> 6) * 1024 + (row & 7) * 128 +
                                            ((((k & 63) >> 3) ^ (row & 7)) << 4)) + (k & 7);
      *p = __float2half_rn(__fdiv_rn(__fmaf_rn(__fsub_rn(sv, 1.f), __fmul_rn(w, rm), __half2float(*p)), sv));
    }
  }
  fence_proxy_async_smem();  // the bulk copies read the blocks next
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int b = 0; b < 2; ++b)
      if (tn * 2 + b < g.nst)
        bulk_store(g.out + (static_cast<size_t>(kb) * g.nst + tn * 2 + b) * 16384, blk + b * 16384, 16384u);
    bulk_commit_group();
    bulk_wait_group_all();
  }
}

struct DxArgs {
  const float* rowscale;  // [M]
  uint16_t* dX;           // [M][K] (reduce kernel)
  float* part;            // [S][M][K] partial sums (S > 1)
  int M, K;
  int two;                // dZ in two terms (M <= 128)
  int nst;                // 64-channel steps of the whole reduction
  int tiles_k, tiles_m, S, units, ncl, gm;
};

struct alignas(64) DxParams {
  CUtensorMap tmA;  // scaled dZ fp16 [M][N] (two terms: [2 M][N]), 64 x 128 boxes, 128-byte swizzle
  CUtensorMap tmB;  // operand blocks as rows of 128 bytes, 128 rows a block
  CUtensorMap tmX;  // dX fp16 [M][K], 64 x 128 boxes (two terms: 64 x 64), 128-byte swizzle (stores)
  DxArgs g;
};

struct DxCfg {
  static constexpr int S = 5;                        // stages
  static constexpr int kStage = 32768;               // 16 KB of dZ rows + 16 KB of operand
  static constexpr int kOffY = S * kStage;           // output: two 128-token x 128-input chunks
  static constexpr int kChunk = 32768;
  static constexpr int kOffBar = kOffY + 2 * kChunk;
  static constexpr int kSmem = kOffBar + 256 + 1024;  // + alignment slack
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (2 + kEpiWarps);
  static_assert(kSmem <= 232448, "input gradient pair kernel shared memory above 227 KB");
};

// Unit u: reduction range u % S of tile u / S.  Tiles are visited in groups
// of gm token tiles, the token tile fastest, so the pairs that run together
// share operand blocks and dZ rows.
struct DxUnit {
  int tk, tm, sp, j0, j1;
};
__device__ __forceinline__ DxUnit dx_unit(const DxArgs& g, int u) {
  DxUnit w;
  const int t = u / g.S;
  w.sp = u - t * g.S;
  const int per = g.gm * g.tiles_k;
  const int grp = t / per;
  const int r = t - grp * per;
  const int g0 = grp * g.gm;
  const int gs = g.tiles_m - g0 < g.gm ? g.tiles_m - g0 : g.gm;
  w.tm = g0 + r % gs;
  w.tk = r / gs;
  w.j0 = static_cast<int>(static_cast<long long>(w.sp) * g.nst / g.S);
  w.j1 = static_cast<int>(static_cast<long long>(w.sp + 1) * g.nst / g.S);
  return w;
}

__global__ void __launch_bounds__(DxCfg::kThreads, 1) dx_pair_kernel(const __grid_constant__ DxParams prm) {
  using C = DxCfg;
  const DxArgs& g = prm.g;
  constexpr int S = C::S;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [S] (the even CTA's are used)
  uint64_t* empty = full + S;                                        // [S] (each CTA's own)
  uint64_t* acc_full = empty + S;                                    // [2] each CTA's own
  uint64_t* acc_empty = acc_full + 2;                                // [2] the even CTA's
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int crk = static_cast<int>(cluster_ctarank());
  const int cid = static_cast<int>(cluster_id_x());
  const bool leader = crk == 0;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * C::kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 1) {
    tma_prefetch_desc(&prm.tmA);
    tma_prefetch_desc(&prm.tmB);
    tma_prefetch_desc(&prm.tmX);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync_all();  // both CTAs' barriers exist before either touches the other's
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      griddep_wait();  // dZ and the operand come from the previous kernels
      const uint32_t lfull0 = mapa_shared(smem_u32(&full[0]), 0);
      int gi = 0;
      bool ok = true;
      for (int u = cid; ok && u < g.units; u += g.ncl) {
        const DxUnit w = dx_unit(g, u);
        const int m0 = w.tm * 256 + crk * 128;               // this CTA's 128 rows of dZ
        const int b0 = (2 * w.tk + crk) * g.nst;             // this CTA's 128 inputs
        for (int j = w.j0; j < w.j1; ++j, ++gi) {
          const int s = gi % S;
          if (gi >= S && !mbar_wait(&empty[s], static_cast<uint32_t>(gi / S - 1) & 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (leader) mbar_arrive_expect_tx(&full[s], 2u * C::kStage);
          unsigned char* A = smem + s * C::kStage;
          const uint32_t lb = lfull0 + static_cast<uint32_t>(8 * s);
          tma_load_2d_pair(A, &prm.tmA, lb, j * 64, m0);
          tma_load_2d_pair(A + 16384, &prm.tmB, lb, 0, (b0 + j) * 128);
        }
      }
      // every stage this CTA filled has been consumed by the pair's MMAs (so
      // its copies have landed) before the CTA can leave
      const uint64_t t0 = globaltimer_ns();  // one limit for the whole ring
      for (int t = gi - 1; t >= 0 && t >= gi - S; --t) {
        while (!mbar_try_wait_sleep(&empty[t % S], static_cast<uint32_t>(t / S) & 1u, 1000000u) &&
               globaltimer_ns() - t0 < QLIN_DRAIN_NS) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ pair MMA (even CTA)
    if (leader) {
      constexpr uint32_t idesc = idesc_f16_f32(256, 256) | (1u << 16);  // B MN-major
      const uint64_t adesc0 = sdesc_k_sw128(smem_u32(smem));
      const uint64_t bdesc0 = sdesc_mn_sw128(smem_u32(smem + 16384), 1024, 2048);
      int gi = 0, ti = 0;
      bool ok = true, issued = false;
      for (int u = cid; ok && u < g.units; u += g.ncl, ++ti) {
        const DxUnit w = dx_unit(g, u);
        const int buf = ti & 1;
        if (ti > 1 && !warp_agree(mbar_wait_cluster(&acc_empty[buf], static_cast<uint32_t>((ti >> 1) - 1) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * 256);
        for (int j = w.j0; j < w.j1; ++j, ++gi) {
          const int s = gi % S;
          if (!warp_wait(&full[s], static_cast<uint32_t>(gi / S) & 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          issued = true;
          const uint64_t ad = adesc0 + static_cast<uint64_t>(s * (C::kStage >> 4));
          const uint64_t bd = bdesc0 + static_cast<uint64_t>(s * (C::kStage >> 4));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 channels: 32 bytes of a dZ row, two channel groups
              mma_f16_pair(d, ad + 2 * k, bd + (4096 >> 4) * k, idesc, (j > w.j0 || k > 0) ? 1u : 0u);
            mma_commit_pair(&empty[s], 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) mma_commit_pair(&acc_full[buf], 0x3);
        __syncwarp();
      }
      // every pair MMA has completed before tensor memory can be freed
      if (issued) {
        if (elect_one()) mma_commit_pair(mma_done, 0x1);
        __syncwarp();
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait_sleep(mma_done, 0u, 1000000u) && globaltimer_ns() - t0 < QLIN_DRAIN_NS) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    // TMEM lane = token, column = input.  Two groups of four warps: group
    // grp takes inputs 64 grp .. +63 of each 128-input chunk.
    const int ep = warp - 2;
    const int grp = ep >> 2;
    const int quad = warp & 3;  // TMEM lanes 32*quad .. +31
    const int row = quad * 32 + lane;
    const int trow = g.two ? row >> 1 : row;     // its token among the CTA's, which its even lane writes
    const bool mine = !g.two || !(lane & 1);
    const bool issuer = ep == 0 && lane == 0;
    griddep_wait();  // the rows' factors come from a previous kernel
    int ti = 0;
    bool ok = true;
    for (int u = cid; u < g.units; u += g.ncl, ++ti) {
      const DxUnit w = dx_unit(g, u);
      const int buf = ti & 1;
      const int m0 = g.two ? crk * 64 : w.tm * 256 + crk * 128;
      const int m = m0 + trow;
      const int k0 = w.tk * 256;
      const uint32_t lempty = mapa_shared(smem_u32(&acc_empty[buf]), 0);
      const float f = m < g.M && g.S == 1 ? g.rowscale[m] : 1.f;
      if (ok) ok = mbar_wait(&acc_full[buf], static_cast<uint32_t>(ti >> 1) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t tacc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(buf * 256);
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        unsigned char* yb = smem + C::kOffY + c * C::kChunk + grp * 16384 + trow * 128;
        if (g.S == 1) {
          if (issuer) bulk_wait_group_read1();  // the store of this chunk's previous contents has read them
          named_bar_sync(1, 256);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = c * 128 + grp * 64 + q * 16;
          uint32_t r[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = 0u;
          if (ok) {
            tmem_ld16(tacc + col, r);
            tmem_ld_wait();
          }
          if (g.two) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(__shfl_xor_sync(0xffffffffu, r[j], 1)));
          }
          if (g.S > 1) {
            if (mine && m < g.M && k0 + col < g.K) {  // K % 32 == 0: sixteen inputs or none
              float4* dst = reinterpret_cast<float4*>(g.part + (static_cast<size_t>(w.sp) * g.M + m) * g.K + k0 + col);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                dst[e] = make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                     __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3]));
            }
          } else {
            uint32_t hw[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              hw[e] = h2_as_u32(__floats2half2_rn(__fmul_rn(__uint_as_float(r[2 * e]), f),
                                                  __fmul_rn(__uint_as_float(r[2 * e + 1]), f)));
            if (mine) {
              *reinterpret_cast<uint4*>(yb + (((2 * q) ^ (trow & 7)) << 4)) = make_uint4(hw[0], hw[1], hw[2], hw[3]);
              *reinterpret_cast<uint4*>(yb + (((2 * q + 1) ^ (trow & 7)) << 4)) = make_uint4(hw[4], hw[5], hw[6], hw[7]);
            }
          }
        }
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (leader) mbar_arrive(&acc_empty[buf]);
            else mbar_arrive_remote(lempty);
          }
        }
        if (g.S == 1) {
          fence_proxy_async_smem();  // the rows are read by the bulk copies next
          named_bar_sync(1, 256);
          if (issuer) {
            for (int b = 0; b < 2; ++b) {
              const int k = k0 + c * 128 + b * 64;
              if (k < g.K && m0 < g.M) tma_store_2d(&prm.tmX, smem + C::kOffY + c * C::kChunk + b * 16384, k, m0);
            }
            bulk_commit_group();
          }
        }
      }
    }
    if (issuer) bulk_wait_group_all();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its pair may still signal or read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// dX = rowscale * (sum of the S partial sums, in order), rounded once; eight
// inputs per thread.
__global__ void __launch_bounds__(256) dx_reduce_kernel(const __grid_constant__ DxArgs g) {
  griddep_launch_dependents();
  griddep_wait();
  const size_t mk = static_cast<size_t>(g.M) * g.K;
  const size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (i >= mk) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
  for (int sp = 0; sp < g.S; ++sp) {
    const float4* p = reinterpret_cast<const float4*>(g.part + sp * mk + i);
    const float4 x = __ldcg(p), y = __ldcg(p + 1);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    b.x += y.x; b.y += y.y; b.z += y.z; b.w += y.w;
  }
  const float f = g.rowscale[i / g.K];
  *reinterpret_cast<uint4*>(g.dX + i) =
      make_uint4(h2_as_u32(__floats2half2_rn(__fmul_rn(a.x, f), __fmul_rn(a.y, f))),
                 h2_as_u32(__floats2half2_rn(__fmul_rn(a.z, f), __fmul_rn(a.w, f))),
                 h2_as_u32(__floats2half2_rn(__fmul_rn(b.x, f), __fmul_rn(b.y, f))),
                 h2_as_u32(__floats2half2_rn(__fmul_rn(b.z, f), __fmul_rn(b.w, f))));
}

}  // namespace qlin
