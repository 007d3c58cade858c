// gemm_fused.cuh -- the fused layers (epilogue.cuh) for many-token calls, on
// two SMs at a time.
//
// Operands, loads and products are those of gemm_pair.cuh with the operands'
// roles exchanged: the pair's 256 tokens are the rows of the product (tensor
// memory lanes) and 256 channels its columns, so a thread of the epilogue owns
// one token and neighbouring channels.  Gate and up values of a product then
// meet in one thread, channels leave as 16-byte pieces, and the arithmetic
// runs on fp32 pairs.
//
// What bounds a call beside the products is the time the tensor cores stand
// still between tiles (with the epilogue between them, 4 us a tile against
// 0.3 us a K-block).  So the accumulator is given back as soon as it is in
// registers -- 128 loads a thread, no arithmetic -- and everything else runs
// under the next tile's products.  Without outliers two accumulators alternate
// and nothing waits.  With outliers the second half of tensor memory holds the
// compensation: it is committed and given back apart, so the main accumulator
// is drained under the compensation's products.  Measured: INT8 2048 -> 8192
// at 4736 tokens, GELU, no outliers, 72 us (2200 TOPS) against 94 with one
// accumulator and the channels as the product's rows.
//
// The tiles of a short last wave run as halves of 128 channels, each left to
// the epilogue group of its channels.
//
// Warps 0..3 control (0 loads, 1 tensor memory and products), warps 4..11
// epilogue in two groups of four, group g taking channels 128 g .. +127 of the
// tile; the control warps give registers to the epilogue (setmaxnreg: 128 x
// 40 + 256 x 208 of the 384 x 168 launched).
#pragma once

#include "gemm_pair.cuh"

namespace qlin {

struct FusedPairArgs {
  const float* cscale;
  float cmul;  // factor on c_n (1, or 1/16 for per-channel INT4 widened to 16 q)
  const float* a;
  int M, N, nO;
  int kb;   // 128-wide K-blocks
  int ntn;  // 128-channel tiles of the weights
  int ncs;  // 64-wide outlier slices
  int tiles_n2, tiles_m, gm, ncl;
  int whole, units;  // tiles 0 .. whole - 1, then the other tiles' halves
  EpiArgs epi;
};

struct alignas(64) FusedPairParams {
  CUtensorMap tmA;   // weight blocks as rows of 128 bytes
  CUtensorMap tmAh;  // the same, boxes of half a block
  CUtensorMap tmX;   // Xq int8 [M][K], 128 x 128 boxes, 128-byte swizzle
  CUtensorMap tmU;   // U fp16 [2M][nOp], 64 x 128 boxes, 128-byte swizzle
  CUtensorMap tmWo;  // W_O^T blocks as rows of 128 bytes
  CUtensorMap tmWoh;
  CUtensorMap tmY;   // Y fp16 [M][N], gated [M][N / 2]: 64 x 128 boxes, 128-byte swizzle (stores)
  CUtensorMap tmZ;   // Z fp16 [M][N], the same boxes
  CUtensorMap tmR;   // residual fp16 [M][N], the same boxes (loads)
  FusedPairArgs g;
};

struct FusedPairCfg {
  static constexpr int S = 5;                                 // stages of weight + token rows
  static constexpr int kOffY = S * kPairStage;                // four boxes of 128 tokens x 64 channels
  static constexpr int kOffSc = kOffY + 4 * 16384;            // c'_n of the tile's 256 channels
  static constexpr int kOffBar = kOffSc + 1024;
  static constexpr int kSmem = kOffBar + 256 + 1024;          // + alignment slack
  static constexpr int kEpiWarps = 8;
  static constexpr int kThreads = 32 * (4 + kEpiWarps);
  static_assert(kSmem <= 232448, "fused pair kernel shared memory above 227 KB");
};

template <int R>
__device__ __forceinline__ void setmaxnreg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void setmaxnreg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// Unit u -> (256-channel tile, token tile, half): whole tiles (half -1), then
// the first and second 128 channels of the tiles that are left.  Token tiles
// come in groups of gm, the token tile fastest (pair_tile_coords).
__device__ __forceinline__ void fused_unit_coords(const FusedPairArgs& g, int u, int& tn2, int& tm, int& half) {
  half = u < g.whole ? -1 : (u - g.whole) & 1;
  const int t = u < g.whole ? u : g.whole + ((u - g.whole) >> 1);
  const int per = g.gm * g.tiles_n2;
  const int grp = t / per;
  const int w = t - grp * per;
  const int g0 = grp * g.gm;
  const int gs = g.tiles_m - g0 < g.gm ? g.tiles_m - g0 : g.gm;
  tm = g0 + w % gs;
  tn2 = w / gs;
}

template <int EPI, int ACT>
__global__ void __launch_bounds__(FusedPairCfg::kThreads, 1) gemm_fused_kernel(const __grid_constant__ FusedPairParams prm) {
  using C = FusedPairCfg;
  const FusedPairArgs& g = prm.g;
  constexpr int S = C::S;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kOffBar);  // [S] (the even CTA's are used)
  uint64_t* empty = full + S;                                        // [S] (each CTA's own)
  uint64_t* main_full = empty + S;                                   // [2] each CTA's own
  uint64_t* main_empty = main_full + 2;                              // [2] the even CTA's
  uint64_t* comp_full = main_empty + 2;                              // each CTA's own
  uint64_t* comp_empty = comp_full + 1;                              // the even CTA's
  uint64_t* res_full = comp_empty + 1;                               // [2] residual boxes of each epilogue group
  uint64_t* mma_done = res_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int crk = static_cast<int>(cluster_ctarank());
  const int cid = static_cast<int>(cluster_id_x());
  const bool leader = crk == 0;
  const bool comp = g.nO > 0;
  const int nbuf = comp ? 1 : 2;
  const int T = g.kb + 2 * g.ncs;

  if (warp == 0 && lane == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&main_full[b], 1);
      mbar_init(&main_empty[b], 2 * C::kEpiWarps);
      mbar_init(&res_full[b], 1);
    }
    mbar_init(comp_full, 1);
    mbar_init(comp_empty, 2 * C::kEpiWarps);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 1) {
    tma_prefetch_desc(&prm.tmA);
    tma_prefetch_desc(&prm.tmX);
    tma_prefetch_desc(&prm.tmY);
    if (comp) {
      tma_prefetch_desc(&prm.tmU);
      tma_prefetch_desc(&prm.tmWo);
    }
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

  if (warp < 4) {
    setmaxnreg_dec<40>();
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        griddep_wait();  // Xq, U and widened weights come from the previous kernels
        const uint32_t lfull0 = mapa_shared(smem_u32(&full[0]), 0);
        int gi = 0;
        bool ok = true;
        for (int u = cid; ok && u < g.units; u += g.ncl) {
          int tn2, tm, half;
          fused_unit_coords(g, u, tn2, tm, half);
          // the channels this CTA loads: a block of 128, or half of one
          const int ctile = 2 * tn2 + (half < 0 ? crk : half);
          const int c0 = half < 0 ? 0 : crk * 64;
          const CUtensorMap* mapA = half < 0 ? &prm.tmA : &prm.tmAh;
          const CUtensorMap* mapWo = half < 0 ? &prm.tmWo : &prm.tmWoh;
          const uint32_t bytes = 2u * (half < 0 ? kPairStage : kPairStage - 8192);
          const int m0 = tm * 256 + crk * 128;  // its 128 tokens
          for (int r = 0; r < T; ++r, ++gi) {
            const int s = gi % S;
            if (gi >= S && !mbar_wait(&empty[s], static_cast<uint32_t>(gi / S - 1) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            if (leader) mbar_arrive_expect_tx(&full[s], bytes);
            unsigned char* W = smem + s * kPairStage;
            unsigned char* X = W + 16384;
            const uint32_t lb = lfull0 + static_cast<uint32_t>(8 * s);
            if (r < g.kb) {
              tma_load_2d_pair(W, mapA, lb, 0, (ctile * g.kb + r) * 128 + c0);
              tma_load_2d_pair(X, &prm.tmX, lb, r * 128, m0);
            } else {
              const int j = r - g.kb;
              const int lo = j >= g.ncs ? 1 : 0;  // U rows [0, M) hold hi, [M, 2M) hold lo
              const int ib = j - lo * g.ncs;
              tma_load_2d_pair(W, mapWo, lb, 0, (ctile * g.ncs + ib) * 128 + c0);
              tma_load_2d_pair(X, &prm.tmU, lb, ib * 64, lo * g.M + m0);
            }
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
    } else if (warp == 1 && leader) {
      // ---------------------------------------------------------- pair MMA (even CTA)
      const uint64_t xdesc0 = sdesc_k_sw128(smem_u32(smem + 16384));  // rows: tokens
      const uint64_t wdesc0 = sdesc_k_sw128(smem_u32(smem));          // columns: channels
      int gi = 0, ti = 0;
      bool ok = true, issued = false;
      for (int u = cid; ok && u < g.units; u += g.ncl, ++ti) {
        const int buf = ti % nbuf, use = ti / nbuf;
        const uint32_t idesc_main = u < g.whole ? idesc_s8_s32(256, 256) : idesc_s8_s32(256, 128);
        const uint32_t idesc_comp = u < g.whole ? idesc_f16_f32(256, 256) : idesc_f16_f32(256, 128);
        if (use > 0 && !warp_agree(mbar_wait_cluster_poll(&main_empty[buf], static_cast<uint32_t>(use - 1) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(buf * 256);
        for (int r = 0; r < T; ++r, ++gi) {
          const int s = gi % S;
          if (!warp_wait(&full[s], static_cast<uint32_t>(gi / S) & 1u, abort_flag)) {
            ok = false;
            break;
          }
          if (r == g.kb && ti > 0 &&
              !warp_agree(mbar_wait_cluster_poll(comp_empty, static_cast<uint32_t>(ti - 1) & 1u, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          issued = true;
          const uint64_t xd = xdesc0 + static_cast<uint64_t>(s * (kPairStage >> 4));
          const uint64_t wd = wdesc0 + static_cast<uint64_t>(s * (kPairStage >> 4));
          if (elect_one()) {
            if (r < g.kb) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_i8_pair(d, xd + 2 * k, wd + 2 * k, idesc_main, (r > 0 || k > 0) ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f16_pair(tmem + 256, xd + 2 * k, wd + 2 * k, idesc_comp, (r > g.kb || k > 0) ? 1u : 0u);
            }
            mma_commit_pair(&empty[s], 0x3);
            if (r == g.kb - 1) mma_commit_pair(&main_full[buf], 0x3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (comp && elect_one()) mma_commit_pair(comp_full, 0x3);
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
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    setmaxnreg_inc<208>();
    const EpiArgs& e = g.epi;
    const int grp = (warp - 4) >> 2;
    const int quad = warp & 3;            // TMEM lanes 32*quad .. +31
    const int row = quad * 32 + lane;     // token row of this CTA's 128
    const int gt = threadIdx.x - 128 - grp * 128;
    const bool issuer = gt == 0;          // of the group's stores
    const int gbar = 1 + grp;             // the group's named barrier
    float* sc = reinterpret_cast<float*>(smem + C::kOffSc) + grp * 128;
    constexpr int kOut = EPI == kEpiGated ? 1 : 2;  // 64-channel output boxes of a group
    unsigned char* box0 = smem + C::kOffY + grp * 2 * 16384 + row * 128;
    const int sw = row & 7;
    const int F = EPI == kEpiGated ? g.N >> 1 : g.N;  // channels of Y
    griddep_wait();  // a[] comes from the previous kernel
    int ti = 0, tr = 0;  // units of the pair; those with channels of this group
    int loads = 0;       // the issuer's residual loads, one a unit as long as no wait gives up
    bool ok = true;
    for (int u = cid; u < g.units; u += g.ncl, ++ti) {
      int tn2, tm, half;
      fused_unit_coords(g, u, tn2, tm, half);
      const int buf = ti % nbuf, use = ti / nbuf;
      if (half == 1 - grp) {  // the other group's 128 channels: only give the accumulators back
        if (ok) ok = mbar_wait(&main_full[buf], static_cast<uint32_t>(use) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&main_empty[buf]), 0));
        if (comp) {
          if (ok) ok = mbar_wait(comp_full, static_cast<uint32_t>(ti) & 1u, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(comp_empty), 0));
        }
        continue;
      }
      const int n0 = tn2 * 256 + grp * 128;  // the group's first channel
      const int m0 = tm * 256 + crk * 128;
      const int m = m0 + row;
      // the group's boxes leave through TMA; `store` hands them over once every
      // thread of the group has written
      auto take_boxes = [&] {
        if (issuer) bulk_wait_group_read0();
        named_bar_sync(gbar, 128);
      };
      // the issuer has taken the boxes: the residual on its way into them.  Not
      // after a wait gave up: the issuer then no longer waits for a load's
      // bytes before it would arm the barrier and fill the boxes again.
      auto load_residual = [&] {
        if (!ok) return;
        ++loads;
        int n = 0;
        for (int b = 0; b < 2; ++b) n += n0 + 64 * b < g.N && m0 < g.M ? 1 : 0;
        mbar_arrive_expect_tx(&res_full[grp], static_cast<uint32_t>(n) * 16384u);
        for (int b = 0; b < n; ++b)
          tma_load_2d(smem + C::kOffY + (grp * 2 + b) * 16384, &prm.tmR, &res_full[grp], n0 + 64 * b, m0);
      };
      auto store_boxes = [&](const CUtensorMap* map, int boxes, int width) {
        fence_proxy_async_smem();
        named_bar_sync(gbar, 128);
        if (issuer) {
          const int x0 = (tn2 * 2 + grp) * 64 * boxes;
          for (int b = 0; b < boxes; ++b)
            if (x0 + 64 * b < width && m0 < g.M)
              tma_store_2d(map, smem + C::kOffY + (grp * 2 + b) * 16384, x0 + 64 * b, m0);
          bulk_commit_group();
        }
      };
      named_bar_sync(gbar, 128);  // the previous tile's factors have been used
      sc[gt] = n0 + gt < g.N ? __fmul_rn(g.cscale[n0 + gt], g.cmul) : 0.f;
      const float am = m < g.M ? g.a[m] : 0.f;
      const bool residual = EPI == kEpiAct && e.residual;
      if (residual && !e.Z && issuer) {  // (with Z the boxes hold that first)
        bulk_wait_group_read0();
        load_residual();
      }
      named_bar_sync(gbar, 128);
      if (ok) ok = mbar_wait(&main_full[buf], static_cast<uint32_t>(use) & 1u, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half < 0 ? grp * 128 : 0);
      uint32_t r[128];
      if (ok) {
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(trow + static_cast<uint32_t>(buf * 256 + 32 * q), r + 32 * q);
        tmem_ld_wait();
      } else {
#pragma unroll
        for (int q = 0; q < 128; ++q) r[q] = 0u;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&main_empty[buf]), 0));
      // v = c'_n acc, then + comp, * a_m, + bias: the operations and roundings
      // of the unfused epilogue
      f32x2 v[64];
#pragma unroll
      for (int q = 0; q < 32; ++q) {
        const float4 c = *reinterpret_cast<const float4*>(sc + 4 * q);
        v[2 * q] = f2_mul(f2_pack(c.x, c.y), f2_pack(static_cast<float>(static_cast<int32_t>(r[4 * q])),
                                                     static_cast<float>(static_cast<int32_t>(r[4 * q + 1]))));
        v[2 * q + 1] = f2_mul(f2_pack(c.z, c.w), f2_pack(static_cast<float>(static_cast<int32_t>(r[4 * q + 2])),
                                                         static_cast<float>(static_cast<int32_t>(r[4 * q + 3]))));
      }
      if (comp) {
        if (ok) ok = mbar_wait(comp_full, static_cast<uint32_t>(ti) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        if (ok) {
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            uint32_t u[16];
            tmem_ld16(trow + static_cast<uint32_t>(256 + 16 * q), u);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[8 * q + j] = f2_add(v[8 * q + j], f2_pack(__uint_as_float(u[2 * j]), __uint_as_float(u[2 * j + 1])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(comp_empty), 0));
      }
      const f32x2 a2 = f2_both(am);
#pragma unroll
      for (int q = 0; q < 64; ++q) v[q] = f2_mul(v[q], a2);
      if (e.bias) {
#pragma unroll
        for (int q = 0; q < 32; ++q) {  // all lanes read one address; N is a multiple of 16
          if (n0 + 4 * q < g.N) {
            const float4 b = __ldg(reinterpret_cast<const float4*>(e.bias + n0) + q);
            v[2 * q] = f2_add(v[2 * q], f2_pack(b.x, b.y));
            v[2 * q + 1] = f2_add(v[2 * q + 1], f2_pack(b.z, b.w));
          }
        }
      }
      if (!residual || e.Z) take_boxes();
      if (e.Z) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const f32x2 o[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          *reinterpret_cast<uint4*>(box0 + (q >> 3) * 16384 + (((q & 7) ^ sw) << 4)) = f2_to_h8(o);
        }
        store_boxes(&prm.tmZ, 2, g.N);
        if (residual && issuer) {
          bulk_wait_group_read0();
          load_residual();
        }
        if (!residual) take_boxes();
      }
      if (residual) {
        if (ok) ok = mbar_wait(&res_full[grp], static_cast<uint32_t>(tr) & 1u, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
      }
      if (EPI == kEpiGated) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {  // eight gate and up pairs -> eight channels
          f32x2 h[4], up[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 p0 = f2_unpack(v[8 * q + 2 * j]), p1 = f2_unpack(v[8 * q + 2 * j + 1]);
            h[j] = f2_pack(p0.x, p1.x);
            up[j] = f2_pack(p0.y, p1.y);
          }
          act_pairs<4>(ACT, h);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = f2_mul(h[j], up[j]);
          *reinterpret_cast<uint4*>(box0 + ((q ^ sw) << 4)) = f2_to_h8(h);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          uint4* at = reinterpret_cast<uint4*>(box0 + (q >> 3) * 16384 + (((q & 7) ^ sw) << 4));
          f32x2 o[4] = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
          act_pairs<4>(ACT, o);
          if (residual) {
            f32x2 x[4];
            h8_to_f2(*at, x);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = f2_add(o[j], x[j]);
          }
          *at = f2_to_h8(o);
        }
      }
      store_boxes(&prm.tmY, kOut, F);
      ++tr;
    }
    if (issuer) {
      bulk_wait_group_all();
      // a residual box still on its way (only after a wait gave up) lands before the CTA leaves
      if (!ok) drain_ring(&res_full[grp], 1, loads);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its pair may still signal or read it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

}  // namespace qlin
