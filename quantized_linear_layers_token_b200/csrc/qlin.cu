// qlin.cu -- the C ABI declared in include/qlin.h: host-side validation,
// TMA descriptor encoding, launch selection.  All kernels live in the
// headers included below so the library is one translation unit (the device
// error word needs no relocatable device code).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <atomic>
#include <mutex>

#include "qlin.h"
#include "act_quant.cuh"
#include "gemm.cuh"
#include "gemm_fused.cuh"
#include "gemm_pair.cuh"
#include "backward.cuh"
#include "dact.cuh"
#include "dx_pair.cuh"
#include "gptq.cuh"
#include "norm.cuh"
#include "offq.cuh"
#include "pack.cuh"
#include "smooth.cuh"

using namespace qlin;

namespace {

thread_local char t_last_error[512] = "";

qlin_status fail(qlin_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_last_error, sizeof(t_last_error), fmt, ap);
  va_end(ap);
  return st;
}

#define QLIN_CUDA_TRY(expr)                                                                    \
  do {                                                                                         \
    cudaError_t e_ = (expr);                                                                   \
    if (e_ != cudaSuccess)                                                                     \
      return fail(QLIN_ERR_CUDA, "%s failed: %s", #expr, cudaGetErrorString(e_));              \
  } while (0)

#define QLIN_LAUNCH_CHECK(what)                                                                \
  do {                                                                                         \
    cudaError_t e_ = cudaGetLastError();                                                       \
    if (e_ != cudaSuccess) return fail(QLIN_ERR_CUDA, "%s launch failed: %s", what,           \
                                       cudaGetErrorString(e_));                                \
  } while (0)

constexpr size_t kAlign = 256;

// What every workspace starts with, wherever its call puts the rest: all that
// must be zero on entry and is left zero, at one place for every layer, token
// count and entry point, so that any of them may follow another on a workspace.
struct WorkspaceHead {
  unsigned cnt[512];       // counters of split tiles: one per persistent CTA of the GEMM, two per split
                           // tile of a launch on CTA pairs, one per split tile of the input gradient
  unsigned momentum[64];   // completion counter of each problem's momentum update
  unsigned cmax[4096];     // outlier column maxima, as many as a layer may have
};
constexpr int kHeadCounters = 512;
static_assert(sizeof(WorkspaceHead) == QLIN_WORKSPACE_HEAD && QLIN_WORKSPACE_HEAD % kAlign == 0, "include/qlin.h");
static_assert(kMaxGrid <= kHeadCounters && 2 * 2 * kMaxPairs <= kHeadCounters && kMaxProbs <= 64, "counters of a launch");
WorkspaceHead* head_of(void* workspace) { return static_cast<WorkspaceHead*>(workspace); }
size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
int pad8(int n) { return (n + 7) / 8 * 8; }

qlin_status check_shape(int32_t K, int32_t N, int32_t fmt, int32_t nO) {
  if (fmt != QLIN_W4_PERCHANNEL && fmt != QLIN_W4_G128 && fmt != QLIN_W8_PERCHANNEL)
    return fail(QLIN_ERR_ARG, "unknown weight format %d", fmt);
  if (K <= 0 || N <= 0 || nO < 0) return fail(QLIN_ERR_ARG, "negative or zero size K=%d N=%d n_outlier=%d", K, N, nO);
  if (K % 32 != 0 || K > 65536) return fail(QLIN_ERR_SHAPE, "K=%d must be a multiple of 32, at most 65536", K);
  if (N % 16 != 0) return fail(QLIN_ERR_SHAPE, "N=%d must be a multiple of 16", N);
  if (fmt == QLIN_W4_G128 && K % 128 != 0) return fail(QLIN_ERR_SHAPE, "g128 needs K %% 128 == 0 (K=%d)", K);
  if (nO > K || nO > 4096) return fail(QLIN_ERR_SHAPE, "n_outlier=%d must be <= min(K, 4096)", nO);
  return QLIN_OK;
}

struct Layout {
  size_t codes, chan, group, fold, oidx, wot, wmax, total;
};

Layout weights_layout(int32_t K, int32_t N, int32_t fmt, int32_t nO) {
  Layout L{};
  size_t off = 0;
  const size_t tiles_n = (N + 127) / 128, kb = (K + 127) / 128, ib = (nO + 63) / 64;
  const size_t codes_b = tiles_n * kb * ((fmt == QLIN_W8_PERCHANNEL) ? 16384 : 8192);
  L.codes = off; off = round_up(off + codes_b, kAlign);
  L.chan = off; off = round_up(off + size_t(N) * 4, kAlign);
  const size_t gb = (fmt == QLIN_W4_G128) ? size_t(K / 128) * N * 2 : 0;
  L.group = off; off = round_up(off + gb, kAlign);
  L.fold = off; off = round_up(off + gb, kAlign);
  L.oidx = off; off = round_up(off + size_t(nO) * 4, kAlign);
  L.wot = off; off = round_up(off + tiles_n * ib * 16384, kAlign);
  L.wmax = off; off = round_up(off + size_t(nO) * 4, kAlign);
  L.total = off;
  return L;
}

qlin_status check_weights(const qlin_weights* w) {
  if (!w) return fail(QLIN_ERR_ARG, "weights descriptor is NULL");
  qlin_status st = check_shape(w->K, w->N, w->fmt, w->n_outlier);
  if (st != QLIN_OK) return st;
  if (w->n_outlier_pad != pad8(w->n_outlier))
    return fail(QLIN_ERR_ARG, "n_outlier_pad=%d must be n_outlier rounded up to 8 (%d)", w->n_outlier_pad, pad8(w->n_outlier));
  if (w->fmt == QLIN_W4_G128 && w->group != 128) return fail(QLIN_ERR_ARG, "g128 format needs group=128");
  if (w->fmt != QLIN_W4_G128 && w->group != 0) return fail(QLIN_ERR_ARG, "per-channel formats need group=0");
  if (!w->codes || !w->chan_scale) return fail(QLIN_ERR_ARG, "codes/chan_scale is NULL");
  if (w->fmt == QLIN_W4_G128 && (!w->group_scale || !w->fold_ratio)) return fail(QLIN_ERR_ARG, "g128 scales are NULL");
  if (w->n_outlier > 0 && (!w->outlier_idx || !w->W_Ot || !w->wmax_O))
    return fail(QLIN_ERR_ARG, "outlier buffers are NULL");
  if (!aligned16(w->codes) || !aligned16(w->chan_scale) || (w->group_scale && !aligned16(w->group_scale)) ||
      (w->fold_ratio && !aligned16(w->fold_ratio)) || (w->W_Ot && !aligned16(w->W_Ot)) ||
      (w->outlier_idx && !aligned16(w->outlier_idx)) || (w->wmax_O && !aligned16(w->wmax_O)))
    return fail(QLIN_ERR_ALIGN, "a weights buffer is not 16-byte aligned");
  return QLIN_OK;
}

// ---------------------------------------------------------------- TMA maps
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

qlin_status get_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return fail(QLIN_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  return QLIN_OK;
}

// 2-D map over a row-major [outer][inner] array of `esize`-byte elements.
qlin_status make_map(CUtensorMap* map, const void* base, CUtensorMapDataType dt, int esize, uint64_t inner,
                     uint64_t outer, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw) {
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {inner * static_cast<uint64_t>(esize)};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(QLIN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return QLIN_OK;
}

// ---------------------------------------------------------------- launches
// Test and measurement knobs (qlin_debug_set); the defaults are the tuned
// behaviour.  Kernels are launched with programmatic dependent launch, so
// each may start its prologue (and the GEMM its weight stream) while the
// previous kernel in the stream finishes; every kernel waits on the grid
// dependency before it reads what the previous one wrote.
std::atomic<long long> g_knob[11] = {{1}, {1}, {0}, {0}, {256}, {512}, {kFusedMomentumMaxM}, {2000000000LL}, {2}, {0}, {0}};

long long knob(int k) { return g_knob[k].load(std::memory_order_relaxed); }

bool cluster_disabled() { return knob(QLIN_KNOB_CLUSTER) == 0; }

int forced_cluster_size() {
  const long long v = knob(QLIN_KNOB_CLUSTER_SIZE);
  return (v == 2 || v == 4 || v == 8) ? static_cast<int>(v) : 0;
}

bool pdl_enabled() { return knob(QLIN_KNOB_PDL) != 0; }

// `cluster` > 1 launches thread-block clusters of that many CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_kc(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, int cluster,
                      Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (pdl_enabled()) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_k(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                     Args... args) {
  return launch_kc(kern, grid, block, smem, stream, 1, args...);
}

// Raise a kernel's shared-memory limit, once on each device (the attribute
// belongs to the device's context).
template <auto Kern>
cudaError_t allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

int sm_count() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!cached[dev]) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    cached[dev] = n;
  }
  return cached[dev];
}

// CTAs a GEMM may use at most (QLIN_KNOB_MAX_CTAS; default all SMs).
int gemm_cta_cap() {
  const long long v = knob(QLIN_KNOB_MAX_CTAS);
  const int sms = sm_count();
  return (v > 0 && v < sms) ? static_cast<int>(v) : sms;
}

// INT4 layers on CTA pairs up to this many tokens convert their codes inside
// the GEMM instead of widening them ahead (QLIN_KNOB_CONVERT_MAX_M; 0 never).
long long convert_max_m() { return knob(QLIN_KNOB_CONVERT_MAX_M); }

// QLIN_KNOB_MAX_TOKEN_TILE = 64 or 128 caps the token tile.
int max_bt() {
  const long long x = knob(QLIN_KNOB_MAX_TOKEN_TILE);
  return (x == 64 || x == 128) ? static_cast<int>(x) : 256;
}

int pick_bt(int M) {
  int bt = 256;
  if (M <= 16) bt = 16;
  else if (M <= 32) bt = 32;
  else if (M <= 64) bt = 64;
  else if (M <= 128) bt = 128;
  return bt < max_bt() ? bt : max_bt();
}

// Work decomposition of one GEMM launch over one or more problems that
// share the token count M (same on the host for workspace sizes and for the
// launch).
struct GemmPlan {
  int bt, grid, split, widen, nprob;
  long long tiles;         // tiles of every problem
  GemmProb pr[kMaxProbs];  // per problem: shape, tiles and iteration offsets (pointers unset)
  size_t acc_off, comp_off, w8_off, total;  // shared scratch (after the problems' U operands)
  size_t u_off[kMaxProbs];                           // each problem's compensation operand U
  // CTA-pair launch (one problem, 256 x 256 tiles): pairs, whole tiles and
  // the stream-K tail's step boundaries and partial slots
  int pair_ncl, pair_dp;
  long long pair_sk_tiles;
  size_t pacc_off, pcomp_off;
  unsigned pair_bnd[kMaxPairs + 1];
};

bool use_pair(const GemmPlan& p, const qlin_weights* w);
template <int FMT>
int pair_max_clusters();

// Work split of a launch on CTA pairs over `tiles` tiles of T steps (the
// last T - kb of them the outlier compensation, never split).  Whole tiles
// in raster order while they fill whole waves; when the last wave would be
// partly empty, the last full wave and the remainder are instead divided by
// steps into one contiguous range per pair (stream-K), so every pair ends
// at about the same time.  With eight or more full waves the empty part of
// the last one is small and tiles stay whole.
void pair_split(GemmPlan& p, long long tiles, int T, int kb, int maxc, bool may_split) {
  if (maxc > kMaxPairs) maxc = kMaxPairs;
  p.pair_sk_tiles = 0;
  for (int c = 0; c <= kMaxPairs; ++c) p.pair_bnd[c] = 0u;
  const long long full = tiles / maxc, rem = tiles % maxc;
  if (!may_split || knob(QLIN_KNOB_PAIR_SPLIT) == 0 || rem == 0 || full >= 8 || maxc < 2) {
    p.pair_ncl = static_cast<int>(tiles < maxc ? tiles : maxc);
    p.pair_dp = static_cast<int>(tiles);
    return;
  }
  p.pair_ncl = maxc;
  p.pair_dp = static_cast<int>(full >= 1 ? (full - 1) * maxc : 0);
  p.pair_sk_tiles = tiles - p.pair_dp;
  const unsigned long long total = static_cast<unsigned long long>(p.pair_sk_tiles) * T;
  unsigned prev = 0;
  for (int c = 0; c <= p.pair_ncl; ++c) {
    unsigned long long b = total * c / p.pair_ncl;
    const unsigned long long r = b % T;
    if (r > static_cast<unsigned long long>(kb) && r < static_cast<unsigned long long>(T))
      b = (r - kb <= T - r) ? b - (r - kb) : b + (T - r);  // not inside a compensation run
    if (c == p.pair_ncl) b = total;
    unsigned v = static_cast<unsigned>(b);
    if (v < prev) v = prev;
    p.pair_bnd[c] = v;
    prev = v;
  }
}

// From this many tokens the INT4 formats widen their weights once per call
// and run the INT8 kernel (QLIN_KNOB_WIDEN_MIN_M; 0 turns it off).
int widen_min_m() { return static_cast<int>(knob(QLIN_KNOB_WIDEN_MIN_M)); }

// CTAs per tile of a fused launch that has fewer than four tiles per SM: 1
// for whole tiles, 2, 4 or 8 for ranges that end with the tiles (token tiles
// of 128 and 256), 0 to leave tiles of up to 64 tokens to the cluster and
// stream-K splits of the launch.  The least of estimated times in us, from
// measurements on B200: a pipeline step (512, 256 or 128 inputs of a tile at
// token tiles of 16, up to 64, above) by format, the exchange of a cluster
// round, the fix-up of stream-K or of n partial tiles of mv tokens.  At 64
// tokens of 4096 -> 11008 whole tiles take 16 to 19 us against 26 to 29 split;
// at 200 tokens 30 to 35 against 69; 11008 -> 4096 at 200 tokens takes 56 to
// 67 us whole, 50 to 52 in four ranges and 82 to 83 in one per SM.
int fused_tile_ctas(const GemmProb& g, int bt, int fmt, long long tiles, int sms) {
  const int f = fmt == QLIN_W4_G128 ? 1 : (fmt == QLIN_W8_PERCHANNEL ? 2 : 0);
  const double T = g.T;
  if (bt >= 128) {
    static const double step[3] = {0.43, 0.57, 0.35};
    const double mv = g.M < bt ? g.M : bt;
    int best = 1;
    double least = T * step[f];
    for (int n = 2; n <= 8 && n <= g.T && tiles * n <= sms; n *= 2) {
      const double us = T / n * step[f] + 8.0 + 0.016 * mv * n;
      if (us < least) {
        least = us;
        best = n;
      }
    }
    return best;
  }
  static const double step16[3] = {0.53, 1.13, 0.78}, step64[3] = {0.42, 0.70, 0.50};
  const double st = bt == 16 ? step16[f] : step64[f];
  const double fixup = bt == 16 ? 8.0 : (bt == 32 ? 15.0 : 21.0);
  const double round = bt == 16 ? (f == 1 ? 1.2 : 1.8) : (bt == 32 ? 2.0 : 3.7);
  const double drain = bt == 16 ? 1.0 : (bt == 32 ? 1.5 : 2.0);
  const double whole = static_cast<double>((tiles + sms - 1) / sms) * (T * st + drain);
  double split = T * tiles / sms * st + fixup;
  for (int cs = 2; cs <= 8 && cs <= g.nk; cs *= 2) {
    const double us = static_cast<double>((tiles + sms / cs - 1) / (sms / cs)) * ((T + cs - 1) / cs * st + round);
    if (us < split) split = us;
  }
  return whole < split ? 1 : 0;
}

// `fused` launches (a fused epilogue, one problem) keep whole tiles on CTA
// pairs, widen INT4 ahead of them, and split tiles by fused_tile_ctas.
GemmPlan plan_gemm_group(int M, const qlin_weights* const* ws, int n, bool fused = false) {
  GemmPlan p{};
  p.nprob = n;
  p.bt = pick_bt(M);
  // Fused INT8 layers on CTA pairs from 97 tokens on (4096 -> 4096 at 128
  // tokens 19.0 against 22.3 us, 1024 -> 1024 10.3 against 12.4; at 70 tokens
  // of 11008 -> 4096 36 against 30).
  if (fused && ws[0]->fmt == QLIN_W8_PERCHANNEL && M > 96 && p.bt == 128 && max_bt() == 256) p.bt = 256;
  const int ks = gemm_ks(p.bt);
  bool any_outliers = false;
  unsigned it = 0;
  for (int q = 0; q < n; ++q) {
    const qlin_weights* w = ws[q];
    GemmProb& g = p.pr[q];
    g.M = M;
    g.N = w->N;
    g.K = w->K;
    g.nO = w->n_outlier;
    g.tiles_n = (w->N + 127) / 128;
    g.tiles_m = (M + p.bt - 1) / p.bt;
    g.kb = (w->K + 127) / 128;
    g.nk = (g.kb + ks - 1) / ks;
    g.ncs = w->n_outlier > 0 ? (w->n_outlier + 63) / 64 : 0;
    g.nc = (p.bt <= 64) ? g.ncs : 2 * g.ncs;
    g.T = g.nk + g.nc;
    g.gm = 1;
    g.it0 = it;
    it += static_cast<unsigned>(static_cast<long long>(g.tiles_n) * g.tiles_m * g.T);
    p.tiles += static_cast<long long>(g.tiles_n) * g.tiles_m;
    any_outliers = any_outliers || w->n_outlier > 0;
  }
  long long iters = 0;
  for (int q = 0; q < n; ++q) iters += static_cast<long long>(p.pr[q].tiles_n) * p.pr[q].tiles_m * p.pr[q].T;
  const int sms = gemm_cta_cap();
  // Split tiles (stream-K or cluster split-K) when whole tiles would leave
  // SMs idle or badly balanced.  Token tiles of 128/256 have partials of
  // 64-128 KiB, so they split only when there are fewer tiles than SMs.
  // Groups of decode problems split too: their tiles differ in length (K),
  // and only split points give every CTA the same number of iterations.
  p.split = (p.tiles < (p.bt >= 128 ? 1LL : 4LL) * sms || (n > 1 && p.bt <= 64)) ? 1 : 0;
  long long units = p.split ? iters : p.tiles;
  // (a forced cluster setting keeps the splits it asks for)
  if (fused && p.split && sms >= 8 && (p.bt > 64 || !(cluster_disabled() || forced_cluster_size()))) {
    const int ctas = fused_tile_ctas(p.pr[0], p.bt, ws[0]->fmt, p.tiles, sms);
    if (ctas == 1) p.split = 0;
    if (ctas >= 1) units = p.tiles * ctas;  // ranges of one tile each: every ctas-th boundary is a tile start
  }
  const int cap = sms < kMaxGrid ? sms : kMaxGrid;
  p.grid = static_cast<int>(units < cap ? units : cap);
  if (p.grid < 1) p.grid = 1;
  // Raster order of many-token problems: the CTAs running at once should
  // share weight tiles and reuse activation tiles from L2.  All token tiles
  // in one group when the INT8 activations (M x K) fit well inside L2, else
  // groups of about sqrt(grid * 128 / BT) token tiles (the size that
  // minimises the activation bytes plus the weight bytes one wave of CTAs
  // touches).
  for (int q = 0; q < n; ++q) {
    GemmProb& g = p.pr[q];
    if (g.tiles_m <= 1) continue;
    const double x_bytes = static_cast<double>(M) * g.K;
    int gm = static_cast<int>(std::lround(std::sqrt(static_cast<double>(p.grid) * 128.0 / p.bt)));
    if (x_bytes <= 48.0 * 1024 * 1024) gm = g.tiles_m;
    g.gm = gm < 1 ? 1 : (gm > g.tiles_m ? g.tiles_m : gm);
  }
  size_t off = 0;
  for (int q = 0; q < n; ++q) {
    p.u_off[q] = off;
    off = round_up(off + (ws[q]->n_outlier > 0 ? size_t(2) * M * ws[q]->n_outlier_pad * 2 : 0), kAlign);
  }
  const size_t slot_bytes = size_t(p.bt) * 128 * 4;
  p.acc_off = off;
  off = round_up(off + (p.split ? size_t(2) * p.grid * slot_bytes : 0), kAlign);
  p.comp_off = off;
  off = round_up(off + (p.split && any_outliers ? size_t(2) * p.grid * slot_bytes : 0), kAlign);
  // A fused launch widens from its second token tile on.  g128 layers gain at
  // every size measured (at 257 tokens 4096 -> 11008 41 against 54 us, 4096 ->
  // 2 x 11008 70 against 75, 8192 -> 2 x 28672 299 against 310).  Per-channel ones,
  // whose codes cost less to convert inside the kernel, gain where they are small
  // (4096 -> 4096 24 against 28, 4096 -> 11008 41 against 45) and lose towards the
  // limit below (4096 -> 2 x 11008 69.5 against 61 at 257 tokens, 84 against 80 at
  // 700); past it they widen as other launches do.  And in the first tile of 256
  // while the layer is small for the tokens (4096
  // -> 4096 at 129 tokens 25.3 against 28.3 us, at 256 25.4 against 33.5; 1024
  // -> 1024 14 against 17 and 21; but 4096 -> 11008 at 129 36 against 30).
  int widen_from = widen_min_m();
  if (fused && widen_from > 0) {
    const long long weights = static_cast<long long>(ws[0]->K) * ws[0]->N;
    if (widen_from > 257 && (ws[0]->fmt == QLIN_W4_G128 || weights <= 100000000LL)) widen_from = 257;
    if (widen_from > 129 && weights <= 131072LL * M) widen_from = 129;
  }
  p.widen = (n == 1 && ws[0]->fmt != QLIN_W8_PERCHANNEL && p.bt == 256 && widen_from > 0 && M >= widen_from) ? 1 : 0;
  p.w8_off = off;
  off = round_up(off + (p.widen ? size_t(p.pr[0].tiles_n) * p.pr[0].kb * 16384 : 0), kAlign);
  p.pair_ncl = 0;
  p.pair_dp = 0;
  p.pair_sk_tiles = 0;
  p.pacc_off = p.pcomp_off = off;
  if (n == 1 && use_pair(p, ws[0])) {
    const GemmProb& q = p.pr[0];
    const bool conv = p.widen && M <= convert_max_m() && !fused;
    const int maxc = !conv ? pair_max_clusters<kFmtW8>()
                           : (ws[0]->fmt == QLIN_W4_PERCHANNEL ? pair_max_clusters<kFmtW4PC>()
                                                                : pair_max_clusters<kFmtW4G128>());
    const long long tiles = static_cast<long long>((q.tiles_n + 1) / 2) * q.tiles_m;
    pair_split(p, tiles, q.kb + 2 * q.ncs, q.kb, maxc > 0 ? maxc : 1, !fused);
    // Fused tiles that would fill at most half of the last wave become two
    // half tiles each (128 channels; less than twice the speed, since a half
    // loads all of the tile's tokens): INT8 4096 -> 4096 at 512 tokens 23.1
    // against 25.4 us, 1024 -> 1024 at 512 13.6 against 15.9, 4096 -> 11008
    // at 1000 tokens 51.0 against 53.4.
    const long long rem = maxc > 0 ? tiles % maxc : 0;
    if (fused && 2 * rem <= maxc) {
      p.pair_dp = static_cast<int>(tiles - rem);
      p.pair_ncl = static_cast<int>(tiles + rem < maxc ? tiles + rem : maxc);
    }
    if (p.pair_sk_tiles > 0) {
      const size_t part = size_t(2) * 256 * 128 * 4;  // one slot: both CTAs' 128 channels x 256 tokens
      off = round_up(off + size_t(2) * p.pair_ncl * part, kAlign);
      p.pcomp_off = off;
      off = round_up(off + (ws[0]->n_outlier > 0 ? size_t(p.pair_ncl) * part : 0), kAlign);
    }
  }
  p.total = off;
  return p;
}

// A GEMM launch's scratch (laid out by the plan) and the counters of its split
// tiles, zero on entry and left zero.
struct GemmScratch {
  char* p;
  unsigned* cnt;
};

GemmPlan plan_gemm(int M, const qlin_weights* w, bool fused = false) { return plan_gemm_group(M, &w, 1, fused); }

constexpr int kGroupMaxM = 64;  // token counts a grouped launch takes (decode-sized tiles)

// ---------------------------------------------------------------- GEMM launch
template <int FMT, int BT, int MAXP, int EPI>
qlin_status launch_gemm_t(GemmParams<MAXP>& prm, cudaStream_t stream) {
  using C = GemmCfg<FMT, BT>;
  auto kern = gemm_kernel<FMT, BT, MAXP, EPI>;
  const cudaError_t attr_err = allow_smem<gemm_kernel<FMT, BT, MAXP, EPI>>(C::kSmemBytes);
  if (attr_err != cudaSuccess) return fail(QLIN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(attr_err));
  GemmArgs& args = prm.g;
  // Single-problem launches whose token tiles (up to 64) would be split
  // (decode): cluster split-K when it is expected to beat global-memory
  // stream-K.  Costs in units of one pipeline step, fitted to B200
  // measurements of the 7B decode shapes: a cluster round costs its longest
  // rank range plus the exchange of BT x 128 partials through distributed
  // shared memory (about 0.5 / 2 / 7.5 steps at BT = 16 / 32 / 64);
  // stream-K costs its per-CTA iterations plus the global fixup chain
  // (about 7 / 12 / 28 steps).  QLIN_KNOB_CLUSTER_SIZE forces a size.
  if (MAXP == 1 && C::kCluster && args.split && !cluster_disabled()) {
    const GemmProb& g0 = prm.pr[0];
    const double xchg = BT <= 16 ? 0.5 : (BT <= 32 ? 2.0 : 7.5);
    const double fixup = BT <= 16 ? 7.0 : (BT <= 32 ? 12.0 : 28.0);
    const int forced = forced_cluster_size();
    const long long iters = static_cast<long long>(g0.tiles_n) * g0.tiles_m * g0.T;
    const double streamk_cost = static_cast<double>((iters + args.grid - 1) / args.grid) + fixup;
    const long long tiles = static_cast<long long>(g0.tiles_n) * g0.tiles_m;
    static int max_clusters[9] = {-1, -1, -1, -1, -1, -1, -1, -1, -1};  // per cluster size, this instantiation
    int best_cs = 0, best_ncl = 0;
    double best_cost = streamk_cost;
    // compensation run of the last rank: its steps plus sending a BT x slice
    // fp32 partial (about BT / 32 steps at cs = 4)
    for (int cs = 2; cs <= 8; cs *= 2) {
      int cb[9];
      const double ccost = (g0.T - g0.nk) + (g0.nO > 0 ? BT / 32.0 * 4.0 / cs : 0.0);
      const double span = cluster_bounds(g0.T, g0.nk, cs, ccost, cb);
      if (span < 0) continue;
      if (max_clusters[cs] < 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cs * ((sm_count() + cs - 1) / cs)));
        cfg.blockDim = dim3(C::kThreads);
        cfg.dynamicSmemBytes = C::kSmemBytes;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = static_cast<unsigned>(cs);
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
          cudaGetLastError();
          n = 0;
        }
        max_clusters[cs] = n;
      }
      int ncl = static_cast<int>(max_clusters[cs] < tiles ? max_clusters[cs] : tiles);
      if (ncl * cs > gemm_cta_cap()) ncl = gemm_cta_cap() / cs;
      if (ncl < 1) continue;
      double cost = static_cast<double>((tiles + ncl - 1) / ncl) * (span + xchg);
      if (forced) cost = forced == cs ? -1.0 : 1e30;
      if (cost < best_cost) {
        best_cs = cs;
        best_ncl = ncl;
        best_cost = cost;
      }
    }
    if (best_cs) {
      args.cs = best_cs;
      args.ncl = best_ncl;
      args.grid = best_cs * best_ncl;
      cluster_bounds(g0.T, g0.nk, best_cs,
                     (g0.T - g0.nk) + (g0.nO > 0 ? BT / 32.0 * 4.0 / best_cs : 0.0), args.cb);
    }
  }
  cudaError_t e = launch_kc(kern, dim3(args.grid), dim3(C::kThreads), C::kSmemBytes, stream, args.cs, prm);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "gemm_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

// Grouped launches (MAXP > 1) take decode-sized token tiles only (<= 64).
template <int FMT, int MAXP, int EPI = kEpiPlain>
qlin_status launch_gemm_fmt(int bt, GemmParams<MAXP>& prm, cudaStream_t stream) {
  switch (bt) {
    case 16: return launch_gemm_t<FMT, 16, MAXP, EPI>(prm, stream);
    case 32: return launch_gemm_t<FMT, 32, MAXP, EPI>(prm, stream);
    case 64: return launch_gemm_t<FMT, 64, MAXP, EPI>(prm, stream);
    default:
      if constexpr (MAXP == 1) {
        if (bt == 128) return launch_gemm_t<FMT, 128, 1, EPI>(prm, stream);
        return launch_gemm_t<FMT, 256, 1, EPI>(prm, stream);
      } else {
        return fail(QLIN_ERR_SHAPE, "grouped GEMMs take at most %d tokens", kGroupMaxM);
      }
  }
}

// The same with the epilogue variant chosen at run time (one problem).
template <int FMT>
qlin_status launch_gemm_epi(int epi, int bt, GemmParams<1>& prm, cudaStream_t stream) {
  if (epi == kEpiGated) return launch_gemm_fmt<FMT, 1, kEpiGated>(bt, prm, stream);
  if (epi == kEpiAct) return launch_gemm_fmt<FMT, 1, kEpiAct>(bt, prm, stream);
  return launch_gemm_fmt<FMT, 1>(bt, prm, stream);
}

// ---------------------------------------------------------------- CTA-pair GEMM (many tokens)
template <int FMT>
int pair_max_clusters() {
  static int n = -1;
  static std::once_flag once;
  std::call_once(once, [] {
    if (cudaFuncSetAttribute(gemm_pair_kernel<FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             PairCfg<FMT>::kSmem) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
      return;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * ((sm_count() + 1) / 2)));
    cfg.blockDim = dim3(PairCfg<FMT>::kThreads);
    cfg.dynamicSmemBytes = PairCfg<FMT>::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, gemm_pair_kernel<FMT>, &cfg) != cudaSuccess) {
      cudaGetLastError();
      c = 0;
    }
    n = c;
  });
  return n;
}

// Whether a single-problem launch runs on CTA pairs: 256-token tiles with
// INT8 operands (the INT8 format, or INT4 widened once per call); by default
// whenever the operands allow, even with fewer 256 x 256 pair tiles than
// pairs on the GPU (QLIN_KNOB_PAIR_MMA: 0 never, 1 only from one full wave).
bool use_pair(const GemmPlan& p, const qlin_weights* w) {
  const long long mode = knob(QLIN_KNOB_PAIR_MMA);
  if (mode == 0 || p.nprob != 1 || p.bt != 256) return false;
  if (!(w->fmt == QLIN_W8_PERCHANNEL || p.widen)) return false;
  const int ncl = pair_max_clusters<kFmtW8>();
  if (ncl < 1) return false;
  const long long tiles = static_cast<long long>((p.pr[0].tiles_n + 1) / 2) * p.pr[0].tiles_m;
  return mode == 2 ? tiles >= 1 : tiles >= ncl;
}

// FMT = kFmtW8: INT8 weight rows by TMA from `codes8` (the INT8 format, or
// INT4 widened ahead); kFmtW4PC / kFmtW4G128: the layer's packed INT4 codes,
// converted inside the kernel.
template <int FMT>
qlin_status launch_gemm_pair(const GemmPlan& p, const qlin_weights* w, const int8_t* Xq, const float* a, uint16_t* Y,
                             int32_t* acc_debug, const GemmScratch& gws, const uint8_t* codes8, float cmul, cudaStream_t stream) {
  PairParams prm;
  memset(&prm, 0, sizeof(prm));
  PairArgs& g = prm.g;
  const GemmProb& q = p.pr[0];
  const int M = q.M;
  g.codes = static_cast<const uint8_t*>(w->codes);
  g.rfold = w->fold_ratio;
  g.cscale = w->chan_scale;
  g.cmul = cmul;
  g.a = a;
  g.Y = Y;
  g.acc_debug = acc_debug;
  g.M = M;
  g.N = w->N;
  g.nO = w->n_outlier;
  g.kb = q.kb;
  g.ntn = q.tiles_n;
  g.ncs = q.ncs;
  g.T = q.kb + 2 * q.ncs;
  g.tiles_n2 = (q.tiles_n + 1) / 2;
  g.tiles_m = q.tiles_m;
  g.tiles = g.tiles_n2 * g.tiles_m;
  const double x_bytes = static_cast<double>(M) * w->K;
  const int maxc = pair_max_clusters<FMT>();
  if (maxc < 1) return fail(QLIN_ERR_CUDA, "gemm_pair_kernel: no 2-CTA cluster fits");
  int gm = static_cast<int>(std::lround(std::sqrt(static_cast<double>(maxc) * 256.0 / 256.0)));
  if (x_bytes <= 48.0 * 1024 * 1024) gm = g.tiles_m;
  g.gm = gm < 1 ? 1 : (gm > g.tiles_m ? g.tiles_m : gm);
  if (p.pair_ncl < 1 || p.pair_ncl > maxc) return fail(QLIN_ERR_CUDA, "gemm_pair_kernel: plan of %d pairs, %d fit", p.pair_ncl, maxc);
  g.ncl = p.pair_ncl;
  g.dp = p.pair_dp;
  for (int c = 0; c <= kMaxPairs; ++c) g.bnd[c] = p.pair_bnd[c];
  g.ws_acc = reinterpret_cast<int32_t*>(gws.p + p.pacc_off);
  g.ws_comp = reinterpret_cast<float*>(gws.p + p.pcomp_off);
  g.ws_cnt = gws.cnt;
  qlin_status st = QLIN_OK;
  if (FMT == kFmtW8) {
    st = make_map(&prm.tmA, codes8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                  static_cast<uint64_t>(q.tiles_n) * q.kb * 128, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != QLIN_OK) return st;
  }
  st = make_map(&prm.tmX, Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->K, M, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  if (w->n_outlier > 0) {
    st = make_map(&prm.tmU, gws.p + p.u_off[0], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->n_outlier_pad,
                  2 * static_cast<uint64_t>(M), 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QLIN_OK) return st;
    st = make_map(&prm.tmWo, w->W_Ot, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                  static_cast<uint64_t>(q.tiles_n) * q.ncs * 128, 128, 128, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != QLIN_OK) return st;
  }
  st = make_map(&prm.tmY, Y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->N, M, 128, 256, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != QLIN_OK) return st;
  cudaError_t e = allow_smem<gemm_pair_kernel<FMT>>(PairCfg<FMT>::kSmem);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "gemm_pair_kernel attribute: %s", cudaGetErrorString(e));
  e = launch_kc(gemm_pair_kernel<FMT>, dim3(static_cast<unsigned>(2 * g.ncl)),
                            dim3(PairCfg<FMT>::kThreads), PairCfg<FMT>::kSmem, stream, 2, prm);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "gemm_pair_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

// A fused layer on CTA pairs.  INT8 weight rows from `codes8` (the INT8
// format, or INT4 widened ahead).
template <int EPI, int ACT>
qlin_status launch_fused_t(const GemmPlan& p, const qlin_weights* w, const int8_t* Xq, const float* a, uint16_t* Y,
                           const GemmScratch& gws, const uint8_t* codes8, float cmul, cudaStream_t stream, const EpiArgs& epi) {
  FusedPairParams prm;
  memset(&prm, 0, sizeof(prm));
  FusedPairArgs& g = prm.g;
  const GemmProb& q = p.pr[0];
  const int M = q.M;
  g.cscale = w->chan_scale;
  g.cmul = cmul;
  g.a = a;
  g.M = M;
  g.N = w->N;
  g.nO = w->n_outlier;
  g.kb = q.kb;
  g.ntn = q.tiles_n;
  g.ncs = q.ncs;
  g.tiles_n2 = (q.tiles_n + 1) / 2;
  g.tiles_m = q.tiles_m;
  g.ncl = p.pair_ncl;
  g.whole = p.pair_dp;
  g.units = 2 * g.tiles_n2 * g.tiles_m - g.whole;
  g.epi = epi;
  int gm = static_cast<int>(std::lround(std::sqrt(static_cast<double>(g.ncl))));
  if (static_cast<double>(M) * w->K <= 48.0 * 1024 * 1024) gm = g.tiles_m;
  g.gm = gm < 1 ? 1 : (gm > g.tiles_m ? g.tiles_m : gm);
  qlin_status st = QLIN_OK;
  for (int h = 0; h < 2 && st == QLIN_OK; ++h)
    st = make_map(h ? &prm.tmAh : &prm.tmA, codes8, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                  static_cast<uint64_t>(q.tiles_n) * q.kb * 128, 128, 128 >> h, CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != QLIN_OK) return st;
  st = make_map(&prm.tmX, Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->K, M, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  if (w->n_outlier > 0) {
    st = make_map(&prm.tmU, gws.p + p.u_off[0], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->n_outlier_pad,
                  2 * static_cast<uint64_t>(M), 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QLIN_OK) return st;
    for (int h = 0; h < 2 && st == QLIN_OK; ++h)
      st = make_map(h ? &prm.tmWoh : &prm.tmWo, w->W_Ot, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128,
                    static_cast<uint64_t>(q.tiles_n) * q.ncs * 128, 128, 128 >> h, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (st != QLIN_OK) return st;
  }
  const int F = EPI == kEpiGated ? w->N / 2 : w->N;
  st = make_map(&prm.tmY, Y, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, F, M, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  if (epi.Z) {
    st = make_map(&prm.tmZ, epi.Z, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->N, M, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QLIN_OK) return st;
  }
  if (epi.residual) {
    st = make_map(&prm.tmR, epi.residual, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->N, M, 64, 128,
                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QLIN_OK) return st;
  }
  constexpr auto kern = gemm_fused_kernel<EPI, ACT>;
  cudaError_t e = allow_smem<kern>(FusedPairCfg::kSmem);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "gemm_fused_kernel attribute: %s", cudaGetErrorString(e));
  e = launch_kc(kern, dim3(static_cast<unsigned>(2 * g.ncl)), dim3(FusedPairCfg::kThreads), FusedPairCfg::kSmem, stream,
                2, prm);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "gemm_fused_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

template <int EPI>
qlin_status launch_fused_act(const GemmPlan& p, const qlin_weights* w, const int8_t* Xq, const float* a, uint16_t* Y,
                             const GemmScratch& gws, const uint8_t* codes8, float cmul, cudaStream_t stream, const EpiArgs& epi) {
  switch (epi.act) {
    case kActRelu: return launch_fused_t<EPI, kActRelu>(p, w, Xq, a, Y, gws, codes8, cmul, stream, epi);
    case kActGelu: return launch_fused_t<EPI, kActGelu>(p, w, Xq, a, Y, gws, codes8, cmul, stream, epi);
    case kActGeluTanh: return launch_fused_t<EPI, kActGeluTanh>(p, w, Xq, a, Y, gws, codes8, cmul, stream, epi);
    case kActSilu: return launch_fused_t<EPI, kActSilu>(p, w, Xq, a, Y, gws, codes8, cmul, stream, epi);
    default: return launch_fused_t<EPI, kActNone>(p, w, Xq, a, Y, gws, codes8, cmul, stream, epi);
  }
}

// INT8 operands on CTA pairs, with the epilogue variant chosen at run time.
qlin_status launch_pair_w8(const GemmPlan& p, const qlin_weights* w, const int8_t* Xq, const float* a, uint16_t* Y,
                           int32_t* acc_debug, const GemmScratch& gws, const uint8_t* codes8, float cmul, cudaStream_t stream,
                           const EpiArgs* epi, int variant) {
  if (variant == kEpiGated) return launch_fused_act<kEpiGated>(p, w, Xq, a, Y, gws, codes8, cmul, stream, *epi);
  if (variant == kEpiAct) return launch_fused_act<kEpiAct>(p, w, Xq, a, Y, gws, codes8, cmul, stream, *epi);
  return launch_gemm_pair<kFmtW8>(p, w, Xq, a, Y, acc_debug, gws, codes8, cmul, stream);
}

// One GEMM launch over the problems of a plan.  Per problem q: weights
// ws[q], the INT8 activations Xq[q], token scales a[q], output Y[q] and
// (optional) acc_debug[q]; `gws` is the scratch laid out by the plan (each
// problem's U, then the shared split-K slots and counters).  `epi` and
// `variant`: a fused epilogue (one problem, no acc_debug).
template <int MAXP>
qlin_status launch_gemm_group(const GemmPlan& p, const qlin_weights* const* ws, const int8_t* const* Xq,
                              const float* const* a, uint16_t* const* Y, int32_t* const* acc_debug, const GemmScratch& gws,
                              cudaStream_t stream, const EpiArgs* epi = nullptr, int variant = kEpiPlain) {
  qlin_status st = get_encoder();
  if (st != QLIN_OK) return st;
  static_assert(sizeof(GemmParams<MAXP>) <= 32000, "kernel parameter space");
  GemmParams<MAXP> prm;
  memset(&prm, 0, sizeof(prm));
  GemmArgs& args = prm.g;
  const int M = p.pr[0].M;
  long long iters = 0;
  for (int q = 0; q < p.nprob; ++q) {
    const qlin_weights* w = ws[q];
    GemmProb& g = prm.pr[q];
    g = p.pr[q];
    g.codes = static_cast<const uint8_t*>(w->codes);
    g.rfold = w->fold_ratio;
    g.wot = w->W_Ot;
    g.cscale = w->chan_scale;
    g.a = a[q];
    g.Y = Y[q];
    g.acc_debug = acc_debug ? acc_debug[q] : nullptr;
    g.cmul = 1.f;
    iters += static_cast<long long>(g.tiles_n) * g.tiles_m * g.T;
    st = make_map(&prm.tmX[q], Xq[q], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w->K, M, 128, p.bt,
                  CU_TENSOR_MAP_SWIZZLE_128B);
    if (st != QLIN_OK) return st;
    if (w->n_outlier > 0) {
      st = make_map(&prm.tmU[q], gws.p + p.u_off[q], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, w->n_outlier_pad,
                    2 * static_cast<uint64_t>(M), 64, p.bt, CU_TENSOR_MAP_SWIZZLE_128B);
      if (st != QLIN_OK) return st;
    }
  }
  if (iters >= (1LL << 31)) return fail(QLIN_ERR_SHAPE, "problem too large (%lld tile iterations)", iters);
  args.ws_acc = reinterpret_cast<int32_t*>(gws.p + p.acc_off);
  args.ws_comp = reinterpret_cast<float*>(gws.p + p.comp_off);
  args.ws_cnt = gws.cnt;
  args.nprob = p.nprob;
  args.grid = p.grid;
  args.split = p.split;
  args.total = static_cast<unsigned>(iters);
  args.cs = 1;
  args.ncl = 0;
  args.wdep = p.widen ? 1 : 0;
  if (epi) args.epi = *epi;
  gemm_boundaries(prm.pr, p.nprob, p.grid, p.split, args.bnd);
  const int fmt = ws[0]->fmt;
  if (p.widen && MAXP == 1 && !epi && use_pair(p, ws[0]) && p.pr[0].M <= convert_max_m()) {
    // INT4 on CTA pairs, converted inside the kernel (no widening pass)
    const qlin_weights* w = ws[0];
    const float cm = fmt == QLIN_W4_PERCHANNEL ? 0.0625f : 1.f;
    return fmt == QLIN_W4_PERCHANNEL
               ? launch_gemm_pair<kFmtW4PC>(p, w, Xq[0], a[0], Y[0], acc_debug ? acc_debug[0] : nullptr, gws, nullptr,
                                            cm, stream)
               : launch_gemm_pair<kFmtW4G128>(p, w, Xq[0], a[0], Y[0], acc_debug ? acc_debug[0] : nullptr, gws,
                                              nullptr, cm, stream);
  }
  if (p.widen) {
    const qlin_weights* w = ws[0];
    uint8_t* w8 = reinterpret_cast<uint8_t*>(gws.p + p.w8_off);
    const unsigned nblk = static_cast<unsigned>(p.pr[0].tiles_n) * static_cast<unsigned>(p.pr[0].kb);
    const uint8_t* codes = static_cast<const uint8_t*>(w->codes);
    const uint16_t* rf = reinterpret_cast<const uint16_t*>(w->fold_ratio);
    cudaError_t e = fmt == QLIN_W4_PERCHANNEL
                        ? launch_k(widen_w4_kernel<kFmtW4PC>, dim3(nblk), dim3(256), 0, stream, codes, rf, w->N,
                                   p.pr[0].kb, w8)
                        : launch_k(widen_w4_kernel<kFmtW4G128>, dim3(nblk), dim3(256), 0, stream, codes, rf, w->N,
                                   p.pr[0].kb, w8);
    if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "widen_w4_kernel launch failed: %s", cudaGetErrorString(e));
    prm.pr[0].codes = w8;
    prm.pr[0].cmul = fmt == QLIN_W4_PERCHANNEL ? 0.0625f : 1.f;
    if (MAXP == 1 && use_pair(p, w))
      return launch_pair_w8(p, w, Xq[0], a[0], Y[0], acc_debug ? acc_debug[0] : nullptr, gws, w8, prm.pr[0].cmul, stream,
                            epi, variant);
    if constexpr (MAXP == 1) return launch_gemm_epi<kFmtW8>(variant, p.bt, prm, stream);
    else return launch_gemm_fmt<kFmtW8, MAXP>(p.bt, prm, stream);
  }
  if (MAXP == 1 && fmt == QLIN_W8_PERCHANNEL && use_pair(p, ws[0]))
    return launch_pair_w8(p, ws[0], Xq[0], a[0], Y[0], acc_debug ? acc_debug[0] : nullptr, gws,
                          static_cast<const uint8_t*>(ws[0]->codes), 1.f, stream, epi, variant);
  if constexpr (MAXP == 1) {
    if (epi) {
      switch (fmt) {
        case QLIN_W4_PERCHANNEL: return launch_gemm_epi<kFmtW4PC>(variant, p.bt, prm, stream);
        case QLIN_W4_G128: return launch_gemm_epi<kFmtW4G128>(variant, p.bt, prm, stream);
        default: return launch_gemm_epi<kFmtW8>(variant, p.bt, prm, stream);
      }
    }
  }
  switch (fmt) {
    case QLIN_W4_PERCHANNEL: return launch_gemm_fmt<kFmtW4PC, MAXP>(p.bt, prm, stream);
    case QLIN_W4_G128: return launch_gemm_fmt<kFmtW4G128, MAXP>(p.bt, prm, stream);
    default: return launch_gemm_fmt<kFmtW8, MAXP>(p.bt, prm, stream);
  }
}

// Single-problem GEMM launch.
qlin_status launch_gemm(const qlin_weights* w, const int8_t* Xq, const float* a, int M, uint16_t* Y,
                        int32_t* acc_debug, const GemmScratch& gws, cudaStream_t stream) {
  const GemmPlan p = plan_gemm(M, w);
  return launch_gemm_group<1>(p, &w, &Xq, &a, &Y, acc_debug ? &acc_debug : nullptr, gws, stream);
}

// Single-problem GEMM launch with a fused epilogue.
qlin_status launch_gemm_fused(const GemmPlan& p, const qlin_weights* w, const int8_t* Xq, const float* a, uint16_t* Y,
                              const GemmScratch& gws, cudaStream_t stream, const EpiArgs& epi, int variant) {
  return launch_gemm_group<1>(p, &w, &Xq, &a, &Y, nullptr, gws, stream, &epi, variant);
}

// ---------------------------------------------------------------- act quant
// Up to this many tokens the momentum update runs inside the quantization
// kernel (every CTA gathers all rows' outlier values); above it a separate
// column-max kernel gathers them once (QLIN_KNOB_FUSED_MOMENTUM_MAX_M).
int fused_momentum_max_m() { return static_cast<int>(knob(QLIN_KNOB_FUSED_MOMENTUM_MAX_M)); }

constexpr int kQuantSmemMax = 232448 - 1024;  // 227 KB per CTA, less room for the kernel's static shared memory

size_t act_ws_bytes(const qlin_weights* w) { return w->n_outlier > 0 ? sizeof(WorkspaceHead) : 0; }

// Activations of one quantization problem (outputs and scratch per problem).
struct QuantIO {
  const uint16_t* X;
  float* s;
  int8_t* Xq;
  float* a;
  int8_t* XqO;
  uint16_t* U;   // compensation operand (qlin_forward), or null
  unsigned* cmax;     // outlier column maxima and completion counter (update only):
  unsigned* counter;  // zero on entry, left zero
};

template <int T, int VPT, bool FUSED, int MAXP>
qlin_status launch_quant_v(const QuantGroup<MAXP>& qg, int rows, size_t smem, cudaStream_t stream) {
  constexpr auto kern = quant_kernel<T, VPT, FUSED, MAXP>;
  const cudaError_t attr = allow_smem<kern>(kQuantSmemMax);
  if (attr != cudaSuccess) return fail(QLIN_ERR_CUDA, "quant_kernel attribute: %s", cudaGetErrorString(attr));
  cudaError_t e = launch_k(kern, dim3(rows), dim3(T), smem, stream, qg);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "quant_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

// A row costs a chain of loads and barriers, so calls with many more rows than
// CTAs of 512 threads fit on the GPU at once (four an SM) take a row with fewer
// threads and have more rows under way: 4096 inputs, 41 of them outliers, 8192
// rows in 21 instead of 38 us, 1024 inputs in 11 instead of 28; at 1000 rows
// of 4096 inputs 512 threads are even.
template <bool FUSED, int MAXP>
qlin_status launch_quant_f(const QuantGroup<MAXP>& qg, int rows, int vpt, size_t smem, cudaStream_t stream) {
  if constexpr (!FUSED && MAXP == 1) {
    const int nvec = qg.pr[0].K / 8, few = 4 * sm_count();
    if ((nvec <= 128 && rows > few) || (nvec <= 512 && rows > 2 * few))
      return launch_quant_v<128, 4, FUSED, MAXP>(qg, rows, smem, stream);
    if (nvec <= 1024 && rows > 2 * few) return launch_quant_v<256, 4, FUSED, MAXP>(qg, rows, smem, stream);
    if (nvec <= 2048 && rows > 2 * few) return launch_quant_v<256, 8, FUSED, MAXP>(qg, rows, smem, stream);
  }
  if (vpt <= 1) return launch_quant_v<512, 1, FUSED, MAXP>(qg, rows, smem, stream);
  if (vpt <= 2) return launch_quant_v<512, 2, FUSED, MAXP>(qg, rows, smem, stream);
  if (vpt <= 4) return launch_quant_v<512, 4, FUSED, MAXP>(qg, rows, smem, stream);
  if (vpt <= 8) return launch_quant_v<512, 8, FUSED, MAXP>(qg, rows, smem, stream);
  return launch_quant_v<512, 16, FUSED, MAXP>(qg, rows, smem, stream);
}

// Stage 1 for one problem or a group (same M): the momentum update (fused
// into the quantization kernel up to the fused-momentum token count, else a
// column-max kernel per problem first), then one quantization launch with a
// CTA per token row of every problem.
template <int MAXP>
qlin_status launch_quant_group(const qlin_weights* const* ws, const QuantIO* io, int n, int M, float gamma,
                               int update, cudaStream_t stream) {
  if (M == 0) return QLIN_OK;
  QuantGroup<MAXP> qg;
  memset(&qg, 0, sizeof(qg));
  qg.gamma = gamma;
  qg.nprob = n;
  bool any_update = false;
  int maxK = 0;
  size_t smem = 0;
  for (int q = 0; q < n; ++q) {
    const qlin_weights* w = ws[q];
    const int K = w->K, nO = w->n_outlier;
    QuantProb& p = qg.pr[q];
    p.X = io[q].X;
    p.O = static_cast<const int32_t*>(w->outlier_idx);
    p.s = io[q].s;
    p.Xq = io[q].Xq;
    p.a = io[q].a;
    p.XqO = io[q].XqO;
    p.U = io[q].U;
    p.wmaxO = w->wmax_O;
    p.counter = io[q].counter;
    p.K = K;
    p.nO = nO;
    p.nOp = w->n_outlier_pad;
    p.M = M;
    p.row0 = q * M;
    any_update = any_update || (update && nO > 0);
    if (K > maxK) maxK = K;
    const size_t sm = size_t(K) * 2 + size_t(nO) * 16;
    if (sm > smem) smem = sm;
  }
  if (smem > size_t(kQuantSmemMax))
    return fail(QLIN_ERR_SHAPE, "K=%d with its outliers needs %zu bytes of shared memory", maxK, smem);
  const int nvec = maxK / 8;
  const int vpt = (nvec + kQuantThreads - 1) / kQuantThreads;
  if (vpt > 16) return fail(QLIN_ERR_SHAPE, "K=%d too large for the quantization kernel", maxK);
  const bool fused = any_update && M <= fused_momentum_max_m();
  if (any_update && !fused) {
    for (int q = 0; q < n; ++q) {
      const qlin_weights* w = ws[q];
      const int nO = w->n_outlier;
      if (nO == 0) continue;
      const int grid = colmax_grid(M);
      cudaError_t e = launch_k(colmax_kernel, dim3(grid), dim3(256), size_t(nO) * 8, stream, io[q].X, M, w->K,
                               static_cast<const int32_t*>(w->outlier_idx), nO, io[q].cmax, 1,
                               static_cast<const float*>(w->wmax_O), io[q].s, gamma, io[q].counter);
      if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "colmax_kernel launch failed: %s", cudaGetErrorString(e));
    }
  }
  const int rows = n * M;
  return fused ? launch_quant_f<true, MAXP>(qg, rows, vpt, smem, stream)
               : launch_quant_f<false, MAXP>(qg, rows, vpt, smem, stream);
}

qlin_status launch_quant(const uint16_t* X, int M, const qlin_weights* w, float* s, float gamma, int update,
                         int8_t* Xq, float* a, int8_t* XqO, uint16_t* U, unsigned* cmax, unsigned* counter, cudaStream_t stream) {
  const QuantIO io{X, s, Xq, a, XqO, U, cmax, counter};
  return launch_quant_group<1>(&w, &io, 1, M, gamma, update, stream);
}

size_t gemm_ws_bytes(int M, const qlin_weights* w, bool fused = false) {
  return M > 0 ? plan_gemm(M, w, fused).total : 0;
}

struct FwdLayout {
  size_t xq, a, xqo, gemm, total;
};

FwdLayout forward_layout(int M, const qlin_weights* w, bool fused = false) {
  FwdLayout L{};
  size_t off = sizeof(WorkspaceHead);
  L.xq = off; off = round_up(off + size_t(M) * w->K, kAlign);
  L.a = off; off = round_up(off + size_t(M) * 4, kAlign);
  L.xqo = off; off = round_up(off + size_t(M) * w->n_outlier, kAlign);
  L.gemm = off; off = round_up(off + gemm_ws_bytes(M, w, fused), kAlign);
  L.total = off;
  return L;
}

// Workspace of a grouped forward: the head, per problem Xq, a and XqO, then
// the GEMM launch's scratch (every problem's U and the shared split-K slots).
struct GroupLayout {
  size_t xq[kMaxProbs], a[kMaxProbs], xqo[kMaxProbs];
  size_t gemm, total;
  GemmPlan plan;
};

GroupLayout group_layout(int M, const qlin_weights* const* ws, int n) {
  GroupLayout L{};
  size_t off = sizeof(WorkspaceHead);
  for (int q = 0; q < n; ++q) {
    const qlin_weights* w = ws[q];
    L.xq[q] = off; off = round_up(off + size_t(M) * w->K, kAlign);
    L.a[q] = off; off = round_up(off + size_t(M) * 4, kAlign);
    L.xqo[q] = off; off = round_up(off + size_t(M) * w->n_outlier, kAlign);
  }
  L.plan = plan_gemm_group(M > 0 ? M : 1, ws, n);
  L.gemm = off;
  off = round_up(off + (M > 0 ? L.plan.total : 0), kAlign);
  L.total = off;
  return L;
}

qlin_status check_group(int32_t count, const qlin_weights* const* w, int32_t M) {
  if (count < 1 || count > kMaxProbs) return fail(QLIN_ERR_SHAPE, "count=%d must be in [1, %d]", count, kMaxProbs);
  if (!w) return fail(QLIN_ERR_ARG, "weights array is NULL");
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (M > kGroupMaxM) return fail(QLIN_ERR_SHAPE, "M=%d: grouped forwards take at most %d tokens", M, kGroupMaxM);
  for (int q = 0; q < count; ++q) {
    qlin_status st = check_weights(w[q]);
    if (st != QLIN_OK) return fail(st, "problem %d: %s", q, t_last_error);
    if (w[q]->fmt != w[0]->fmt) return fail(QLIN_ERR_ARG, "problem %d: every problem must have the same format", q);
  }
  return QLIN_OK;
}

}  // namespace

// ---------------------------------------------------------------- allocation-free quantization
// Fixed scratch for qlin_quant_act_noalloc: the outlier column maxima and the
// completion counter of the momentum update.  It is a file-scope device
// array, so every GPU that loads this library holds it (4.25 KiB: 1024 + 64
// words) until the process exits, and every call on a device shares the same
// copy.
#define QLIN_NOALLOC_MAX_OUTLIERS 1024
static __device__ __align__(256) unsigned g_noalloc_scratch[QLIN_NOALLOC_MAX_OUTLIERS + 64];

namespace {

constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
unsigned* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the scratch on the current device.  In host code the
// symbol names a host-side shadow, not device memory, so the address is
// looked up once per device (with that device current) and cached.
qlin_status noalloc_scratch(unsigned** out) {
  int dev = -1;
  QLIN_CUDA_TRY(cudaGetDevice(&dev));
  if (dev < 0 || dev >= kMaxDevices) return fail(QLIN_ERR_CUDA, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (!g_noalloc_ptr[dev]) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess || !p)
      return fail(QLIN_ERR_CUDA, "cudaGetSymbolAddress(scratch) failed: %s", cudaGetErrorString(e));
    g_noalloc_ptr[dev] = static_cast<unsigned*>(p);
  }
  *out = g_noalloc_ptr[dev];
  return QLIN_OK;
}

// ---------------------------------------------------------------- backward
// Work plan of the input gradient: whole 256 x 256 tiles fill complete
// waves of one CTA per SM; when the grid is under two waves, the tiles of
// the ragged last wave are split into tsplit ranges of the channel steps (at
// most 8, at most one range per step) so that wave has as many CTAs as SMs,
// and their fp32 partials go through the workspace.  Without a workspace
// every tile is whole.
struct BwdPlan {
  int ntk, tiles, full, tsplit;
  size_t part_off, bytes;
};

BwdPlan plan_backward(int M, const qlin_weights* w, bool split) {
  BwdPlan p{};
  p.ntk = (w->K + 255) / 256;
  p.tiles = p.ntk * ((M + 255) / 256);
  p.full = p.tiles;
  p.tsplit = 1;
  const int sms = sm_count();
  const int nsteps = (w->N + 63) / 64;
  const int tail = p.tiles % sms;
  // only below two waves: with more, CTAs of different lengths already
  // interleave across the wave boundaries and the partials cost more than
  // the idle SMs of the last wave (measured on 3.5-wave grids)
  if (split && tail > 0 && tail <= kHeadCounters && p.tiles < 2 * sms) {
    int S = sms / tail;
    if (S > 8) S = 8;
    if (S > nsteps) S = nsteps;
    if (S >= 2) {
      p.full = p.tiles - tail;
      p.tsplit = S;
    }
  }
  const int ntail = p.tiles - p.full;
  p.part_off = sizeof(WorkspaceHead);
  p.bytes = ntail ? round_up(p.part_off + size_t(ntail) * (p.tsplit - 1) * 65536 * 4, kAlign) : 0;
  return p;
}

template <int FMT>
qlin_status launch_backward_t(const CUtensorMap& tm, const BwdArgs& args, cudaStream_t stream) {
  using C = BwdCfg<FMT>;
  auto kern = backward_dx_kernel<FMT>;
  static std::once_flag attr_once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(attr_once, [&] {
    attr_err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (attr_err != cudaSuccess) return fail(QLIN_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(attr_err));
  const dim3 grid(static_cast<unsigned>(args.full + (args.ntk * ((args.M + 255) / 256) - args.full) * args.tsplit));
  cudaError_t e = launch_k(kern, grid, dim3(C::kThreads), C::kSmemBytes, stream, tm, args);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "backward_dx_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

// ---------------------------------------------------------------- packing
// Quantize and pack from one weight source (checked by the caller).
template <typename Src>
qlin_status pack_from(const Src src, const int32_t* O_host, const qlin_weights* w, cudaStream_t stream) {
  const int K = w->K, N = w->N, nO = w->n_outlier;
  if (nO > 0) {
    if (!O_host) return fail(QLIN_ERR_ARG, "O_host is NULL with n_outlier=%d", nO);
    for (int i = 0; i < nO; ++i) {
      if (O_host[i] < 0 || O_host[i] >= K) return fail(QLIN_ERR_ARG, "O[%d]=%d outside [0, K)", i, O_host[i]);
      if (i > 0 && O_host[i] <= O_host[i - 1]) return fail(QLIN_ERR_ARG, "O is not strictly increasing at %d", i);
    }
  }
  const int threads = 128;
  const int blocks = (N + threads - 1) / threads;
  uint8_t* codes = static_cast<uint8_t*>(w->codes);
  const Layout L = weights_layout(K, N, w->fmt, nO);
  QLIN_CUDA_TRY(cudaMemsetAsync(codes, 0, L.chan - L.codes, stream));  // tile padding is zero
  switch (w->fmt) {
    case QLIN_W4_PERCHANNEL:
      pack_per_channel_kernel<7, true, Src><<<blocks, threads, 0, stream>>>(src, K, N, codes, w->chan_scale);
      break;
    case QLIN_W8_PERCHANNEL:
      pack_per_channel_kernel<127, false, Src><<<blocks, threads, 0, stream>>>(src, K, N, codes, w->chan_scale);
      break;
    default:
      pack_group_kernel<128, Src><<<blocks, threads, 0, stream>>>(src, K, N, codes, w->chan_scale, w->group_scale,
                                                             w->fold_ratio);
  }
  QLIN_LAUNCH_CHECK("pack kernel");
  if (nO > 0) {
    QLIN_CUDA_TRY(cudaMemcpyAsync(w->outlier_idx, O_host, size_t(nO) * 4, cudaMemcpyHostToDevice, stream));
    QLIN_CUDA_TRY(cudaMemsetAsync(w->W_Ot, 0, L.wmax - L.wot, stream));
    pack_outliers_kernel<Src><<<nO, 256, 0, stream>>>(src, N, w->outlier_idx, nO, w->W_Ot, w->wmax_O);
    QLIN_LAUNCH_CHECK("pack_outliers_kernel");
  }
  return QLIN_OK;
}

// ---------------------------------------------------------------- fused layers and norms
qlin_status check_act(int32_t act) {
  if (act < QLIN_ACT_NONE || act > QLIN_ACT_SILU) return fail(QLIN_ERR_ARG, "unknown activation %d", act);
  return QLIN_OK;
}

qlin_status forward_fused(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma, int32_t update,
                          const EpiArgs& epi, int variant, uint16_t* Y, void* workspace, size_t ws_bytes,
                          cudaStream_t stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  st = check_act(epi.act);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  if (M == 0) return QLIN_OK;
  const int nO = w->n_outlier;
  if (!X || !Y) return fail(QLIN_ERR_ARG, "X/Y is NULL");
  if (nO > 0 && !s) return fail(QLIN_ERR_ARG, "s is NULL with n_outlier=%d", nO);
  if (epi.Z && epi.Z == Y) return fail(QLIN_ERR_ARG, "Z and Y are the same buffer");
  if (epi.Z && epi.Z == epi.residual) return fail(QLIN_ERR_ARG, "Z and residual are the same buffer");
  if (!aligned16(X) || !aligned16(Y) || (s && !aligned16(s)) || (epi.bias && !aligned16(epi.bias)) ||
      (epi.residual && !aligned16(epi.residual)) || (epi.Z && !aligned16(epi.Z)))
    return fail(QLIN_ERR_ALIGN, "X/Y/s/bias/residual/Z is not 16-byte aligned");
  const FwdLayout L = forward_layout(M, w, true);
  if (ws_bytes < L.total || !workspace) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + L.xq);
  float* a = reinterpret_cast<float*>(ws + L.a);
  int8_t* XqO = nO > 0 ? reinterpret_cast<int8_t*>(ws + L.xqo) : nullptr;
  WorkspaceHead* head = head_of(workspace);
  const GemmScratch gws{ws + L.gemm, head->cnt};
  const GemmPlan p = plan_gemm(M, w, true);
  uint16_t* U = nO > 0 ? reinterpret_cast<uint16_t*>(gws.p + p.u_off[0]) : nullptr;
  st = launch_quant(X, M, w, s, gamma, update, Xq, a, XqO, U, head->cmax, head->momentum, stream);
  if (st != QLIN_OK) return st;
  return launch_gemm_fused(p, w, Xq, a, Y, gws, stream, epi, variant);
}

// Row groups of a column-sum launch over M rows of `nv` 8-element vectors
// (128 per CTA): about four CTAs per SM, at least eight rows each.
int column_groups(int M, int nv) {
  const int gx = (nv + 127) / 128;
  const int want = (4 * sm_count() + gx - 1) / gx;
  const int most = (M - 1) / 8 + 1;
  const int G = want < most ? want : most;
  return G < 1 ? 1 : (G > 65535 ? 65535 : G);
}

// Partial column sums [G][K] (twice that, dgamma then dbeta, for a norm) to
// their totals.
template <int W>
qlin_status launch_column_sum(const float* part, int G, int K, float* out0, float* out1, cudaStream_t stream) {
  cudaError_t e = launch_k(column_sum_kernel<W>, dim3((K + 31) / 32, out1 ? 2 : 1), dim3(32 * W), 0, stream, part, G, K,
                           out0, out1);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "column_sum_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

// Work split of the fused layers' input gradient: 256 x 256 tiles on CTA
// pairs, their reduction cut into S ranges when that shortens the longest
// pair's work: a unit costs its steps (about 0.28 us each) and some eight
// more for its pipeline's ends, a split the traffic of its partial sums.
struct DxPlan {
  int tiles_k, tiles_m, S, units, ncl, nst, gm;
  int two;  // dZ in two fp16 terms: both fit in one tile's rows
};

int dx_max_clusters() {
  static int n = -1;
  static std::once_flag once;
  std::call_once(once, [] {
    n = 0;
    if (cudaFuncSetAttribute(dx_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, DxCfg::kSmem) != cudaSuccess) {
      cudaGetLastError();
      return;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * ((sm_count() + 1) / 2)));
    cfg.blockDim = dim3(DxCfg::kThreads);
    cfg.dynamicSmemBytes = DxCfg::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, dx_pair_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      c = 0;
    }
    n = c;
  });
  return n;
}

DxPlan plan_dx(int M, const qlin_weights* w) {
  DxPlan p{};
  const int pairs = dx_max_clusters() > 0 ? dx_max_clusters() : 1;
  p.two = M <= 128 ? 1 : 0;
  p.tiles_k = (w->K + 255) / 256;
  p.tiles_m = (M + 255) / 256;
  p.nst = (w->N + 63) / 64;
  const long long tiles = static_cast<long long>(p.tiles_k) * p.tiles_m;
  double best = 0.0;
  for (int S = 1; S <= 16 && S <= p.nst; ++S) {
    const double waves = static_cast<double>((tiles * S + pairs - 1) / pairs);
    const double traffic = S > 1 ? 8.0 * S * M * w->K / 1.7e6 + 20.0 : 0.0;  // bytes over about 6 TB/s and a launch, in steps
    const double cost = waves * ((p.nst + S - 1) / S + 8.0) + traffic;
    if (S == 1 || cost < best) {
      best = cost;
      p.S = S;
    }
  }
  const long long units = tiles * p.S;
  p.units = static_cast<int>(units);
  p.ncl = static_cast<int>(units < pairs ? units : pairs);
  p.gm = p.tiles_m < 9 ? p.tiles_m : 9;
  return p;
}

constexpr int kRingRoom = 220 * 1024;  // of an SM's shared memory, for every ring on it

// A row ring's shape: threads, vectors per thread, rows per group, stages and
// persistent CTAs per SM (0 where the ring does not fit).
struct RingPlan {
  int threads, vpt, rows, ctas, stages;
  size_t smem;
};

// Threads that own `vpt` of nv vectors each, in whole warps.
int ring_threads(int nv, int vpt) { return ((nv + vpt - 1) / vpt + 31) / 32 * 32; }

int ring_ctas(const RingPlan& p, int threads_per_sm) {
  const int fit = static_cast<int>(kRingRoom / p.smem);
  int most = threads_per_sm / p.threads;
  if (most > 16) most = 16;  // more would only lengthen the sums over the CTAs
  return fit < most ? fit : most;
}

// Norms over `arrays` arrays of M rows.  A thread has about 32 values of a
// row in hand (backward: 16 of two rows, whose column sums it keeps): with
// fewer, what a row costs beside its values -- waits, reductions, addresses --
// outweighs them.  Short rows are taken four or two at a time.
RingPlan norm_ring_plan(int M, int K, int arrays, bool backward) {
  RingPlan p{};
  const int nv = K / 8;
  if (nv > 2048) return p;
  p.vpt = nv <= 32 ? 1 : (nv <= 64 || (backward && nv <= 1024) ? 2 : 4);
  p.rows = 4 / p.vpt;
  p.threads = ring_threads(nv, p.vpt);
  for (;; p.rows = 1) {
    const size_t stage = size_t(p.rows) * arrays * K * 2;
    p.stages = kRingStages;
    p.smem = p.stages * stage;
    p.ctas = ring_ctas(p, 512);
    RingPlan two = p;
    two.stages = 2;
    two.smem = two.stages * stage;
    two.ctas = ring_ctas(two, 512);
    if (two.ctas > p.ctas) p = two;
    // one row at a time where groups would leave SMs idle or do not fit
    if (p.rows == 1 || (p.ctas > 0 && (M - 1) / p.rows + 1 >= sm_count())) break;
  }
  return p;
}

template <auto Kern, typename Args>
cudaError_t launch_ring(const RingPlan& p, unsigned grid, cudaStream_t stream, const Args& g) {
  cudaError_t e = allow_smem<Kern>(kRingRoom);
  if (e != cudaSuccess) return e;
  return launch_k(Kern, dim3(grid), dim3(p.threads), p.smem, stream, g);
}

unsigned ring_grid(const RingPlan& p, int M) {
  if (p.ctas == 0 || M < 1) return 0;
  const int groups = (M - 1) / p.rows + 1, most = sm_count() * p.ctas;
  return static_cast<unsigned>(groups < most ? groups : most);
}

// The ring of the activation's backward pass: two or three stages of a Z and
// a dY row (ctas = 0 where two do not fit, or a thread would own more than
// six vectors).
RingPlan dact_ring_plan(int N, bool gated, bool has_z) {
  RingPlan p{};
  const int nv = N / 8;
  const size_t stage = size_t(N) * ((has_z ? 2 : 0) + (gated ? 1 : 2));
  const size_t room = kRingRoom;
  p.vpt = (nv + kDactRingThreads - 1) / kDactRingThreads;
  p.threads = ring_threads(nv, p.vpt);
  p.rows = 1;
  p.stages = static_cast<int>(room / stage < size_t(kRingStages) ? room / stage : kRingStages);
  if (p.stages < 2 || p.vpt > 6) return p;
  p.smem = stage * p.stages;
  p.ctas = ring_ctas(p, kDactRingThreads);
  return p;
}

// Workspace of a fused layer's backward pass: the widened weight operand, the
// scaled dZ, the rows' factors, the partial sums of split tiles and of the
// bias's gradient.
struct FusedBwdLayout {
  size_t wide, dz, rows, dxpart, part, total;
  DxPlan dx;
  int G;
};
FusedBwdLayout fused_bwd_layout(int M, const qlin_weights* w) {
  FusedBwdLayout L{};
  L.dx = plan_dx(M, w);
  size_t off = sizeof(WorkspaceHead);  // not used, left as it is
  L.wide = off; off = round_up(off + size_t((w->K + 127) / 128) * L.dx.nst * 16384, kAlign);
  L.dz = off; off = round_up(off + size_t(L.dx.two ? 2 : 1) * M * w->N * 2, kAlign);
  L.rows = off; off = round_up(off + size_t(M) * 4, kAlign);
  L.dxpart = off; off = round_up(off + (L.dx.S > 1 ? size_t(L.dx.S) * M * w->K * 4 : 0), kAlign);
  // partial rows of the bias's gradient: one per CTA of a ring kernel (whose
  // shape depends on what it reads), else one per row group
  L.G = column_groups(M, w->N / 8);
  int most = L.G;
  for (int v = 0; v < 3; ++v) {
    const int n = static_cast<int>(ring_grid(dact_ring_plan(w->N, v == 2, v >= 1), M));
    if (n > most) most = n;
  }
  L.part = off; off = round_up(off + size_t(most) * w->N * 4, kAlign);
  L.total = off;
  return L;
}

template <bool GATED, bool ACC>
cudaError_t launch_dact_ring(const RingPlan& p, unsigned grid, const DactArgs& g, cudaStream_t stream) {
  switch (p.vpt) {
    case 1: return launch_ring<dact_ring_kernel<GATED, 1, ACC>>(p, grid, stream, g);
    case 2: return launch_ring<dact_ring_kernel<GATED, 2, ACC>>(p, grid, stream, g);
    case 3: return launch_ring<dact_ring_kernel<GATED, 3, ACC>>(p, grid, stream, g);
    case 4: return launch_ring<dact_ring_kernel<GATED, 4, ACC>>(p, grid, stream, g);
    case 5: return launch_ring<dact_ring_kernel<GATED, 5, ACC>>(p, grid, stream, g);
    default: return launch_ring<dact_ring_kernel<GATED, 6, ACC>>(p, grid, stream, g);
  }
}

template <int FMT>
cudaError_t launch_dx_widen(const DxWidenArgs& a, cudaStream_t stream) {
  const unsigned sums = a.dbias ? static_cast<unsigned>((a.N + 31) / 32) : 0u;
  return launch_k(dx_widen_kernel<FMT>, dim3(static_cast<unsigned>(a.blocks) + sums), dim3(256), 0, stream, a);
}

// dX from the scaled dZ and the widened operand.
qlin_status launch_dx(const qlin_weights* w, int M, const FusedBwdLayout& L, char* ws, uint16_t* dX, cudaStream_t stream) {
  qlin_status st = get_encoder();
  if (st != QLIN_OK) return st;
  if (dx_max_clusters() < 1) return fail(QLIN_ERR_CUDA, "dx_pair_kernel: no 2-CTA cluster fits");
  const DxPlan& p = L.dx;
  const uint64_t kb = (w->K + 127) / 128;
  DxParams prm;
  memset(&prm, 0, sizeof(prm));
  DxArgs& g = prm.g;
  g.rowscale = reinterpret_cast<const float*>(ws + L.rows);
  g.dX = dX;
  g.part = reinterpret_cast<float*>(ws + L.dxpart);
  g.M = M;
  g.K = w->K;
  g.nst = p.nst;
  g.tiles_k = p.tiles_k;
  g.tiles_m = p.tiles_m;
  g.S = p.S;
  g.units = p.units;
  g.ncl = p.ncl;
  g.gm = p.gm;
  g.two = p.two;
  st = make_map(&prm.tmA, ws + L.dz, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w->N, static_cast<uint64_t>(p.two ? 2 : 1) * M, 64,
                128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  st = make_map(&prm.tmB, ws + L.wide, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, 128, kb * p.nst * 128, 128, 128,
                CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st != QLIN_OK) return st;
  st = make_map(&prm.tmX, dX, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w->K, M, 64, p.two ? 64 : 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  cudaError_t e = allow_smem<dx_pair_kernel>(DxCfg::kSmem);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dx_pair_kernel attribute: %s", cudaGetErrorString(e));
  e = launch_kc(dx_pair_kernel, dim3(static_cast<unsigned>(2 * p.ncl)), dim3(DxCfg::kThreads), DxCfg::kSmem,
                            stream, 2, prm);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dx_pair_kernel launch failed: %s", cudaGetErrorString(e));
  if (p.S > 1) {
    const size_t blocks = (size_t(M) * w->K / 8 + 255) / 256;
    e = launch_k(dx_reduce_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, g);
    if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dx_reduce_kernel launch failed: %s", cudaGetErrorString(e));
  }
  return QLIN_OK;
}

template <bool GATED>
qlin_status backward_fused(const qlin_weights* w, const uint16_t* dY, const uint16_t* Z, int32_t act, int32_t M,
                           const float* s, uint16_t* dX, float* dbias, void* workspace, size_t ws_bytes,
                           cudaStream_t stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  st = check_act(act);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (M > 65535 * 128) return fail(QLIN_ERR_SHAPE, "M=%d exceeds %d", M, 65535 * 128);
  if (dbias && !aligned16(dbias)) return fail(QLIN_ERR_ALIGN, "dbias is not 16-byte aligned");
  if (M == 0) {  // no rows: the bias's gradient is a sum over nothing
    if (dbias) QLIN_CUDA_TRY(cudaMemsetAsync(dbias, 0, size_t(w->N) * 4, stream));
    return QLIN_OK;
  }
  const int nO = w->n_outlier;
  const bool needs_z = GATED || act != QLIN_ACT_NONE;
  if (size_t((w->K + 127) / 128) * ((w->N + 63) / 64) * 128 >= size_t(1) << 31)
    return fail(QLIN_ERR_SHAPE, "K=%d N=%d: the widened weights exceed 2^31 rows of 128 bytes", w->K, w->N);
  if (!dX && !dbias) return fail(QLIN_ERR_ARG, "dX and dbias are both NULL");
  if (!dY || (needs_z && !Z)) return fail(QLIN_ERR_ARG, "dY/Z is NULL");
  if (nO > 0 && dX && !s) return fail(QLIN_ERR_ARG, "s is NULL with n_outlier=%d", nO);
  if (!aligned16(dY) || (Z && !aligned16(Z)) || (dX && !aligned16(dX)) || (s && !aligned16(s)))
    return fail(QLIN_ERR_ALIGN, "dY/Z/dX/s is not 16-byte aligned");
  const FusedBwdLayout L = fused_bwd_layout(M, w);
  if (ws_bytes < L.total || !workspace) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  DactArgs g{};
  g.dY = dY;
  g.Z = Z;
  g.cscale = w->chan_scale;
  g.dZ = reinterpret_cast<uint16_t*>(ws + L.dz);
  g.two = L.dx.two;
  g.rowscale = reinterpret_cast<float*>(ws + L.rows);
  g.part = reinterpret_cast<float*>(ws + L.part);
  g.cmul = w->fmt == QLIN_W4_PERCHANNEL ? 0.0625f : 1.f;
  g.M = M;
  g.N = w->N;
  g.act = act;
  g.G = L.G;
  const RingPlan ring = dact_ring_plan(w->N, GATED, needs_z);
  cudaError_t e;
  int parts = L.G;  // partial rows of the bias's gradient
  if (ring.ctas > 0) {
    const unsigned grid = ring_grid(ring, M);
    g.stages = ring.stages;
    if (!dX) g.dZ = nullptr;
    e = dbias ? launch_dact_ring<GATED, true>(ring, grid, g, stream) : launch_dact_ring<GATED, false>(ring, grid, g, stream);
    if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dact_ring_kernel launch failed: %s", cudaGetErrorString(e));
    parts = static_cast<int>(grid);
  } else {
    if (dbias) {
      e = launch_k(dact_columns_kernel<GATED>, dim3((w->N / 8 + 127) / 128, L.G), dim3(128), 0, stream, g);
      if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dact_columns_kernel launch failed: %s", cudaGetErrorString(e));
    }
    if (dX) {
      e = launch_k(dact_rows_kernel<GATED>, dim3(static_cast<unsigned>(M)), dim3(kDactThreads), 0, stream, g);
      if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dact_rows_kernel launch failed: %s", cudaGetErrorString(e));
    }
  }
  // eight warps: the order in which the widening kernel adds them
  if (!dX) return launch_column_sum<8>(g.part, parts, w->N, dbias, nullptr, stream);
  DxWidenArgs a{};
  a.codes = static_cast<const uint8_t*>(w->codes);
  a.rfold = w->fold_ratio;
  a.wot = w->W_Ot;
  a.cscale = w->chan_scale;
  a.oidx = w->outlier_idx;
  a.s = s;
  a.out = reinterpret_cast<uint8_t*>(ws + L.wide);
  a.N = w->N;
  a.nO = nO;
  a.kb = (w->K + 127) / 128;
  a.nst = L.dx.nst;
  a.nib = (nO + 63) / 64;
  a.part = g.part;
  a.dbias = dbias;
  a.blocks = (w->N + 127) / 128 * a.kb;
  a.G = parts;
  e = w->fmt == QLIN_W4_PERCHANNEL ? launch_dx_widen<kFmtW4PC>(a, stream)
      : w->fmt == QLIN_W4_G128     ? launch_dx_widen<kFmtW4G128>(a, stream)
                                   : launch_dx_widen<kFmtW8>(a, stream);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "dx_widen_kernel launch failed: %s", cudaGetErrorString(e));
  return launch_dx(w, M, L, ws, dX, stream);
}

qlin_status check_norm(int32_t M, int32_t K, int32_t kind) {
  if (kind != QLIN_NORM_LAYER && kind != QLIN_NORM_RMS) return fail(QLIN_ERR_ARG, "unknown norm kind %d", kind);
  if (M < 0 || K <= 0) return fail(QLIN_ERR_ARG, "bad sizes M=%d K=%d", M, K);
  if (K % 32 != 0 || K > 65536) return fail(QLIN_ERR_SHAPE, "K=%d must be a multiple of 32, at most 65536", K);
  return QLIN_OK;
}

template <int T, int VPT>
cudaError_t launch_norm_t(const NormFwdArgs& g, cudaStream_t stream) {
  const unsigned grid = T == 32 ? (static_cast<unsigned>(g.M) + 3) / 4 : static_cast<unsigned>(g.M);
  return launch_k(norm_forward_kernel<T, VPT>, dim3(grid), dim3(T == 32 ? 128 : T), 0, stream, g);
}

template <bool ACC>
cudaError_t launch_norm_backward_ring(const RingPlan& p, unsigned grid, const NormBwdArgs& g, cudaStream_t stream) {
  if (p.vpt == 4) return launch_ring<norm_backward_ring_kernel<4, 1, ACC>>(p, grid, stream, g);
  if (p.vpt == 2)
    return p.rows == 2 ? launch_ring<norm_backward_ring_kernel<2, 2, ACC>>(p, grid, stream, g)
                       : launch_ring<norm_backward_ring_kernel<2, 1, ACC>>(p, grid, stream, g);
  return p.rows == 4 ? launch_ring<norm_backward_ring_kernel<1, 4, ACC>>(p, grid, stream, g)
                     : launch_ring<norm_backward_ring_kernel<1, 1, ACC>>(p, grid, stream, g);
}

cudaError_t launch_norm_forward_ring(const RingPlan& p, unsigned grid, const NormFwdArgs& g, cudaStream_t stream) {
  // only calls with more rows than persistent CTAs come here: groups are full
  if (p.vpt == 4) return launch_ring<norm_forward_ring_kernel<4, 1>>(p, grid, stream, g);
  if (p.vpt == 2) return launch_ring<norm_forward_ring_kernel<2, 2>>(p, grid, stream, g);
  return launch_ring<norm_forward_ring_kernel<1, 4>>(p, grid, stream, g);
}

// Partial rows of dgamma and dbeta: one per CTA of the ring kernel, else one
// per row group of the column kernel.  The workspace covers both (whether
// dres is given decides whether and how a ring fits).
struct NormBwdLayout {
  RingPlan ring[2];  // without and with dres
  int G;             // row groups of the column kernel
  size_t part, total;
};
NormBwdLayout norm_bwd_layout(int M, int K) {
  NormBwdLayout L{};
  L.G = column_groups(M, K / 8);
  int most = L.G;
  for (int r = 0; r < 2; ++r) {
    L.ring[r] = norm_ring_plan(M, K, 2 + r, true);
    const int n = static_cast<int>(ring_grid(L.ring[r], M));
    if (n > most) most = n;
  }
  L.part = sizeof(WorkspaceHead);  // the head is not used, left as it is
  L.total = M > 0 ? round_up(L.part + size_t(2) * most * K * 4, kAlign) : 0;
  return L;
}

}  // namespace

// ====================================================================== C ABI
extern "C" {

const char* qlin_status_string(qlin_status s) {
  switch (s) {
    case QLIN_OK: return "QLIN_OK";
    case QLIN_ERR_ARG: return "QLIN_ERR_ARG";
    case QLIN_ERR_SHAPE: return "QLIN_ERR_SHAPE";
    case QLIN_ERR_ALIGN: return "QLIN_ERR_ALIGN";
    case QLIN_ERR_WORKSPACE: return "QLIN_ERR_WORKSPACE";
    case QLIN_ERR_CUDA: return "QLIN_ERR_CUDA";
    case QLIN_ERR_TIMEOUT: return "QLIN_ERR_TIMEOUT";
  }
  return "QLIN_UNKNOWN_STATUS";
}

const char* qlin_last_error(void) { return t_last_error; }

qlin_status qlin_weights_bytes(int32_t K, int32_t N, int32_t fmt, int32_t n_outlier, size_t* bytes) {
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  qlin_status st = check_shape(K, N, fmt, n_outlier);
  if (st != QLIN_OK) return st;
  *bytes = weights_layout(K, N, fmt, n_outlier).total;
  return QLIN_OK;
}

qlin_status qlin_weights_bind(qlin_weights* w, int32_t K, int32_t N, int32_t fmt, int32_t n_outlier, void* base,
                              size_t bytes) {
  if (!w || !base) return fail(QLIN_ERR_ARG, "weights descriptor or base is NULL");
  qlin_status st = check_shape(K, N, fmt, n_outlier);
  if (st != QLIN_OK) return st;
  if (reinterpret_cast<uintptr_t>(base) % kAlign) return fail(QLIN_ERR_ALIGN, "base must be 256-byte aligned");
  Layout L = weights_layout(K, N, fmt, n_outlier);
  if (bytes < L.total) return fail(QLIN_ERR_WORKSPACE, "buffer of %zu bytes < %zu needed", bytes, L.total);
  char* b = static_cast<char*>(base);
  memset(w, 0, sizeof(*w));
  w->K = K;
  w->N = N;
  w->fmt = fmt;
  w->group = fmt == QLIN_W4_G128 ? 128 : 0;
  w->n_outlier = n_outlier;
  w->n_outlier_pad = pad8(n_outlier);
  w->codes = b + L.codes;
  w->chan_scale = reinterpret_cast<float*>(b + L.chan);
  if (fmt == QLIN_W4_G128) {
    w->group_scale = reinterpret_cast<uint16_t*>(b + L.group);
    w->fold_ratio = reinterpret_cast<uint16_t*>(b + L.fold);
  }
  if (n_outlier > 0) {
    w->outlier_idx = reinterpret_cast<int32_t*>(b + L.oidx);
    w->W_Ot = reinterpret_cast<uint16_t*>(b + L.wot);
    w->wmax_O = reinterpret_cast<float*>(b + L.wmax);
  }
  return QLIN_OK;
}

qlin_status qlin_pack_weights(const uint16_t* W, const int32_t* O_host, const qlin_weights* w, void* stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!W) return fail(QLIN_ERR_ARG, "W is NULL");
  if (!aligned16(W)) return fail(QLIN_ERR_ALIGN, "W is not 16-byte aligned");
  return pack_from(WeightSource{W, w->N}, O_host, w, static_cast<cudaStream_t>(stream));
}

qlin_status qlin_pack_gated(const uint16_t* W_gate, const uint16_t* W_up, const int32_t* O_host, const qlin_weights* w,
                            void* stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!W_gate || !W_up) return fail(QLIN_ERR_ARG, "W_gate/W_up is NULL");
  if (!aligned16(W_gate) || !aligned16(W_up)) return fail(QLIN_ERR_ALIGN, "W_gate/W_up is not 16-byte aligned");
  return pack_from(GatedSource{W_gate, W_up, w->N / 2}, O_host, w, static_cast<cudaStream_t>(stream));
}

qlin_status qlin_quant_act_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  *bytes = act_ws_bytes(w);
  return QLIN_OK;
}

qlin_status qlin_quant_act(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma,
                           int32_t update_momentum, int8_t* Xq, float* a, int8_t* XqO, void* workspace,
                           size_t ws_bytes, void* stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  const int nO = w->n_outlier;
  if (M > 0 && (!X || !Xq || !a)) return fail(QLIN_ERR_ARG, "X/Xq/a is NULL");
  if (nO > 0 && M > 0 && (!s || !XqO)) return fail(QLIN_ERR_ARG, "s/XqO is NULL with n_outlier=%d", nO);
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  if ((X && !aligned16(X)) || (Xq && !aligned16(Xq)) || (a && !aligned16(a)) || (s && !aligned16(s)) ||
      (XqO && !aligned16(XqO)))
    return fail(QLIN_ERR_ALIGN, "an activation buffer is not 16-byte aligned");
  const size_t need = (update_momentum ? act_ws_bytes(w) : 0);
  if (ws_bytes < need || (need && !workspace)) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  WorkspaceHead* head = head_of(workspace);
  return launch_quant(X, M, w, s, gamma, update_momentum, Xq, a, XqO, nullptr, need ? head->cmax : nullptr,
                      need ? head->momentum : nullptr, static_cast<cudaStream_t>(stream));
}

qlin_status qlin_quant_act_noalloc(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma,
                                   int32_t update_momentum, int8_t* Xq, float* a, int8_t* XqO, void* stream_) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  const int nO = w->n_outlier;
  if (nO > QLIN_NOALLOC_MAX_OUTLIERS)
    return fail(QLIN_ERR_SHAPE, "n_outlier=%d exceeds the %d outlier channels the fixed scratch of "
                "qlin_quant_act_noalloc holds; use qlin_quant_act with a workspace", nO, QLIN_NOALLOC_MAX_OUTLIERS);
  if (M > 0 && (!X || !Xq || !a)) return fail(QLIN_ERR_ARG, "X/Xq/a is NULL");
  if (nO > 0 && M > 0 && (!s || !XqO)) return fail(QLIN_ERR_ARG, "s/XqO is NULL with n_outlier=%d", nO);
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  if ((X && !aligned16(X)) || (Xq && !aligned16(Xq)) || (a && !aligned16(a)) || (s && !aligned16(s)) ||
      (XqO && !aligned16(XqO)))
    return fail(QLIN_ERR_ALIGN, "an activation buffer is not 16-byte aligned");
  if (M == 0) return QLIN_OK;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  unsigned* scratch = nullptr;
  if (update_momentum && nO > 0) {
    st = noalloc_scratch(&scratch);
    if (st != QLIN_OK) return st;
    // The scratch keeps whatever the previous call left: clear the maxima
    // and the counter (they must start at zero) before this call uses them.
    QLIN_CUDA_TRY(cudaMemsetAsync(scratch, 0, (size_t(nO) + 1) * sizeof(unsigned), stream));
  }
  return launch_quant(X, M, w, s, gamma, update_momentum, Xq, a, XqO, nullptr, scratch, scratch ? scratch + nO : nullptr,
                      stream);
}

qlin_status qlin_outlier_colmax(const uint16_t* X, int32_t M, const qlin_weights* w, float* cmax, void* stream_) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  const int nO = w->n_outlier;
  if (nO == 0) return QLIN_OK;
  if (!cmax || (M > 0 && !X)) return fail(QLIN_ERR_ARG, "X/cmax is NULL");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  QLIN_CUDA_TRY(cudaMemsetAsync(cmax, 0, size_t(nO) * 4, stream));
  if (M == 0) return QLIN_OK;
  const int grid = colmax_grid(M);
  colmax_kernel<<<grid, 256, size_t(nO) * 8, stream>>>(X, M, w->K, w->outlier_idx, nO,
                                                        reinterpret_cast<unsigned*>(cmax), 0, nullptr, nullptr,
                                                        0.f, nullptr);
  QLIN_LAUNCH_CHECK("colmax_kernel");
  return QLIN_OK;
}

qlin_status qlin_momentum_update(const qlin_weights* w, const float* cmax, float* s, float gamma, void* stream) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  const int nO = w->n_outlier;
  if (nO == 0) return QLIN_OK;
  if (!cmax || !s) return fail(QLIN_ERR_ARG, "cmax/s is NULL");
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  momentum_kernel<<<(nO + 255) / 256, 256, 0, static_cast<cudaStream_t>(stream)>>>(cmax, w->wmax_O, s, gamma, nO);
  QLIN_LAUNCH_CHECK("momentum_kernel");
  return QLIN_OK;
}

qlin_status qlin_gemm_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  const size_t scratch = gemm_ws_bytes(M, w);
  *bytes = scratch ? sizeof(WorkspaceHead) + scratch : 0;
  return QLIN_OK;
}

qlin_status qlin_gemm(const qlin_weights* w, const int8_t* Xq, const float* a, const int8_t* XqO, const float* s,
                      int32_t M, uint16_t* Y, int32_t* acc_debug, void* workspace, size_t ws_bytes,
                      void* stream_) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (M == 0) return QLIN_OK;
  const int nO = w->n_outlier;
  if (!Xq || !a || !Y) return fail(QLIN_ERR_ARG, "Xq/a/Y is NULL");
  if (nO > 0 && (!XqO || !s)) return fail(QLIN_ERR_ARG, "XqO/s is NULL with n_outlier=%d", nO);
  if (!aligned16(Xq) || !aligned16(a) || !aligned16(Y) || (acc_debug && !aligned16(acc_debug)) ||
      (XqO && !aligned16(XqO)) || (s && !aligned16(s)))
    return fail(QLIN_ERR_ALIGN, "a GEMM buffer is not 16-byte aligned");
  const size_t scratch = gemm_ws_bytes(M, w), need = scratch ? sizeof(WorkspaceHead) + scratch : 0;
  if (ws_bytes < need || (need && !workspace)) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, need);
  if (need && reinterpret_cast<uintptr_t>(workspace) % kAlign)
    return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  GemmScratch gws{nullptr, nullptr};
  if (need) gws = GemmScratch{static_cast<char*>(workspace) + sizeof(WorkspaceHead), head_of(workspace)->cnt};
  if (nO > 0) {
    uint16_t* U = reinterpret_cast<uint16_t*>(gws.p + plan_gemm(M, w).u_off[0]);
    const size_t total = size_t(M) * w->n_outlier_pad;
    comp_operand_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, stream>>>(XqO, s, M, nO,
                                                                                       w->n_outlier_pad, U);
    QLIN_LAUNCH_CHECK("comp_operand_kernel");
  }
  return launch_gemm(w, Xq, a, M, Y, acc_debug, gws, stream);
}

qlin_status qlin_backward_dx_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  *bytes = M > 0 ? plan_backward(M, w, true).bytes : 0;
  return QLIN_OK;
}

qlin_status qlin_backward_dx(const qlin_weights* w, const uint16_t* dY, int32_t M, const float* s, uint16_t* dX,
                             void* workspace, size_t ws_bytes, void* stream_) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (M > 65535 * 128) return fail(QLIN_ERR_SHAPE, "M=%d exceeds %d", M, 65535 * 128);
  if (M == 0) return QLIN_OK;
  if (workspace && reinterpret_cast<uintptr_t>(workspace) % kAlign)
    return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const int nO = w->n_outlier;
  if (!dY || !dX) return fail(QLIN_ERR_ARG, "dY/dX is NULL");
  if (nO > 0 && !s) return fail(QLIN_ERR_ARG, "s is NULL with n_outlier=%d", nO);
  if (!aligned16(dY) || !aligned16(dX) || (s && !aligned16(s)))
    return fail(QLIN_ERR_ALIGN, "a backward buffer is not 16-byte aligned");
  st = get_encoder();
  if (st != QLIN_OK) return st;
  CUtensorMap tm;
  st = make_map(&tm, dY, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, w->N, M, 64, 256, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  BwdArgs args;
  args.codes = static_cast<const uint8_t*>(w->codes);
  args.rfold = w->fold_ratio;
  args.wot = w->W_Ot;
  args.cscale = w->chan_scale;
  args.oidx = w->outlier_idx;
  args.s = s;
  args.dX = dX;
  args.M = M;
  args.N = w->N;
  args.K = w->K;
  args.nO = nO;
  args.kbs = (w->K + 127) / 128;
  args.nib = (nO + 63) / 64;
  args.nsteps = (w->N + 63) / 64;
  // the split plan needs the whole workspace it asks for; with none (or a
  // smaller one) every tile runs whole
  BwdPlan p = plan_backward(M, w, true);
  if (p.bytes && (!workspace || ws_bytes < p.bytes)) p = plan_backward(M, w, false);
  args.ntk = p.ntk;
  args.full = p.full;
  args.tsplit = p.tsplit;
  args.part = p.bytes ? reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_off) : nullptr;
  args.cnt = p.bytes ? head_of(workspace)->cnt : nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  switch (w->fmt) {
    case QLIN_W4_PERCHANNEL: return launch_backward_t<kFmtW4PC>(tm, args, stream);
    case QLIN_W4_G128: return launch_backward_t<kFmtW4G128>(tm, args, stream);
    default: return launch_backward_t<kFmtW8>(tm, args, stream);
  }
}

qlin_status qlin_forward_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  *bytes = forward_layout(M, w).total;
  return QLIN_OK;
}

qlin_status qlin_forward(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma,
                         int32_t update_momentum, uint16_t* Y, void* workspace, size_t ws_bytes, void* stream_) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (M < 0) return fail(QLIN_ERR_ARG, "M=%d is negative", M);
  if (M == 0) return QLIN_OK;
  const int nO = w->n_outlier;
  if (!X || !Y) return fail(QLIN_ERR_ARG, "X/Y is NULL");
  if (nO > 0 && !s) return fail(QLIN_ERR_ARG, "s is NULL with n_outlier=%d", nO);
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  if (!aligned16(X) || !aligned16(Y) || (s && !aligned16(s)))
    return fail(QLIN_ERR_ALIGN, "X/Y/s is not 16-byte aligned");
  FwdLayout L = forward_layout(M, w);
  if (ws_bytes < L.total || !workspace) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + L.xq);
  float* a = reinterpret_cast<float*>(ws + L.a);
  int8_t* XqO = nO > 0 ? reinterpret_cast<int8_t*>(ws + L.xqo) : nullptr;
  WorkspaceHead* head = head_of(workspace);
  const GemmScratch gws{ws + L.gemm, head->cnt};
  uint16_t* U = nO > 0 ? reinterpret_cast<uint16_t*>(gws.p + plan_gemm(M, w).u_off[0]) : nullptr;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  st = launch_quant(X, M, w, s, gamma, update_momentum, Xq, a, XqO, U, head->cmax, head->momentum, stream);
  if (st != QLIN_OK) return st;
  return launch_gemm(w, Xq, a, M, Y, nullptr, gws, stream);
}

qlin_status qlin_forward_act_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  *bytes = forward_layout(M, w, true).total;
  return QLIN_OK;
}

qlin_status qlin_forward_act(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma,
                             int32_t update_momentum, int32_t act, const float* bias, const uint16_t* residual,
                             uint16_t* Z, uint16_t* Y, void* workspace, size_t ws_bytes, void* stream) {
  const EpiArgs e{bias, residual, Z, act};
  return forward_fused(X, M, w, s, gamma, update_momentum, e, kEpiAct, Y, workspace, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

qlin_status qlin_forward_gated_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  return qlin_forward_act_workspace(M, w, bytes);
}

qlin_status qlin_forward_gated(const uint16_t* X, int32_t M, const qlin_weights* w, float* s, float gamma,
                               int32_t update_momentum, int32_t act, const float* bias, uint16_t* Z, uint16_t* H,
                               void* workspace, size_t ws_bytes, void* stream) {
  const EpiArgs e{bias, nullptr, Z, act};
  return forward_fused(X, M, w, s, gamma, update_momentum, e, kEpiGated, H, workspace, ws_bytes,
                       static_cast<cudaStream_t>(stream));
}

qlin_status qlin_backward_act_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  qlin_status st = check_weights(w);
  if (st != QLIN_OK) return st;
  if (!bytes || M < 0) return fail(QLIN_ERR_ARG, "bad arguments");
  *bytes = M > 0 ? fused_bwd_layout(M, w).total : 0;
  return QLIN_OK;
}

qlin_status qlin_backward_act(const qlin_weights* w, const uint16_t* dY, const uint16_t* Z, int32_t act, int32_t M,
                              const float* s, uint16_t* dX, float* dbias, void* workspace, size_t ws_bytes,
                              void* stream) {
  return backward_fused<false>(w, dY, Z, act, M, s, dX, dbias, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

qlin_status qlin_backward_gated_workspace(int32_t M, const qlin_weights* w, size_t* bytes) {
  return qlin_backward_act_workspace(M, w, bytes);
}

qlin_status qlin_backward_gated(const qlin_weights* w, const uint16_t* dH, const uint16_t* Z, int32_t act, int32_t M,
                                const float* s, uint16_t* dX, float* dbias, void* workspace, size_t ws_bytes,
                                void* stream) {
  return backward_fused<true>(w, dH, Z, act, M, s, dX, dbias, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
}

qlin_status qlin_norm_forward(const uint16_t* X, int32_t M, int32_t K, int32_t kind, const float* gamma,
                              const float* beta, float eps, uint16_t* Y, float* mean, float* rstd, void* stream_) {
  qlin_status st = check_norm(M, K, kind);
  if (st != QLIN_OK) return st;
  if (!(eps > 0.f) || std::isinf(eps)) return fail(QLIN_ERR_ARG, "eps=%g must be positive and finite", double(eps));
  if (M == 0) return QLIN_OK;
  if (!X || !gamma || !Y) return fail(QLIN_ERR_ARG, "X/gamma/Y is NULL");
  if (!aligned16(X) || !aligned16(gamma) || !aligned16(Y) || (beta && !aligned16(beta)) || (mean && !aligned16(mean)) ||
      (rstd && !aligned16(rstd)))
    return fail(QLIN_ERR_ALIGN, "a norm buffer is not 16-byte aligned");
  const RingPlan ring = norm_ring_plan(M, K, 1, false);
  const NormFwdArgs g{X,    gamma, beta, Y, kind == QLIN_NORM_RMS ? nullptr : mean,
                      rstd, M,     K,    kind == QLIN_NORM_RMS, eps, ring.stages};
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  const int nv = K / 8;
  cudaError_t e;
  if (ring.ctas > 0 && M > sm_count() * ring.ctas && ring.rows * ring.vpt == 4)
    e = launch_norm_forward_ring(ring, ring_grid(ring, M), g, stream);
  else if (nv <= 32) e = launch_norm_t<32, 1>(g, stream);
  else if (nv <= 128) e = launch_norm_t<32, 4>(g, stream);
  else if (nv <= 512) e = launch_norm_t<128, 4>(g, stream);
  else if (nv <= 1024) e = launch_norm_t<256, 4>(g, stream);
  else if (nv <= 2048) e = launch_norm_t<512, 4>(g, stream);
  else e = launch_norm_t<1024, 8>(g, stream);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "norm_forward_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

qlin_status qlin_norm_backward_workspace(int32_t M, int32_t K, size_t* bytes) {
  qlin_status st = check_norm(M, K, QLIN_NORM_LAYER);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = norm_bwd_layout(M, K).total;
  return QLIN_OK;
}

qlin_status qlin_norm_backward(const uint16_t* dY, const uint16_t* X, int32_t M, int32_t K, int32_t kind,
                               const float* gamma, const float* mean, const float* rstd, const uint16_t* dres,
                               uint16_t* dX, float* dgamma, float* dbeta, void* workspace, size_t ws_bytes,
                               void* stream_) {
  qlin_status st = check_norm(M, K, kind);
  if (st != QLIN_OK) return st;
  const bool rms = kind == QLIN_NORM_RMS;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if ((dgamma && !aligned16(dgamma)) || (dbeta && !aligned16(dbeta)))
    return fail(QLIN_ERR_ALIGN, "dgamma/dbeta is not 16-byte aligned");
  if (M == 0) {  // no rows: sums over nothing
    if (dgamma) QLIN_CUDA_TRY(cudaMemsetAsync(dgamma, 0, size_t(K) * 4, stream));
    if (dbeta) QLIN_CUDA_TRY(cudaMemsetAsync(dbeta, 0, size_t(K) * 4, stream));
    return QLIN_OK;
  }
  if (!dX && !dgamma && !dbeta) return fail(QLIN_ERR_ARG, "dX, dgamma and dbeta are all NULL");
  if (!dY || !X || !gamma || !rstd || (!rms && !mean)) return fail(QLIN_ERR_ARG, "dY/X/gamma/mean/rstd is NULL");
  if (!aligned16(dY) || !aligned16(X) || !aligned16(gamma) || !aligned16(rstd) || (mean && !aligned16(mean)) ||
      (dres && !aligned16(dres)) || (dX && !aligned16(dX)))
    return fail(QLIN_ERR_ALIGN, "a norm buffer is not 16-byte aligned");
  NormBwdArgs g{dY, X, gamma, rms ? nullptr : mean, rstd, dres, dX, nullptr, M, K, rms, 0, 0};
  const NormBwdLayout L = norm_bwd_layout(M, K);
  const RingPlan& ring = L.ring[dres ? 1 : 0];
  const bool acc = dgamma || dbeta;
  if (acc) {
    if (ws_bytes < L.total || !workspace) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
    if (reinterpret_cast<uintptr_t>(workspace) % kAlign)
      return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
    g.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.part);
  }
  if (ring.ctas > 0) {
    const unsigned grid = ring_grid(ring, M);
    g.stages = ring.stages;
    cudaError_t e = acc ? launch_norm_backward_ring<true>(ring, grid, g, stream)
                        : launch_norm_backward_ring<false>(ring, grid, g, stream);
    if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "norm_backward_ring_kernel launch failed: %s", cudaGetErrorString(e));
    return acc ? launch_column_sum<32>(g.part, static_cast<int>(grid), K, dgamma, dbeta, stream) : QLIN_OK;
  }
  if (acc) {
    g.G = L.G;
    // before dX, which may replace dY or X
    cudaError_t e = launch_k(norm_columns_kernel, dim3((K / 8 + 127) / 128, L.G), dim3(128), 0, stream, g);
    if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "norm_columns_kernel launch failed: %s", cudaGetErrorString(e));
    st = launch_column_sum<32>(g.part, L.G, K, dgamma, dbeta, stream);
    if (st != QLIN_OK) return st;
  }
  if (!dX) return QLIN_OK;
  const dim3 grid(static_cast<unsigned>(M));
  cudaError_t e = launch_k(norm_rows_kernel<512>, grid, dim3(512), 0, stream, g);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "norm_rows_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

#ifdef QLIN_TRACE
// Diagnostic builds only: point the GEMM's phase stamps at a device buffer
// of [grid][32] int64 (NULL turns them off).
QLIN_API int qlin_trace_set(long long* p) {
  return static_cast<int>(cudaMemcpyToSymbol(qlin::g_trace, &p, sizeof(p)));
}
QLIN_API int qlin_steps_set(long long* p) {
  return static_cast<int>(cudaMemcpyToSymbol(qlin::g_steps, &p, sizeof(p)));
}
#endif

qlin_status qlin_forward_grouped_workspace(int32_t count, const qlin_weights* const* w, int32_t M, size_t* bytes) {
  qlin_status st = check_group(count, w, M);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = group_layout(M, w, count).total;
  return QLIN_OK;
}

qlin_status qlin_forward_grouped(int32_t count, const qlin_weights* const* w, const uint16_t* const* X,
                                 float* const* s, uint16_t* const* Y, int32_t M, float gamma,
                                 int32_t update_momentum, void* workspace, size_t ws_bytes, void* stream_) {
  qlin_status st = check_group(count, w, M);
  if (st != QLIN_OK) return st;
  if (!(gamma >= 0.f && gamma <= 1.f)) return fail(QLIN_ERR_ARG, "gamma=%g outside [0, 1]", double(gamma));
  if (M == 0) return QLIN_OK;
  if (!X || !Y || !s) return fail(QLIN_ERR_ARG, "X/Y/s array is NULL");
  for (int q = 0; q < count; ++q) {
    if (!X[q] || !Y[q]) return fail(QLIN_ERR_ARG, "problem %d: X/Y is NULL", q);
    if (w[q]->n_outlier > 0 && !s[q]) return fail(QLIN_ERR_ARG, "problem %d: s is NULL with n_outlier=%d", q,
                                                  w[q]->n_outlier);
    if (!aligned16(X[q]) || !aligned16(Y[q]) || (s[q] && !aligned16(s[q])))
      return fail(QLIN_ERR_ALIGN, "problem %d: X/Y/s is not 16-byte aligned", q);
    for (int r = 0; r < q; ++r)
      if (Y[r] == Y[q]) return fail(QLIN_ERR_ARG, "problems %d and %d write the same Y", r, q);
  }
  const GroupLayout L = group_layout(M, w, count);
  if (ws_bytes < L.total || !workspace) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  char* ws = static_cast<char*>(workspace);
  WorkspaceHead* head = head_of(workspace);
  const GemmScratch gws{ws + L.gemm, head->cnt};
  QuantIO io[kMaxProbs];
  const int8_t* xq[kMaxProbs];
  const float* av[kMaxProbs];
  uint16_t* yv[kMaxProbs];
  for (int q = 0; q < count; ++q) {
    const bool o = w[q]->n_outlier > 0;
    io[q] = QuantIO{X[q], s[q], reinterpret_cast<int8_t*>(ws + L.xq[q]), reinterpret_cast<float*>(ws + L.a[q]),
                    o ? reinterpret_cast<int8_t*>(ws + L.xqo[q]) : nullptr,
                    o ? reinterpret_cast<uint16_t*>(gws.p + L.plan.u_off[q]) : nullptr, head->cmax, head->momentum + q};
    xq[q] = io[q].Xq;
    av[q] = io[q].a;
    yv[q] = Y[q];
  }
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  st = launch_quant_group<kMaxProbs>(w, io, count, M, gamma, update_momentum, stream);
  if (st != QLIN_OK) return st;
  return launch_gemm_group<kMaxProbs>(L.plan, w, xq, av, yv, nullptr, gws, stream);
}

namespace {
struct GptqLayout {
  size_t st, f, a, total;
};
GptqLayout gptq_layout(int K) {
  GptqLayout L{};
  L.st = 0;
  L.f = round_up(sizeof(GjScratch), kAlign);
  L.a = round_up(L.f + size_t(K) * 8, kAlign);
  L.total = round_up(L.a + size_t(K) * K * 8, kAlign);
  return L;
}
qlin_status check_gptq_shape(int32_t K, int32_t N) {
  if (K < 1 || N < 1) return fail(QLIN_ERR_ARG, "K=%d N=%d must be positive", K, N);
  if (K > 16384) return fail(QLIN_ERR_SHAPE, "K=%d exceeds 16384", K);
  return QLIN_OK;
}
}  // namespace

qlin_status qlin_gptq_workspace(int32_t K, int32_t N, size_t* bytes) {
  qlin_status st = check_gptq_shape(K, N);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = gptq_layout(K).total;
  return QLIN_OK;
}

qlin_status qlin_gptq_quantize(const double* X, int32_t ns, int32_t K, int32_t N, double* W, const double* scale,
                               int32_t qmax, int8_t* codes, double* Hinv, int32_t* singular, void* workspace,
                               size_t ws_bytes, void* stream_) {
  qlin_status st = check_gptq_shape(K, N);
  if (st != QLIN_OK) return st;
  if (ns < 1) return fail(QLIN_ERR_ARG, "ns=%d must be positive", ns);
  if (qmax < 1 || qmax > 127) return fail(QLIN_ERR_ARG, "qmax=%d outside [1, 127]", qmax);
  if (!X || !W || !scale || !codes || !Hinv || !workspace) return fail(QLIN_ERR_ARG, "a GPTQ buffer is NULL");
  if ((reinterpret_cast<uintptr_t>(X) | reinterpret_cast<uintptr_t>(W) | reinterpret_cast<uintptr_t>(scale) |
       reinterpret_cast<uintptr_t>(Hinv)) & 7u)
    return fail(QLIN_ERR_ALIGN, "fp64 buffers must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const GptqLayout L = gptq_layout(K);
  if (ws_bytes < L.total) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  GjScratch* scr = reinterpret_cast<GjScratch*>(ws + L.st);
  double* f = reinterpret_cast<double*>(ws + L.f);
  double* a = reinterpret_cast<double*>(ws + L.a);
  QLIN_CUDA_TRY(cudaMemsetAsync(scr, 0, sizeof(GjScratch), stream));
  // H = 2 X^T X into the working matrix; the inverse starts as the identity
  const unsigned th = static_cast<unsigned>((K + kHessTile - 1) / kHessTile);
  gptq_hessian_kernel<<<dim3(th, th), 256, 0, stream>>>(X, ns, K, a);
  QLIN_LAUNCH_CHECK("gptq_hessian_kernel");
  const size_t kk = size_t(K) * K;
  gptq_identity_kernel<<<static_cast<unsigned>((kk + 255) / 256), 256, 0, stream>>>(Hinv, K);
  QLIN_LAUNCH_CHECK("gptq_identity_kernel");
  // Gauss-Jordan elimination with partial pivoting: a -> I, Hinv -> H^-1
  const unsigned cb = static_cast<unsigned>((K + 255) / 256);
  const unsigned ex = cb < 4 ? cb : 4;
  for (int c = 0; c < K; ++c) {
    gj_pivot_kernel<<<1, 1024, 0, stream>>>(a, K, c, scr, f);
    gj_swap_scale_kernel<<<cb, 256, 0, stream>>>(a, Hinv, K, c, scr);
    gj_eliminate_kernel<<<dim3(ex, static_cast<unsigned>(K)), 256, 0, stream>>>(a, Hinv, K, c, scr, f);
  }
  QLIN_LAUNCH_CHECK("Gauss-Jordan kernels");
  // column-sequential quantization with compensation on a working copy of H^-1
  QLIN_CUDA_TRY(cudaMemcpyAsync(a, Hinv, kk * 8, cudaMemcpyDeviceToDevice, stream));
  constexpr int kRows = 64;
  for (int i = 0; i < K; ++i) {
    const int rem = K - i - 1;
    const int yw = rem > 0 ? (rem + kRows - 1) / kRows : 1;
    const int yd = rem > 0 ? (rem + kRows - 1) / kRows : 0;
    const int xa = (N + 255) / 256, xd = (rem + 255) / 256;
    const unsigned gx = static_cast<unsigned>(xa > xd ? xa : xd);
    gptq_step_kernel<<<dim3(gx, static_cast<unsigned>(yw + yd)), 256, 0, stream>>>(W, codes, scale, a, K, N, i, qmax,
                                                                                  kRows, yw, scr);
  }
  QLIN_LAUNCH_CHECK("gptq_step_kernel");
  if (singular) QLIN_CUDA_TRY(cudaMemcpyAsync(singular, &scr->singular, 4, cudaMemcpyDeviceToDevice, stream));
  return QLIN_OK;
}

namespace {
struct SmoothLayout {
  size_t cmax, wmax, xall, sv, xh, wh, packed, xq, a, cnt, gemm, y, acc, ref, total;
  Layout wl;
};
SmoothLayout smooth_layout(int M, int K, int N) {
  SmoothLayout L{};
  size_t off = 0;
  L.cmax = off; off = round_up(off + size_t(K) * 4, kAlign);
  L.wmax = off; off = round_up(off + size_t(K) * 4, kAlign);
  L.xall = off; off = round_up(off + 16, kAlign);
  L.sv = off; off = round_up(off + size_t(K) * 4, kAlign);
  L.xh = off; off = round_up(off + size_t(M) * K * 2, kAlign);
  L.wh = off; off = round_up(off + size_t(K) * N * 2, kAlign);
  L.wl = weights_layout(K, N, QLIN_W4_PERCHANNEL, 0);
  L.packed = off; off = round_up(off + L.wl.total, kAlign);
  L.xq = off; off = round_up(off + size_t(M) * K, kAlign);
  L.a = off; off = round_up(off + size_t(M) * 4, kAlign);
  qlin_weights w{};
  w.K = K; w.N = N; w.fmt = QLIN_W4_PERCHANNEL; w.n_outlier = 0; w.n_outlier_pad = 0;
  L.cnt = off; off = round_up(off + sizeof(WorkspaceHead::cnt), kAlign);
  L.gemm = off; off = round_up(off + gemm_ws_bytes(M, &w), kAlign);
  L.y = off; off = round_up(off + size_t(M) * N * 2, kAlign);
  L.acc = off; off = round_up(off + size_t(M) * N * 4, kAlign);
  L.ref = off; off = round_up(off + size_t(M) * N * 4, kAlign);
  L.total = off;
  return L;
}
qlin_status check_smooth(int32_t M, int32_t K, int32_t N, int32_t G) {
  if (M < 1 || G < 1 || G > 64) return fail(QLIN_ERR_ARG, "M=%d must be >= 1 and G=%d in [1, 64]", M, G);
  return check_shape(K, N, QLIN_W4_PERCHANNEL, 0);
}
}  // namespace

qlin_status qlin_smooth_search_workspace(int32_t M, int32_t K, int32_t N, int32_t G, size_t* bytes) {
  qlin_status st = check_smooth(M, K, N, G);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = smooth_layout(M, K, N).total;
  return QLIN_OK;
}

qlin_status qlin_smooth_search(const uint16_t* X, int32_t M, int32_t K, const uint16_t* W, int32_t N, int32_t G,
                               double* loss, int32_t* best, float* s_best, void* workspace, size_t ws_bytes,
                               void* stream_) {
  qlin_status st = check_smooth(M, K, N, G);
  if (st != QLIN_OK) return st;
  if (!X || !W || !loss || !workspace) return fail(QLIN_ERR_ARG, "X/W/loss/workspace is NULL");
  if (!aligned16(X) || !aligned16(W) || (reinterpret_cast<uintptr_t>(loss) & 7u) ||
      (s_best && (reinterpret_cast<uintptr_t>(s_best) & 3u)) || (best && (reinterpret_cast<uintptr_t>(best) & 3u)))
    return fail(QLIN_ERR_ALIGN, "X/W must be 16-byte aligned, loss 8, best and s_best 4");
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const SmoothLayout L = smooth_layout(M, K, N);
  if (ws_bytes < L.total) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  char* ws = static_cast<char*>(workspace);
  unsigned* cmax = reinterpret_cast<unsigned*>(ws + L.cmax);
  float* wmax = reinterpret_cast<float*>(ws + L.wmax);
  float* xall = reinterpret_cast<float*>(ws + L.xall);
  float* sv = reinterpret_cast<float*>(ws + L.sv);
  uint16_t* Xh = reinterpret_cast<uint16_t*>(ws + L.xh);
  uint16_t* Wh = reinterpret_cast<uint16_t*>(ws + L.wh);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + L.xq);
  float* a = reinterpret_cast<float*>(ws + L.a);
  uint16_t* Y = reinterpret_cast<uint16_t*>(ws + L.y);
  int32_t* acc = reinterpret_cast<int32_t*>(ws + L.acc);
  float* ref = reinterpret_cast<float*>(ws + L.ref);
  qlin_weights w{};
  st = qlin_weights_bind(&w, K, N, QLIN_W4_PERCHANNEL, 0, ws + L.packed, L.wl.total);
  if (st != QLIN_OK) return st;
  QLIN_CUDA_TRY(cudaMemsetAsync(cmax, 0, size_t(K) * 4, stream));
  QLIN_CUDA_TRY(cudaMemsetAsync(ws + L.cnt, 0, sizeof(WorkspaceHead::cnt), stream));  // split-K counters start at zero
  QLIN_CUDA_TRY(cudaMemsetAsync(loss, 0, size_t(G) * 8, stream));
  smooth_colmax_kernel<<<dim3((K + 255) / 256, (M + 63) / 64), 256, 0, stream>>>(X, M, K, cmax);
  smooth_rowmax_kernel<<<K, 256, 0, stream>>>(W, N, wmax);
  smooth_allmax_kernel<<<1, 1024, 0, stream>>>(cmax, K, xall);
  QLIN_LAUNCH_CHECK("smoothing maxima");
  const size_t mk = size_t(M) * K, kn = size_t(K) * N, mn = size_t(M) * N;
  for (int j = 0; j < G; ++j) {
    smooth_factors_kernel<<<(K + 255) / 256, 256, 0, stream>>>(cmax, wmax, xall, K, j, G, sv);
    smooth_apply_x_kernel<<<static_cast<unsigned>((mk + 255) / 256), 256, 0, stream>>>(X, sv, M, K, Xh);
    smooth_apply_w_kernel<<<static_cast<unsigned>((kn + 255) / 256), 256, 0, stream>>>(W, sv, K, N, Wh);
    QLIN_LAUNCH_CHECK("smoothing kernels");
    // the layer's quantizers and integer product on the smoothed tensors
    st = qlin_pack_weights(Wh, nullptr, &w, stream);
    if (st != QLIN_OK) return st;
    st = launch_quant(Xh, M, &w, nullptr, 0.f, 0, Xq, a, nullptr, nullptr, nullptr, nullptr, stream);
    if (st != QLIN_OK) return st;
    st = launch_gemm(&w, Xq, a, M, Y, acc, GemmScratch{ws + L.gemm, reinterpret_cast<unsigned*>(ws + L.cnt)}, stream);
    if (st != QLIN_OK) return st;
    smooth_ref_kernel<<<dim3((N + kRefTile - 1) / kRefTile, (M + kRefTile - 1) / kRefTile), 256, 0, stream>>>(
        X, W, sv, M, K, N, ref);
    smooth_loss_kernel<<<static_cast<unsigned>((mn + 255) / 256), 256, 0, stream>>>(acc, a, w.chan_scale, ref, M,
                                                                                    N, loss + j);
    QLIN_LAUNCH_CHECK("smoothing loss");
  }
  smooth_pick_kernel<<<1, 256, 0, stream>>>(loss, G, cmax, wmax, xall, K, best, s_best);
  QLIN_LAUNCH_CHECK("smooth_pick_kernel");
  return QLIN_OK;
}

// ---------------------------------------------------------------- OffQ
namespace {
// d (+1/-1, d_0 = +1) as a bit mask: bit i set when d_i = -1.
qlin_status offq_signs(const int8_t* d, uint4* out) {
  if (!d) return fail(QLIN_ERR_ARG, "signs is NULL");
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  for (int i = 0; i < 128; ++i) {
    if (d[i] != 1 && d[i] != -1) return fail(QLIN_ERR_ARG, "signs[%d] = %d is not +1 or -1", i, int(d[i]));
    if (d[i] < 0) w[i >> 5] |= 1u << (i & 31);
  }
  if (w[0] & 1u) return fail(QLIN_ERR_ARG, "signs[0] must be +1 (row 0 of D H is all ones)");
  *out = make_uint4(w[0], w[1], w[2], w[3]);
  return QLIN_OK;
}

qlin_status check_offq_shape(int32_t M, int32_t K, int32_t N) {
  if (M < 0 || K <= 0 || N <= 0) return fail(QLIN_ERR_ARG, "bad sizes M=%d K=%d N=%d", M, K, N);
  if (K % 128 || K > 65536) return fail(QLIN_ERR_SHAPE, "OffQ needs K %% 128 == 0 and K <= 65536 (K=%d)", K);
  if (N % 16 || N > 1048576) return fail(QLIN_ERR_SHAPE, "N=%d must be a multiple of 16 and <= 2^20", N);
  return QLIN_OK;
}

size_t offq_codes_size(int32_t K, int32_t N) { return size_t((N + 127) / 128) * (K / 128) * 8192; }
size_t offq_wide_size(int32_t K, int32_t N) { return size_t((N + 127) / 128) * (K / 128) * 16384; }

struct OffqLayout {
  size_t xq = 0, scale = 0, offset = 0, wide = 0, total = 0;
};
OffqLayout offq_layout(int32_t M, int32_t K, int32_t N, bool with_act) {
  OffqLayout L;
  size_t o = 0;
  if (with_act) {
    L.xq = o;
    o = round_up(o + size_t(M) * K, kAlign);
    L.scale = o;
    o = round_up(o + size_t(M) * (K / 128) * 4, kAlign);
    L.offset = o;
    o = round_up(o + size_t(M) * (K / 128) * 4, kAlign);
  }
  L.wide = o;
  L.total = round_up(o + offq_wide_size(K, N), kAlign);
  return L;
}

int offq_gemm_smem_ok() {
  static int ok = -1;
  static std::once_flag once;
  std::call_once(once, [] {
    ok = cudaFuncSetAttribute(offq_gemm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOffqSmem) ==
         cudaSuccess;
    if (!ok) cudaGetLastError();
  });
  return ok;
}

qlin_status launch_offq_quant(const uint16_t* X, int32_t M, int32_t K, uint4 sg, int8_t* Xq, float* scale,
                              float* offset, cudaStream_t stream) {
  const long long units = static_cast<long long>(M) * (K / 128);
  const long long blocks = (units + kOffqQuantThreads / 4 - 1) / (kOffqQuantThreads / 4);
  if (blocks > 0x7fffffffLL) return fail(QLIN_ERR_SHAPE, "M * K too large");
  cudaError_t e = launch_k(offq_quant_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kOffqQuantThreads), 0,
                           stream, X, M, K, sg, Xq, scale, offset);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "offq_quant_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}

qlin_status launch_offq_gemm(const int8_t* Xq, const float* scale, const float* offset, int32_t M, int32_t K,
                             int32_t N, const uint8_t* codes, const float* chan_scale, const float* colsum,
                             uint16_t* Y, uint8_t* wide, cudaStream_t stream) {
  qlin_status st = get_encoder();
  if (st != QLIN_OK) return st;
  if (!offq_gemm_smem_ok()) return fail(QLIN_ERR_CUDA, "offq_gemm_kernel: shared memory attribute refused");
  const int kb = K / 128;
  const int tiles_n = (N + 127) / 128;
  const unsigned nblk = static_cast<unsigned>(tiles_n) * static_cast<unsigned>(kb);
  cudaError_t e = launch_k(widen_w4_kernel<kFmtW4PC>, dim3(nblk), dim3(256), 0, stream, codes,
                           static_cast<const uint16_t*>(nullptr), N, kb, wide);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "widen_w4_kernel launch failed: %s", cudaGetErrorString(e));
  OffqParams prm;
  memset(&prm, 0, sizeof(prm));
  OffqArgs& g = prm.g;
  g.scale = scale;
  g.offset = offset;
  g.colsum = colsum;
  g.cscale = chan_scale;
  g.wide = wide;
  g.Y = Y;
  g.M = M;
  g.N = N;
  g.G = kb;
  g.tiles_m = (M + 127) / 128;
  g.tiles = g.tiles_m * tiles_n;
  st = make_map(&prm.tmX, Xq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, K, M, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != QLIN_OK) return st;
  const int cap = gemm_cta_cap();
  const int grid = g.tiles < cap ? g.tiles : cap;
  e = launch_k(offq_gemm_kernel, dim3(static_cast<unsigned>(grid)), dim3(kOffqThreads), kOffqSmem, stream, prm);
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "offq_gemm_kernel launch failed: %s", cudaGetErrorString(e));
  return QLIN_OK;
}
}  // namespace

qlin_status qlin_offq_codes_bytes(int32_t K, int32_t N, size_t* bytes) {
  qlin_status st = check_offq_shape(0, K, N);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = offq_codes_size(K, N);
  return QLIN_OK;
}

qlin_status qlin_offq_rotate_weights(const uint16_t* W, int32_t K, int32_t N, const int8_t* signs, float* Wr,
                                     void* stream_) {
  qlin_status st = check_offq_shape(0, K, N);
  if (st != QLIN_OK) return st;
  uint4 sg;
  st = offq_signs(signs, &sg);
  if (st != QLIN_OK) return st;
  if (!W || !Wr) return fail(QLIN_ERR_ARG, "W/Wr is NULL");
  if (!aligned16(W) || !aligned16(Wr)) return fail(QLIN_ERR_ALIGN, "W/Wr is not 16-byte aligned");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  offq_rotate_kernel<<<dim3((N + 31) / 32, K / 128), 256, 0, stream>>>(W, K, N, sg, Wr);
  QLIN_LAUNCH_CHECK("offq_rotate_kernel");
  return QLIN_OK;
}

qlin_status qlin_offq_pack(const uint16_t* W, int32_t K, int32_t N, const int8_t* signs, uint8_t* codes,
                           float* chan_scale, float* colsum, float* Wr, void* stream_) {
  qlin_status st = qlin_offq_rotate_weights(W, K, N, signs, Wr, stream_);
  if (st != QLIN_OK) return st;
  if (!codes || !chan_scale || !colsum) return fail(QLIN_ERR_ARG, "codes/chan_scale/colsum is NULL");
  if (!aligned16(codes) || !aligned16(chan_scale) || !aligned16(colsum))
    return fail(QLIN_ERR_ALIGN, "codes/chan_scale/colsum is not 16-byte aligned");
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  QLIN_CUDA_TRY(cudaMemsetAsync(codes, 0, offq_codes_size(K, N), stream));  // padding channels stay zero
  offq_pack_kernel<<<(N + 127) / 128, 128, 0, stream>>>(Wr, K, N, codes, chan_scale, colsum);
  QLIN_LAUNCH_CHECK("offq_pack_kernel");
  return QLIN_OK;
}

qlin_status qlin_offq_quant_act(const uint16_t* X, int32_t M, int32_t K, const int8_t* signs, int8_t* Xq,
                                float* scale, float* offset, void* stream_) {
  qlin_status st = check_offq_shape(M, K, 16);
  if (st != QLIN_OK) return st;
  uint4 sg;
  st = offq_signs(signs, &sg);
  if (st != QLIN_OK) return st;
  if (M == 0) return QLIN_OK;
  if (!X || !Xq || !scale || !offset) return fail(QLIN_ERR_ARG, "X/Xq/scale/offset is NULL");
  if (!aligned16(X) || !aligned16(Xq) || (reinterpret_cast<uintptr_t>(scale) & 3u) ||
      (reinterpret_cast<uintptr_t>(offset) & 3u))
    return fail(QLIN_ERR_ALIGN, "X/Xq must be 16-byte aligned, scale/offset 4");
  return launch_offq_quant(X, M, K, sg, Xq, scale, offset, static_cast<cudaStream_t>(stream_));
}

qlin_status qlin_offq_gemm_workspace(int32_t M, int32_t K, int32_t N, size_t* bytes) {
  qlin_status st = check_offq_shape(M, K, N);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = offq_layout(M, K, N, false).total;
  return QLIN_OK;
}

qlin_status qlin_offq_gemm(const int8_t* Xq, const float* scale, const float* offset, int32_t M, int32_t K,
                           int32_t N, const uint8_t* codes, const float* chan_scale, const float* colsum, uint16_t* Y,
                           void* workspace, size_t ws_bytes, void* stream_) {
  qlin_status st = check_offq_shape(M, K, N);
  if (st != QLIN_OK) return st;
  if (M == 0) return QLIN_OK;
  if (!Xq || !scale || !offset || !codes || !chan_scale || !colsum || !Y || !workspace)
    return fail(QLIN_ERR_ARG, "a pointer argument is NULL");
  if (!aligned16(Xq) || !aligned16(codes) || !aligned16(chan_scale) || !aligned16(colsum) || !aligned16(Y) ||
      (reinterpret_cast<uintptr_t>(scale) & 3u) || (reinterpret_cast<uintptr_t>(offset) & 3u))
    return fail(QLIN_ERR_ALIGN, "Xq/codes/chan_scale/colsum/Y must be 16-byte aligned, scale/offset 4");
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const OffqLayout L = offq_layout(M, K, N, false);
  if (ws_bytes < L.total) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  uint8_t* wide = static_cast<uint8_t*>(workspace) + L.wide;
  return launch_offq_gemm(Xq, scale, offset, M, K, N, codes, chan_scale, colsum, Y, wide,
                          static_cast<cudaStream_t>(stream_));
}

qlin_status qlin_offq_forward_workspace(int32_t M, int32_t K, int32_t N, size_t* bytes) {
  qlin_status st = check_offq_shape(M, K, N);
  if (st != QLIN_OK) return st;
  if (!bytes) return fail(QLIN_ERR_ARG, "bytes is NULL");
  *bytes = offq_layout(M, K, N, true).total;
  return QLIN_OK;
}

qlin_status qlin_offq_forward(const uint16_t* X, int32_t M, int32_t K, int32_t N, const int8_t* signs,
                              const uint8_t* codes, const float* chan_scale, const float* colsum, uint16_t* Y,
                              void* workspace, size_t ws_bytes, void* stream_) {
  qlin_status st = check_offq_shape(M, K, N);
  if (st != QLIN_OK) return st;
  uint4 sg;
  st = offq_signs(signs, &sg);
  if (st != QLIN_OK) return st;
  if (M == 0) return QLIN_OK;
  if (!X || !codes || !chan_scale || !colsum || !Y || !workspace) return fail(QLIN_ERR_ARG, "a pointer argument is NULL");
  if (!aligned16(X) || !aligned16(codes) || !aligned16(chan_scale) || !aligned16(colsum) || !aligned16(Y))
    return fail(QLIN_ERR_ALIGN, "X/codes/chan_scale/colsum/Y is not 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) % kAlign) return fail(QLIN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const OffqLayout L = offq_layout(M, K, N, true);
  if (ws_bytes < L.total) return fail(QLIN_ERR_WORKSPACE, "workspace %zu < %zu", ws_bytes, L.total);
  char* ws = static_cast<char*>(workspace);
  int8_t* Xq = reinterpret_cast<int8_t*>(ws + L.xq);
  float* scale = reinterpret_cast<float*>(ws + L.scale);
  float* offset = reinterpret_cast<float*>(ws + L.offset);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  st = launch_offq_quant(X, M, K, sg, Xq, scale, offset, stream);
  if (st != QLIN_OK) return st;
  return launch_offq_gemm(Xq, scale, offset, M, K, N, codes, chan_scale, colsum, Y,
                          reinterpret_cast<uint8_t*>(ws + L.wide), stream);
}

qlin_status qlin_debug_set(int32_t k, int64_t value, int64_t* previous) {
  if (k < 0 || k > QLIN_KNOB_PAIR_SPLIT) return fail(QLIN_ERR_ARG, "unknown knob %d", k);
  bool ok = true;
  switch (k) {
    case QLIN_KNOB_PDL:
    case QLIN_KNOB_CLUSTER:
    case QLIN_KNOB_PAIR_SPLIT: ok = value == 0 || value == 1; break;
    case QLIN_KNOB_CLUSTER_SIZE: ok = value == 0 || value == 2 || value == 4 || value == 8; break;
    case QLIN_KNOB_MAX_TOKEN_TILE: ok = value == 64 || value == 128 || value == 256; break;
    case QLIN_KNOB_PAIR_MMA: ok = value >= 0 && value <= 2; break;
    default: ok = value >= 0;
  }
  if (!ok) return fail(QLIN_ERR_ARG, "invalid value %lld for knob %d", static_cast<long long>(value), k);
  if (k == QLIN_KNOB_WAIT_NS) {
    const unsigned long long v = static_cast<unsigned long long>(value);
    QLIN_CUDA_TRY(cudaMemcpyToSymbol(qlin::g_wait_ns, &v, sizeof(v)));
  }
  const long long old = g_knob[k].exchange(value);
  if (previous) *previous = old;
  return QLIN_OK;
}

qlin_status qlin_debug_get(int32_t k, int64_t* value) {
  if (k < 0 || k > QLIN_KNOB_PAIR_SPLIT || !value) return fail(QLIN_ERR_ARG, "unknown knob %d or NULL value", k);
  *value = g_knob[k].load();
  return QLIN_OK;
}

qlin_status qlin_poll_device_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(QLIN_ERR_CUDA, "stream error: %s", cudaGetErrorString(e));
  int flag = 0;
  QLIN_CUDA_TRY(cudaMemcpyFromSymbol(&flag, qlin::g_device_error, sizeof(int)));
  if (flag) {
    const int zero = 0;
    QLIN_CUDA_TRY(cudaMemcpyToSymbol(qlin::g_device_error, &zero, sizeof(int)));
    return fail(QLIN_ERR_TIMEOUT, "a device-side bounded wait gave up (code %d)", flag);
  }
  return QLIN_OK;
}

}  // extern "C"
