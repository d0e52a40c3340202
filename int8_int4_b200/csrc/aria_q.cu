// aria_q.cu -- the C ABI of libaria_q.so (declared in include/aria_q.h):
// host-side validation, tensor-map encoding, tile / split planning and
// launches of the sm_100a kernels. One translation unit, so the device
// status word is a single symbol without relocatable device code.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "aria_q.h"
#include "act.cuh"
#include "gated_bwd.cuh"
#include "ptx.cuh"
#include "qgemm.cuh"
#include "quant_kernels.cuh"
#include "smallm.cuh"
#include "tgemm.cuh"

#define ARIA_API extern "C" __attribute__((visibility("default")))

namespace {

thread_local char g_msg[512] = "";

aria_status fail(aria_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

aria_status cuda_fail(cudaError_t e, const char* what) {
  return fail(ARIA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int64_t kMaxDim = (int64_t{1} << 31) - 1;

// ------------------------------------------------------------ tensor maps ---
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// 2-D row-major tensor [rows, cols] of `esize`-byte elements; box {bc, br}.
aria_status make_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int esize,
                     int64_t rows, int64_t cols, int bc, int br, CUtensorMapSwizzle sw) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(ARIA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols * esize)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(bc), static_cast<cuuint32_t>(br)};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ARIA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ARIA_OK;
}

// ---------------------------------------------------------- device facts ---
struct DevInfo {
  int sms = 148;
  int smem_optin = 232448;
};

constexpr int kMaxDevices = 64;

int current_device() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
  return dev;
}

DevInfo dev_info() {
  static DevInfo info[kMaxDevices];
  static bool done[kMaxDevices] = {};
  static std::mutex mu;
  const int dev = current_device();
  std::lock_guard<std::mutex> g(mu);
  if (dev >= 0 && dev < kMaxDevices && !done[dev]) {
    cudaDeviceGetAttribute(&info[dev].sms, cudaDevAttrMultiProcessorCount, dev);
    cudaDeviceGetAttribute(&info[dev].smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    done[dev] = true;
  }
  return (dev >= 0 && dev < kMaxDevices) ? info[dev] : DevInfo{};
}

// ----------------------------------------------------------------- GEMM ---
struct Plan {
  aria::GemmParams p;
  dim3 grid;
  int threads;
  size_t smem;
};

// `epi`: aria::EpiMode. A gated tile holds 64 channels of either projection,
// so its plan is that of a GEMM with 2 N weight rows.
aria_status plan_gemm(int kind, int epi, int64_t M, int64_t N, int64_t K, Plan* out) {
  using namespace aria;
  const DevInfo di = dev_info();
  GemmParams p{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  const int unitK = kind == kQ4 ? 256 : (kind == kF16 ? 64 : 128);
  p.units = static_cast<int>((K + unitK - 1) / unitK);

  // Token tile: up to 256. W8A8 at M <= 512 uses narrower tiles (<= 160):
  // more output tiles fill the SMs, and without a dequant stage the per-tile
  // cost of a narrower MMA is small (measured: 15-25 % faster at M = 432).
  int max_bn = 256;
  if ((kind == kW8A8 || kind == kS32 || kind == kF16) && M <= 512) max_bn = 160;
#if defined(ARIA_MAX_BN)
  max_bn = ARIA_MAX_BN;  // tuning builds only
#endif
  auto tile_for = [&](int mt_try, int* bn_out) {  // token tile for mt_try token tiles
    int b = static_cast<int>((M + mt_try - 1) / mt_try);
    b = (b + 15) / 16 * 16;
    *bn_out = b;
    return static_cast<int>((M + b - 1) / b);
  };
  int bn = 0;
  int mt = tile_for(static_cast<int>((M + max_bn - 1) / max_bn), &bn);
  const int chans = epi == kEpiGated ? tile_chans<kEpiGated>() : tile_chans<kEpiPlain>();
  const int nt = static_cast<int>((N + chans - 1) / chans);
  // q8/q4 with a few hundred tokens: the dequant work per K block is the
  // same for any token tile, and a split-K launch costs several us of
  // cluster reduction. Measured at M = 432 (d = 1536 linears): prefer the
  // token tile that fills the most SMs (at least two thirds) without split-K;
  // otherwise one tile narrower than the widest when K is short (fewer
  // ranks to reduce), the widest when K is long (less K per rank).
  bool dq_policy = (kind == kQ8 || kind == kQ4) && M >= 128 && M <= 512;
#if defined(ARIA_MAX_BN)
  dq_policy = false;  // tuning builds pin the tile
#endif
  if (dq_policy && epi != kEpiPlain) {
    // The same choice by estimated time (the rule below is tuned to the plain
    // linears; two gated projections have twice the tiles, and where they lie
    // between half and two thirds of the SMs it would halve the token tile
    // into two waves: q8 6144 x 1536 at M = 203 21.6 against 13.5 us). A K
    // block takes about 0.21 us and 0.0009 per token of the tile (0.08 more
    // when the weights go through shared memory), a split-K exchange 1.2 us and
    // 0.014 per token.
    const int mt0 = mt;
    double best = 0.0;
    int best_mt = mt0;
    const double nkb = static_cast<double>((K + 63) / 64);
    for (int m_try = mt0; m_try <= mt0 + 2; ++m_try) {
      int b = 0;
      const int m_eff = tile_for(m_try, &b);
      const int64_t t = static_cast<int64_t>(nt) * m_eff;
      const int64_t s = t < di.sms ? std::min<int64_t>({8, di.sms / t, p.units}) : 1;
      const int64_t waves = (t * s + di.sms - 1) / di.sms;
      const double kb = 0.21 + 0.0009 * b + (t <= di.sms ? 0.0 : 0.08);
      const double us = waves * (nkb / s * kb + 1.0) + (s > 1 ? 1.2 + 0.014 * b : 0.0) + 0.3 * (m_try - mt0);
      if (best == 0.0 || us < best) {
        best = us;
        best_mt = m_try;
      }
    }
    mt = tile_for(best_mt, &bn);
  } else if (dq_policy) {
    const int mt0 = mt;
    int best_mt = 0, best_tiles = 0;
    for (int m_try = mt0; m_try <= mt0 + 2; ++m_try) {
      int b = 0;
      const int m_eff = tile_for(m_try, &b);
      const int64_t t = static_cast<int64_t>(nt) * m_eff;
      if (t <= di.sms && 3 * t >= 2 * static_cast<int64_t>(di.sms) && t > best_tiles) {
        best_tiles = static_cast<int>(t);
        best_mt = m_try;
      }
    }
    if (best_mt == 0) best_mt = K <= 2048 ? mt0 + 1 : mt0;
    mt = tile_for(best_mt, &bn);
  }
  // Many tokens (several tiles per CTA): the persistent CTAs take the tiles
  // round-robin, so the slowest CTA does ceil(tiles / SMs) of them. Pick the
  // token tile (a multiple of 16 in [128, 256]) that minimises that count
  // times the tile's width plus a fixed per-tile cost (16 token-columns'
  // worth), e.g. 176 instead of 256 for N = 1536 at M = 4096: 288 tiles in
  // two nearly full waves instead of 192 in two waves of which one is 30 %
  // full.
  bool wave_policy = M > 512;
#if defined(ARIA_MAX_BN)
  wave_policy = false;  // tuning builds pin the tile
#endif
  if (wave_policy) {
    int64_t best_cost = -1;
    for (int b = 256; b >= 128; b -= 16) {
      const int64_t m_t = (M + b - 1) / b;
      const int64_t waves = (static_cast<int64_t>(nt) * m_t + di.sms - 1) / di.sms;
      const int64_t cost = waves * (b + 16);
      if (best_cost < 0 || cost < best_cost) {
        best_cost = cost;
        bn = b;
        mt = static_cast<int>(m_t);
      }
    }
  }
  // W8A8 with few weight-row tiles and a short K: the narrowest token tile
  // that still leaves at least two thirds of the SMs busy without split-K
  // (measured at M = 432, N = K = 1536: 48-token tiles 6.8 us against 9.3 us
  // for 144-token tiles in 3-way split-K clusters; at K = 6144 the split
  // stays faster)
  bool narrow_policy = kind == kW8A8 && M <= 512 && K <= 2048 && static_cast<int64_t>(nt) * mt < di.sms;
#if defined(ARIA_MAX_BN)
  narrow_policy = false;  // tuning builds pin the tile
#endif
  if (narrow_policy) {
    for (int b = bn - 16; b >= 48; b -= 16) {
      const int64_t m_t = (M + b - 1) / b;
      const int64_t t = static_cast<int64_t>(nt) * m_t;
      if (t > di.sms) break;
      if (3 * t >= 2 * static_cast<int64_t>(di.sms)) {
        bn = b;
        mt = static_cast<int>(m_t);
        break;
      }
    }
  }
  p.BN = bn;
  const int64_t tiles = static_cast<int64_t>(nt) * mt;
  if (tiles > (int64_t{1} << 30)) return fail(ARIA_ERR_UNSUPPORTED, "too many tiles");
  p.tiles_n = nt;
  p.tiles = static_cast<int>(tiles);

  // split-K upper bound; the launcher lowers it until the clusters fit in one wave
  int splits = 1;
  if (tiles < di.sms) splits = static_cast<int>(std::min<int64_t>(8, di.sms / tiles));
  splits = std::max(1, std::min(splits, p.units));
#if defined(ARIA_FORCE_SPLITS)
  splits = std::max(1, std::min(std::min(ARIA_FORCE_SPLITS, p.units), static_cast<int>(di.sms / tiles)));  // tuning builds only
#endif
  p.splits = splits;

  const bool dq = (kind == kQ8 || kind == kQ4);
  // q8/q4 with one tile per CTA (every split-K CTA has one too): the A
  // operand lives in tensor memory, so a stage holds only the activation
  // tile; the ring depth stays <= 8 (8 A slots of 32 TMEM columns)
  const bool ta = dq && tiles <= di.sms;
  p.tmem_a = ta ? 1 : 0;
  const uint32_t a_tile = ta ? 0u : kATile;
  const uint32_t out_bytes = kind == kS32 ? 4 : 2;
  const uint32_t epi_warps = dq ? 4 : 8;
  const uint32_t stage_bytes = epi_warps * warp_stage(epi, out_bytes);
  const uint32_t sxd_bytes = 2 * aria::kTileBnMax * 4;  // W8A8 token scales, two m-tiles
  p.x_stage = static_cast<uint32_t>(bn) * 128u;
  p.raw_stage = kind == kQ8 ? kATile : (kind == kQ4 ? kATile + kQ4ScaleTile : 0);
  p.raw_stage = (p.raw_stage + 1023u) & ~1023u;
  const int64_t budget = static_cast<int64_t>(di.smem_optin) - 1024 - 512 - stage_bytes - sxd_bytes;
  // stage ring: one A tile + one X tile per stage (one MMA commit each);
  // q8/q4 also keep a ring of raw packed weight tiles for the dequant warps
  int nr = 0, na = 0, nx = 0;
  const int64_t st_bytes = a_tile + p.x_stage;
  int k_max = 8;
#if defined(ARIA_MAX_STAGES)
  k_max = ARIA_MAX_STAGES;  // tuning builds only
#endif
  for (int k = k_max; k >= 2 && na == 0; --k) {
    if (!dq) {
      if (k * st_bytes <= budget) na = k;
      continue;
    }
    for (int r = 4; r >= 2; --r)
      if (k * st_bytes + static_cast<int64_t>(r) * p.raw_stage <= budget) {
        na = k;
        nr = r;
        break;
      }
  }
  if (na == 0) return fail(ARIA_ERR_UNSUPPORTED, "tile does not fit in shared memory");
  nx = na;
  p.n_raw = nr;
  p.n_a = na;
  p.n_x = nx;
  p.off_raw = 0;
  p.off_a = p.off_raw + nr * p.raw_stage;
  p.off_x = p.off_a + na * a_tile;
  p.off_stage = p.off_x + nx * p.x_stage;
  p.off_sxd = p.off_stage + stage_bytes;
  p.off_bar = p.off_sxd + sxd_bytes;
  // the split-K partial tile (BN rows x 512 B) overlays the stage rings
  if (static_cast<uint32_t>(bn) * 512u > p.off_stage) p.splits = splits = 1;
  // warps 0..3 help with the last tile's epilogue when their store boxes (and
  // W8A8 token scales) fit in the activation ring
  const uint64_t helper_bytes = 4ull * warp_stage(epi, out_bytes) + 4ull * kTileBnMax;
  p.helpers = static_cast<uint64_t>(nx) * p.x_stage >= helper_bytes ? 1 : 0;
  const uint32_t nbar = 2 * (nr + na) + 6;  // raw, stage, 2 acc_full, 2 acc_empty, mma_drain, acc_last
  const size_t smem = 1024 + p.off_bar + nbar * 8 + 16;
  if (smem > static_cast<size_t>(di.smem_optin)) return fail(ARIA_ERR_UNSUPPORTED, "shared memory plan too large");

  out->p = p;
  out->grid = dim3(static_cast<unsigned>(std::min<int64_t>(tiles, di.sms)), 1, 1);
  out->threads = 384;
  out->smem = smem;
  return ARIA_OK;
}

// Trace builds: each GEMM launch gets the next trace row block (see
// ARIA_STAMP); 0 otherwise.
#ifdef ARIA_TRACE
std::atomic<int> g_trace_launches{0};
int next_trace_launch() { return g_trace_launches.fetch_add(1); }
#else
int next_trace_launch() { return 0; }
#endif

// programmatic dependent launch: the kernel may start while the previous
// kernel in the stream drains; it waits (griddepcontrol.wait) before reading
// anything that kernel may write (the weights of aria_qgemm and the packed
// weights of the feed-forward operators are the one exception, see the
// stream-order note of aria_qgemm in the header)
void set_pdl(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* attr) {
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs++;
  cfg.attrs = attr;
}

// how many clusters of `size` CTAs of this kernel can be resident at once on
// the current device (cached per device, size and shared-memory footprint;
// queried outside any capture on first use)
template <int KIND, int EPI>
int max_clusters(int size, int threads, size_t smem) {
  static std::mutex mu;
  static int cache_dev[64], cache_size[64], cache_n[64];
  static size_t cache_smem[64];
  static int used = 0;
  const int dev = current_device();
  std::lock_guard<std::mutex> g(mu);
  for (int i = 0; i < used; ++i)
    if (cache_dev[i] == dev && cache_size[i] == size && cache_smem[i] == smem) return cache_n[i];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(size, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, aria::qgemm_kernel<KIND, EPI>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (used < 64) {
    cache_dev[used] = dev;
    cache_size[used] = size;
    cache_smem[used] = smem;
    cache_n[used] = n;
    ++used;
  }
  return n;
}

// Raise a kernel's dynamic shared-memory limit to the device's opt-in
// maximum, once per kernel and device (the attribute is per device).
template <typename F>
aria_status opt_in_smem(F* kfn, bool (&done)[kMaxDevices], std::mutex& mu) {
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return fail(ARIA_ERR_UNSUPPORTED, "device index %d", dev);
  std::lock_guard<std::mutex> g(mu);
  if (done[dev]) return ARIA_OK;
  cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       dev_info().smem_optin);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  done[dev] = true;
  return ARIA_OK;
}

template <int KIND, int EPI = aria::kEpiPlain>
aria_status launch_gemm(const Plan& pl, const CUtensorMap& tw, const CUtensorMap& ts,
                        const CUtensorMap& tx, cudaStream_t st,
                        const aria::GatedMaps<EPI>& tu = aria::GatedMaps<EPI>{}) {
  auto kfn = aria::qgemm_kernel<KIND, EPI>;
  static bool attr_done[kMaxDevices] = {};
  static std::mutex attr_mu;
  aria_status as = opt_in_smem(kfn, attr_done, attr_mu);
  if (as != ARIA_OK) return as;
  aria::GemmParams prm = pl.p;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = pl.grid;
  cfg.blockDim = dim3(pl.threads, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = 0;
  // largest split whose clusters are all co-resident (one wave)
  while (prm.splits > 1 && max_clusters<KIND, EPI>(prm.splits, pl.threads, pl.smem) < prm.tiles) --prm.splits;
  if (prm.splits > 1) {
    cfg.gridDim = dim3(prm.splits, prm.tiles, 1);
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = prm.splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    cfg.attrs = attr;
  }
  set_pdl(cfg, attr);
  prm.trace_launch = next_trace_launch();
  cudaError_t e = cudaLaunchKernelEx(&cfg, kfn, tw, ts, tx, prm, tu);
  if (e != cudaSuccess) return cuda_fail(e, "qgemm launch");
  return ARIA_OK;
}

// ------------------------------------------------------------- few tokens ---
// Plan of the few-token weight-only GEMM (smallm_kernel): the smallest
// cluster size S (K split) that keeps each warp's activation chunks in
// registers and the activations read per CTA at or below 32 KB, with the
// rows divided over as many clusters as the SMs hold. False when no plan
// fits (then the tensor-core kernel runs).
struct SmallPlan {
  aria::SmallParams p;
  int grid = 0, tb = 1, ch = 8;
  size_t smem = 0;
};

constexpr int64_t kSmallMaxTokens = 16;
constexpr size_t kSmallSmemBudget = 110 * 1024;  // two CTAs per SM
constexpr size_t kSmallSmemMost = 220 * 1024;    // one

template <int KIND, int TB, int CH, int GP, int EPI>
int small_max_clusters(int size, size_t smem) {
  static std::mutex mu;
  static int cache_dev[64], cache_size[64], cache_n[64];
  static size_t cache_smem[64];
  static int used = 0;
  const int dev = current_device();
  std::lock_guard<std::mutex> g(mu);
  for (int i = 0; i < used; ++i)
    if (cache_dev[i] == dev && cache_size[i] == size && cache_smem[i] == smem) return cache_n[i];
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(size, 1, 1);
  cfg.blockDim = dim3(aria::kSmThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, aria::smallm_kernel<KIND, TB, CH, GP, EPI>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  if (used < 64) {
    cache_dev[used] = dev;
    cache_size[used] = size;
    cache_smem[used] = smem;
    cache_n[used] = n;
    ++used;
  }
  return n;
}

// shared-memory layout of a plan with `clusters` clusters of S CTAs
// (`rpc` weight rows per output channel: 2 for the gated epilogue)
bool small_layout(int kind, int64_t M, int64_t N, int64_t K, int S, int clusters, int tb, int gp, int rpc,
                  aria::SmallParams* p, size_t* smem) {
  using namespace aria;
  const int num = kind == kF16 ? 2 : 1, den = kind == kQ4 ? 2 : 1;
  p->S = S;
  p->kslice = static_cast<int>(K / S);
  p->rows_base = static_cast<int>(N / clusters);
  p->rows_rem = static_cast<int>(N % clusters);
  const int rmax = (p->rows_base + (p->rows_rem ? 1 : 0)) * rpc;
  p->r_pad = (rmax + 15) / 16 * 16;
  const uint32_t slice = static_cast<uint32_t>(p->kslice) * num / den;
  p->wrow = slice + 16;
  auto up = [](uint64_t v, uint64_t a) { return (v + a - 1) / a * a; };
  uint64_t off = up(static_cast<uint64_t>(rmax) * p->wrow, 128);
  p->off_sc = static_cast<uint32_t>(off);
  if (kind == kQ4) off = up(off + static_cast<uint64_t>(rmax) * (p->kslice / 16), 128);
  p->off_red = static_cast<uint32_t>(off);
  off += static_cast<uint64_t>(kSmWarps) * tb * 8 * sm_red_stride(gp) * 4;
  p->off_part = static_cast<uint32_t>(up(off, 128));
  off = p->off_part + (S > 1 ? static_cast<uint64_t>(tb) * 8 * (p->r_pad + 4) * 4 : 0);
  p->off_bar = static_cast<uint32_t>(up(off, 16));
  p->off_sw = p->off_bar + 16;  // q8 channel scales of the rows
  *smem = p->off_sw + static_cast<uint64_t>(rmax) * 4;
  (void)M;
  // Two CTAs per SM: the next launch's weights stream beside this one. The
  // gated operator's weights may be too many for that and still stream faster
  // one CTA per SM than through the tensor-core kernel (q8, 6144 x 1536, one
  // token: 6.0 against 10.1 us), up to 8 tokens (16 tokens, 1536 x 6144: 11.8
  // against 11.5).
  return *smem <= (rpc == 2 && tb == 1 ? kSmallSmemMost : kSmallSmemBudget);
}

template <int KIND, int TB, int CH, int GP, int EPI>
bool plan_small_t(int64_t M, int64_t N, int64_t K, SmallPlan* out) {
  using namespace aria;
  const DevInfo di = dev_info();
  const int unit = KIND == kQ4 ? 256 : 64;
  constexpr int rpc = EPI == kEpiGated ? 2 : 1;
  if (K % unit) return false;
  int best_s = 0;
  for (int S = 1; S <= 8; ++S) {
    if (K % (static_cast<int64_t>(S) * unit)) continue;
    const int64_t kslice = K / S;
    if ((kslice / 64 + kSmWarps - 1) / kSmWarps > CH) continue;  // activation chunks in registers
    best_s = S;
    if (M * kslice * 2 <= 32768) break;  // activations read per CTA: small enough
  }
  if (best_s == 0) return false;
  const int S = best_s;
  int clusters = static_cast<int>(std::min<int64_t>(di.sms / S, N));
  SmallParams p{};
  size_t smem = 0;
  if (!small_layout(KIND, M, N, K, S, clusters, TB, GP, rpc, &p, &smem)) return false;
  if (S > 1) {
    const int fit = small_max_clusters<KIND, TB, CH, GP, EPI>(S, smem);
    if (fit < 1) return false;
    if (fit < clusters) {
      clusters = fit;
      if (!small_layout(KIND, M, N, K, S, clusters, TB, GP, rpc, &p, &smem)) return false;
    }
  }
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  out->p = p;
  out->grid = clusters * S;
  out->tb = TB;
  out->ch = CH;
  out->smem = smem;
  return true;
}

// 16-row groups per pass for one token block: a gated channel has two rows
template <int EPI>
constexpr int small_groups() { return EPI == aria::kEpiGated ? 6 : 4; }

template <int EPI>
bool plan_small(int kind, int64_t M, int64_t N, int64_t K, SmallPlan* out) {
  using namespace aria;
  if (M > kSmallMaxTokens) return false;
  const bool two = M > 8;
  constexpr int gp = small_groups<EPI>();
  switch (kind) {
    case kQ8: return two ? plan_small_t<kQ8, 2, 4, 2, EPI>(M, N, K, out) : plan_small_t<kQ8, 1, 6, gp, EPI>(M, N, K, out);
    case kQ4: return two ? plan_small_t<kQ4, 2, 4, 2, EPI>(M, N, K, out) : plan_small_t<kQ4, 1, 6, gp, EPI>(M, N, K, out);
    case kF16: return two ? plan_small_t<kF16, 2, 4, 2, EPI>(M, N, K, out) : plan_small_t<kF16, 1, 6, gp, EPI>(M, N, K, out);
  }
  return false;
}

template <int KIND, int TB, int CH, int GP, int EPI>
aria_status launch_small_t(const SmallPlan& pl, cudaStream_t st) {
  auto kfn = aria::smallm_kernel<KIND, TB, CH, GP, EPI>;
  static bool attr_done[kMaxDevices] = {};
  static std::mutex attr_mu;
  aria_status as = opt_in_smem(kfn, attr_done, attr_mu);
  if (as != ARIA_OK) return as;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(pl.grid), 1, 1);
  cfg.blockDim = dim3(aria::kSmThreads, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.numAttrs = 0;
  if (pl.p.S > 1) {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = pl.p.S;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    cfg.attrs = attr;
  }
  set_pdl(cfg, attr);
  aria::SmallParams sp = pl.p;
  sp.trace_launch = next_trace_launch();
  cudaError_t e = cudaLaunchKernelEx(&cfg, kfn, sp);
  if (e != cudaSuccess) return cuda_fail(e, "few-token GEMM launch");
  return ARIA_OK;
}

template <int KIND, int EPI>
aria_status launch_small_kind(const SmallPlan& pl, cudaStream_t st) {
  return pl.tb == 2 ? launch_small_t<KIND, 2, 4, 2, EPI>(pl, st)
                    : launch_small_t<KIND, 1, 6, small_groups<EPI>(), EPI>(pl, st);
}

template <int EPI>
aria_status launch_small(int kind, const SmallPlan& pl, cudaStream_t st) {
  using namespace aria;
  switch (kind) {
    case kQ8: return launch_small_kind<kQ8, EPI>(pl, st);
    case kQ4: return launch_small_kind<kQ4, EPI>(pl, st);
    case kF16: return launch_small_kind<kF16, EPI>(pl, st);
  }
  return fail(ARIA_ERR_INVALID_ARG, "unknown kind");
}

aria_status check_gemm_shape(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return fail(ARIA_ERR_INVALID_ARG, "sizes must be positive and < 2^31 (M=%lld N=%lld K=%lld)",
                (long long)M, (long long)N, (long long)K);
  if (N < 16 || N % 16) return fail(ARIA_ERR_UNSUPPORTED, "N must be a positive multiple of 16");
  if (K < 16 || K % 16) return fail(ARIA_ERR_UNSUPPORTED, "K must be a positive multiple of 16");
  return ARIA_OK;
}

}  // namespace

// ================================================================= ABI ===

ARIA_API const char* aria_status_string(aria_status s) {
  switch (s) {
    case ARIA_OK: return "ARIA_OK";
    case ARIA_ERR_INVALID_ARG: return "ARIA_ERR_INVALID_ARG";
    case ARIA_ERR_UNSUPPORTED: return "ARIA_ERR_UNSUPPORTED";
    case ARIA_ERR_MISALIGNED: return "ARIA_ERR_MISALIGNED";
    case ARIA_ERR_CUDA: return "ARIA_ERR_CUDA";
    case ARIA_ERR_TIMEOUT: return "ARIA_ERR_TIMEOUT";
  }
  return "ARIA_ERR_UNKNOWN";
}

ARIA_API const char* aria_last_error_message(void) { return g_msg; }

ARIA_API aria_status aria_qpack_size(aria_format fmt, int group, int64_t N, int64_t K,
                                     size_t* wq_bytes, size_t* scale_bytes) {
  if (!wq_bytes || !scale_bytes) return fail(ARIA_ERR_INVALID_ARG, "NULL output pointer");
  if (N < 1 || K < 1 || N > kMaxDim || K > kMaxDim)
    return fail(ARIA_ERR_INVALID_ARG, "N and K must be in [1, 2^31)");
  if (fmt == ARIA_FMT_Q8 || fmt == ARIA_FMT_W8A8) {
    if (group != 0) return fail(ARIA_ERR_UNSUPPORTED, "q8 scales are per output channel: group must be 0");
    *wq_bytes = static_cast<size_t>(N) * K;
    *scale_bytes = static_cast<size_t>(N) * 4;
    return ARIA_OK;
  }
  if (fmt == ARIA_FMT_F16)
    return fail(ARIA_ERR_UNSUPPORTED, "fp16 weights are used as they are, not packed");
  if (fmt == ARIA_FMT_Q4) {
    if (group != 32) return fail(ARIA_ERR_UNSUPPORTED, "q4 supports group = 32 only");
    if (K % 32) return fail(ARIA_ERR_UNSUPPORTED, "q4 needs K % 32 == 0");
    *wq_bytes = static_cast<size_t>(N) * (K / 2);
    *scale_bytes = static_cast<size_t>(N) * (K / 32) * 2;
    return ARIA_OK;
  }
  return fail(ARIA_ERR_INVALID_ARG, "unknown format %d", (int)fmt);
}

ARIA_API aria_status aria_qpack(aria_format fmt, int group, const void* W, int64_t N, int64_t K,
                                void* Wq, void* scales, void* stream) {
  size_t wb = 0, sb = 0;
  aria_status s = aria_qpack_size(fmt, group, N, K, &wb, &sb);
  if (s != ARIA_OK) return s;
  if (!W || !Wq || !scales) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  if (!aligned16(W) || !aligned16(Wq) || !aligned16(scales))
    return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.stream = st;
  set_pdl(cfg, attr);
  cudaError_t e;
  if (fmt == ARIA_FMT_Q4) {
    const int64_t nchunk = N * (K / 8);
    const int64_t blocks = std::min<int64_t>((nchunk + 255) / 256, int64_t{dev_info().sms} * 16);
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(256);
    e = cudaLaunchKernelEx(&cfg, aria::pack_q4_kernel, static_cast<const __half*>(W), nchunk,
                           static_cast<uint32_t*>(Wq), static_cast<__half*>(scales));
  } else {
    if (K % 16) return fail(ARIA_ERR_UNSUPPORTED, "q8 needs K % 16 == 0");
    cfg.gridDim = dim3(static_cast<unsigned>(N));
    cfg.blockDim = dim3(aria::kRowThreads);
    e = cudaLaunchKernelEx(&cfg, aria::row_quant_i8_kernel, static_cast<const __half*>(W),
                           static_cast<int>(K), static_cast<int8_t*>(Wq), static_cast<float*>(scales),
                           false);
  }
  if (e != cudaSuccess) return cuda_fail(e, "pack launch");
  return ARIA_OK;
}

ARIA_API aria_status aria_act_quant(const void* X, int64_t M, int64_t K, int8_t* Xq, float* sx,
                                    void* stream) {
  if (!X || !Xq || !sx) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  if (M < 1 || K < 1 || M > kMaxDim || K > kMaxDim)
    return fail(ARIA_ERR_INVALID_ARG, "M and K must be in [1, 2^31)");
  if (K % 16) return fail(ARIA_ERR_UNSUPPORTED, "K must be a multiple of 16");
  if (!aligned16(X) || !aligned16(Xq) || !aligned16(sx))
    return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.gridDim = dim3(static_cast<unsigned>(M));
  cfg.blockDim = dim3(aria::kRowThreads);
  set_pdl(cfg, attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, aria::row_quant_i8_kernel, static_cast<const __half*>(X),
                                     static_cast<int>(K), Xq, sx, true);
  if (e != cudaSuccess) return cuda_fail(e, "act_quant launch");
  return ARIA_OK;
}

// Workspace of the fused W8A8 call: [0, 256) the grid barrier {arrivals,
// generation}; then the token scales fp32 [M]; then the codes int8 [M,K], at
// 256-byte aligned offsets (TMA reads the codes).
struct FusedWs {
  unsigned* gbar;
  float* sx;
  int8_t* xq;
};

constexpr size_t kWsHeader = 256;

size_t fused_ws_bytes(int64_t M, int64_t K) {
  const size_t sx = (static_cast<size_t>(M) * 4 + 255) / 256 * 256;
  return kWsHeader + sx + static_cast<size_t>(M) * static_cast<size_t>(K);
}

FusedWs fused_ws(void* ws, int64_t M) {
  uint8_t* b = static_cast<uint8_t*>(ws);
  const size_t sx = (static_cast<size_t>(M) * 4 + 255) / 256 * 256;
  return FusedWs{reinterpret_cast<unsigned*>(b), reinterpret_cast<float*>(b + kWsHeader),
                 reinterpret_cast<int8_t*>(b + kWsHeader + sx)};
}

// the failure-detection self-test's settings of a launch (defaults: none)
struct SelfTest {
  uint64_t wait_ns = 0;
  int drop_first_stage = 0;
};

// what the kEpiAct and kEpiGated epilogues take besides a GEMM's arguments
struct EpiArgs {
  int act = ARIA_ACT_NONE;
  const void* res = nullptr;     // kEpiAct
  const void* Wu = nullptr;      // kEpiGated: the up projection
  const void* scales_u = nullptr;
  const void* bias_u = nullptr;
  void* G = nullptr;             // kEpiGated: the pre-activations
  void* U = nullptr;
  bool w_late = false;           // no weight load before the dependency wait
};

// Whether a feed-forward operator's weights may come from the preceding
// kernel. fp16 weights are ordinary tensors that any kernel may have written
// by ordinary stores (an optimiser's, a cast, a merge of two weights), and a
// call that keeps the pre-activations is a training step's in any format.
// Packed weights otherwise follow aria_qgemm's rule.
static bool weights_late(int kind, const void* kept) { return kind == aria::kF16 || kept; }

static aria_status check_gemm_sizes(int kind, int64_t M, int64_t N, int64_t K) {
  using namespace aria;
  aria_status s = check_gemm_shape(M, N, K);
  if (s != ARIA_OK) return s;
  if (kind == kQ4 && K % 256) return fail(ARIA_ERR_UNSUPPORTED, "q4 GEMM needs K % 256 == 0");
  // exact int32 accumulation: |acc| <= K * 127^2 must stay below 2^31
  if ((kind == kW8A8 || kind == kS32) && K * 127 * 127 > INT32_MAX)
    return fail(ARIA_ERR_UNSUPPORTED, "int8 GEMM needs K * 127^2 < 2^31 (K <= %lld), got K=%lld",
                (long long)(INT32_MAX / (127 * 127)), (long long)K);
  return ARIA_OK;
}

// a weight's tensor maps: `rows` rows of 128 packed bytes (fp16: of 64
// elements) per box, and for q4 the group scales
static aria_status weight_maps(int kind, const void* W, const void* scales, int64_t N, int64_t K, int rows,
                               CUtensorMap* tw, CUtensorMap* ts) {
  using namespace aria;
  aria_status s;
  if (kind == kQ4) {
    if ((s = make_map(tw, W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K / 2, 128, rows,
                      CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK) return s;
    return make_map(ts, scales, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, N, K / 32, 8, rows,
                    CU_TENSOR_MAP_SWIZZLE_NONE);
  }
  if (kind == kF16)
    return make_map(tw, W, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, N, K, 64, rows, CU_TENSOR_MAP_SWIZZLE_128B);
  return make_map(tw, W, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, N, K, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int EPI>
static aria_status qgemm_impl(int kind, int64_t M, int64_t N, int64_t K, const void* X,
                              const float* sx, const void* Wq, const void* scales,
                              const void* bias, const float* steer, float alpha,
                              const float* alpha_dev, void* Y, cudaStream_t st, const EpiArgs& ea,
                              const void* xf16 = nullptr, const FusedWs* ws = nullptr,
                              const SelfTest& selftest = SelfTest{}) {
  using namespace aria;
  aria_status s = check_gemm_sizes(kind, M, N, K);
  if (s != ARIA_OK) return s;
  // a handful of tokens: the weight-streaming kernel, when its plan fits
  SmallPlan sp;
  if (!xf16 && !selftest.drop_first_stage && plan_small<EPI>(kind, M, N, K, &sp)) {
    sp.p.W = static_cast<const uint8_t*>(Wq);
    sp.p.Wsc = kind == kQ4 ? static_cast<const __half*>(scales) : nullptr;
    sp.p.sw = kind == kQ8 ? static_cast<const float*>(scales) : nullptr;
    sp.p.X = static_cast<const __half*>(X);
    sp.p.bias = static_cast<const __half*>(bias);
    sp.p.steer = (steer && (alpha_dev || alpha != 0.0f)) ? steer : nullptr;
    sp.p.alpha = sp.p.steer ? alpha : 0.0f;
    sp.p.alpha_dev = sp.p.steer ? alpha_dev : nullptr;
    sp.p.Y = static_cast<__half*>(Y);
    sp.p.w_late = ea.w_late;
    sp.p.act = ea.act;
    sp.p.res = static_cast<const __half*>(ea.res);
    sp.p.W_u = static_cast<const uint8_t*>(ea.Wu);
    sp.p.Wsc_u = kind == kQ4 ? static_cast<const __half*>(ea.scales_u) : nullptr;
    sp.p.sw_u = kind == kQ8 ? static_cast<const float*>(ea.scales_u) : nullptr;
    sp.p.bias_u = static_cast<const __half*>(ea.bias_u);
    sp.p.G = static_cast<__half*>(ea.G);
    sp.p.U = static_cast<__half*>(ea.U);
    return launch_small<EPI>(kind, sp, st);
  }
  Plan pl;
  if ((s = plan_gemm(kind, EPI, M, N, K, &pl)) != ARIA_OK) return s;
  CUtensorMap tw, ts, tx;
  std::memset(&ts, 0, sizeof(ts));
  const int bn = pl.p.BN;
  GatedMaps<EPI> tu;
  const int wrows = tile_chans<EPI>();
  if ((s = weight_maps(kind, Wq, scales, N, K, wrows, &tw, &ts)) != ARIA_OK) return s;
  if constexpr (EPI == kEpiGated) {
    std::memset(&tu, 0, sizeof(tu));
    if ((s = weight_maps(kind, ea.Wu, ea.scales_u, N, K, wrows, &tu.W, &tu.S)) != ARIA_OK) return s;
  }
  if (kind == kQ8 || kind == kQ4 || kind == kF16) {
    if ((s = make_map(&tx, X, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, M, K, 64, bn,
                      CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK) return s;
  } else {
    if ((s = make_map(&tx, X, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, M, K, 128, bn,
                      CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK) return s;
  }
  pl.p.sw = static_cast<const float*>((kind == kQ4 || kind == kF16) ? nullptr : scales);
  pl.p.sx = sx;
  pl.p.bias = static_cast<const __half*>(bias);
  // skip, not "+ 0*v": a host alpha of 0 drops the vector here; a device
  // alpha is tested in the kernel
  pl.p.steer = (steer && (alpha_dev || alpha != 0.0f)) ? steer : nullptr;
  pl.p.alpha = pl.p.steer ? alpha : 0.0f;
  pl.p.alpha_dev = pl.p.steer ? alpha_dev : nullptr;
  pl.p.Y = Y;
  pl.p.wait_ns = selftest.wait_ns;
  pl.p.drop_first_stage = selftest.drop_first_stage;
  if (xf16) {  // W8A8 with the activation quantisation in this launch
    pl.p.xf16 = static_cast<const __half*>(xf16);
    pl.p.xq_ws = ws->xq;
    pl.p.sx_ws = ws->sx;
    pl.p.gbar = ws->gbar;
    pl.p.sx = ws->sx;
  }
  pl.p.w_late = ea.w_late;
  pl.p.act = ea.act;
  pl.p.res = static_cast<const __half*>(ea.res);
  pl.p.sw_u = static_cast<const float*>((kind == kQ4 || kind == kF16) ? nullptr : ea.scales_u);
  pl.p.bias_u = static_cast<const __half*>(ea.bias_u);
  pl.p.G = static_cast<__half*>(ea.G);
  pl.p.U = static_cast<__half*>(ea.U);
  switch (kind) {
    case kQ8: return launch_gemm<kQ8, EPI>(pl, tw, tw, tx, st, tu);
    case kQ4: return launch_gemm<kQ4, EPI>(pl, tw, ts, tx, st, tu);
    case kW8A8: return launch_gemm<kW8A8, EPI>(pl, tw, tw, tx, st, tu);
    case kF16: return launch_gemm<kF16, EPI>(pl, tw, tw, tx, st, tu);
  }
  if constexpr (EPI == kEpiPlain) {
    if (kind == kS32) return launch_gemm<kS32>(pl, tw, tw, tx, st);
  }
  return fail(ARIA_ERR_INVALID_ARG, "unknown kind");
}

// argument checks shared by aria_qgemm and aria_qgemm_steer_dev; sets *kind
static aria_status check_qgemm_args(aria_format fmt, int group, const void* X, const float* sx,
                                    const void* Wq, const void* scales, const void* bias,
                                    const float* steer_vec, const void* Y, int* kind) {
  if (!X || !Wq || !Y) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  if (fmt == ARIA_FMT_Q8 || fmt == ARIA_FMT_W8A8) {
    if (group != 0) return fail(ARIA_ERR_UNSUPPORTED, "q8 scales are per output channel: group must be 0");
    *kind = fmt == ARIA_FMT_Q8 ? aria::kQ8 : aria::kW8A8;
  } else if (fmt == ARIA_FMT_Q4) {
    if (group != 32) return fail(ARIA_ERR_UNSUPPORTED, "q4 supports group = 32 only");
    *kind = aria::kQ4;
  } else if (fmt == ARIA_FMT_F16) {
    if (group != 0) return fail(ARIA_ERR_UNSUPPORTED, "fp16 weights have no groups: group must be 0");
    *kind = aria::kF16;
  } else {
    return fail(ARIA_ERR_INVALID_ARG, "unknown format %d", (int)fmt);
  }
  if (*kind == aria::kF16) {
    if (scales) return fail(ARIA_ERR_INVALID_ARG, "fp16 weights take no scales (pass NULL)");
  } else if (!scales) {
    return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  }
  if (*kind == aria::kW8A8 && !sx) return fail(ARIA_ERR_INVALID_ARG, "W8A8 needs sx");
  if (*kind != aria::kW8A8 && sx) return fail(ARIA_ERR_INVALID_ARG, "sx is for W8A8 only");
  for (const void* q : {X, static_cast<const void*>(sx), Wq, scales, bias,
                        static_cast<const void*>(steer_vec), Y})
    if (q && !aligned16(q)) return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  return ARIA_OK;
}

ARIA_API aria_status aria_qgemm(aria_format fmt, int group, int64_t M, int64_t N, int64_t K,
                                const void* X, const float* sx, const void* Wq, const void* scales,
                                const void* bias, const float* steer_vec, float alpha, void* Y,
                                void* stream) {
  int kind = 0;
  aria_status s = check_qgemm_args(fmt, group, X, sx, Wq, scales, bias, steer_vec, Y, &kind);
  if (s != ARIA_OK) return s;
  return qgemm_impl<aria::kEpiPlain>(kind, M, N, K, X, sx, Wq, scales, bias, steer_vec, alpha, nullptr, Y,
                                     static_cast<cudaStream_t>(stream), EpiArgs{});
}

ARIA_API aria_status aria_qgemm_steer_dev(aria_format fmt, int group, int64_t M, int64_t N,
                                          int64_t K, const void* X, const float* sx,
                                          const void* Wq, const void* scales, const void* bias,
                                          const float* steer_vec, const float* alpha_dev, void* Y,
                                          void* stream) {
  int kind = 0;
  aria_status s = check_qgemm_args(fmt, group, X, sx, Wq, scales, bias, steer_vec, Y, &kind);
  if (s != ARIA_OK) return s;
  if (steer_vec && !alpha_dev)
    return fail(ARIA_ERR_INVALID_ARG, "a steering vector needs a device alpha");
  if (alpha_dev && (reinterpret_cast<uintptr_t>(alpha_dev) & 3u))
    return fail(ARIA_ERR_MISALIGNED, "alpha_dev must be 4-byte aligned");
  return qgemm_impl<aria::kEpiPlain>(kind, M, N, K, X, sx, Wq, scales, bias, steer_vec, 0.0f, alpha_dev, Y,
                                     static_cast<cudaStream_t>(stream), EpiArgs{});
}

ARIA_API aria_status aria_w8a8_workspace_size(int64_t M, int64_t K, size_t* bytes) {
  if (!bytes) return fail(ARIA_ERR_INVALID_ARG, "NULL output pointer");
  if (M < 1 || K < 1 || M > kMaxDim || K > kMaxDim)
    return fail(ARIA_ERR_INVALID_ARG, "M and K must be in [1, 2^31)");
  *bytes = fused_ws_bytes(M, K);
  return ARIA_OK;
}

ARIA_API aria_status aria_qgemm_w8a8_fused(int64_t M, int64_t N, int64_t K, const void* X,
                                           const void* Wq, const float* sw, const void* bias,
                                           const float* steer_vec, float alpha,
                                           const float* alpha_dev, void* Y, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (!X || !Wq || !sw || !Y || !workspace) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  for (const void* q : {X, static_cast<const void*>(Wq), static_cast<const void*>(sw), bias,
                        static_cast<const void*>(steer_vec), static_cast<const void*>(Y)})
    if (q && !aligned16(q)) return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ARIA_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
  if (alpha_dev && (reinterpret_cast<uintptr_t>(alpha_dev) & 3u))
    return fail(ARIA_ERR_MISALIGNED, "alpha_dev must be 4-byte aligned");
  aria_status s = check_gemm_shape(M, N, K);
  if (s != ARIA_OK) return s;
  if (workspace_bytes < fused_ws_bytes(M, K))
    return fail(ARIA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes,
                fused_ws_bytes(M, K));
  const FusedWs ws = fused_ws(workspace, M);
  return qgemm_impl<aria::kEpiPlain>(aria::kW8A8, M, N, K, ws.xq, ws.sx, Wq, sw, bias, steer_vec, alpha, alpha_dev, Y,
                                     static_cast<cudaStream_t>(stream), EpiArgs{}, X, &ws);
}

// ------------------------------------------------- no-allocation variant ---
// Scratch of aria_qgemm_w8a8_fused_noalloc: a file-scope device array that
// every GPU loading this library holds until the process exits. Host code
// must not pass the symbol itself to a kernel (on the host it names a
// stand-in, not device memory): its device address comes from
// cudaGetSymbolAddress, once per device, with that device current.
constexpr size_t kNoAllocScratchBytes = size_t{32} << 20;  // 32 MiB
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

static aria_status noalloc_scratch(void** out) {
  static void* addr[kMaxDevices] = {};
  static std::mutex mu;
  const int dev = current_device();
  if (dev < 0 || dev >= kMaxDevices) return fail(ARIA_ERR_UNSUPPORTED, "device index %d", dev);
  std::lock_guard<std::mutex> g(mu);
  if (!addr[dev]) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetSymbolAddress of the static scratch");
    addr[dev] = p;
  }
  *out = addr[dev];
  return ARIA_OK;
}

ARIA_API aria_status aria_qgemm_w8a8_fused_noalloc(int64_t M, int64_t N, int64_t K, const void* X,
                                                   const void* Wq, const float* sw, const void* bias,
                                                   const float* steer_vec, float alpha,
                                                   const float* alpha_dev, void* Y, void* stream) {
  if (!X || !Wq || !sw || !Y) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  for (const void* q : {X, static_cast<const void*>(Wq), static_cast<const void*>(sw), bias,
                        static_cast<const void*>(steer_vec), static_cast<const void*>(Y)})
    if (q && !aligned16(q)) return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (alpha_dev && (reinterpret_cast<uintptr_t>(alpha_dev) & 3u))
    return fail(ARIA_ERR_MISALIGNED, "alpha_dev must be 4-byte aligned");
  aria_status s = check_gemm_shape(M, N, K);
  if (s != ARIA_OK) return s;
  const size_t need = fused_ws_bytes(M, K);
  if (need > kNoAllocScratchBytes)
    return fail(ARIA_ERR_UNSUPPORTED,
                "M=%lld K=%lld needs %zu bytes of scratch; the static scratch holds %zu "
                "(256 + 4*M rounded up to 256 + M*K must fit)",
                (long long)M, (long long)K, need, kNoAllocScratchBytes);
  void* scratch = nullptr;
  if ((s = noalloc_scratch(&scratch)) != ARIA_OK) return s;
  // the grid barrier's words must start at zero; the array keeps whatever
  // the last call left (a call that gave up leaves them non-zero)
  cudaError_t e = cudaMemsetAsync(scratch, 0, kWsHeader, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "clearing the static scratch's barrier");
  const FusedWs ws = fused_ws(scratch, M);
  return qgemm_impl<aria::kEpiPlain>(aria::kW8A8, M, N, K, ws.xq, ws.sx, Wq, sw, bias, steer_vec, alpha, alpha_dev, Y,
                                     static_cast<cudaStream_t>(stream), EpiArgs{}, X, &ws);
}

ARIA_API aria_status aria_qgemm_s32(int64_t M, int64_t N, int64_t K, const int8_t* Xq,
                                    const int8_t* Wq, int32_t* C, void* stream) {
  if (!Xq || !Wq || !C) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(C))
    return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  return qgemm_impl<aria::kEpiPlain>(aria::kS32, M, N, K, Xq, nullptr, Wq, Wq, nullptr, nullptr, 0.0f, nullptr, C,
                                     static_cast<cudaStream_t>(stream), EpiArgs{});
}

ARIA_API aria_status aria_selftest_bounded_wait(int64_t M, int64_t N, int64_t K, const int8_t* Xq,
                                               const float* sx, const int8_t* Wq, const float* sw,
                                               void* Y, uint32_t wait_limit_us, void* stream) {
  if (!Xq || !sx || !Wq || !sw || !Y) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  for (const void* q : {static_cast<const void*>(Xq), static_cast<const void*>(sx),
                        static_cast<const void*>(Wq), static_cast<const void*>(sw),
                        static_cast<const void*>(Y)})
    if (!aligned16(q)) return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (wait_limit_us < 1 || wait_limit_us > 4000000u)
    return fail(ARIA_ERR_INVALID_ARG, "wait_limit_us must be in [1, 4e6]");
  SelfTest t;
  t.wait_ns = static_cast<uint64_t>(wait_limit_us) * 1000u;
  t.drop_first_stage = 1;
  return qgemm_impl<aria::kEpiPlain>(aria::kW8A8, M, N, K, Xq, sx, Wq, sw, nullptr, nullptr, 0.0f, nullptr, Y,
                                     static_cast<cudaStream_t>(stream), EpiArgs{}, nullptr, nullptr, t);
}

// ------------------------------------------- feed-forward operators ---
namespace {

bool bad_act(int act) { return act < ARIA_ACT_NONE || act > ARIA_ACT_GELU_TANH; }

// [a, a + na) and [b, b + nb) share a byte
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

size_t x_bytes(int kind, int64_t M, int64_t K) {
  return static_cast<size_t>(M) * K * (kind == aria::kW8A8 ? 1 : 2);
}

size_t weight_bytes(int kind, int64_t N, int64_t K) {
  const size_t nk = static_cast<size_t>(N) * K;
  return kind == aria::kF16 ? nk * 2 : kind == aria::kQ4 ? nk / 2 : nk;
}

// ---- the token-major kernel's plan and launch
struct TgPlan {
  aria::TgParams p;
  aria::TgMaps m;
  int grid = 0;
  size_t smem = 0;
};

// Ring and shared-memory layout for tiles of 256 rows x `bn` accumulator
// columns (a gradient's B is MN-major: boxes of 64 columns).
aria_status plan_tg(int mode, int bn, TgPlan* out) {
  using namespace aria;
  const DevInfo di = dev_info();
  std::memset(&out->p, 0, sizeof(out->p));
  std::memset(&out->m, 0, sizeof(out->m));
  TgParams& p = out->p;
  p.BN = bn;
  const bool grad = mode == kTgGrad;
  const uint32_t a_stage = tg_kb_per_stage(mode) * kTgATile;
  p.b_stage = static_cast<uint32_t>(tg_kb_per_stage(mode) * (grad ? (bn / 2 + 63) / 64 * 64 : bn / 2)) * 128u;
  const uint32_t col_bytes = grad ? 0 : 2 * 3 * kTgAccCols * 4;
  const uint32_t out_bytes = kTgEpiWarps * tg_slots(mode) * kTgBox;
  const int64_t budget = static_cast<int64_t>(di.smem_optin) - 1024 - 512 - col_bytes - out_bytes;
  const int ns = static_cast<int>(std::min<int64_t>(8, budget / (a_stage + p.b_stage)));
  if (ns < 2) return fail(ARIA_ERR_UNSUPPORTED, "tile does not fit in shared memory");
  p.nstage = ns;
  p.off_a = 0;
  p.off_b = static_cast<uint32_t>(ns) * a_stage;
  p.off_out = p.off_b + static_cast<uint32_t>(ns) * p.b_stage;
  p.off_col = p.off_out + out_bytes;
  p.off_bar = p.off_col + col_bytes;
  out->smem = 1024 + p.off_bar + (2 * ns + 5 + kTgEpiWarps * tg_slots(mode)) * 8 + 16;
  if (out->smem > static_cast<size_t>(di.smem_optin))
    return fail(ARIA_ERR_UNSUPPORTED, "shared memory plan too large");
  return ARIA_OK;
}

template <int MODE, bool I8>
aria_status launch_tg(TgPlan& pl, cudaStream_t st) {
  auto kfn = aria::tgemm_kernel<MODE, I8>;
  static bool attr_done[kMaxDevices] = {};
  static std::mutex attr_mu;
  aria_status as = opt_in_smem(kfn, attr_done, attr_mu);
  if (as != ARIA_OK) return as;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pl.p.nunit), 1, 1);
  cfg.blockDim = dim3(aria::kTgThreads, 1, 1);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.numAttrs = 1;
  cfg.attrs = attr;
  set_pdl(cfg, attr);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kfn, pl.m, pl.p);
  if (e != cudaSuccess) return cuda_fail(e, "token-major GEMM launch");
  return ARIA_OK;
}

aria_status half_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int box_rows) {
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows, cols, 64, box_rows,
                  CU_TENSOR_MAP_SWIZZLE_128B);
}

// fp32 partials [parts][rows][cols]: 32 x 32 boxes of one part
aria_status partial_map(CUtensorMap* m, const void* base, int parts, int64_t rows, int64_t cols) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(ARIA_ERR_CUDA, "cuTensorMapEncodeTiled unavailable");
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(parts)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols) * 4, static_cast<cuuint64_t>(rows) * cols * 4};
  cuuint32_t box[3] = {32, 32, 1}, estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ARIA_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ARIA_OK;
}

// an fp16 output [rows, cols] of the token-major kernel: 32 x 32 boxes
aria_status out_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
  return make_map(m, base, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, rows, cols, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

// The forward operators on the token-major kernel (fp16, W8A8): the tile
// width, and whether it is expected to be faster than the channel-major one.
//
// Times in us, a model of the two kernels: a K block of a pair takes
// max(2 BN, 256 + BN) cycles (the tensor core's and the shared memory's), one
// of the channel-major kernel 2 (128 + BN); a tile's epilogue overlaps the
// next tile's mainloop in part, and the last one stands alone. The five
// remaining constants are fitted to a sweep over five weight shapes and nine
// token counts from 48 to 4096 (180 cases of either operator, the linear with
// a residual), where the choice then costs 0.6 % over the best of the four
// variants on average, and 0.5 % (11 % at most) on 100 cases of five weight
// shapes outside the fit, 8192 x 2048 to 1280 x 5120.
struct TgChoice {
  int bn = 256;
  double us = 0.0;
};

TgChoice choose_tg(bool gated, int64_t M, int64_t N, int64_t nkb) {
  TgChoice best;
  const int64_t pairs = dev_info().sms / 2, tr = (M + 2 * aria::kTgRows - 1) / (2 * aria::kTgRows);
  for (int bn : {256, 192, 128}) {
    const int chans = gated ? bn / 2 : bn;
    const int64_t waves = (tr * ((N + chans - 1) / chans) + pairs - 1) / pairs;
    const double kb = std::max(2 * bn, 256 + bn) / 1850.0;  // us per K block at 1850 cycles per us
    const double epi = bn / 64 * (gated ? 0.45 : 1.0);      // a tile's epilogue
    const double main = static_cast<double>(nkb) * kb;
    const double t = 2.8 + epi + static_cast<double>(waves) * (1.5 + std::max(main, epi) + 0.75 * std::min(main, epi));
    if (best.us == 0.0 || t < best.us) best = TgChoice{bn, t};
  }
  return best;
}

// Measured: gated fp16 over N = 6144, K = 1536 takes 12.8 us against 21.1 at
// M = 203 and 110 against 163 at M = 4096, but over N = 1536, K = 6144 (few
// tiles, which only the channel-major kernel splits along K) 28 against 24 at
// M = 432; a linear with residual, W8A8 at M = 4096, N = 1536, K = 6144 33
// against 39, at K = 1536 18.4 against 17.6.
bool use_tg(int kind, bool gated, int64_t M, int64_t N, int64_t K, int* bn) {
  using namespace aria;
  if ((kind != kF16 && kind != kW8A8) || M < 128 || M > (1 << 30)) return false;  // (row indices: 32 bits)
  const int64_t nkb = (K * (kind == kF16 ? 2 : 1) + 127) / 128;
  const TgChoice tg = choose_tg(gated, M, N, nkb);
  *bn = tg.bn;
  Plan pl;
  if (plan_gemm(kind, gated ? kEpiGated : kEpiAct, M, N, K, &pl) != ARIA_OK) return false;
  const int64_t sms = dev_info().sms, ctas = static_cast<int64_t>(pl.p.tiles) * pl.p.splits;
  const double kb = 2.0 * (128 + pl.p.BN) / 1850.0, epi = pl.p.BN * 0.022;
  const double main = static_cast<double>(nkb) / pl.p.splits * kb;
  // (6.0 for a split launch: its exchange and the epilogue behind it, fitted to
  // fp16 and W8A8; plan_gemm's estimate of q8's and q4's exchange is another fit)
  const double chan = 0.5 + (pl.p.splits > 1 ? 6.0 : epi) +
                      static_cast<double>((ctas + sms - 1) / sms) * (std::max(main, epi) + 0.8 * std::min(main, epi));
  return tg.us < chan;
}

template <int MODE>
aria_status forward_tg(int kind, int bn, int64_t M, int64_t N, int64_t K, const void* X, const float* sx, const void* W,
                       const void* scales, const void* bias, const float* steer, float alpha,
                       const float* alpha_dev, void* Y, const EpiArgs& ea, cudaStream_t st) {
  using namespace aria;
  const bool i8 = kind == kW8A8;
  TgPlan pl;
  const int kelems = i8 ? 128 : 64;
  aria_status s = plan_tg(MODE, bn, &pl);
  if (s != ARIA_OK) return s;
  TgParams& p = pl.p;
  const int chans = MODE == kTgGated ? p.BN / 2 : p.BN;
  const int64_t tr = (M + 2 * kTgRows - 1) / (2 * kTgRows), tiles = tr * ((N + chans - 1) / chans);
  if (tiles > (int64_t{1} << 30)) return fail(ARIA_ERR_UNSUPPORTED, "too many tiles");
  p.R = static_cast<int>(M);
  p.C = static_cast<int>(N);
  p.nkb = static_cast<int>((K + kelems - 1) / kelems);
  p.tiles_r = static_cast<int>(tr);
  p.tiles = static_cast<int>(tiles);
  p.nunit = static_cast<int>(std::min<int64_t>(tiles, dev_info().sms / 2));
  p.act = ea.act;
  p.sx = sx;
  p.sw[0] = i8 ? static_cast<const float*>(scales) : nullptr;
  p.sw[1] = i8 ? static_cast<const float*>(ea.scales_u) : nullptr;
  p.bias[0] = static_cast<const __half*>(bias);
  p.bias[1] = static_cast<const __half*>(ea.bias_u);
  p.steer = (steer && (alpha_dev || alpha != 0.0f)) ? steer : nullptr;
  p.alpha = p.steer ? alpha : 0.0f;
  p.alpha_dev = p.steer ? alpha_dev : nullptr;
  p.res = ea.res != nullptr;
  p.save = ea.G != nullptr;
  if (ea.res && (s = out_map(&pl.m.R, ea.res, M, N)) != ARIA_OK) return s;
  if ((s = out_map(&pl.m.D[0], Y, M, N)) != ARIA_OK) return s;
  if (ea.G && ((s = out_map(&pl.m.D[1], ea.G, M, N)) != ARIA_OK || (s = out_map(&pl.m.D[2], ea.U, M, N)) != ARIA_OK))
    return s;
  const auto dt = i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int es = i8 ? 1 : 2;
  const int brows = p.BN / 2;  // rows of one B box: one CTA's half of the columns
  if ((s = make_map(&pl.m.A[0], X, dt, es, M, K, kelems, kTgRows, CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK) return s;
  if ((s = make_map(&pl.m.B[0], W, dt, es, N, K, kelems, brows, CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK) return s;
  if (MODE == kTgGated &&
      (s = make_map(&pl.m.B[1], ea.Wu, dt, es, N, K, kelems, brows, CU_TENSOR_MAP_SWIZZLE_128B)) != ARIA_OK)
    return s;
  return i8 ? launch_tg<MODE, true>(pl, st) : launch_tg<MODE, false>(pl, st);
}

// ---- the backward pass. Workspace: dG, dU fp16 [M,N], the column partials
// fp32 [P][2N], and where dX's k is split its partials fp32 [S][M][K], each
// from a 256-byte boundary.
constexpr int kBwdBn = 256;        // columns of a gradient tile
constexpr int kBwdMaxParts = 16;
constexpr int kBwdItemMin = 5;     // ring stages' time that an item's epilogue takes: no item costs less

// The longest time of a unit, in ring stages (128 of k), when `units` pairs take n0 items of
// length l0 first and then n1 <= l0 long ones; the caps go to *sc.
int64_t bwd_makespan(int units, int64_t n0, int64_t l0, int64_t n1, int64_t l1, aria::TgSched* sc) {
  sc->q = static_cast<int>(n0 / units);
  sc->r = static_cast<int>(n0 % units);
  const int64_t long_a = (sc->q + 1) * l0, long_b = sc->q * l0;
  // smallest end time that leaves room for all items of the other type
  int64_t lo = sc->r ? long_a : long_b, hi = lo + (n1 / units + 1) * l1;
  auto room = [&](int64_t t) {
    return sc->r * ((t - long_a) / l1) + static_cast<int64_t>(units - sc->r) * ((t - long_b) / l1);
  };
  while (lo < hi) {
    const int64_t t = lo + (hi - lo) / 2;
    if (room(t) >= n1) hi = t;
    else lo = t + 1;
  }
  sc->wb = static_cast<int>((lo - long_b) / l1);
  sc->wa = sc->r ? static_cast<int>((lo - long_a) / l1) : sc->wb;
  return lo;
}

struct BwdPlan {
  int rows = 32, P = 1;   // rows per block of the elementwise kernel, blocks along M
  int parts = 1;          // shares of a dX tile's k
  int units = 1;
  aria::TgSched sched{};
};

BwdPlan make_bwd_plan(int64_t M, int64_t N, int64_t K, bool dx, bool dw, int units) {
  using namespace aria;
  BwdPlan pl;
  // at most 64 partials per column (their sum is read once more), and at
  // least 32 rows per block, two for each of its 16 row lanes, whose loads
  // are then in flight together
  pl.rows = static_cast<int>(std::max<int64_t>(32, ((M + 63) / 64 + 15) / 16 * 16));
  pl.P = static_cast<int>((M + pl.rows - 1) / pl.rows);
  auto tiles = [](int64_t rows, int64_t cols) {
    return (rows + 2 * kTgRows - 1) / (2 * kTgRows) * ((cols + kBwdBn - 1) / kBwdBn);
  };
  const int64_t tx = dx ? tiles(M, K) : 0, lx = 2 * ((N + 127) / 128);
  const int64_t tw = dw ? 2 * tiles(N, K) : 0, lw = std::max<int64_t>(kBwdItemMin, (M + 127) / 128);
  // Shares of k for dX: more than one costs a further launch that reads the
  // fp32 partials back, about 5 stages' time, and every partial is written and
  // read once more (a stage takes about 0.6 us; all pairs together write and
  // read partials at about 4 TB/s)
  int64_t best = -1;
  for (int s = 1; s <= kBwdMaxParts && s <= lx; ++s) {
    if (s > 1 && (!dx || tx * s > 4 * units)) break;
    const int64_t l = std::max<int64_t>(kBwdItemMin, (lx + s - 1) / s);
    TgSched sc{};
    int64_t t;
    if (l >= lw || !dw) {
      t = bwd_makespan(units, tx * s, l, tw, lw, &sc);
      sc.first = 0;
    } else {
      t = bwd_makespan(units, tw, lw, tx * s, l, &sc);
      sc.first = 1;
    }
    if (s > 1) t += 5 + s * (M * K * 8 / 4000) / 600;
    if (best < 0 || t < best) {
      best = t;
      sc.n[0] = static_cast<int>(tx * s);
      sc.n[1] = static_cast<int>(tw);
      pl.sched = sc;
      pl.parts = s;
    }
  }
  pl.units = static_cast<int>(std::min<int64_t>(units, std::max<int64_t>(1, tx * pl.parts + tw)));
  return pl;
}

// The plan of the sizes asked for last (it takes a few us to make, and a
// training loop asks for the same one three times a call).
BwdPlan bwd_plan(int64_t M, int64_t N, int64_t K, bool dx, bool dw) {
  struct Entry {
    int64_t M = 0, N = 0, K = 0;
    int units = 0;
    BwdPlan pl;
  };
  static thread_local Entry last[4];
  const int units = dev_info().sms / 2;
  Entry& e = last[(dx ? 1 : 0) + (dw ? 2 : 0)];
  if (e.M != M || e.N != N || e.K != K || e.units != units)
    e = Entry{M, N, K, units, make_bwd_plan(M, N, K, dx, dw, units)};
  return e.pl;
}

// keeps every byte count below 2^48 (no device holds such tensors)
aria_status check_bwd_size(int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMost = int64_t{1} << 40;
  if (N > kMaxDim / 2 || M > kMaxDim / 2 || K > kMaxDim / 2)
    return fail(ARIA_ERR_UNSUPPORTED, "gated backward: sizes must be below 2^30");
  if (M > kMost / N || M > kMost / K || N > kMost / K)
    return fail(ARIA_ERR_UNSUPPORTED, "gated backward: a tensor of 2^40 elements or more");
  return ARIA_OK;
}

struct BwdLayout {
  size_t off_du = 0, off_part = 0, off_x = 0, bytes = 0;
};

BwdLayout bwd_layout(int64_t M, int64_t N, int64_t K, int P, int parts) {
  BwdLayout l;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  l.off_du = up(static_cast<size_t>(M) * N * 2);
  l.off_part = 2 * l.off_du;
  l.off_x = l.off_part + up(static_cast<size_t>(P) * 2 * N * 4);
  l.bytes = l.off_x + (parts > 1 ? up(static_cast<size_t>(parts) * M * K * 4) : 0);
  return l;
}

}  // namespace

ARIA_API aria_status aria_qgemm_act(aria_format fmt, int group, int64_t M, int64_t N, int64_t K,
                                    const void* X, const float* sx, const void* Wq, const void* scales,
                                    const void* bias, aria_act act, const void* residual,
                                    const float* steer_vec, float alpha, const float* alpha_dev, void* Y,
                                    void* stream) {
  int kind = 0;
  aria_status s = check_qgemm_args(fmt, group, X, sx, Wq, scales, bias, steer_vec, Y, &kind);
  if (s != ARIA_OK) return s;
  if (bad_act(act)) return fail(ARIA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  if (residual && !aligned16(residual))
    return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (alpha_dev && (reinterpret_cast<uintptr_t>(alpha_dev) & 3u))
    return fail(ARIA_ERR_MISALIGNED, "alpha_dev must be 4-byte aligned");
  if ((s = check_gemm_sizes(kind, M, N, K)) != ARIA_OK) return s;
  const size_t yb = static_cast<size_t>(M) * N * 2;
  if (residual != Y && overlap(residual, yb, Y, yb))
    return fail(ARIA_ERR_INVALID_ARG, "the residual may be Y itself, but not overlap it otherwise");
  if (overlap(X, x_bytes(kind, M, K), Y, yb) || overlap(Wq, weight_bytes(kind, N, K), Y, yb))
    return fail(ARIA_ERR_INVALID_ARG, "Y overlaps X or the weights");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!steer_vec) alpha_dev = nullptr;
  EpiArgs ea;
  ea.w_late = weights_late(kind, nullptr);
  if (act == ARIA_ACT_NONE && !residual)  // the plain GEMM, byte for byte
    return qgemm_impl<aria::kEpiPlain>(kind, M, N, K, X, sx, Wq, scales, bias, steer_vec, alpha, alpha_dev, Y,
                                       st, ea);
  ea.act = act;
  ea.res = residual;
  int bn = 0;
  if (use_tg(kind, false, M, N, K, &bn))
    return forward_tg<aria::kTgAct>(kind, bn, M, N, K, X, sx, Wq, scales, bias, steer_vec, alpha, alpha_dev, Y, ea, st);
  return qgemm_impl<aria::kEpiAct>(kind, M, N, K, X, sx, Wq, scales, bias, steer_vec, alpha, alpha_dev, Y, st,
                                   ea);
}

ARIA_API aria_status aria_qgemm_gated(aria_format fmt, int group, int64_t M, int64_t N, int64_t K,
                                      const void* X, const float* sx, const void* Wg, const void* scales_g,
                                      const void* Wu, const void* scales_u, const void* bias_g,
                                      const void* bias_u, aria_act act, void* H, void* G, void* U,
                                      void* stream) {
  int kind = 0;
  aria_status s = check_qgemm_args(fmt, group, X, sx, Wg, scales_g, bias_g, nullptr, H, &kind);
  if (s != ARIA_OK) return s;
  if ((s = check_qgemm_args(fmt, group, X, sx, Wu, scales_u, bias_u, nullptr, H, &kind)) != ARIA_OK) return s;
  if (bad_act(act)) return fail(ARIA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  if (!G != !U) return fail(ARIA_ERR_INVALID_ARG, "G and U are kept both or neither");
  if ((G && !aligned16(G)) || (U && !aligned16(U)))
    return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if ((s = check_gemm_sizes(kind, M, N, K)) != ARIA_OK) return s;
  if (N > kMaxDim / 2) return fail(ARIA_ERR_UNSUPPORTED, "gated: N must be below 2^30");
  const size_t yb = static_cast<size_t>(M) * N * 2;
  if (overlap(G, yb, U, yb) || overlap(G, yb, H, yb) || overlap(U, yb, H, yb))
    return fail(ARIA_ERR_INVALID_ARG, "H, G and U must not overlap");
  for (const void* o : {static_cast<const void*>(H), static_cast<const void*>(G), static_cast<const void*>(U)})
    if (overlap(X, x_bytes(kind, M, K), o, yb) || overlap(Wg, weight_bytes(kind, N, K), o, yb) ||
        overlap(Wu, weight_bytes(kind, N, K), o, yb))
      return fail(ARIA_ERR_INVALID_ARG, "an output overlaps X or a weight");
  EpiArgs ea;
  ea.w_late = weights_late(kind, G);
  ea.act = act;
  ea.Wu = Wu;
  ea.scales_u = scales_u;
  ea.bias_u = bias_u;
  ea.G = G;
  ea.U = U;
  int bn = 0;
  if (use_tg(kind, true, M, N, K, &bn))
    return forward_tg<aria::kTgGated>(kind, bn, M, N, K, X, sx, Wg, scales_g, bias_g, nullptr, 0.0f, nullptr, H, ea,
                                      static_cast<cudaStream_t>(stream));
  return qgemm_impl<aria::kEpiGated>(kind, M, N, K, X, sx, Wg, scales_g, bias_g, nullptr, 0.0f, nullptr, H,
                                     static_cast<cudaStream_t>(stream), ea);
}

ARIA_API aria_status aria_gated_bwd_workspace_size(int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return fail(ARIA_ERR_INVALID_ARG, "NULL output pointer");
  if (M < 1 || N < 1 || K < 1 || M > kMaxDim || N > kMaxDim || K > kMaxDim)
    return fail(ARIA_ERR_INVALID_ARG, "M, N and K must be in [1, 2^31)");
  aria_status s = check_bwd_size(M, N, K);
  if (s != ARIA_OK) return s;
  // enough for every subset of the gradients
  size_t need = 0;
  for (int dw = 0; dw < 2; ++dw) {
    const BwdPlan pl = bwd_plan(M, N, K, true, dw != 0);
    need = std::max(need, bwd_layout(M, N, K, pl.P, pl.parts).bytes);
  }
  *bytes = need;
  return ARIA_OK;
}

ARIA_API aria_status aria_gated_bwd(aria_act act, int64_t M, int64_t N, int64_t K, const void* dH,
                                    const void* G, const void* U, const void* X, const void* Wg,
                                    const void* Wu, void* dX, void* dWg, void* dWu, void* dbg, void* dbu,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  using namespace aria;
  if (!dH || !G || !U || !workspace) return fail(ARIA_ERR_INVALID_ARG, "NULL device pointer");
  if (!dWg != !dWu) return fail(ARIA_ERR_INVALID_ARG, "dWg and dWu are computed both or neither");
  if (!dbg != !dbu) return fail(ARIA_ERR_INVALID_ARG, "dbg and dbu are computed both or neither");
  if (!dX && !dWg && !dbg) return fail(ARIA_ERR_INVALID_ARG, "no output is asked for");
  if (dX && (!Wg || !Wu)) return fail(ARIA_ERR_INVALID_ARG, "dX needs Wg and Wu");
  if (dWg && !X) return fail(ARIA_ERR_INVALID_ARG, "dWg and dWu need X");
  if (bad_act(act)) return fail(ARIA_ERR_INVALID_ARG, "unknown activation %d", (int)act);
  for (const void* q : {dH, G, U, X, Wg, Wu, static_cast<const void*>(dX), static_cast<const void*>(dWg),
                        static_cast<const void*>(dWu), static_cast<const void*>(dbg),
                        static_cast<const void*>(dbu)})
    if (q && !aligned16(q)) return fail(ARIA_ERR_MISALIGNED, "device pointers must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ARIA_ERR_MISALIGNED, "the workspace must be 256-byte aligned");
  aria_status s = check_gemm_shape(M, N, K);
  if (s != ARIA_OK) return s;
  if ((s = check_bwd_size(M, N, K)) != ARIA_OK) return s;
  const BwdPlan bp = bwd_plan(M, N, K, dX != nullptr, dWg != nullptr);
  const BwdLayout l = bwd_layout(M, N, K, bp.P, bp.parts);
  if (workspace_bytes < l.bytes)
    return fail(ARIA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, l.bytes);
  {
    // outputs share no byte with an input, the workspace or one another
    const size_t mn = static_cast<size_t>(M) * N * 2, mk = static_cast<size_t>(M) * K * 2,
                 nk = static_cast<size_t>(N) * K * 2, nb = static_cast<size_t>(N) * 2;
    const struct { const void* p; size_t n; } out[6] = {{dX, mk}, {dWg, nk}, {dWu, nk}, {dbg, nb}, {dbu, nb},
                                                        {workspace, l.bytes}},
        in[6] = {{dH, mn}, {G, mn}, {U, mn}, {X, mk}, {Wg, nk}, {Wu, nk}};
    for (int i = 0; i < 6; ++i) {
      for (int j = 0; j < 6; ++j)
        if (overlap(out[i].p, out[i].n, in[j].p, in[j].n))
          return fail(ARIA_ERR_INVALID_ARG, "an output or the workspace overlaps an input");
      for (int j = i + 1; j < 6; ++j)
        if (overlap(out[i].p, out[i].n, out[j].p, out[j].n))
          return fail(ARIA_ERR_INVALID_ARG, "outputs and the workspace must not overlap");
    }
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  __half* dG = (dX || dWg) ? reinterpret_cast<__half*>(ws) : nullptr;
  __half* dU = (dX || dWg) ? reinterpret_cast<__half*>(ws + l.off_du) : nullptr;
  float* part = dbg ? reinterpret_cast<float*>(ws + l.off_part) : nullptr;
  // the column sums are added by idle warps of the products' launch, or, where
  // a last launch is needed anyway, by that one
  const bool finish = bp.parts > 1 || (!dX && !dWg);
  float* xpart = reinterpret_cast<float*>(ws + l.off_x);
  const int64_t count = bp.parts > 1 ? M * K : 0;
  const int64_t nb = part ? (2 * N + 63) / 64 : 0, nx = (count / 4 + 255) / 256;
  if (nb + nx > kMaxDim) return fail(ARIA_ERR_UNSUPPORTED, "too many elements");
  // everything that can be refused comes before the first launch
  TgPlan pl;
  if (dX || dWg) {
    if ((s = plan_tg(kTgGrad, kBwdBn, &pl)) != ARIA_OK) return s;
    pl.p.sched = bp.sched;
    pl.p.nunit = bp.units;
    pl.p.M = static_cast<int>(M);
    pl.p.N = static_cast<int>(N);
    pl.p.K = static_cast<int>(K);
    pl.p.parts = bp.parts;
    if (part && !finish)
      pl.p.colsum = ColSum{part, static_cast<__half*>(dbg), static_cast<__half*>(dbu), bp.P, static_cast<int>(N)};
    if (dX) {
      if ((s = half_map(&pl.m.A[0], dG, M, N, kTgRows)) != ARIA_OK) return s;
      if ((s = half_map(&pl.m.A[1], dU, M, N, kTgRows)) != ARIA_OK) return s;
      if ((s = half_map(&pl.m.B[0], Wg, N, K, 128)) != ARIA_OK) return s;
      if ((s = half_map(&pl.m.B[1], Wu, N, K, 128)) != ARIA_OK) return s;
      if ((s = bp.parts > 1 ? partial_map(&pl.m.D[0], xpart, bp.parts, M, K) : out_map(&pl.m.D[0], dX, M, K)) !=
          ARIA_OK)
        return s;
    }
    if (dWg) {
      if ((s = half_map(&pl.m.A[2], dG, M, N, 128)) != ARIA_OK) return s;
      if ((s = half_map(&pl.m.A[3], dU, M, N, 128)) != ARIA_OK) return s;
      if ((s = half_map(&pl.m.B[2], X, M, K, 128)) != ARIA_OK) return s;
      if ((s = out_map(&pl.m.D[1], dWg, N, K)) != ARIA_OK) return s;
      if ((s = out_map(&pl.m.D[2], dWu, N, K)) != ARIA_OK) return s;
    }
  }
  {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.stream = st;
    cfg.gridDim = dim3(static_cast<unsigned>((N + kGbCols - 1) / kGbCols), static_cast<unsigned>(bp.P));
    cfg.blockDim = dim3(kGbThreads);
    set_pdl(cfg, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, gated_bwd_kernel, static_cast<const __half*>(dH),
                                       static_cast<const __half*>(G), static_cast<const __half*>(U), dG, dU, part,
                                       static_cast<int>(M), static_cast<int>(N), bp.rows, static_cast<int>(act));
    if (e != cudaSuccess) return cuda_fail(e, "gated backward launch");
  }
  if ((dX || dWg) && (s = launch_tg<kTgGrad, false>(pl, st)) != ARIA_OK) return s;
  if (finish) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.stream = st;
    cfg.gridDim = dim3(static_cast<unsigned>(nb + nx));
    cfg.blockDim = dim3(256);
    set_pdl(cfg, attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, bwd_finish_kernel, static_cast<const float*>(part),
                                       static_cast<__half*>(dbg), static_cast<__half*>(dbu), bp.P,
                                       static_cast<int>(N), static_cast<int>(nb), static_cast<const float*>(xpart),
                                       static_cast<__half*>(dX), bp.parts, count);
    if (e != cudaSuccess) return cuda_fail(e, "gated backward's last launch");
  }
  return ARIA_OK;
}

ARIA_API aria_status aria_device_status(void* stream) {
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronize");
  unsigned v = 0, site = 0, zero = 0;
  if ((e = cudaMemcpyFromSymbol(&v, aria::g_status, sizeof(v))) != cudaSuccess)
    return cuda_fail(e, "read status word");
  if (v) {
    cudaMemcpyFromSymbol(&site, aria::g_wait_site, sizeof(site));
    cudaMemcpyToSymbol(aria::g_status, &zero, sizeof(zero));
    return fail(ARIA_ERR_TIMEOUT, "a bounded wait ran out in a kernel (site %u)", site);
  }
  return ARIA_OK;
}

#ifdef ARIA_TRACE
// trace builds only: copy the per-CTA phase stamps to host memory
ARIA_API int aria_trace_read(void* host, size_t bytes) {
  return static_cast<int>(cudaMemcpyFromSymbol(host, aria::g_trace, bytes));
}
ARIA_API int aria_trace_clear(void) {
  static long long zero[8192 * 24];
  g_trace_launches = 0;
  return static_cast<int>(cudaMemcpyToSymbol(aria::g_trace, zero, sizeof(zero)));
}
#endif
