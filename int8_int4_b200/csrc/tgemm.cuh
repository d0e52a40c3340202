// tgemm.cuh -- token-major GEMM on the tensor cores (tcgen05): the
// feed-forward operators over many tokens, forward and backward.
//
//   D[r, c] = sum over k of A[r, k] * B[c, k]
//
// with fp16 (or, forward, int8) operands that may each lie in memory with k
// contiguous ("K-major") or with their row index contiguous ("MN-major"), so
// that the gradients need no transposed copies:
//
//   forward     rows = tokens,   columns = channels, k = input features
//               A = X K-major, B = W K-major; gated: the columns of a tile are
//               BN/2 gate channels and the BN/2 up channels beside them, so
//               one thread holds both pre-activations of its outputs
//   dX          rows = tokens,   columns = input features, k = channels, of
//               the gate and then of the up projection (two sources)
//               A = dG, dU K-major, B = Wg, Wu MN-major
//   dWg, dWu    rows = channels, columns = input features, k = tokens
//               A = dG, dU MN-major, B = X MN-major (two problems)
//
// Beside qgemm.cuh, whose tiles have the weight channels as MMA rows: here
// the rows are the tile's 128 (or, over a CTA pair, 256) tokens. The
// epilogue then needs no transpose, and a pair of CTAs shares one
// 256 x BN tile (cta_group::2), each holding half of B: a K block moves 32 KB
// through each SM's shared memory for 128 x 256 x 64 products, where one
// CTA alone moves 48 KB. The tensor core reads shared memory at 128 bytes
// per cycle, which is what bounds the single-CTA form.
//
// Roles of a CTA (12 warps): warp 0 TMA producer, warp 1 TMEM allocation and
// MMA issue (the pair's first CTA issues for both), warps 2 and 3 the column
// sums that a backward call still has to add up (see ColSum), warps 4..11
// epilogue. Two accumulators of up to 256 columns in TMEM: a tile's epilogue
// overlaps the next tile's mainloop. Every wait is bounded.
//
// Few tiles (a gradient dX over few tokens, whose k is long): CG = 1 and a
// cluster of S CTAs divides k; the partial tiles meet in shared memory and
// are added in rank order (deterministic, no atomics, no global scratch).
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "act.cuh"
#include "ptx.cuh"

namespace aria {

enum TgMode : int { kTgStore = 0, kTgAct = 1, kTgGated = 2 };

constexpr int kTgThreads = 384;
constexpr int kTgEpiWarps = 8;
constexpr int kTgRows = 128;              // rows per CTA
constexpr uint32_t kTgATile = 16384;      // 128 rows x 64 fp16 (or 128 int8) of k
constexpr uint32_t kTgAccCols = 256;
constexpr int kTgMaxSplits = 8;

constexpr uint32_t kTgBox = 32 * 64;      // output box of a warp: 32 rows x 32 fp16
constexpr int kTgSlots = 2;               // store boxes per epilogue warp
constexpr uint32_t kTgStageBytes = kTgEpiWarps * kTgSlots * kTgBox;

struct TgMaps {
  CUtensorMap A[2], B[2];
  CUtensorMap D[3];  // outputs: one per problem; gated: H, G, U
};

// Column sums left over from an earlier kernel of the call: P rows of fp32
// partials [P][2 n] whose two halves become fp16 sums of n columns each.
struct ColSum {
  const float* part;  // null: none
  __half* out0;
  __half* out1;
  int P, n;
};

struct TgParams {
  int R, C;                // output rows and columns of one problem
  int nkb;                 // K blocks (128 bytes of k) of one source
  int nsrc;                // sources summed into one output
  int BN;                  // accumulator columns per tile (gated: 2 x channels)
  int tiles_r, tiles_c, tiles;  // tiles: over all problems (tiles_r per problem)
  int nstage, splits;
  uint32_t b_stage;        // bytes of this CTA's part of a B tile
  uint32_t off_a, off_b, off_out, off_col, off_bar;
  // epilogue
  int act;
  const float* sx;         // int8: token scales [R]
  const float* sw[2];      // int8: channel scales (gated: gate, up)
  const __half* bias[2];
  const float* steer;      // kTgAct
  float alpha;
  const float* alpha_dev;
  const __half* res;       // kTgAct: [R,C] or null; may be D itself
  __half* D[2];            // split-K: outputs, one per problem
  int save;                // kTgGated: keep the pre-activations
  ColSum colsum;
};

// MN-major operand in the 128-byte swizzle layout: boxes of 64 row indexes
// (128 bytes) x 64 k; 8 k apart = 1024 bytes (SBO), the next 64 row indexes
// 8 KB further (LBO).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;   // LBO
  d |= static_cast<uint64_t>(1024 >> 4) << 32;   // SBO
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <int CG, bool I8>
__device__ __forceinline__ void tg_mma(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc,
                                       uint32_t accumulate) {
#define ARIA_TG_MMA(group, kind)                                                   \
  asm volatile(                                                                    \
      "{\n\t.reg .pred e, p;\n\t"                                                  \
      "elect.sync _|e, 0xffffffff;\n\t"                                            \
      "setp.ne.b32 p, %4, 0;\n\t"                                                  \
      "@e tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)                                \
      : "memory")
  if constexpr (CG == 2) {
    if constexpr (I8) ARIA_TG_MMA("2", "i8");
    else ARIA_TG_MMA("2", "f16");
  } else {
    if constexpr (I8) ARIA_TG_MMA("1", "i8");
    else ARIA_TG_MMA("1", "f16");
  }
#undef ARIA_TG_MMA
}

// the completion of all MMAs issued so far arrives on this barrier, in both
// CTAs of a pair
template <int CG>
__device__ __forceinline__ void tg_commit(uint64_t* bar) {
  if constexpr (CG == 2) {
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
        "mov.b16 m, 3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::
            "r"(smem_u32(bar))
        : "memory");
  } else {
    umma_commit_elect(bar);
  }
}

// a CTA of a pair loads its own part of a tile and reports to the pair's
// first CTA (`bar`: that CTA's barrier as a cluster address)
template <int CG>
__device__ __forceinline__ void tg_load(const CUtensorMap* m, uint32_t bar, void* dst, int32_t x, int32_t y) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

__device__ __forceinline__ void st_dsmem_wait_visible() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// 32 results of this lane's row -> its 64 bytes of the warp's store box
// (64-byte swizzle: 16-byte piece j of row r at j ^ (r / 2 % 4), which spreads
// eight lanes' stores over all banks)
__device__ __forceinline__ void tg_box_row(uint8_t* box, int lane, const F2 (&y)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 v;
    __half2* h = reinterpret_cast<__half2*>(&v);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __float22half2_rn(f2_get(y[4 * j + i]));
    *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = v;
  }
}

// fp32 pre-activations of 32 columns: accumulators, scales, bias
template <bool I8>
__device__ __forceinline__ void tg_pre(const uint32_t (&v)[32], float sx, const float* sw, const float* bias,
                                       F2 (&z)[16]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 b = reinterpret_cast<const float4*>(bias)[q];
    if constexpr (I8) {
      const float4 s = reinterpret_cast<const float4*>(sw)[q];
      const F2 x2 = f2(sx);
      const F2 a0 = f2(__int2float_rn(static_cast<int32_t>(v[4 * q])), __int2float_rn(static_cast<int32_t>(v[4 * q + 1])));
      const F2 a1 = f2(__int2float_rn(static_cast<int32_t>(v[4 * q + 2])), __int2float_rn(static_cast<int32_t>(v[4 * q + 3])));
      z[2 * q] = f2_fma(f2_mul(a0, x2), f2(s.x, s.y), f2(b.x, b.y));
      z[2 * q + 1] = f2_fma(f2_mul(a1, x2), f2(s.z, s.w), f2(b.z, b.w));
    } else {
      z[2 * q] = f2_add(f2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1])), f2(b.x, b.y));
      z[2 * q + 1] = f2_add(f2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3])), f2(b.z, b.w));
    }
  }
}

// CG: CTAs sharing a tile (1 or 2). AMN, BMN: operand MN-major.
template <int MODE, bool I8, int CG, bool AMN, bool BMN>
__global__ void __launch_bounds__(kTgThreads, 1)
    tgemm_kernel(const __grid_constant__ TgMaps tm, const TgParams p) {
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t base_u32 = smem_u32(dyn_smem);
  uint8_t* smem = dyn_smem + (((base_u32 + 1023u) & ~1023u) - base_u32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kKElems = I8 ? 128 : 64;  // k per 128-byte block

  const bool split = CG == 1 && p.splits > 1;
  const int rank = (CG == 2 || split) ? static_cast<int>(cluster_ctarank()) : 0;
  const int crank = CG == 2 ? rank : 0;                        // place in the pair
  const int unit = static_cast<int>(blockIdx.x) / (split ? p.splits : CG);
  const int nunit = static_cast<int>(gridDim.x) / (split ? p.splits : CG);
  const int kb_all = p.nkb * p.nsrc;
  const int kb0 = split ? static_cast<int>(static_cast<int64_t>(kb_all) * rank / p.splits) : 0;
  const int kb1 = split ? static_cast<int>(static_cast<int64_t>(kb_all) * (rank + 1) / p.splits) : kb_all;

  uint8_t* abuf = smem + p.off_a;
  uint8_t* bbuf = smem + p.off_b;
  float* col = reinterpret_cast<float*>(smem + p.off_col);  // [2 tiles][3][kTgAccCols]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
  uint64_t* empty = full + p.nstage;
  uint64_t* acc_full = empty + p.nstage;   // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2], the pair's first CTA's
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.nstage; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, CG * kTgEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < 2; ++i) {
      prefetch_tmap(&tm.A[i]);
      prefetch_tmap(&tm.B[i]);
    }
  }
  if (warp == 1) {
    if constexpr (CG == 2) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                   "r"(2 * kTgAccCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(tmem_slot, 2 * kTgAccCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // tile -> problem, row tile (fastest: neighbours share B), column tile
  auto tile_at = [&](int t, int& prob, int& r0, int& tc) {
    const int per = p.tiles_r * p.tiles_c;
    prob = t / per;
    const int q = t % per;
    r0 = (q % p.tiles_r) * (kTgRows * CG) + crank * kTgRows;
    tc = q / p.tiles_r;
  };

  int issued = 0;
  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    const uint32_t full0 = CG == 2 ? mapa_shared(smem_u32(full), 0) : smem_u32(full);
    const uint32_t tx = CG * (kTgATile + p.b_stage);
    const int bn_cta = p.BN / CG;  // this CTA's columns of B
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = unit; t < p.tiles && ok; t += nunit) {
      int prob, r0, tc;
      tile_at(t, prob, r0, tc);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(ok = mbar_wait_warp(empty + s, ph ^ 1, abort_flag, 40))) break;
        if (lane == 0) {
          const int src = kb / p.nkb, x = (kb - src * p.nkb) * kKElems;
          if (crank == 0) mbar_arrive_expect_tx(full + s, tx);
          const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
          uint8_t* a = abuf + s * kTgATile;
          uint8_t* b = bbuf + s * p.b_stage;
          const CUtensorMap* ma = &tm.A[p.nsrc == 2 ? src : prob];
          if constexpr (AMN) {
            tg_load<CG>(ma, bar, a, r0, x);
            tg_load<CG>(ma, bar, a + 8192, r0 + 64, x);
          } else {
            tg_load<CG>(ma, bar, a, x, r0);
          }
          if constexpr (MODE == kTgGated) {
            // CTA pair: the first CTA brings the gate's channels, the second
            // the up projection's; a lone CTA brings both
            const int c0 = tc * (p.BN / 2);
            if constexpr (CG == 2) {
              tg_load<CG>(&tm.B[crank], bar, b, x, c0);
            } else {
              tg_load<CG>(&tm.B[0], bar, b, x, c0);
              tg_load<CG>(&tm.B[1], bar, b + (p.b_stage >> 1), x, c0);
            }
          } else {
            const int c0 = tc * p.BN + crank * bn_cta;
            const CUtensorMap* mb = &tm.B[p.nsrc == 2 ? src : 0];
            if constexpr (BMN) {
              for (int j = 0; j < bn_cta; j += 64) tg_load<CG>(mb, bar, b + j * 128, c0 + j, x);
            } else {
              tg_load<CG>(mb, bar, b, x, c0);
            }
          }
        }
        ++issued;
        if (++s == p.nstage) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (crank == 0) {
      uint32_t idesc = I8 ? idesc_s8_s32(p.BN) : idesc_f16_f32(p.BN);
      if (CG == 2) idesc += (128u >> 4) << 24;  // M = 256
      if (AMN) idesc |= 1u << 15;
      if (BMN) idesc |= 1u << 16;
      int ti = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = unit; t < p.tiles && ok; t += nunit, ++ti) {
        const int b = ti & 1;
        if (!(ok = mbar_wait_warp(acc_empty + b, ((ti >> 1) & 1) ^ 1, abort_flag, 41))) break;
        if constexpr (CG == 2) st_dsmem_wait_visible();  // the peer's arrivals
        tc_fence_after();
        const uint32_t dt = tmem_base + b * kTgAccCols;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!(ok = mbar_wait_warp(full + s, ph, abort_flag, 42))) break;
          tc_fence_after();
          const uint32_t a_u = smem_u32(abuf + s * kTgATile), b_u = smem_u32(bbuf + s * p.b_stage);
          const uint64_t ad = AMN ? sdesc_mn_sw128(a_u) : sdesc_sw128(a_u);
          const uint64_t bd = BMN ? sdesc_mn_sw128(b_u) : sdesc_sw128(b_u);
#pragma unroll
          for (int j = 0; j < 4; ++j)  // K-major: 32 bytes per step; MN-major: 16 rows of 128 bytes
            tg_mma<CG, I8>(dt, ad + (AMN ? 128 : 2) * j, bd + (BMN ? 128 : 2) * j, idesc, (kb > kb0) | (j > 0));
          tg_commit<CG>(empty + s);
          if (++s == p.nstage) { s = 0; ph ^= 1u; }
        }
        tg_commit<CG>(acc_full + b);
      }
    }
  } else if (warp < 4) {
    // --------------------------------- column sums of an earlier kernel
    // One thread per output, the partials in order; their loads are
    // independent, so eight are in flight.
    if (MODE == kTgStore && p.colsum.part) {
      const ColSum& cs = p.colsum;
      const int n2 = 2 * cs.n;
      for (int c = static_cast<int>(blockIdx.x) * 64 + (warp - 2) * 32 + lane; c < n2;
           c += static_cast<int>(gridDim.x) * 64) {
        float sum = 0.0f;
#pragma unroll 8
        for (int i = 0; i < cs.P; ++i) sum += ld_dep_f32(cs.part + static_cast<int64_t>(i) * n2 + c);
        const __half h = __float2half_rn(sum);
        if (c < cs.n) cs.out0[c] = h;
        else cs.out1[c - cs.n] = h;
      }
    }
  } else if (!split) {
    // ----------------------------------------------------------- epilogue
    const int e = warp - 4, te = threadIdx.x - 128;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int cg = e >> 2;  // this warp takes chunks cg, cg + 2, ...
    const int chans = MODE == kTgGated ? p.BN / 2 : p.BN;
    const uint32_t release0 = CG == 2 ? mapa_shared(smem_u32(acc_empty), 0) : smem_u32(acc_empty);
    const float alpha = (MODE == kTgAct && p.steer) ? (p.alpha_dev ? *p.alpha_dev : p.alpha) : 0.0f;
    // column constants of a tile, one tile ahead: bias, scale, steering
    auto col_load = [&](int t, float (&cv)[3]) {
      cv[0] = cv[2] = 0.0f;
      cv[1] = 1.0f;
      if constexpr (MODE == kTgStore) return;
      if (t >= p.tiles || te >= p.BN) return;
      int prob, r0, tc;
      tile_at(t, prob, r0, tc);
      const bool up = MODE == kTgGated && te >= chans;
      const int c = tc * chans + (up ? te - chans : te);
      if (c >= p.C) return;
      const __half* bp = up ? p.bias[1] : p.bias[0];
      if (bp) cv[0] = __half2float(__ushort_as_half(ld_dep_u16(bp + c)));
      if constexpr (I8) cv[1] = ld_dep_f32((up ? p.sw[1] : p.sw[0]) + c);
      if (MODE == kTgAct && alpha != 0.0f) cv[2] = alpha * ld_dep_f32(p.steer + c);
    };
    float cv[3];
    col_load(unit, cv);
    uint8_t* boxes = smem + p.off_out + e * (kTgSlots * kTgBox);
    int ti = 0, nst = 0;
    for (int t = unit; t < p.tiles; t += nunit, ++ti) {
      const int b = ti & 1;
      int prob, r0, tc;
      tile_at(t, prob, r0, tc);
      float* cb = col + b * 3 * kTgAccCols;
      if constexpr (MODE != kTgStore) {
#pragma unroll
        for (int k = 0; k < 3; ++k) cb[k * kTgAccCols + te] = cv[k];
        named_bar(1, kTgEpiWarps * 32);  // and every reader of this buffer two tiles ago is done
        col_load(t + nunit, cv);
      }
      const int rw = r0 + (warp & 3) * 32, r = rw + lane;  // this warp's first row, this lane's row
      const bool row_in = r < p.R;
      const int64_t ro = static_cast<int64_t>(r) * p.C;
      float sx = 1.0f;
      if constexpr (I8) sx = row_in ? ld_dep_f32(p.sx + r) : 0.0f;
      bool ok = mbar_wait(acc_full + b, (ti >> 1) & 1, abort_flag, 43);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;  // (stays with the named barriers of later tiles)
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_off + b * kTgAccCols;
      // units of 32 columns; a result goes through a store box of the warp's
      // own and leaves by TMA, which clips the box at the tensor's edges
      auto box_store = [&](const CUtensorMap* m, const F2 (&y)[16], int c0) {
        uint8_t* box = boxes + (nst & (kTgSlots - 1)) * kTgBox;
        ++nst;
        if (lane == 0) bulk_wait_read<kTgSlots - 1>();  // the box's last store has read it
        __syncwarp();
        tg_box_row(box, lane, y);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rw < p.R) tma_store_2d(m, box, c0, rw);
          bulk_commit();
        }
      };
      const int nunit32 = (chans + 31) / 32;
      for (int c = cg; c < nunit32; c += 2) {
        const int c0 = tc * chans + c * 32;
        if (c0 >= p.C) break;
        uint32_t v[32];
        tmem_ld32(tacc + c * 32, v);
        F2 z[16];
        if constexpr (MODE == kTgStore) {
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 16; ++i) z[i] = f2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
          box_store(&tm.D[prob], z, c0);
        } else if constexpr (MODE == kTgAct) {
          uint4 rv[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            rv[j] = make_uint4(0u, 0u, 0u, 0u);
            if (p.res && row_in && c0 + 8 * j < p.C) rv[j] = ld_dep_v4(p.res + ro + c0 + 8 * j);  // C % 16 == 0
          }
          tmem_ld_wait();
          tg_pre<I8>(v, sx, cb + kTgAccCols + c * 32, cb + c * 32, z);
          with_act(p.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = act_fwd2<decltype(tag)::value>(z[i]);
          });
          if (alpha != 0.0f) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float4 f = reinterpret_cast<const float4*>(cb + 2 * kTgAccCols + c * 32)[q];
              z[2 * q] = f2_add(z[2 * q], f2(f.x, f.y));
              z[2 * q + 1] = f2_add(z[2 * q + 1], f2(f.z, f.w));
            }
          }
          if (p.res) {
            const __half2* hr = reinterpret_cast<const __half2*>(rv);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 f = __half22float2(hr[i]);
              z[i] = f2_add(z[i], f2(f.x, f.y));
            }
          }
          box_store(&tm.D[0], z, c0);
        } else {
          uint32_t w[32];
          tmem_ld32(tacc + chans + c * 32, w);
          tmem_ld_wait();
          F2 u[16];
          tg_pre<I8>(v, sx, cb + kTgAccCols + c * 32, cb + c * 32, z);
          tg_pre<I8>(w, sx, cb + kTgAccCols + chans + c * 32, cb + chans + c * 32, u);
          if (p.save) {
            box_store(&tm.D[1], z, c0);
            box_store(&tm.D[2], u, c0);
          }
          with_act(p.act, [&](auto tag) {
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = f2_mul(act_fwd2<decltype(tag)::value>(z[i]), u[i]);
          });
          box_store(&tm.D[0], z, c0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (CG == 2) mbar_arrive_cluster(release0 + b * 8u);
        else mbar_arrive(acc_empty + b);
      }
    }
    if (lane == 0) bulk_wait_all();
  }

  // -------------------------------------------- split-K: cluster reduction
  // One tile per cluster. The partial tile goes to shared memory as fp32
  // rows of BN + 4 words (the pad spreads a warp's 16-byte stores, one row
  // per lane, over the banks); after a cluster barrier rank q adds rows
  // [128 q / S, 128 (q + 1) / S) in rank order and stores them.
  if (split) {
    const bool ok = mbar_wait_warp(acc_full, 0, abort_flag, 44);
    float* red = reinterpret_cast<float*>(smem);
    const uint32_t stride = static_cast<uint32_t>(p.BN) + 4u;
    tc_fence_after();
    {
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      float* rr = red + ((warp & 3) * 32 + lane) * stride;
      for (int c = warp >> 2; c < p.BN / 16; c += 3) {
        uint32_t v[16];
        tmem_ld16(tmem_base + lane_off + c * 16, v);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<uint4*>(rr + c * 16 + 4 * q) =
              ok ? make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    __syncwarp();
    cluster_sync();
    int prob, r0, tc;
    tile_at(unit, prob, r0, tc);
    const int rb = kTgRows * rank / p.splits, re = kTgRows * (rank + 1) / p.splits;
    const int per_row = p.BN / 8;  // 8 columns per thread
    const uint32_t red_u32 = smem_u32(smem);
    for (int i = threadIdx.x; i < (re - rb) * per_row; i += kTgThreads) {
      const int row = rb + i / per_row, c8 = (i % per_row) * 8;
      const int r = r0 + row, c = tc * p.BN + c8;
      if (r >= p.R || c >= p.C) continue;  // C % 16 == 0
      uint4 a[kTgMaxSplits][2];
#pragma unroll
      for (int q = 0; q < kTgMaxSplits; ++q) {
        if (q < p.splits) {
          const uint32_t ad = mapa_shared(red_u32 + (row * stride + c8) * 4u, q);
          a[q][0] = ld_dsmem_v4(ad);
          a[q][1] = ld_dsmem_v4(ad + 16u);
        }
      }
      float y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = 0.0f;
#pragma unroll
      for (int q = 0; q < kTgMaxSplits; ++q) {
        if (q < p.splits) {
          const uint32_t w[8] = {a[q][0].x, a[q][0].y, a[q][0].z, a[q][0].w, a[q][1].x, a[q][1].y, a[q][1].z, a[q][1].w};
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] += __uint_as_float(w[k]);
        }
      }
      uint4 o;
      __half2* h = reinterpret_cast<__half2*>(&o);
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
      *reinterpret_cast<uint4*>(p.D[prob] + static_cast<int64_t>(r) * p.C + c) = o;
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer still reads its partials
  }

  // ---------------------------------------------------------------- teardown
  const bool aborted = *abort_flag != 0;
  if (warp == 0 && aborted && issued > 0 && lane == 0) {
    // loads in flight write this CTA's shared memory: allow them 100 us to
    // land (a pair's loads report to its first CTA, so the second cannot
    // wait on a barrier of its own)
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) __nanosleep(1000);
  }
  if (warp == 1 && crank == 0 && __any_sync(0xffffffffu, aborted)) {
    tg_commit<CG>(drain);
    mbar_wait_drain(drain, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();  // the pair's MMAs, commits and arrivals are done
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * kTgAccCols)
                   : "memory");
    else
      tmem_dealloc(tmem_base, 2 * kTgAccCols);
  }
}

}  // namespace aria
