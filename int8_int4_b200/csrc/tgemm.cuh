// tgemm.cuh -- token-major GEMM on the tensor cores (tcgen05): the
// feed-forward operators over many tokens, and their gradients.
//
//   D[r, c] = sum over k of A[r, k] * B[c, k]
//
// with fp16 (or, forward, int8) operands that may each lie in memory with k
// contiguous ("K-major") or with their row index contiguous ("MN-major"), so
// that the gradients need no transposed copies:
//
//   forward     rows = tokens,   columns = channels, k = input features
//               A = X K-major, B = W K-major; gated: the columns of a tile are
//               128 gate channels and the 128 up channels beside them, so
//               one thread holds both pre-activations of its outputs
//   dX          rows = tokens,   columns = input features, k = channels, of
//               the gate and then of the up projection (two sources)
//               A = dG, dU K-major, B = Wg, Wu MN-major
//   dWg, dWu    rows = channels, columns = input features, k = tokens
//               A = dG, dU MN-major, B = X MN-major
//
// Beside qgemm.cuh, whose tiles have the weight channels as MMA rows: here
// the rows are tokens (or, for dW, channels), and a pair of CTAs shares one
// 256-row tile (cta_group::2), each holding its 128 rows of A and half of B.
// A K block then moves 32 KB into each SM for 128 x 256 x 64 products where a
// lone CTA moves 48 KB, and shared memory, which the tensor core reads at 128
// bytes per cycle, keeps up with it: fp16 at M = 8192, N = K = 8192 ran at
// 1390 TFLOP/s with its epilogue taken out and 1240-1280 with it, cuBLAS at
// 1373 (both under the power cap). Loads alone took 295 ns per K block, the
// MMAs alone 300, both 350 (at 1.3 tiles per pair) to 480 (power-capped).
//
// Roles of a CTA (12 warps): warp 0 TMA producer, warp 1 TMEM allocation and
// MMA issue (the pair's first CTA issues for both), warps 2 and 3 the column
// sums that a backward call still has to add up (see ColSum), warps 4..11
// epilogue. Two accumulators of up to 256 columns in TMEM: a tile's epilogue
// overlaps the next tile's mainloop. The epilogue works on packed fp32 pairs
// and writes through small swizzled boxes that leave by TMA; with scalar
// arithmetic and 16-byte stores per row it was what bounded the forward
// operators (M = 4096, N = 6144, K = 1536: gated fp16 with its
// pre-activations 136 against 121 us, gated W8A8 77-86 against 62, fp16 with
// GELU 75 against 67). Every wait is bounded.
//
// The two gradients run in ONE launch, over one list of work items: dX tiles
// have a long k (2 N), dW tiles a short one (M), and the pairs take the long
// ones first and fill up with the short ones (see TgSched).
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "act.cuh"
#include "ptx.cuh"

namespace aria {

enum TgMode : int { kTgGrad = 0, kTgAct = 1, kTgGated = 2 };

constexpr int kTgEpiWarps = 8;
constexpr int kTgThreads = 128 + 32 * kTgEpiWarps;
constexpr int kTgEpiStep = kTgEpiWarps / 4;  // warps per TMEM lane quarter: they share a tile's column units
constexpr int kTgRows = 128;              // rows per CTA; a pair's tile has twice as many
constexpr uint32_t kTgATile = 16384;      // 128 rows x 64 fp16 (or 128 int8) of k
constexpr uint32_t kTgAccCols = 256;      // = the epilogue's threads, which load a tile's column constants
constexpr uint32_t kTgBox = 32 * 64;      // output box of a warp: 32 rows x 32 fp16
// Boxes per epilogue warp (two together hold 32 x 32 fp32), and K blocks per
// ring stage. A box of an MN-major operand is 64 rows wide, so a K block of a
// gradient takes three or four TMA copies where a forward one takes two, and
// each further copy costs about 40 ns; two K blocks per stage bring it back
// to two of 16 KB each (backward at M, N, K = 4096, 6144, 1536: 254 against
// 288 us).
__host__ __device__ constexpr int tg_slots(int mode) { return mode == kTgGrad ? 2 : 3; }
__host__ __device__ constexpr int tg_kb_per_stage(int mode) { return mode == kTgGrad ? 2 : 1; }

struct TgMaps {
  CUtensorMap A[4];  // forward: X; gradients: dG, dU as rows of tokens, then as rows of channels
  CUtensorMap B[3];  // forward: W (gated: gate, up); gradients: Wg, Wu, X
  CUtensorMap D[3];  // forward: Y or H, G, U; gradients: dX (split k: its fp32 partials), dWg, dWu
  CUtensorMap R;     // kTgAct: the residual
};

// Column sums left over from an earlier kernel of the call: P rows of fp32
// partials [P][2 n] whose two halves become fp16 sums of n columns each.
struct ColSum {
  const float* part;  // null: none
  __half* out0;
  __half* out1;
  int P, n;
};

// Work items of a gradient launch. An item of type 0 is one of `parts` equal
// shares of the k of a dX tile, an item of type 1 a dW tile. Units (pairs)
// 0 .. r - 1 take q + 1 items of the longer type, the others q; then every
// unit takes items of the other type up to a cap chosen by the host so that
// all end at about the same time: wa for the first r units, wb >= wa for the
// others.
struct TgSched {
  int first;              // the longer type
  int n[2];               // items of either type
  int q, r, wa, wb;
};

struct TgParams {
  int R, C;                // forward: output rows and columns
  int nkb;                 // forward: K blocks (128 bytes of k), one per stage
  int BN;                  // accumulator columns per tile (gated: 2 x channels)
  int tiles_r, tiles, nunit;
  int nstage;
  uint32_t b_stage;        // bytes of this CTA's part of B in a stage
  uint32_t off_a, off_b, off_out, off_col, off_bar;
  // gradients
  TgSched sched;
  int M, N, K, parts;      // tokens, channels, input features; shares of a dX tile's k
  // forward epilogue
  int act;
  const float* sx;         // int8: token scales [R]
  const float* sw[2];      // int8: channel scales (gated: gate, up)
  const __half* bias[2];
  const float* steer;      // kTgAct
  float alpha;
  const float* alpha_dev;
  int res;                 // kTgAct: add the residual (may be Y itself)
  int save;                // kTgGated: keep the pre-activations
  ColSum colsum;
};

// MN-major operand in the 128-byte swizzle layout: boxes of 64 row indexes
// (128 bytes) x 128 k; 8 k apart = 1024 bytes (SBO), the next 64 row indexes
// 16 KB further (LBO).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>(16384 >> 4) << 16;  // LBO
  d |= static_cast<uint64_t>(1024 >> 4) << 32;   // SBO
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <bool I8>
__device__ __forceinline__ void tg_mma(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (I8)
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
        : "memory");
}

// the completion of all MMAs issued so far arrives on this barrier of both
// CTAs
__device__ __forceinline__ void tg_commit(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
      "mov.b16 m, 3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::
          "r"(smem_u32(bar))
      : "memory");
}

// a CTA loads its own part of a tile into its own shared memory and reports
// to the pair's first CTA (`bar`: that CTA's barrier as a cluster address)
__device__ __forceinline__ void tg_load(const CUtensorMap* m, uint32_t bar, void* dst, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// a load that reports to a barrier of this CTA
__device__ __forceinline__ void tg_load_local(const CUtensorMap* m, uint64_t* bar, void* dst, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
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

// 32 accumulators of this lane's row -> its 128 bytes of a 32 x 32 fp32 box
// (128-byte swizzle)
__device__ __forceinline__ void tg_box_row_f32(uint8_t* box, int lane, const uint32_t (&v)[32]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}

// One work item as a CTA of a pair sees it.
struct TgItem {
  int type;        // gradients: 0 = dX, 1 = dW
  int src;         // dW: 0 = gate, 1 = up; dX: the share of k
  int r0, c0;      // this CTA's first row; the tile's first column
  int kb0, kb1;    // ring stages of k
};

template <int MODE, bool I8>
__global__ void __launch_bounds__(kTgThreads, 1)
    tgemm_kernel(const __grid_constant__ TgMaps tm, const TgParams p) {
  extern __shared__ uint8_t dyn_smem[];
  const uint32_t base_u32 = smem_u32(dyn_smem);
  uint8_t* smem = dyn_smem + (((base_u32 + 1023u) & ~1023u) - base_u32);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kKElems = I8 ? 128 : 64;  // k per 128-byte block
  constexpr int kKbs = tg_kb_per_stage(MODE), kSlots = tg_slots(MODE);
  constexpr uint32_t kAStage = kKbs * kTgATile;

  const int crank = static_cast<int>(cluster_ctarank());  // place in the pair
  const int unit = static_cast<int>(blockIdx.x) >> 1;
  const int chans = MODE == kTgGated ? p.BN / 2 : p.BN;   // output columns per tile

  uint8_t* abuf = smem + p.off_a;
  uint8_t* bbuf = smem + p.off_b;
  float* col = reinterpret_cast<float*>(smem + p.off_col);  // forward: [2 tiles][3][kTgAccCols]
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + p.off_bar);
  uint64_t* empty = full + p.nstage;
  uint64_t* acc_full = empty + p.nstage;   // [2]
  uint64_t* acc_empty = acc_full + 2;      // [2], the pair's first CTA's
  uint64_t* drain = acc_empty + 2;
  uint64_t* res_full = drain + 1;          // kTgAct: [kTgEpiWarps][slots]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(res_full + kTgEpiWarps * kSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.nstage; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(acc_full + i, 1);
      mbar_init(acc_empty + i, 2 * kTgEpiWarps);
    }
    mbar_init(drain, 1);
    for (int i = 0; i < kTgEpiWarps * kSlots; ++i) mbar_init(res_full + i, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if constexpr (MODE != kTgGrad) {  // (a gradient launch fills only the maps that it uses)
      prefetch_tmap(&tm.A[0]);
      prefetch_tmap(&tm.B[0]);
      prefetch_tmap(&tm.D[0]);
    }
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(2 * kTgAccCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // The unit's i-th item; false behind its last one. Neighbouring units take
  // neighbouring items at the same time, so their operands meet in L2.
  auto item_at = [&](int i, TgItem& it) -> bool {
    int idx;
    if constexpr (MODE == kTgGrad) {
      const TgSched& sc = p.sched;
      const int nl = sc.q + (unit < sc.r);  // items of the longer type
      if (i < nl) {
        it.type = sc.first;
        idx = i * p.nunit + unit;
      } else {
        it.type = sc.first ^ 1;
        const int j = i - nl;
        if (j < sc.wa) {
          idx = j * p.nunit + unit;
        } else {
          if (unit < sc.r || j >= sc.wb) return false;
          idx = sc.wa * p.nunit + (j - sc.wa) * (p.nunit - sc.r) + (unit - sc.r);
        }
      }
      if (idx >= sc.n[it.type]) return false;
      const int tiles_c = (p.K + p.BN - 1) / p.BN;
      if (it.type == 0) {
        const int kb_all = 2 * ((p.N + 127) / 128);
        const int tile = idx / p.parts;
        it.src = idx - tile * p.parts;
        it.kb0 = static_cast<int>(static_cast<int64_t>(kb_all) * it.src / p.parts);
        it.kb1 = static_cast<int>(static_cast<int64_t>(kb_all) * (it.src + 1) / p.parts);
        it.r0 = (tile / tiles_c) * (2 * kTgRows);
        it.c0 = (tile % tiles_c) * p.BN;
      } else {
        const int per = sc.n[1] / 2;  // tiles of one projection
        it.src = idx >= per;
        const int tile = idx - it.src * per;
        it.kb0 = 0;
        it.kb1 = (p.M + 127) / 128;
        it.r0 = (tile / tiles_c) * (2 * kTgRows);
        it.c0 = (tile % tiles_c) * p.BN;
      }
    } else {
      idx = i * p.nunit + unit;
      if (idx >= p.tiles) return false;
      it.type = it.src = 0;
      it.r0 = (idx % p.tiles_r) * (2 * kTgRows);
      it.c0 = (idx / p.tiles_r) * chans;
      it.kb0 = 0;
      it.kb1 = p.nkb;
    }
    it.r0 += crank * kTgRows;
    return true;
  };

  int issued = 0;
  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    const uint32_t full0 = mapa_shared(smem_u32(full), 0);
    const uint32_t tx = 2 * (kAStage + p.b_stage);   // both CTAs' bytes
    const int bn_cta = p.BN / 2;                     // this CTA's columns of B
    int s = 0;
    uint32_t ph = 0;
    bool ok = true;
    TgItem it;
    for (int i = 0; ok && item_at(i, it); ++i) {
      for (int kb = it.kb0; kb < it.kb1; ++kb) {
        if (!(ok = mbar_wait_warp(empty + s, ph ^ 1, abort_flag, 40))) break;
        if (lane == 0) {
          if (crank == 0) mbar_arrive_expect_tx(full + s, tx);
          const uint32_t bar = full0 + static_cast<uint32_t>(s) * 8u;
          uint8_t* a = abuf + s * kAStage;
          uint8_t* b = bbuf + s * p.b_stage;
          if constexpr (MODE == kTgGrad) {
            const CUtensorMap* mb;
            int x;
            if (it.type == 0) {
              const int nst = (p.N + 127) / 128, src = kb >= nst;
              x = (kb - src * nst) * 128;
              tg_load(&tm.A[src], bar, a, x, it.r0);
              tg_load(&tm.A[src], bar, a + kTgATile, x + 64, it.r0);
              mb = &tm.B[src];
            } else {
              x = kb * 128;
              tg_load(&tm.A[2 + it.src], bar, a, it.r0, x);
              tg_load(&tm.A[2 + it.src], bar, a + kTgATile, it.r0 + 64, x);
              mb = &tm.B[2];
            }
            const int c = it.c0 + crank * bn_cta;
            for (int j = 0; j < bn_cta; j += 64) tg_load(mb, bar, b + j * 256, c + j, x);
          } else {
            const int x = kb * kKElems;
            tg_load(&tm.A[0], bar, a, x, it.r0);
            // gated: the first CTA brings the gate's channels, the second
            // the up projection's
            if constexpr (MODE == kTgGated) tg_load(&tm.B[crank], bar, b, x, it.c0);
            else tg_load(&tm.B[0], bar, b, x, it.c0 + crank * bn_cta);
          }
        }
        ++issued;
        if (++s == p.nstage) { s = 0; ph ^= 1u; }
      }
    }
  } else if (warp == 1) {
    // --------------------------------------------------------- MMA issuer
    if (crank == 0) {
      // M = 256
      const uint32_t idesc0 = (I8 ? idesc_s8_s32(p.BN) : idesc_f16_f32(p.BN)) + ((128u >> 4) << 24);
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      TgItem it;
      for (int i = 0; ok && item_at(i, it); ++i) {
        const int b = i & 1;
        if (!(ok = mbar_wait_warp(acc_empty + b, ((i >> 1) & 1) ^ 1, abort_flag, 41))) break;
        asm volatile("fence.acq_rel.cluster;" ::: "memory");  // the peer's arrivals
        tc_fence_after();
        const uint32_t dt = tmem_base + b * kTgAccCols;
        // MN-major operands: bits 15 (A) and 16 (B)
        const bool amn = MODE == kTgGrad && it.type == 1;
        constexpr bool bmn = MODE == kTgGrad;
        const uint32_t idesc = idesc0 | (amn ? 1u << 15 : 0u) | (bmn ? 1u << 16 : 0u);
        // 16 k further, in descriptor units of 16 bytes: 32 bytes of a K-major
        // row, or 16 rows of 128 bytes; the second K block of a stage lies
        // kTgATile further (K-major), or 64 such rows
        const uint32_t astep = amn ? 128 : 2, ablock = amn ? 512 : kTgATile / 16;
        const int klim = MODE != kTgGrad ? 0 : it.type == 0 ? p.N : p.M;
        const int kper = MODE != kTgGrad || it.type == 1 ? 1 << 30 : (p.N + 127) / 128;  // stages per source
        for (int kb = it.kb0; kb < it.kb1; ++kb) {
          if (!(ok = mbar_wait_warp(full + s, ph, abort_flag, 42))) break;
          tc_fence_after();
          const uint32_t a_u = smem_u32(abuf + s * kAStage), b_u = smem_u32(bbuf + s * p.b_stage);
          const uint64_t ad = amn ? sdesc_mn_sw128(a_u) : sdesc_sw128(a_u);
          const uint64_t bd = bmn ? sdesc_mn_sw128(b_u) : sdesc_sw128(b_u);
#pragma unroll
          for (int h = 0; h < kKbs; ++h) {
            // a second K block wholly beyond the sum's end holds zeros
            if (h == 1 && (kb >= kper ? kb - kper : kb) * 128 + 64 >= klim) break;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              tg_mma<I8>(dt, ad + ablock * h + astep * j, bd + (bmn ? 512 * h + 128 * j : 2 * j), idesc,
                         (kb > it.kb0) | (h > 0) | (j > 0));
          }
          tg_commit(empty + s);
          if (++s == p.nstage) { s = 0; ph ^= 1u; }
        }
        tg_commit(acc_full + b);
      }
    }
  } else if (warp < 4) {
    // --------------------------------- column sums of an earlier kernel
    // One thread per output; four interleaved sums, joined as
    // bwd_finish_kernel joins its four threads', so that either gives the same
    // bytes.
    if (MODE == kTgGrad && p.colsum.part) {
      const ColSum& cs = p.colsum;
      const int n2 = 2 * cs.n;
      for (int c = static_cast<int>(blockIdx.x) * 64 + (warp - 2) * 32 + lane; c < n2;
           c += static_cast<int>(gridDim.x) * 64) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const float* pc = cs.part + c;
        int i = 0;
        for (; i + 4 <= cs.P; i += 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) sum[q] += ld_dep_f32(pc + static_cast<int64_t>(i + q) * n2);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q)
          if (i + q < cs.P) sum[q] += ld_dep_f32(pc + static_cast<int64_t>(i + q) * n2);
        const __half h = __float2half_rn((sum[0] + sum[1]) + (sum[2] + sum[3]));
        if (c < cs.n) cs.out0[c] = h;
        else cs.out1[c - cs.n] = h;
      }
    }
  } else {
    // ----------------------------------------------------------- epilogue
    const int e = warp - 4, te = threadIdx.x - 128;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int cg = e >> 2;  // this warp takes 32-column units cg, cg + kTgEpiStep, ...
    const uint32_t release0 = mapa_shared(smem_u32(acc_empty), 0);
    const float alpha = (MODE == kTgAct && p.steer) ? (p.alpha_dev ? *p.alpha_dev : p.alpha) : 0.0f;
    // column constants of an item, one item ahead: bias, scale, steering
    auto col_load = [&](bool valid, const TgItem& it, float (&cv)[3]) {
      cv[0] = cv[2] = 0.0f;
      cv[1] = 1.0f;
      if (!valid || te >= p.BN) return;
      const bool up = MODE == kTgGated && te >= chans;
      const int c = it.c0 + (up ? te - chans : te);
      if (c >= p.C) return;
      const __half* bp = up ? p.bias[1] : p.bias[0];
      if (bp) cv[0] = __half2float(__ushort_as_half(ld_dep_u16(bp + c)));
      if constexpr (I8) cv[1] = ld_dep_f32((up ? p.sw[1] : p.sw[0]) + c);
      if (MODE == kTgAct && alpha != 0.0f) cv[2] = alpha * ld_dep_f32(p.steer + c);
    };
    uint8_t* boxes = smem + p.off_out + e * (kSlots * kTgBox);
    float cv[3];
    TgItem it, nx;
    bool valid = item_at(0, nx);
    if constexpr (MODE != kTgGrad) col_load(valid, nx, cv);
    int slot = 0;       // the next unit's box
    uint32_t rph = 0;   // parity of its residual's arrival
    // kTgAct: the residual of a unit is loaded by TMA into the box that will
    // carry the unit's result, kSlots - 1 units ahead and across items (the
    // lane reads its row of the box, adds, and writes the sum in its place).
    // Read directly, 16 bytes per row and lane, it took longer: W8A8 with relu
    // at M = 4096, N = 6144, K = 1536 49 against 44 us, the down projection 39
    // against 38.
    TgItem pit;
    int pi = 0, pc = cg, pslot = 0;
    bool pvalid = valid;
    pit = nx;
    auto res_issue = [&] {  // lane 0 issues the load of the next unit in line
      if (!pvalid) return;
      if (lane == 0) {
        bulk_wait_read<1>();  // all but the newest store have read their boxes
        uint64_t* bar = res_full + e * kSlots + pslot;
        mbar_arrive_expect_tx(bar, kTgBox);
        tg_load_local(&tm.R, bar, boxes + pslot * kTgBox, pit.c0 + pc * 32, pit.r0 + (warp & 3) * 32);
      }
      if (++pslot == kSlots) pslot = 0;
      pc += kTgEpiStep;
      if (pc * 32 >= chans || pit.c0 + pc * 32 >= p.C) {
        pc = cg;
        do {  // (a narrow last column tile may hold no unit of this warp)
          pvalid = item_at(++pi, pit);
        } while (pvalid && pit.c0 + pc * 32 >= p.C);
      }
    };
    if (MODE == kTgAct && p.res) {
      while (pvalid && pit.c0 + pc * 32 >= p.C) pvalid = item_at(++pi, pit);
      for (int k = 0; k < kSlots - 1; ++k) res_issue();
    }
    for (int i = 0; valid; ++i) {
      it = nx;
      valid = item_at(i + 1, nx);
      const int b = i & 1;
      float* cb = col + b * 3 * kTgAccCols;
      if constexpr (MODE != kTgGrad) {
#pragma unroll
        for (int k = 0; k < 3; ++k) cb[k * kTgAccCols + te] = cv[k];
        named_bar(1, kTgEpiWarps * 32);  // and every reader of this buffer two items ago is done
        col_load(valid, nx, cv);
      }
      const int rw = it.r0 + (warp & 3) * 32, r = rw + lane;  // this warp's first row, this lane's row
      const int rows = MODE == kTgGrad ? (it.type == 0 ? p.M : p.N) : p.R;
      const int cols = MODE == kTgGrad ? p.K : p.C;
      const bool row_in = r < rows;
      float sx = 1.0f;
      if constexpr (I8) sx = row_in ? ld_dep_f32(p.sx + r) : 0.0f;
      bool ok = mbar_wait(acc_full + b, (i >> 1) & 1, abort_flag, 43);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) continue;  // (stays with the named barriers of later items)
      tc_fence_after();
      const uint32_t tacc = tmem_base + lane_off + b * kTgAccCols;
      // units of 32 columns; a result goes through one of the warp's boxes and
      // leaves by TMA, which clips the box at the tensor's edges
      if constexpr (MODE == kTgGrad) {  // the fp32 box of a share of k covers two others
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
      }
      auto box_store = [&](const CUtensorMap* m, const F2 (&y)[16], int c0) {
        uint8_t* box = boxes + slot * kTgBox;
        if (++slot == kSlots) slot = 0;
        if (MODE != kTgAct || !p.res) {  // (with a residual the box is the warp's since its load was issued)
          if (lane == 0) bulk_wait_read<kSlots - 1>();  // the box's last store has read it
          __syncwarp();
        }
        tg_box_row(box, lane, y);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rw < rows) tma_store_2d(m, box, c0, rw);
          bulk_commit();
        }
      };
      const int nunit32 = (chans + 31) / 32;
      for (int c = cg; c < nunit32; c += kTgEpiStep) {
        const int c0 = it.c0 + c * 32;
        if (c0 >= cols) break;
        uint32_t v[32];
        tmem_ld32(tacc + c * 32, v);
        F2 z[16];
        if constexpr (MODE == kTgGrad) {
          tmem_ld_wait();
          if (it.type == 0 && p.parts > 1) {
            // a share of k: fp32, through both boxes
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
            tg_box_row_f32(boxes, lane, v);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (rw < rows) tma_store_3d(&tm.D[0], boxes, c0, rw, it.src);
              bulk_commit();
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
            box_store(&tm.D[it.type == 0 ? 0 : 1 + it.src], z, c0);
          }
        } else if constexpr (MODE == kTgAct) {
          tmem_ld_wait();
          tg_pre<I8>(v, sx, cb + kTgAccCols + c * 32, cb + c * 32, z);
          with_act(p.act, [&](auto tag) {
#pragma unroll
            for (int j = 0; j < 16; ++j) z[j] = act_fwd2<decltype(tag)::value>(z[j]);
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
            mbar_wait(res_full + e * kSlots + slot, rph, abort_flag, 45);
            if (slot == kSlots - 1) rph ^= 1u;
            __syncwarp();
            const uint8_t* box = boxes + slot * kTgBox;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 rv = *reinterpret_cast<const uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
              const __half2* hr = reinterpret_cast<const __half2*>(&rv);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(hr[k]);
                z[4 * j + k] = f2_add(z[4 * j + k], f2(f.x, f.y));
              }
            }
          }
          box_store(&tm.D[0], z, c0);
          if (p.res) res_issue();
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
            for (int j = 0; j < 16; ++j) z[j] = f2_mul(act_fwd2<decltype(tag)::value>(z[j]), u[j]);
          });
          box_store(&tm.D[0], z, c0);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(release0 + b * 8u);
    }
    if (lane == 0) bulk_wait_all();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  const bool aborted = *abort_flag != 0;
  if (warp == 0 && aborted && issued > 0 && lane == 0) {
    // loads in flight write this CTA's shared memory: allow them 100 us to
    // land (a pair's loads report to its first CTA, so the second cannot
    // wait on a barrier of its own)
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000ull) __nanosleep(1000);
  }
  if (warp == 1 && crank == 0 && __any_sync(0xffffffffu, aborted)) {
    tg_commit(drain);
    mbar_wait_drain(drain, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's MMAs, commits and arrivals are done
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(2 * kTgAccCols)
                 : "memory");
  }
}

}  // namespace aria
