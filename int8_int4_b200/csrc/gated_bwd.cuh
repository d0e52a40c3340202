// gated_bwd.cuh -- the elementwise part of the gated feed-forward's backward
// pass:
//
//   dG = dH * U * act'(G),   dU = dH * act(G)
//
// from the kept pre-activations, and the column sums of both (the bias
// gradients) from the unrounded fp32 values. dG and dU are rounded to fp16,
// once: they are the operands of the two products that follow, whose other
// operands are fp16 too. An element of at least 2^-14 is off by 2^-11 of
// itself, independent from element to element, which adds about as much to
// those products as rounding their results does (2.9e-4 against 2.1e-4 in
// norm). A smaller element is off by up to 2^-25, its bits among the
// subnormals, and one above 65504 becomes infinite: dH's scale has to keep
// the two within that range, as it has to for dH itself, which is fp16. (A
// scale of the kernel's own would have to be known before the first element
// is rounded: one more pass over the three inputs.)
//
// Memory-bound: 6 bytes read and 4 written per element. A block covers 128
// columns x `rows` rows, 16 threads along the columns (8 each, 16-byte
// accesses) and 16 row lanes; a thread adds its columns over its rows, the
// row lanes meet in shared memory, and each block leaves one row of
// partials, which the last launch of the call adds in order (no atomics).
#pragma once

#include <cuda_fp16.h>
#include <cstdint>

#include "act.cuh"
#include "ptx.cuh"

namespace aria {

constexpr int kGbThreads = 256;
constexpr int kGbCols = 128;

__global__ void __launch_bounds__(kGbThreads, 3)
    gated_bwd_kernel(const __half* __restrict__ dH, const __half* __restrict__ G, const __half* __restrict__ U,
                     __half* __restrict__ dG, __half* __restrict__ dU, float* __restrict__ part, int M, int N,
                     int rows, int act) {
  __shared__ float red[2][16][kGbCols];
  pdl_wait();  // the inputs may come from the preceding kernel; the outputs may be in its hands
  pdl_launch_dependents();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int c = blockIdx.x * kGbCols + tx * 8;
  const int rb = blockIdx.y * rows, re = rb + min(rows, M - rb);
  F2 sg[4], su[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) sg[i] = su[i] = f2(0.0f);
  if (c < N) {  // N % 16 == 0: 8 columns are wholly in or out
    with_act(act, [&](auto tag) {
      // two rows' loads are always in flight: the next row's and the one's
      // behind it
      uint4 v[2][3];
      auto load = [&](int r, uint4 (&w)[3]) {
        if (r >= re) return;
        const int64_t o = static_cast<int64_t>(r) * N + c;
        w[0] = ld_dep_v4(dH + o);
        w[1] = ld_dep_v4(G + o);
        w[2] = ld_dep_v4(U + o);
      };
      auto row = [&](int r, const uint4 (&w)[3]) {
        const __half2* h2 = reinterpret_cast<const __half2*>(&w[0]);
        const __half2* g2 = reinterpret_cast<const __half2*>(&w[1]);
        const __half2* u2 = reinterpret_cast<const __half2*>(&w[2]);
        uint4 og, ou;
        __half2* og2 = reinterpret_cast<__half2*>(&og);
        __half2* ou2 = reinterpret_cast<__half2*>(&ou);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 hv = __half22float2(h2[i]), gv = __half22float2(g2[i]), uv = __half22float2(u2[i]);
          const F2 h = f2(hv.x, hv.y);
          F2 fa, da;
          act_fwd_bwd2<decltype(tag)::value>(f2(gv.x, gv.y), fa, da);
          const F2 a = f2_mul(f2_mul(h, f2(uv.x, uv.y)), da), b = f2_mul(h, fa);
          sg[i] = f2_add(sg[i], a);
          su[i] = f2_add(su[i], b);
          og2[i] = __float22half2_rn(f2_get(a));
          ou2[i] = __float22half2_rn(f2_get(b));
        }
        if (dG) {
          const int64_t o = static_cast<int64_t>(r) * N + c;
          *reinterpret_cast<uint4*>(dG + o) = og;
          *reinterpret_cast<uint4*>(dU + o) = ou;
        }
      };
      load(rb + ty, v[0]);
      load(rb + ty + 16, v[1]);
      for (int r = rb + ty; r < re; r += 32) {
        row(r, v[0]);
        load(r + 32, v[0]);
        if (r + 16 < re) {
          row(r + 16, v[1]);
          load(r + 48, v[1]);
        }
      }
    });
  }
  if (!part) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    *reinterpret_cast<float2*>(&red[0][ty][tx * 8 + 2 * i]) = f2_get(sg[i]);
    *reinterpret_cast<float2*>(&red[1][ty][tx * 8 + 2 * i]) = f2_get(su[i]);
  }
  __syncthreads();
  const int half = threadIdx.x >> 7, cc = threadIdx.x & 127;
  const int col = blockIdx.x * kGbCols + cc;
  if (col < N) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[half][i][cc];
    part[static_cast<int64_t>(blockIdx.y) * 2 * N + static_cast<int64_t>(half) * N + col] = s;
  }
}

// The end of a call whose products could not finish everything themselves:
// the column partials' sums (`part`, P rows of [2 n]; blocks 0 .. nb - 1, 64
// columns each, four threads per column so that all of its at most 64 loads
// are in flight at once) and dX from the S fp32 partials [S][count] of its
// split k (the blocks behind them). Both are added in a fixed order.
__global__ void __launch_bounds__(256)
    bwd_finish_kernel(const float* __restrict__ part, __half* __restrict__ db0, __half* __restrict__ db1, int P,
                      int n, int nb, const float* __restrict__ xpart, __half* __restrict__ dX, int S,
                      int64_t count) {
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < nb) {
    __shared__ float quarter[4][64];
    const int cc = threadIdx.x & 63, qr = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + cc;
    float s = 0.0f;
    if (c < 2 * n) {
#pragma unroll 16
      for (int i = qr; i < P; i += 4) s += ld_dep_f32(part + static_cast<int64_t>(i) * 2 * n + c);
    }
    quarter[qr][cc] = s;
    __syncthreads();
    if (qr == 0 && c < 2 * n) {
      const __half h = __float2half_rn((quarter[0][cc] + quarter[1][cc]) + (quarter[2][cc] + quarter[3][cc]));
      if (c < n) db0[c] = h;
      else db1[c - n] = h;
    }
    return;
  }
  const int64_t e = (static_cast<int64_t>(blockIdx.x - nb) * 256 + threadIdx.x) * 4;  // count % 16 == 0
  if (e >= count) return;
  F2 a = f2(0.0f), b = f2(0.0f);
#pragma unroll 4
  for (int i = 0; i < S; ++i) {
    const uint4 v = ld_dep_v4(xpart + static_cast<int64_t>(i) * count + e);
    a = f2_add(a, f2(__uint_as_float(v.x), __uint_as_float(v.y)));
    b = f2_add(b, f2(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  uint2 o;
  __half2* h = reinterpret_cast<__half2*>(&o);
  h[0] = __float22half2_rn(f2_get(a));
  h[1] = __float22half2_rn(f2_get(b));
  *reinterpret_cast<uint2*>(dX + e) = o;
}

}  // namespace aria
