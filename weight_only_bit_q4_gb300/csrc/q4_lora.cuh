// Low-rank adapters beside a shared projection: what the kernels that apply them share.
//
//   y[t, n] = (W x_t)[n] + sc_a sum_{r < rank_a} B_a[n, r] u[t, r],   u[t, r] = sum_k A_a[r, k] x[t, k],
//   a = ids[t] (a outside [0, L): no adapter, the second term is absent).
//
// u is computed first ("shrink", lora_shrink_tile), in ks partial sums along K that its
// readers add in order; the second product joins the shared projection's FP32 sum before
// the one bf16 rounding.
#pragma once

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

constexpr int kShrinkThreads = 256;
constexpr int kShrinkWarps = kShrinkThreads / 32;
constexpr int kShrinkRanks = 64;    // ranks per round
constexpr int kLoraMaxRank = 256;

// Adapter of token t and its rank (0: none).  ids, ranks and scales may have been written by
// an earlier kernel of the stream: coherent loads.
__device__ __forceinline__ int lora_adapter(const LoraArgs& lo, int64_t t, int* rank) {
  const int a = (int)ld_global_u32(lo.ids + t);
  if (a < 0 || a >= lo.L) {
    *rank = 0;
    return -1;
  }
  int r = lo.R;
  if (lo.ranks != nullptr) {
    const int ra = (int)ld_global_u32(lo.ranks + a);
    r = ra < 0 ? 0 : ra < lo.R ? ra : lo.R;
  }
  *rank = r;
  return r > 0 ? a : -1;
}

// sum over the K partials, in order
__device__ __forceinline__ float lora_u(const LoraArgs& lo, int64_t T, int64_t t, int r) {
  float v = 0.f;
  for (int s = 0; s < lo.ks; ++s) v += __uint_as_float(ld_global_u32(lo.u + ((int64_t)s * T + t) * lo.R + r));
  return v;
}

// sum of 8 products of a row chunk of B (ranks r0 .. r0 + 7, those past `rank` left out
// whatever bits they hold) with u
__device__ __forceinline__ float lora_dot8(uint4 b, const float* u, int left, float v) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
  if (left >= 8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v = fmaf(bf16lo(w[i]), u[2 * i], v);
      v = fmaf(bf16hi(w[i]), u[2 * i + 1], v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * i < left) v = fmaf(bf16lo(w[i]), u[2 * i], v);
      if (2 * i + 1 < left) v = fmaf(bf16hi(w[i]), u[2 * i + 1], v);
    }
  }
  return v;
}

__device__ __forceinline__ void lora_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// u of 8 tokens over one share of K, by kShrinkThreads threads (all of them; ends with a
// barrier).  MMA rows are ranks, columns are tokens, both operands bf16 as they are (exact
// products, FP32 sums): thread (g, c) takes 8 consecutive K values of rank g, of rank g + 8
// and of token g, one 16-byte load each, and feeds two MMAs.  Tokens of the tile may have
// different adapters: each adapter present is multiplied with all 8 columns and only its
// own columns are kept.  The warps share K in steps of 32; their sums meet in `red`
// (kShrinkWarps x 8 x kShrinkRanks floats), added in warp order.
__device__ __forceinline__ void lora_shrink_tile(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, int64_t tile,
                                                 int split, float* red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t t0 = 8 * tile;
  // K shares: whole steps of 32
  const int64_t steps = (K + 31) / 32;
  const int64_t s0 = steps * split / lo.ks, s1 = steps * (split + 1) / lo.ks;
  int rank = 0;
  const int mine = t0 + g < T ? lora_adapter(lo, t0 + g, &rank) : -1;
  const unsigned active = __ballot_sync(0xffffffffu, mine >= 0 && c == 0);
  for (int rc = 0; rc < lo.R; rc += kShrinkRanks) {
    unsigned todo = active;
    while (todo) {
      const int lead = __ffs(todo) - 1;
      const int a = __shfl_sync(0xffffffffu, mine, lead);
      const int ra = __shfl_sync(0xffffffffu, rank, lead);
      todo &= ~__ballot_sync(0xffffffffu, mine == a && c == 0);
      const int ntile = (ra - rc + 15) / 16 < kShrinkRanks / 16 ? (ra - rc + 15) / 16 : kShrinkRanks / 16;
      float acc[kShrinkRanks / 16][4];
#pragma unroll
      for (int n = 0; n < kShrinkRanks / 16; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      const uint16_t* A = lo.a + ((int64_t)a * lo.R + rc) * K;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      for (int64_t st = s0 + warp; st < s1; st += kShrinkWarps) {
        const int64_t k = 32 * st + 8 * c;   // K is a multiple of 8
        const bool in = k < K;
        const uint4 xv = in && mine == a ? ld_global_u4(x + (t0 + g) * K + k) : zero;
#pragma unroll
        for (int n = 0; n < kShrinkRanks / 16; ++n) {
          if (n >= ntile) break;
          const int r = 16 * n + g;
          const uint4 p = in && rc + r < ra ? ld_global_u4(A + (int64_t)r * K + k) : zero;
          const uint4 q = in && rc + r + 8 < ra ? ld_global_u4(A + (int64_t)(r + 8) * K + k) : zero;
          lora_mma(acc[n], p.x, q.x, p.y, q.y, xv.x, xv.y);
          lora_mma(acc[n], p.z, q.z, p.w, q.w, xv.z, xv.w);
        }
      }
      // columns 2c, 2c + 1 of this thread: kept if the token is this adapter's
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = 2 * c + j;
        const int ca = __shfl_sync(0xffffffffu, mine, 4 * col);
        if (ca != a) continue;
#pragma unroll
        for (int n = 0; n < kShrinkRanks / 16; ++n) {
          red[(warp * 8 + col) * kShrinkRanks + 16 * n + g] = acc[n][j];
          red[(warp * 8 + col) * kShrinkRanks + 16 * n + g + 8] = acc[n][2 + j];
        }
      }
    }
    __syncthreads();
    const int nr = lo.R - rc < kShrinkRanks ? lo.R - rc : kShrinkRanks;
    for (int e = threadIdx.x; e < 8 * kShrinkRanks; e += kShrinkThreads) {
      const int col = e / kShrinkRanks, r = e % kShrinkRanks;
      if (r >= nr || !((active >> (4 * col)) & 1u)) continue;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kShrinkWarps; ++w) v += red[(w * 8 + col) * kShrinkRanks + r];
      if (lo.scales != nullptr) {
        const int a = (int)ld_global_u32(lo.ids + t0 + col);
        v *= __uint_as_float(ld_global_u32(lo.scales + a));
      }
      lo.u[((int64_t)split * T + t0 + col) * lo.R + rc + r] = v;
    }
    __syncthreads();
  }
}

}  // namespace q4
