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
constexpr int kShrinkTokens = 16;   // tokens per tile
constexpr int kShrinkFloats = kShrinkWarps * kShrinkTokens * kShrinkRanks;
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

// sum over the K partials, in order; kAhead loads in flight (one after the other they cost the
// reader a trip to L2 each)
template <int kAhead = 8>
__device__ __forceinline__ float lora_u(const LoraArgs& lo, int64_t T, int64_t t, int r) {
  const float* at = lo.u + t * lo.R + r;
  const int64_t step = T * lo.R;
  float v = 0.f;
  for (int s = 0; s < lo.ks; s += kAhead) {
    float f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) f[i] = s + i < lo.ks ? __uint_as_float(ld_global_u32(at + (s + i) * step)) : 0.f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) v += f[i];
  }
  return v;
}

// v as two bf16 terms (bits): hi + lo, relative error 2^-17; Inf and NaN: hi alone.  A finite v
// whose nearest bf16 would be infinite takes the largest finite one.
__device__ __forceinline__ void lora_terms(float v, uint32_t& hi, uint32_t& lo) {
  const bool finite = fabsf(v) < INFINITY;
  hi = float_to_bf16_bits(v);
  if (finite && (hi & 0x7FFFu) == 0x7F80u) --hi;
  lo = finite ? (uint32_t)float_to_bf16_bits(v - __uint_as_float(hi << 16)) : 0u;
}

// Two bf16 values with Inf and NaN taken as zero.
__device__ __forceinline__ uint32_t lora_finite2(uint32_t w) {
  return w & ~__vcmpeq2(w & 0x7F807F80u, 0x7F807F80u);
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

// Tokens of a chunk sorted by adapter and cut into tiles of at most `per` tokens of one
// adapter, so that a tile reads one adapter's rows once.  Built by every CTA that works on
// the chunk (kLoraChunk tokens cost about half a microsecond): each thread counts, for its
// token, the tokens that come before it.
constexpr int kLoraChunk = 128;

struct LoraLists {
  __align__(16) int ids[kLoraChunk];   // adapter of every token (kNoAdapter: none); then tile numbers
  short order[kLoraChunk];    // token numbers in the chunk, by adapter
  int adapter[kLoraChunk];    // per tile
  short rank[kLoraChunk];
  short first[kLoraChunk], count[kLoraChunk];
  int heads[kLoraChunk / 32];
  int ntiles;
};
constexpr int kNoAdapter = 0x7FFFFFFF;

// All threads of a CTA of at least kLoraChunk threads; ends with a barrier.  Tokens without an
// adapter get tiles too (adapter kNoAdapter, the last ones).
__device__ __forceinline__ void lora_build_lists(const LoraArgs& lo, int64_t t0, int n, int per, LoraLists& L) {
  const int i = threadIdx.x;
  int id = kNoAdapter, rank = 0;
  if (i < n) {
    const int a = lora_adapter(lo, t0 + i, &rank);
    if (a >= 0) id = a;
  }
  if (n <= 32) {   // one warp: adapters in the order of their first tokens (the none last)
    if (i < 32) {
      const unsigned live = n < 32 ? (1u << n) - 1u : 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, id) & live;
      const int before = __popc(same & ((1u << i) - 1u)), equal = __popc(same);
      const bool on = i < n, lead = on && before == 0;
      const unsigned none = __ballot_sync(0xffffffffu, i < n && id == kNoAdapter);
      const unsigned leads = __ballot_sync(0xffffffffu, lead && id != kNoAdapter);
      // sorted position and tile number of the adapter's first token: sums over the leads before it
      int pos = 0, k = 0;
      for (unsigned m = leads; m; m &= m - 1u) {
        const int l = __ffs(m) - 1;
        const int cnt = __shfl_sync(0xffffffffu, equal, l);
        if (id == kNoAdapter || l < __ffs(same) - 1) {
          pos += cnt;
          k += (cnt + per - 1) / per;
        }
      }
      if (on) L.order[pos + before] = (short)i;
      if (on && before % per == 0) {
        const int at = k + before / per;
        L.adapter[at] = id;
        L.rank[at] = (short)rank;
        L.first[at] = (short)(pos + before);
        L.count[at] = (short)(equal - before < per ? equal - before : per);
      }
      // tiles: those of the adapters, then of the tokens without one
      int total = 0;
      for (unsigned m = leads; m; m &= m - 1u) total += (__shfl_sync(0xffffffffu, equal, __ffs(m) - 1) + per - 1) / per;
      total += (__popc(none) + per - 1) / per;
      if (i == 0) L.ntiles = total;
    }
    __syncthreads();
    return;
  }
  if (i < kLoraChunk) L.ids[i] = id;
  __syncthreads();
  int less = 0, before = 0, equal = 0;
  if (i < n) {
    const int4* ids = reinterpret_cast<const int4*>(L.ids);
    for (int j = 0; j < n; j += 4) {   // (places past n hold kNoAdapter and count for nothing below)
      const int4 o4 = ids[j / 4];
      const int o[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const bool same = o[q] == id && j + q < n;
        less += o[q] < id;
        equal += same;
        before += same && j + q < i;
      }
    }
  }
  // tile heads, numbered in sorted order
  const int pos = less + before;
  __syncthreads();
  if (i < kLoraChunk) L.ids[i] = 0;
  __syncthreads();
  const bool head = i < n && before % per == 0;
  if (i < n) L.order[pos] = (short)i;
  if (head) L.ids[pos] = 1;
  __syncthreads();
  const int lane = i & 31;
  const bool mark = i < kLoraChunk && L.ids[i] != 0;
  const unsigned bal = __ballot_sync(0xffffffffu, mark);
  if (i < kLoraChunk && lane == 0) L.heads[i >> 5] = __popc(bal);
  __syncthreads();
  if (mark) {
    int k = __popc(bal & ((1u << lane) - 1u));
    for (int w = 0; w < (i >> 5); ++w) k += L.heads[w];
    L.ids[i] = k + 1;   // (only this thread reads or writes this place)
  }
  if (i == 0) {
    int k = 0;
    for (int w = 0; w < kLoraChunk / 32; ++w) k += L.heads[w];
    L.ntiles = k;
  }
  __syncthreads();
  if (head) {
    const int k = L.ids[pos] - 1;
    L.adapter[k] = id;
    L.rank[k] = (short)rank;
    L.first[k] = (short)pos;
    L.count[k] = (short)(equal - before < per ? equal - before : per);
  }
  __syncthreads();
}

// u of a tile (up to 16 tokens of one adapter) over one share of K, by kShrinkThreads threads.
// MMA rows are ranks, columns are tokens (two column tiles), both operands bf16 as they are
// (exact products, FP32 sums): thread (g, c) takes 8 consecutive K values of ranks g and
// g + 8 and of tokens g and g + 8, one 16-byte load each, and feeds two MMAs per rank tile and
// column tile.  The warps share K in steps of 32, with the loads of several steps in flight;
// their sums meet in `red` (kShrinkWarps x kShrinkTokens x kShrinkRanks floats), added in warp
// order.
template <int NR>
__device__ __forceinline__ void lora_shrink_ranks(const uint16_t* A, const uint16_t* x0, const uint16_t* x1, bool wide, int rows,
                                                  int64_t K, int64_t s0, int64_t s1, float* red) {
  constexpr int kSteps = NR == 1 ? 4 : NR == 2 ? 3 : 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  float acc[NR][2][4];
#pragma unroll
  for (int n = 0; n < NR; ++n)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.f;
  for (int64_t st = s0 + warp; st < s1; st += kSteps * kShrinkWarps) {
    uint4 xa[kSteps], xb[kSteps], p[kSteps][NR], q[kSteps][NR];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int64_t k = 32 * (st + u * kShrinkWarps) + 8 * c;   // K is a multiple of 8
      const bool in = st + u * kShrinkWarps < s1 && k < K;
      xa[u] = in ? ld_global_u4(x0 + k) : zero;
      xb[u] = in && wide ? ld_global_u4(x1 + k) : zero;
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const int r = 16 * n + g;
        p[u][n] = in && r < rows ? ld_global_u4(A + (int64_t)r * K + k) : zero;
        q[u][n] = in && r + 8 < rows ? ld_global_u4(A + (int64_t)(r + 8) * K + k) : zero;
      }
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        lora_mma(acc[n][0], p[u][n].x, q[u][n].x, p[u][n].y, q[u][n].y, xa[u].x, xa[u].y);
        lora_mma(acc[n][0], p[u][n].z, q[u][n].z, p[u][n].w, q[u][n].w, xa[u].z, xa[u].w);
        if (wide) {
          lora_mma(acc[n][1], p[u][n].x, q[u][n].x, p[u][n].y, q[u][n].y, xb[u].x, xb[u].y);
          lora_mma(acc[n][1], p[u][n].z, q[u][n].z, p[u][n].w, q[u][n].w, xb[u].z, xb[u].w);
        }
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int col = 8 * (j >> 1) + 2 * c + (j & 1);
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      red[(warp * kShrinkTokens + col) * kShrinkRanks + 16 * n + g] = acc[n][j >> 1][j & 1];
      red[(warp * kShrinkTokens + col) * kShrinkRanks + 16 * n + g + 8] = acc[n][j >> 1][2 + (j & 1)];
    }
  }
}

__device__ __forceinline__ void lora_shrink_tile(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, int64_t t0,
                                                 int tile, int split, const LoraLists& L, float* red) {
  const int a = L.adapter[tile], rank = L.rank[tile], first = L.first[tile], count = L.count[tile];
  const int g = (threadIdx.x & 31) >> 2;
  const int64_t steps = (K + 31) / 32;
  const int64_t s0 = steps * split / lo.ks, s1 = steps * (split + 1) / lo.ks;
  // an empty column's sums are dropped
  const uint16_t* x0 = x + (t0 + L.order[first + (g < count ? g : 0)]) * K;
  const uint16_t* x1 = x + (t0 + L.order[first + (g + 8 < count ? g + 8 : 0)]) * K;
  const float sc = lo.scales != nullptr ? __uint_as_float(ld_global_u32(lo.scales + a)) : 1.f;
  for (int rc = 0; rc < lo.R; rc += kShrinkRanks) {
    const uint16_t* A = lo.a + ((int64_t)a * lo.R + rc) * K;
    const int rows = rank - rc;
    if (rows > 32) lora_shrink_ranks<4>(A, x0, x1, count > 8, rows, K, s0, s1, red);
    else if (rows > 16) lora_shrink_ranks<2>(A, x0, x1, count > 8, rows, K, s0, s1, red);
    else if (rows > 0) lora_shrink_ranks<1>(A, x0, x1, count > 8, rows, K, s0, s1, red);
    __syncthreads();
    // (ranks past the adapter's are zero, whatever the buffer holds there)
    const int nr = lo.R - rc < kShrinkRanks ? lo.R - rc : kShrinkRanks;
    for (int e = threadIdx.x; e < count * kShrinkRanks; e += kShrinkThreads) {
      const int col = e / kShrinkRanks, r = e % kShrinkRanks;
      if (r >= nr) continue;
      float v = 0.f;
      if (r < rows) {
#pragma unroll
        for (int w = 0; w < kShrinkWarps; ++w) v += red[(w * kShrinkTokens + col) * kShrinkRanks + r];
      }
      lo.u[((int64_t)split * T + t0 + L.order[first + col]) * lo.R + rc + r] = sc * v;
    }
    __syncthreads();
  }
}

// Tiles of a chunk of n tokens, at most.
__host__ __device__ inline int lora_max_tiles(int n, int per, int64_t L) {
  const int64_t some = n / per + (L + 1 < n ? L + 1 : n);
  return (int)(some < n ? some : n);
}

// What the expand kernel needs to know of a tile, left by the shrink kernel (lo.tiles): adapter
// (kNoAdapter: tokens without one; -1: no such tile), rank, tokens, and their numbers in the chunk.
struct __align__(16) LoraTile {
  int adapter, rank, count, pad;
  short order[kShrinkTokens];
};
static_assert(kLoraTileBytes == sizeof(LoraTile), "workspace of the tile records");

// One CTA of the shrink product: number q of lora_shrink_blocks().
__device__ __forceinline__ void lora_shrink_block(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, int64_t q,
                                                  LoraLists& L, float* red) {
  const int n0 = (int)(T < kLoraChunk ? T : kLoraChunk);
  const int tiles = lora_max_tiles(n0, kShrinkTokens, lo.L);
  const int split = (int)(q % lo.ks);
  const int64_t chunk = q / lo.ks / tiles;
  const int tile = (int)(q / lo.ks - chunk * tiles);
  const int64_t t0 = chunk * kLoraChunk;
  const int n = (int)(T - t0 < kLoraChunk ? T - t0 : kLoraChunk);
  lora_build_lists(lo, t0, n, kShrinkTokens, L);
  const bool there = tile < L.ntiles;
  if (lo.tiles != nullptr && split == 0 && threadIdx.x < kShrinkTokens) {
    LoraTile* rec = static_cast<LoraTile*>(lo.tiles) + chunk * tiles + tile;
    const int count = there ? L.count[tile] : 0;
    rec->order[threadIdx.x] = (int)threadIdx.x < count ? L.order[L.first[tile] + threadIdx.x] : (short)0;
    if (threadIdx.x == 0) {
      rec->adapter = there ? L.adapter[tile] : -1;
      rec->rank = there ? L.rank[tile] : 0;
      rec->count = count;
    }
  }
  if (there && L.adapter[tile] != kNoAdapter) lora_shrink_tile(lo, x, K, T, t0, tile, split, L, red);
}

__host__ inline int64_t lora_shrink_blocks(const LoraArgs& lo, int64_t T) {
  const int n0 = (int)(T < kLoraChunk ? T : kLoraChunk);
  return (T + kLoraChunk - 1) / kLoraChunk * lora_max_tiles(n0, kShrinkTokens, lo.L) * lo.ks;
}

}  // namespace q4
