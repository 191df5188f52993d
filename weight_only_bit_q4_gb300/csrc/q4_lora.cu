// The two products of the low-rank adapters that run beside the shared projection: the
// shrink kernel (u = A x, for the decode GEMV and the tile route; the streaming warp-MMA
// route runs it inside its operand pass) and, for the tile route, either the expand kernel (the
// FP32 term delta[t, n] = sum_r B_a[n, r] u[t, r], from which its accumulators start) or, with
// few adapters of low rank, the spread kernel (u as an operand of the tile kernel, which takes the
// second product as a few more K groups).
//
// Bound: the adapters' rows.  A few tokens read each distinct adapter's A and B once
// (2 rank (K + N) bytes); with many tokens the FP32 term, written and read once through
// L2, is the cost.
#include "q4_lora.cuh"

namespace q4 {

namespace {

__global__ void __launch_bounds__(kShrinkThreads)
q4_lora_shrink_kernel(const LoraArgs lo, const uint16_t* x, int64_t K, int64_t T) {
  __shared__ float red[kShrinkFloats];
  __shared__ LoraLists L;
  // The next kernel launches after the wait: when it starts, everything before this call
  // is complete and only u is still being written.
  pdl_wait_previous();
  pdl_launch_dependents();
  lora_shrink_block(lo, x, K, T, blockIdx.x, L, red);
}

// One CTA: a tile of up to 16 tokens of one adapter (MMA rows) x `rows` weight rows.  u enters
// as two bf16 terms u = hi + lo (relative error 2^-17), B as it is.  A warp forms 32 weight
// rows at a time as four MMA column tiles whose columns are dealt so that a thread ends with
// 8 consecutive rows of a token: column g of tile i is weight row 8 (g / 2) + 2 i + g % 2.
constexpr int kExpandThreads = 256;
constexpr int kExpandTokens = kShrinkTokens;
constexpr int kExpandPitch = kLoraMaxRank / 2 + 4;   // 32-bit words per token

__global__ void __launch_bounds__(kExpandThreads, 3)   // three CTAs per SM: one wave, mostly
q4_lora_expand_kernel(const LoraArgs lo, float* delta, int64_t pitch, int64_t N, int64_t T, int rows, int tiles) {
  __shared__ __align__(16) uint32_t uh[kExpandTokens * kExpandPitch], ul[kExpandTokens * kExpandPitch];   // bf16 pairs
  // (The tile kernel launches next: the shrink kernel let this one launch after its own wait, so
  // everything but u, the tile records and delta is final by then.)
  pdl_launch_dependents();
  pdl_wait_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const LoraTile* rec = static_cast<const LoraTile*>(lo.tiles) + blockIdx.x;
  const uint4 head = ld_global_u4(rec);
  const int a = (int)head.x, rank = (int)head.y, count = (int)head.z;
  if (a < 0) return;
  const int64_t t0 = (int64_t)(blockIdx.x / tiles) * kLoraChunk;
  const short* order = rec->order;
  const int64_t nb = (int64_t)blockIdx.y * rows;
  const uint16_t* B = lo.b + (int64_t)(a == kNoAdapter ? 0 : a) * N * lo.R;
  const int row_g = 8 * (g >> 1) + (g & 1);   // + 2 i: the weight row of column g of tile i
  // the four B fragments of rows n0r .. n0r + 31 for the ranks from r0 on
  auto load_b = [&](int64_t n0r, int r0, uint2 (&b)[4]) {
    const int r = r0 + 4 * c, left = rank - r;   // this thread's four ranks
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i] = make_uint2(0u, 0u);
      const int64_t row = n0r + row_g + 2 * i;
      if (row < N && left > 0) b[i] = ld_global_u2(B + row * lo.R + r);   // R is a multiple of 8
    }
  };
  auto trim = [&](int r0, uint2 (&b)[4]) {   // what lies past the adapter's rank is not used
    const int left = rank - (r0 + 4 * c);
    if (left < 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (left < 2) b[i].x &= 0xFFFFu;
        if (left < 3) b[i].y = 0u;
        else b[i].y &= 0xFFFFu;
      }
    }
  };
  auto multiply = [&](int r0, uint2 (&b)[4], float (&d)[4][4]) {
    trim(r0, b);
    const int at = g * kExpandPitch + (r0 + 4 * c) / 2, at8 = at + 8 * kExpandPitch;
    const uint2 h0 = *reinterpret_cast<const uint2*>(uh + at), h8 = *reinterpret_cast<const uint2*>(uh + at8);
    const uint2 l0 = *reinterpret_cast<const uint2*>(ul + at), l8 = *reinterpret_cast<const uint2*>(ul + at8);
    uint32_t top = 0u;   // largest magnitudes of this thread's B
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lora_mma(d[i], h0.x, h8.x, h0.y, h8.y, b[i].x, b[i].y);
      top = __vmaxu2(top, __vmaxu2(b[i].x & 0x7FFF7FFFu, b[i].y & 0x7FFF7FFFu));
    }
    // An infinite B times u is the first term's: the second, 0 or of either sign, would make it NaN.
    if (__any_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16) >= 0x7F80u)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = make_uint2(lora_finite2(b[i].x), lora_finite2(b[i].y));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) lora_mma(d[i], l0.x, l8.x, l0.y, l8.y, b[i].x, b[i].y);
  };
  // Row steps of 32 per warp; four fragment sets in flight: four row steps of one rank step
  // (rank <= 16), or one row step of four rank steps.
  constexpr int kStride = 32 * (kExpandThreads / 32);
  const bool narrow = rank <= 16;
  const int64_t n1 = nb + 32 * warp;
  uint2 b[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (narrow ? q * kStride < rows : 16 * q < rank) load_b(narrow ? n1 + q * kStride : n1, narrow ? 0 : 16 * q, b[q]);
  }
  const int words = (rank + 15) / 16 * 8;   // whole steps of 16 ranks
  for (int e = threadIdx.x; e < kExpandTokens * words; e += kExpandThreads) {
    const int col = e / words, w = e - col * words;
    uint32_t h = 0u, l = 0u;
    if (col < count) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 2 * w + j;
        const float v = r < rank ? lora_u(lo, T, t0 + order[col], r) : 0.f;
        uint32_t hi, lw;
        lora_terms(v, hi, lw);
        h |= hi << (16 * j);
        l |= lw << (16 * j);
      }
    }
    uh[col * kExpandPitch + w] = h;
    ul[col * kExpandPitch + w] = l;
  }
  __syncthreads();
  // rows n0r + 8c .. + 7 of tokens g and g + 8 (the pitch is a multiple of 8 floats: whole
  // vectors, past N too)
  auto store = [&](int64_t n0r, const float (&d)[4][4]) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = g + 8 * j;
      if (col < count && n0r + 8 * c < pitch) {
        float4* o = reinterpret_cast<float4*>(delta + (t0 + order[col]) * pitch + n0r + 8 * c);
        o[0] = make_float4(d[0][2 * j], d[0][2 * j + 1], d[1][2 * j], d[1][2 * j + 1]);
        o[1] = make_float4(d[2][2 * j], d[2][2 * j + 1], d[3][2 * j], d[3][2 * j + 1]);
      }
    }
  };
  if (narrow) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t n0r = n1 + q * kStride;
      if (q * kStride >= rows || n0r >= N) break;
      float d[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
      if (rank > 0) multiply(0, b[q], d);
      store(n0r, d);
    }
    return;
  }
  for (int64_t n0r = n1; n0r < nb + rows && n0r < N; n0r += kStride) {
    float d[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
    for (int r0 = 0; r0 < rank; r0 += 64) {
      if (n0r > n1 || r0 > 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (r0 + 16 * q < rank) load_b(n0r, r0 + 16 * q, b[q]);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (r0 + 16 * q < rank) multiply(r0 + 16 * q, b[q], d);
    }
    store(n0r, d);
  }
}

// u as the tile route's further groups read it: [T][groups][64] bf16, groups 2 b and 2 b + 1 the
// terms hi and lo of columns 64 b .. 64 b + 63 of all adapters' ranks side by side; a token's own
// adapter's columns hold u, the others zeros.  A thread writes 8 columns.
constexpr int kSpreadThreads = 256;

__global__ void __launch_bounds__(kSpreadThreads)
q4_lora_spread_kernel(const LoraArgs lo, uint16_t* u, int groups, int64_t T) {
  pdl_launch_dependents();   // (as the expand kernel: all but u is final by now)
  pdl_wait_previous();
  const int chunks = groups * 4;   // of 8 columns, per token
  const int64_t i = (int64_t)blockIdx.x * kSpreadThreads + threadIdx.x;
  const int64_t t = i / chunks;
  if (t >= T) return;
  const int q = (int)(i - t * chunks), a = 8 * q / lo.R, r0 = 8 * q - a * lo.R;
  uint4 hi = make_uint4(0u, 0u, 0u, 0u), lw = hi;
  if (a < lo.L && (int)ld_global_u32(lo.ids + t) == a) {
    const int rank = lo.ranks == nullptr ? lo.R : min(max((int)ld_global_u32(lo.ranks + a), 0), lo.R);
    uint32_t h[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = r0 + j < rank ? lora_u(lo, T, t, r0 + j) : 0.f;
      lora_terms(v, h[j], l[j]);
    }
    hi = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    lw = make_uint4(l[0] | l[1] << 16, l[2] | l[3] << 16, l[4] | l[5] << 16, l[6] | l[7] << 16);
  }
  uint4* o = reinterpret_cast<uint4*>(u + (t * groups + 2 * (q >> 3)) * 64) + (q & 7);
  o[0] = hi;
  o[8] = lw;
}

cudaLaunchConfig_t pdl_config(dim3 grid, unsigned threads, cudaStream_t stream, cudaLaunchAttribute* at) {
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

// K shares of the shrink product: at most as many as keep a share at 256 K values (one step per
// warp), and about one CTA per SM for the tiles that the tokens are likely to make (each sorts its chunk first).  With more
// than 32 tokens at most 8: the expand kernel's every CTA adds the shares of its tokens.
int lora_splits(int64_t K, int64_t T, int64_t L) {
  const int64_t n0 = T < kLoraChunk ? T : kLoraChunk, chunks = (T + kLoraChunk - 1) / kLoraChunk;
  const int64_t likely = chunks * (n0 / kShrinkTokens + ((L + 1 < n0 ? L + 1 : n0) + 1) / 2);
  int64_t ks = (K + 255) / 256;
  const int64_t most = 168 / likely;
  if (ks > most) ks = most;
  if (T > 32 && ks > 8) ks = 8;
  return (int)(ks < 1 ? 1 : ks);
}

int64_t lora_shrink_grid(const LoraArgs& lo, int64_t T) { return lora_shrink_blocks(lo, T); }

int64_t lora_records(int64_t T, int64_t L) {
  return (T + kLoraChunk - 1) / kLoraChunk * lora_max_tiles((int)(T < kLoraChunk ? T : kLoraChunk), kShrinkTokens, L);
}

int64_t lora_delta_pitch(int64_t N) { return (N + 7) / 8 * 8; }

int lora_shrink_launch(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)lora_shrink_blocks(lo, T), 1, 1), kShrinkThreads, stream, at);
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_lora_shrink_kernel, lo, x, K, T), "lora: shrink kernel launch");
}

int lora_expand_launch(const LoraArgs& lo, float* delta, int64_t N, int64_t T, cudaStream_t stream) {
  const int n0 = (int)(T < kLoraChunk ? T : kLoraChunk);
  const int64_t tiles = lora_records(T, lo.L);
  // a warp's 32 rows per CTA where that fills the GPU about once, else four times as many
  const int rows = tiles * ((N + 255) / 256) <= 608 ? 256 : 1024;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)tiles, (unsigned)((N + rows - 1) / rows), 1), kExpandThreads,
                                            stream, at);
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_lora_expand_kernel, lo, delta, lora_delta_pitch(N), N, T, rows,
                                       lora_max_tiles(n0, kExpandTokens, lo.L)),
                    "lora: expand kernel launch");
}

// The tile route's second product as further K groups, two per 64 ranks of all adapters together
// (hi and lo).  Against delta it saves the FP32 term's way through memory and lets the tile kernel
// start before u is complete, but multiplies every token by every adapter, and the groups' A
// stages come by plain loads.  Measured (K = 5120): 2 groups always win (N = 6144: 26.0 us for
// 31.6 at T = 40, 44.8 for 55.5 at 256, 110.5 for 118.1 at 1024), 4 do from K = 4096 on (29.6 for
// 32.0, 48.5 for 56.3, 117.5 for 118.6; K = 2048: 20.4 for 19.5), 8 lose (35.0 for 31.9).
int64_t lora_groups(int64_t K, int64_t L, int64_t R) {
  const int64_t g = L <= 16 ? 2 * ((L * R + 63) / 64) : 8;   // (R is at least 8)
  return g <= 2 || (g <= 4 && K >= 4096) ? g : 0;
}

int lora_spread_launch(const LoraArgs& lo, uint16_t* u, int groups, int64_t T, cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  const int64_t n = T * groups * 4;
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((n + kSpreadThreads - 1) / kSpreadThreads), 1, 1), kSpreadThreads,
                                            stream, at);
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_lora_spread_kernel, lo, u, groups, T), "lora: spread kernel launch");
}

}  // namespace q4
