// The two products of the low-rank adapters that run beside the shared projection: the
// shrink kernel (u = A x, for the decode GEMV and the tile route; the streaming warp-MMA
// route runs it inside its operand pass) and the expand kernel (the tile route's FP32 term
// delta[t, n] = sum_r B_a[n, r] u[t, r], from which its accumulators start).
//
// Bound: the adapters' rows.  A few tokens read each distinct adapter's A and B once
// (2 rank (K + N) bytes); with many tokens the FP32 term, written and read once through
// L2, is the cost.
#include "q4_lora.cuh"

namespace q4 {

namespace {

__global__ void __launch_bounds__(kShrinkThreads)
q4_lora_shrink_kernel(const LoraArgs lo, const uint16_t* x, int64_t K, int64_t T) {
  __shared__ float red[kShrinkWarps * 8 * kShrinkRanks];
  // The next kernel launches after the wait: when it starts, everything before this call
  // is complete and only u is still being written.
  pdl_wait_previous();
  pdl_launch_dependents();
  lora_shrink_tile(lo, x, K, T, blockIdx.x / lo.ks, (int)(blockIdx.x % lo.ks), red);
}

// One CTA: 8 tokens x kExpandRows weight rows.  MMA rows are weight rows, columns tokens,
// K the ranks; u enters as two bf16 terms u = hi + lo (relative error 2^-17), B as it is.
constexpr int kExpandThreads = 256;
constexpr int kExpandRows = 1024;

__global__ void __launch_bounds__(kExpandThreads)
q4_lora_expand_kernel(const LoraArgs lo, float* delta, int64_t N, int64_t T) {
  __shared__ uint32_t uh[8 * kLoraMaxRank], ul[8 * kLoraMaxRank];   // bf16 pairs' halves, one word per value
  pdl_launch_dependents();
  pdl_wait_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t t0 = 8 * (int64_t)blockIdx.x;
  int rank = 0;
  const int mine = t0 + g < T ? lora_adapter(lo, t0 + g, &rank) : -1;
  const unsigned active = __ballot_sync(0xffffffffu, mine >= 0 && c == 0);
  const int Rp = (lo.R + 15) / 16 * 16;
  for (int e = threadIdx.x; e < 8 * Rp; e += kExpandThreads) {
    const int col = e / Rp, r = e % Rp;
    float v = 0.f;
    if (r < lo.R && ((active >> (4 * col)) & 1u)) v = lora_u(lo, T, t0 + col, r);
    const uint16_t hi = float_to_bf16_bits(v);
    const float rest = v - __uint_as_float((uint32_t)hi << 16);
    uh[col * kLoraMaxRank + r] = hi;
    ul[col * kLoraMaxRank + r] = fabsf(v) < INFINITY ? float_to_bf16_bits(rest) : 0u;
  }
  __syncthreads();
  const int64_t nb = (int64_t)blockIdx.y * kExpandRows;
  for (int64_t n0 = nb + 16 * warp; n0 < nb + kExpandRows && n0 < N; n0 += 16 * (kExpandThreads / 32)) {
    const int64_t ra_ = n0 + g, rb_ = n0 + g + 8;
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    unsigned todo = active;
    while (todo) {
      const int lead = __ffs(todo) - 1;
      const int a = __shfl_sync(0xffffffffu, mine, lead);
      const int ra = __shfl_sync(0xffffffffu, rank, lead);
      todo &= ~__ballot_sync(0xffffffffu, mine == a && c == 0);
      const uint16_t* B = lo.b + (int64_t)a * N * lo.R;
      const bool col_in = mine == a;
      for (int r0 = 0; r0 < ra; r0 += 16) {
        const int r = r0 + 4 * c;      // this thread's four ranks
        const int left = ra - r;
        auto row = [&](int64_t n) {
          uint2 v = make_uint2(0u, 0u);
          if (n < N && left > 0) {
            v = ld_global_u2(B + n * lo.R + r);   // r + 3 < R: R is a multiple of 8
            if (left < 4) {                       // what is past the adapter's rank is not used
              if (left < 2) v.x &= 0xFFFFu;
              if (left < 3) v.y = 0u;
              else v.y &= 0xFFFFu;
            }
          }
          return v;
        };
        const uint2 p = row(ra_), q = row(rb_);
        uint32_t h[4] = {0u, 0u, 0u, 0u}, l[4] = {0u, 0u, 0u, 0u};
        if (col_in) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[i] = uh[g * kLoraMaxRank + r + i];
            l[i] = ul[g * kLoraMaxRank + r + i];
          }
        }
        lora_mma(d, p.x, q.x, p.y, q.y, h[0] | (h[1] << 16), h[2] | (h[3] << 16));
        lora_mma(d, p.x, q.x, p.y, q.y, l[0] | (l[1] << 16), l[2] | (l[3] << 16));
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t t = t0 + 2 * c + j;
      if (t >= T) continue;
      if (ra_ < N) delta[t * N + ra_] = d[j];
      if (rb_ < N) delta[t * N + rb_] = d[2 + j];
    }
  }
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

// K shares of the shrink pass: at most as many as keep a share at 256 K values (one step per
// warp), and no more CTAs than about two per SM.
int lora_splits(int64_t K, int64_t T) {
  const int64_t tiles = (T + 7) / 8;
  int64_t ks = (K + 255) / 256;
  const int64_t most = 304 / tiles;
  if (ks > most) ks = most;
  return (int)(ks < 1 ? 1 : ks);
}

int lora_shrink_launch(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, cudaStream_t stream) {
  const int64_t blocks = (T + 7) / 8 * lo.ks;
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)blocks, 1, 1), kShrinkThreads, stream, at);
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_lora_shrink_kernel, lo, x, K, T), "lora: shrink kernel launch");
}

int lora_expand_launch(const LoraArgs& lo, float* delta, int64_t N, int64_t T, cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = pdl_config(dim3((unsigned)((T + 7) / 8), (unsigned)((N + kExpandRows - 1) / kExpandRows), 1),
                                            kExpandThreads, stream, at);
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_lora_expand_kernel, lo, delta, N, T), "lora: expand kernel launch");
}

}  // namespace q4
