// Attention over whole prompts: causal, grouped heads, sequences packed after one another.
//
// For token t (row i of its sequence) and query head h of group g:
//     y = sum_{j <= i} p_j v_j / sum_{j <= i} p_j,  p_j = 2^((q . k_j) scale log2 e - m),
// over the tokens j of the same sequence, m the running maximum.  Scores, maxima and sums are FP32.
// P enters the second product as bf16, its operands' type (V is bf16): 2^-9 of each weight,
// as much as the output's own rounding.
#include <cfloat>

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kPtThreads = 128;
constexpr int kPtM = 64, kPtN = 64;   // query rows and keys of a tile

struct PtParams {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t ldq, ldk, ldv, ldo;
  const int32_t* cu;        // [S + 1]
  int64_t T;
  int S, Hq, G, D, tiles;
  float c;                  // scale * log2 e
};

// Rows [a, b) of sequence s, within the tensors whatever cu holds.
__device__ __forceinline__ void pt_rows(const PtParams& p, int s, int64_t& a, int64_t& b) {
  a = (int32_t)ld_global_u32(p.cu + s);
  b = (int32_t)ld_global_u32(p.cu + s + 1);
  a = a < 0 ? 0 : a > p.T ? p.T : a;
  b = b < a ? a : b > p.T ? p.T : b;
}

__device__ __forceinline__ void pt_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ float pt_ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}

__device__ __forceinline__ uint32_t pt_pack(float lo, float hi) {
  return (uint32_t)float_to_bf16_bits(lo) | (uint32_t)float_to_bf16_bits(hi) << 16;
}

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint4 w) {
  const uint32_t x = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(x & 0xFFFFu, x >> 16) >= 0x7F80u;
}

// The same with those as zeros.
__device__ __forceinline__ uint4 finite_only(uint4 w) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((x[i] & 0x7F80u) == 0x7F80u) x[i] &= 0xFFFF0000u;
    if ((x[i] & 0x7F800000u) == 0x7F800000u) x[i] &= 0xFFFFu;
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// The tile `index` of all sequences' query tiles, the last tiles of a sequence first: its
// sequence's rows and its number within the sequence.  False: there are fewer tiles.
struct PtTile {
  int64_t a, b;
  int tile;
};
__device__ __forceinline__ bool pt_find(const PtParams& p, int64_t index, PtTile* found, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found->tile = -1;
  int64_t before = 0;
  for (int s0 = 0; s0 < p.S; s0 += kPtThreads) {
    int64_t a = 0, b = 0;
    if (s0 + tid < p.S) pt_rows(p, s0 + tid, a, b);
    const int64_t n = (b - a + kPtM - 1) / kPtM;
    int64_t upto = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kPtThreads / 32; ++w) {
      if (w < warp) upto += sums[w];
      all += sums[w];
    }
    upto += before;
    if (index < upto && index >= upto - n) {
      found->a = a;
      found->b = b;
      found->tile = (int)(upto - 1 - index);
    }
    before += all;
    if (index < before) break;   // (uniform)
  }
  __syncthreads();
  return found->tile >= 0;
}

template <int DP>
__global__ void __launch_bounds__(kPtThreads) q4_prompt_kernel(const PtParams p) {
  constexpr int pitch = DP * 2 + 16;   // bytes
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ PtTile found;
  __shared__ int64_t sums[kPtThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const uint32_t sq = smem_u32(smem), sk = sq + kPtM * pitch, sv = sk + kPtN * pitch;
  pdl_launch_dependents();
  pdl_wait_previous();
  const int h = blockIdx.x % p.Hq;
  if (!pt_find(p, blockIdx.x / p.Hq, &found, sums)) return;
  const int64_t row0 = found.a;
  const int len = (int)(found.b - found.a), q0 = found.tile * kPtM;
  auto load = [&](const uint16_t* src, int64_t ld, int head, uint32_t dst, int from) {
    for (int i = tid; i < kPtM * (DP / 8); i += kPtThreads) {
      const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (from + r < len && d < p.D) w = ld_global_u4(src + (row0 + from + r) * ld + (int64_t)head * p.D + d);
      st_shared_v4(dst + (uint32_t)(r * pitch + d * 2), w);
    }
  };
  load(p.q, p.ldq, h, sq, q0);
  __syncthreads();
  uint32_t qa[DP / 16][4];
#pragma unroll
  for (int i = 0; i < DP / 16; ++i)
    ldsm4(qa[i], sq + (uint32_t)((warp * 16 + (lane & 15)) * pitch + i * 32 + (lane >> 4) * 16));
  float o[DP / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < DP / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int rows[2] = {q0 + warp * 16 + g, q0 + warp * 16 + g + 8};
  const int hk = h / p.G;
  for (int k0 = 0; k0 < min(len, q0 + kPtM); k0 += kPtN) {
    __syncthreads();
    load(p.k, p.ldk, hk, sk, k0);
    const bool edge = k0 + kPtN > q0;   // some rows do not see all of these keys
    int odd = 0;
    for (int i = tid; i < kPtN * (DP / 8); i += kPtThreads) {
      const int r = i / (DP / 8), d = (i - r * (DP / 8)) * 8;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (k0 + r < len && d < p.D) w = ld_global_u4(p.v + (row0 + k0 + r) * p.ldv + (int64_t)hk * p.D + d);
      if (edge && not_finite(w)) {   // 0 times infinity would reach rows that do not see this key
        odd = 1;
        w = finite_only(w);
      }
      st_shared_v4(sv + (uint32_t)(r * pitch + d * 2), w);
    }
    odd = __syncthreads_or(odd);
    float s[kPtN / 8][4];
#pragma unroll
    for (int n = 0; n < kPtN / 8; ++n) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < DP / 16; i += 2) {
        uint32_t b[4];
        ldsm4(b, sk + (uint32_t)((n * 8 + (lane & 7)) * pitch + i * 32 + (lane >> 3) * 16));
        pt_mma(s[n], qa[i], b[0], b[1]);
        pt_mma(s[n], qa[i + 1], b[2], b[3]);
      }
    }
    float top[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < kPtN / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] *= p.c;
        if (edge && k0 + n * 8 + 2 * c + (e & 1) > rows[e >> 1]) s[n][e] = -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const float f = top[r] == m[r] ? 1.f : pt_ex2(m[r] - top[r]);
      m[r] = top[r];
      l[r] *= f;
#pragma unroll
      for (int i = 0; i < DP / 8; ++i) {
        o[i][2 * r] *= f;
        o[i][2 * r + 1] *= f;
      }
      if (top[r] == -INFINITY) top[r] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < kPtN / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = pt_ex2(s[n][e] - top[e >> 1]);
        l[e >> 1] += s[n][e];
      }
#pragma unroll
    for (int n = 0; n < kPtN / 16; ++n) {
      const uint32_t pa[4] = {pt_pack(s[2 * n][0], s[2 * n][1]), pt_pack(s[2 * n][2], s[2 * n][3]),
                              pt_pack(s[2 * n + 1][0], s[2 * n + 1][1]), pt_pack(s[2 * n + 1][2], s[2 * n + 1][3])};
#pragma unroll
      for (int i = 0; i < DP / 8; i += 2) {
        uint32_t b[4];
        ldsm4t(b, sv + (uint32_t)((n * 16 + (lane & 15)) * pitch + (i + (lane >> 4)) * 16));
        pt_mma(o[i], pa, b[0], b[1]);
        pt_mma(o[i + 1], pa, b[2], b[3]);
      }
    }
    if (odd) {   // what was left out above, for the rows that see it
      for (int j = k0; j < min(len, k0 + kPtN); ++j) {
        const uint16_t* src = p.v + (row0 + j) * p.ldv + (int64_t)hk * p.D;
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) {
          if (8 * i >= p.D) break;
          const uint4 w = ld_global_u4(src + 8 * i);
          if (!not_finite(w)) continue;
          const uint32_t x = c == 0 ? w.x : c == 1 ? w.y : c == 2 ? w.z : w.w;
          const float v2[2] = {bf16lo(x), bf16hi(x)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (j <= rows[e >> 1] && !(fabsf(v2[e & 1]) <= FLT_MAX)) o[i][e] += v2[e & 1];
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (rows[r] >= len) continue;
    const float f = 1.f / l[r];
    uint16_t* dst = p.out + (row0 + rows[r]) * p.ldo + (int64_t)h * p.D;
#pragma unroll
    for (int i = 0; i < DP / 8; ++i)
      if (8 * i < p.D) *reinterpret_cast<uint32_t*>(dst + 8 * i + 2 * c) = pt_pack(o[i][2 * r] * f, o[i][2 * r + 1] * f);
  }
}

template <int DP>
int pt_run(const PtParams& p, unsigned blocks, cudaStream_t stream) {
  constexpr int smem = 3 * kPtM * (DP * 2 + 16);
  static bool set[64] = {};
  int dev = 0;
  if (cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return Q4LIN_ERR_CUDA;
  if (dev >= 64 || !set[dev]) {
    if (cuda_check(cudaFuncSetAttribute(q4_prompt_kernel<DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                   "prompt_attention: cudaFuncSetAttribute(max dynamic shared memory)"))
      return Q4LIN_ERR_CUDA;
    if (dev < 64) set[dev] = true;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kPtThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_prompt_kernel<DP>, p), "prompt_attention: kernel launch");
}

}  // namespace

int prompt_launch(const PromptArgs& a) {
  PtParams p{a.q, a.k, a.v, a.out, a.ldq, a.ldk, a.ldv, a.ldo, a.cu, a.T, (int)a.S, (int)a.Hq, (int)(a.Hq / a.Hk), (int)a.D, 0,
             a.scale * 1.4426950408889634f};
  // tiles: at most one that is not full per sequence
  const int64_t blocks = ((a.T + kPtM - 1) / kPtM + a.S) * a.Hq;
  if (blocks > 0x7fffffff) {
    set_error_detail("prompt_attention: too many tokens for one launch");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  return a.D <= 64 ? pt_run<64>(p, (unsigned)blocks, a.stream) : pt_run<128>(p, (unsigned)blocks, a.stream);
}

}  // namespace q4
