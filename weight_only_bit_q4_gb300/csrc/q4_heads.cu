// Query / key head norms with the position rotation, in one pass over the heads
// of a projection's output.
//
// For every token t and head h (D values v) of the query and the key rows:
//     z_i = v_i / sqrt(mean_j v_j^2 + eps) * w_i            (w: one weight per column,
//                                                             queries and keys apart)
//     first rot columns, angle i of position p = pos[t]:
//       halves       (z_i, z_{i+rot/2})  -> (z_i c - z_{i+rot/2} s, z_{i+rot/2} c + z_i s)
//       interleaved  (z_{2i}, z_{2i+1})  -> (z_{2i} c - z_{2i+1} s, z_{2i+1} c + z_{2i} s)
//     with (c, s) = table[p]; the other columns stay z_i.
// FP32 throughout, one rounding to bf16.
//
// Bound: the bytes of the heads, read once and written once (2 + 2 per value); the
// table rows and norm weights are shared by all heads of a token.
//
// Split: LPH = 8, 16 or 32 lanes own one head, 8 columns (one 16-byte load) each, so the
// mean of squares and the exchange with the partner column of the halves form are
// shuffles inside a warp.  A lane group takes up to kHeads heads of one token whose
// loads are issued together, and holds the token's (c, s) of its columns in registers
// for all of them; with few tokens a group takes one head, so that even one token
// spreads over the lanes of several CTAs.
#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kQkThreads = 256;
constexpr int kHeads = 4;   // heads in flight per lane group

struct QkParams {
  const uint16_t* src[2];
  uint16_t* dst[2];
  const uint16_t* w[2];
  int64_t lds[2], ldd[2];   // row strides in elements
  const float* table;       // [P, rot]: rot/2 cosines, then rot/2 sines
  const int32_t* pos;
  int64_t T, P;
  int hq, heads;            // query heads, query + key heads
  int D, rot, gpt;          // lane groups per token
  float eps;
};

template <int LPH, bool kInter>
__global__ void __launch_bounds__(kQkThreads) q4_qk_norm_rope_kernel(const QkParams p) {
  pdl_launch_dependents();
  pdl_wait_previous();
  const int64_t gid = ((int64_t)blockIdx.x * kQkThreads + threadIdx.x) / LPH;
  const int l = threadIdx.x % LPH;
  const int64_t t = gid / p.gpt;
  const int part = (int)(gid - t * p.gpt);
  // whole lane groups leave together; the shuffles below name only their own lanes
  const unsigned mask = LPH == 32 ? 0xffffffffu : ((1u << (LPH & 31)) - 1u) << ((threadIdx.x & 31) / LPH * LPH);
  if (t >= p.T) return;
  const int32_t pos = (int32_t)ld_global_u32(p.pos + t);
  if (pos < 0 || pos >= p.P) return;   // padding: this token's outputs stay as they are
  const int col = 8 * l, half = p.rot / 2;
  const bool in = col < p.D, turned = col < p.rot;
  float c[8], s[8];
  if (turned) {
    const float* row = p.table + (int64_t)pos * p.rot;
    if constexpr (kInter) {
      const float4 cc = ld_global_f4(row + col / 2), ss = ld_global_f4(row + half + col / 2);
      const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c[i] = cv[i / 2];
        s[i] = (i & 1) ? sv[i / 2] : -sv[i / 2];
      }
    } else {
      const bool second = col >= half;
      const float* base = row + (second ? col - half : col);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const float4 cc = ld_global_f4(base + 4 * v), ss = ld_global_f4(base + half + 4 * v);
        const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[4 * v + i] = cv[i];
          s[4 * v + i] = second ? sv[i] : -sv[i];
        }
      }
    }
  }
  // the lane that holds the partner columns (halves form); others exchange with themselves
  const int self = threadIdx.x & 31;
  const int mate = kInter || !turned ? self : self + (col < half ? half / 8 : -(half / 8));
  const float inv_d = 1.f / (float)p.D;

  for (int h0 = part; h0 < p.heads; h0 += kHeads * p.gpt) {
    uint4 v[kHeads];
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * p.gpt;
      const int side = h >= p.hq;
      const int hh = side ? h - p.hq : h;
      v[j] = in && h < p.heads ? ld_global_u4(p.src[side] + t * p.lds[side] + (int64_t)hh * p.D + col)
                               : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * p.gpt;
      if (h >= p.heads) break;   // uniform over the lane group
      const int side = h >= p.hq;
      const int hh = side ? h - p.hq : h;
      const uint32_t raw[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      float a[8], ss = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[2 * i] = bf16lo(raw[i]);
        a[2 * i + 1] = bf16hi(raw[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      uint32_t wr[4] = {0u, 0u, 0u, 0u};
      if (in) {
        const uint4 wv = ld_global_u4(p.w[side] + col);
        wr[0] = wv.x; wr[1] = wv.y; wr[2] = wv.z; wr[3] = wv.w;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[2 * i] = a[2 * i] * r * bf16lo(wr[i]);
        a[2 * i + 1] = a[2 * i + 1] * r * bf16hi(wr[i]);
      }
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = kInter ? a[i ^ 1] : __shfl_sync(mask, a[i], mate);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float y0 = turned ? fmaf(a[i], c[i], z[i] * s[i]) : a[i];
        const float y1 = turned ? fmaf(a[i + 1], c[i + 1], z[i + 1] * s[i + 1]) : a[i + 1];
        o[i / 2] = (uint32_t)float_to_bf16_bits(y0) | ((uint32_t)float_to_bf16_bits(y1) << 16);
      }
      if (in)
        *reinterpret_cast<uint4*>(p.dst[side] + t * p.ldd[side] + (int64_t)hh * p.D + col) =
            make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int LPH>
int qk_launch(const QkParams& p, bool inter, unsigned blocks, cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kQkThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(inter ? cudaLaunchKernelEx(&cfg, q4_qk_norm_rope_kernel<LPH, true>, p)
                          : cudaLaunchKernelEx(&cfg, q4_qk_norm_rope_kernel<LPH, false>, p),
                    "qk_norm_rope: kernel launch");
}

}  // namespace

int qk_norm_rope_launch(const QkArgs& a) {
  QkParams p{};
  p.src[0] = a.q; p.src[1] = a.k;
  p.dst[0] = a.q_out; p.dst[1] = a.k_out;
  p.w[0] = a.q_weight; p.w[1] = a.k_weight;
  p.lds[0] = a.ldq; p.lds[1] = a.ldk;
  p.ldd[0] = a.ldqo; p.ldd[1] = a.ldko;
  p.table = a.table;
  p.pos = a.pos;
  p.T = a.T;
  p.P = a.P;
  p.hq = (int)a.Hq;
  p.heads = (int)(a.Hq + a.Hk);
  p.D = (int)a.D;
  p.rot = (int)a.rot;
  p.eps = a.eps;
  const int lph = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  // heads per lane group: one while all groups of one head each still fit the GPU at once
  // (152 SMs x 2048 threads), else kHeads
  const int64_t threads1 = a.T * p.heads * lph;
  const int hpg = threads1 <= (int64_t)152 * 2048 ? 1 : kHeads;
  p.gpt = (p.heads + hpg - 1) / hpg;
  const int64_t blocks = (a.T * p.gpt * lph + kQkThreads - 1) / kQkThreads;
  if (blocks > 0x7fffffff) {
    set_error_detail("qk_norm_rope: too many tokens for one launch");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  if (lph == 8) return qk_launch<8>(p, a.interleaved, (unsigned)blocks, a.stream);
  if (lph == 16) return qk_launch<16>(p, a.interleaved, (unsigned)blocks, a.stream);
  return qk_launch<32>(p, a.interleaved, (unsigned)blocks, a.stream);
}

}  // namespace q4
