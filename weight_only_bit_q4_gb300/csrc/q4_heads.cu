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
// Split: LPH = 8, 16 or 32 lanes own one head, 8 columns each as two runs of four (8-byte
// loads): in the halves form the columns 4 l .. and rot/2 + 4 l .., so that a rotation stays
// inside a thread, otherwise 8 adjacent columns.  A lane group takes up to kHeads heads of one
// token whose loads are issued together, and holds the token's (c, s) of its columns and the
// norm weights in registers for all of them; with few tokens a group takes one head, so that
// even one token spreads over the lanes of several CTAs.  Arithmetic on pairs (packed FP32):
// the pass is close enough to the issue rate that scalar arithmetic and partner shuffles
// cost it a third.
#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kQkThreads = 128;
constexpr int kHeads = 5;   // heads in flight per lane group

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

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

__device__ __forceinline__ float2 unpack2(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

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
  const int half = p.rot / 2;
  const bool in = 8 * l < p.D, turned = 8 * l < p.rot;
  const int c0 = !kInter && turned ? 4 * l : 8 * l, c1 = !kInter && turned ? half + 4 * l : 8 * l + 4;
  // head h: the query rows, then (h counted on) the key rows
  const uint16_t* src_q = p.src[0] + t * p.lds[0];
  const uint16_t* src_k = p.src[1] + t * p.lds[1] - (int64_t)p.hq * p.D;
  uint16_t* dst_q = p.dst[0] + t * p.ldd[0];
  uint16_t* dst_k = p.dst[1] + t * p.ldd[1] - (int64_t)p.hq * p.D;
  // the heads' loads first: they depend on nothing, the table's on the position
  uint2 v0[kHeads], v1[kHeads];
  auto load_heads = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * p.gpt;
      v0[j] = v1[j] = make_uint2(0u, 0u);
      if (in && h < p.heads) {
        const uint16_t* s = (h < p.hq ? src_q : src_k) + h * p.D;
        v0[j] = ld_global_u2(s + c0);
        v1[j] = ld_global_u2(s + c1);
      }
    }
  };
  load_heads(part);
  const int32_t pos = (int32_t)ld_global_u32(p.pos + t);
  uint2 wq0 = make_uint2(0u, 0u), wq1 = wq0, wk0 = wq0, wk1 = wq0;
  if (in) {
    if (p.hq > 0) {
      wq0 = ld_global_u2(p.w[0] + c0);
      wq1 = ld_global_u2(p.w[0] + c1);
    }
    if (p.hq < p.heads) {
      wk0 = ld_global_u2(p.w[1] + c0);
      wk1 = ld_global_u2(p.w[1] + c1);
    }
  }
  if (pos < 0 || pos >= p.P) return;   // padding: this token's outputs stay as they are
  // four angles: of columns c0 .. c0 + 3 (halves), or of the pairs 8l / 2 .. + 3 (interleaved)
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turned) {
    const float* row = p.table + (int64_t)pos * p.rot + 4 * l;
    c = ld_global_f4(row);
    s = ld_global_f4(row + half);
  }
  const float inv_d = 1.f / (float)p.D;

  for (int h0 = part; h0 < p.heads; h0 += kHeads * p.gpt) {
    if (h0 != part) load_heads(h0);
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      const int h = h0 + j * p.gpt;
      if (h >= p.heads) break;   // uniform over the lane group
      const bool key = h >= p.hq;
      float2 a[4] = {unpack2(v0[j].x), unpack2(v0[j].y), unpack2(v1[j].x), unpack2(v1[j].y)};
      float2 q = fmul2(a[0], a[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) q = ffma2(a[i], a[i], q);
      float ss = q.x + q.y;
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(mask, ss, o);
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float2 rr = make_float2(r, r);
      a[0] = fmul2(fmul2(a[0], rr), unpack2(key ? wk0.x : wq0.x));
      a[1] = fmul2(fmul2(a[1], rr), unpack2(key ? wk0.y : wq0.y));
      a[2] = fmul2(fmul2(a[2], rr), unpack2(key ? wk1.x : wq1.x));
      a[3] = fmul2(fmul2(a[3], rr), unpack2(key ? wk1.y : wq1.y));
      if (turned) {   // (columns past rot keep their bits: an infinity there does not meet a zero sine)
        if constexpr (kInter) {
          const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a[i] = make_float2(fmaf(a[i].x, cv[i], -a[i].y * sv[i]), fmaf(a[i].y, cv[i], a[i].x * sv[i]));
        } else {
          const float2 cc[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)}, sn[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float2 u = a[i], w = a[2 + i];
            a[i] = ffma2(u, cc[i], fmul2(make_float2(-w.x, -w.y), sn[i]));
            a[2 + i] = ffma2(w, cc[i], fmul2(u, sn[i]));
          }
        }
      }
      if (in) {
        uint16_t* d = (key ? dst_k : dst_q) + h * p.D;
        *reinterpret_cast<uint2*>(d + c0) = make_uint2(pack2(a[0]), pack2(a[1]));
        *reinterpret_cast<uint2*>(d + c1) = make_uint2(pack2(a[2]), pack2(a[3]));
      }
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
