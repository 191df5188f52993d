// Mixture-of-experts layer with Q4_G64_FP16 experts, for a few tokens.
//
//   router    l[t, e] = sum_h x[t, h] wr[e, h] (+ bias[e]),  p = softmax(l[t, :]),
//             the top_k experts of each token by l (ties: the lowest e first), their p
//             (divided by their sum if asked);
//   gate/up   h[t, j, f] = silu(g) u,  g = sum_k W_gate[e, f, k] x[t, k],  u likewise with
//             W_up, e = ids[t, j], silu(z) = z / (1 + e^-z);
//   down      y[t, n] = bf16( sum_j p[t, j] sum_f W_down[e, n, f] h[t, j, f] ).
//
// The router (with the conversion of x beside it), gate/up, down and, for more slots, a sum
// over the choices: kernels chained by programmatic dependent launch.  Bound: the packed weights of
// the experts that some token chose, each read once; the kernels below therefore sort
// the (token, choice) slots by expert and stream each chosen expert's rows once for all
// of its tokens that fit a tile (up to 8 token columns, fewer where columns are long).
//
// Products.  mma.sync m16n8k16 (fp16 x fp16 -> fp32); the 64 weights of a scale group go
// through four MMAs into a fresh D, then acc += s D in FP32.  A: a masked nibble pair is the
// fp16 subnormal pattern q 2^-24 (16 q 2^-24 for the odd nibbles, which meet B / 16), one AND
// per two weights.  B: the vector v as fp16 at a power of two 2^-e that puts its largest |v|
// in [2^14, 2^15); D starts from the group's zero-point term -8 2^-24 sum v, and 2^(24 + e) is
// undone on the FP32 sum.
//   gate/up: v = x (bf16), exact down to 2^-27 of the largest |x| and within 2^-35 of it
//     below (the odd nibbles' sixteenth costs four bits).
//   down: v = h (FP32), as two fp16 terms v = hi + lo (relative error 2^-22; one term, 2^-11,
//     shows in y: 1e-4 of its rms, and single bf16 steps).  In a tile of up to four slots the lo
//     terms are columns of their own, which would be empty otherwise (kPairs); in a wider one
//     their products follow the hi terms' into the same D.  Against one term: 20.1 us for 20.2
//     (1 token, 8 of 64, 2048 x 768), 32.7 for 32.4 (4, 2 of 8, 5120 x 1408), 32.9 for 32.2 (19,
//     3 of 20, 1992 x 1016), 89.4 for 88.4 (64, 8 of 128, 2048 x 768), 82 for 72.7 with 32
//     tokens per expert (64, 4 of 8, 2048 x 2048).
//
// Operand layout, as in the streaming warp-MMA route: the K order inside an MMA is free as
// long as A and B agree, so thread (g = lane / 4, c = lane % 4) takes the 16 weights
// k = 16 c .. 16 c + 15 of a group (8 code bytes per row) and the same 16 values of token
// column g (two 16-byte loads of fragments stored in the pairs (k, k + 4) of the masks).
//
// A warp takes one tile of 8 columns at a time.  Two (16 tokens of an expert per pass over its rows)
// spill registers, and lost at every load: 64 tokens x 8 of 64, 2048 x 768 98 us for 70; x 2 of 8,
// 5120 x 1408 112 for 83; 512 x 1 of 8, 4096 x 2048 305 for 218; no gain anywhere.
//
// A unit is 16 MT MMA rows = two boxes of 8 MT weight rows: gate rows f0 .. over up rows
// f0 .. (a thread then holds g and u of the same f and token), or 16 MT rows of W_down.
// Box row of MMA row g is 2g mod 8 (+ 1 from g = 4): in the 128-byte-swizzled box the
// 8-byte code loads of a half warp then hit 16 different bank pairs.
//
// Streaming.  Every warp owns a ring of shared-memory slots, one sub-box (two boxes of
// 8 MT rows x 256 weights, TMA) each, and works through its own sequence of (unit,
// sub-box): lane 0 refills a slot as soon as the warp has read it, across unit borders, so
// no warp waits for another.  The columns of a CTA's next few tiles lie in shared memory
// beside the rings; read through L1 instead they cost the whole layer 12 us of
// 103 at 64 tokens x 8 of 128 experts (one term of h).  Gate/up copies what the operand pass has converted
// (bulk copies; plain loads by all warps spill and cost 9 us there); down converts h itself, in
// every CTA that needs the slot (a conversion kernel between the products took 3.6 us of 90.7).
//
// Three forms, by the number of slots S = T top_k of a pass and the items of a CTA (moe_plan):
//   S <= kLatSlots, and every slot's h fits shared memory: latency.  MT = 1, the K range of a unit
//     shared by up to 4 warps (partial sums joined in shared memory); every CTA of the down product
//     converts all of h itself, owns whole units and adds its slots' sums in shared memory.  (At 80
//     registers a down CTA of 8 warps fits beside the gate/up CTA and starts early, but both then
//     spill and run at half speed: one token of 8 of 64 experts took 25.8 us against 22.2.)
//   otherwise: throughput.  MT = 2 (each B fragment feeds
//     two MMA row tiles); the (tile, unit) pairs are dealt evenly over all CTAs, the slots'
//     sums of the down product go to the workspace and a last kernel adds them in the order of
//     the choices;
//   or, for a product with few items per CTA (moe_joins) or with long columns, joined: the same with
//     MT = 1 and the K range of an item shared by up to 4 warps, as in the latency form, whose
//     gate/up it is.
// Long F: the joined down product runs in chunks of F columns, a launch each, so that a tile keeps
// its four or eight slots; the last kernel adds the chunks' sums.
//
// Every mbarrier wait is bounded (kSpinLimit): on expiry the kernel records
// Q4LIN_ERR_TIMEOUT, the warps stop computing, pass the CTA barriers and drain the
// copies that they issued.
#include <cmath>

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

__device__ int g_moe_status = 0;

constexpr int kLatSlots = 16;               // up to here the latency form
enum { kThroughput = 0, kLatency = 1, kJoined = 2 };
constexpr int kMaxParts = 4;                // warps that share the K range of an item, at most
constexpr int kMoeWarps = 16;
__host__ __device__ constexpr int slot_bytes(int mt) { return 2 * 8 * mt * 128; }
constexpr int kMaxSlots = 512;              // (token, choice) pairs per pass
constexpr int kMaxExperts = 1024;

// ----------------------------------------------------------------- router
constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 512;
constexpr int kRouteMma = 4;      // tokens from which the products run on the tensor cores

struct RouterParams {
  const uint16_t* x;      // [T, H]
  const uint16_t* w;      // [E, H]
  const float* bias;      // [E] or NULL
  int32_t* ids;           // [T, k]
  float* weights;         // [T, k]
  int64_t T, H;
  int E, k, renorm;
  // the operand pass of the experts' first pass, beside the router (prep_tokens 0: none)
  uint8_t* xf;            // fragments, zero-point terms, powers of two: see moe_prep_token
  float* zs;
  float* ft;
  int prep_tokens;
  int clusters;           // clusters that route; the CTAs of the others prepare one token each
  int parts;              // shares of H per expert (E * parts <= 128, or 1)
};

// Eight values (k .. k + 7) as fp16 at scale s1 (s16 = s1 / 16 for the odd ones) in B-fragment
// order -- registers (0, 4), (1, 5) / 16, (2, 6), (3, 7) / 16 -- and the sum of what the MMA
// will see of them.
__device__ __forceinline__ uint4 moe_fragment(const float (&f)[8], float s1, float s16, float& sum) {
  uint32_t b[4];
  sum = 0.f;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float sc = (q & 1) ? s16 : s1;
    const __half2 h = __floats2half2_rn(f[q] * sc, f[q + 4] * sc);
    const float2 v = __half22float2(h);
    b[q] = *reinterpret_cast<const uint32_t*>(&h);
    sum += (v.x + v.y) * ((q & 1) ? 16.f : 1.f);
  }
  return make_uint4(b[0], b[1], b[2], b[3]);
}

// The same as two fp16 terms v = hi + lo (relative error 2^-22, which the sum need not follow).
__device__ __forceinline__ uint4 moe_fragment2(const float (&f)[8], float s1, float s16, uint4& low, float& sum) {
  uint32_t b[4], l[4];
  float v[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float sc = (q & 1) ? s16 : s1;
    v[q] = f[q] * sc;
    v[q + 4] = f[q + 4] * sc;
    const __half2 h = __floats2half2_rn(v[q], v[q + 4]);
    const float2 r = __half22float2(h);
    const __half2 lo = __floats2half2_rn(v[q] - r.x, v[q + 4] - r.y);
    b[q] = *reinterpret_cast<const uint32_t*>(&h);
    l[q] = *reinterpret_cast<const uint32_t*>(&lo);
  }
  sum = ((v[0] + v[4]) + (v[2] + v[6])) + 16.f * ((v[1] + v[5]) + (v[3] + v[7]));
  low = make_uint4(l[0], l[1], l[2], l[3]);
  return make_uint4(b[0], b[1], b[2], b[3]);
}

constexpr float kZeroTerm = -8.f * 5.9604644775390625e-8f;   // -8 2^-24
constexpr float kCodePower = 16777216.f;                       // 2^24

__host__ __device__ inline int64_t moe_groups(int64_t H) { return (H + 63) / 64; }
__host__ __device__ inline int64_t moe_zs_pitch(int64_t H) { return (moe_groups(H) + 3) / 4 * 4; }

// Where run i of 8 K values goes inside a column's fragments: group i / 8 (128 bytes), the
// first or second 8 of thread c = (i % 8) / 2.
__device__ __forceinline__ int moe_fragment_at(int i) { return (i >> 3) * 128 + (i & 1) * 64 + ((i & 7) >> 1) * 16; }

// Operand pass of one token, by all threads of a CTA (a multiple of 32, at most 512): x as
// fp16 fragments, zeros past H; per group its zero-point term; and 2^(24 + e).  Tokens
// holding Inf or NaN keep e = 0 so that those values propagate.
__device__ __forceinline__ void moe_prep_token(const uint16_t* x, int64_t H, uint8_t* xf, float* zs, float* ft) {
  __shared__ uint32_t wmax[16];
  const int tid = threadIdx.x, nth = blockDim.x;
  const int nv = (int)(H / 8), nv64 = (int)((H + 63) / 64) * 8;
  uint32_t m2 = 0;
  for (int i = tid; i < nv; i += nth) {
    const uint4 v = ld_global_u4(x + 8 * (int64_t)i);
    m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
  }
  const uint32_t own = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
  if ((tid & 31) == 0) wmax[tid >> 5] = own;
  __syncthreads();
  uint32_t mx = wmax[0];
  for (int w = 1; w < nth / 32; ++w) mx = max(mx, wmax[w]);
  const int E = (int)(mx >> 7);   // bf16 biased exponent of the largest |x|
  const int e = (mx == 0 || E == 255) ? 0 : min(max(E - 141, -100), 100);
  const float s1 = exp2i(-e), s16 = exp2i(-e - 4);
  // 8 values per thread; the 8 threads of a group are adjacent lanes (nv64 is a multiple of 8)
  for (int i = tid; i - (tid & 31) < nv64; i += nth) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (i < nv) v = ld_global_u4(x + 8 * (int64_t)i);
    const float f[8] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y), bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w)};
    float sum;
    const uint4 b = moe_fragment(f, s1, s16, sum);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < nv64) {
      *reinterpret_cast<uint4*>(xf + moe_fragment_at(i)) = b;
      if ((i & 7) == 0) zs[i >> 3] = kZeroTerm * sum;
    }
  }
  if (tid == 0) *ft = exp2i(24 + e);
}

// The same of one slot's h (FP32, F values), by one warp and as two terms.  The first 256 kRuns
// values are read once and held in registers between the maximum and the conversion, the others
// are read for both, 256 kRest at a time (together; one after the other they cost a trip to L2
// each, but the throughput form has no registers left for more than one).
template <int kRuns, int kRest>
__device__ __forceinline__ void moe_prep_slot(const float* h, int F, uint8_t* hf, float* zs, float* ft) {
  constexpr int kLanes = 32;
  const int lane = threadIdx.x % kLanes;
  const int nv = F / 8, nv64 = (F + 63) / 64 * 8;
  float4 keep[kRuns][2];
  uint32_t mx = 0;   // FP32 magnitude bits
  auto load = [&](int i, float4 (&v)[2]) {
    v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < nv) {
      v[0] = ld_global_f4(h + 8 * (int64_t)i);
      v[1] = ld_global_f4(h + 8 * (int64_t)i + 4);
    }
  };
  auto magnitude = [&](const float4 (&v)[2]) {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      mx = max(max(max(mx, __float_as_uint(v[q].x) & 0x7FFFFFFFu), max(__float_as_uint(v[q].y) & 0x7FFFFFFFu, __float_as_uint(v[q].z) & 0x7FFFFFFFu)),
               __float_as_uint(v[q].w) & 0x7FFFFFFFu);
  };
  for (int i0 = kRuns * kLanes; i0 < nv64; i0 += kRest * kLanes) {
    float4 v[kRest][2];
#pragma unroll
    for (int u = 0; u < kRest; ++u) load(i0 + u * kLanes + lane, v[u]);
#pragma unroll
    for (int u = 0; u < kRest; ++u) magnitude(v[u]);
  }
#pragma unroll
  for (int u = 0; u < kRuns; ++u) load(lane + u * kLanes, keep[u]);
#pragma unroll
  for (int u = 0; u < kRuns; ++u) magnitude(keep[u]);
  mx = __reduce_max_sync(0xffffffffu, mx);
  const int E = (int)(mx >> 23);
  // (h, the product of two sums, may have any FP32 magnitude; 2^(24 + e) might be none, so the
  // sums take 2^24 and 2^e one after the other)
  const int e = (mx == 0 || E == 255) ? 0 : min(max(E - 141, -126), 113);
  const float s1 = exp2i(-e), s16 = exp2i(-e - 4);
  auto convert = [&](int i, const float4 (&v)[2]) {   // whole warps; the 8 lanes of a group are adjacent
    const float f[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    float sum;
    uint4 low;
    const uint4 b = moe_fragment2(f, s1, s16, low, sum);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < nv64) {
      *reinterpret_cast<uint4*>(hf + moe_fragment_at(i)) = b;
      *reinterpret_cast<uint4*>(hf + 16 * nv64 + moe_fragment_at(i)) = low;   // (second terms behind the first)
      if ((i & 7) == 0) {   // (both terms' zero points with the first)
        zs[i >> 3] = kZeroTerm * sum;
        zs[moe_zs_pitch(F) + (i >> 3)] = 0.f;
      }
    }
  };
#pragma unroll
  for (int u = 0; u < kRuns; ++u)
    if (u * kLanes < nv64) convert(lane + u * kLanes, keep[u]);
  for (int i0 = kRuns * kLanes; i0 < nv64; i0 += kRest * kLanes) {
    float4 v[kRest][2];
#pragma unroll
    for (int u = 0; u < kRest; ++u) load(i0 + u * kLanes + lane, v[u]);
#pragma unroll
    for (int u = 0; u < kRest; ++u)
      if (i0 + u * kLanes < nv64) convert(i0 + u * kLanes + lane, v[u]);
  }
  if (lane == 0) *ft = exp2i(e);
}

__device__ __forceinline__ void moe_prep_at(const RouterParams& p, int64_t t) {
  moe_prep_token(p.x + t * p.H, p.H, p.xf + (size_t)t * moe_groups(p.H) * 128, p.zs + t * moe_zs_pitch(p.H), p.ft + t);
}

// The operand pass alone (experts whose routing the caller has done): one CTA per token.
__global__ void __launch_bounds__(256) q4_moe_prep_kernel(const RouterParams p) {
  pdl_launch_dependents();
  pdl_wait_previous();
  moe_prep_at(p, blockIdx.x);
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                               uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The top_k of one token's logits (lg: `parts` sums of each expert, part after part), by one
// warp.  kV: values per lane.  Each lane keeps its values as order-preserving integers (0: never
// chosen -- -inf, NaN, what is already chosen) and its best one; a pick is a warp maximum of the
// keys and a minimum over the experts that have it.
template <int kV>
__device__ __forceinline__ void moe_pick(const RouterParams& p, const float* lg, int64_t t) {
  const int lane = threadIdx.x & 31;
  uint32_t key[kV];
  uint32_t best = 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0u;
    if (e < p.E) {
      float v = lg[e];
      for (int q = 1; q < p.parts; ++q) v += lg[q * p.E + e];
      const uint32_t b = __float_as_uint(v);
      if (v > -INFINITY) key[i] = (b & 0x80000000u) ? ~b : b | 0x80000000u;
      best = max(best, key[i]);
    }
  }
  auto value = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); };
  const uint32_t top = __reduce_max_sync(0xffffffffu, best);
  const float m = value(top);
  auto ex = [&](uint32_t k) { return k == top ? 1.f : expf(value(k) - m); };   // m may be +inf
  float z = 0.f;
  if (!p.renorm) {
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (key[i] != 0u) z += ex(key[i]);
    z = warp_sum(z);
  }
  uint32_t mine = 0u;   // lane j keeps pick j (k <= 32)
  int mine_id = -1;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t k = __reduce_max_sync(0xffffffffu, best);
    if (k == 0u) break;   // none left
    int at = p.E;
    if (best == k) {
#pragma unroll
      for (int i = kV - 1; i >= 0; --i)
        if (key[i] == k) at = lane + 32 * i;
    }
    const int id = __reduce_min_sync(0xffffffffu, at);
    if (lane == j) {
      mine = k;
      mine_id = id;
    }
    if (lane == (id & 31)) {
      best = 0u;
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if (lane + 32 * i == id) key[i] = 0u;
        best = max(best, key[i]);
      }
    }
  }
  const float pe = mine != 0u ? ex(mine) : 0.f;
  if (p.renorm) z = warp_sum(pe);
  if (lane < p.k) {
    p.ids[t * p.k + lane] = mine_id;
    p.weights[t * p.k + lane] = mine_id >= 0 ? pe / z : 0.f;
  }
}

// The 16-bit values [k0, k1) of a row to L2 (16-byte aligned at both ends).
__device__ __forceinline__ void prefetch_run(const uint16_t* row, int64_t k0, int64_t k1) {
  const int64_t bytes = 2 * (k1 - k0);
  if (bytes > 0) bulk_prefetch_l2(row + k0, (uint32_t)(bytes < 32768 ? bytes : 32768));
}

// One cluster per TT tokens: its 128 warps share the experts (with few experts several warps
// share the H of one), a warp's lanes share its H; the sums meet in the shared memory of the
// cluster's first CTA, whose first warps pick the top_k of one token each.
template <int TT>
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads, 2)
q4_moe_router_kernel(const RouterParams p) {
  __shared__ float logit[TT][kMaxExperts];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * TT;
  if ((int)blockIdx.x >= p.clusters * kRouteCluster) {   // whole clusters
    pdl_wait_previous();
    const int t = (int)blockIdx.x - p.clusters * kRouteCluster;
    if (t < p.prep_tokens) moe_prep_at(p, t);
    return;
  }
  constexpr int kWarps = kRouteThreads / 32;
  const int64_t nv = p.H / 8;
  constexpr int kAhead = TT == 1 ? 4 : 2;   // loads of this many steps in flight
  uint4 wv[kAhead];
  auto load_w = [&](const uint16_t* wr, int64_t i, int64_t i1) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) wv[q] = i + 32 * q < i1 ? ld_global_u4(wr + 8 * (i + 32 * q)) : make_uint4(0u, 0u, 0u, 0u);
  };
  const int w0 = warp * kRouteCluster + (int)rank;
  if (w0 < p.E * p.parts && lane == 0) {   // (to L2 only: a kernel before this one may still write them)
    const int e = w0 / p.parts, part = w0 - e * p.parts;
    prefetch_run(p.w + (int64_t)e * p.H, 8 * (nv * part / p.parts), 8 * (nv * (part + 1) / p.parts));
  }
  cluster_sync();   // every CTA of the cluster runs before its shared memory is written
  pdl_wait_previous();
  for (int w = w0; w < p.E * p.parts; w += kRouteCluster * kWarps) {
    const int e = w / p.parts, part = w - e * p.parts;
    const int64_t i0 = nv * part / p.parts, i1 = nv * (part + 1) / p.parts;
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    const uint16_t* wr = p.w + (int64_t)e * p.H;
    for (int64_t i = i0 + lane; i < i1; i += 32 * kAhead) {
      uint4 xv[kAhead][TT];
      load_w(wr, i, i1);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const bool in = i + 32 * q < i1;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const int64_t tt = t0 + t < p.T ? t0 + t : p.T - 1;
          xv[q][t] = in ? ld_global_u4(p.x + tt * p.H + 8 * (i + 32 * q)) : zero;
        }
      }
#pragma unroll
      for (int q = 0; q < kAhead; ++q) {
        const uint32_t ww[4] = {wv[q].x, wv[q].y, wv[q].z, wv[q].w};
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          const uint32_t xx[4] = {xv[q][t].x, xv[q][t].y, xv[q][t].z, xv[q][t].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[t] = fmaf(bf16lo(ww[k]), bf16lo(xx[k]), acc[t]);
            acc[t] = fmaf(bf16hi(ww[k]), bf16hi(xx[k]), acc[t]);
          }
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = warp_sum(acc[t]);
    if (lane == 0) {
      const float b = p.bias != nullptr && part == 0 ? __uint_as_float(ld_global_u32(p.bias + e)) : 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) {   // part after part: [parts][E]
        const uint32_t dst = mapa_shared(smem_u32(&logit[t][part * p.E + e]), 0);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(acc[t] + b) : "memory");
      }
    }
  }
  cluster_sync();
  if (rank != 0 || warp >= TT || t0 + warp >= p.T) return;
  // ---- one warp per token: softmax statistics, then top_k picks
  if (p.E <= 128) moe_pick<4>(p, logit[warp], t0 + warp);   // (four values per lane, in registers)
  else moe_pick<kMaxExperts / 32>(p, logit[warp], t0 + warp);
}

// The same for more tokens, eight to a cluster, on the tensor cores: mma.sync m16n8k16
// (bf16 x bf16 -> FP32) over tiles of 16 experts, the H of a tile shared by a CTA's 16 warps and,
// with few tiles, by several CTAs.  K order inside an MMA is free: thread (g, c) takes the eight
// values k = 8 c .. 8 c + 7 of every 32, of two experts' rows and of token g, one 16-byte load each
// for two MMAs.  The warps' sums meet in shared memory, then in the CTA of the token's rank,
// which picks.  Latency-bound: every load of a warp's share is in flight at once up to H = 2048.
// The router alone, against the form above (two tokens a
// cluster): 17.3 us for 48.8 (512 tokens, 128 experts, H = 2048), 6.5 for 6.7 (64), 5.1 for 4.7 (4).
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads, 2)
q4_moe_router_mma_kernel(const RouterParams p) {
  constexpr int kWarps = kRouteThreads / 32, kSteps = 4;
  __shared__ float logit[kMaxExperts];
  __shared__ __align__(16) float part_sum[kWarps][16][8];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  const int rank = (int)cluster_ctarank();
  const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * 8;
  if ((int)blockIdx.x >= p.clusters * kRouteCluster) {   // whole clusters
    pdl_wait_previous();
    const int t = (int)blockIdx.x - p.clusters * kRouteCluster;
    if (t < p.prep_tokens) moe_prep_at(p, t);
    return;
  }
  const int units = (p.E + 15) / 16 * p.parts;
  const int steps = (int)((p.H + 31) / 32), shares = p.parts * kWarps;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 w0[kSteps], w1[kSteps];
  auto load_w = [&](int unit, int st, int end) {
    const int e = unit / p.parts * 16 + g;   // (rows past E: the last one again, dropped below)
    const uint16_t* r0 = p.w + (int64_t)(e < p.E ? e : p.E - 1) * p.H;
    const uint16_t* r1 = p.w + (int64_t)(e + 8 < p.E ? e + 8 : p.E - 1) * p.H;
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int64_t k = 32 * (int64_t)(st + q) + 8 * c;
      const bool in = st + q < end && k < p.H;
      w0[q] = in ? ld_global_u4(r0 + k) : zero;
      w1[q] = in ? ld_global_u4(r1 + k) : zero;
    }
  };
  auto first_step = [&](int unit, int w) { return (int)((int64_t)steps * (unit % p.parts * kWarps + w) / shares); };
  // the first unit's weights to L2 (only that: a kernel before this one may still write them)
  if (rank < units && lane < 16) {
    const int e = rank / p.parts * 16 + lane;
    const int64_t k1 = 32 * (int64_t)first_step(rank, warp + 1);
    if (e < p.E) prefetch_run(p.w + (int64_t)e * p.H, 32 * (int64_t)first_step(rank, warp), k1 < p.H ? k1 : p.H);
  }
  cluster_sync();   // every CTA of the cluster runs before its shared memory is written
  pdl_wait_previous();
  const uint16_t* xr = p.x + (t0 + g < p.T ? t0 + g : p.T - 1) * p.H;
  for (int unit = rank; unit < units; unit += kRouteCluster) {
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    const int end = first_step(unit, warp + 1);
    for (int st = first_step(unit, warp); st < end; st += kSteps) {
      uint4 xv[kSteps];
      load_w(unit, st, end);
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        const int64_t k = 32 * (int64_t)(st + q) + 8 * c;
        xv[q] = st + q < end && k < p.H ? ld_global_u4(xr + k) : zero;
      }
#pragma unroll
      for (int q = 0; q < kSteps; ++q) {
        mma_bf16_16816(d, w0[q].x, w1[q].x, w0[q].y, w1[q].y, xv[q].x, xv[q].y);
        mma_bf16_16816(d, w0[q].z, w1[q].z, w0[q].w, w1[q].w, xv[q].z, xv[q].w);
      }
    }
    *reinterpret_cast<float2*>(&part_sum[warp][g][2 * c]) = make_float2(d[0], d[1]);
    *reinterpret_cast<float2*>(&part_sum[warp][g + 8][2 * c]) = make_float2(d[2], d[3]);
    __syncthreads();
    if (threadIdx.x < 128) {
      const int e = unit / p.parts * 16 + (int)(threadIdx.x >> 3), part = unit % p.parts, t = threadIdx.x & 7;
      float v = p.bias != nullptr && part == 0 && e < p.E ? __uint_as_float(ld_global_u32(p.bias + e)) : 0.f;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += part_sum[w][threadIdx.x >> 3][t];
      v += sum;
      if (e < p.E)
        asm volatile("st.shared::cluster.f32 [%0], %1;"
                     ::"r"(mapa_shared(smem_u32(&logit[part * p.E + e]), (uint32_t)t)), "f"(v)
                     : "memory");
    }
    __syncthreads();
  }
  cluster_sync();
  if (warp != 0 || t0 + rank >= p.T) return;
  if (p.E <= 128) moe_pick<4>(p, logit, t0 + rank);
  else moe_pick<kMaxExperts / 32>(p, logit, t0 + rank);
}

// ----------------------------------------------------------------- slots by expert
struct MoeParams {
  const uint8_t* xf;       // operand pass: fragments [T][groups][128], terms [T][pitch], powers [T]
  const float* zs;
  const float* ft;
  const int32_t* ids;      // [T, k]
  const float* weights;    // [T, k]
  const uint16_t* s_gu;    // [E, 2F, Hp/64]
  const uint16_t* s_dn;    // [E, H, Fp/64]
  float* h;                // [T k][F] (down: from the launch's first column on)
  float* part;             // [chunks][T k][H] sums of the down product, but in the latency form
  uint16_t* y;             // [T, H]
  int64_t H, F;
  int kn;                  // columns of the launch: H, or (down) a chunk of F
  int E, k, slots;         // slots = T k of this pass
  int chunks;              // launches of the down product
  int depth;               // ring slots per warp
  int per;                 // columns per tile, at most (8, fewer where a column is long)
  int gtiles;              // tiles whose columns lie in shared memory together
  uint32_t col_bytes;      // shared memory of a column
  uint32_t bar_off, cnt_off, wcnt_off, order_off, tiles_off, misc_off, pow_off, sum_off, col_off;   // shared memory
};

// Shared-memory lists of one CTA: the tiles (up to 8 slots of one expert) in
// expert order.
struct MoeLists {
  int* cnt;        // [E] first positions
  uint8_t* wcnt;   // [16][E] slots per warp and expert
  int* order;      // [slots] by expert: slot number | token << 16
  int2* tiles;     // [max tiles] (expert, first position | count << 16)
  int* ntiles;
};

__host__ __device__ inline int moe_max_tiles(int slots, int E, int per) {
  // every expert adds at most one partly filled tile
  return slots / per + (slots < E ? slots : E);
}

// Builds the lists from the pass's ids (all threads of the CTA; ends with a barrier).  Slots
// whose id is outside [0, E) are left out.  Inside an expert the slots keep their order: the
// units of a tile are spread over CTAs, which must all put the same slots into it.
__device__ __forceinline__ void moe_build_lists(const MoeParams& p, const MoeLists& L, int per) {
  const int tid = threadIdx.x, nth = blockDim.x;
  if (p.slots <= 32) {   // one warp, one load: experts in the order of their first slots
    if (tid < 32) {
      int e = tid < p.slots ? (int)ld_global_u32(p.ids + tid) : -1;
      if (e >= p.E) e = -1;
      const bool on = e >= 0;
      const unsigned same = __match_any_sync(0xffffffffu, on ? e : -1);
      const int n = __popc(same), rank = __popc(same & ((1u << tid) - 1u));
      const bool lead = on && rank == 0;
      int a = lead ? n : 0, b = lead ? (n + per - 1) / per : 0;
      const int slots_here = a, tiles_here = b;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a2 = __shfl_up_sync(0xffffffffu, a, o), b2 = __shfl_up_sync(0xffffffffu, b, o);
        if (tid >= o) {
          a += a2;
          b += b2;
        }
      }
      const int pos = a - slots_here;
      const int base = __shfl_sync(0xffffffffu, pos, __ffs(same) - 1);
      if (on) L.order[base + rank] = tid | (tid / p.k) << 16;
      for (int i = 0; i < tiles_here; ++i) {
        const int left = n - i * per;
        L.tiles[b - tiles_here + i] = make_int2(e, (pos + i * per) | ((left < per ? left : per) << 16));
      }
      if (tid == 31) *L.ntiles = b;
    }
    __syncthreads();
    return;
  }
  // One slot per thread (S <= kMaxSlots = the threads of the throughput form): ranks inside a
  // warp by matching, counts per (warp, expert), then sums over the warps and the experts.
  const int warp = tid >> 5, lane = tid & 31, warps = nth / 32;
  uint32_t* z = reinterpret_cast<uint32_t*>(L.wcnt);
  for (int i = tid; i < (warps * p.E + 3) / 4; i += nth) z[i] = 0u;
  int e = tid < p.slots ? (int)ld_global_u32(p.ids + tid) : -1;
  if (e < 0 || e >= p.E) e = -1;
  __syncthreads();
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && rank == 0) L.wcnt[warp * p.E + e] = (uint8_t)__popc(same);
  __syncthreads();
  if (warp == 0) {  // exclusive sums over the experts, 32 at a time
    int base = 0, tbase = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int x = e0 + lane;
      int n = 0;
      if (x < p.E)
        for (int w = 0; w < warps; ++w) n += L.wcnt[w * p.E + x];
      const int nt = (n + per - 1) / per;
      int a = n, b = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a2 = __shfl_up_sync(0xffffffffu, a, o), b2 = __shfl_up_sync(0xffffffffu, b, o);
        if (lane >= o) {
          a += a2;
          b += b2;
        }
      }
      const int pos = base + a - n, tp = tbase + b - nt;
      for (int i = 0; i < nt; ++i) {
        const int left = n - i * per;
        L.tiles[tp + i] = make_int2(x, (pos + i * per) | ((left < per ? left : per) << 16));
      }
      if (x < p.E) L.cnt[x] = pos;
      base += __shfl_sync(0xffffffffu, a, 31);
      tbase += __shfl_sync(0xffffffffu, b, 31);
    }
    if (lane == 0) *L.ntiles = tbase;
  }
  __syncthreads();
  if (e >= 0) {
    int at = L.cnt[e] + rank;
    for (int w = 0; w < warp; ++w) at += L.wcnt[w * p.E + e];
    L.order[at] = tid | (tid / p.k) << 16;
  }
  __syncthreads();
}

// ----------------------------------------------------------------- the product of a unit
// D = A . B + C
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The 16 weights of two code words as eight A registers, pairs (k, k + 4), (k + 1, k + 5),
// (k + 2, k + 6), (k + 3, k + 7) and the same of k + 8: fp16 patterns q 2^-24 (even registers)
// and 16 q 2^-24 (odd ones).
__device__ __forceinline__ void decode_pairs(uint2 w, uint32_t (&a)[8]) {
  const uint32_t v0 = w.x >> 8, v1 = w.y >> 8;
  a[0] = w.x & 0x000F000Fu;
  a[1] = w.x & 0x00F000F0u;
  a[2] = v0 & 0x000F000Fu;
  a[3] = v0 & 0x00F000F0u;
  a[4] = w.y & 0x000F000Fu;
  a[5] = w.y & 0x00F000F0u;
  a[6] = v1 & 0x000F000Fu;
  a[7] = v1 & 0x00F000F0u;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// What a warp holds of one unit while it runs through the unit's K range: where its rows'
// scales (global memory) and its B columns (shared memory) start.  Plain loads (not the
// volatile ones) in the loops, so that the compiler can overlap the groups of a sub-box; the
// waits before them are compiler barriers.
template <int MT>
struct MoeUnit {
  const uint16_t* s0[MT];    // scales of MMA rows g and g + 8
  const uint16_t* s1[MT];
  const uint8_t* b;          // fragments of thread column g
  const float* z[2];         // zero-point terms of token columns 2c, 2c + 1
};

// acc[m] += the products of the sub-box with the groups G0 .. G0 + 3 (kFull: all of them
// exist; kTwo: and those of the second terms, groups * 128 bytes behind the first).
template <int MT, bool kFull, bool kTwo>
__device__ __forceinline__ void moe_sub_box(const uint8_t* slot, const uint32_t (&off)[4], int G0, int groups,
                                            const MoeUnit<MT>& un, float (&acc)[MT][4]) {
  __half2 s0[MT][2], s1[MT][2];   // (the plane rows hold an even number of scales)
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (kFull || G0 + 2 * i < groups) {
        s0[m][i] = *reinterpret_cast<const __half2*>(un.s0[m] + G0 + 2 * i);
        s1[m][i] = *reinterpret_cast<const __half2*>(un.s1[m] + G0 + 2 * i);
      }
    }
  float4 z[2];   // the four groups' terms (the rows are padded to a multiple of four)
#pragma unroll
  for (int j = 0; j < 2; ++j) z[j] = *reinterpret_cast<const float4*>(un.z[j] + G0);
#pragma unroll
  for (int gl = 0; gl < 4; ++gl) {
    const int G = G0 + gl;
    if (!kFull && G >= groups) break;
    uint32_t a0[MT][8], a1[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      decode_pairs(*reinterpret_cast<const uint2*>(slot + off[gl] + 1024 * m), a0[m]);
      decode_pairs(*reinterpret_cast<const uint2*>(slot + off[gl] + 1024 * (MT + m)), a1[m]);
    }
    const uint8_t* at = un.b + (size_t)G * 128;
    const uint4 b0 = *reinterpret_cast<const uint4*>(at), b1 = *reinterpret_cast<const uint4*>(at + 64);
    uint4 c0, c1;
    if constexpr (kTwo) {
      c0 = *reinterpret_cast<const uint4*>(at + (size_t)groups * 128);
      c1 = *reinterpret_cast<const uint4*>(at + (size_t)groups * 128 + 64);
    }
    const float za = gl == 0 ? z[0].x : gl == 1 ? z[0].y : gl == 2 ? z[0].z : z[0].w;
    const float zb = gl == 0 ? z[1].x : gl == 1 ? z[1].y : gl == 2 ? z[1].z : z[1].w;
    const float zz[4] = {za, zb, za, zb};
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      float d[4];
      mma_f16_16816(d, a0[m][0], a1[m][0], a0[m][1], a1[m][1], b0.x, b0.y, zz);
      mma_f16_16816(d, a0[m][2], a1[m][2], a0[m][3], a1[m][3], b0.z, b0.w, d);
      mma_f16_16816(d, a0[m][4], a1[m][4], a0[m][5], a1[m][5], b1.x, b1.y, d);
      mma_f16_16816(d, a0[m][6], a1[m][6], a0[m][7], a1[m][7], b1.z, b1.w, d);
      if constexpr (kTwo) {
        mma_f16_16816(d, a0[m][0], a1[m][0], a0[m][1], a1[m][1], c0.x, c0.y, d);
        mma_f16_16816(d, a0[m][2], a1[m][2], a0[m][3], a1[m][3], c0.z, c0.w, d);
        mma_f16_16816(d, a0[m][4], a1[m][4], a0[m][5], a1[m][5], c1.x, c1.y, d);
        mma_f16_16816(d, a0[m][6], a1[m][6], a0[m][7], a1[m][7], c1.z, c1.w, d);
      }
      const float sa = (gl & 1) ? __high2float(s0[m][gl >> 1]) : __low2float(s0[m][gl >> 1]);
      const float sb = (gl & 1) ? __high2float(s1[m][gl >> 1]) : __low2float(s1[m][gl >> 1]);
      acc[m][0] = fmaf(sa, d[0], acc[m][0]);
      acc[m][1] = fmaf(sa, d[1], acc[m][1]);
      acc[m][2] = fmaf(sb, d[2], acc[m][2]);
      acc[m][3] = fmaf(sb, d[3], acc[m][3]);
    }
  }
}

// A column in shared memory (down: a slot's two): the fragments, then the zero-point terms, an odd
// number of 64-byte units in all, so that the 64-byte reads of neighbouring columns meet different
// banks.
__host__ __device__ inline uint32_t moe_column_bytes(int64_t K, int terms) {
  return (uint32_t)((terms * (moe_groups(K) * 128 + moe_zs_pitch(K) * 4) + 127) / 128 * 128 + 64);
}

// Shared-memory layout: rings (1024-byte aligned) and their barriers, lists, the columns'
// powers of two, the latency form's exchange buffer -- gate/up, the accumulators of the K parts (one
// 16-byte word per thread, two rounds); down, the slots' sums of every K part, their powers of
// two, weights and whether they count -- and the columns: gtiles tiles of them (latency form,
// down: every slot's).
// Warps that share the K range of an item, where a CTA's `items` are dealt to its warps in rounds:
// as few as pass all items in the shortest time (rounds / parts).
__host__ __device__ inline int moe_parts(int items, int nsb) {
  int best = 1, cost = kMaxParts * ((items + kMoeWarps - 1) / kMoeWarps);
  for (int kp = 2; kp <= kMaxParts && kp <= nsb; kp *= 2) {
    const int c = kMaxParts / kp * ((items * kp + kMoeWarps - 1) / kMoeWarps);
    if (c < cost) {
      best = kp;
      cost = c;
    }
  }
  return best;
}

__host__ inline uint32_t moe_layout(MoeParams& p, int mt, bool down, int form) {
  p.bar_off = (uint32_t)(kMoeWarps * p.depth * slot_bytes(mt));
  p.cnt_off = p.bar_off + (uint32_t)(kMoeWarps * p.depth * 8 + 8);
  p.wcnt_off = p.cnt_off + (p.slots <= 32 ? 0u : (uint32_t)p.E * 4);
  p.tiles_off = (p.wcnt_off + (p.slots <= 32 ? 0u : (uint32_t)(kMoeWarps * p.E + 4)) + 7) / 8 * 8;
  p.order_off = p.tiles_off + (uint32_t)moe_max_tiles(p.slots, p.E, p.per) * 8;
  p.misc_off = p.order_off + (uint32_t)p.slots * 4;
  p.pow_off = p.misc_off + 16;
  p.sum_off = (p.pow_off + (uint32_t)(p.gtiles * p.per) * 4 + 15) / 16 * 16;
  uint32_t at = p.sum_off;
  const bool own = down && form == kLatency;
  if (form != kThroughput) at += own ? (uint32_t)(p.slots * (kMaxParts * 64 + 12)) : (uint32_t)(2 * 32 * kMoeWarps * 16);
  p.col_off = (at + 127) / 128 * 128;
  return p.col_off + (uint32_t)(own ? p.slots : p.gtiles * p.per) * p.col_bytes;
}

// kDown false: gate/up units, h written; true: down units, y (latency) or part written.
// kPairs (down, tiles of up to four slots): the second terms in columns of their own.
template <int MT, bool kDown, int kForm, bool kPairs>
__global__ void __launch_bounds__(32 * kMoeWarps, 1)
q4_moe_kernel(const __grid_constant__ CUtensorMap tm, const MoeParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  static_assert(!kPairs || kDown, "pairs of columns: the down product");
  constexpr bool kTwo = kDown && !kPairs;   // the second terms' products follow the first
  constexpr int kRows = 8 * MT, kWarps = kMoeWarps, kThreads = 32 * kWarps;
  const int kPer = p.per;
  const uint32_t col_bar = sbase + p.bar_off + 8u * (uint32_t)(kWarps * p.depth);
  constexpr uint32_t kSlot = slot_bytes(MT);
  MoeLists L;
  L.cnt = reinterpret_cast<int*>(smem + p.cnt_off);
  L.wcnt = smem + p.wcnt_off;
  L.order = reinterpret_cast<int*>(smem + p.order_off);
  L.tiles = reinterpret_cast<int2*>(smem + p.tiles_off);
  L.ntiles = reinterpret_cast<int*>(smem + p.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + p.misc_off + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  if (lane == 0) {   // a warp's barriers are its own
    for (int i = 0; i < p.depth; ++i) mbar_init(sbase + p.bar_off + 8u * (uint32_t)(warp * p.depth + i), 1);
    if (warp == 0) {   // (the columns' barrier: every warp's, behind the lists' CTA barriers)
      mbar_init(col_bar, 1);
      *abort_flag = 0;
      prefetch_tmap(&tm);
    }
    fence_mbar_init();
  }
  __syncwarp();
  // Order of the chain: the gate/up kernel waits for everything before it, then lets the
  // down kernel launch.  So when the down kernel starts, ids, weights and planes are final
  // and only h is still being written: it sorts the slots and fills its rings before its
  // own wait.
  if constexpr (!kDown) {
    pdl_wait_previous();
    pdl_launch_dependents();
  } else {
    pdl_launch_dependents();
  }
  moe_build_lists(p, L, kPer);
  const int ntiles = *L.ntiles;

  const int K = p.kn;
  const int nsb = (K + 255) / 256;
  const int groups = (K + 63) / 64, gpad = (K + 127) / 128 * 2;
  const int grow = (int)(((kDown ? p.F : p.H) + 127) / 128 * 2);      // scales per weight row
  const int64_t rows_e = kDown ? p.H : 2 * p.F;                        // weight rows per expert
  const int64_t last_row = (int64_t)p.E * rows_e - 1;
  const int nu = (int)(kDown ? (p.H + 2 * kRows - 1) / (2 * kRows) : (p.F + kRows - 1) / kRows);   // units per expert
  const uint16_t* scales = kDown ? p.s_dn : p.s_gu;
  // Work.  Latency form, down: whole units [u0, u1), all tiles of each.  Otherwise a range
  // [u0, u1) of the numbers tile * nu + unit, so that a CTA's warps share an expert's tokens
  // (the host bounds nu * tiles below 2^31).  kp warps share the K range of an item.
  constexpr bool kOwn = kDown && kForm == kLatency, kJoin = kForm != kThroughput && !kOwn;
  const int all = kOwn ? nu : nu * ntiles, grid = (int)gridDim.x, bid = (int)blockIdx.x;
  const int share = all / grid, more = all - share * grid;   // the first `more` CTAs take one more
  const int u0 = bid * share + (bid < more ? bid : more), u1 = u0 + share + (bid < more ? 1 : 0);
  int kp = 1;
  if constexpr (kOwn) {   // the same for every unit
    while (kp < kMaxParts && 2 * kp * ntiles <= kWarps && 2 * kp <= nsb) kp *= 2;
  }
  if constexpr (kJoin) kp = moe_parts(share + (more > 0 ? 1 : 0), nsb);   // the same for every CTA
  const int kps = 31 - __clz(kp);                  // kp is a power of two
  const int wpr = kWarps >> kps;                   // items per round of the warps
  const int wnum = warp >> kps, kpart = warp & (kp - 1);
  const int sb0 = (nsb * kpart) >> kps, sb1 = (nsb * (kpart + 1)) >> kps;
  // The numbers are worked off in groups of gtiles tiles, whose columns lie in shared memory
  // together: group by group, numbers group start + wnum, + wpr, ...
  const int tile_a = !kOwn && nu > 0 ? u0 / nu : 0;
  auto group_end = [&](int tile0) { return tile0 + p.gtiles < ntiles && (tile0 + p.gtiles) * nu < u1 ? (tile0 + p.gtiles) * nu : u1; };
  // The items of this warp, in order: a position that steps without divisions.
  struct Pos {
    int tile, unit, left;   // left: more than 0 while inside the range (kOwn: units to its end)
    int tile0, gend;        // the group's first tile and end
  };
  // moves q from number u of its group on to the first one that is this warp's
  auto settle = [&](Pos& q, int u) {
    while (u >= q.gend && q.gend < u1) {
      q.tile0 += p.gtiles;
      u = q.gend + wnum;
      q.gend = group_end(q.tile0);
      q.tile = q.tile0;
      q.unit = u - q.tile * nu;
    }
    q.left = wnum < wpr ? (u < u1 ? u1 - u : 0) : 0;
    if (q.left > 0)
      while (q.unit >= nu) {
        q.unit -= nu;
        ++q.tile;
      }
  };
  auto start = [&]() -> Pos {
    if constexpr (kOwn) return {wnum, u0, wnum < ntiles && wnum < wpr ? u1 - u0 : 0, 0, 0};
    Pos q{tile_a, u0 + wnum - tile_a * nu, 0, tile_a, group_end(tile_a)};
    if (u0 < u1) settle(q, u0 + wnum);
    return q;
  };
  auto step = [&](Pos& q) {
    if constexpr (kOwn) {
      q.tile += wpr;
      if (q.tile >= ntiles) {
        q.tile = wnum;
        ++q.unit;
        --q.left;
      }
    } else {
      q.unit += wpr;
      settle(q, u1 - q.left + wpr);
    }
  };
  uint8_t* ring = smem + (size_t)(warp * p.depth) * kSlot;
  const uint32_t bars = sbase + p.bar_off + (uint32_t)(warp * p.depth * 8);
  // ---- issue side (lane 0): the warp's items once more, sub-box by sub-box, `depth` ahead
  Pos is = start();
  int is_sb = sb0, is_slot = 0, is_row = 0, is_exp = 0;
  int issued = 0;
  auto issue = [&]() {
    if (is_sb == sb0) {
      is_exp = L.tiles[is.tile].x;
      is_row = (kDown ? 2 * kRows : kRows) * is.unit;
    }
    const uint32_t bar = bars + 8u * (uint32_t)is_slot;
    mbar_expect_tx(bar, kSlot);
    tma_load_4d(smem_u32(ring) + (uint32_t)is_slot * kSlot, &tm, bar, is_sb * 128, is_row, 0, is_exp);   // rows past the expert's: zeros
    ++issued;
    if (++is_slot == p.depth) is_slot = 0;
    if (++is_sb == sb1) {
      is_sb = sb0;
      step(is);
    }
  };
  if (lane == 0)
    for (int d = 0; d < p.depth && is.left > 0; ++d) issue();
  // scale lines of a unit's rows: one row per lane
  const int nl = (sb1 - sb0) * 8 / 128 + 1;   // 128-byte lines past the first, at most
  auto scale_row = [&](const Pos& q) -> const uint8_t* {
    const int64_t base = (int64_t)L.tiles[q.tile].x * rows_e + (int64_t)q.unit * (kDown ? 2 * kRows : kRows);
    int64_t row = base + (kDown || lane < kRows ? lane : p.F + lane - kRows);
    row = row < last_row ? row : last_row;
    return reinterpret_cast<const uint8_t*>(scales + row * grow + 4 * sb0);
  };
  auto for_scale_lines = [&](const Pos& q, auto&& f) {
    if (lane < 2 * kRows) {
      const uint8_t* a = scale_row(q);
      const int most = (gpad - 4 * sb0) * 2 - 4;
      for (int i = 0; i <= nl; ++i) f(a + (128 * i < most ? 128 * i : most));
    }
  };
  float* wsm = nullptr;   // kOwn: the slots' weights, and which of them count
  int* von = nullptr;
  if constexpr (kOwn) {
    wsm = reinterpret_cast<float*>(smem + p.sum_off) + p.slots * (kMaxParts * 16 + 1);
    von = reinterpret_cast<int*>(wsm + p.slots);
    if ((int)threadIdx.x < p.slots) {
      const int id = p.ids[threadIdx.x];
      wsm[threadIdx.x] = p.weights[threadIdx.x];
      von[threadIdx.x] = id >= 0 && id < p.E;
    }
  }
  const Pos first_item = start();
  if (first_item.left > 0) for_scale_lines(first_item, [&](const uint8_t* a) { prefetch_l2(a); });
  // The B columns: x of a token (gate/up) or h of a slot (down): fragments, terms and powers.
  const float* power = p.ft;   // (down: set below)
  const uint32_t fbytes = (uint32_t)groups * (kDown ? 256u : 128u), zbytes = (uint32_t)moe_zs_pitch(K) * 4u;
  uint8_t* cols = smem + p.col_off;
  if constexpr (kDown) pdl_wait_previous();
  if constexpr (kOwn) {   // a warp per slot converts h
    float* fsm = reinterpret_cast<float*>(smem + p.sum_off) + p.slots * kMaxParts * 16;
    for (int s = warp; s < p.slots; s += kWarps) {
      uint8_t* at = cols + s * p.col_bytes;
      moe_prep_slot<3, MT == 1 ? 3 : 1>(p.h + s * p.F, K, at, reinterpret_cast<float*>(at + fbytes), fsm + s);
    }
    power = fsm;
    __syncthreads();
  }
  // The columns of the tiles from tile0 to the one of number gend - 1, tile after tile.  Gate/up:
  // bulk copies by warp 0 of what the operand pass has converted.  Down: a warp per column
  // converts h, in every CTA that needs the slot.
  float* cpow = reinterpret_cast<float*>(smem + p.pow_off);   // down: the columns' powers
  auto stage_columns = [&](int tile0, int gend) {
    const int last = (gend - 1) / nu;
    if constexpr (kDown) {
      int before = 0;
      for (int t = tile0; t <= last; ++t) {
        const int2 tl = L.tiles[t];
        const int count = tl.y >> 16;
        for (int i = (warp - before) & (kWarps - 1); i < count; i += kWarps) {
          const int at = (t - tile0) * kPer + i;
          uint8_t* dst = cols + at * p.col_bytes;
          moe_prep_slot<3, MT == 1 ? 3 : 1>(p.h + (L.order[(tl.y & 0xFFFF) + i] & 0xFFFF) * p.F, K, dst, reinterpret_cast<float*>(dst + fbytes),
                           cpow + at);
        }
        before += count;
      }
    } else {
      int n = 0;
      for (int t = tile0; t <= last; ++t) n += L.tiles[t].y >> 16;
      if (lane == 0) mbar_expect_tx(col_bar, (uint32_t)n * (fbytes + zbytes));
      __syncwarp();
      for (int t = tile0; t <= last; ++t) {
        const int2 tl = L.tiles[t];
        if (lane < (tl.y >> 16)) {
          const int64_t src = L.order[(tl.y & 0xFFFF) + lane] >> 16;
          const uint32_t dst = smem_u32(cols) + (uint32_t)((t - tile0) * kPer + lane) * p.col_bytes;
          bulk_g2s(dst, p.xf + src * fbytes, fbytes, col_bar);
          bulk_g2s(dst + fbytes, reinterpret_cast<const uint8_t*>(p.zs) + src * zbytes, zbytes, col_bar);
        }
      }
    }
  };

  bool ok = true;
  int slot = 0;
  uint32_t phase = 0;
  float* sums = reinterpret_cast<float*>(smem + p.sum_off);
  const int r = (2 * g & 7) + (g >> 2);
  uint32_t off[4];   // this thread's code bytes of the sub-box's four groups, in the swizzled box
#pragma unroll
  for (int gl = 0; gl < 4; ++gl)
    off[gl] = (uint32_t)r * 128u + (((((uint32_t)(2 * gl + (c >> 1))) ^ (uint32_t)r) << 4) | (uint32_t)((c & 1) << 3));
  // products of an item over this warp's K part; next: the item after it
  auto compute = [&](const Pos& q, const Pos& next, float (&acc)[MT][4], int& first, int& count) {
    const int2 tl = L.tiles[q.tile];
    first = tl.y & 0xFFFF;
    count = tl.y >> 16;
    MoeUnit<MT> un;
    const int64_t row0 = (int64_t)tl.x * rows_e + (int64_t)q.unit * (kDown ? 2 * kRows : kRows);
    const int64_t row1 = row0 + (kDown ? (int64_t)kRows : p.F);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      // rows past the plane (a last, partly filled unit): their results are dropped
      const int64_t q0 = row0 + 8 * m + r, q1 = row1 + 8 * m + r;
      un.s0[m] = scales + (q0 < last_row ? q0 : last_row) * grow;
      un.s1[m] = scales + (q1 < last_row ? q1 : last_row) * grow;
    }
    // empty columns take the tile's first one; their results are dropped
    const uint8_t* tcols = cols + (kOwn ? 0u : (uint32_t)((q.tile - q.tile0) * kPer) * p.col_bytes);
    auto column = [&](int i) -> const uint8_t* {
      const int k = i < count ? i : 0;
      return tcols + (uint32_t)(kOwn ? L.order[first + k] & 0xFFFF : k) * p.col_bytes;
    };
    // (kPairs: column i is the first term of slot i, column 4 + i its second)
    const uint32_t bterm = kPairs && g >= 4 ? fbytes / 2 : 0u, zterm = kPairs && c >= 2 ? zbytes : 0u;
    constexpr int width = kPairs ? 3 : 7;
    un.b = column(g & width) + bterm + 16 * c;
    un.z[0] = reinterpret_cast<const float*>(column(2 * c & width) + fbytes + zterm);
    un.z[1] = reinterpret_cast<const float*>(column((2 * c & width) + 1) + fbytes + zterm);
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
    if (next.left > 0) for_scale_lines(next, [&](const uint8_t* a) { prefetch_l2(a); });   // the next unit's scales
    for (int sb = sb0; sb < sb1; ++sb) {
      // every lane polls and the warp votes (a lane's answer is its own, and warp_wait wants the
      // whole warp): two instructions where the copy has landed
      if (ok && !__all_sync(0xffffffffu, mbar_try_wait(bars + 8u * (uint32_t)slot, phase)))
        ok = warp_wait(bars + 8u * (uint32_t)slot, phase, abort_flag, &g_moe_status);
      if (ok) {
        if (!kTwo && 4 * (sb + 1) <= groups)   // (with two terms the whole box's loads do not fit the registers)
          moe_sub_box<MT, true, kTwo>(ring + slot * kSlot, off, 4 * sb, groups, un, acc);
        else
          moe_sub_box<MT, false, kTwo>(ring + slot * kSlot, off, 4 * sb, groups, un, acc);
        __threadfence_block();   // every lane's reads of the slot lie before its refill
        __syncwarp();
        if (lane == 0 && is.left > 0) issue();   // refill the slot just read
        if (++slot == p.depth) {
          slot = 0;
          phase ^= 1;
        }
      }
    }
    if constexpr (kPairs) {   // the second terms' sums, of columns 4 .. 7, to the threads of the first terms' (c = 0, 1)
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] += __shfl_down_sync(0xffffffffu, acc[m][j], 2);
    }
  };

  // The columns of the group at hand (not kOwn): staged once all warps are past the one before.
  int group = 0;
  auto enter_group = [&](int tile0, int gend) {
    if (group > 0) __syncthreads();
    if constexpr (kDown) {
      stage_columns(tile0, gend);
      __syncthreads();
    } else {
      if (warp == 0) stage_columns(tile0, gend);
      if (ok) ok = warp_wait(col_bar, (uint32_t)(group & 1), abort_flag, &g_moe_status);
    }
    ++group;
  };
  Pos pos = start();
  auto activate = [&](const float (&acc)[MT][4], int first, int count, int unit) {
    // thread (g, c) holds gate and up of row f of token columns 2c, 2c + 1
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = 2 * c + j;
      if (col >= count) continue;
      const int o = L.order[first + col];
      const float F = power[o >> 16];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t f = kRows * (int64_t)unit + 8 * m;
        if (f >= p.F) continue;
        const float gt = F * acc[m][j], up = F * acc[m][2 + j];
        const float h = gt / (1.f + expf(-gt)) * up;
        p.h[(int64_t)(o & 0xFFFF) * p.F + f + r] = h;
      }
    }
  };
  // pcol: the tile's first staged column
  auto store = [&](const float (&acc)[MT][4], int first, int count, int unit, int pcol) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = 2 * c + j;
      if (col >= count) continue;
      const int s = L.order[first + col] & 0xFFFF;
      const float F = kOwn ? power[s] : cpow[pcol + col];
      if constexpr (kOwn) {
        sums[(kpart * p.slots + s) * 16 + r] = F * (kCodePower * acc[0][j]);
        sums[(kpart * p.slots + s) * 16 + 8 + r] = F * (kCodePower * acc[0][2 + j]);
      } else {
        const int64_t n0 = 2 * kRows * (int64_t)unit;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int64_t ra = n0 + 8 * m + r, rb = ra + kRows;
          if (ra < p.H) p.part[(int64_t)s * p.H + ra] = F * (kCodePower * acc[m][j]);
          if (rb < p.H) p.part[(int64_t)s * p.H + rb] = F * (kCodePower * acc[m][2 + j]);
        }
      }
    }
  };
  if constexpr (!kOwn) {
    int parity = 0;
    int tile0 = tile_a, gstart = u0;
    while (gstart < u1) {
      const int gend = group_end(tile0);
      enter_group(tile0, gend);
      // with K parts, all warps pass the same rounds (they meet to join their sums)
      for (int base = gstart; base < gend; base += wpr) {
        const bool have = pos.left > 0 && pos.tile0 == tile0;
        if (kp == 1 && !have) break;
        const Pos q = pos;
        if (have) step(pos);
        float acc[MT][4];
        int first = 0, count = 0;
        if (have) compute(q, pos, acc, first, count);
        if constexpr (kJoin) {
          if (kp > 1) {   // part 0 adds the others' accumulators, in order
            float4* ex = reinterpret_cast<float4*>(sums) + parity * kThreads;
            parity ^= 1;
            if (have && kpart > 0) ex[threadIdx.x] = make_float4(acc[0][0], acc[0][1], acc[0][2], acc[0][3]);
            __syncthreads();
            if (!have || kpart > 0) continue;
            for (int i = 1; i < kp; ++i) {
              const float4 v = ex[threadIdx.x + 32 * i];
              acc[0][0] += v.x;
              acc[0][1] += v.y;
              acc[0][2] += v.z;
              acc[0][3] += v.w;
            }
          }
        }
        if (!ok || !have) continue;
        if constexpr (kDown) store(acc, first, count, q.unit, (q.tile - q.tile0) * kPer);
        else activate(acc, first, count, q.unit);
      }
      gstart = gend;
      tile0 += p.gtiles;
    }
  } else {
    const int tokens = p.slots / p.k;
    for (int unit = u0; unit < u1; ++unit) {   // (without any tile: y = +0)
      while (pos.left > 0 && pos.unit == unit) {
        const Pos q = pos;
        step(pos);
        float acc[MT][4];
        int first, count;
        compute(q, pos, acc, first, count);
        if (ok) store(acc, first, count, unit, 0);
      }
      __syncthreads();
      if (!*abort_flag) {   // y of the unit's rows: the slots' sums in the order of the choices
        const int64_t n0 = 16 * (int64_t)unit;
        // lane 16 h + row: token 2 i + h
        for (int t = 2 * warp + (lane >> 4); t < tokens; t += 2 * kWarps) {
          const int rr = lane & 15;
          float v = 0.f;
#pragma unroll 4
          for (int j = 0; j < p.k; ++j) {
            const int s = t * p.k + j;
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i)
              if (i < kp) part += sums[(i * p.slots + s) * 16 + rr];
            v = von[s] ? fmaf(wsm[s], part, v) : v;
          }
          if (n0 + rr < p.H) p.y[(int64_t)t * p.H + n0 + rr] = float_to_bf16_bits(v);
        }
      }
      __syncthreads();   // the sums are free again
    }
  }
  if constexpr (!kDown) {
    if (!ok && threadIdx.x == 0 && group > 0) mbar_drain(col_bar, (uint32_t)((group - 1) & 1));
  }
  if (!ok && lane == 0)   // aborted: let the copies already issued land before the CTA exits
    for (int d = issued > p.depth ? issued - p.depth : 0; d < issued; ++d)
      mbar_drain(bars + 8u * (uint32_t)(d % p.depth), (uint32_t)((d / p.depth) & 1));
}

// Throughput form, after the down product: y[t, n] = sum_j p[t, j] part[t k + j, n] in the order
// of the choices; four columns per thread (H is a multiple of 8).  The choices (final since the
// gate/up kernel) are read before the wait, and eight parts are in flight at once: one after the
// other, each behind its choice, they cost about 1.5 us more at 64 tokens x 8.
constexpr int kReduceThreads = 128;

// kMany: the down product ran in chunks of F (with their loop in it, the kernel takes 106 registers
// for 38, and 64 tokens x 8 of 128 took 92 us for 87).
template <bool kMany>
__global__ void __launch_bounds__(kReduceThreads) q4_moe_reduce_kernel(const MoeParams p) {
  pdl_launch_dependents();
  constexpr int kAtOnce = 8;
  const int q = (int)(p.H / 4);
  const int64_t i = (int64_t)blockIdx.x * kReduceThreads + threadIdx.x;
  const int64_t t = i / q;
  const bool mine = t < p.slots / p.k;
  const int64_t n = 4 * (i - t * q);
  float w[kAtOnce];
  bool on[kAtOnce];   // (the part of a choice outside [0, E) was not written)
  auto choices = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool in = mine && j0 + j < p.k;
      const int id = in ? (int)ld_global_u32(p.ids + t * p.k + j0 + j) : -1;
      w[j] = in ? __uint_as_float(ld_global_u32(p.weights + t * p.k + j0 + j)) : 0.f;
      on[j] = id >= 0 && id < p.E;
    }
  };
  choices(0);
  pdl_wait_previous();
  if (!mine) return;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < p.k; j0 += kAtOnce) {
    if (j0 > 0) choices(j0);
    float4 f[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) f[j] = on[j] ? ld_global_f4(p.part + (t * p.k + j0 + j) * p.H + n) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 1; kMany && c < p.chunks; ++c) {   // the sums of the further chunks of columns, in order
      float4 m[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        m[j] = on[j] ? ld_global_f4(p.part + ((int64_t)c * p.slots + t * p.k + j0 + j) * p.H + n) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) f[j] = make_float4(f[j].x + m[j].x, f[j].y + m[j].y, f[j].z + m[j].z, f[j].w + m[j].w);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (!on[j]) continue;
      v[0] = fmaf(w[j], f[j].x, v[0]);
      v[1] = fmaf(w[j], f[j].y, v[1]);
      v[2] = fmaf(w[j], f[j].z, v[2]);
      v[3] = fmaf(w[j], f[j].w, v[3]);
    }
  }
  uint2 o;
  o.x = (uint32_t)float_to_bf16_bits(v[0]) | ((uint32_t)float_to_bf16_bits(v[1]) << 16);
  o.y = (uint32_t)float_to_bf16_bits(v[2]) | ((uint32_t)float_to_bf16_bits(v[3]) << 16);
  *reinterpret_cast<uint2*>(p.y + t * p.H + n) = o;
}

int moe_sm_count() {
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && cached[dev]) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < 64) cached[dev] = n;
  return n;
}

// Dynamic shared memory at most; what is left of the SM's 256 KB is the L1 of the scales.
constexpr uint32_t kMoeSmem = 208 * 1024;

// Shared-memory plan of a launch (the tile width per, the ring's depth, the tiles held together):
// columns of one or two tiles beside rings of two slots per warp; then as many slots (up to four)
// as there is room for, and more tiles together, where they are short.  Long columns: fewer per
// tile.  0: a column of this length does not fit at all.
uint32_t moe_fit(MoeParams& p, bool down, int form) {
  const int mt = form == kThroughput ? 2 : 1;
  const bool own = down && form == kLatency;
  const int tokens = p.slots / p.k;   // (an expert gets a token once, as a rule)
  p.col_bytes = moe_column_bytes(p.kn, down ? 2 : 1);
  p.per = tokens < 8 ? tokens : 8;
  p.depth = 2;
  p.gtiles = own ? 1 : 2;
  uint32_t bytes = moe_layout(p, mt, down, form);
  if (bytes > kMoeSmem && p.gtiles > 1) {
    p.gtiles = 1;
    bytes = moe_layout(p, mt, down, form);
  }
  while (bytes > kMoeSmem && p.per > 1) {
    --p.per;
    bytes = moe_layout(p, mt, down, form);
  }
  if (bytes > kMoeSmem) return 0;
  while (p.depth < 4) {
    MoeParams q = p;
    ++q.depth;
    const uint32_t more = moe_layout(q, mt, down, form);
    if (more > kMoeSmem) break;
    p = q;
    bytes = more;
  }
  while (!own && p.gtiles < 8) {
    MoeParams q = p;
    ++q.gtiles;
    const uint32_t more = moe_layout(q, mt, down, form);
    if (more > kMoeSmem) break;
    p = q;
    bytes = more;
  }
  return bytes;
}

template <int MT, bool kDown, int kForm, bool kPairs = false>
int moe_kernel_launch(const CUtensorMap& tm, const MoeParams& p, uint32_t bytes, int sms, cudaStream_t stream) {
  static bool attr[64] = {};
  int dev = 0;
  if (cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return Q4LIN_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cuda_check(cudaFuncSetAttribute(q4_moe_kernel<MT, kDown, kForm, kPairs>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)kMoeSmem),
                   "moe: cudaFuncSetAttribute"))
      return Q4LIN_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  if (bytes == 0) {   // (moe_plan leaves no such form: a kernel without its shared memory would write past it)
    set_error_detail("moe: this form does not fit shared memory");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  int grid = sms;
  if (kDown && kForm == kLatency) {   // whole units
    const int64_t nu = (p.H + 15) / 16;
    if (grid > nu) grid = (int)nu;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(32 * kMoeWarps, 1, 1);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_moe_kernel<MT, kDown, kForm, kPairs>, tm, p),
                    kDown ? "moe: down kernel launch" : "moe: gate/up kernel launch");
}

template <bool kDown>
int moe_kernel_form(int form, const CUtensorMap& tm, const MoeParams& p, uint32_t bytes, int sms, cudaStream_t stream) {
  if constexpr (kDown) {
    if (p.per <= 4) {
      if (form == kLatency) return moe_kernel_launch<1, true, kLatency, true>(tm, p, bytes, sms, stream);
      if (form == kJoined) return moe_kernel_launch<1, true, kJoined, true>(tm, p, bytes, sms, stream);
      return moe_kernel_launch<2, true, kThroughput, true>(tm, p, bytes, sms, stream);
    }
    if (form == kLatency) return moe_kernel_launch<1, true, kLatency>(tm, p, bytes, sms, stream);
  }
  // (the latency form's gate/up is the joined one)
  if (form != kThroughput) return moe_kernel_launch<1, kDown, kJoined>(tm, p, bytes, sms, stream);
  return moe_kernel_launch<2, kDown, kThroughput>(tm, p, bytes, sms, stream);
}

// Joined or throughput, by the likely number of a CTA's items (slots spread evenly over the
// experts).  With less than one long item per SM sub-partition the item's own latency is the
// time, and shorter items with shared K win: down product of 19 tokens x 6 of 9, 584 x 1944, 1.1
// items: the layer takes 37 us for 60; gate/up of 32 x 2 of 8, 2048 x 768, 2.5 items: 26.0 for
// 32.4; of 16 x 2 of 8, 4096 x 1024, 3.3 items: 34.5 for 44.4.  With more, the longer items'
// cheaper bytes do: 19 x 3 of 20, 1992 x 1016, 8 items: 35.4 for 32.6 in either product; 64 x 8 of
// 128, 2048 x 768, 40 items: 108.6 for 88.8 (gate/up), 97.3 for 88.8 (down); even at 4.3.
bool moe_joins(int slots, int64_t E, int64_t rows, int sms) {
  const double none = std::pow(1.0 - 1.0 / (double)E, (double)slots);
  return (double)E * (1.0 - none) * (double)((rows + 15) / 16) < 4.0 * sms;
}

MoeParams moe_params(int tokens, int64_t H, int64_t F, int64_t E, int k) {
  MoeParams p{};
  p.H = H;
  p.F = F;
  p.E = (int)E;
  p.k = k;
  p.slots = tokens * k;
  p.kn = (int)H;
  p.chunks = 1;
  return p;
}

// How a pass of `tokens` tokens runs (its sizes decide alone): the forms of its two products, and the
// chunks of F columns (a launch of the down product each) with their length.
struct MoePlan {
  int gu_form, dn_form, chunks, len;
};

// False: a column of H values does not fit shared memory beside the rings.
bool moe_plan(int tokens, int64_t H, int64_t F, int64_t E, int k, int sms, MoePlan* pl) {
  const MoeParams p = moe_params(tokens, H, F, E, k);
  auto fit = [&](bool down, int form, int64_t columns) {   // the tile width, 0: does not fit
    MoeParams q = p;
    q.kn = (int)columns;
    return moe_fit(q, down, form) != 0 ? q.per : 0;
  };
  pl->gu_form = moe_joins(p.slots, E, F, sms) || fit(false, kThroughput, H) == 0 ? kJoined : kThroughput;
  if (fit(false, pl->gu_form, H) == 0) return false;
  pl->chunks = 1;
  pl->len = (int)F;
  // (64 KB of columns and less: 20.4 us for 21.8, one token x 8 of 64, 2048 x 768; 134 KB: 30.6 for
  // 35.2, 16 tokens x 1 of 8, 2048 x 2048, and 40.5 for 39.1, 2 x 8 of 16)
  if (p.slots <= kLatSlots && fit(true, kLatency, F) > 0) {
    pl->gu_form = pl->dn_form = kLatency;
    return true;
  }
  // The throughput form only with whole tiles.  Narrower ones decode their rows again for every few
  // slots, and joined they are wider (its rings are half as large): 4 tokens x 2 of 8, 4096 x 14336,
  // one column for four: 259 us for 170.
  const int width = tokens < 8 ? tokens : 8;
  pl->dn_form = moe_joins(p.slots, E, H / 2, sms) || fit(true, kThroughput, F) < width ? kJoined : kThroughput;
  if (pl->dn_form == kThroughput) return true;
  // Chunks of F that keep tiles of four slots, of eight where an expert gets more than four on
  // average: 64 tokens x 2 of 8, 4096 x 14336: 716 us in one launch (two slots per tile), 592 with
  // four, 551 with eight; 16 tokens: 274, 215, 247; 8 tokens, 6144 x 32768: 727, 588, 662.
  const int even = p.slots > 4 * E ? 8 : 4, want = even < tokens ? even : tokens;
  const int nsb = (int)((F + 255) / 256);
  for (int c = 1; c <= nsb; ++c) {
    pl->len = (nsb + c - 1) / c * 256;
    pl->chunks = (nsb * 256 + pl->len - 1) / pl->len;
    if (fit(true, kJoined, pl->len < F ? pl->len : F) >= want) return true;
  }
  return false;
}

// Workspace parts of one pass, each 256-byte aligned.
struct MoeWs {
  size_t xf, zs, ft, h, part, total;
};

MoeWs moe_ws(int tokens, int64_t H, int64_t F, int k, const MoePlan& pl) {
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  const size_t S = (size_t)tokens * (size_t)k;
  MoeWs w;
  w.xf = 0;
  w.zs = w.xf + up((size_t)tokens * (size_t)moe_groups(H) * 128);
  w.ft = w.zs + up((size_t)tokens * (size_t)moe_zs_pitch(H) * 4);
  w.h = w.ft + up((size_t)tokens * 4);
  w.part = w.h + up(S * (size_t)F * 4);
  w.total = w.part + (pl.dn_form == kLatency ? 0 : up((size_t)pl.chunks * S * (size_t)H * 4));
  return w;
}

cudaLaunchConfig_t moe_config(unsigned blocks, unsigned threads, cudaStream_t stream, cudaLaunchAttribute* at) {
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cfg;
}

}  // namespace

int moe_pass_tokens(int64_t T, int k) {
  const int most = kMaxSlots / k;
  return (int)(T < most ? T : most);
}

namespace {

// The plans of a call's passes: the full one's and, where there is one, the last, shorter one's.
// f(plan, tokens); false: a pass has none.
template <typename Fn>
bool moe_plans(int64_t T, int64_t H, int64_t F, int64_t E, int k, Fn&& f) {
  const int tp = moe_pass_tokens(T, k), last = (int)(T % tp), sms = moe_sm_count();
  MoePlan pl;
  if (!moe_plan(tp, H, F, E, k, sms, &pl)) return false;
  f(pl, tp);
  if (last == 0) return true;
  if (!moe_plan(last, H, F, E, k, sms, &pl)) return false;
  f(pl, last);
  return true;
}

}  // namespace

bool moe_supported(int64_t T, int64_t H, int64_t F, int64_t E, int k) {
  return moe_plans(T, H, F, E, k, [](const MoePlan&, int) {});
}

size_t moe_workspace_bytes(int64_t T, int64_t H, int64_t F, int64_t E, int k) {
  size_t most = 0;
  const bool ok = moe_plans(T, H, F, E, k, [&](const MoePlan& pl, int tokens) {
    const size_t b = moe_ws(tokens, H, F, k, pl).total;
    most = b > most ? b : most;
  });
  return ok ? most : 0;
}

int moe_router_launch(const MoeArgs& a) {
  RouterParams p{};
  p.x = a.x;
  p.w = a.w_router;
  p.bias = a.bias;
  p.ids = a.ids_out;
  p.weights = a.weights_out;
  p.T = a.T;
  p.H = a.H;
  p.E = (int)a.E;
  p.k = a.k;
  p.renorm = a.renorm;
  const int tt = a.T < kRouteMma ? (a.T == 1 ? 1 : 2) : 8;   // tokens per cluster
  const int64_t clusters = (a.T + tt - 1) / tt;
  p.clusters = (int)clusters;
  const int tiles = (int)((a.E + 15) / 16);
  if (tt == 8) p.parts = tiles >= kRouteCluster ? 1 : kRouteCluster / tiles;
  else p.parts = a.E >= 128 ? 1 : (int)(128 / a.E);
  int64_t prep = 0;
  if (a.workspace != nullptr) {   // the whole layer: the experts' first operand pass beside the router
    const int tp = moe_pass_tokens(a.T, a.k);
    MoePlan pl;
    if (!moe_plan(tp, a.H, a.F, a.E, a.k, moe_sm_count(), &pl)) return Q4LIN_ERR_UNSUPPORTED_SHAPE;
    const MoeWs w = moe_ws(tp, a.H, a.F, a.k, pl);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.xf = ws + w.xf;
    p.zs = reinterpret_cast<float*>(ws + w.zs);
    p.ft = reinterpret_cast<float*>(ws + w.ft);
    p.prep_tokens = tp;
    prep = (tp + kRouteCluster - 1) / kRouteCluster;
  }
  cudaLaunchAttribute at[1];
  const cudaLaunchConfig_t cfg = moe_config((unsigned)((clusters + prep) * kRouteCluster), kRouteThreads, a.stream, at);
  cudaError_t e;
  switch (tt) {
    case 1: e = cudaLaunchKernelEx(&cfg, q4_moe_router_kernel<1>, p); break;
    case 2: e = cudaLaunchKernelEx(&cfg, q4_moe_router_kernel<2>, p); break;
    default: e = cudaLaunchKernelEx(&cfg, q4_moe_router_mma_kernel, p); break;
  }
  return cuda_check(e, "moe: router kernel launch");
}

int moe_experts_launch(const MoeArgs& a, bool prepared) {
  const int64_t Hp = k_pad(a.H), Fp = k_pad(a.F);
  const int sms = moe_sm_count();
  const int pass = moe_pass_tokens(a.T, a.k);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  for (int64_t t0 = 0; t0 < a.T; t0 += pass) {
    const int tp = (int)(a.T - t0 < pass ? a.T - t0 : pass);
    MoePlan pl;
    if (!moe_plan(tp, a.H, a.F, a.E, a.k, sms, &pl)) return Q4LIN_ERR_UNSUPPORTED_SHAPE;
    // (code bytes, rows, gate / up, expert): one copy brings the gate rows and the up rows of a
    // unit (down: one run of twice as many rows)
    const uint32_t gbox = pl.gu_form == kThroughput ? 16 : 8, dbox = pl.dn_form == kThroughput ? 16 : 8;
    CUtensorMap gu;
    const uint64_t gd[4] = {(uint64_t)(Hp / 2), (uint64_t)a.F, 2, (uint64_t)a.E};
    const uint64_t gs[3] = {(uint64_t)(Hp / 2), (uint64_t)(a.F * (Hp / 2)), (uint64_t)(2 * a.F * (Hp / 2))};
    const uint32_t gb[4] = {128, gbox, 2, 1};
    if (!encode_map_4d(&gu, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq_gu, gd, gs, gb, CU_TENSOR_MAP_SWIZZLE_128B)) {
      set_error_detail("moe: cuTensorMapEncodeTiled failed (or is unavailable)");
      return Q4LIN_ERR_CUDA;
    }
    const MoeWs w = moe_ws(tp, a.H, a.F, a.k, pl);
    if (!prepared || t0 > 0) {
      RouterParams r{};
      r.x = a.x + t0 * a.H;
      r.H = a.H;
      r.xf = ws + w.xf;
      r.zs = reinterpret_cast<float*>(ws + w.zs);
      r.ft = reinterpret_cast<float*>(ws + w.ft);
      cudaLaunchAttribute at[1];
      const cudaLaunchConfig_t cfg = moe_config((unsigned)tp, 256, a.stream, at);
      if (cuda_check(cudaLaunchKernelEx(&cfg, q4_moe_prep_kernel, r), "moe: operand pass launch")) return Q4LIN_ERR_CUDA;
    }
    MoeParams p = moe_params(tp, a.H, a.F, a.E, a.k);
    p.xf = ws + w.xf;
    p.zs = reinterpret_cast<const float*>(ws + w.zs);
    p.ft = reinterpret_cast<const float*>(ws + w.ft);
    p.ids = a.ids + t0 * a.k;
    p.weights = a.weights + t0 * a.k;
    p.s_gu = a.s_gu;
    p.s_dn = a.s_dn;
    p.h = reinterpret_cast<float*>(ws + w.h);
    p.part = reinterpret_cast<float*>(ws + w.part);
    p.y = a.y + t0 * a.H;
    p.chunks = pl.chunks;
    // a chunk of the down product: its columns, map and shared memory
    MoeParams d;
    CUtensorMap dn;
    uint32_t dbytes = 0;
    auto chunk = [&](int c) -> bool {
      const int64_t k0 = (int64_t)c * pl.len, left = a.F - k0;
      d = p;
      d.kn = (int)(left < pl.len ? left : pl.len);
      d.h = p.h + k0;
      d.s_dn = p.s_dn + k0 / 64;
      d.part = p.part + (int64_t)c * p.slots * a.H;
      dbytes = moe_fit(d, true, pl.dn_form);
      const uint64_t dd[4] = {(uint64_t)((Fp - k0) / 2), (uint64_t)a.H, 1, (uint64_t)a.E};
      const uint64_t ds[3] = {(uint64_t)(Fp / 2), (uint64_t)(a.H * (Fp / 2)), (uint64_t)(a.H * (Fp / 2))};
      const uint32_t db[4] = {128, 2 * dbox, 1, 1};
      return encode_map_4d(&dn, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq_dn + k0 / 2, dd, ds, db, CU_TENSOR_MAP_SWIZZLE_128B);
    };
    MoeParams g = p;
    const uint32_t gbytes = moe_fit(g, false, pl.gu_form);
    bool encoded = chunk(0);   // (before the first launch: the two follow one another closely)
    if (const int rc = moe_kernel_form<false>(pl.gu_form, gu, g, gbytes, sms, a.stream)) return rc;
    for (int c = 0; c < pl.chunks; ++c) {
      if (c > 0) encoded = chunk(c);
      if (!encoded) {
        set_error_detail("moe: cuTensorMapEncodeTiled failed (or is unavailable)");
        return Q4LIN_ERR_CUDA;
      }
      if (const int rc = moe_kernel_form<true>(pl.dn_form, dn, d, dbytes, sms, a.stream)) return rc;
    }
    if (pl.dn_form != kLatency) {
      cudaLaunchAttribute at[1];
      const int64_t n = (int64_t)tp * (a.H / 4);
      const cudaLaunchConfig_t cfg = moe_config((unsigned)((n + kReduceThreads - 1) / kReduceThreads), kReduceThreads, a.stream, at);
      if (cuda_check(pl.chunks > 1 ? cudaLaunchKernelEx(&cfg, q4_moe_reduce_kernel<true>, p)
                                   : cudaLaunchKernelEx(&cfg, q4_moe_reduce_kernel<false>, p),
                     "moe: reduction launch"))
        return Q4LIN_ERR_CUDA;
    }
  }
  return Q4LIN_OK;
}

int moe_status(int* value, bool clear) {
  if (cudaMemcpyFromSymbol(value, g_moe_status, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_moe_status, &zero, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  }
  return Q4LIN_OK;
}

}  // namespace q4
