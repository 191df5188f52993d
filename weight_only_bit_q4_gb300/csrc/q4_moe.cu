// Mixture-of-experts layer with Q4_G64_FP16 experts, for a few tokens.
//
//   router    l[t, e] = sum_h x[t, h] wr[e, h] (+ bias[e]),  p = softmax(l[t, :]),
//             the top_k experts of each token by l (ties: the lowest e first), their p
//             (divided by their sum if asked);
//   gate/up   h[t, j, f] = silu(g) u,  g = sum_k W_gate[e, f, k] x[t, k],  u likewise with
//             W_up, e = ids[t, j], silu(z) = z / (1 + e^-z);
//   down      y[t, n] = bf16( sum_j p[t, j] sum_f W_down[e, n, f] h[t, j, f] ).
//
// Three kernels chained by programmatic dependent launch.  Bound: the packed weights of
// the experts that some token chose, each read once; the kernels below therefore sort
// the (token, choice) slots by expert and stream each chosen expert's rows once for all
// of its tokens (8 token columns per MMA tile, up to kMaxNT tiles at a time).
//
// Products.  mma.sync m16n8k16 on bf16 operands with FP32 accumulation.  A: the codes as
// exact bf16 integers q - 8 (|q - 8| <= 8): a masked nibble pair OR-ed into the mantissa
// of 128 is the bf16 pair 128 + q, minus 136.  B, gate/up: x as it is (bf16), so every
// product is exact.  B, down: h in FP32 is split into two bf16 terms h = hi + lo (relative
// error 2^-17; one bf16 rounding of h alone would put about 1e-3 rms(y) of error into y),
// two MMAs.  The 64 weights of a scale group go through four (eight) MMAs into a fresh
// accumulator D, then acc += s D in FP32.
//
// Operand layout, as in the streaming warp-MMA route: the K order inside an MMA is free as
// long as A and B agree, so thread (g = lane / 4, c = lane % 4) takes the 16 weights
// k = 16 c .. 16 c + 15 of a group (8 code bytes per row) and the same 16 values of token
// column g (two 16-byte loads), and pairs them as the nibble masks do: (k, k + 4).
//
// A unit is 16 MMA rows = two boxes of 8 weight rows: gate rows f0 .. f0 + 7 over up rows
// f0 .. f0 + 7 (a thread then holds g and u of the same f and token), or 16 rows of
// W_down.  Box row of MMA row g is 2g mod 8 (+ 1 from g = 4): in the 128-byte-swizzled
// box the 8-byte code loads of a half warp then hit 16 different bank pairs.
//
// Streaming.  Every warp owns a ring of shared-memory slots, one sub-box (two boxes of
// 8 rows x 256 weights, 2 KB, TMA) each, and works through its own sequence of
// (unit, sub-box): lane 0 refills a slot as soon as the warp has read it, across unit
// borders, so no warp waits for another and the ring is the only buffering.
//
// Every mbarrier wait is bounded (kSpinLimit): on expiry the kernel records
// Q4LIN_ERR_TIMEOUT, the warps stop computing, pass the CTA barriers and drain the
// copies that they issued.
#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

__device__ int g_moe_status = 0;

constexpr int kMoeWarps = 8;
constexpr int kMoeThreads = 32 * kMoeWarps;
constexpr int kBoxBytes = 8 * 128;
constexpr int kSlotBytes = 2 * kBoxBytes;   // one sub-box: 16 rows x 256 weights
constexpr int kMaxNT = 4;                   // token tiles of 8 handled together
constexpr int kMaxSlots = 512;              // (token, choice) pairs per pass
constexpr int kMaxExperts = 1024;

// ----------------------------------------------------------------- router
constexpr int kRouteCluster = 8;
constexpr int kRouteThreads = 512;
constexpr int kRouteTokens = 4;   // tokens per cluster

struct RouterParams {
  const uint16_t* x;      // [T, H]
  const uint16_t* w;      // [E, H]
  const float* bias;      // [E] or NULL
  int32_t* ids;           // [T, k]
  float* weights;         // [T, k]
  int64_t T, H;
  int E, k, renorm;
};

// One cluster per kRouteTokens tokens: its 128 warps share the experts, a warp's lanes
// share H; the logits meet in the shared memory of the cluster's first CTA, whose first
// warps pick the top_k of one token each.
template <int TT>
__global__ void __cluster_dims__(kRouteCluster, 1, 1) __launch_bounds__(kRouteThreads)
q4_moe_router_kernel(const RouterParams p) {
  __shared__ float logit[TT][kMaxExperts];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t t0 = (int64_t)(blockIdx.x / kRouteCluster) * TT;
  cluster_sync();   // every CTA of the cluster runs before its shared memory is written
  pdl_wait_previous();
  constexpr int kWarps = kRouteThreads / 32;
  const int64_t nv = p.H / 8;
  for (int e = warp * kRouteCluster + (int)rank; e < p.E; e += kRouteCluster * kWarps) {
    float acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = 0.f;
    const uint16_t* wr = p.w + (int64_t)e * p.H;
#pragma unroll 4
    for (int64_t i = lane; i < nv; i += 32) {
      const uint4 wv = ld_global_u4(wr + 8 * i);
      const uint32_t ww[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int64_t tt = t0 + t < p.T ? t0 + t : p.T - 1;
        const uint4 xv = ld_global_u4(p.x + tt * p.H + 8 * i);
        const uint32_t xx[4] = {xv.x, xv.y, xv.z, xv.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[t] = fmaf(bf16lo(ww[q]), bf16lo(xx[q]), acc[t]);
          acc[t] = fmaf(bf16hi(ww[q]), bf16hi(xx[q]), acc[t]);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = warp_sum(acc[t]);
    if (lane == 0) {
      const float b = p.bias != nullptr ? __uint_as_float(ld_global_u32(p.bias + e)) : 0.f;
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint32_t dst = mapa_shared(smem_u32(&logit[t][e]), 0);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(acc[t] + b) : "memory");
      }
    }
  }
  cluster_sync();
  if (rank != 0 || warp >= TT || t0 + warp >= p.T) return;
  // ---- one warp per token: softmax statistics, then top_k picks
  float* lg = logit[warp];
  constexpr float kNone = -INFINITY;   // never chosen: -inf, NaN and what is already chosen
  float m = kNone;
  for (int e = lane; e < p.E; e += 32) {
    const float v = lg[e];
    if (!(v > kNone)) lg[e] = kNone;   // NaN too
    else m = fmaxf(m, v);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  auto ex = [&](float v) { return v == m ? 1.f : expf(v - m); };   // m may be +inf
  float z = 0.f;
  for (int e = lane; e < p.E; e += 32) {
    const float v = lg[e];
    if (v > kNone) z += ex(v);
  }
  z = warp_sum(z);
  __syncwarp();
  float chosen = 0.f, mine = 0.f;   // lane j keeps pick j (k <= 32)
  int mine_id = -1;
  for (int j = 0; j < p.k; ++j) {
    float best = kNone;
    int at = -1;
    for (int e = lane; e < p.E; e += 32) {
      const float v = lg[e];
      if (v > best) {
        best = v;
        at = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, best, o);
      const int oa = __shfl_xor_sync(0xffffffffu, at, o);
      if (oa >= 0 && (at < 0 || ov > best || (ov == best && oa < at))) {
        best = ov;
        at = oa;
      }
    }
    const float pe = at >= 0 ? ex(best) : 0.f;
    chosen += pe;
    if (lane == j) {
      mine = pe;
      mine_id = at;
    }
    if (at >= 0 && lane == (at & 31)) lg[at] = kNone;
    __syncwarp();
  }
  if (lane < p.k) {
    const int64_t o = (t0 + warp) * p.k + lane;
    p.ids[o] = mine_id;
    p.weights[o] = mine_id >= 0 ? mine / (p.renorm ? chosen : z) : 0.f;
  }
}

// ----------------------------------------------------------------- slots by expert
struct MoeParams {
  const uint16_t* x;       // [T, H] bf16 (first token of the pass)
  const int32_t* ids;      // [T, k]
  const float* weights;    // [T, k]
  const uint16_t* s_gu;    // [E, 2F, Hp/64]
  const uint16_t* s_dn;    // [E, H, Fp/64]
  uint16_t* h_hi;          // [T k, F] bf16 high and low terms of h
  uint16_t* h_lo;
  uint16_t* y;             // [T, H]
  int64_t H, F;
  int E, k, slots;         // slots = T k of this pass
  int depth;               // ring slots per warp
};

// Shared-memory lists of one CTA: the tiles (up to 8 kMaxNT slots of one expert) in
// expert order.
struct MoeLists {
  int* cnt;        // [E] slots per expert, then the fill positions
  int* order;      // [slots] slot numbers by expert
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
  const int tid = threadIdx.x;
  for (int e = tid; e < p.E; e += kMoeThreads) L.cnt[e] = 0;
  __syncthreads();
  for (int s = tid; s < p.slots; s += kMoeThreads) {
    const int e = (int)ld_global_u32(p.ids + s);
    if (e >= 0 && e < p.E) atomicAdd(&L.cnt[e], 1);
  }
  __syncthreads();
  if (tid < 32) {  // exclusive sums over the experts, 32 at a time
    int base = 0, tbase = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int e = e0 + tid;
      const int n = e < p.E ? L.cnt[e] : 0;
      const int nt = (n + per - 1) / per;
      int a = n, b = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a2 = __shfl_up_sync(0xffffffffu, a, o), b2 = __shfl_up_sync(0xffffffffu, b, o);
        if (tid >= o) {
          a += a2;
          b += b2;
        }
      }
      const int pos = base + a - n, tp = tbase + b - nt;
      for (int i = 0; i < nt; ++i) {
        const int left = n - i * per;
        L.tiles[tp + i] = make_int2(e, (pos + i * per) | ((left < per ? left : per) << 16));
      }
      if (e < p.E) L.cnt[e] = pos;
      base += __shfl_sync(0xffffffffu, a, 31);
      tbase += __shfl_sync(0xffffffffu, b, 31);
    }
    if (tid == 0) *L.ntiles = tbase;
  }
  __syncthreads();
  if (tid < 32) {  // fill in slot order, 32 slots at a time: rank among the equal ids of the 32
    for (int s0 = 0; s0 < p.slots; s0 += 32) {
      const int s = s0 + tid;
      int e = s < p.slots ? (int)ld_global_u32(p.ids + s) : -1;
      if (e >= p.E) e = -1;
      const unsigned same = __match_any_sync(0xffffffffu, e);
      const int at = e >= 0 ? L.cnt[e] : 0;
      __syncwarp();
      if (e >= 0) {
        L.order[at + __popc(same & ((1u << tid) - 1u))] = s;
        if ((same >> tid) == 1u) L.cnt[e] = at + __popc(same);   // the highest lane of the id
      }
      __syncwarp();
    }
  }
  __syncthreads();
}

// ----------------------------------------------------------------- the product of a unit
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Code words w0, w1 (weights k .. k + 15) as eight bf16 pairs q - 8: (k, k + 4), (k + 1, k + 5),
// (k + 2, k + 6), (k + 3, k + 7), and the same of k + 8.
__device__ __forceinline__ void decode_pairs_bf16(uint2 w, uint32_t (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = bf16x2_sub136(((w.x >> (4 * i)) & 0x000F000Fu) | 0x43004300u);
    a[4 + i] = bf16x2_sub136(((w.y >> (4 * i)) & 0x000F000Fu) | 0x43004300u);
  }
}

// 8 consecutive bf16 values as the four pairs of decode_pairs_bf16.
__device__ __forceinline__ void pair_up(uint4 v, uint32_t* b) {
  b[0] = __byte_perm(v.x, v.z, 0x5410);
  b[1] = __byte_perm(v.x, v.z, 0x7632);
  b[2] = __byte_perm(v.y, v.w, 0x5410);
  b[3] = __byte_perm(v.y, v.w, 0x7632);
}

__device__ __forceinline__ uint2 lds_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

// acc[n] += the products of one sub-box (256 K values from k0) of one unit with the token
// columns of its tiles.  brow[n]: this thread's column of tile n (NULL: an empty column);
// with kSplit, blow[n] holds the low terms.
template <int NT, bool kSplit>
__device__ __forceinline__ void moe_sub_box(uint32_t slot, int g, int c, int64_t k0, int64_t K, const float (&sa)[4],
                                            const float (&sb)[4], const uint16_t* const (&brow)[NT],
                                            const uint16_t* const (&blow)[NT], int nt, float (&acc)[NT][4]) {
  const int r = (2 * g & 7) + (g >> 2);
  const uint32_t row0 = slot + (uint32_t)r * 128u, row1 = row0 + kBoxBytes;
#pragma unroll
  for (int gl = 0; gl < 4; ++gl) {
    const int64_t kg = k0 + 64 * gl;
    if (kg >= K) break;
    const uint32_t off = ((((uint32_t)(2 * gl + (c >> 1))) ^ (uint32_t)r) << 4) | (uint32_t)((c & 1) << 3);
    uint32_t a0[8], a1[8];
    decode_pairs_bf16(lds_v2(row0 + off), a0);
    decode_pairs_bf16(lds_v2(row1 + off), a1);
    const int64_t kt = kg + 16 * c;   // this thread's 16 values; K is a multiple of 8
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (NT > 1 && n >= nt) break;
      const bool v0 = brow[n] != nullptr && kt < K, v1 = brow[n] != nullptr && kt + 8 < K;
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      uint32_t b[8];
      pair_up(v0 ? ld_global_u4(brow[n] + kt) : zero, b);
      pair_up(v1 ? ld_global_u4(brow[n] + kt + 8) : zero, b + 4);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; i += 2) mma_bf16(d, a0[i], a1[i], a0[i + 1], a1[i + 1], b[i], b[i + 1]);
      if constexpr (kSplit) {
        pair_up(v0 ? ld_global_u4(blow[n] + kt) : zero, b);
        pair_up(v1 ? ld_global_u4(blow[n] + kt + 8) : zero, b + 4);
#pragma unroll
        for (int i = 0; i < 8; i += 2) mma_bf16(d, a0[i], a1[i], a0[i + 1], a1[i + 1], b[i], b[i + 1]);
      }
      acc[n][0] = fmaf(sa[gl], d[0], acc[n][0]);
      acc[n][1] = fmaf(sa[gl], d[1], acc[n][1]);
      acc[n][2] = fmaf(sb[gl], d[2], acc[n][2]);
      acc[n][3] = fmaf(sb[gl], d[3], acc[n][3]);
    }
  }
}

// The four group scales of a row from group G on (the plane rows hold an even number of
// scales, so pairs are 4-byte aligned; groups past the row read as zero).
__device__ __forceinline__ void load_scales(const uint16_t* row, int G, int groups, uint32_t (&w)[2]) {
  w[0] = G < groups ? ld_global_u32(row + G) : 0u;
  w[1] = G + 2 < groups ? ld_global_u32(row + G + 2) : 0u;
}

__device__ __forceinline__ void scales_f32(const uint32_t (&w)[2], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    s[2 * i] = fp16_bits_to_float((uint16_t)(w[i] & 0xFFFFu));
    s[2 * i + 1] = fp16_bits_to_float((uint16_t)(w[i] >> 16));
  }
}

// Shared-memory layout: rings (1024-byte aligned), barriers, lists, then (down) the slot sums.
struct MoeLayout {
  uint32_t bar_off, cnt_off, order_off, tiles_off, misc_off, sum_off, total;
};

__host__ __device__ inline MoeLayout moe_layout(int depth, int E, int slots, int per, bool down) {
  MoeLayout L;
  L.bar_off = (uint32_t)(kMoeWarps * depth * kSlotBytes);
  L.cnt_off = L.bar_off + (uint32_t)(kMoeWarps * depth * 8);
  L.tiles_off = (L.cnt_off + (uint32_t)E * 4 + 7) / 8 * 8;
  L.order_off = L.tiles_off + (uint32_t)moe_max_tiles(slots, E, per) * 8;
  L.misc_off = L.order_off + (uint32_t)slots * 4;
  L.sum_off = (L.misc_off + 8 + 15) / 16 * 16;
  L.total = L.sum_off + (down ? (uint32_t)slots * 64 : 0u);
  return L;
}

// kDown false: gate/up units, h written; true: down units, y written.
template <int NT, bool kDown>
__global__ void __launch_bounds__(kMoeThreads, 2)
q4_moe_kernel(const __grid_constant__ CUtensorMap tm, const MoeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  constexpr int kPer = 8 * NT;
  const MoeLayout S = moe_layout(p.depth, p.E, p.slots, kPer, kDown);
  MoeLists L;
  L.cnt = reinterpret_cast<int*>(smem + S.cnt_off);
  L.order = reinterpret_cast<int*>(smem + S.order_off);
  L.tiles = reinterpret_cast<int2*>(smem + S.tiles_off);
  L.ntiles = reinterpret_cast<int*>(smem + S.misc_off);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S.misc_off + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMoeWarps * p.depth; ++i) mbar_init(sbase + S.bar_off + 8u * (uint32_t)i, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tm);
  }
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

  const int64_t K = kDown ? p.F : p.H;
  const int nsb = (int)((K + 255) / 256);
  const int groups = (int)((K + 63) / 64), grow = (int)(((K + 127) / 128 * 128) / 64);
  const int64_t rows_e = kDown ? p.H : 2 * p.F;                        // weight rows per expert
  const int nu = (int)(kDown ? (p.H + 15) / 16 : p.F / 8);              // units per expert
  const uint16_t* scales = kDown ? p.s_dn : p.s_gu;
  // Units of this CTA.  Gate/up: (tile, unit) pairs in tile order, a contiguous range per CTA
  // (its warps then share one expert's tokens), dealt to the warps in turn.  Down: every
  // gridDim-th unit with all tiles, the tiles dealt to the warps.  (The host bounds
  // nu * tiles below 2^31.)
  int u0, u1;
  if constexpr (!kDown) {
    const int64_t all = (int64_t)nu * ntiles;
    u0 = (int)((int64_t)blockIdx.x * all / gridDim.x);
    u1 = (int)((int64_t)(blockIdx.x + 1) * all / gridDim.x);
  } else {
    u0 = (int)blockIdx.x;
    u1 = nu;
  }
  // this warp's items: unit u0 + warp, + 8, ... (gate/up); per unit, tiles warp, warp + 8, ... (down)
  const int per_unit = ntiles > warp ? (ntiles - warp + kMoeWarps - 1) / kMoeWarps : 0;
  auto row_base = [&](int tile, int unit, int64_t& row0, int64_t& row1) {
    row0 = (int64_t)L.tiles[tile].x * rows_e + (kDown ? 16 : 8) * (int64_t)unit;
    row1 = row0 + (kDown ? 8 : p.F);
  };
  const uint32_t ring0 = sbase + (uint32_t)(warp * p.depth * kSlotBytes);
  const uint32_t bars = sbase + S.bar_off + (uint32_t)(warp * p.depth * 8);
  // ---- issue side (lane 0): the warp's items once more, sub-box by sub-box, `depth` ahead
  int is_unit = kDown ? u0 : 0, is_tile = kDown ? warp : 0, is_flat = u0 + warp, is_sb = 0, is_slot = 0;
  int64_t is_row0 = 0, is_row1 = 0;
  int64_t issued = 0;
  bool more = kDown ? (u0 < nu && per_unit > 0) : is_flat < u1;
  auto issue = [&]() {
    if (is_sb == 0) {
      if constexpr (!kDown) {
        is_tile = is_flat / nu;
        is_unit = is_flat - is_tile * nu;
      }
      row_base(is_tile, is_unit, is_row0, is_row1);
    }
    const uint32_t bar = bars + 8u * (uint32_t)is_slot, dst = ring0 + (uint32_t)is_slot * kSlotBytes;
    mbar_expect_tx(bar, kSlotBytes);
    tma_load_2d(dst, &tm, bar, is_sb * 128, (int32_t)is_row0);
    tma_load_2d(dst + kBoxBytes, &tm, bar, is_sb * 128, (int32_t)is_row1);
    ++issued;
    if (++is_slot == p.depth) is_slot = 0;
    if (++is_sb == nsb) {
      is_sb = 0;
      if constexpr (!kDown) {
        is_flat += kMoeWarps;
        more = is_flat < u1;
      } else {
        is_tile += kMoeWarps;
        if (is_tile >= ntiles) {
          is_tile = warp;
          is_unit += (int)gridDim.x;
          more = is_unit < nu;
        }
      }
    }
  };
  if (lane == 0)
    for (int d = 0; d < p.depth && more; ++d) issue();
  if constexpr (kDown) pdl_wait_previous();

  bool ok = true;
  int slot = 0;
  uint32_t phase = 0;
  float* sums = reinterpret_cast<float*>(smem + S.sum_off);   // down: [slots][16]
  // down: one round per unit; gate/up: a single round over the CTA's range
  for (int round = kDown ? u0 : 0; round < (kDown ? nu : 1); round += kDown ? (int)gridDim.x : 1) {
    const int i_end = kDown ? ntiles : u1;
    for (int i = kDown ? warp : u0 + warp; i < i_end; i += kMoeWarps) {
      const int tile = kDown ? i : i / nu, unit = kDown ? round : i - tile * nu;
      const int2 tl = L.tiles[tile];
      const int first = tl.y & 0xFFFF, count = tl.y >> 16;
      const int nt = (count + 7) / 8;
      const int r = (2 * g & 7) + (g >> 2);
      int64_t row0, row1;
      row_base(tile, unit, row0, row1);
      if (kDown && 16 * (int64_t)unit + 8 >= p.H) row1 = row0;   // no second box: its results are dropped
      row0 += r;
      row1 += r;
      const uint16_t* srow0 = scales + row0 * grow;
      const uint16_t* srow1 = scales + row1 * grow;
      const uint16_t* brow[NT];
      const uint16_t* blow[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int s = 8 * n + g < count ? L.order[first + 8 * n + g] : -1;
        brow[n] = blow[n] = nullptr;
        if (s >= 0) {
          brow[n] = kDown ? p.h_hi + (int64_t)s * p.F : p.x + (int64_t)(s / p.k) * p.H;
          if (kDown) blow[n] = p.h_lo + (int64_t)s * p.F;
        }
      }
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
      uint32_t w0[2], w1[2];
      load_scales(srow0, 0, groups, w0);
      load_scales(srow1, 0, groups, w1);
      for (int sb = 0; sb < nsb; ++sb) {
        float sa[4], sc[4];
        scales_f32(w0, sa);
        scales_f32(w1, sc);
        if (sb + 1 < nsb) {   // the next sub-box's scales
          load_scales(srow0, 4 * (sb + 1), groups, w0);
          load_scales(srow1, 4 * (sb + 1), groups, w1);
        }
        ok = ok && warp_wait(bars + 8u * (uint32_t)slot, phase, abort_flag, &g_moe_status);
        if (ok) {
          moe_sub_box<NT, kDown>(ring0 + (uint32_t)slot * kSlotBytes, g, c, 256 * (int64_t)sb, K, sa, sc, brow, blow, nt, acc);
          __syncwarp();
          if (lane == 0 && more) issue();   // refill the slot just read
          if (++slot == p.depth) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) continue;
      // ---- the unit's results: thread (g, c) holds MMA rows g, g + 8 of token columns 2c, 2c + 1
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (NT > 1 && n >= nt) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int col = 8 * n + 2 * c + j;
          if (col >= count) continue;
          const int s = L.order[first + col];
          if constexpr (kDown) {
            sums[s * 16 + r] = acc[n][j];
            sums[s * 16 + 8 + r] = acc[n][2 + j];
          } else {
            const float gt = acc[n][j], up = acc[n][2 + j];
            const float h = gt / (1.f + expf(-gt)) * up;
            const uint16_t hi = float_to_bf16_bits(h);
            const float rest = h - __uint_as_float((uint32_t)hi << 16);
            const int64_t o = (int64_t)s * p.F + 8 * (int64_t)unit + r;
            p.h_hi[o] = hi;
            // an infinite or NaN h has no low term
            p.h_lo[o] = fabsf(h) < INFINITY ? float_to_bf16_bits(rest) : (uint16_t)0;
          }
        }
      }
    }
    if constexpr (kDown) {
      __syncthreads();
      const int64_t n0 = 16 * (int64_t)round;
      const int tokens = p.slots / p.k;
      if (!*abort_flag) {
        for (int e = threadIdx.x; e < tokens * 16; e += kMoeThreads) {
          const int t = e >> 4, rr = e & 15;
          if (n0 + rr >= p.H) continue;
          float v = 0.f;
          for (int j = 0; j < p.k; ++j) {   // in the order of the choices
            const int s = t * p.k + j;
            const int id = (int)ld_global_u32(p.ids + s);
            if (id >= 0 && id < p.E) v = fmaf(__uint_as_float(ld_global_u32(p.weights + s)), sums[s * 16 + rr], v);
          }
          p.y[(int64_t)t * p.H + n0 + rr] = float_to_bf16_bits(v);
        }
      }
      __syncthreads();   // the sums are free again
    }
  }
  if (!ok && lane == 0)   // aborted: let the copies already issued land before the CTA exits
    for (int64_t d = issued > p.depth ? issued - p.depth : 0; d < issued; ++d)
      mbar_drain(bars + 8u * (uint32_t)(d % p.depth), (uint32_t)((d / p.depth) & 1));
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

constexpr int kMoeSmem = 112 * 1024;   // dynamic shared memory at most (two CTAs per SM)

template <int NT, bool kDown>
int moe_kernel_launch(const CUtensorMap& tm, const MoeParams& p0, int sms, cudaStream_t stream) {
  static bool attr[64] = {};
  int dev = 0;
  if (cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return Q4LIN_ERR_CUDA;
  if (dev >= 64 || !attr[dev]) {
    if (cuda_check(cudaFuncSetAttribute(q4_moe_kernel<NT, kDown>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoeSmem),
                   "moe: cudaFuncSetAttribute"))
      return Q4LIN_ERR_CUDA;
    if (dev < 64) attr[dev] = true;
  }
  MoeParams p = p0;
  p.depth = 8;
  MoeLayout L = moe_layout(p.depth, p.E, p.slots, 8 * NT, kDown);
  while (p.depth > 2 && L.total + 1024 > kMoeSmem) L = moe_layout(--p.depth, p.E, p.slots, 8 * NT, kDown);
  if (L.total + 1024 > kMoeSmem) {
    set_error_detail("moe: the slot lists do not fit shared memory");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * sms), 1, 1);
  cfg.blockDim = dim3(kMoeThreads, 1, 1);
  cfg.dynamicSmemBytes = L.total + 1024;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_moe_kernel<NT, kDown>, tm, p), kDown ? "moe: down kernel launch" : "moe: gate/up kernel launch");
}

template <bool kDown>
int moe_kernel_nt(int nt, const CUtensorMap& tm, const MoeParams& p, int sms, cudaStream_t stream) {
  if (nt <= 1) return moe_kernel_launch<1, kDown>(tm, p, sms, stream);
  if (nt <= 2) return moe_kernel_launch<2, kDown>(tm, p, sms, stream);
  return moe_kernel_launch<kMaxNT, kDown>(tm, p, sms, stream);
}

}  // namespace

int moe_pass_tokens(int64_t T, int k) {
  const int most = kMaxSlots / k;
  return (int)(T < most ? T : most);
}

size_t moe_workspace_bytes(int64_t T, int64_t F, int k) {
  const size_t one = ((size_t)moe_pass_tokens(T, k) * (size_t)k * (size_t)F * 2 + 255) / 256 * 256;
  return 2 * one;
}

int moe_launch_count(int64_t T, int k) {
  const int tp = moe_pass_tokens(T, k);
  return 2 * (int)((T + tp - 1) / tp);
}

int moe_router_launch(const MoeArgs& a) {
  RouterParams p{a.x, a.w_router, a.bias, a.ids_out, a.weights_out, a.T, a.H, (int)a.E, a.k, a.renorm};
  const int tt = a.T < kRouteTokens ? (a.T == 1 ? 1 : 2) : kRouteTokens;
  const int64_t clusters = (a.T + tt - 1) / tt;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(clusters * kRouteCluster), 1, 1);
  cfg.blockDim = dim3(kRouteThreads, 1, 1);
  cfg.stream = a.stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  cudaError_t e;
  switch (tt) {
    case 1: e = cudaLaunchKernelEx(&cfg, q4_moe_router_kernel<1>, p); break;
    case 2: e = cudaLaunchKernelEx(&cfg, q4_moe_router_kernel<2>, p); break;
    default: e = cudaLaunchKernelEx(&cfg, q4_moe_router_kernel<kRouteTokens>, p); break;
  }
  return cuda_check(e, "moe: router kernel launch");
}

int moe_experts_launch(const MoeArgs& a) {
  const int64_t Hp = k_pad(a.H), Fp = k_pad(a.F);
  CUtensorMap gu, dn;
  if (!encode_map_2d(&gu, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq_gu, (uint64_t)(Hp / 2), (uint64_t)(a.E * 2 * a.F),
                     (uint64_t)(Hp / 2), 128, 8, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_map_2d(&dn, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.wq_dn, (uint64_t)(Fp / 2), (uint64_t)(a.E * a.H),
                     (uint64_t)(Fp / 2), 128, 8, CU_TENSOR_MAP_SWIZZLE_128B)) {
    set_error_detail("moe: cuTensorMapEncodeTiled failed (or is unavailable)");
    return Q4LIN_ERR_CUDA;
  }
  const int sms = moe_sm_count();
  const int pass = moe_pass_tokens(a.T, a.k);
  const size_t one = moe_workspace_bytes(a.T, a.F, a.k) / 2;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  for (int64_t t0 = 0; t0 < a.T; t0 += pass) {
    const int tp = (int)(a.T - t0 < pass ? a.T - t0 : pass);
    MoeParams p{};
    p.x = a.x + t0 * a.H;
    p.ids = a.ids + t0 * a.k;
    p.weights = a.weights + t0 * a.k;
    p.s_gu = a.s_gu;
    p.s_dn = a.s_dn;
    p.h_hi = reinterpret_cast<uint16_t*>(ws);
    p.h_lo = reinterpret_cast<uint16_t*>(ws + one);
    p.y = a.y + t0 * a.H;
    p.H = a.H;
    p.F = a.F;
    p.E = (int)a.E;
    p.k = a.k;
    p.slots = tp * a.k;
    // token tiles handled together: as many as one expert can get when every token chooses it
    const int nt = (tp + 7) / 8;
    if (const int rc = moe_kernel_nt<false>(nt, gu, p, sms, a.stream)) return rc;
    if (const int rc = moe_kernel_nt<true>(nt, dn, p, sms, a.stream)) return rc;
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
