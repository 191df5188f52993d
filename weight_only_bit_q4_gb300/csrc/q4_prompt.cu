// Attention over whole prompts: causal, grouped heads, sequences packed after one another.
//
// For token t (row i of its sequence) and query head h of group g:
//     y = sum_{j <= i} p_j v_j / sum_{j <= i} p_j,  p_j = 2^((q . k_j) scale log2 e - m),
// over the tokens j of the same sequence.  Scores, maxima and sums are FP32.  P enters the second
// product as bf16, its operands' type (V is bf16): 2^-9 of each weight, as much as the output's
// own rounding.
//
// Bound: the tensor cores (4 D operations per query head and pair of tokens that see each other);
// beside them the exponentials, one per pair.
//
// Split: a CTA (one per SM) owns two tiles of 128 query rows, A and B, that read the same keys: two
// heads of a group where there is an even number of them, else two runs of rows of a head.  Blocks
// of 128 keys stream through shared memory (TMA, 128-byte swizzle), from the diagonal down.
//   warps 4-7, 8-11  softmax of A, of B: a thread owns a row.  It reads its 128 scores from tensor
//                    memory, and writes P (bf16) over them.  The reference m moves only when a
//                    score passes it by 2^8 (P and the sums then hold up to 2^8 times more, far
//                    from any end); only then is the row of O in tensor memory rescaled, by the
//                    same thread: the block's scores are complete only after the last P V.
//   warp 0           issues the MMAs: per block and tile P V (P from tensor memory, V as an
//                    MN-major operand), then the next block's Q K^T into the same columns.
//                    While A's are computed, B's softmax runs, and the other way round.
//   warp 1           issues the copies.
//   warps 2, 3       look blocks of V that hold keys some rows must not see over for values that are
//                    not finite (0 times infinity would reach those rows).  They become zeros for
//                    the MMA; the rows that see such a key add it at the end.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kPtThreads = 384;
constexpr int kPtTile = 128;          // rows of a tile, keys of a block
constexpr float kPtSlack = 8.f;       // log2 of how far a score may pass its row's reference
constexpr int kPtSoftRegs = 224, kPtOtherRegs = 56;
// the shares of three warpgroups come out of the registers at launch (168 a thread)
static_assert(2 * kPtSoftRegs + kPtOtherRegs <= 3 * 168, "register split");
constexpr uint32_t kPtBoxBytes = 64 * 2 * kPtTile;   // 64 columns of a tile
constexpr int kPtK = 2, kPtV = 3;     // stages of K and of V (all that shared memory holds for D = 128)
__device__ int g_prompt_status = 0;

struct PtParams {
  CUtensorMap mq, mk, mv;   // (D, heads, T)
  const uint16_t* v;
  uint16_t* out;
  int64_t ldv, ldo;
  const int32_t* cu;        // [S + 1]
  int64_t T;
  int S, Hq, Hk, G, D;
  int heads2;               // 1: the tiles are two heads, 0: two runs of rows
  int pairs;                // units per run of rows
  float c;                  // |scale| log2 e
  int negate;               // the scale is negative: Q enters negated
};

// Rows [a, b) of sequence s, within the tensors whatever cu holds.
__device__ __forceinline__ void pt_rows(const PtParams& p, int s, int64_t& a, int64_t& b) {
  a = (int32_t)ld_global_u32(p.cu + s);
  b = (int32_t)ld_global_u32(p.cu + s + 1);
  a = a < 0 ? 0 : a > p.T ? p.T : a;
  b = b < a ? a : b > p.T ? p.T : b;
}

__device__ __forceinline__ float pt_ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}

__device__ __forceinline__ uint32_t pt_pack(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float2 pt_fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
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

// The run of rows `index` of all sequences' runs (of `rows` rows), the last runs of a sequence
// first: its sequence's rows and its number within the sequence.  False: there are fewer.
struct PtRun {
  int64_t a, b;
  int run;
};
__device__ __forceinline__ bool pt_find(const PtParams& p, int rows, int64_t index, PtRun* found, int64_t* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found->run = -1;
  int64_t before = 0;
  for (int s0 = 0; s0 < p.S; s0 += kPtThreads) {
    int64_t a = 0, b = 0;
    if (s0 + tid < p.S) pt_rows(p, s0 + tid, a, b);
    const int64_t n = (b - a + rows - 1) / rows;
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
      found->run = (int)(upto - 1 - index);
    }
    before += all;
    if (index < before) break;   // (uniform)
  }
  __syncthreads();
  return found->run >= 0;
}

__device__ __forceinline__ void pt_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int d, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(d), "r"(h), "r"(t)
      : "memory");
}

// Shared-memory descriptor of V as the second operand: its rows are keys (the K dimension), 64
// columns (N) in a 128-byte line; 8 keys are 1024 bytes, the next 64 columns a box further on.
__device__ __forceinline__ uint64_t pt_v_desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kPtBoxBytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

template <int DB>   // 64-column boxes of a head
struct PtSmem {
  static constexpr uint32_t tile = DB * kPtBoxBytes;
  static constexpr uint32_t q = 0, k = 2 * tile, v = k + kPtK * tile, bars = v + kPtV * tile;
  // barriers: Q; K full, empty; V full, empty; per tile scores, P (with its operands), O; all MMAs done
  static constexpr uint32_t qf = bars, kf = qf + 8, ke = kf + 8 * kPtK, vf = ke + 8 * kPtK,
                            ve = vf + 8 * kPtV, sf = ve + 8 * kPtV, pf = sf + 16, of = pf + 16, done = of + 16, end = done + 8;
  static constexpr uint32_t alloc = end + 1024;   // (the base is aligned to 1024)
};

// Tensor memory: scores and P of tile x, O of tile x.
__device__ __forceinline__ uint32_t pt_s_col(int x) { return 128u * (uint32_t)x; }
__device__ __forceinline__ uint32_t pt_o_col(int x) { return 256u + 128u * (uint32_t)x; }

template <int DB>
__global__ void __launch_bounds__(kPtThreads, 1) q4_prompt_kernel(const __grid_constant__ PtParams p) {
  using SM = PtSmem<DB>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ PtRun found;
  __shared__ int64_t sums[kPtThreads / 32];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ volatile int odd_flag;   // V held a value that is not finite
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  pdl_launch_dependents();
  if (tid == 0) {
    abort_flag = 0;
    odd_flag = 0;
    mbar_init(base + SM::qf, 1);
    for (int i = 0; i < kPtK; ++i) {
      mbar_init(base + SM::kf + 8 * i, 1);
      mbar_init(base + SM::ke + 8 * i, 1);
    }
    for (int i = 0; i < kPtV; ++i) {
      mbar_init(base + SM::vf + 8 * i, 1);
      mbar_init(base + SM::ve + 8 * i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(base + SM::sf + 8 * x, 1);
      mbar_init(base + SM::pf + 8 * x, 6);   // four softmax warps, warps 2 and 3
      mbar_init(base + SM::of + 8 * x, 1);
    }
    mbar_init(base + SM::done, 1);
    fence_mbar_init();
    prefetch_tmap(&p.mq);
    prefetch_tmap(&p.mk);
    prefetch_tmap(&p.mv);
  }
  pdl_wait_previous();
  const int unit = blockIdx.x % p.pairs;
  const int64_t run = blockIdx.x / p.pairs;
  const int run_rows = p.heads2 ? kPtTile : 2 * kPtTile;
  if (!pt_find(p, run_rows, run, &found, sums)) return;   // (the whole CTA, nothing in flight)
  if (warp == 0) tmem_alloc(smem_u32(&tmem_base), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  const int64_t row0 = found.a;
  const int len = (int)(found.b - found.a);
  // tile x: its first row and head; the blocks of keys that it sees
  const int q0[2] = {found.run * run_rows, found.run * run_rows + (p.heads2 ? 0 : kPtTile)};
  const int head[2] = {p.heads2 ? 2 * unit : unit, p.heads2 ? 2 * unit + 1 : unit};
  const int n0 = (min(len, q0[0] + kPtTile) + kPtTile - 1) / kPtTile;
  const int n1 = q0[1] < len ? (min(len, q0[1] + kPtTile) + kPtTile - 1) / kPtTile : 0;
  const int n = max(n0, n1), hk = head[0] / p.G;
  const int edge = q0[0] / kPtTile;    // blocks from here on hold keys that some row does not see
  bool ok = true;

  if (warp >= 4) {
    // ------------------------------------------------ softmax
    setmaxnreg_inc<kPtSoftRegs>();
    const int x = (warp >> 2) - 1, nx = x ? n1 : n0;
    const int row = (x ? q0[1] : q0[0]) + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + pt_s_col(x), to = tmem + lanes + pt_o_col(x);
    float m = -INFINITY;
    float2 l = make_float2(0.f, 0.f);
    const float2 c2 = make_float2(p.c, p.c);
    for (int i = 0; i < nx && ok; ++i) {
      const int kb = nx - 1 - i;
      ok = warp_wait_vote(base + SM::sf + 8 * x, (uint32_t)(i & 1), &abort_flag, &g_prompt_status);
      if (!ok) break;
      tc_fence_after();
      uint32_t r[4][32];
#pragma unroll
      for (int j = 0; j < 4; ++j) tmem_ld32(ts + 32 * j, r[j]);
      tmem_ld_wait();
      if (kb * kPtTile + kPtTile - 1 > (x ? q0[1] : q0[0])) {
        const int see = row - kb * kPtTile;   // keys 0 .. see of the block
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * j + e > see) r[j][e] = 0xFF800000u;
      }
      float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          top = fmaxf(top, fmaxf(__uint_as_float(r[j][e]), __uint_as_float(r[j][e + 1])));
          top2 = fmaxf(top2, fmaxf(__uint_as_float(r[j][e + 2]), __uint_as_float(r[j][e + 3])));
        }
      top = fmaxf(top, top2) * p.c;
      const bool up = top > m + kPtSlack || (m == -INFINITY && top > m);
      if (__any_sync(0xffffffffu, up)) {
        const float f = up ? pt_ex2(m - top) : 1.f;
        if (up) m = top;
        l = pt_fmul2(l, make_float2(f, f));
        if (i > 0) {   // (the first P V overwrites O)
#pragma unroll 1
          for (int j = 0; j < 2 * DB; ++j) {
            uint32_t o[32];
            tmem_ld32(to + 32 * j, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(to + 32 * j, o);
          }
        }
      }
      const float mu = m == -INFINITY ? 0.f : -m;
      const float2 m2 = make_float2(mu, mu);
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        uint32_t w[32];
#pragma unroll
        for (int e = 0; e < 64; e += 2) {
          const float2 t = ffma2(make_float2(__uint_as_float(r[j + (e >> 5)][e & 31]), __uint_as_float(r[j + (e >> 5)][(e & 31) + 1])), c2, m2);
          const float2 pr = make_float2(pt_ex2(t.x), pt_ex2(t.y));
          l = fadd2(l, pr);
          w[e >> 1] = pt_pack(pr.x, pr.y);
        }
        tmem_st32(ts + 16 * j, w);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_release(base + SM::pf + 8 * x, lane);
    }
    // ------------------------------------------------ the rows of O
    if (nx > 0 && ok) ok = warp_wait_vote(base + SM::of + 8 * x, 0, &abort_flag, &g_prompt_status);
    if (nx > 0 && ok) {
      tc_fence_after();
      const float inv = 1.f / (l.x + l.y);
      const bool odd = odd_flag != 0;
      uint16_t* dst = p.out + (row0 + row) * p.ldo + (int64_t)(x ? head[1] : head[0]) * p.D;
#pragma unroll 1
      for (int j = 0; j < 2 * DB; ++j) {
        uint32_t o[32];
        tmem_ld32(to + 32 * j, o);
        tmem_ld_wait();
        if (odd && row < len)   // the keys left out of the products, for the rows that see them
          for (int key = edge * kPtTile; key <= row; ++key) {
            const uint16_t* src = p.v + (row0 + key) * p.ldv + (int64_t)hk * p.D + 32 * j;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (32 * j + 8 * b >= p.D) break;
              const uint4 w = ld_global_u4(src + 8 * b);
              if (!not_finite(w)) continue;
              const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float val = e & 1 ? bf16hi(ws[e >> 1]) : bf16lo(ws[e >> 1]);
                if (!(fabsf(val) <= FLT_MAX)) o[8 * b + e] = __float_as_uint(__uint_as_float(o[8 * b + e]) + val);
              }
            }
          }
        if (row < len)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (32 * j + 8 * b < p.D) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pt_pack(__uint_as_float(o[8 * b + 2 * e]) * inv, __uint_as_float(o[8 * b + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + 32 * j + 8 * b) = make_uint4(w[0], w[1], w[2], w[3]);
            }
      }
    }
    tc_fence_before();
  } else {
    setmaxnreg_dec<kPtOtherRegs>();
    if (warp == 0) {
      // ---------------------------------------------- MMAs
      const int steps = (p.D + 15) / 16;
      const uint32_t is = idesc_kind_f16(kPtTile, kPtTile, 1) | (p.negate ? 1u << 13 : 0u);
      const uint32_t io = idesc_kind_f16(kPtTile, 16, 1) + ((uint32_t)(steps - 1) << 18) | 1u << 16;   // N = D, V is N-major
      // descriptors as 32-bit halves; the low one counts in 16 bytes
      const uint64_t qd = sw128_desc(base + SM::q), kd = sw128_desc(base + SM::k), vd = pt_v_desc(base + SM::v);
      const uint32_t kmajor = (uint32_t)(qd >> 32), nmajor = (uint32_t)(vd >> 32);
      const bool one = elect_one();
      auto scores = [&](auto lo, auto hi, int x, uint32_t st) {   // k-steps lo .. hi - 1 of Q K^T
        const uint32_t a = (uint32_t)qd + (uint32_t)x * (SM::tile >> 4), b = (uint32_t)kd + st * (SM::tile >> 4);
        if (one) {
#pragma unroll
          for (int s = lo.value; s < hi.value; ++s)
            if (s < steps) {
              constexpr uint32_t box = kPtBoxBytes >> 4;
              mma_f16_ss(tmem + pt_s_col(x), a + (uint32_t)(s >> 2) * box + 2u * (s & 3), kmajor,
                         b + (uint32_t)(s >> 2) * box + 2u * (s & 3), kmajor, is, s > 0);
            }
        }
      };
      using Lo = std::integral_constant<int, 0>;
      using Mid = std::integral_constant<int, DB == 2 ? 5 : 2>;
      using Hi = std::integral_constant<int, 4 * DB>;
      auto values = [&](int x, uint32_t st, uint32_t join) {   // P V
        const uint32_t b = (uint32_t)vd + st * (SM::tile >> 4);
        if (one) {
#pragma unroll
          for (int s = 0; s < kPtTile / 16; ++s)
            mma_f16_ts32(tmem + pt_o_col(x), tmem + pt_s_col(x) + 8u * s, b + 128u * s, nmajor, io, s > 0 ? 1u : join);
        }
      };
      auto commit = [&](uint32_t bar) {
        if (one) mma_commit(bar);
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = warp_wait_vote(bar, parity, &abort_flag, &g_prompt_status);
        return ok;
      };
      // block i of the loop is keys (n - 1 - i) * 128 on; tile x takes part from its own last block on
      const int from0 = n - n0, from1 = n1 > 0 ? n - n1 : n;
      const uint32_t pf = base + SM::pf, sf = base + SM::sf;
      uint32_t vs = 0, ks = 0, ph0 = 0, ph1 = 0;   // stages of V of block i and of K of block i + 1; phases
      if (wait(base + SM::qf, 0) && wait(base + SM::kf, 0)) {
        for (int x = 0; x < 2; ++x)
          if ((x ? from1 : from0) == 0) {
            scores(Lo{}, Hi{}, x, 0);
            commit(sf + 8 * x);
          }
        commit(base + SM::ke);
      }
      // The barrier of a tile's P stands for V of the block and K of the next one too (warps 2 and 3 wait
      // for those).  It is looked up once in the middle of the other tile's Q K^T: a wait's own
      // latency (some 300 cycles beside two softmax warps) then lies behind work in the queue.
      bool there = false;
      for (int i = 0; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        if (more && ++ks == kPtK) ks = 0;
        if (i >= from0) {
          if (!there && !wait(pf, ph0)) break;
          ph0 ^= 1u;
          tc_fence_after();
          values(0, vs, i > from0);
          if (!more) commit(base + SM::of);
        }
        const bool s0 = more && i + 1 >= from0, s1 = more && i + 1 >= from1;
        if (s0) scores(Lo{}, Mid{}, 0, ks);
        there = i >= from1 && warp_test(pf + 8, ph1);
        if (s0) {
          scores(Mid{}, Hi{}, 0, ks);
          commit(sf);
        }
        if (i >= from1) {
          if (!there && !wait(pf + 8, ph1)) break;
          ph1 ^= 1u;
          tc_fence_after();
          values(1, vs, i > from1);
          if (!more) commit(base + SM::of + 8);
        }
        commit(base + SM::ve + 8 * vs);
        if (++vs == kPtV) vs = 0;
        if (s1) scores(Lo{}, Mid{}, 1, ks);
        there = s0 && warp_test(pf, ph0);
        if (s1) {
          scores(Mid{}, Hi{}, 1, ks);
          commit(sf + 8);
        }
        if (more) commit(base + SM::ke + 8 * ks);
      }
      // nothing is in flight behind this
      commit(base + SM::done);
      if (one) mbar_drain(base + SM::done, 0);
    } else if (warp == 1 && lane == 0) {
      // ---------------------------------------------- copies
      mbar_expect_tx(base + SM::qf, (n1 > 0 ? 2 : 1) * SM::tile);
      for (int x = 0; x < (n1 > 0 ? 2 : 1); ++x)
        for (int b = 0; b < DB; ++b)
          pt_load(base + SM::q + (uint32_t)x * SM::tile + b * kPtBoxBytes, &p.mq, base + SM::qf, 64 * b, head[x], (int)(row0 + q0[x]));
      // the loads of block i, K's and V's: a stage is free once its last use has completed
      int ki = 0, vi = 0;
      auto load = [&](const CUtensorMap* map, uint32_t tiles, uint32_t full, uint32_t empty, int stages, int& i) {
        const int st = i % stages;
        if (i >= stages && !mbar_wait(empty + 8 * st, ((uint32_t)(i / stages) & 1u) ^ 1u, &abort_flag, &g_prompt_status)) return false;
        mbar_expect_tx(full + 8 * st, SM::tile);
        for (int b = 0; b < DB; ++b)
          pt_load(tiles + (uint32_t)st * SM::tile + b * kPtBoxBytes, map, full + 8 * st, 64 * b, hk, (int)row0 + (n - 1 - i) * kPtTile);
        ++i;
        return true;
      };
      while (vi < n) {   // (K of block i + 1 is wanted before V of block i)
        if (ki < n && !load(&p.mk, base + SM::k, base + SM::kf, base + SM::ke, kPtK, ki)) break;
        if (ki == 1 && ki < n && !load(&p.mk, base + SM::k, base + SM::kf, base + SM::ke, kPtK, ki)) break;
        if (!load(&p.mv, base + SM::v, base + SM::vf, base + SM::ve, kPtV, vi)) break;
      }
      // the CTA does not end before its copies have landed
      mbar_drain(base + SM::qf, 0);
      for (int i = max(0, ki - kPtK); i < ki; ++i) mbar_drain(base + SM::kf + 8 * (i % kPtK), (uint32_t)(i / kPtK) & 1u);
      for (int i = max(0, vi - kPtV); i < vi; ++i) mbar_drain(base + SM::vf + 8 * (i % kPtV), (uint32_t)(i / kPtV) & 1u);
    } else if (warp >= 2) {
      // ---------------------------------------------- V at the edge, and word that a block's operands are there
      const int from[2] = {n - n0, n1 > 0 ? n - n1 : n};
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (ok) ok = warp_wait_vote(bar, parity, &abort_flag, &g_prompt_status);
        return ok;
      };
      for (int i = 0; i < n && ok; ++i) {
        if (!wait(base + SM::vf + 8 * (i % kPtV), (uint32_t)(i / kPtV) & 1u)) break;
        if (n - 1 - i >= edge) {
          const uint32_t at = base + SM::v + (uint32_t)(i % kPtV) * SM::tile;
          for (uint32_t o = (uint32_t)(tid - 64) * 16; o < SM::tile; o += 64 * 16) {
            const uint4 w = ld_shared_v4(at + o);
            if (not_finite(w)) {
              st_shared_v4(at + o, finite_only(w));
              odd_flag = 1;
            }
          }
          fence_proxy_async();
        }
        if (i + 1 < n && !wait(base + SM::kf + 8 * ((i + 1) % kPtK), (uint32_t)((i + 1) / kPtK) & 1u)) break;
        for (int x = 0; x < 2; ++x)
          if (i >= from[x]) {
            // (an arrival before the last phase is complete would count for that one)
            if (i > from[x] && !wait(base + SM::pf + 8 * x, (uint32_t)(i - from[x] - 1) & 1u)) break;
            warp_release(base + SM::pf + 8 * x, lane);
          }
      }
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Rows of heads as a tensor (D, heads, T) of boxes of 64 columns of a head and 128 rows.
bool pt_map(CUtensorMap* m, const void* base, int64_t D, int64_t heads, int64_t T, int64_t ld) {
  return encode_map_3d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, {(uint64_t)D, (uint64_t)heads, (uint64_t)T},
                       {(uint64_t)D * 2, (uint64_t)ld * 2}, {64, 1, kPtTile}, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int DB>
int pt_run(const PtParams& p, unsigned blocks, cudaStream_t stream) {
  constexpr int smem = (int)PtSmem<DB>::alloc;
  static bool set[64] = {};
  int dev = 0;
  if (cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return Q4LIN_ERR_CUDA;
  if (dev >= 64 || !set[dev]) {
    if (cuda_check(cudaFuncSetAttribute(q4_prompt_kernel<DB>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
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
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_prompt_kernel<DB>, p), "prompt_attention: kernel launch");
}

}  // namespace

int prompt_launch(const PromptArgs& a) {
  PtParams p{};
  if (!pt_map(&p.mq, a.q, a.D, a.Hq, a.T, a.ldq) || !pt_map(&p.mk, a.k, a.D, a.Hk, a.T, a.ldk) ||
      !pt_map(&p.mv, a.v, a.D, a.Hk, a.T, a.ldv)) {
    set_error_detail("prompt_attention: the tensors cannot be described to the copy engine");
    return Q4LIN_ERR_CUDA;
  }
  p.v = a.v;
  p.out = a.out;
  p.ldv = a.ldv;
  p.ldo = a.ldo;
  p.cu = a.cu;
  p.T = a.T;
  p.S = (int)a.S;
  p.Hq = (int)a.Hq;
  p.Hk = (int)a.Hk;
  p.G = (int)(a.Hq / a.Hk);
  p.D = (int)a.D;
  p.heads2 = p.G % 2 == 0;
  p.pairs = p.heads2 ? p.Hq / 2 : p.Hq;
  // (a scale of 0 becomes the smallest that keeps a masked -inf one)
  p.c = fmaxf(fabsf(a.scale) * 1.4426950408889634f, FLT_TRUE_MIN);
  p.negate = a.scale < 0.f;
  // runs of rows: at most one that is not full per sequence
  const int64_t rows = p.heads2 ? kPtTile : 2 * kPtTile;
  const int64_t blocks = ((a.T + rows - 1) / rows + a.S) * p.pairs;
  if (blocks > 0x7fffffff) {
    set_error_detail("prompt_attention: too many tokens for one launch");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  return a.D <= 64 ? pt_run<1>(p, (unsigned)blocks, a.stream) : pt_run<2>(p, (unsigned)blocks, a.stream);
}

int prompt_status(int* value, bool clear) {
  if (cudaMemcpyFromSymbol(value, g_prompt_status, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_prompt_status, &zero, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  }
  return Q4LIN_OK;
}

}  // namespace q4
