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
// Split: a unit of work is two tiles of 128 query rows, A and B, that read the same keys: two
// heads of a group where there is an even number of them, else two runs of rows of a head.  One CTA per
// SM stays and takes further units off the launch as long as there are any, the costliest first.  Blocks
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
//   warp 2           reports that a block's operands are there.  Before, it looks blocks of V that hold
//                    keys some rows must not see over for values that are not finite (0 times
//                    infinity would reach those rows): they become zeros for the MMA, and the rows
//                    that see such a key add it at the end.
//   warp 3           finds the units, one ahead of the other roles.
//
// Measured (captured calls; in a long row of calls, under the power cap, the first takes 355 to 360 us): 8192
// tokens, 32 + 8 heads of 128: 330 us, 1665 TFLOP/s (0.86 of the measured bf16 rate); 16384
// tokens of seven prompts, 32 + 4 heads: 345 us; 2000 tokens of nine prompts, 28 + 4 heads of 96: 19.1 us;
// 133 tokens: 8.5 us.  With 8192 tokens, 32 + 8 heads of 96 take 310 us, of 64 270: softmax, P V and
// Q K^T of one tile follow one another, and the other tile's products are too short to hide that.
// In the middle of a long prompt (heads of 128) a block of both tiles takes 2600 to 2700 cycles, 2048 of them
// the MMAs' at their nominal rate: Q K^T reads both operands from shared memory, which at 128
// bytes a cycle is all it gives, and the copies write there too (105 cycles for one of these MMAs, 65
// to 75 for one of P V).  A unit costs some 5000 cycles beyond its blocks: its first scores and its
// last P V have nothing of their own beside them, only the neighbouring units'.
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
constexpr int kPtSoftRegs = 216, kPtOtherRegs = 72;
// the shares of three warpgroups come out of the registers at launch (168 a thread)
static_assert(2 * kPtSoftRegs + kPtOtherRegs <= 3 * 168, "register split");
constexpr uint32_t kPtBoxBytes = 64 * 2 * kPtTile;   // 64 columns of a tile
constexpr int kPtK = 2, kPtV = 3;     // stages of K and of V (all that shared memory holds for D = 128)
__device__ int g_prompt_status = 0;

struct PtParams {
  CUtensorMap mq, mk, mv;   // (D, heads, T, 1)
  const uint16_t *k, *v;
  uint16_t* out;
  int64_t ldk, ldv, ldo;
  const int32_t* cu;        // [S + 1]
  int64_t T;
  int S, Hq, Hk, G, D;
  int heads2;               // 1: the tiles are two heads, 0: two runs of rows
  int pairs;                // units per run of rows
  float c;                  // |scale| log2 e
  int negate;               // the scale is negative: Q enters negated
  int wide;                 // the output's rows of heads are 32-byte aligned
};

// Bounded wait with every lane polling and the warp voting: no branch on one lane, no shuffle, so a wait
// whose phase has completed already costs a query and a vote.
__device__ __forceinline__ bool warp_wait_vote(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
  }
  *abort_flag = 1;
  if ((threadIdx.x & 31) == 0) atomicExch(status, (int)Q4LIN_ERR_TIMEOUT);
  return false;
}

// Whether the phase has completed, without waiting; the warp's common answer.
__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// One lane of a converged warp, the same every time.  Code under it stays uniform to the compiler,
// where a test of the lane's number would make it a divergent branch.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

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

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {   // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
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

// Whether one of a row's D values is.  (Not inlined: it is hardly ever called, and its code changed the order of the
// kernel's own: 336 us for 329.)
__device__ __noinline__ bool pt_not_finite(const uint16_t* x, int D) {
  bool any = false;
  for (int d = 0; d < D; d += 8) any = any || not_finite(ld_global_u4(x + d));
  return any;
}

// A unit of work: rows [row0, row0 + len) are its sequence, tiles A and B start at rows q0, q1 of it and
// see n0, n1 blocks of keys; the query head of A (B's is the next, or the same).
struct PtUnit {
  int row0, len, q0, q1, head, n0, n1, there;   // there: 0 ends the CTA's work
};

// Units in the order of their cost: the last runs of all sequences first.  One warp; lane l holds the
// numbers of runs of sequences l, l + 32, .. .  With more sequences than kPtSorted the runs are taken
// sequence by sequence, the last run first (they are short then).
constexpr int kPtSorted = 256;
template <int kHeld>   // sequences held per lane: 1 (up to 32 of them) or 8
struct PtOrder {
  int n[kHeld], row0, len;   // (row0, len: of sequence l, with one per lane)
  int most, level;   // the highest number plus one; that of the last run found
  int64_t before;    // (not sorted) runs of the sequences before s
  int s;
  bool sorted;

  __device__ __forceinline__ void start(const PtParams& p, int rows, int lane) {
    sorted = p.S <= kPtSorted;
    before = 0;
    s = most = row0 = len = 0;
    if (!sorted) return;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      n[k] = 0;
      if (32 * k + lane < p.S) {
        int64_t a, b;
        pt_rows(p, 32 * k + lane, a, b);
        row0 = (int)a;
        len = (int)(b - a);
        n[k] = (int)(((unsigned)len + (unsigned)rows - 1u) / (unsigned)rows);
      }
      most = max(most, n[k]);
    }
    level = most = (int)__reduce_max_sync(0xffffffffu, (unsigned)most);
  }

  // Runs whose number is j or more.
  __device__ __forceinline__ int64_t runs_from(int j) const {
    unsigned c = 0;
#pragma unroll
    for (int k = 0; k < kHeld; ++k) c += (unsigned)max(0, n[k] - j);
    return (int64_t)__reduce_add_sync(0xffffffffu, c);   // (below T / rows + S)
  }

  // The index-th run: its sequence's first row and length, and its number; false: there are fewer.
  __device__ __forceinline__ bool find(const PtParams& p, int rows, int64_t index, int lane, int& first, int& length, int& run) {
    int seq = -1;
    if (!search(p, rows, index, lane, seq, run)) return false;
    if (kHeld == 1 && sorted) {
      first = __shfl_sync(0xffffffffu, row0, seq);
      length = __shfl_sync(0xffffffffu, len, seq);
    } else {
      int64_t a, b;
      pt_rows(p, seq, a, b);
      first = (int)a;
      length = (int)(b - a);
    }
    return true;
  }
  __device__ __forceinline__ bool search(const PtParams& p, int rows, int64_t index, int lane, int& seq, int& run) {
    if (sorted) {
      if (runs_from(0) <= index) return false;
      // the largest number whose runs and those above it are more than index: often the last one's
      int lo = 0, hi = most;
      if (runs_from(level) > index) lo = level;
      else hi = level;
      while (hi - lo > 1) {
        const int mid = lo == level && lo > 0 ? lo + 1 : (lo + hi) / 2;
        if (runs_from(mid) > index) lo = mid;
        else hi = mid;
      }
      level = lo;
      int rank = (int)(index - runs_from(lo + 1));
      run = lo;
      seq = -1;
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const unsigned has = __ballot_sync(0xffffffffu, n[k] > lo);
        if (seq < 0 && rank < __popc(has)) {
          const bool mine = (has >> lane & 1u) && __popc(has & ((1u << lane) - 1u)) == rank;
          seq = 32 * k + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        }
        rank -= __popc(has);
      }
      return true;
    }
    if (index < before) s = 0, before = 0;
    for (; s < p.S; s += 32) {
      int64_t a = 0, b = 0;
      if (s + lane < p.S) pt_rows(p, s + lane, a, b);
      const int runs = (int)((b - a + rows - 1) / rows);
      int64_t upto = runs;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (index < before + all) {
        const bool mine = index < before + upto && index >= before + upto - runs;
        const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        seq = s + from;
        run = __shfl_sync(0xffffffffu, (int)(before + upto - 1 - index), from);
        return true;
      }
      before += all;
    }
    return false;
  }
};

// Takes a CTA that has not started yet off the launch: its number, or none.  The answer (16 bytes) comes
// to shared memory with the barrier's completion.
__device__ __forceinline__ void pt_take(uint32_t answer, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(answer),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool pt_taken(uint32_t answer, uint32_t& block) {
  uint32_t ok, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b64 lo, hi;\n\t"
      "ld.shared.v2.b64 {lo, hi}, [%2];\n\t"
      "mov.b128 h, {lo, hi};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(answer)
      : "memory");
  block = x;
  return ok != 0;
}

__device__ __forceinline__ void pt_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int d, int h, int t) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(d), "r"(h), "r"(t), "r"(0)
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
  // barriers: units full, empty, time to take one; the launch's answer; Q full, empty; K full, empty; V full, empty; per
  // tile scores, P (with its operands), O; all MMAs done
  static constexpr uint32_t uf = bars, ue = uf + 16, go = ue + 16, tk = go + 8, qf = tk + 8, qe = qf + 8, kf = qe + 8, ke = kf + 8 * kPtK, vf = ke + 8 * kPtK,
                            ve = vf + 8 * kPtV, sf = ve + 8 * kPtV, pf = sf + 16, of = pf + 16, done = of + 16, end = done + 8;
  static constexpr uint32_t alloc = end + 1024;   // (the base is aligned to 1024)
};

// Tensor memory: scores and P of tile x, O of tile x.
__device__ __forceinline__ uint32_t pt_s_col(int x) { return 128u * (uint32_t)x; }
__device__ __forceinline__ uint32_t pt_o_col(int x) { return 256u + 128u * (uint32_t)x; }

constexpr int kPtReaders = 11;   // warps that read a unit: MMAs, copies, operands, eight of softmax

template <int DB>
__global__ void __launch_bounds__(kPtThreads, 1) q4_prompt_kernel(const __grid_constant__ PtParams p) {
  using SM = PtSmem<DB>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) uint8_t answer[16];
  __shared__ PtUnit units[2];
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  __shared__ volatile int odd_flag;   // V has held a value that is not finite
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  pdl_launch_dependents();
  if (tid == 0) {
    abort_flag = 0;
    odd_flag = 0;
    mbar_init(base + SM::go, 1);
    mbar_init(base + SM::tk, 1);
    mbar_init(base + SM::qf, 1);
    mbar_init(base + SM::qe, 1);
    for (int i = 0; i < kPtK; ++i) {
      mbar_init(base + SM::kf + 8 * i, 1);
      mbar_init(base + SM::ke + 8 * i, 1);
    }
    for (int i = 0; i < kPtV; ++i) {
      mbar_init(base + SM::vf + 8 * i, 1);
      mbar_init(base + SM::ve + 8 * i, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(base + SM::uf + 8 * x, 1);
      mbar_init(base + SM::ue + 8 * x, kPtReaders);
      mbar_init(base + SM::sf + 8 * x, 1);
      mbar_init(base + SM::pf + 8 * x, 5);   // four softmax warps, warp 2
      mbar_init(base + SM::of + 8 * x, 1);
    }
    mbar_init(base + SM::done, 1);
    fence_mbar_init();
    prefetch_tmap(&p.mq);
    prefetch_tmap(&p.mk);
    prefetch_tmap(&p.mv);
  }
  if (warp == 0) tmem_alloc(smem_u32(&tmem_base), 512);
  pdl_wait_previous();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (ok) ok = warp_wait_vote(bar, parity, &abort_flag, &g_prompt_status);
    return ok;
  };
  // The CTA's units come through two slots; number `u` of them.
  auto next_unit = [&](int u, PtUnit& w) {
    if (!wait(base + SM::uf + 8 * (u & 1), (uint32_t)(u >> 1) & 1u)) return false;
    w = units[u & 1];
    warp_release(base + SM::ue + 8 * (u & 1), lane);
    return w.there != 0;
  };
  PtUnit w;

  if (warp >= 4) {
    // ------------------------------------------------ softmax
    setmaxnreg_inc<kPtSoftRegs>();
    const int x = (warp >> 2) - 1;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + pt_s_col(x), to = tmem + lanes + pt_o_col(x);
    const float2 c2 = make_float2(p.c, p.c);
    uint32_t sph = 0, oph = 0;
    for (int u = 0; next_unit(u, w); ++u) {
      const int nx = x ? w.n1 : w.n0, qx = x ? w.q1 : w.q0;
      if (nx == 0) continue;
      const int row = qx + (warp & 3) * 32 + lane;
      float m = -INFINITY;
      float2 l = make_float2(0.f, 0.f);
      for (int i = 0; i < nx; ++i) {
        const int kb = nx - 1 - i;
        if (!wait(base + SM::sf + 8 * x, sph)) break;
        sph ^= 1u;
        tc_fence_after();
        uint32_t r[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j) tmem_ld32(ts + 32 * j, r[j]);
        tmem_ld_wait();
        if (kb * kPtTile + kPtTile - 1 > qx) {
          const int see = row - kb * kPtTile;   // keys 0 .. see of the block
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (bits, which become predicates several at a time)
            const int last = see - 32 * j;
            const uint32_t keep = last >= 31 ? 0xFFFFFFFFu : last < 0 ? 0u : (2u << last) - 1u;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(keep >> e & 1u)) r[j][e] = 0xFF800000u;
          }
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
          uint32_t pw[32];
#pragma unroll
          for (int e = 0; e < 64; e += 2) {
            const float2 t = ffma2(make_float2(__uint_as_float(r[j + (e >> 5)][e & 31]), __uint_as_float(r[j + (e >> 5)][(e & 31) + 1])), c2, m2);
            const float2 pr = make_float2(pt_ex2(t.x), pt_ex2(t.y));
            l = fadd2(l, pr);
            pw[e >> 1] = pt_pack(pr.x, pr.y);
          }
          tmem_st32(ts + 16 * j, pw);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_release(base + SM::pf + 8 * x, lane);
      }
      // ---------------------------------------------- the rows of O
      if (!wait(base + SM::of + 8 * x, oph)) break;
      oph ^= 1u;
      tc_fence_after();
      const float sum = l.x + l.y, inv = sum > 0.f ? 1.f / sum : __int_as_float(0x7FC00000);   // (no weight at all: NaN)
      const bool odd = odd_flag != 0;
      uint16_t* dst = p.out + ((int64_t)w.row0 + row) * p.ldo + (int64_t)(w.head + (p.heads2 ? x : 0)) * p.D;
#pragma unroll 1
      for (int j = 0; j < 2 * DB; ++j) {
        uint32_t o[32];
        tmem_ld32(to + 32 * j, o);
        tmem_ld_wait();
        if (odd && row < w.len)   // the keys left out of the products, for the rows that see them
          for (int key = w.q0 & ~(kPtTile - 1); key <= row; ++key) {
            const uint16_t* src = p.v + ((int64_t)w.row0 + key) * p.ldv + (int64_t)(w.head / p.G) * p.D + 32 * j;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              if (32 * j + 8 * b >= p.D) break;
              const uint4 v = ld_global_u4(src + 8 * b);
              if (!not_finite(v)) continue;
              // (a score that is not finite is -inf, or the row is NaN in any case: weight 0 times this value)
              const bool none = pt_not_finite(p.k + ((int64_t)w.row0 + key) * p.ldk + (int64_t)(w.head / p.G) * p.D, p.D);
              const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float val = e & 1 ? bf16hi(vs[e >> 1]) : bf16lo(vs[e >> 1]);
                if (!(fabsf(val) <= FLT_MAX))
                  o[8 * b + e] = none ? 0x7FC00000u : __float_as_uint(__uint_as_float(o[8 * b + e]) + val);
              }
            }
          }
        uint32_t ow[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) ow[e] = pt_pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
        if (row < w.len) {
          // (a lane's store is a line of its own, whatever its width: the wider the fewer)
          if (p.wide) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
              if (32 * j + 16 * b < p.D) st_global_32(dst + 32 * j + 16 * b, &ow[8 * b]);
          } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (32 * j + 8 * b < p.D)
                *reinterpret_cast<uint4*>(dst + 32 * j + 8 * b) = make_uint4(ow[4 * b], ow[4 * b + 1], ow[4 * b + 2], ow[4 * b + 3]);
          }
        }
      }
      tc_fence_before();   // (ahead of the arrival that lets the next unit's P V overwrite O)
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
      const uint32_t pf = base + SM::pf, sf = base + SM::sf;
      uint32_t vs = 0, ks = 0, kph = 0, ph0 = 0, ph1 = 0;   // stages of V's and K's next blocks; phases
      auto next_k = [&]() {
        if (++ks == kPtK) {
          ks = 0;
          kph ^= 1u;
        }
      };
      // Q K^T of the first block of unit w (from there on the units' products follow one another without a
      // break: the scores' columns are free as soon as the last unit's P V have been issued)
      auto first = [&](int x) {
        if ((x ? w.n1 : w.n0) == max(w.n0, w.n1)) {
          scores(Lo{}, Hi{}, x, ks);
          commit(sf + 8 * x);
        }
      };
      auto first_done = [&]() {
        commit(base + SM::ke + 8 * ks);
        if (max(w.n0, w.n1) == 1) commit(base + SM::qe);
        next_k();
      };
      bool have = next_unit(0, w) && wait(base + SM::qf, 0) && wait(base + SM::kf + 8 * ks, kph);
      if (have) {
        first(0);
        first(1);
        first_done();
      }
      // The barrier of a tile's P stands for V of the block and K of the next one too (warp 2 waits for
      // those).  It is looked up once in the middle of the other tile's Q K^T: a wait's own latency (some
      // 300 cycles beside two softmax warps) then lies behind work in the queue.
      bool there = false;
      for (int u = 0; have && ok; ++u) {
        const int n = max(w.n0, w.n1);
        // block i of the loop is keys (n - 1 - i) * 128 on; tile x takes part from its own last block on
        const int from0 = n - w.n0, from1 = w.n1 > 0 ? n - w.n1 : n;
        // (A begins with the second block: it has had no P yet, so no word of that block's K either)
        if (from0 > 0 && !wait(base + SM::kf + 8 * ks, kph)) break;
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n;
          if (i == max(0, n - 4)) commit(base + SM::go);
          if (i >= from0) {
            if (!there && !wait(pf, ph0)) break;
            ph0 ^= 1u;
            tc_fence_after();
            values(0, vs, i > from0);
            if (!more) commit(base + SM::of);
          }
          const bool s0 = more && i + 1 >= from0, s1 = more && i + 1 >= from1;
          // the next unit's operands, if they are there already, else behind this unit's last product
          bool early = false, read = false;
          if (!more && warp_test(base + SM::uf + 8 * ((u + 1) & 1), (uint32_t)((u + 1) >> 1) & 1u)) {
            have = next_unit(u + 1, w);
            read = true;
            early = true;
            if (have && warp_test(base + SM::qf, (uint32_t)(u + 1) & 1u) && warp_test(base + SM::kf + 8 * ks, kph)) first(0);
            else if (have) early = false;
          }
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
          there = false;
          if (more) {
            if (s1) scores(Lo{}, Mid{}, 1, ks);
            there = s0 && warp_test(pf, ph0);
            if (s1) {
              scores(Mid{}, Hi{}, 1, ks);
              commit(sf + 8);
            }
            commit(base + SM::ke + 8 * ks);
            if (i + 2 == n) commit(base + SM::qe);
            next_k();
          } else {
            if (!early) {
              if (!read) have = next_unit(u + 1, w);
              if (have && wait(base + SM::qf, (uint32_t)(u + 1) & 1u) && wait(base + SM::kf + 8 * ks, kph)) first(0);
            }
            if (have && ok) {
              first(1);
              first_done();
            }
          }
        }
      }
      // nothing is in flight behind this
      commit(base + SM::done);
      if (one) mbar_drain(base + SM::done, 0);
    } else if (warp == 1) {
      // ---------------------------------------------- copies
      const bool one = elect_one();
      int kc = 0, vc = 0, qc = 0;   // blocks of K and V, and Qs, so far
      auto load = [&](const CUtensorMap* map, uint32_t tiles, uint32_t full, uint32_t empty, int stages, int& count, int t) {
        const int st = count % stages;
        if (count >= stages && !wait(empty + 8 * st, ((uint32_t)(count / stages) & 1u) ^ 1u)) return false;
        if (one) {
          mbar_expect_tx(full + 8 * st, SM::tile);
          for (int b = 0; b < DB; ++b)
            pt_load(tiles + (uint32_t)st * SM::tile + b * kPtBoxBytes, map, full + 8 * st, 64 * b, w.head / p.G, t);
        }
        ++count;
        return true;
      };
      // a stage is free once its last use has completed; K of block i + 1 is wanted before V of block i
      for (int u = 0; next_unit(u, w); ++u) {
        const int n = max(w.n0, w.n1), tiles = w.n1 > 0 ? 2 : 1;
        auto key = [&](int i) { return w.row0 + (n - 1 - i) * kPtTile; };
        if (!load(&p.mk, base + SM::k, base + SM::kf, base + SM::ke, kPtK, kc, key(0))) break;
        if (u > 0 && !wait(base + SM::qe, (uint32_t)(u - 1) & 1u)) break;
        if (one) {
          mbar_expect_tx(base + SM::qf, tiles * SM::tile);
          for (int x = 0; x < tiles; ++x)
            for (int b = 0; b < DB; ++b)
              pt_load(base + SM::q + (uint32_t)x * SM::tile + b * kPtBoxBytes, &p.mq, base + SM::qf, 64 * b,
                      w.head + (p.heads2 ? x : 0), w.row0 + (x ? w.q1 : w.q0));
        }
        qc = u + 1;
        for (int i = 0; i < n && ok; ++i) {
          if (i + 1 < n && !load(&p.mk, base + SM::k, base + SM::kf, base + SM::ke, kPtK, kc, key(i + 1))) break;
          if (!load(&p.mv, base + SM::v, base + SM::vf, base + SM::ve, kPtV, vc, key(i))) break;
        }
      }
      // the CTA does not end before its copies have landed
      if (one) {
        if (qc > 0) mbar_drain(base + SM::qf, (uint32_t)(qc - 1) & 1u);
        for (int i = max(0, kc - kPtK); i < kc; ++i) mbar_drain(base + SM::kf + 8 * (i % kPtK), (uint32_t)(i / kPtK) & 1u);
        for (int i = max(0, vc - kPtV); i < vc; ++i) mbar_drain(base + SM::vf + 8 * (i % kPtV), (uint32_t)(i / kPtV) & 1u);
      }
    } else if (warp == 2) {
      // ---------------------------------------------- V at the edge, and word that a block's operands are there
      int kc = 0, vc = 0, arrived[2] = {0, 0};
      for (int u = 0; next_unit(u, w); ++u) {
        const int n = max(w.n0, w.n1), edge = w.q0 / kPtTile;   // blocks from here on hold keys that some row does not see
        const int from[2] = {n - w.n0, w.n1 > 0 ? n - w.n1 : n};
        ++kc;   // (K of the first block: the MMAs' own wait)
        for (int i = 0; i < n; ++i, ++vc) {
          if (!wait(base + SM::vf + 8 * (vc % kPtV), (uint32_t)(vc / kPtV) & 1u)) break;
          if (n - 1 - i >= edge) {
            const uint32_t at = base + SM::v + (uint32_t)(vc % kPtV) * SM::tile;
            uint32_t top = 0;   // the largest magnitude's bits; 0x7F80 and above: not finite
#pragma unroll 8
            for (uint32_t o = (uint32_t)lane * 16; o < SM::tile; o += 32 * 16) {
              const uint4 v = ld_shared_v4(at + o);
              top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                           __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
            }
            if (max(top & 0xFFFFu, top >> 16) >= 0x7F80u) {
              for (uint32_t o = (uint32_t)lane * 16; o < SM::tile; o += 32 * 16) {
                const uint4 v = ld_shared_v4(at + o);
                if (not_finite(v)) st_shared_v4(at + o, finite_only(v));
              }
              odd_flag = 1;
            }
            fence_proxy_async();
          }
          if (i + 1 < n) {
            if (!wait(base + SM::kf + 8 * (kc % kPtK), (uint32_t)(kc / kPtK) & 1u)) break;
            ++kc;
          }
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (i >= from[x]) {
              // (an arrival before the last phase is complete would count for that one)
              if (arrived[x] > 0 && !wait(base + SM::pf + 8 * x, (uint32_t)(arrived[x] - 1) & 1u)) break;
              warp_release(base + SM::pf + 8 * x, lane);
              ++arrived[x];
            }
        }
      }
    } else {
      // ---------------------------------------------- units
      // A unit is a run of rows and a head (pair); the CTA begins with its own number and takes those
      // of CTAs that have not started, so that long and short runs even out.
      const int rows = p.heads2 ? kPtTile : 2 * kPtTile;
      auto hand_out = [&](auto order) {
        order.start(p, rows, lane);
        uint32_t block = blockIdx.x;
        bool found = true;
        int taken = 0;
        for (int u = 0;; ++u) {
          int first = 0, length = 0, run = 0;
          if (found) {
            const uint32_t at = block / (uint32_t)p.pairs, unit = block - at * (uint32_t)p.pairs;
            found = order.find(p, rows, at, lane, first, length, run);
            if (u >= 2 && !wait(base + SM::ue + 8 * (u & 1), ((uint32_t)(u >> 1) & 1u) ^ 1u)) break;
            if (lane == 0) {
              PtUnit v{};
              if (found) {
                v.row0 = first;
                v.len = length;
                v.q0 = run * rows;
                v.q1 = v.q0 + (p.heads2 ? 0 : kPtTile);
                v.head = (int)unit * (p.heads2 ? 2 : 1);
                v.n0 = (min(v.len, v.q0 + kPtTile) + kPtTile - 1) / kPtTile;
                v.n1 = v.q1 < v.len ? (min(v.len, v.q1 + kPtTile) + kPtTile - 1) / kPtTile : 0;
                v.there = 1;
              }
              units[u & 1] = v;
            }
            warp_release(base + SM::uf + 8 * (u & 1), lane);
          }
          // (the next unit is taken when this one is nearly done: what has been taken early cannot be
          // evened out any more)
          if (found && !wait(base + SM::go, (uint32_t)u & 1u)) break;
          // (behind the last unit there may be CTAs of the launch that have nothing to do: they are taken
          // off too, which costs less than their start)
          if (lane == 0) {
            fence_proxy_async();   // (the last answer has been read)
            mbar_expect_tx(base + SM::tk, 16);
            pt_take(smem_u32(answer), base + SM::tk);
          }
          __syncwarp();
          if (!wait(base + SM::tk, (uint32_t)taken & 1u)) {
            if (lane == 0) mbar_drain(base + SM::tk, (uint32_t)taken & 1u);
            break;
          }
          ++taken;
          const bool more = pt_taken(smem_u32(answer), block);
          __syncwarp();
          if (!more) {   // the end, unless the units have ended before
            if (found) {
              ++u;
              if (u >= 2 && !wait(base + SM::ue + 8 * (u & 1), ((uint32_t)(u >> 1) & 1u) ^ 1u)) break;
              if (lane == 0) units[u & 1] = PtUnit{};
              warp_release(base + SM::uf + 8 * (u & 1), lane);
            }
            break;
          }
        }
      };
      if (p.S <= 32) hand_out(PtOrder<1>{});
      else hand_out(PtOrder<kPtSorted / 32>{});
    }
    __syncwarp();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// Rows of heads as a tensor (D, heads, T, 1) of boxes of 64 columns of a head and 128 rows.
bool pt_map(CUtensorMap* m, const void* base, int64_t D, int64_t heads, int64_t T, int64_t ld) {
  const uint64_t row = (uint64_t)ld * 2;
  return encode_map_4d(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, {(uint64_t)D, (uint64_t)heads, (uint64_t)T, 1},
                       {(uint64_t)D * 2, row, row}, {64, 1, kPtTile, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
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
  p.k = a.k;
  p.v = a.v;
  p.out = a.out;
  p.ldk = a.ldk;
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
  p.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && a.ldo % 16 == 0 && a.D % 16 == 0;
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
