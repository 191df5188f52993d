// What a row of logits says: log probabilities of given tokens, the entropy, the top tokens.
//
// For a row x of V logits, M = max x, S = sum e^(x_v - M):
//     logp(v) = x_v - M - ln S,     entropy = ln S - (sum e^(x_v - M) (x_v - M)) / S,
// and the k largest x in order, ties by the lowest token.  FP32 sums; every thread's are taken about a
// reference of its own that moves only when a logit lies more than kSlack above it, and are brought to M at
// the end.  Both terms of the entropy are >= 0 about M; about a thread's own reference its second sum
// holds terms of both signs, up to kSlack / ln 2 times the first, so what is left of it at M is off by some
// kSlack 2^-23 of the terms above the reference.  With kSlack 8 that is 1e-6 where the entropy is not small,
// and nothing where one logit stands further out (then it is the reference); what rounding leaves below
// 0 is 0.  (With kSlack 40 rows certain to 1e-12 came out as up to 1e-6 of either sign.)
//
// Bound: the bytes of the logits, read once.  One pass: the exponentials, both sums, the
// maximum and the candidates of the top list come from the same registers.
//
// Split: a row belongs to a cluster of 1 .. 8 CTAs (as many as fill the GPU, with few rows), its
// 16-byte chunks dealt to the cluster's threads in turn; what lies before the first and behind
// the last whole chunk goes to the first CTA's and the last CTA's single threads.  Lists: lane i of every warp holds the warp's i-th; a vote per chunk of 32
// vectors decides whether any of its logits beats the last entry, which is rare after the
// first few: a bar made of all threads' maxima over their first batch stands before the lists.  Warps, then CTAs
// (distributed shared memory) are merged in order.
//
// Measured (captured calls): 1024 rows of 131072 bf16 logits 44.5 us, 6.0 TB/s (0.90 of the measured copy rate); 75
// rows of 50001 FP32 logits with the top 5 11.1 us and one row of 131072 with the top 8 8.6 us, which are
// the latencies of the loads, the lists and their merges (without the first batch's bar 36 and 29 us).  The
// lists show with many rows too: 128, 256, 512 rows of 131072 take 13.8, 14.8, 27.5 us, with the top 8
// 24.8, 26.3, 47.7.
#include <cfloat>
#include <type_traits>

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kLpMaxWarps = 16;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr float kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The two halves of cluster_sync.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

struct LpParams {
  const void* x;
  int64_t ld;               // row stride in elements
  const int32_t* tok;       // [T, n]
  float* logp;              // [T, n]
  float* entropy;           // [T] or NULL
  int32_t* ids;             // [T, k]
  float* top;               // [T, k]
  int64_t T;
  int V, n, k, cs;          // cs: CTAs per row
};

__device__ __forceinline__ float ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}

__device__ __forceinline__ float2 lp_fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// Sums about the reference m (in units of ln 2 for a): s = sum 2^t, a = sum 2^t t.
struct Sums {
  float m, s, a, top;   // top: the largest logit so far; -inf: none
};

// The sums of `o` brought to the reference m (o.m <= m up to rounding, or o empty).  About +inf they hold the
// number of infinite logits, and what is finite has nothing.
__device__ __forceinline__ void shift_to(float m, Sums& o) {
  if (o.s == 0.f) {
    o.a = 0.f;
  } else {
    const float t = o.m == m ? 0.f : (o.m - m) * kLog2e, f = ex2(t);
    o.a = f == 0.f && o.s == o.s ? 0.f : f * (o.a + o.s * t);
    o.s *= f;
  }
  o.m = m;
}

// The warp's list: lane i holds the i-th largest (value, token), i < k; unused entries are (-inf, -1).
// Equal values stand in the order of their tokens.
struct TopList {
  float v;
  int id;
};

__device__ __forceinline__ void list_insert(TopList& l, float x, int id, int k, int lane) {
  const int at = __popc(__ballot_sync(0xffffffffu, lane < k && (l.v > x || (l.v == x && l.id < id))));
  const float pv = __shfl_up_sync(0xffffffffu, l.v, 1);
  const int pi = __shfl_up_sync(0xffffffffu, l.id, 1);
  if (lane > at) {
    l.v = pv;
    l.id = pi;
  }
  if (lane == at) {
    l.v = x;
    l.id = id;
  }
}

// Floats above -inf as integers in their order, above 0 (-inf and NaN: 0).  Equal floats have equal keys: adding 0
// makes -0 a +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}

// Lane r gets the r-th largest of the lanes' keys (0 where there are no more above 0), r < k.
__device__ __forceinline__ uint32_t top_keys(uint32_t key, int k, int lane) {
  uint32_t mine = 0;
  for (int r = 0; r < k; ++r) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, key);
    if (top == 0) break;
    if (lane == r) mine = top;
    if (lane == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) key = 0;
  }
  return mine;
}

// The k-th largest of `lists` sorted lists of keys; 0: there are fewer above 0.
__device__ __forceinline__ uint32_t kth_of_lists(const uint32_t (*keys)[kMaxTop], int lists, int k, int lane) {
  int at = 0;
  uint32_t key = lane < lists ? keys[lane][0] : 0u, top = 0;
  for (int r = 0; r < k; ++r) {
    top = __reduce_max_sync(0xffffffffu, key);
    if (top == 0) break;
    if (lane == __ffs(__ballot_sync(0xffffffffu, key == top)) - 1) key = ++at < k ? keys[lane][at] : 0u;
  }
  return top;
}

// Merge of `lists` sorted lists of k entries into lane i's i-th of the result: every lane walks one list.
template <class Load>
__device__ __forceinline__ TopList merge_lists(int lists, int k, int lane, Load load) {
  int at = 0;
  float v = -INFINITY;
  int id = -1;
  if (lane < lists) load(lane, 0, v, id);
  TopList out{-INFINITY, -1};
  for (int r = 0; r < k; ++r) {
    const uint32_t key = order_key(v), top = __reduce_max_sync(0xffffffffu, key);
    if (top == 0) break;   // (uniform: nothing is left)
    const uint32_t first = __reduce_min_sync(0xffffffffu, key == top ? (uint32_t)id : 0xffffffffu);
    const bool mine = key == top && (uint32_t)id == first;
    const float win = __shfl_sync(0xffffffffu, v, __ffs(__ballot_sync(0xffffffffu, mine)) - 1);
    if (lane == r) out = TopList{win, (int)first};
    if (mine) {
      ++at;
      v = -INFINITY;
      id = -1;
      if (at < k) load(lane, at, v, id);
    }
  }
  return out;
}

template <bool kF32>
struct Vec;   // one 16-byte chunk as pairs of FP32 values
template <>
struct Vec<false> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(uint4 w, float2 (&x)[4]) {
    x[0] = make_float2(bf16lo(w.x), bf16hi(w.x));
    x[1] = make_float2(bf16lo(w.y), bf16hi(w.y));
    x[2] = make_float2(bf16lo(w.z), bf16hi(w.z));
    x[3] = make_float2(bf16lo(w.w), bf16hi(w.w));
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(static_cast<const uint16_t*>(p) + i));
    return __uint_as_float((uint32_t)v << 16);
  }
};
template <>
struct Vec<true> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(uint4 w, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    x[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
  static __device__ __forceinline__ float one(const void* p, int64_t i) {
    return __uint_as_float(ld_global_u32(static_cast<const uint32_t*>(p) + i));
  }
};

// Values of `np` pairs join the sums; `vm` is their largest.
template <int NP>
__device__ __forceinline__ void add_values(Sums& r, float& limit, const float2 (&x)[NP], float vm) {
  if (vm > limit) {   // (the first values at all, or far above the reference)
    shift_to(vm, r);
    limit = vm + kSlack;
    if (vm == INFINITY) {   // every +inf counts as 1, whatever is finite as 0
      limit = FLT_MAX;      // (the next one comes here too)
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float e[2] = {x[i].x, x[i].y};
#pragma unroll
        for (int j = 0; j < 2; ++j) r.s += e[j] == INFINITY ? 1.f : e[j] == e[j] ? 0.f : e[j];
      }
      r.top = vm;
      return;
    }
  }
  r.top = fmaxf(r.top, vm);
  const float2 neg = make_float2(-r.m, -r.m), c = make_float2(kLog2e, kLog2e);
  float2 s = make_float2(0.f, 0.f), a = s;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 t = lp_fmul2(fadd2(x[i], neg), c);
    const float2 e = make_float2(ex2(t.x), ex2(t.y));
    s = fadd2(s, e);
    // (a logit of -inf adds nothing: 0 times the bounded t)
    a = ffma2(e, make_float2(fmaxf(t.x, -1e4f), fmaxf(t.y, -1e4f)), a);
  }
  r.s += s.x + s.y;
  r.a += a.x + a.y;
}

struct LpShared {
  alignas(16) Sums sums[kLpMaxWarps];
  float lv[kLpMaxWarps][kMaxTop];
  int li[kLpMaxWarps][kMaxTop];
  alignas(16) Sums cta[kMaxCluster];     // (the cluster's first CTA) what its CTAs have sent
  float cv[kMaxCluster][kMaxTop];
  int ci[kMaxCluster][kMaxTop];
  float row[2];              // M, ln S
  uint32_t keys[kLpMaxWarps][kMaxTop];   // the warps' largest lane maxima of the first batch, in order
};

__device__ __forceinline__ Sums warp_join(Sums r) {
  float m = r.top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (m > -INFINITY) shift_to(m, r);
  // a fixed tree: the same bits every time
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
    r.a += __shfl_xor_sync(0xffffffffu, r.a, o);
  }
  r.m = r.top = m;
  return r;
}

template <bool kF32, bool kTop, int kLpThreads>
__global__ void __launch_bounds__(kLpThreads, 1024 / kLpThreads) q4_logprobs_kernel(const LpParams p) {
  using V = Vec<kF32>;
  constexpr int kLpWarps = kLpThreads / 32;
  constexpr int kBatch = 4;   // chunks added up together per thread, as many more on their way
  __shared__ LpShared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t row = blockIdx.x / (unsigned)p.cs;
  const int rank = (int)(blockIdx.x - (unsigned)row * (unsigned)p.cs);
  pdl_launch_dependents();
  if (p.cs > 1) cluster_arrive();   // (waited for before anything is sent)
  pdl_wait_previous();
  constexpr int64_t esize = kF32 ? 4 : 2;
  const char* x = static_cast<const char*>(p.x) + row * p.ld * esize;
  // whole 16-byte chunks lie between `head` and `head + chunks * V::n`
  const int head = min(p.V, (int)(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / esize));
  const int chunks = (p.V - head) / V::n;
  const char* body = x + head * esize;

  Sums r{0.f, 0.f, 0.f, -INFINITY};
  float limit = -INFINITY;
  TopList list{-INFINITY, -1};
  // What a value has to beat: the list's last entry once it is full, and a bar that k of the CTA's logits
  // reach (its equals still count, for their tokens).
  float last = -INFINITY, bar = -INFINITY;
  int last_id = -1;
  // every lane offers a value (uniform); those that pass go in, one after the other
  auto offer = [&](float v, int id) {
    auto passes = [&](float x, int i) { return x > -INFINITY && x >= bar && (x > last || (x == last && i < last_id)); };
    uint32_t some = __ballot_sync(0xffffffffu, passes(v, id));
    while (some) {
      const int from = __ffs(some) - 1;
      some &= some - 1;
      const float x = __shfl_sync(0xffffffffu, v, from);
      const int i = __shfl_sync(0xffffffffu, id, from);
      if (passes(x, i)) {   // (uniform)
        list_insert(list, x, i, p.k, lane);
        const float lv = __shfl_sync(0xffffffffu, list.v, p.k - 1);
        if (lv > -INFINITY) {   // the list is full
          last = lv;
          last_id = __shfl_sync(0xffffffffu, list.id, p.k - 1);
        }
      }
    }
  };
  // single logits, one per lane (first: warp 0 of the first CTA; last: the last warp of the last)
  auto singles = [&](int from, int count) {
    float v = -INFINITY;
    if (lane < count) v = V::one(x, from + lane);
    const float2 pair[1] = {make_float2(v, -INFINITY)};
    if (lane < count) add_values<1>(r, limit, pair, v);
    if constexpr (kTop) offer(v, from + lane);
  };
  if (rank == 0 && warp == 0 && head > 0) singles(0, head);

  const int step = p.cs * kLpThreads;
  // the next batch is on its way while this one is added up
  uint4 w[kBatch], ahead[kBatch];
  auto fetch = [&](int c0, uint4 (&v)[kBatch]) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int c = c0 + b * step + lane;
      if (c < chunks) v[b] = ld_global_u4(body + (int64_t)c * 16);
    }
  };
  int c0 = rank * kLpThreads + warp * 32;
  fetch(c0, w);
  if constexpr (kTop) {
    // The bar: the k-th largest of the threads' maxima over the first batch, which k values at least reach.
    // (Without it the first chunks would all go through the lists; from the warps' own maxima alone it
    // would let 16 times as many values pass for the rest of the row.)
    float most = -INFINITY;
#pragma unroll
    for (int b = 0; b < kBatch; ++b)
      if (c0 + b * step + lane < chunks) {
        float2 v[V::n / 2];
        V::unpack(w[b], v);
#pragma unroll
        for (int i = 0; i < V::n / 2; ++i) most = fmaxf(most, fmaxf(v[i].x, v[i].y));
      }
    const uint32_t mine = top_keys(order_key(most), p.k, lane);
    sh.keys[warp][lane] = mine;
    __syncthreads();
    const uint32_t key = kth_of_lists(sh.keys, kLpWarps, p.k, lane);
    if (key != 0) bar = __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
  }
  for (; c0 < chunks; c0 += kBatch * step) {
    fetch(c0 + kBatch * step, ahead);
    uint32_t some[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int c = c0 + b * step + lane;
      float2 v[V::n / 2];
      float vm = -INFINITY;
      if (c < chunks) {
        V::unpack(w[b], v);
        vm = fmaxf(v[0].x, v[0].y);
#pragma unroll
        for (int i = 1; i < V::n / 2; ++i) vm = fmaxf(vm, fmaxf(v[i].x, v[i].y));
        add_values<V::n / 2>(r, limit, v, vm);
      }
      if constexpr (kTop)
        some[b] = __ballot_sync(0xffffffffu, vm > -INFINITY && vm >= bar && (vm > last || (vm == last && head + c * V::n < last_id)));
    }
    if constexpr (kTop) {
      // Chunks with a value that may go in, one after the other: read again, a value per lane.  (One place in the
      // code for all of them: with the lists' code behind every value, unrolled, each use of it came from
      // outside the instruction cache, and 128 rows of 131072 took 32 us.)
      uint32_t any = 0;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) any |= some[b];
      if (any) {
#pragma unroll 1
        for (int b = 0; b < kBatch; ++b) {
          uint32_t left = b == 0 ? some[0] : b == 1 ? some[1] : b == 2 ? some[2] : some[3];
          while (left) {
            const int from = __ffs(left) - 1, id = head + (c0 + b * step + from) * V::n + lane;
            left &= left - 1;
            offer(lane < V::n ? V::one(x, id) : -INFINITY, id);
          }
        }
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) w[b] = ahead[b];
  }
  const int tail = head + chunks * V::n;
  if (rank == p.cs - 1 && warp == kLpWarps - 1 && tail < p.V) singles(tail, p.V - tail);

  r = warp_join(r);
  if (lane == 0) sh.sums[warp] = r;
  if (kTop) {
    sh.lv[warp][lane] = list.v;
    sh.li[warp][lane] = list.id;
  }
  __syncthreads();
  if (warp == 0) {
    Sums q = lane < kLpWarps ? sh.sums[lane] : Sums{0.f, 0.f, 0.f, -INFINITY};
    q = warp_join(q);
    if (kTop)
      list = merge_lists(kLpWarps, p.k, lane, [&](int l, int i, float& v, int& id) { v = sh.lv[l][i]; id = sh.li[l][i]; });
    r = q;
  }
  if (p.cs > 1) {
    cluster_wait();   // the cluster's first CTA is there
    if (warp == 0) {
      if (lane == 0)
        st_cluster_v4(mapa_shared(smem_u32(&sh.cta[rank]), 0), r.m, r.s, r.a, r.top);
      if (kTop) {
        st_cluster_u32(mapa_shared(smem_u32(&sh.cv[rank][lane]), 0), __float_as_uint(list.v));
        st_cluster_u32(mapa_shared(smem_u32(&sh.ci[rank][lane]), 0), (uint32_t)list.id);
      }
    }
    cluster_sync();
    if (rank != 0) return;
    if (warp == 0) {
      r = warp_join(lane < p.cs ? sh.cta[lane] : Sums{0.f, 0.f, 0.f, -INFINITY});
      if (kTop) list = merge_lists(p.cs, p.k, lane, [&](int l, int i, float& v, int& id) { v = sh.cv[l][i]; id = sh.ci[l][i]; });
    }
  }
  if (warp == 0) {
    // r.s NaN: a logit was NaN; none above -inf: no distribution
    const bool none = r.top == -INFINITY && r.s == r.s;
    const float ls = logf(r.s);
    if (lane == 0) {
      sh.row[0] = r.top;
      sh.row[1] = none ? INFINITY : ls;
      const float h = ls - r.a / r.s * kLn2;
      if (p.entropy != nullptr) p.entropy[row] = none || h < 0.f ? 0.f : h;
    }
    if (kTop && lane < p.k) {
      p.ids[row * p.k + lane] = list.id;
      p.top[row * p.k + lane] = list.id < 0 ? -INFINITY : (list.v == r.top ? 0.f : list.v - r.top) - ls;
    }
  }
  __syncthreads();
  for (int j = tid; j < p.n; j += kLpThreads) {
    const int v = (int)ld_global_u32(p.tok + row * p.n + j);
    float out = 0.f;   // no token: adds nothing to a sequence's sum
    if (v >= 0 && v < p.V) {
      const float xv = V::one(x, v);
      out = (xv == sh.row[0] ? 0.f : xv - sh.row[0]) - sh.row[1];   // (equal: both may be infinite)
    }
    p.logp[row * p.n + j] = out;
  }
}

template <bool kF32, bool kTop, int kLpThreads>
int lp_launch(const LpParams& p, unsigned blocks, cudaStream_t stream) {
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)p.cs;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
  cfg.blockDim = dim3(kLpThreads, 1, 1);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = p.cs > 1 ? 2 : 1;
  return cuda_check(cudaLaunchKernelEx(&cfg, q4_logprobs_kernel<kF32, kTop, kLpThreads>, p), "token_logprobs: kernel launch");
}

}  // namespace

int logprobs_launch(const LogprobArgs& a) {
  LpParams p{a.logits, a.ld, a.targets, a.logprobs, a.entropy, a.top_ids, a.top_logprobs, a.T, (int)a.V, (int)a.n, a.k, 1};
  // CTAs per row: as many as leave one per SM, each with two batches of chunks at least.  (Measured at one
  // shape: 75 rows of 50001 FP32 logits, top 5, 11.0 us with two, 13.0 with one, 14.6 with four.  It leaves 77
  // to 152 rows of any length one CTA each.)
  const int64_t chunks = a.V * (a.fp32 ? 4 : 2) / 16;
  while (p.cs < kMaxCluster && a.T * p.cs * 2 <= 152 && chunks >= (int64_t)p.cs * 2 * 512 * 2) p.cs *= 2;
  const int64_t blocks = a.T * p.cs;
  if (blocks > 0x7fffffff) {
    set_error_detail("token_logprobs: too many rows for one launch");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  auto go = [&](auto f32, auto top) {
    constexpr bool kF32 = decltype(f32)::value, kTop = decltype(top)::value;
    // many rows: four CTAs of 256 threads per SM, whose beginnings and ends overlap better (1024 rows of 131072
    // bf16 logits: 44.6 us, with two of 512 threads 46.4)
    return a.T > 304 ? lp_launch<kF32, kTop, 256>(p, (unsigned)blocks, a.stream)
                     : lp_launch<kF32, kTop, 512>(p, (unsigned)blocks, a.stream);
  };
  if (a.fp32) return a.k > 0 ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
  return a.k > 0 ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
}

}  // namespace q4
