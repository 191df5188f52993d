// A paged cache of keys and values in 4 bits: writing tokens, reading them back, and the
// attention of new tokens over it.
//
// A value is (q - 8) s, the layer's own Q4_G64 format: per token, head and 64 values one fp16
// scale s = fp16(max |x| / 7), q = rint(x / s) + 8 in [0, 15].  A page holds 64 tokens; the record
// of a page and head is contiguous (K codes, V codes, K scales, V scales), so that one bulk copy
// fetches it, and its codes lie as the tensor cores' A fragments want them:
//   K  [64 tokens][D / 2 bytes], 32-bit words of 8 values (block b), word c (D/32) + j = block
//      4 j + c: thread c of a quad reads its D/32 words of a token in one load, word j of all four
//      threads lies in scale group j / 2;
//   V  [D / 2 rows][64 bytes], row i values 2i (low nibble) and 2i + 1 of every token, token o at
//      byte 16 c + 4 j + 2 e + h (j = o / 16, h = o % 16 / 8, c = o % 8 / 2, e = o % 2): word j of
//      thread c holds its four tokens of k-step j, two values each.
//
// Measured (captured calls): 8192 tokens in and out, 8 heads of 128: 26.3 us (85 MB; bound by issue and by the
// chain of position, page and row of each tile of tokens); attention of 64 sequences of up to 8192
// tokens, 32 + 8 heads of 128: 42.7 us, 4.3 TB/s of codes and scales, with four new tokens each (16 columns)
// 75; five sequences of up to 70001 tokens, four new tokens each, 28 + 4 heads of 64, 96, 128: 44, 59,
// 72 us; one sequence of 1000 tokens: 7.4 us.
#include <type_traits>

#include "q4_internal.h"
#include "q4_sm100.cuh"

namespace q4 {

namespace {

constexpr int kPage = 64;
__device__ int g_kv_status = 0;

__host__ __device__ constexpr int kv_groups(int D) { return (D + 63) / 64; }
__host__ __device__ constexpr int kv_record(int D) { return kPage * D + 4 * kPage * kv_groups(D); }

// Byte of token o in a row of V codes.
__device__ __forceinline__ int v_place(int o) { return 16 * ((o & 7) >> 1) + 4 * (o >> 4) + 2 * (o & 1) + ((o & 15) >> 3); }

__device__ __forceinline__ float2 kv_fmul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<uint64_t*>(&a)), "l"(*reinterpret_cast<uint64_t*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}

// ------------------------------------------------------------------ tokens in and out
struct KvTokParams {
  const uint16_t* src[2];   // k, v rows (append)
  uint16_t* dst[2];         // k, v rows (read)
  int64_t ld[2];
  uint8_t* cache;
  const int32_t* table;     // [S, M]
  const int32_t* rows;      // [T] or NULL: token t is of sequence t
  const int32_t* pos;       // [T]
  int64_t T, S, M, P;
  int Hk, D;
};

// The record and place of token t; false: it has none (padding).
__device__ __forceinline__ bool kv_slot(const KvTokParams& p, int64_t t, int64_t& page, int& o) {
  const int64_t s = p.rows != nullptr ? (int64_t)(int32_t)ld_global_u32(p.rows + t) : t;
  const int64_t at = (int32_t)ld_global_u32(p.pos + t);
  if (s < 0 || s >= p.S || at < 0 || at >= p.M * kPage) return false;
  page = (int32_t)ld_global_u32(p.table + s * p.M + at / kPage);
  o = (int)(at % kPage);
  return page >= 0 && page < p.P;
}

constexpr int kTokThreads = 256;
constexpr int kTokTile = 64;   // tokens of a CTA

// A CTA takes 64 tokens' keys or values of one head; LPR lanes (8 values each) share a row.  V
// codes cross shared memory between token order (a lane has 8 values of a token) and the
// record's order (a lane has a token's byte of a row), so that tokens of a page are written and
// read a row at a time.
struct KvTile {
  int64_t rec[kTokTile];    // byte of the token's record in the cache; < 0: the token has no place
  int place[kTokTile];
};

__device__ __forceinline__ void kv_places(const KvTokParams& p, KvTile& tile, int64_t t0, int h) {
  if (threadIdx.x < kTokTile) {
    int64_t page = -1;
    int o = 0;
    const int64_t t = t0 + threadIdx.x;
    const bool there = t < p.T && kv_slot(p, t, page, o);
    tile.rec[threadIdx.x] = there ? (page * p.Hk + h) * (int64_t)kv_record(p.D) : -1;
    tile.place[threadIdx.x] = o;
  }
}

// Codes (low nibble first) and scale of a lane's eight bf16 values x; top: the bits of the group's largest
// magnitude.  q = rint(x / s) comes from a fixed-point sum with 16 bits behind the point, x (65536 / s) +
// 65536 (8 + 1/2) + 1 (off by less than 0.7 of its last place): its upper half's low nibble is the
// code, unless the lower half is 0, 1 or 2 for one of the values, which then may lie at a half (one value
// in 600 does so exactly).  Those lanes compare x with h s, h the half next to x / s: a product of 5 by
// 11 bits, so that one FMA gives the exact difference's sign.  s = fp16(top / 7) by a product: top / 7
// keeps 2^-15 away from the midpoints of normal fp16 numbers.
__device__ __forceinline__ uint32_t kv_codes(const uint32_t (&x)[4], uint32_t top, uint16_t& scale) {
  scale = 0x7E00u;   // NaN: a group with a value that is not finite reads as NaN
  if (top >= 0x7F80u) return 0x88888888u;
  const float tf = __uint_as_float(top << 16);
  const bool plain = tf >= 0.0005f && tf <= 458000.f;   // (s a normal number, and not cut off)
  const __half s = __float2half_rn(plain ? tf * 0.14285714924335479736f : fminf(__fdiv_rn(tf, 7.f), 65504.f));
  const float sf = __half2float(s), inv = __fdividef(1.f, sf);
  scale = __half_as_ushort(s);
  if (plain) {
    constexpr float base = 12582912.f + 557057.f;   // 1.5 * 2^23: the sum's mantissa counts whole units
    const float up = inv * 65536.f;
    uint32_t n[8], low = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[2 * i] = __float_as_uint(fmaf(bf16lo(x[i]), up, base));
      n[2 * i + 1] = __float_as_uint(fmaf(bf16hi(x[i]), up, base));
      low = __vminu2(low, __byte_perm(n[2 * i], n[2 * i + 1], 0x5410));
    }
    if (min(low & 0xFFFFu, low >> 16) > 2u) {
      auto thirds = [](uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // the third bytes side by side
        return __byte_perm(__byte_perm(a, b, 0x0062), __byte_perm(c, d, 0x0062), 0x5410);
      };
      return (thirds(n[0], n[2], n[4], n[6]) & 0x0F0F0F0Fu) | (thirds(n[1], n[3], n[5], n[7]) << 4 & 0xF0F0F0F0u);
    }
  } else if (sf == 0.f) {
    return 0x88888888u;
  }
  constexpr float magic = 12582912.f;   // adding and taking it off rounds to integers, halves to even
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = i & 1 ? bf16hi(x[i >> 1]) : bf16lo(x[i >> 1]);
    const float h = (fminf(fmaxf(v * inv, -9.f), 8.f) - 0.5f + magic) - magic + 0.5f, r = fmaf(-h, sf, v);
    const float q = r == 0.f ? (h + magic) - magic : r > 0.f ? h + 0.5f : h - 0.5f;
    code |= (__float_as_uint(fminf(fmaxf(q, -8.f), 7.f) + (magic + 8.f)) & 15u) << (4 * i);
  }
  return code;
}

template <int LPR>
__global__ void __launch_bounds__(kTokThreads) q4_kv_append_kernel(const KvTokParams p) {
  constexpr int kRows = kTokThreads / LPR, kPasses = kTokTile / kRows;
  __shared__ KvTile tile;
  __shared__ uint32_t words[kTokTile][17];
  const int tid = threadIdx.x, b = tid % LPR;
  const int side = (int)blockIdx.y >= p.Hk ? 1 : 0, h = (int)blockIdx.y - side * p.Hk;
  const int64_t t0 = (int64_t)blockIdx.x * kTokTile;
  pdl_launch_dependents();
  pdl_wait_previous();
  const bool in = 8 * b < p.D;
  const int64_t ld = side ? p.ld[1] : p.ld[0];
  const uint16_t* src = (side ? p.src[1] : p.src[0]) + (t0 + tid / LPR) * ld + h * p.D + 8 * b;
  const int left = (int)min((int64_t)kTokTile, p.T - t0);
  uint4 w[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i, src += kRows * ld) {
    w[i] = make_uint4(0u, 0u, 0u, 0u);
    if (in && i * kRows + tid / LPR < left) w[i] = ld_global_u4(src);
  }
  kv_places(p, tile, t0, h);
  __syncthreads();
  const int G = kv_groups(p.D), word = ((b & 3) * (p.D / 32) + (b >> 2)) * 4;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + tid / LPR;
    const uint32_t xs[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
    uint32_t top = 0;   // magnitudes of bf16 compare as their bits; above 0x7F7F: not finite
#pragma unroll
    for (int e = 0; e < 4; ++e) top = __vmaxu2(top, xs[e] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    uint16_t scale;
    const uint32_t code = kv_codes(xs, top, scale);
    if (side == 1 && in) words[r][b] = code;
    const int64_t at = tile.rec[r];
    if (at < 0 || !in) continue;
    uint8_t* rec = p.cache + at;
    const int o = tile.place[r];
    if (side == 0) *reinterpret_cast<uint32_t*>(rec + o * (p.D / 2) + word) = code;
    if ((b & 7) == 0) reinterpret_cast<uint16_t*>(rec + 64 * p.D)[side * kPage * G + o * G + (b >> 3)] = scale;
  }
  if (side == 0) return;
  __syncthreads();
  const int r = tid % kTokTile;
  const int64_t at = tile.rec[r];
  if (at < 0) return;
  uint8_t* rec = p.cache + at + 32 * p.D + v_place(tile.place[r]);
  for (int b0 = tid / kTokTile; b0 < p.D / 8; b0 += kTokThreads / kTokTile) {
    const uint32_t code = words[r][b0];
#pragma unroll
    for (int i = 0; i < 4; ++i) rec[(4 * b0 + i) * kPage] = (uint8_t)(code >> (8 * i));
  }
}

template <int LPR>
__global__ void __launch_bounds__(kTokThreads) q4_kv_read_kernel(const KvTokParams p) {
  constexpr int kRows = kTokThreads / LPR, kPasses = kTokTile / kRows;
  __shared__ KvTile tile;
  __shared__ uint32_t words[kTokTile][17];
  const int tid = threadIdx.x, b = tid % LPR;
  const int side = (int)blockIdx.y >= p.Hk ? 1 : 0, h = (int)blockIdx.y - side * p.Hk;
  const int64_t t0 = (int64_t)blockIdx.x * kTokTile;
  pdl_launch_dependents();
  pdl_wait_previous();
  kv_places(p, tile, t0, h);
  __syncthreads();
  if (side == 1) {
    const int r = tid % kTokTile;
    const int64_t at = tile.rec[r];
    if (at >= 0) {
      const volatile uint8_t* rec = p.cache + at + 32 * p.D + v_place(tile.place[r]);
#pragma unroll 4
      for (int b0 = tid / kTokTile; b0 < p.D / 8; b0 += kTokThreads / kTokTile) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = rec[(4 * b0 + i) * kPage];
        words[r][b0] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
      }
    }
    __syncthreads();
  }
  if (8 * b >= p.D) return;
  const int G = kv_groups(p.D);
  const int64_t ld = side ? p.ld[1] : p.ld[0];
  uint16_t* dst = (side ? p.dst[1] : p.dst[0]) + (t0 + tid / LPR) * ld + h * p.D + 8 * b;
  const int word = ((b & 3) * (p.D / 32) + (b >> 2)) * 4;
  uint32_t codes[kPasses];
  uint16_t scales[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + tid / LPR;
    const int64_t at = tile.rec[r];
    if (at < 0) continue;
    const uint8_t* rec = p.cache + at;
    const int o = tile.place[r];
    codes[i] = side ? words[r][b] : ld_global_u32(rec + o * (p.D / 2) + word);
    scales[i] = reinterpret_cast<const volatile uint16_t*>(rec + 64 * p.D)[side * kPage * G + o * G + (b >> 3)];
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i, dst += kRows * ld) {
    if (tile.rec[i * kRows + tid / LPR] < 0) continue;
    const uint32_t code = codes[i];
    const float s = fp16_bits_to_float(scales[i]);
    // the nibbles as FP32 128 + q, then (q - 8) s
    const uint32_t even = code & 0x0F0F0F0Fu, odd = (code >> 4) & 0x0F0F0F0Fu;
    const float2 zero = make_float2(-136.f, -136.f), s2 = make_float2(s, s);
    auto pair = [&](float lo, float hi) {
      const float2 v = kv_fmul2(fadd2(make_float2(lo, hi), zero), s2);
      const __nv_bfloat162 h2 = __floats2bfloat162_rn(v.x, v.y);
      return *reinterpret_cast<const uint32_t*>(&h2);
    };
    const uint32_t out[4] = {pair(f128_plus_byte<0>(even), f128_plus_byte<0>(odd)), pair(f128_plus_byte<1>(even), f128_plus_byte<1>(odd)),
                             pair(f128_plus_byte<2>(even), f128_plus_byte<2>(odd)), pair(f128_plus_byte<3>(even), f128_plus_byte<3>(odd))};
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

template <class Kernel>
int pdl_launch(Kernel kernel, const char* what, dim3 blocks, unsigned threads, size_t smem, cudaStream_t stream, const void* params) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  void* args[1] = {const_cast<void*>(params)};
  return cuda_check(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), args), what);
}

// ------------------------------------------------------------------ attention over the cache
//
// For query column (token i, head) of a sequence of L tokens, over its tokens j < L - n + 1 + i:
//     x_j = scale q . k_j,   y = sum 2^(x_j log2 e - m) v_j / sum 2^(x_j log2 e - m).
// Scores S^T = K q^T on the warp MMAs, 16 tokens x 8 columns: codes become exact fp16 subnormals
// by one AND per pair (q 2^-24; the odd nibbles 16 q 2^-24 meet q / 16), the query enters as fp16
// at a power of two per column that puts its largest value in [2^14, 2^15) (exact down to 2^-28 of
// that), every scale group sums in FP32 and is scaled there:
//     x = sum_g s_g (F D_g + Z_g),  F = 2^24 2^e scale log2 e,  Z_g = -8 2^-24 F sum (x 2^-e).
// Values O^T = V^T P^T likewise, with P_j s_j (per scale group) as the fp16 operand: its rounding,
// 2^-12 of each weight, is an eighth of the output's own.  The reference m of a column absorbs
// the scales' size (m >= max x log2 e + log2 of the page's largest V scale - 14), so that P s
// stays below 2^15 whatever the scales are; what lies 2^28 and more below a page's largest weight times its
// largest scale is a subnormal fp16, off by up to 2^-38 of that product.  The zero points' share,
// 8 sum P s, comes from one more MMA against a fragment of eights.  A subnormal operand is aligned by its
// exponent, not by its leading bit: of the 16 tokens of an MMA, products below 2^-15 of the largest P s
// (odd values 2^-19) are cut off, at most 17 2^-15 of it in all.  That is as much as the
// output's own rounding where that token's value is of its scale's size, and matters only to what stands beside a value
// of 0.  Codes shifted up by 6 bits in their halves would leave 2^-21, for three more shifts a word (64 sequences
// 43.3 us for 42.6, five long ones 60.3 for 58.7).
// (Scores do not show it: neighbours 0.01 apart at 2400 are off by 4e-4, FP32's last place there being 2e-4.)
//
// Bound: the bytes of the codes and scales, read once per 32 columns.  Up to 8 columns the decode's issue is
// close behind (integer pipe 40 %, 1.5 instructions a cycle); with more, the MMAs and the decode of
// two warps per scheduler, all that two tiles' states in registers leave room for (tensor pipe 33 %; with heads of
// 96 ten or twelve warps spill: 74 and 67 us where eight took 61 on the five long sequences).  Heads of
// 128 do not fit with eight warps either: 156 to 172 bytes a thread are spilled, some of them in the
// loop over pages.
//
// Split: the pages of all sequences and heads in a row are cut into equal shares, whatever the
// lengths are.  A share belongs to one warp of a CTA (one CTA per SM) with a ring of record copies and
// a running (m, sum, O) of its own, 8 or 16 columns wide; for 17 to 32 columns to a group of two
// warps that take the same pages.  No barrier joins the groups.  A (sequence, head) inside one share is
// finished there, others leave FP32 partial sums (at most two per share) that a second kernel
// joins in order.  (With a CTA's warps joined by barriers at the end of every segment the 64 sequences
// took 115 us; with a warp per 8 columns, each decoding a page again, the five long ones 132.)
struct KvParams {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* len;
  float* part;              // [shares][2][tiles][part_floats]
  int64_t P;
  int S, M, n, G, Hk, cols, passes;   // columns of a head (n * G) and passes over them
  float c;                  // scale * log2 e
};

constexpr int kKvRecords = 24;    // records in shared memory, over all rings

// A warp takes NT tiles of 8 columns (its codes are decoded once for all of them); kGroup warps share
// a ring and its pages.
template <int NT, int kGroup>
struct KvShape {
  static constexpr int warps = NT == 1 ? 12 : 8;   // (two tiles' states leave no more; heads of 128 spill)
  static constexpr int threads = 32 * warps;
  static constexpr int rings = warps / kGroup, stages = kKvRecords / rings;
};

__host__ __device__ constexpr int part_floats(int D) { return 8 * (D + 2); }

__device__ __forceinline__ int kv_pages(const KvParams& p, int s, int& L) {
  L = (int)ld_global_u32(p.len + s);
  L = L < 0 ? 0 : L;
  const int64_t most = (int64_t)p.M * kPage;
  if (L > most) L = (int)most;
  return (L + kPage - 1) / kPage;
}

// A unit is a page of a segment: a sequence's pages for a head and a pass, sequence by sequence.  (The
// units' number is below 2^31: the entry point refuses more.)  All threads get the total; ends[t]
// holds the units up to the end of thread t's run of sequences.
template <int kThreads>
__device__ __forceinline__ int kv_scan(const KvParams& p, int* ends, int* sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int run = (p.S + kThreads - 1) / kThreads, a = min(p.S, tid * run), b = min(p.S, a + run);
  int upto = 0, L;
  for (int s = a; s < b; ++s) upto += kv_pages(p, s, L);
  upto *= p.Hk * p.passes;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int v = sums[w];
    if (w < warp) upto += v;
    total += v;
  }
  ends[tid] = upto;
  __syncthreads();
  return total;
}

// Shares that the units are cut into: none of them is empty.
__device__ __forceinline__ int kv_shares_used(int total, int most) { return total < most ? total : most; }
__device__ __forceinline__ int kv_share_start(int total, int share, int shares) { return (int)((int64_t)total * share / shares); }

// A walk over units: unit `u` is page `u - seg0` of segment `seg` (head and pass) of sequence s.
struct KvCursor {
  int s, L, pages, seg;
  int seg0;   // first unit of the segment
  // one warp: to the sequence that holds unit u (below the total)
  template <int kThreads>
  __device__ __forceinline__ void start(const KvParams& p, int u, const int* ends, int lane) {
    int t = 0;   // the first run that ends behind u
    for (int t0 = 0; t0 < kThreads; t0 += 32) {
      const unsigned past = __ballot_sync(0xffffffffu, ends[t0 + lane] > u);
      if (past) {
        t = t0 + __ffs(past) - 1;
        break;
      }
    }
    s = t * ((p.S + kThreads - 1) / kThreads);
    seg = 0;
    seg0 = t > 0 ? ends[t - 1] : 0;
    pages = kv_pages(p, s, L);
    seek(p, u);
  }
  __device__ __forceinline__ void seek(const KvParams& p, int u) {
    const int per = p.Hk * p.passes;
    while (u >= seg0 + (per - seg) * pages && s + 1 < p.S) {
      seg0 += (per - seg) * pages;
      seg = 0;
      ++s;
      pages = kv_pages(p, s, L);
    }
    if (u >= seg0 + pages && pages > 0) {
      const int k = min((u - seg0) / pages, per - 1 - seg);
      seg += k;
      seg0 += k * pages;
    }
  }
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float kv_ex2(float t) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// A warp's running state over the pages of a segment.
template <int J, int NT>
struct KvState {
  static constexpr int D = 32 * J, G = kv_groups(D);
  float o[2 * J][NT][4];        // 2^-24 sum q P s; rows of odd values 16 times that
  float z[G][NT][4];        // the same with q = 8 everywhere
  float mm[NT][2], l[NT][2];   // the columns' references, and this thread's tokens' sum of 2^(x - mm)
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < 2 * J; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][t][e] = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[i][t][e] = 0.f;
      mm[t][0] = mm[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
    }
  }
  __device__ __forceinline__ void scale(int t, float f0, float f1) {
#pragma unroll
    for (int i = 0; i < 2 * J; ++i) {
      o[i][t][0] *= f0; o[i][t][1] *= f1; o[i][t][2] *= f0; o[i][t][3] *= f1;
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
      z[i][t][0] *= f0; z[i][t][1] *= f1; z[i][t][2] *= f0; z[i][t][3] *= f1;
    }
    l[t][0] *= f0;
    l[t][1] *= f1;
  }
};

// A warp's query columns as B fragments, and the scores' factors.
template <int J, int NT>
struct KvQuery {
  static constexpr int G = kv_groups(32 * J);
  uint32_t b[NT][J][4];     // b0, b1 of the word's two k-steps
  float f[NT][2], z[NT][G][2];
  int seen[NT][2];            // tokens that columns 2c and 2c + 1 see (columns that are not there: none)

  __device__ __forceinline__ void load(const KvParams& p, int s, int L, int h, int col0, int lane) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int col = col0 + 8 * t + g;
      uint4 w[J];
#pragma unroll
      for (int j = 0; j < J; ++j) w[j] = make_uint4(0u, 0u, 0u, 0u);
      if (col < p.cols) {
        const int i = col / p.G;
        const uint16_t* row = p.q + ((int64_t)s * p.n + i) * p.ldq + (int64_t)(h * p.G + col - i * p.G) * (32 * J);
#pragma unroll
        for (int j = 0; j < J; ++j) w[j] = ld_global_u4(row + 8 * (4 * j + c));
      }
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < J; ++j)
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[j].x & 0x7FFF7FFFu, w[j].y & 0x7FFF7FFFu),
                                     __vmaxu2(w[j].z & 0x7FFF7FFFu, w[j].w & 0x7FFF7FFFu)));
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^-e puts the largest value (exponent field top >> 7) in [2^14, 2^15)
      const int e = min(max((int)(top >> 7), 1), 254) - 127 - 14;
      const int d1 = min(-e, 127);
      const float down = exp2i(d1), down2 = exp2i(-e - d1);
      float zg[G];
#pragma unroll
      for (int i = 0; i < G; ++i) zg[i] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint32_t ws[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
        float x[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = (i & 1 ? bf16hi(ws[i >> 1]) : bf16lo(ws[i >> 1]));
          x[i] = x[i] * down * down2;
          sum += x[i];
        }
        zg[j >> 1] += sum;
        b[t][j][0] = pack_f16(x[0], x[4]);
        b[t][j][1] = pack_f16(x[1] * 0.0625f, x[5] * 0.0625f);
        b[t][j][2] = pack_f16(x[2], x[6]);
        b[t][j][3] = pack_f16(x[3] * 0.0625f, x[7] * 0.0625f);
      }
      // 2^(24 + e) c in two steps, and the zero points' sums over the scaled values: neither leaves FP32's range
      // before the scores do
      const int half = (24 + e) / 2;
      const float fc = p.c * exp2i(half) * exp2i(24 + e - half);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        zg[i] += __shfl_xor_sync(0xffffffffu, zg[i], 1);
        zg[i] += __shfl_xor_sync(0xffffffffu, zg[i], 2);
        zg[i] *= -8.f / 16777216.f * fc;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int from = 4 * (2 * c + k);   // a lane of column 2c + k
        f[t][k] = __shfl_sync(0xffffffffu, fc, from);
#pragma unroll
        for (int i = 0; i < G; ++i) z[t][i][k] = __shfl_sync(0xffffffffu, zg[i], from);
        const int mine = col0 + 8 * t + 2 * c + k;
        seen[t][k] = mine < p.cols ? L - p.n + 1 + mine / p.G : 0;
      }
    }
  }
};

// The scales of a token's groups.
template <int G>
__device__ __forceinline__ void kv_scales(const uint8_t* at, float (&v)[G]) {
  if constexpr (G == 2) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(at));
    v[0] = f.x;
    v[1] = f.y;
  } else {
    v[0] = __half2float(*reinterpret_cast<const __half*>(at));
  }
}

// e with v < 2^e, from fp16's smallest to its largest (infinity counts as that), of v >= 0: the exponent's field as the
// mantissa of 2^23, which takes no conversion.
__device__ __forceinline__ float kv_exponent(float v) {
  return __uint_as_float(0x4B000000u + min(max(__float_as_uint(v) >> 23, 127u - 25u), 127u + 15u)) - (8388608.f + 126.f);
}

// One page (64 tokens from token0 on) joins the warp's state; kEnd: not every column sees all of it.
template <int J, int NT, bool kEnd>
__device__ __forceinline__ void kv_page(KvState<J, NT>& st, const KvQuery<J, NT>& qy, const uint8_t* rec, int token0, int lane) {
  constexpr int D = 32 * J, G = kv_groups(D);
  constexpr uint32_t M0 = 0x000F000Fu, M1 = 0x00F000F0u;
  const int g = lane >> 2, c = lane & 3;
  // (plain loads: the compiler may move them ahead of the products before them)
  const uint8_t *kbase = rec + g * (D / 2) + c * J * 4, *sbase = rec + 64 * D + g * 2 * G;
  float x[4][NT][4];
  float vs[4][2][G];   // V scales of this thread's tokens
  float vtop = 0.f;
  int any = 0;         // tokens that some column sees
  if (kEnd) {
#pragma unroll
    for (int t = 0; t < NT; ++t) any = max(any, max(qy.seen[t][0], qy.seen[t][1]));
    any = max(any, __shfl_xor_sync(0xffffffffu, any, 1));
    any = max(any, __shfl_xor_sync(0xffffffffu, any, 2));
  }
#pragma unroll
  for (int mt = 0; mt < 4; ++mt) {
    float d[G][NT][4];
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[i][t][e] = 0.f;
    uint32_t w[2][J];
    float ks[2][G];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint8_t* at = kbase + (16 * mt + 8 * r) * (D / 2);
      if constexpr (J == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(at);
        w[r][0] = v.x; w[r][1] = v.y; w[r][2] = v.z; w[r][3] = v.w;
      } else if constexpr (J == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(at);
        w[r][0] = v.x; w[r][1] = v.y;
      } else {
#pragma unroll
        for (int j = 0; j < J; ++j) w[r][j] = reinterpret_cast<const uint32_t*>(at)[j];
      }
      kv_scales<G>(sbase + (16 * mt + 8 * r) * 2 * G, ks[r]);
      kv_scales<G>(sbase + (16 * mt + 8 * r) * 2 * G + 128 * G, vs[mt][r]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t h0 = w[0][j] >> 8, h1 = w[1][j] >> 8;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma_16816(d[j >> 1][t], w[0][j] & M0, w[1][j] & M0, w[0][j] & M1, w[1][j] & M1, qy.b[t][j][0], qy.b[t][j][1]);
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma_16816(d[j >> 1][t], h0 & M0, h1 & M0, h0 & M1, h1 & M1, qy.b[t][j][2], qy.b[t][j][3]);
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int r = 0; r < 2; ++r) {   // (columns 2c and 2c + 1 of a token together)
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < G; ++i)
          s = ffma2(make_float2(ks[r][i], ks[r][i]),
                    ffma2(make_float2(qy.f[t][0], qy.f[t][1]), make_float2(d[i][t][2 * r], d[i][t][2 * r + 1]),
                          make_float2(qy.z[t][i][0], qy.z[t][i][1])), s);
        if (kEnd) {
          const int token = token0 + 16 * mt + g + 8 * r;
          if (token >= qy.seen[t][0]) s.x = -INFINITY;
          if (token >= qy.seen[t][1]) s.y = -INFINITY;
        }
        x[mt][t][2 * r] = s.x;
        x[mt][t][2 * r + 1] = s.y;
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      // tokens that no column sees: whatever their scales hold, they are left out
      if (kEnd && token0 + 16 * mt + g + 8 * r >= any)
#pragma unroll
        for (int i = 0; i < G; ++i) vs[mt][r][i] = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) vtop = fmaxf(vtop, fabsf(vs[mt][r][i]));
    }
  }
  // What a column's reference has to stay above, + 14: its largest x plus the exponent of the page's largest V scale
  // (NaN does not count).  At a sequence's end the columns see different tokens, and one's scale must not
  // cost the others their bits: there every x is taken with its own token's scale.
  float top[NT][2];
  if constexpr (kEnd) {
#pragma unroll
    for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float ve = kv_exponent(G == 2 ? fmaxf(fabsf(vs[mt][r][0]), fabsf(vs[mt][r][G - 1])) : fabsf(vs[mt][r][0]));
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) top[t][k] = fmaxf(top[t][k], x[mt][t][2 * r + k] + ve);
      }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        top[t][k] = fmaxf(fmaxf(fmaxf(x[0][t][k], x[0][t][2 + k]), fmaxf(x[1][t][k], x[1][t][2 + k])),
                          fmaxf(fmaxf(x[2][t][k], x[2][t][2 + k]), fmaxf(x[3][t][k], x[3][t][2 + k])));
  }
#pragma unroll
  for (int o = 4; o <= 16; o <<= 1) {
    if (!kEnd) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) top[t][k] = fmaxf(top[t][k], __shfl_xor_sync(0xffffffffu, top[t][k], o));
  }
  const float ve = kEnd ? 0.f : kv_exponent(vtop);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    top[t][0] += ve - 14.f;
    top[t][1] += ve - 14.f;
    if (__any_sync(0xffffffffu, top[t][0] > st.mm[t][0] + 1.f || top[t][1] > st.mm[t][1] + 1.f)) {
      float f[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float m = fmaxf(st.mm[t][k], top[t][k]);
        f[k] = st.mm[t][k] == m ? 1.f : kv_ex2(st.mm[t][k] - m);
        st.mm[t][k] = m;
      }
      st.scale(t, f[0], f[1]);
    }
  }
  // P s as B fragments: [k-step][scale group][tile]
  uint32_t pb[4][G][NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // (a column that has seen nothing yet: its x are -inf, its P 0)
    const float2 m = make_float2(st.mm[t][0] == -INFINITY ? 0.f : -st.mm[t][0], st.mm[t][1] == -INFINITY ? 0.f : -st.mm[t][1]);
    float2 l = make_float2(st.l[t][0], st.l[t][1]);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float2 e = fadd2(make_float2(x[mt][t][2 * r], x[mt][t][2 * r + 1]), m);
        const float2 pr = make_float2(kv_ex2(e.x), kv_ex2(e.y));
        l = fadd2(l, pr);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          float2 ps = kv_fmul2(pr, make_float2(vs[mt][r][i], vs[mt][r][i]));
          if (kEnd) {   // a scale that is not finite stays with the columns that see its token
            if (x[mt][t][2 * r] == -INFINITY) ps.x = 0.f;
            if (x[mt][t][2 * r + 1] == -INFINITY) ps.y = 0.f;
          }
          pb[mt][i][t][r] = movmatrix(pack_f16(ps.x, ps.y));
        }
      }
    st.l[t][0] = l.x;
    st.l[t][1] = l.y;
  }
  const uint8_t* vbase = rec + 32 * D + g * kPage + 16 * c;
#pragma unroll
  for (int i = 0; i < G; ++i)
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma_16816(st.z[i][t], 0x00080008u, 0x00800080u, 0x00080008u, 0x00800080u, pb[s][i][t][0], pb[s][i][t][1]);
#pragma unroll
  for (int md = 0; md < 2 * J; ++md) {
    const uint4 v = *reinterpret_cast<const uint4*>(vbase + md * 8 * kPage);
    const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t h = ws[s] >> 8;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        mma_16816(st.o[md][t], ws[s] & M0, ws[s] & M1, h & M0, h & M1, pb[s][md >> 2][t][0], pb[s][md >> 2][t][1]);
    }
  }
}

// The state's columns in FP32: o in true units times 2^-mm, l over all tokens.
template <int J, int NT>
__device__ __forceinline__ void kv_finish_state(KvState<J, NT>& st) {
  constexpr float up = 16777216.f;   // 2^24
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int md = 0; md < 2 * J; ++md)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.o[md][t][e] = (st.o[md][t][e] - st.z[md >> 2][t][e]) * (e < 2 ? up : up / 16.f);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) st.l[t][k] += __shfl_xor_sync(0xffffffffu, st.l[t][k], o);
  }
}

// They as tiles of [8][D] values, then the references, then the sums.
template <int J, int NT>
__device__ __forceinline__ void kv_put(float* dst, const KvState<J, NT>& st, int lane) {
  constexpr int D = 32 * J;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t, dst += part_floats(D)) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int md = 0; md < 2 * J; ++md)
        *reinterpret_cast<float2*>(dst + (2 * c + k) * D + 16 * md + 2 * g) = make_float2(st.o[md][t][k], st.o[md][t][2 + k]);
    if (g == 0)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        dst[8 * D + 2 * c + k] = st.mm[t][k];
        dst[8 * (D + 1) + 2 * c + k] = st.l[t][k];
      }
  }
}

// The finished columns as bf16 rows; a column that saw no token gives zeros.
template <int J, int NT>
__device__ __forceinline__ void kv_write(const KvParams& p, int s, int h, int col0, const KvState<J, NT>& st, int lane) {
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int col = col0 + 8 * t + 2 * (lane & 3) + k;
      if (col >= p.cols) continue;
      const int i = col / p.G;
      const bool empty = st.mm[t][k] == -INFINITY && st.l[t][k] == 0.f;
      const float r = 1.f / st.l[t][k];
      uint16_t* row = p.out + ((int64_t)s * p.n + i) * p.ldo + (int64_t)(h * p.G + col - i * p.G) * (32 * J);
#pragma unroll
      for (int md = 0; md < 2 * J; ++md) {
        const float a = empty ? 0.f : st.o[md][t][k] * r, b = empty ? 0.f : st.o[md][t][2 + k] * r;
        *reinterpret_cast<uint32_t*>(row + 16 * md + 2 * (lane >> 2)) =
            (uint32_t)float_to_bf16_bits(a) | (uint32_t)float_to_bf16_bits(b) << 16;
      }
    }
}

// Bounded wait with every lane polling and the warp voting: no branch on one lane, no shuffle, so a wait
// whose phase has completed already costs a query and a vote.
__device__ __forceinline__ bool kv_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status) {
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort_flag)) return false;
  }
  *abort_flag = 1;
  if ((threadIdx.x & 31) == 0) atomicExch(status, (int)Q4LIN_ERR_TIMEOUT);
  return false;
}

template <int J>
struct KvSmem {
  static constexpr int rec = kv_record(32 * J);
  static constexpr int bars = kKvRecords * rec;                // per record: copied, free
  static constexpr int alloc = bars + kKvRecords * 16;
};

template <int J, int NT, int kGroup>
__global__ void __launch_bounds__(KvShape<NT, kGroup>::threads, 1) q4_kv_attention_kernel(const KvParams p) {
  using SM = KvSmem<J>;
  using Shape = KvShape<NT, kGroup>;
  constexpr int kKvThreads = Shape::threads, kRings = Shape::rings, kStages = Shape::stages;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int ends[kKvThreads], sums[Shape::warps];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, group = warp / kGroup, member = warp % kGroup;
  const uint32_t base = smem_u32(smem);
  const uint32_t ring = base + (uint32_t)(group * kStages * SM::rec), bars = base + SM::bars + 16u * (uint32_t)(group * kStages);
  if (tid < kKvRecords) {
    mbar_init(base + SM::bars + 16u * tid, 1);
    mbar_init(base + SM::bars + 16u * tid + 8, kGroup);
  }
  if (tid == 0) abort_flag = 0;
  fence_mbar_init();
  pdl_wait_previous();
  // (not before the wait: the second kernel reads the lengths as soon as it runs)
  pdl_launch_dependents();
  const int total = kv_scan<kKvThreads>(p, ends, sums);
  // (few units: their shares lie in as many CTAs as there are)
  const int shares = kv_shares_used(total, (int)gridDim.x * kRings), share = group * (int)gridDim.x + (int)blockIdx.x;
  if (share >= shares) return;   // (no barrier of the CTA follows)
  const int u0 = kv_share_start(total, share, shares), u1 = kv_share_start(total, share + 1, shares);

  KvCursor here;
  here.start<kKvThreads>(p, u0, ends, lane);
  // copies run kStages ahead of their use; the group's first warp issues them
  KvCursor ahead = here;
  int next = u0, used = 0, filled = 0;
  uint32_t there = 0;       // per stage: a page was copied
  int32_t held = -1;        // lane l: page of unit held0 + l, up to held1 (of one segment)
  int held0 = u0, held1 = u0;
  bool ok = true;
  auto look = [&]() {
    if (next < u1 && next >= held1) {
      ahead.seek(p, next);
      held0 = next;
      held1 = min(min(ahead.seg0 + ahead.pages, u1), next + 32);
      if (next + lane < held1) held = (int32_t)ld_global_u32(p.table + (int64_t)ahead.s * p.M + (next - ahead.seg0) + lane);
    }
  };
  auto issue = [&]() {      // (every warp keeps the books)
    if (next >= u1) return;
    const int st = filled % kStages;
    const int32_t page = __shfl_sync(0xffffffffu, held, next - held0);
    const bool good = page >= 0 && page < p.P;   // a page that is not there: its tokens are left out
    there = good ? there | 1u << st : there & ~(1u << st);
    if (good && member == 0 && lane == 0) {
      const uint32_t bar = bars + 16u * (uint32_t)st;
      mbar_expect_tx(bar, SM::rec);
      bulk_load(ring + (uint32_t)(st * SM::rec), p.cache + ((int64_t)page * p.Hk + ahead.seg / p.passes) * SM::rec, SM::rec, bar);
    }
    ++filled;
    ++next;
    look();
  };
  __syncwarp();
  look();
  for (int i = 0; i < kStages; ++i) issue();

  KvState<J, NT> st;
  KvQuery<J, NT> qy;
  uint32_t phases = 0;      // per stage: the parity of its next copy
  for (int u = u0; u < u1 && ok;) {
    here.seek(p, u);
    const int end = min(here.seg0 + here.pages, u1);   // this share's units of the segment
    const int h = here.seg / p.passes, col0 = ((here.seg - h * p.passes) * kGroup + member) * 8 * NT;
    const bool whole = end - u == here.pages;
    st.clear();
    qy.load(p, here.s, here.L, h, col0, lane);
    for (; u < end; ++u) {
      const int s = used % kStages;
      if (there >> s & 1u) {
        ok = kv_wait(bars + 16u * (uint32_t)s, phases >> s & 1u, &abort_flag, &g_kv_status);
        if (!ok) break;
        phases ^= 1u << s;
        const int token0 = (u - here.seg0) * kPage;
        // (the last n - 1 tokens are seen by some columns only)
        if (token0 + kPage <= here.L - p.n + 1)
          kv_page<J, NT, false>(st, qy, smem + (group * kStages + s) * SM::rec, token0, lane);
        else
          kv_page<J, NT, true>(st, qy, smem + (group * kStages + s) * SM::rec, token0, lane);
      }
      if constexpr (kGroup == 1) {
        ++used;
        __threadfence_block();
        __syncwarp();
        issue();
      } else {
        // The record before this one is refilled: the group's other warps are likely done with it.  Every warp waits
        // for that: a run of pages that are not there has no copies to hold the others back, and the phase's one
        // bit does not tell two rounds of the ring apart.
        warp_release(bars + 16u * (uint32_t)s + 8, lane);
        const int b = used - 1;
        ++used;
        if (b >= 0) {
          if (next < u1) {
            ok = kv_wait(bars + 16u * (uint32_t)(b % kStages) + 8, (uint32_t)(b / kStages) & 1u, &abort_flag, &g_kv_status);
            if (!ok) break;
          }
          issue();
        }
      }
    }
    kv_finish_state(st);
    if (!ok) break;
    if (whole) {
      kv_write(p, here.s, h, col0, st, lane);
    } else {
      // (a share's first segment may have begun in an earlier share, its last may go on: slots 0 and 1)
      const int slot = here.seg0 > u0 ? 1 : 0;
      kv_put(p.part + (((int64_t)share * 2 + slot) * kGroup + member) * NT * part_floats(32 * J), st, lane);
    }
  }
  // nothing is left in flight, after a wait that ran out either
  if (!ok && member == 0 && lane == 0)
    for (int i = used; i < filled; ++i)
      if (there >> (i % kStages) & 1u) mbar_drain(bars + 16u * (uint32_t)(i % kStages), phases >> (i % kStages) & 1u);
}

// Segments that lie in several shares, and sequences without tokens.  D / 2 threads hold a column, two
// values each.  kSplit: a CTA takes one column, its groups of threads the partial sums in turn (few
// long segments); otherwise a CTA takes a segment, its groups the columns (many short ones).
constexpr int kKvJoin = 256;
template <int J, int kTiles, bool kSplit>
__global__ void __launch_bounds__(kKvJoin) q4_kv_combine_kernel(const KvParams p, int most) {
  constexpr int D = 32 * J, kLanes = kKvJoin / (D / 2);
  __shared__ int ends[kKvJoin], sums[kKvJoin / 32];
  // Ahead of the wait for the first kernel stand the lengths only: that kernel lets this one start after
  // its own wait, so what it found complete is complete here.
  const int tid = threadIdx.x, per = p.Hk * p.passes, lane = tid / (D / 2), d = tid - lane * (D / 2);
  const int total = kv_scan<kKvJoin>(p, ends, sums);
  const int shares = kv_shares_used(total, most);
  const int run = (p.S + kKvJoin - 1) / kKvJoin;
  const int64_t pitch = (int64_t)2 * kTiles * part_floats(D);
  const int s = blockIdx.x / per, seg = blockIdx.x - s * per, h = seg / p.passes, pass = seg - h * p.passes, t = s / run;
  const int cols = min(8 * kTiles, p.cols - pass * 8 * kTiles);
  int L, a = t > 0 ? ends[t - 1] : 0;
  for (int i = t * run; i < s; ++i) a += kv_pages(p, i, L) * per;
  const int pages = kv_pages(p, s, L);
  a += seg * pages;
  int c0 = 0, n = 0;   // the segment's shares
  if (pages > 0) {
    c0 = (int)((((int64_t)a + 1) * shares - 1) / total);
    n = (int)(((int64_t)(a + pages) * shares - 1) / total) - c0 + 1;
  }
  // a share's slot: 1 only where the segment begins inside it, behind another (that is its first share's case)
  const int64_t head = n > 0 && a > kv_share_start(total, c0, shares) ? kTiles * part_floats(D) : 0;
  pdl_launch_dependents();
  pdl_wait_previous();   // (by every CTA: this kernel does not end before the first one)
  if (n == 1 || (int)blockIdx.y >= cols) return;   // finished by its share; a narrower last pass
  auto at = [&](int c, int local) {
    return p.part + (c0 + c) * pitch + (c == 0 ? head : 0) + (local >> 3) * part_floats(D);
  };
  // partial sums from, from + step, .. of column `local`, two values of it: eight at a time on their way
  auto join = [&](int local, int d, int from, int step, float& m, float2& o, float& l) {
    const int v = (local & 7) * D + 2 * d, k = 8 * D + (local & 7);
    m = -INFINITY;
    l = 0.f;
    o = make_float2(0.f, 0.f);
    for (int c = from; c < n; c += 8 * step) {
      float mc[8], lc[8], top = m;
      float2 oc[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mc[i] = -INFINITY;
        lc[i] = 0.f;
        oc[i] = make_float2(0.f, 0.f);
        if (c + i * step < n) {
          const float* q = at(c + i * step, local);
          mc[i] = q[k];
          lc[i] = q[k + 8];
          oc[i] = *reinterpret_cast<const float2*>(q + v);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, mc[i]);
      const float f0 = m == top ? 1.f : kv_ex2(m - top);   // (equal references, both -inf among them, need no factor)
      o = kv_fmul2(o, make_float2(f0, f0));
      l *= f0;
      m = top;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = mc[i] == m ? 1.f : kv_ex2(mc[i] - m);
        o = ffma2(oc[i], make_float2(f, f), o);
        l = fmaf(lc[i], f, l);
      }
    }
  };
  auto write = [&](int local, int d, float m, float2 o, float l) {
    const int col = pass * 8 * kTiles + local, i = col / p.G;
    const bool empty = m == -INFINITY && l == 0.f;
    const float r = 1.f / l;
    uint16_t* row = p.out + ((int64_t)s * p.n + i) * p.ldo + (int64_t)(h * p.G + col - i * p.G) * D;
    *reinterpret_cast<uint32_t*>(row + 2 * d) =
        empty ? 0u : (uint32_t)float_to_bf16_bits(o.x * r) | (uint32_t)float_to_bf16_bits(o.y * r) << 16;
  };
  float m, l;
  float2 o;
  if constexpr (!kSplit) {
    if (lane >= kLanes) return;
    for (int local = lane; local < cols; local += kLanes) {
      join(local, d, 0, 1, m, o, l);
      write(local, d, m, o, l);
    }
  } else {
    __shared__ float2 red[kLanes][D / 2];
    __shared__ float ms[kLanes], ls[kLanes];
    const int local = blockIdx.y;
    if (lane < kLanes) {
      join(local, d, lane, kLanes, m, o, l);
      red[lane][d] = o;
      if (d == 0) {
        ms[lane] = m;
        ls[lane] = l;
      }
    }
    __syncthreads();
    if (tid >= D / 2) return;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) top = fmaxf(top, ms[i]);
    l = 0.f;
    o = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kLanes; ++i) {
      const float f = ms[i] == top ? 1.f : kv_ex2(ms[i] - top);
      l = fmaf(ls[i], f, l);
      o = ffma2(red[i][tid], make_float2(f, f), o);
    }
    write(local, tid, top, o, l);
  }
}

int kv_sms() {
  static int cache[64] = {};
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64) {
    if (cache[dev] == 0 && cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) cache[dev] = sms;
    if (cache[dev] != 0) return cache[dev];
  }
  return sms;
}

template <int J, int NT, int kGroup>
int kv_attention_run(const KvParams& p, cudaStream_t stream) {
  using SM = KvSmem<J>;
  static bool set[64] = {};
  int dev = 0;
  if (cuda_check(cudaGetDevice(&dev), "cudaGetDevice")) return Q4LIN_ERR_CUDA;
  if (dev >= 64 || !set[dev]) {
    if (cuda_check(cudaFuncSetAttribute(q4_kv_attention_kernel<J, NT, kGroup>, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::alloc),
                   "kv4_attention: cudaFuncSetAttribute(max dynamic shared memory)"))
      return Q4LIN_ERR_CUDA;
    if (dev < 64) set[dev] = true;
  }
  const int sms = kv_sms();
  const int st = pdl_launch(q4_kv_attention_kernel<J, NT, kGroup>, "kv4_attention: kernel launch", dim3((unsigned)sms, 1, 1), KvShape<NT, kGroup>::threads, SM::alloc, stream, &p);
  if (st != Q4LIN_OK) return st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const int64_t segments = (int64_t)p.S * p.Hk * p.passes;
  const int cols = p.cols < 8 * NT * kGroup ? p.cols : 8 * NT * kGroup;
  // In rounds of eight partial sums on their way, a CTA's beginning counted as two, for a segment three times as
  // long as the mean: the columns of a segment one after the other, or a CTA per column (its groups of
  // threads share the sums) in as many waves as the GPU holds of them, four per SM.  (16 sequences of up to
  // 8192 tokens, 16 columns: 47 us and 35; 32 columns in two passes: 77 and 95.)
  const int64_t parts = 3 * sms * KvShape<NT, kGroup>::rings / segments + 1, held = 4 * sms;
  const int64_t whole = 2 + (cols + 3) / 4 * ((parts + 7) / 8), quarter = (segments * cols + held - 1) / held * (2 + (parts + 31) / 32);
  const bool split = quarter < whole;
  cfg.gridDim = dim3((unsigned)segments, (unsigned)(split ? cols : 1), 1);
  cfg.blockDim = dim3(kKvJoin, 1, 1);
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int shares = sms * KvShape<NT, kGroup>::rings;
  return cuda_check(split ? cudaLaunchKernelEx(&cfg, q4_kv_combine_kernel<J, NT * kGroup, true>, p, shares)
                          : cudaLaunchKernelEx(&cfg, q4_kv_combine_kernel<J, NT * kGroup, false>, p, shares),
                    "kv4_attention: combine launch");
}

// Tiles of a pass, 8 columns each: one warp with one or two, or two warps with two each.
int kv_tiles(int64_t cols) { return cols <= 8 ? 1 : cols <= 16 ? 2 : 4; }

}  // namespace

int64_t kv_page_bytes(int64_t D) { return kv_record((int)D); }

// Two partial sums per share and tile: 12 or 16 tiles per SM.
int64_t kv_workspace_bytes(int64_t D) { return (int64_t)kv_sms() * 16 * 2 * part_floats((int)D) * 4; }

int64_t kv_passes(int64_t cols) { return (cols + 8 * kv_tiles(cols) - 1) / (8 * kv_tiles(cols)); }

int kv_tokens_launch(const KvTokArgs& a, bool append) {
  KvTokParams p{};
  p.src[0] = a.k; p.src[1] = a.v;
  p.dst[0] = a.k_out; p.dst[1] = a.v_out;
  p.ld[0] = a.ldk; p.ld[1] = a.ldv;
  p.cache = a.cache;
  p.table = a.table;
  p.rows = a.rows;
  p.pos = a.pos;
  p.T = a.T; p.S = a.S; p.M = a.M; p.P = a.P;
  p.Hk = (int)a.Hk;
  p.D = (int)a.D;
  const int lpr = a.D == 64 ? 8 : 16;
  const dim3 blocks((unsigned)((a.T + kTokTile - 1) / kTokTile), (unsigned)(2 * a.Hk), 1);
  if (blocks.y > 65535) {
    set_error_detail("kv4: too many heads for one launch");
    return Q4LIN_ERR_UNSUPPORTED_SHAPE;
  }
  if (append)
    return lpr == 8 ? pdl_launch(q4_kv_append_kernel<8>, "kv4_append: kernel launch", blocks, kTokThreads, 0, a.stream, &p)
                    : pdl_launch(q4_kv_append_kernel<16>, "kv4_append: kernel launch", blocks, kTokThreads, 0, a.stream, &p);
  return lpr == 8 ? pdl_launch(q4_kv_read_kernel<8>, "kv4_read: kernel launch", blocks, kTokThreads, 0, a.stream, &p)
                  : pdl_launch(q4_kv_read_kernel<16>, "kv4_read: kernel launch", blocks, kTokThreads, 0, a.stream, &p);
}

int kv_attention_launch(const KvAttnArgs& a) {
  KvParams p{};
  p.q = a.q; p.out = a.out;
  p.ldq = a.ldq; p.ldo = a.ldo;
  p.cache = a.cache;
  p.table = a.table;
  p.len = a.len;
  p.part = static_cast<float*>(a.workspace);
  p.P = a.P;
  p.S = (int)a.S; p.M = (int)a.M; p.n = (int)a.n;
  p.Hk = (int)a.Hk; p.G = (int)(a.Hq / a.Hk);
  p.cols = p.n * p.G;
  p.passes = (int)kv_passes(p.cols);
  p.c = a.scale * 1.4426950408889634f;
  const int tiles = kv_tiles(p.cols);
  auto pick = [&](auto j) {
    constexpr int J = decltype(j)::value;
    return tiles == 1   ? kv_attention_run<J, 1, 1>(p, a.stream)
           : tiles == 2 ? kv_attention_run<J, 2, 1>(p, a.stream)
                        : kv_attention_run<J, 2, 2>(p, a.stream);
  };
  if (a.D == 64) return pick(std::integral_constant<int, 2>{});
  if (a.D == 96) return pick(std::integral_constant<int, 3>{});
  return pick(std::integral_constant<int, 4>{});
}

int kv_status(int* value, bool clear) {
  if (cudaMemcpyFromSymbol(value, g_kv_status, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  if (clear) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_kv_status, &zero, sizeof(int)) != cudaSuccess) return Q4LIN_ERR_CUDA;
  }
  return Q4LIN_OK;
}

}  // namespace q4
