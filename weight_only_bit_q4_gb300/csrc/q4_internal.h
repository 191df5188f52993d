// Host-side declarations shared by the q4lin translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace q4 {

// Records why a call failed (thread-local; read by q4lin_last_error_detail)
// and returns Q4LIN_ERR_CUDA when `e` is an error, Q4LIN_OK otherwise.
int cuda_check(cudaError_t e, const char* where);
void set_error_detail(const char* what);

// Low-rank adapters of LinearLora: y += scales[a] B_a (A_a x), a = ids[t].
struct LoraArgs {
  const uint16_t* a;      // [L, R, K] bf16
  const uint16_t* b;      // [L, N, R] bf16
  const int32_t* ids;     // [T]; outside [0, L): no adapter
  const float* scales;    // [L] or NULL (1)
  const int32_t* ranks;   // [L] or NULL (R); clamped to [0, R]
  float* u;               // [ks, T, R] partial sums of A x along K, already scaled
  int L, R, ks;
  void* tiles;            // tile route: lora_records(T, L) records of kLoraTileBytes; else NULL
};
constexpr int kLoraTileBytes = 48;

struct LinearArgs {
  const uint8_t* wq;
  const uint16_t* scales;
  const uint16_t* x;
  uint16_t* y;
  int64_t N, K, T;
  void* workspace;
  cudaStream_t stream;
  int fmt = 0;                   // weight format (0: Q4G64; 1: Q5G64, 2: Q6G64, 3: W8G32)
  const uint8_t* wh = nullptr;   // Q5G64 / Q6G64: the high-bit plane
  const uint16_t* r = nullptr;   // LinearAdd: bf16 residual [T, N] (tile route)
  // fused forms on the exact tile route: 1 = LinearSwiGLU (wq / scales hold 2N rows, gate then
  // up; y is [T, N]), 2 = LinearPair (a second weight wq_b / scales_b of n_b rows into y_b)
  int mode = 0;
  const uint8_t* wq_b = nullptr;
  const uint16_t* scales_b = nullptr;
  uint16_t* y_b = nullptr;
  int64_t n_b = 0;
  // LinearLora: the adapters (GEMV and warp-MMA routes apply them in their epilogues; on the
  // tile route, mode 3, the accumulators start from the FP32 term delta [T, lora_delta_pitch(N)];
  // mode 4: the second product as lora_groups further K groups over lora_u [T][lora_groups][64])
  const LoraArgs* lora = nullptr;
  const float* delta = nullptr;
  const uint16_t* lora_u = nullptr;
  int lora_groups = 0;
};

// The adapters' two products beside the projection (q4_lora.cu).
int lora_splits(int64_t K, int64_t T, int64_t L);
int64_t lora_shrink_grid(const LoraArgs& lo, int64_t T);   // CTAs
int64_t lora_records(int64_t T, int64_t L);
int64_t lora_delta_pitch(int64_t N);                        // floats per token row of delta
int lora_shrink_launch(const LoraArgs& lo, const uint16_t* x, int64_t K, int64_t T, cudaStream_t stream);
int lora_expand_launch(const LoraArgs& lo, float* delta, int64_t N, int64_t T, cudaStream_t stream);
int64_t lora_groups(int64_t K, int64_t L, int64_t R);       // 64-wide groups of u as bf16 terms; 0: delta instead
int lora_spread_launch(const LoraArgs& lo, uint16_t* u, int groups, int64_t T, cudaStream_t stream);

// The weight planes are stored for K rounded up to a multiple of 128
// (linear-benchmark.md section 4, K_pad); columns k >= K are padding.
inline int64_t k_pad(int64_t K) { return (K + 127) / 128 * 128; }

// CUDA-core GEMV: each weight is decoded once per block of up to 4 tokens.
int gemv_launch(const LinearArgs& a);
size_t gemv_workspace_bytes(int64_t N, int64_t K, int64_t T);
int gemv_launch_count(int64_t N, int64_t K, int64_t T);
// Whether the streaming kernel (1..4 tokens, one launch) has a shared-memory plan for
// (N, K, T) on the current device.
bool gemv_stream_ok(int64_t N, int64_t K, int64_t T, int fmt = 0);
// One token with an adapter of rank R on the streaming GEMV (LinearArgs::lora).
bool gemv_lora_ok(int64_t N, int64_t K, int R);
int gemv_lora_launch(const LinearArgs& a);
// The sibling formats (fmt 1..3) run on the streaming GEMV only.
int gemv_launch_fmt(const LinearArgs& a);

// tcgen05 tile routes: one CTA per 128-row x BN-token output tile (per K
// share when split across a cluster), group partials in tensor memory.
struct TcPlan {
  int bn;              // token tile (MMA N)
  int splitk;          // cluster size along K of the main launch
  int64_t main_tiles;  // output tiles of the main launch (all of them without a tail launch)
  int tail_splitk;     // cluster size along K of the tail launch over the other tiles (0 = none)
};
// fmt: 0 Q4G64, 1 Q5G64, 2 Q6G64 (the latter two on token tiles up to 128 wide)
TcPlan tc_plan(int route, int64_t N, int64_t K, int64_t T, int sms, int fmt = 0);
TcPlan tc_plan_current_device(int route, int64_t N, int64_t K, int64_t T, int fmt = 0);
int tc_launch(const LinearArgs& a, int route);
// The folded tile routes (Q4LIN_ROUTE_TC, Q4LIN_ROUTE_TC_SPLITK) need workspace for
// their fp16 operands and launch a prep kernel first; the exact route needs none.
size_t tc_workspace_bytes(int route, int64_t N, int64_t K, int64_t T);
int tc_launch_count(int route, int64_t N, int64_t K, int64_t T, int fmt = 0);
// The fp16 tile route with its operand scratch in a fixed device array instead of
// a caller workspace (q4lin_linear_fp16_static): whether (N, K, T) fits, and the call.
bool tc_fp16_static_fits(int64_t N, int64_t K, int64_t T);
int tc_fp16_static_launch(const LinearArgs& a);
bool tc_supported(int64_t N, int64_t K, int64_t T);

// A 2-D tensor map (inner extent, outer extent, row pitch in bytes, box); false if the
// driver's encoder is unavailable or refuses the arguments.
bool encode_map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swizzle);
// A 4-D tensor map (extents, byte strides of dimensions 1..3, box).
bool encode_map_4d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, const uint64_t (&dims)[4],
                   const uint64_t (&strides)[3], const uint32_t (&box)[4], CUtensorMapSwizzle swizzle);

// Streaming warp-MMA route (a few tokens; any T in passes of 32): an operand pass
// writes X as fp16 MMA fragments into the workspace, then one persistent kernel
// streams the weights.  Whether it has a shared-memory plan for (N, K, T), its
// workspace, its launch count and the call.
// fmt: 0 Q4G64, 1 Q5G64, 2 Q6G64, 3 W8G32
bool mma_supported(int64_t N, int64_t K, int64_t T, int fmt = 0);
size_t mma_workspace_bytes(int64_t N, int64_t K, int64_t T, int fmt = 0);
int mma_launch_count(int64_t N, int64_t K, int64_t T, int fmt = 0);
// fused: the one-launch form without workspace (up to 8 tokens, where the whole-K operands
// fit in shared memory), for the entry points that take no workspace
// (swiglu: LinearSwiGLU with N = F output rows over a 2F-row weight)
bool mma_fused_supported(int64_t N, int64_t K, int64_t T, int fmt = 0, bool swiglu = false);
int mma_launch(const LinearArgs& a, bool fused = false);
// LinearLora on the two-kernel form, up to 32 tokens: the operand pass also runs the shrink
// product, the streaming kernel's band epilogue adds the second one.
bool mma_lora_supported(int64_t N, int64_t K, int64_t T, int R);
size_t mma_lora_workspace_bytes(int64_t N, int64_t K, int64_t T, int R);
int mma_status(int* value, bool clear);

// Query / key head norms with the position rotation (strides in elements).
struct QkArgs {
  const uint16_t *q, *k, *q_weight, *k_weight;
  const float* table;      // [P, rot] fp32: cosines, then sines
  const int32_t* pos;      // [T]
  uint16_t *q_out, *k_out;
  int64_t ldq, ldk, ldqo, ldko;
  int64_t T, Hq, Hk, D, rot, P;
  float eps;
  bool interleaved;
  cudaStream_t stream;
};
int qk_norm_rope_launch(const QkArgs& a);

// Mixture-of-experts layer with Q4 experts (any T in passes of at most 512 (token, choice) slots).
struct MoeArgs {
  const uint16_t* x;          // [T, H]
  const uint16_t* w_router;   // [E, H] (router only)
  const float* bias;          // [E] or NULL (router only)
  int32_t* ids_out;           // [T, k] (router only)
  float* weights_out;
  const int32_t* ids;         // [T, k] (experts only)
  const float* weights;
  const uint8_t *wq_gu, *wq_dn;    // [E, 2F, Hp/2], [E, H, Fp/2]
  const uint16_t *s_gu, *s_dn;     // [E, 2F, Hp/64], [E, H, Fp/64]
  uint16_t* y;                // [T, H]
  int64_t T, H, F, E;
  int k, renorm;
  void* workspace;
  cudaStream_t stream;
};
// Whether every pass of these sizes has a plan (a column of H values fits shared memory).
bool moe_supported(int64_t T, int64_t H, int64_t F, int64_t E, int k);
size_t moe_workspace_bytes(int64_t T, int64_t H, int64_t F, int64_t E, int k);
// With a workspace the router also runs the experts' first operand pass into it (prepared).
int moe_router_launch(const MoeArgs& a);
int moe_experts_launch(const MoeArgs& a, bool prepared);
int moe_status(int* value, bool clear);

// Attention over whole prompts: causal, packed sequences (strides in elements).
struct PromptArgs {
  const uint16_t *q, *k, *v;
  uint16_t* out;
  int64_t ldq, ldk, ldv, ldo;
  const int32_t* cu;       // [S + 1]
  int64_t T, S, Hq, Hk, D;
  float scale;
  cudaStream_t stream;
};
int prompt_launch(const PromptArgs& a);
int prompt_status(int* value, bool clear);

// The paged 4-bit cache: tokens in (append: k, v -> cache) and out (cache -> k_out, v_out).
struct KvTokArgs {
  const uint16_t *k, *v;
  uint16_t *k_out, *v_out;
  int64_t ldk, ldv;
  uint8_t* cache;
  const int32_t *table, *rows, *pos;
  int64_t T, S, M, P, Hk, D;
  cudaStream_t stream;
};
int64_t kv_page_bytes(int64_t D);
int kv_tokens_launch(const KvTokArgs& a, bool append);
// Attention of n new tokens per sequence over the cache.
struct KvAttnArgs {
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, ldo;
  const uint8_t* cache;
  const int32_t *table, *len;
  int64_t S, n, Hq, Hk, D, M, P;
  float scale;
  void* workspace;
  cudaStream_t stream;
};
int64_t kv_passes(int64_t cols);   // passes over a head's cols = n Hq / Hk query columns
int64_t kv_workspace_bytes(int64_t D);
int kv_attention_launch(const KvAttnArgs& a);
int kv_status(int* value, bool clear);

// Log probabilities of given tokens, entropy and top tokens of rows of logits.
struct LogprobArgs {
  const void* logits;
  int64_t ld;
  const int32_t* targets;
  float *logprobs, *entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int64_t T, V, n;
  int k;
  bool fp32;
  cudaStream_t stream;
};
int logprobs_launch(const LogprobArgs& a);

// Reads (and optionally clears) the device error word of one translation unit.
int gemv_status(int* value, bool clear);
int tc_status(int* value, bool clear);
int probe_status(int* value, bool clear);

// Diagnostics: HBM read probe and the bounded-wait expiry check.
int hbm_read_probe(const void* src, size_t bytes, uint32_t* sink, int blocks, cudaStream_t stream);
// Copies `bytes` (a multiple of 2; both pointers 16-byte aligned and device-accessible,
// page-locked host memory included) in stream order, chained by programmatic launch.
int stage_copy(const void* src, void* dst, size_t bytes, cudaStream_t stream);
int wait_expiry(uint32_t limit, int* out, cudaStream_t stream);

}  // namespace q4
