// Host-side interface of the 4-bit key/value cache kernels (kv4_*.cu), beside internal.h.
#pragma once

#include <atomic>

#include "internal.h"

namespace dsv4 {

// launch_pdl of a kernel that takes more than 48 KiB of dynamic shared memory. The attribute that allows it is
// set once per kernel and device (setting it costs about as much as a launch), and again where a launch
// fails after that (a device reset drops it).
template <auto Kernel, typename... Args>
cudaError_t launch_large(dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args... args) {
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  for (bool again = false;; again = true) {
    const bool set = allowed.load(std::memory_order_relaxed) & bit;
    if (!set || again) {
      e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
      allowed.fetch_or(bit, std::memory_order_relaxed);
    }
    e = launch_pdl(Kernel, grid, block, smem, st, 1, args...);
    if (e == cudaSuccess || !set || again) return e;
    cudaGetLastError();
  }
}

constexpr int kKv4Block = 32;               // channels that share one power-of-two scale
constexpr int kKv4ExpMin = -23;             // scale exponents: every code times its scale is then
constexpr int kKv4ExpMax = 13;              // an exact fp16 (and bf16) value

struct Kv4Cache {
  uint8_t *k_codes, *v_codes;    // [num_pages][Hk][256][D / 2]
  uint8_t *k_scales, *v_scales;  // [num_pages][Hk][256][D / 32]
  const int32_t *block_table;    // [B][max_blocks]
  int num_pages, max_blocks;
};

// Head norms and rotation of new tokens (cache.k_codes null: q and k to q_out and k_out;
// otherwise q to q_out, k and v to the cache).
struct Kv4HeadsLaunch {
  int B, T, Hq, Hk, D;
  const void *q, *k, *v;                  // rows of D values, heads contiguous
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  dsv4_dtype in_dt, out_dt;               // F32 or BF16
  const float *gamma_q, *gamma_k;         // [D], null: no norm
  float eps;
  int rope_dims;
  float rope_base;
  double rope_theta1 = 1.0;               // filled by the launcher
  const int32_t *cu_seqlens, *start_pos;
  void *q_out, *k_out;                    // [T][H][D]
  uint16_t *k_stored, *v_stored;          // [T][Hk][D] bf16, optional (cache only)
  Kv4Cache cache;
  uint32_t *d_status;
};
cudaError_t launch_kv4_heads(const Kv4HeadsLaunch &p, cudaStream_t st);

struct Kv4AttnLaunch {
  int B, T, Hq, Hk, D;
  int max_new;              // the most new tokens of a sequence (chooses the kernel, nothing else)
  const uint16_t *q;        // [T][Hq][D] bf16
  int64_t q_stride;         // elements between tokens
  const int32_t *cu_seqlens, *start_pos;
  Kv4Cache cache;
  float softmax_scale;      // > 0
  uint16_t *out;            // [T][Hq][D] bf16
  float *lse;               // [T][Hq] or null
  uint32_t *d_status;
};
// how the form for many rows per sequence shares out a call
struct Kv4PromptShape {
  int row_blocks;     // blocks of 256 rows of each sequence and key/value head
  int whole, splits;  // units that one CTA takes; CTAs of each of the others
};
Kv4PromptShape kv4_prompt_shape(const Kv4AttnLaunch &p);
int64_t kv4_prompt_most_parts(const Kv4AttnLaunch &p);  // of any call whose sizes are no larger

// which kernel takes a call: of sizes and the codes' alignment alone
struct Kv4AttnPlan {
  dsv4_kv4_form form;
  int rows;              // of a row tile
  Kv4PromptShape shape;  // DSV4_KV4_PROMPT
};
Kv4AttnPlan kv4_attention_plan(const Kv4AttnLaunch &p);
size_t kv4_attention_workspace_bytes(const Kv4AttnLaunch &p, const Kv4AttnPlan &plan);
size_t kv4_attention_workspace_limit(const Kv4AttnLaunch &p);  // of any call whose sizes are no larger
cudaError_t launch_kv4_attention(const Kv4AttnLaunch &p, const Kv4AttnPlan &plan, void *ws, cudaStream_t st);
size_t kv4_prompt_workspace_bytes(int dim, int64_t parts);  // parts: CTAs that share units
inline int64_t kv4_prompt_parts(const Kv4AttnLaunch &p, const Kv4PromptShape &g) {
  return (static_cast<int64_t>(g.row_blocks) * p.B * p.Hk - g.whole) * g.splits;
}
cudaError_t launch_kv4_prompt(const Kv4AttnLaunch &p, const Kv4PromptShape &g, void *ws, cudaStream_t st);

}  // namespace dsv4
