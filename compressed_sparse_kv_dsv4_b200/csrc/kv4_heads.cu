// Head norms, position rotation and the 4-bit cache append (vLLM's fused "Q-norm + KV RoPE +
// K insert", here for separate key and value heads):
//
//   y = RoPE_p( x / sqrt(mean(x^2) + eps) * gamma )      each query and key head
//   cache row = round4(y) for keys, round4(v) for values
//
// round4 works on blocks of 32 channels: the scale is 2^k with the smallest k in [-23, 13]
// that has amax <= 6 * 2^k (0 for a zero block), the codes are e2m1, nearest with ties to even,
// saturating. amax = 1.f * 2^e needs k = e - 2 where 1.f <= 1.5 (6 = 1.5 * 2^2) and e - 1
// otherwise, so k comes from the exponent and mantissa bits without a logarithm. A block that
// holds an infinity or a NaN is stored as scale byte 255, which reads as NaN.
//
// One pass, bound by memory: a token's rows are its query heads, key heads and value heads;
// D / 8 neighbouring lanes (at most a warp) hold one row, 8 values (16 bytes of bf16) each, so
// the row's sum of squares and a block's amax are a few shuffles. A block of 256 threads takes
// a few tokens at a time; the angles of a token (float64, the most expensive arithmetic here)
// are worked out once by one thread per pair and token and shared by all its heads.
#include "common.cuh"
#include "kv4.h"

namespace dsv4 {

namespace {

constexpr int kHThreads = 256;
constexpr int kHTokens = 4;   // tokens of a block's step
constexpr int kHPairs = 256;  // rotated pairs at most (D <= 512)

struct HeadsParams {
  Kv4HeadsLaunch a;
  int rows;        // rows of a token: Hq + Hk (+ Hk value rows)
  int row_split;   // blocks along y, each on every row_split-th group of rows
  int tok_blocks;  // blocks along x
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int E, bool F32>
__device__ __forceinline__ void load_vals(const void *base, int64_t off, float (&x)[E]) {
  if constexpr (F32) {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + off);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 v = __ldcs(p + i);
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + off);
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      const uint4 v = __ldcs(p + i);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) x[8 * i + 2 * k] = bf16_lo(w[k]), x[8 * i + 2 * k + 1] = bf16_hi(w[k]);
    }
  }
}

template <int E>
__device__ __forceinline__ void store_vals(void *base, dsv4_dtype dt, int64_t off, const float (&x)[E]) {
  if (dt == DSV4_F32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + off);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else {
    uint4 *p = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off);
#pragma unroll
    for (int i = 0; i < E / 8; ++i)
      p[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                        pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  }
}

// two floats -> one byte of e2m1 codes (lo in the low nibble): nearest even, saturating at 6
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Scale byte of a block with the given amax (a non-finite amax: 255).
__device__ __forceinline__ int block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  if (u >= 0x7F800000u) return 255;
  if (u == 0) return 127;
  const int e = static_cast<int>(u >> 23) - 127;
  const int k = (u & 0x7FFFFFu) <= 0x400000u ? e - 2 : e - 1;
  return min(max(k, kKv4ExpMin), kKv4ExpMax) + 127;
}

template <int D, bool F32>
__global__ void __launch_bounds__(kHThreads) kv4_heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int E = D <= 256 ? 8 : D / 32;  // values of a row per lane
  constexpr int L = D / E;                  // lanes of a row
  constexpr int G = kHThreads / L;          // rows of a block at a time
  const Kv4HeadsLaunch &p = P.a;
  __shared__ float2 turn[kHTokens][kHPairs];
  __shared__ int first_sh;
  __shared__ int64_t pos_sh[kHTokens], cell_sh[kHTokens];  // position (-1: no such token), page * 256 + row (-1: none)
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  const bool cached = p.cache.k_codes != nullptr;
  pdl_wait();
  pdl_launch_dependents();

  float gq[E], gk[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    gq[i] = p.gamma_q ? p.gamma_q[l * E + i] : 1.f;
    gk[i] = p.gamma_k ? p.gamma_k[l * E + i] : 1.f;
  }
  const int pairs = p.rope_dims / 2, rope_at = D - p.rope_dims;

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kHTokens; t0 < p.T;
       t0 += static_cast<int64_t>(P.tok_blocks) * kHTokens) {
    const int nt = p.T - t0 < kHTokens ? static_cast<int>(p.T - t0) : kHTokens;
    // the sequence of the first token: as many as end at or before it
    __syncthreads();
    if (tid == 0) first_sh = 0;
    __syncthreads();
    int before = 0;
    for (int i = tid; i < p.B; i += kHThreads) before += p.cu_seqlens[i + 1] <= t0;
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if ((tid & 31) == 0 && before) atomicAdd(&first_sh, before);
    __syncthreads();
    if (tid < nt) {
      const int64_t t = t0 + tid;
      int s = first_sh;
      while (s < p.B && p.cu_seqlens[s + 1] <= t) ++s;
      int64_t pos = -1, cell = -1;
      if (s < p.B && p.cu_seqlens[s] <= t) {
        const int64_t start = p.start_pos[s];
        if (start < 0) {
          report(p.d_status, DSV4_DEV_BAD_LENGTH);
        } else {
          pos = start + (t - p.cu_seqlens[s]);
          if (cached) {
            const int64_t blk = pos / DSV4_PAGE_POSITIONS;
            if (blk >= p.cache.max_blocks) {
              report(p.d_status, DSV4_DEV_BAD_LENGTH);
            } else {
              const int page = p.cache.block_table[static_cast<int64_t>(s) * p.cache.max_blocks + blk];
              if (page < 0 || page >= p.cache.num_pages) report(p.d_status, DSV4_DEV_BAD_PAGE);
              else cell = static_cast<int64_t>(page) * DSV4_PAGE_POSITIONS + pos % DSV4_PAGE_POSITIONS;
            }
          }
        }
      }
      pos_sh[tid] = pos;
      cell_sh[tid] = cell;
    }
    __syncthreads();
    for (int i = tid; i < nt * pairs; i += kHThreads) {
      const int j = i / pairs, pr = i % pairs;
      float c = 1.f, s = 0.f;
      if (pos_sh[j] >= 0) rope_cos_sin(pos_sh[j], pr, p.rope_theta1, &c, &s);
      turn[j][pr] = make_float2(c, s);
    }
    __syncthreads();

    // rows (token j, row r): group y of the grid takes every row_split-th set of G rows
    const int total = nt * P.rows;
    for (int base = static_cast<int>(blockIdx.y) * G; base < total; base += P.row_split * G) {
      const int it = base + g;
      const bool in = it < total;
      const int j = in ? it / P.rows : 0, r = in ? it % P.rows : 0;
      const int64_t t = t0 + j;
      const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.Hk;
      const int h = is_q ? r : (is_v ? r - p.Hq - p.Hk : r - p.Hq);
      const bool live = in && pos_sh[j] >= 0 && (is_q || !cached || cell_sh[j] >= 0);
      float x[E];
      if (live) {
        const void *src = is_q ? p.q : (is_v ? p.v : p.k);
        const int64_t stride = is_q ? p.q_stride : (is_v ? p.v_stride : p.k_stride);
        load_vals<E, F32>(src, t * stride + static_cast<int64_t>(h) * D + l * E, x);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = 0.f;
      }
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      if (!is_v) {
        if (is_q ? p.gamma_q != nullptr : p.gamma_k != nullptr) {
          const float inv = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
          for (int i = 0; i < E; ++i) x[i] *= inv * (is_q ? gq[i] : gk[i]);
        }
#pragma unroll
        for (int i = 0; i < E; i += 2) {
          const int d = l * E + i - rope_at;  // even: rope_dims, D and E are
          if (d >= 0) {
            const float2 cs = turn[j][d >> 1];
            const float a = x[i], b = x[i + 1];
            x[i] = a * cs.x - b * cs.y;
            x[i + 1] = a * cs.y + b * cs.x;
          }
        }
      }
      if (!cached || is_q) {
        if (live) {
          const int64_t off = (t * (is_q ? p.Hq : p.Hk) + h) * D + l * E;
          store_vals<E>(is_q ? p.q_out : p.k_out, p.out_dt, off, x);
        }
      }
      if (cached) {  // (every lane of the warp takes the shuffles)
        if constexpr (D <= 128) {
          uint32_t am = 0;  // largest |x| as bits: a NaN is above infinity
#pragma unroll
          for (int i = 0; i < E; ++i) am = max(am, __float_as_uint(x[i]) & 0x7FFFFFFFu);
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
          am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
          if (live && !is_q) {
            const int sb = block_scale(__uint_as_float(am));
            const float up = __uint_as_float(static_cast<uint32_t>(sb == 255 ? 0 : 254 - sb) << 23);  // 2^-k
            uint32_t w = 0;
            if (sb != 255) {
#pragma unroll
              for (int i = 0; i < 4; ++i) w |= e2m1_pair(x[2 * i] * up, x[2 * i + 1] * up) << (8 * i);
            }
            const int64_t cell = cell_sh[j];
            const int64_t row = ((cell / DSV4_PAGE_POSITIONS) * p.Hk + h) * DSV4_PAGE_POSITIONS +
                                cell % DSV4_PAGE_POSITIONS;
            reinterpret_cast<uint32_t *>((is_v ? p.cache.v_codes : p.cache.k_codes) + row * (D / 2))[l] = w;
            if ((l & 3) == 0) (is_v ? p.cache.v_scales : p.cache.k_scales)[row * (D / kKv4Block) + l / 4] = sb;
            uint16_t *stored = is_v ? p.v_stored : p.k_stored;
            if (stored) {
              const float sc = __uint_as_float(sb == 255 ? 0x7FC00000u : static_cast<uint32_t>(sb) << 23);
              float y[E];
#pragma unroll
              for (int i = 0; i < E; ++i) y[i] = e2m1_to_float((w >> (4 * i)) & 15u) * sc;
              store_vals<E>(stored, DSV4_BF16, (t * p.Hk + h) * D + l * E, y);
            }
          }
        }
      }
    }
  }
}

template <bool F32>
cudaError_t launch_typed(HeadsParams &P, cudaStream_t st) {
  const int D = P.a.D;
  const int G = kHThreads / (D <= 256 ? D / 8 : 32);
  const int steps = (P.a.T + kHTokens - 1) / kHTokens;
  // Few tokens: the rows of a step spread over blocks, one set of G rows each, until the card
  // is filled; many tokens: one block takes all rows of a step (the angles once), and blocks
  // walk over the steps.
  const int per_step = (kHTokens < P.a.T ? kHTokens : P.a.T) * P.rows;
  const int sets = (per_step + G - 1) / G;
  const int want = sm_count() * 8;
  P.tok_blocks = steps < want ? steps : want;
  int split = want / P.tok_blocks;
  split = split < 1 ? 1 : (split > sets ? sets : split);
  P.row_split = split;
  const dim3 grid(P.tok_blocks, split);
  switch (D) {
    case 64: return launch_pdl(kv4_heads_kernel<64, F32>, grid, dim3(kHThreads), 0, st, 1, P);
    case 128: return launch_pdl(kv4_heads_kernel<128, F32>, grid, dim3(kHThreads), 0, st, 1, P);
    case 256: return launch_pdl(kv4_heads_kernel<256, F32>, grid, dim3(kHThreads), 0, st, 1, P);
    case 512: return launch_pdl(kv4_heads_kernel<512, F32>, grid, dim3(kHThreads), 0, st, 1, P);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv4_heads(const Kv4HeadsLaunch &q, cudaStream_t st) {
  HeadsParams P{};
  P.a = q;
  P.a.rope_theta1 = rope_theta1(q.rope_base, q.rope_dims);
  P.rows = q.Hq + q.Hk + (q.cache.k_codes ? q.Hk : 0);
  return q.in_dt == DSV4_F32 ? launch_typed<true>(P, st) : launch_typed<false>(P, st);
}

}  // namespace dsv4
