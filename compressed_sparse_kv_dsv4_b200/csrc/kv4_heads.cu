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
// up to eight tokens at a time, two rows per thread in flight; the angles of a token are
// worked out once, by one thread per pair and token, and shared by all its heads.
//
// Rounding to 4 bits makes a whole step out of one bit of float32 next to a border, so the float32
// part is kept in the textbook's order: squares rounded, then summed (four neighbours in turn at 128
// channels, channels 32 apart at 64; then halves onto halves), x * (1 / rms) * gamma, products of the
// rotation rounded before their difference; angle, sine and cosine in float64.
#include "kv4_device.cuh"

namespace dsv4 {

namespace {

constexpr int kHThreads = 256;
constexpr int kHTokens = 8;   // tokens of a block's step, at most
constexpr int kHPairs = 256;  // rotated pairs at most (D <= 512)

struct HeadsParams {
  Kv4HeadsLaunch a;
  int row_split;   // blocks along y, each on every row_split-th group of rows
  int tok_blocks;  // blocks along x
  int step;        // tokens of a block's step
  uint32_t div_q, div_k;  // ceil(2^32 / Hq), ceil(2^32 / Hk): row numbers (below 2^17) over heads (up to 2^14)
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

// Sum over a row of the squares x_i^2, each rounded, in the order the file's head gives: a lane's E values
// and the L lanes of the row.
template <int D, int E>
__device__ __forceinline__ float sum_squares(const float (&x)[E]) {
  constexpr int L = D / E;
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  if constexpr (D == 64) {  // 32 columns of two, 32 channels apart: lanes 4 apart hold a column's two
    const int l = threadIdx.x & 7;
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __fmul_rn(x[i], x[i]);
    // each exchange keeps half of the columns: lane bit 2 the first or last four, then two, then one
    float d[4], e[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float send = (l & 4) ? c[i] : c[i + 4], keep = (l & 4) ? c[i + 4] : c[i];
      d[i] = keep + __shfl_xor_sync(kAll, send, 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // columns 16 apart: lanes 2 apart
      const float send = (l & 2) ? d[i] : d[i + 2], keep = (l & 2) ? d[i + 2] : d[i];
      e[i] = keep + __shfl_xor_sync(kAll, send, 2);
    }
    const float send = (l & 1) ? e[0] : e[1], keep = (l & 1) ? e[1] : e[0];
    float s = keep + __shfl_xor_sync(kAll, send, 1);  // columns 8 apart: neighbouring lanes
    // lane l now has the column of eight whose bits are l's, high to low: 4, 2 and 1 apart
    s += __shfl_xor_sync(kAll, s, 4);
    s += __shfl_xor_sync(kAll, s, 2);
    return s + __shfl_xor_sync(kAll, s, 1);
  } else {  // columns of four neighbours: a lane's E / 4, then halves onto halves
    float c[E / 4];
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      c[i] = __fadd_rn(__fmul_rn(x[4 * i], x[4 * i]), __fmul_rn(x[4 * i + 1], x[4 * i + 1]));
      c[i] = __fadd_rn(c[i], __fmul_rn(x[4 * i + 2], x[4 * i + 2]));
      c[i] = __fadd_rn(c[i], __fmul_rn(x[4 * i + 3], x[4 * i + 3]));
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < E / 4; ++i) c[i] += __shfl_xor_sync(kAll, c[i], o);
#pragma unroll
    for (int o = E / 8; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) c[i] += c[i + o];
    return c[0];
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

template <int D, bool F32>
__global__ void __launch_bounds__(kHThreads, D <= 256 ? 4 : 3) kv4_heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int E = D <= 256 ? 8 : D / 32;  // values of a row per lane
  constexpr int L = D / E;                  // lanes of a row
  constexpr int G = kHThreads / L;          // rows of a block at a time
  const Kv4HeadsLaunch &p = P.a;
  __shared__ __align__(16) float2 turn[kHTokens][kHPairs];  // cos and sin of a token's pairs
  __shared__ __align__(16) float gamma[2][D];               // of queries and of keys
  __shared__ int first_sh;
  __shared__ int64_t pos_sh[kHTokens], cell_sh[kHTokens];  // position (-1: no such token), page * 256 + row (-1: none)
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  const bool cached = p.cache.k_codes != nullptr;
  const int pairs = p.rope_dims / 2, rope_at = D - p.rope_dims;
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < 2 * D; i += kHThreads) {
    const float *src = i < D ? p.gamma_q : p.gamma_k;
    gamma[i / D][i % D] = src ? src[i % D] : 1.f;
  }

  // Row number -> the row: query rows of the step's tokens first, then keys, then values.
  struct Row {
    int kind, j, h;  // 0 query, 1 key, 2 value (3: none); token of the step; head
  };
  auto row_of = [&](int it, int nt) {
    Row r;
    const int nq = nt * p.Hq, nk = nt * p.Hk;
    r.kind = it < nq ? 0 : (it < nq + nk ? 1 : (cached && it < nq + 2 * nk ? 2 : 3));
    const uint32_t at = r.kind == 0 ? it : (r.kind == 1 ? it - nq : (r.kind == 2 ? it - nq - nk : 0));
    r.j = r.kind == 3 ? 0 : static_cast<int>(r.kind == 0 ? __umulhi(at, P.div_q) : __umulhi(at, P.div_k));
    if ((r.kind == 0 ? p.Hq : p.Hk) == 1) r.j = static_cast<int>(at);  // (2^32 / 1 does not fit)
    r.h = static_cast<int>(at) - r.j * (r.kind == 0 ? p.Hq : p.Hk);
    return r;
  };
  auto load_row = [&](const Row &r, int64_t t0, float(&x)[E]) {
    if (r.kind == 3) {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = 0.f;
      return;
    }
    const void *src = r.kind == 0 ? p.q : (r.kind == 1 ? p.k : p.v);
    const int64_t stride = r.kind == 0 ? p.q_stride : (r.kind == 1 ? p.k_stride : p.v_stride);
    load_vals<E, F32>(src, (t0 + r.j) * stride + r.h * D + l * E, x);
  };
  auto finish_row = [&](const Row &r, int64_t t0, float(&x)[E]) {
    const float sum = sum_squares<D, E>(x);
    const bool live = r.kind < 3 && pos_sh[r.j] >= 0 && (r.kind == 0 || !cached || cell_sh[r.j] >= 0);
    const int64_t t = t0 + r.j;
    if (r.kind < 2) {
      if (r.kind == 0 ? p.gamma_q != nullptr : p.gamma_k != nullptr) {
        const float inv = rsqrtf(__fadd_rn(sum * (1.f / D), p.eps));
        const float4 *gm = reinterpret_cast<const float4 *>(&gamma[r.kind][l * E]);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const float4 w = gm[i];
          x[4 * i] = __fmul_rn(__fmul_rn(x[4 * i], inv), w.x);
          x[4 * i + 1] = __fmul_rn(__fmul_rn(x[4 * i + 1], inv), w.y);
          x[4 * i + 2] = __fmul_rn(__fmul_rn(x[4 * i + 2], inv), w.z);
          x[4 * i + 3] = __fmul_rn(__fmul_rn(x[4 * i + 3], inv), w.w);
        }
      }
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const int d = l * E + i - rope_at;  // even: rope_dims, D and E are
        if (d >= 0) {
          const float2 cs = turn[r.j][d >> 1];
          const float a = x[i], b = x[i + 1];
          x[i] = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
          x[i + 1] = __fadd_rn(__fmul_rn(a, cs.y), __fmul_rn(b, cs.x));
        }
      }
      if (r.kind == 0 || !cached) {
        if (live) {
          const int64_t off = (t * (r.kind == 0 ? p.Hq : p.Hk) + r.h) * D + l * E;
          store_vals<E>(r.kind == 0 ? p.q_out : p.k_out, p.out_dt, off, x);
        }
      }
    }
    if constexpr (D <= 128) {
      if (cached) {  // (every lane of the warp takes the shuffles)
        float am = fabsf(x[0]);
#pragma unroll
        for (int i = 1; i < E; ++i) am = max_nan(am, fabsf(x[i]));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        if (live && r.kind != 0) {
          const int sb = block_scale(am);
          const float up = __uint_as_float(static_cast<uint32_t>(sb == 255 ? 0 : 254 - sb) << 23);  // 2^-k
          uint32_t w = 0;
          if (sb != 255) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w |= e2m1_pair(x[2 * i] * up, x[2 * i + 1] * up) << (8 * i);
          }
          const int64_t cell = cell_sh[r.j];
          const int64_t row = ((cell / DSV4_PAGE_POSITIONS) * p.Hk + r.h) * DSV4_PAGE_POSITIONS + cell % DSV4_PAGE_POSITIONS;
          const bool is_v = r.kind == 2;
          reinterpret_cast<uint32_t *>((is_v ? p.cache.v_codes : p.cache.k_codes) + row * (D / 2))[l] = w;
          if ((l & 3) == 0) (is_v ? p.cache.v_scales : p.cache.k_scales)[row * (D / kKv4Block) + l / 4] = sb;
          uint16_t *stored = is_v ? p.v_stored : p.k_stored;
          if (stored) {
            const float sc = __uint_as_float(sb == 255 ? 0x7FC00000u : static_cast<uint32_t>(sb) << 23);
            uint32_t h[4];
            e2m1x8_to_half2(w, h);
            float y[E];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
              y[2 * i] = f.x * sc, y[2 * i + 1] = f.y * sc;
            }
            store_vals<E>(stored, DSV4_BF16, (t * p.Hk + r.h) * D + l * E, y);
          }
        }
      }
    }
  };

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.step; t0 < p.T; t0 += static_cast<int64_t>(P.tok_blocks) * P.step) {
    const int nt = p.T - t0 < P.step ? static_cast<int>(p.T - t0) : P.step;
    const int total = nt * (p.Hq + (cached ? 2 : 1) * p.Hk);
    // the first rows' loads, which need no position, are under way while the positions are looked up
    int base = static_cast<int>(blockIdx.y) * 2 * G;
    Row ra = row_of(base + g, nt), rb = row_of(base + G + g, nt);
    float xa[E], xb[E];
    load_row(ra, t0, xa);
    load_row(rb, t0, xb);
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
      double c = 1.0, s = 0.0;
      if (pos_sh[j] >= 0) {
        double th = 1.0, b = p.rope_theta1;  // theta1^pr by binary powering
        for (int e = pr; e; e >>= 1) {
          if (e & 1) th *= b;
          b *= b;
        }
        sincos(static_cast<double>(pos_sh[j]) * th, &s, &c);
      }
      turn[j][pr] = make_float2(static_cast<float>(c), static_cast<float>(s));
    }
    __syncthreads();

    // two rows per thread at a time; group y of the grid takes every row_split-th set of 2 G rows
    for (;;) {
      finish_row(ra, t0, xa);
      finish_row(rb, t0, xb);
      base += P.row_split * 2 * G;
      if (base >= total) break;
      ra = row_of(base + g, nt), rb = row_of(base + G + g, nt);
      load_row(ra, t0, xa);
      load_row(rb, t0, xb);
    }
  }
}

template <bool F32>
cudaError_t launch_typed(HeadsParams &P, cudaStream_t st) {
  const int D = P.a.D;
  const int64_t pass = 2 * (kHThreads / (D <= 256 ? D / 8 : 32));  // rows of a block at a time
  const int rows = P.a.Hq + (P.a.cache.k_codes ? 2 : 1) * P.a.Hk;
  // Few tokens: a token a step, its rows spread over blocks until the card is filled; many tokens: up to eight
  // a step, all their rows on one block (the lookups and angles once), and blocks walk over the steps.
  const int want = sm_count() * 8;
  const int step = P.a.T / want;
  P.step = step < 1 ? 1 : (step > kHTokens ? kHTokens : step);
  const int steps = (P.a.T + P.step - 1) / P.step;
  const int64_t sets = (static_cast<int64_t>(P.step) * rows + pass - 1) / pass;
  P.tok_blocks = steps < want ? steps : want;
  const int64_t split = want / P.tok_blocks;
  P.row_split = static_cast<int>(split < 1 ? 1 : (split > sets ? sets : split));
  P.div_q = P.a.Hq > 1 ? static_cast<uint32_t>(((1ull << 32) + P.a.Hq - 1) / P.a.Hq) : 0;
  P.div_k = P.a.Hk > 1 ? static_cast<uint32_t>(((1ull << 32) + P.a.Hk - 1) / P.a.Hk) : 0;
  const dim3 grid(P.tok_blocks, P.row_split);
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
  return q.in_dt == DSV4_F32 ? launch_typed<true>(P, st) : launch_typed<false>(P, st);
}

}  // namespace dsv4
