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
#include <type_traits>

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
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a lane's E values of a row as they lie in memory, and as floats
template <int E, bool F32>
struct Raw {
  static constexpr int kWords = F32 ? E / 4 : E / 8;  // 16 bytes each
  uint4 w[kWords];
  __device__ __forceinline__ void load(const void *base, int64_t off) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(base) + off * (F32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&x)[E]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (F32) x[4 * i + k] = __uint_as_float(v[k]);
        else x[8 * i + 2 * k] = bf16_lo(v[k]), x[8 * i + 2 * k + 1] = bf16_hi(v[k]);
      }
    }
  }
};

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
      p[i] = make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                        pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
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

// Sine and cosine of `a` (finite, |a| below 2^31), to about 1e-11 absolute, rounded once to float32: the nearest
// multiple k of pi/2 is taken off with two constants (pi/2 to 107 bits), the rest, within pi/4, goes into
// the Taylor polynomials up to r^11 and r^12 (next terms 7e-12 and 4e-13), and k's low bits turn the quadrant. The
// library's float64 sincos took the step of one token from 4.4 to 15 us where few pairs are worked out per block.
__device__ __forceinline__ float2 cos_sin(double a) {
  constexpr double kHi = 1.5707963267948966, kLo = 6.123233995736766e-17, kInv = 0.6366197723675814;
  const double k = rint(a * kInv);
  const double r = fma(-k, kLo, fma(-k, kHi, a)), q = r * r;
  double s = fma(q, -1.0 / 39916800.0, 1.0 / 362880.0);
  s = fma(s, q, -1.0 / 5040.0);
  s = fma(s, q, 1.0 / 120.0);
  s = fma(s, q, -1.0 / 6.0);
  s = fma(s * q, r, r);
  double c = fma(q, 1.0 / 479001600.0, -1.0 / 3628800.0);
  c = fma(c, q, 1.0 / 40320.0);
  c = fma(c, q, -1.0 / 720.0);
  c = fma(c, q, 1.0 / 24.0);
  c = fma(c, q, -0.5);
  c = fma(c, q, 1.0);
  const int n = static_cast<int>(static_cast<int64_t>(k)) & 3;
  const float fs = static_cast<float>(s), fc = static_cast<float>(c);
  const float x = (n & 1) ? fs : fc, y = (n & 1) ? fc : fs;
  return make_float2(n == 1 || n == 2 ? -x : x, n >= 2 ? -y : y);
}

enum { kQuery, kKey, kValue };

// A thread's rows of one kind in a step: row number it = first, first + S, ... below total, which is head it % H of
// token it / H. Divisions only at the start: the walk adds S = dj * H + dh.
struct RowWalk {
  int j, h, left;      // token of the step, head, rows still to come (this one included)
  int64_t in, out;     // element offsets of the row from the step's first token in the input and the dense output
  __device__ __forceinline__ void begin(int first, int S, int H, int total, int64_t stride, int D) {
    left = first < total ? (total - first + S - 1) / S : 0;
    j = first / H;
    h = first - j * H;
    in = j * stride + h * D;
    out = static_cast<int64_t>(first) * D;
  }
  __device__ __forceinline__ void next(int S, int dj, int dh, int H, int64_t stride, int D) {
    --left;
    j += dj;
    h += dh;
    in += dj * stride + dh * D;
    out += static_cast<int64_t>(S) * D;
    if (h >= H) {
      h -= H;
      ++j;
      in += stride - H * D;
    }
  }
};

template <int D, bool F32>
__global__ void __launch_bounds__(kHThreads, D <= 256 ? 4 : 3) kv4_heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int E = D <= 256 ? 8 : D / 32;  // values of a row per lane
  constexpr int L = D / E;                  // lanes of a row
  constexpr int G = kHThreads / L;          // rows of a block at a time
  const Kv4HeadsLaunch &p = P.a;
  __shared__ __align__(16) float2 turn[kHTokens][kHPairs];  // cos and sin of a token's pairs
  __shared__ __align__(16) float gamma[2][D];               // of queries and of keys
  __shared__ int64_t pos_sh[kHTokens], cell_sh[kHTokens];  // position (-1: no such token), page * 256 + row (-1: none)
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  const bool cached = p.cache.k_codes != nullptr;
  const int pairs = p.rope_dims / 2, rope_at = D - p.rope_dims;
  const bool aligned = rope_at % 8 == 0;  // a lane's pairs are all turned or none, and start at a multiple of four
  pdl_wait();
  pdl_launch_dependents();
  for (int i = tid; i < 2 * D; i += kHThreads) {
    const float *src = i < D ? p.gamma_q : p.gamma_k;
    gamma[i / D][i % D] = src ? src[i % D] : 1.f;
  }
  const int first = static_cast<int>(blockIdx.y) * G + g, S = P.row_split * G;
  const int djq = p.Hq ? S / p.Hq : 0, dhq = S - djq * p.Hq, djk = p.Hk ? S / p.Hk : 0, dhk = S - djk * p.Hk;

  using Row = Raw<E, F32>;
  // one row: x in, results out
  auto finish = [&](auto kind_tag, const Row &raw, const RowWalk &w, bool in, int64_t t0) {
    constexpr int kKind = decltype(kind_tag)::value;
    float x[E];
    raw.values(x);
    bool live = in && pos_sh[w.j] >= 0;
    if (kKind != kQuery && cached) live = live && cell_sh[w.j] >= 0;
    if constexpr (kKind != kValue) {
      if ((kKind == kQuery ? p.gamma_q : p.gamma_k) != nullptr) {
        const float inv = rsqrtf(__fadd_rn(sum_squares<D, E>(x) * (1.f / D), p.eps));
        const float4 *gm = reinterpret_cast<const float4 *>(&gamma[kKind][l * E]);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const float4 m = gm[i];
          x[4 * i] = __fmul_rn(__fmul_rn(x[4 * i], inv), m.x);
          x[4 * i + 1] = __fmul_rn(__fmul_rn(x[4 * i + 1], inv), m.y);
          x[4 * i + 2] = __fmul_rn(__fmul_rn(x[4 * i + 2], inv), m.z);
          x[4 * i + 3] = __fmul_rn(__fmul_rn(x[4 * i + 3], inv), m.w);
        }
      }
      auto rotate = [&](int i, float c, float s) {
        const float a = x[i], b = x[i + 1];
        x[i] = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        x[i + 1] = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
      };
      const int d0 = l * E - rope_at;  // even: rope_dims, D and E are
      if (aligned) {
        if (d0 + E > 0) {
          const float4 *cs = reinterpret_cast<const float4 *>(&turn[w.j][0]) + d0 / 4;
#pragma unroll
          for (int i = 0; i < E; i += 4) {
            if (E > 8 && d0 + i < 0) continue;  // (16 values of a lane, 8 of them turned)
            const float4 v = cs[i / 4];
            rotate(i, v.x, v.y);
            rotate(i + 2, v.z, v.w);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < E; i += 2)
          if (d0 + i >= 0) rotate(i, turn[w.j][(d0 + i) >> 1].x, turn[w.j][(d0 + i) >> 1].y);
      }
      if (kKind == kQuery || !cached) {
        const int64_t off = t0 * (kKind == kQuery ? p.Hq : p.Hk) * D + w.out + l * E;
        if (live) store_vals<E>(kKind == kQuery ? p.q_out : p.k_out, p.out_dt, off, x);
        return;
      }
    }
    if constexpr (D <= 128 && kKind != kQuery) {
      float am = fabsf(x[0]);
#pragma unroll
      for (int i = 1; i < E; ++i) am = max_nan(am, fabsf(x[i]));
      am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
      am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
      if (live) {
        const int sb = block_scale(am);
        const float up = __uint_as_float(static_cast<uint32_t>(sb == 255 ? 0 : 254 - sb) << 23);  // 2^-k
        uint32_t c = 0;
        if (sb != 255) {
#pragma unroll
          for (int i = 0; i < 4; ++i) c |= e2m1_pair(x[2 * i] * up, x[2 * i + 1] * up) << (8 * i);
        }
        const int64_t cell = cell_sh[w.j];
        const int64_t row = (cell / DSV4_PAGE_POSITIONS * p.Hk + w.h) * DSV4_PAGE_POSITIONS + cell % DSV4_PAGE_POSITIONS;
        reinterpret_cast<uint32_t *>((kKind == kValue ? p.cache.v_codes : p.cache.k_codes) + row * (D / 2))[l] = c;
        if ((l & 3) == 0) (kKind == kValue ? p.cache.v_scales : p.cache.k_scales)[row * (D / kKv4Block) + l / 4] = sb;
        uint16_t *stored = kKind == kValue ? p.v_stored : p.k_stored;
        if (stored) {
          const float sc = __uint_as_float(sb == 255 ? 0x7FC00000u : static_cast<uint32_t>(sb) << 23);
          uint32_t h[4];
          e2m1x8_to_half2(c, h);
          float y[E];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            y[2 * i] = f.x * sc, y[2 * i + 1] = f.y * sc;
          }
          store_vals<E>(stored, DSV4_BF16, t0 * p.Hk * D + w.out + l * E, y);
        }
      }
    }
  };
  // all rows of one kind; `raw` holds the first
  auto pass = [&](auto kind_tag, Row raw, RowWalk w, int total, int64_t t0) {
    constexpr int kKind = decltype(kind_tag)::value;
    const int H = kKind == kQuery ? p.Hq : p.Hk, dj = kKind == kQuery ? djq : djk, dh = kKind == kQuery ? dhq : dhk;
    const int64_t stride = kKind == kQuery ? p.q_stride : (kKind == kKey ? p.k_stride : p.v_stride);
    const void *src = kKind == kQuery ? p.q : (kKind == kKey ? p.k : p.v);
    const int64_t base = t0 * stride + l * E;
    // as many turns for every thread of the block: the row sums are warp-wide
    for (int at = static_cast<int>(blockIdx.y) * G; at < total; at += S) {
      RowWalk n = w;
      n.next(S, dj, dh, H, stride, D);
      Row next;
      if (n.left > 0) next.load(src, base + n.in);
      else next.zero();
      const bool in = w.left > 0;
      if (!in) w.j = 0;  // (a thread without a row in the last turn)
      finish(kind_tag, raw, w, in, t0);
      raw = next;
      w = n;
    }
  };

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.step; t0 < p.T; t0 += static_cast<int64_t>(P.tok_blocks) * P.step) {
    const int nt = p.T - t0 < P.step ? static_cast<int>(p.T - t0) : P.step;
    // the first rows' loads, which need no position, are under way while the positions are looked up
    RowWalk wq{}, wk{}, wv{};
    Row rq, rk, rv;
    rq.zero(), rk.zero(), rv.zero();
    if (p.Hq) wq.begin(first, S, p.Hq, nt * p.Hq, p.q_stride, D);
    if (p.Hk) wk.begin(first, S, p.Hk, nt * p.Hk, p.k_stride, D);
    if (wq.left > 0) rq.load(p.q, t0 * p.q_stride + l * E + wq.in);
    if (wk.left > 0) rk.load(p.k, t0 * p.k_stride + l * E + wk.in);
    if (cached) {
      wv.begin(first, S, p.Hk, nt * p.Hk, p.v_stride, D);
      if (wv.left > 0) rv.load(p.v, t0 * p.v_stride + l * E + wv.in);
    }
    __syncthreads();  // (the step before has read its positions and angles)
    if (tid < 32) {
      // The sequence of the step's first token: as many as end at or before it, found 32 probes at a time.
      int lo = 0, hi = p.B;
      while (hi > lo) {
        const int width = (hi - lo + 31) / 32, at = lo + (tid + 1) * width - 1;
        const int c = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && p.cu_seqlens[at + 1] <= t0));
        hi = min(hi, lo + (c + 1) * width - 1);
        lo += c * width;
      }
      if (tid < nt) {
        const int64_t t = t0 + tid;
        int s = lo;
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
    }
    __syncthreads();
    for (int i = tid; i < nt * pairs; i += kHThreads) {
      const int j = i / pairs, pr = i % pairs;
      if (pos_sh[j] >= 0) {
        double th = 1.0, b = p.rope_theta1;  // theta1^pr by binary powering
        for (int e = pr; e; e >>= 1) {
          if (e & 1) th *= b;
          b *= b;
        }
        turn[j][pr] = cos_sin(static_cast<double>(pos_sh[j]) * th);
      }
    }
    __syncthreads();
    pass(std::integral_constant<int, kQuery>{}, rq, wq, nt * p.Hq, t0);
    pass(std::integral_constant<int, kKey>{}, rk, wk, nt * p.Hk, t0);
    if (cached) pass(std::integral_constant<int, kValue>{}, rv, wv, nt * p.Hk, t0);
  }
}

template <bool F32>
cudaError_t launch_typed(HeadsParams &P, cudaStream_t st) {
  const int D = P.a.D;
  const int64_t G = kHThreads / (D <= 256 ? D / 8 : 32);  // rows of a block at a time
  // As many tokens a step, up to eight, as let all steps run at once (four blocks an SM); with fewer tokens than
  // that, a step's rows spread over blocks; with more, blocks walk over the steps.
  const int want = sm_count() * 4;
  const int step = (P.a.T + want - 1) / want;
  P.step = step > kHTokens ? kHTokens : step;
  const int steps = (P.a.T + P.step - 1) / P.step;
  const int64_t sets = (static_cast<int64_t>(P.step) * (P.a.Hq > P.a.Hk ? P.a.Hq : P.a.Hk) + G - 1) / G;
  P.tok_blocks = steps < want ? steps : want;
  const int64_t split = want / P.tok_blocks;
  P.row_split = static_cast<int>(split < 1 ? 1 : (split > sets ? sets : split));
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
