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
// One pass, bound by memory: a token's rows are its query heads, key heads and value heads.
// D / 16 neighbouring lanes hold one row, each two pieces of 8 values half a row apart (with half of the
// channels rotated, no lane works on the other half in vain), so the row's sum of squares and a block's amax are a few
// shuffles. A block of 256 threads takes up to eight tokens at a time, with two to three rows per thread on
// their way into shared memory (cp.async, each thread its own pieces, so nothing waits for anything but its
// own data); the angles of a token are worked out once, by one thread per pair and token, and shared by all its heads.
//
// Measured: 8 x 4096 tokens of 64 query and 8 key heads of 128 channels in bf16 197 us (1.21 GB, 93% of the measured copy
// rate), appended with 8 value heads 222 us (1.38 GB, 95%), both captured; as calls among others 212 us (87%) and 250 us (84%).
// As many bytes of 256 or 512 channels 225 us, in float32 280 us at 128 channels and 300 us at 256 and 512 (two turns
// of rows are on their way there, not three).
//
// Rounding to 4 bits makes a whole step out of one bit of float32 next to a border, so the float32 part keeps the order of the
// plain float32 program that it is compared with (perf/operators.py), whose row sums go by four neighbours in turn at 128 channels
// and by channels 32 apart at 64, then halves onto halves: codes next to a border then agree. 256 and 512 channels, which are not
// rounded to 4 bits, take the order of 128. Squares are rounded, then summed; x * (1 / rms) * gamma; products of the rotation
// are rounded before their difference; angle, sine and cosine in float64.
#include <type_traits>

#include "kv4_device.cuh"

namespace dsv4 {

namespace {

constexpr int kHThreads = 256;
// tokens of a block's step, at most (512 channels: by shared memory)
__host__ __device__ constexpr int step_tokens(int D) { return D <= 256 ? 8 : 4; }

struct HeadsParams {
  Kv4HeadsLaunch a;
  int row_split;   // blocks along y, each on every row_split-th group of rows
  int tok_blocks;  // blocks along x
  int step;        // tokens of a block's step
  // of query rows and of key rows: heads, ceil(2^32 / heads), and S = row_split * G = dj * heads + dh
  int heads[2], dj[2], dh[2];
  uint32_t per_head[2], per_split;
};

// a / b by its reciprocal m = ceil(2^32 / b): exact while a * b < 2^32 (rows of a step, below 2^17, over heads up to
// 2^14; sets of rows, below 2^18, over at most some hundred blocks)
__device__ __forceinline__ int over(int a, int b, uint32_t m) { return b == 1 ? a : static_cast<int>(__umulhi(a, m)); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a lane's two pieces of 8 values of a row as they lie in memory, and as floats
template <bool F32>
struct Raw {
  static constexpr int kWords = F32 ? 4 : 2;  // 16 bytes each, half of them a piece's
  uint4 w[kWords];
  __device__ __forceinline__ void values(float (&x)[16]) const {
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

// eight values x[0..7] at element `off`
__device__ __forceinline__ void store_piece(void *base, dsv4_dtype dt, int64_t off, const float *x) {
  if (dt == DSV4_F32) {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + off);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + off) =
        make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
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

// Sum over a row of the squares x_i^2, each rounded, in the order the file's head gives: a lane's two pieces and
// the L = D / 16 lanes of the row. An exchange in which each lane keeps half of its columns takes half the shuffles.
template <int D>
__device__ __forceinline__ float sum_squares(const float (&x)[16]) {
  constexpr uint32_t kAll = 0xFFFFFFFFu;
  float q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) q[i] = __fmul_rn(x[i], x[i]);
  if constexpr (D == 64) {  // 32 columns of two channels 32 apart: a lane's pieces; lane l has columns 8 l ..
    const int l = threadIdx.x & 3;
    float d[4], e[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] += q[i + 8];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // columns 16 apart: lanes 2 apart
      d[i] = ((l & 2) ? q[i + 4] : q[i]) + __shfl_xor_sync(kAll, (l & 2) ? q[i] : q[i + 4], 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)  // 8 apart: neighbouring lanes
      e[i] = ((l & 1) ? d[i + 2] : d[i]) + __shfl_xor_sync(kAll, (l & 1) ? d[i] : d[i + 2], 1);
    // the lane has two of the eight sums that are left, the others' numbers are in its lane bits: 4 apart, 2, 1
#pragma unroll
    for (int o = 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < 2; ++i) e[i] += __shfl_xor_sync(kAll, e[i], o);
    return e[0] + e[1];
  } else {  // columns of four neighbours: four a lane
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = ((q[4 * i] + q[4 * i + 1]) + q[4 * i + 2]) + q[4 * i + 3];
    c[0] += c[2];  // half a row apart
    c[1] += c[3];
    constexpr int L = D / 16;
    const bool up = threadIdx.x & (L / 2);
    float s = (up ? c[1] : c[0]) + __shfl_xor_sync(kAll, up ? c[0] : c[1], L / 2);
#pragma unroll
    for (int o = L / 4; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    return s + __shfl_xor_sync(kAll, s, L / 2);
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sine and cosine of `a` (|a| below 2^48: the entry points see to it), to about 1e-13 absolute beside the angle's own rounding, rounded once to
// float32: the nearest multiple k of pi/2 is taken off with two constants (pi/2 to 107 bits), the rest, within pi/4, goes
// into the Taylor polynomials up to r^13 and r^14 (next terms 2e-14 and 1e-15), and k's low bits turn the quadrant.
// (The library's float64 sincos, which also reduces angles beyond that range, took a one-token call from 4.2 to 4.4 us.)
__device__ __forceinline__ float2 cos_sin(double a) {
  constexpr double kHi = 1.5707963267948966, kLo = 6.123233995736766e-17, kInv = 0.6366197723675814;
  const double k = rint(a * kInv);
  const double r = fma(-k, kLo, fma(-k, kHi, a)), q = r * r;
  double s = fma(q, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  s = fma(s, q, 1.0 / 362880.0);
  s = fma(s, q, -1.0 / 5040.0);
  s = fma(s, q, 1.0 / 120.0);
  s = fma(s, q, -1.0 / 6.0);
  s = fma(s * q, r, r);
  double c = fma(q, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  c = fma(c, q, -1.0 / 3628800.0);
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
  int H, dj, dh;
  __device__ __forceinline__ void begin(const HeadsParams &P, int which, int first, int total, int turns, int S) {
    H = P.heads[which];
    dj = P.dj[which];
    dh = P.dh[which];
    j = over(first, H, P.per_head[which]);
    h = first - j * H;
    left = turns - (first + (turns - 1) * S >= total);  // (the last turn may have no row for this thread)
  }
  __device__ __forceinline__ void next() {
    --left;
    j += dj;
    h += dh;
    if (h >= H) h -= H, ++j;
  }
};

template <int D, bool F32>
__global__ void __launch_bounds__(kHThreads, 3) kv4_heads_kernel(const __grid_constant__ HeadsParams P) {
  constexpr int L = D / 16;         // lanes of a row
  constexpr int G = kHThreads / L;  // rows of a block at a time
  constexpr int kSize = F32 ? 4 : 2;
  const Kv4HeadsLaunch &p = P.a;
  // of two neighbouring pairs both cosines, then both sines, of a token; of four neighbouring channels the even
  // ones' weights, then the odd ones', of queries and of keys: as the packed arithmetic takes them
  __shared__ __align__(16) float turn[step_tokens(D)][D];
  __shared__ __align__(16) float gamma[2][D];
  __shared__ int64_t pos_sh[step_tokens(D)], cell_sh[step_tokens(D)];  // position (-1: no such token), page * 256 + row (-1: none)
  const int tid = threadIdx.x, l = tid % L, g = tid / L;
  const bool cached = p.cache.k_codes != nullptr;
  const int pairs = p.rope_dims / 2, rope_at = D - p.rope_dims;
  const bool aligned = rope_at % 8 == 0;  // a lane's pairs are all turned or none, and start at a multiple of four
  pdl_wait();  // (the only kernel of its call: it releases nothing early, the next call may read these rows at its start)
  for (int i = tid; i < 2 * D; i += kHThreads) {
    const float *src = i < D ? p.gamma_q : p.gamma_k;
    const int d = i % D;
    gamma[i / D][(d & ~3) + (d & 1) * 2 + (d >> 1 & 1)] = src ? src[d] : 1.f;
  }
  const int first = static_cast<int>(blockIdx.y) * G + g, S = P.row_split * G;
  using Row = Raw<F32>;
  constexpr int kDepth = F32 ? 2 : 3;  // turns whose rows are on their way
  __shared__ uint4 ring[kDepth][Row::kWords][kHThreads];

  // one row: x in, results out
  auto finish = [&](auto kind_tag, const Row &raw, const RowWalk &w, bool in, int64_t t0, int64_t out) {
    constexpr int kKind = decltype(kind_tag)::value;
    float x[16];
    raw.values(x);
    bool live = in && pos_sh[w.j] >= 0;
    if (kKind != kQuery && cached) live = live && cell_sh[w.j] >= 0;
    if constexpr (kKind != kValue) {
      if ((kKind == kQuery ? p.gamma_q : p.gamma_k) != nullptr) {
        const float inv = rsqrtf(__fadd_rn(sum_squares<D>(x) * (1.f / D), p.eps));
        const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(&gamma[kKind][i / 8 * (D / 2) + l * 8 + i % 8]);
          unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(x[i], x[i + 2]), inv2), m.x), x[i], x[i + 2]);
          unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(x[i + 1], x[i + 3]), inv2), m.y), x[i + 1], x[i + 3]);
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int d0 = c * (D / 2) + l * 8 - rope_at;  // even: rope_dims and D are
        if (aligned) {
          if (d0 >= 0) {
            const ulonglong2 *cs = reinterpret_cast<const ulonglong2 *>(&turn[w.j][d0]);
#pragma unroll
            for (int i = 8 * c; i < 8 * c + 8; i += 4) {
              const ulonglong2 v = cs[(i & 4) / 4];
              const uint64_t a = pack_f32x2(x[i], x[i + 2]), b = pack_f32x2(x[i + 1], x[i + 3]);
              // (sums one by one: a packed sum of packed products is made one operation, .rn or not)
              float p0, p1, q0, q1, r0, r1, s0, s1;
              unpack_f32x2(mul_f32x2(a, v.x), p0, p1);
              unpack_f32x2(mul_f32x2(b, v.y), q0, q1);
              unpack_f32x2(mul_f32x2(a, v.y), r0, r1);
              unpack_f32x2(mul_f32x2(b, v.x), s0, s1);
              x[i] = __fsub_rn(p0, q0), x[i + 2] = __fsub_rn(p1, q1);
              x[i + 1] = __fadd_rn(r0, s0), x[i + 3] = __fadd_rn(r1, s1);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; i += 2)
            if (d0 + i >= 0) {
              const int pr = (d0 + i) >> 1;
              const float co = turn[w.j][(pr >> 1) * 4 + (pr & 1)], si = turn[w.j][(pr >> 1) * 4 + (pr & 1) + 2];
              const float a = x[8 * c + i], b = x[8 * c + i + 1];
              x[8 * c + i] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si));
              x[8 * c + i + 1] = __fadd_rn(__fmul_rn(a, si), __fmul_rn(b, co));
            }
        }
      }
      if (kKind == kQuery || !cached) {
        if (live) {
          store_piece(kKind == kQuery ? p.q_out : p.k_out, p.out_dt, out, x);
          store_piece(kKind == kQuery ? p.q_out : p.k_out, p.out_dt, out + D / 2, x + 8);
        }
        return;
      }
    }
    if constexpr (D <= 128 && kKind != kQuery) {
      int64_t row = 0;
      if (live) {
        const int64_t cell = cell_sh[w.j];
        row = (cell / DSV4_PAGE_POSITIONS * p.Hk + w.h) * DSV4_PAGE_POSITIONS + cell % DSV4_PAGE_POSITIONS;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float *y = x + 8 * c;
        float am = fabsf(y[0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) am = max_nan(am, fabsf(y[i]));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max_nan(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        if (!live) continue;
        const int sb = block_scale(am);
        const float up = __uint_as_float(static_cast<uint32_t>(sb == 255 ? 0 : 254 - sb) << 23);  // 2^-k
        uint32_t code = 0;
        if (sb != 255) {
#pragma unroll
          for (int i = 0; i < 4; ++i) code |= e2m1_pair(y[2 * i] * up, y[2 * i + 1] * up) << (8 * i);
        }
        reinterpret_cast<uint32_t *>((kKind == kValue ? p.cache.v_codes : p.cache.k_codes) + row * (D / 2))[c * (D / 16) + l] = code;
        if ((l & 3) == 0)
          (kKind == kValue ? p.cache.v_scales : p.cache.k_scales)[row * (D / kKv4Block) + c * (D / 64) + l / 4] = sb;
        uint16_t *stored = kKind == kValue ? p.v_stored : p.k_stored;
        if (stored) {
          const float sc = __uint_as_float(sb == 255 ? 0x7FC00000u : static_cast<uint32_t>(sb) << 23);
          uint32_t h[4];
          e2m1x8_to_half2(code, h);
          float z[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            z[2 * i] = f.x * sc, z[2 * i + 1] = f.y * sc;
          }
          store_piece(stored, DSV4_BF16, out + c * (D / 2), z);
        }
      }
    }
  };
  // turns of a kind: as many for every thread of the block (the row sums are warp-wide)
  auto turns_of = [&](int heads, int nt) {
    const int sets = (nt * heads + G - 1) / G - static_cast<int>(blockIdx.y);
    return sets > 0 ? over(sets + P.row_split - 1, P.row_split, P.per_split) : 0;
  };
  // The step's turns, all kinds in a row, are loaded kDepth ahead; `at` walks over the rows to be loaded.
  RowWalk at;
  int kind = 0, to_load = 0;  // turns of the kind still to be loaded
  const char *src = nullptr;
  int64_t stride = 0;
  auto load_kind = [&](int k, int nt, int64_t t0) {
    kind = k;
    const int heads = k == kQuery ? p.Hq : p.Hk;
    to_load = k == kValue && !cached ? 0 : turns_of(heads, nt);
    at.begin(P, k == kQuery ? 0 : 1, first, nt * heads, to_load, S);
    stride = (k == kQuery ? p.q_stride : (k == kKey ? p.k_stride : p.v_stride)) * kSize;
    src = static_cast<const char *>(k == kQuery ? p.q : (k == kKey ? p.k : p.v)) + t0 * stride + l * (8 * kSize);
  };
  auto load_turn = [&](int slot, int nt, int64_t t0) {
    while (to_load == 0 && kind < kValue) load_kind(kind + 1, nt, t0);
    if (to_load > 0) {
      if (at.left > 0) {
        const char *row = src + at.j * stride + at.h * (D * kSize);
        constexpr int kHalf = Row::kWords / 2;  // 16-byte words of a piece
#pragma unroll
        for (int i = 0; i < Row::kWords; ++i)
          cp_async16(&ring[slot][i][tid], row + i / kHalf * (D / 2 * kSize) + i % kHalf * 16);
      }
      at.next();
      --to_load;
    }
    cp_async_commit();
  };
  // all rows of one kind; `turn_no`: turns of the step so far
  auto pass = [&](auto kind_tag, int &turn_no, int nt, int64_t t0) {
    constexpr int kKind = decltype(kind_tag)::value;
    const int H = kKind == kQuery ? p.Hq : p.Hk;
    int n = turns_of(H, nt);
    RowWalk w;
    w.begin(P, kKind == kQuery ? 0 : 1, first, nt * H, n, S);
    int64_t out = (t0 * H + first) * D + l * 8;
    for (; n > 0; --n) {
      const int slot = turn_no % kDepth;
      ++turn_no;
      asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");  // this thread's part of the turn is there
      const bool in = w.left > 0;
      Row raw;
#pragma unroll
      for (int i = 0; i < Row::kWords; ++i) raw.w[i] = in ? ring[slot][i][tid] : make_uint4(0, 0, 0, 0);
      load_turn(slot, nt, t0);
      if (!in) w.j = 0;  // (no row in the last turn: the thread takes part in the warp's sums)
      finish(kind_tag, raw, w, in, t0, out);
      w.next();
      out += static_cast<int64_t>(S) * D;
    }
  };

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * P.step; t0 < p.T; t0 += static_cast<int64_t>(P.tok_blocks) * P.step) {
    const int nt = p.T - t0 < P.step ? static_cast<int>(p.T - t0) : P.step;
    // the first rows' loads, which need no position, are under way while the positions are looked up
    load_kind(kQuery, nt, t0);
#pragma unroll 1
    for (int i = 0; i < kDepth; ++i) load_turn(i, nt, t0);
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
        const float2 cs = cos_sin(static_cast<double>(pos_sh[j]) * th);
        turn[j][(pr >> 1) * 4 + (pr & 1)] = cs.x;
        turn[j][(pr >> 1) * 4 + (pr & 1) + 2] = cs.y;
      }
    }
    __syncthreads();
    int turn_no = 0;
    pass(std::integral_constant<int, kQuery>{}, turn_no, nt, t0);
    pass(std::integral_constant<int, kKey>{}, turn_no, nt, t0);
    if (cached) pass(std::integral_constant<int, kValue>{}, turn_no, nt, t0);
  }
  cp_async_wait_all();
}

template <bool F32>
cudaError_t launch_typed(HeadsParams &P, cudaStream_t st) {
  const int D = P.a.D;
  const int64_t G = kHThreads / (D / 16);  // rows of a block at a time
  // As many tokens a step, up to eight, as let all steps run at once (three blocks an SM); with fewer tokens than
  // that, a step's rows spread over blocks; with more, blocks walk over the steps.
  const int want = sm_count() * 3;
  const int step = (P.a.T + want - 1) / want;
  P.step = step > step_tokens(D) ? step_tokens(D) : step;
  const int steps = (P.a.T + P.step - 1) / P.step;
  const int64_t sets = (static_cast<int64_t>(P.step) * (P.a.Hq > P.a.Hk ? P.a.Hq : P.a.Hk) + G - 1) / G;
  P.tok_blocks = steps < want ? steps : want;
  const int64_t split = want / P.tok_blocks;
  P.row_split = static_cast<int>(split < 1 ? 1 : (split > sets ? sets : split));
  const int S = P.row_split * static_cast<int>(G);
  for (int k = 0; k < 2; ++k) {
    const int heads = k == 0 ? P.a.Hq : P.a.Hk;
    P.heads[k] = heads;
    if (heads == 0) continue;
    P.dj[k] = S / heads;
    P.dh[k] = S % heads;
    P.per_head[k] = static_cast<uint32_t>(((1ull << 32) + heads - 1) / heads);
  }
  P.per_split = static_cast<uint32_t>(((1ull << 32) + P.row_split - 1) / P.row_split);
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
