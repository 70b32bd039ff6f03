// Attention over the 4-bit key/value cache, rows in small tiles: decode steps, draft tokens.
//
// Query token i of sequence s sits at position p = start + i and sees positions 0..p:
//   o = sum_j softmax_j( scale * q . k_j ) v_j,   lse = ln sum_j exp( scale * q . k_j )
// The rows that share a key/value head's keys are the G = Hq / Hk query heads of each new token;
// a unit of work is a row tile of R = 8 NT of them, of one key/value head of one sequence.
//
// Bound by memory when the rows are few: each cached value is 4.25 bits and is used once per
// row tile. So all units' keys, in tiles of 64 (or 128), form one line that is cut into equal slices,
// one per CTA, whatever the sequences' lengths: every CTA reads the same number of bytes, and a
// long sequence is split over many CTAs. A unit that one CTA has whole is written directly; the
// parts of the others go through the workspace and kv4_combine_kernel joins them (a fixed
// order, so results do not depend on timing; where the line is cut depends on the batch).
//
// Inside a CTA each of four warps takes every fourth tile whole: it brings its tiles into two to four
// stages of its own, half a tile each, with bulk copies (codes and scales of a head's rows are contiguous within a page), and
// does the products, an online softmax of its own and the weighted sum of values in registers; the
// warps' sums are joined at the end of the slice's part of the unit. With no producer between them the warps
// meet only there, and sixteen of them fit an SM at 128 registers. What bounds the kernel is their
// instructions, some 1340 a tile of 16384 values at 128 channels (conversions, products with the scales,
// 64 matrix products): 263 us for four sequences of 262144 positions (1.14 GB, 66% of the measured copy rate), 195 us
// with the arithmetic left out. (The form further down, whose scores are made on the tensor cores, takes long contexts
// of up to eight rows at 128 channels: 233 us.)
// The matrix products are mma.sync m16n8k16 (fp16 operands, fp32 sums) with
// keys (S^T = K Q^T) and channels (O^T = V^T P^T) on the 16-row side and rows on the 8-column
// side: a decode step has G rows, far fewer than a tcgen05 tile's 128, and the operand is made in
// registers from 4-bit codes, where mma.sync takes it without a trip through shared memory.
//  - Codes become fp16 pairs with the hardware's e2m1x2 conversion; a product with the block's
//    power of two is exact (|value| <= 49152, a multiple of 2^-24).
//  - q (bf16) is scaled by a power of two per row into fp16's range, which is exact but for
//    elements 2^-39 below the row's largest.
//  - P is rounded to fp16 (relative 2^-11 / 2, of weights scaled by 2^14); its sum is fp32 of the
//    unrounded weights, so lse carries no rounding of P.
// The channel order of the products is free: a lane takes 16 consecutive bytes of a key's codes
// (K) and D/16 of a value's (V), and Q's fragments and the output's addresses follow that order.
// A value block with scale 255 (NaN) counts as zero in the product; the smallest such position is
// noted per block of channels and rows that see it become NaN at the end, so that a row for which
// the position is masked is not touched by it.
#include <type_traits>

#include "kv4_device.cuh"

namespace dsv4 {

namespace {

constexpr int kTile = 64;       // keys of a warp's turn
constexpr int kWarps = 4;
constexpr int kThreadsA = 32 * kWarps;
constexpr float kPOff = 14.f;   // weights are held times 2^14
constexpr int kMinKeysLog2 = 8; // keys of a slice, at least 256 (a tile for each warp)

struct AttnParams {
  Kv4AttnLaunch a;
  float *part_o;     // [2 slots][R][D] per CTA: unnormalised sums
  float2 *part_ml;   // [2 slots][R] per CTA: maximum (log2) and sum
  int ctas;
  int group;         // query heads of a key/value head
  int key_log2;      // keys of a tile of the line: 64 or 128
};

// ---------------------------------------------------------------- the line of work

// a / b where both are >= 0 and mostly below 2^32 (a 64-bit division takes some hundred instructions)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

struct Line {
  const Kv4AttnLaunch *p;
  int G, R, r_log2;  // rows of a tile: a power of two
  int key_log2;      // keys of a tile
  __device__ __forceinline__ int row_tiles(const Seq &q) const {
    return static_cast<int>((static_cast<int64_t>(q.len) * G + R - 1) >> r_log2);
  }
  __device__ __forceinline__ int tiles(const Seq &q) const { return (q.n + (1 << key_log2) - 1) >> key_log2; }
  __device__ __forceinline__ int64_t weight(int s, bool tell = false) const {
    Seq q;
    if (!seq_info(*p, s, &q, tell)) return 0;
    return static_cast<int64_t>(p->Hk) * row_tiles(q) * tiles(q);
  }
};

// prefix[i]: tiles of the sequences before i * chunk; prefix[n]: all. Called by all `n` threads of
// the block (n a multiple of 32, up to 1024).
__device__ __forceinline__ int64_t line_prefix(const Line &ln, int n, int chunk, int64_t *prefix, int64_t *warp_sums) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine = 0;
  for (int i = 0; i < chunk; ++i) {
    const int64_t s = static_cast<int64_t>(tid) * chunk + i;
    if (s < ln.p->B) mine += ln.weight(static_cast<int>(s), blockIdx.x == 0);
  }
  int64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += up;
  }
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int64_t base = 0, all = 0;
  for (int w = 0; w < n / 32; ++w) {
    if (w < warp) base += warp_sums[w];
    all += warp_sums[w];
  }
  prefix[tid] = base + inc - mine;
  if (tid == n - 1) prefix[n] = all;
  __syncthreads();
  return all;
}

// Walks the units of [at, end) of the line. Every role of a CTA walks the same one.
struct Walk {
  Line ln;
  int64_t at, end;
  int s, row_tiles, tiles, kvh, rt;  // the unit that `at` lies in
  int tile;                          // and the tile in it
  Seq q;

  __device__ __forceinline__ void begin(const Line &line, const int64_t *prefix, int n, int chunk, int64_t from,
                                        int64_t to) {
    ln = line;
    at = from;
    end = to;
    int lo = 0, hi = n;  // the last thread's chunk that starts at or before `from`
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (prefix[mid] <= from) lo = mid;
      else hi = mid;
    }
    int64_t base = prefix[lo];
    s = lo * chunk;
    for (;; ++s) {
      const int64_t w = ln.weight(s);
      if (base + w > from) break;
      base += w;
    }
    load(from - base);
  }
  __device__ __forceinline__ void load(int64_t off) {
    seq_info(*ln.p, s, &q, false);
    row_tiles = ln.row_tiles(q);
    tiles = ln.tiles(q);
    const int64_t unit = quotient(off, tiles), head = quotient(unit, row_tiles);
    tile = static_cast<int>(off - unit * tiles);
    kvh = static_cast<int>(head);
    rt = static_cast<int>(unit - head * row_tiles);
  }
  // the part of the current unit that lies in the slice: tiles [tile, stop)
  __device__ __forceinline__ int stop() const {
    const int64_t left = end - at;
    return left < tiles - tile ? tile + static_cast<int>(left) : tiles;
  }
  __device__ __forceinline__ bool next() {  // false: the slice is done
    at += stop() - tile;
    if (at >= end) return false;
    tile = 0;
    if (++rt == row_tiles) {
      rt = 0;
      if (++kvh == ln.p->Hk) {
        kvh = 0;
        do ++s;
        while (ln.weight(s) == 0);
        load(0);
      }
    }
    return true;
  }
  // positions that any row of the unit sees
  __device__ __forceinline__ int unit_limit() const {
    const int64_t last = min(static_cast<int64_t>(q.len) * ln.G, static_cast<int64_t>(rt + 1) * ln.R) - 1;
    return min(q.n, q.start + static_cast<int>(quotient(last, ln.G)) + 1);
  }
  // positions that row r of the unit sees (0: there is no such row)
  __device__ __forceinline__ int row_limit(int r) const {
    const int64_t row = static_cast<int64_t>(rt) * ln.R + r;
    if (row >= static_cast<int64_t>(q.len) * ln.G) return 0;
    return min(q.n, q.start + static_cast<int>(quotient(row, ln.G)) + 1);
  }
  // [token][head] index of row r
  __device__ __forceinline__ int64_t row_index(int r) const {
    const int64_t row = static_cast<int64_t>(rt) * ln.R + r;
    const int64_t i = quotient(row, ln.G);
    return (q.tok0 + i) * ln.p->Hq + kvh * ln.G + (row - i * ln.G);
  }
};

__device__ __forceinline__ int64_t slice_at(int64_t all, int ctas, int c) {
  // (all is at most 2^31 tokens' row tiles times 2^25 tiles; the quotient form stays in 64 bits)
  const int64_t each = quotient(all, ctas);
  return each * c + quotient((all - each * ctas) * c, ctas);
}
__device__ __forceinline__ int slices(int64_t all, int ctas, int key_log2) {
  const int least_log2 = kMinKeysLog2 - key_log2;
  const int64_t most = (all + (1 << least_log2) - 1) >> least_log2;
  return most < ctas ? static_cast<int>(most) : ctas;
}

// ---------------------------------------------------------------- fragments

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// four 8x8 matrices of 16-bit values from shared memory; lane i gives the address of row i % 8 of matrix i / 8
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Row of a 16-key group that fragment row g (0..7) stands for: neighbouring pairs differ in parity
// (a quarter warp's 16-byte reads of two 64-byte rows touch all banks), and so do the even ones
// (the four rows of a value read meet two to a bank, not four).
__device__ __forceinline__ int key_of(int g) { return (g & 4) + ((0x2130 >> (4 * (g & 3))) & 3); }

// CTAs of an SM, at 128, 168 or 255 registers a thread. (Four with eight rows at 128 channels against three: 263 us and
// 272 us for four sequences of 262144; but with 16 rows the sums spill, 42 us against 34 us for draft tokens.)
constexpr int resident_ctas(int D, int NT) { return NT == 1 ? 4 : (D == 64 ? 3 : 2); }

template <int D, int NT>
struct StepShape {
  static constexpr int kCodes = kTile * D / 2, kScales = kTile * D / kKv4Block;
  static constexpr int kStages = D == 64 ? 4 : (NT == 1 ? 2 : 3);  // of a warp, half a tile each
  static constexpr int kResident = resident_ctas(D, NT);
};

template <int D, int NT>
struct alignas(128) AttnSmem {
  using Sh = StepShape<D, NT>;
  struct alignas(128) Stage {
    uint8_t c[Sh::kCodes], s[Sh::kScales];
  } stage[kWarps][Sh::kStages];
  // Q as the first product's fragments: of row r, 8 values for each step and half of it, two per lane of the four
  // (rows 16 bytes more than a multiple of 128 apart: the eight rows of a matrix meet different banks)
  uint16_t q[8 * NT][D + 8];
  float o[kWarps][8 * NT][D + 4];  // the warps' sums, joined at the end of a unit's part
  float2 ml[kWarps][8 * NT];
  int64_t index[8 * NT];           // [token][head] of the unit's rows
  int lim[8 * NT];                 // positions that they see (0: no such row)
  int64_t prefix[kThreadsA + 1], warp_sums[kThreadsA / 32];
  uint64_t full[kWarps][Sh::kStages];
  int bad[kWarps][Sh::kStages];    // the stage's page does not exist
  int nan_at[D / kKv4Block];       // smallest position with a NaN value block
  int abort_flag;
};

// The warps' sums of a unit's part together, by all 32 kWarps threads: to the output where the part is the whole unit.
template <int D, int R, class Smem>
__device__ __forceinline__ void join_part(const AttnParams &P, Smem &S, const Walk &w, int stop) {
  const Kv4AttnLaunch &p = P.a;
  const int tid = threadIdx.x;
  const bool whole = w.tile == 0 && stop == w.tiles;
  const int part = 2 * static_cast<int>(blockIdx.x) + (w.tile == 0 ? 1 : 0);
  constexpr int V4 = D / 4;
  for (int e = tid; e < R * V4; e += 32 * kWarps) {
    const int r = e / V4, d = e % V4 * 4;
    const int rl = S.lim[r];
    if (rl == 0) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, S.ml[k][r].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const float2 ml = S.ml[k][r];
      const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - mx);
      const float4 v = *reinterpret_cast<const float4 *>(&S.o[k][r][d]);
      sum = fmaf(ml.y, f, sum);
      acc.x = fmaf(v.x, f, acc.x), acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z), acc.w = fmaf(v.w, f, acc.w);
    }
    if (mx == -INFINITY && sum == 0.f && row_sees(p, w.s, w.tile, stop, w.ln.key_log2, rl)) mx = kLeast;
    if (S.nan_at[d / kKv4Block] < rl) acc.x = acc.y = acc.z = acc.w = __uint_as_float(0x7FC00000u);
    if (whole) {
      const int64_t row = S.index[r];
      const float inv = row_inverse(mx, sum);
      const uint2 b = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
      *reinterpret_cast<uint2 *>(p.out + row * D + d) = b;
      if (d == 0 && p.lse) p.lse[row] = row_lse(mx, sum, kPOff);
    } else {
      *reinterpret_cast<float4 *>(P.part_o + (static_cast<int64_t>(part) * R + r) * D + d) = acc;
      if (d == 0) P.part_ml[part * R + r] = make_float2(mx, sum);
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreadsA, StepShape<D, NT>::kResident)
    kv4_step_kernel(const __grid_constant__ AttnParams P) {
  constexpr int R = 8 * NT, KS = D / 16, MT = kTile / 16;
  using Sh = StepShape<D, NT>;
  constexpr int NS = Sh::kStages;
  extern __shared__ uint8_t smem_raw[];
  using Smem = AttnSmem<D, NT>;
  Smem &S = *reinterpret_cast<Smem *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const Kv4AttnLaunch &p = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kWarps * NS; ++i) mbar_init(&S.full[0][0] + i, 2);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();  // (the join follows in this call)
  const Line line{&p, P.group, R, 31 - __clz(R), P.key_log2};
  const int chunk = (p.B + kThreadsA - 1) / kThreadsA;
  const int64_t all = line_prefix(line, kThreadsA, chunk, S.prefix, S.warp_sums);
  const int ctas = slices(all, P.ctas, P.key_log2);
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const int64_t from = slice_at(all, ctas, blockIdx.x), to = slice_at(all, ctas, blockIdx.x + 1);
  Walk w;
  w.begin(line, S.prefix, kThreadsA, chunk, from, to);
  fence_proxy_async_global();  // the cache's rows may come from the kernel before, by plain stores

  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t q_at = smem_u32(&S.q[lane & 7][8 * (lane >> 3)]);
  uint32_t issued = 0, used = 0;  // this warp's tiles
  bool dead = false;
  // The warp's next half tile into its next stage: keys (half 0) or values of tile t of u's unit. Lane 0 copies the
  // codes and lane 1 the scales, in the same instructions.
  const uint32_t row_bytes = lane == 0 ? D / 2 : D / kKv4Block;
  const uint8_t *const src_k = lane == 0 ? p.cache.k_codes : p.cache.k_scales;
  const uint8_t *const src_v = lane == 0 ? p.cache.v_codes : p.cache.v_scales;
  auto fetch = [&](const Walk &u, int t, int half) {
    const uint32_t slot = issued % NS;
    if (lane < 2) {
      const int page = p.cache.block_table[static_cast<int64_t>(u.s) * p.cache.max_blocks + t / (DSV4_PAGE_POSITIONS / kTile)];
      const bool bad = static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.cache.num_pages);
      uint64_t *bar = &S.full[warp][slot];
      S.bad[warp][slot] = bad;
      if (bad) {
        report(p.d_status, DSV4_DEV_BAD_PAGE);
        mbar_arrive(bar);
      } else {
        const int64_t row = static_cast<int64_t>(page) * (p.Hk * DSV4_PAGE_POSITIONS) +
                            (u.kvh * DSV4_PAGE_POSITIONS + t % (DSV4_PAGE_POSITIONS / kTile) * kTile);
        typename Smem::Stage &T = S.stage[warp][slot];
        mbar_arrive_expect_tx(bar, row_bytes * kTile);
        bulk_load(lane == 0 ? T.c : T.s, (half ? src_v : src_k) + row * row_bytes, row_bytes * kTile, bar);
      }
    }
    ++issued;
  };
  // tiles of the unit's part that any of its rows sees: [u.tile, ...); warp w takes the w-th, (w + 4)-th, ...
  auto seen = [&](const Walk &u) { return max(min(u.stop(), (u.unit_limit() + kTile - 1) / kTile) - u.tile, 0); };
  auto fetch_half = [&](const Walk &u, int count, int h) {  // half tile h of the warp's
    const int i = warp + (h >> 1) * kWarps;
    if (i < count) fetch(u, u.tile + i, h & 1);
  };
  auto fetch_first = [&](const Walk &u) {
    const int count = seen(u);
#pragma unroll
    for (int h = 0; h < NS; ++h) fetch_half(u, count, h);
  };
  // waits for the warp's next stage; negative: gave up
  auto arrived = [&]() -> int {
    const uint32_t slot = used % NS;
    const bool ok = !dead && mbar_spin(&S.full[warp][slot], (used / NS) & 1, &S.abort_flag);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      dead = true;
      return -1;
    }
    ++used;
    return static_cast<int>(slot);
  };
  bool first = true;
  for (;;) {
      const int stop = w.stop(), limit = w.unit_limit();
      const int count = seen(w);
      // lane r knows row r: the positions it sees (0: there is no such row) and where it is
      int my_lim = 0, my_head = 0;
      int64_t my_tok = 0;
      if (lane < R) {
        const int64_t row = (static_cast<int64_t>(w.rt) << line.r_log2) + lane;
        if (row < static_cast<int64_t>(w.q.len) * line.G) {
          const int64_t i = quotient(row, line.G);
          my_lim = min(w.q.n, w.q.start + static_cast<int>(i) + 1);
          my_tok = w.q.tok0 + i;
          my_head = w.kvh * line.G + static_cast<int>(row - i * line.G);
          if (warp == 0) S.index[lane] = my_tok * p.Hq + my_head;
        }
        if (warp == 0) S.lim[lane] = my_lim;
      }
      // Q fragments: column g of tile nt is row 8 nt + g; a lane's channels of step j are D/4 t4 + 4 j ..+3
      uint32_t qf[NT][KS][2];
      float rs[NT][2];   // log2 score per product, of columns 2 t4 and 2 t4 + 1
      int lim[NT][2];
      int least = limit; // positions that every row sees
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int rl = __shfl_sync(0xFFFFFFFFu, my_lim, 8 * nt + g);
        const int64_t tok = __shfl_sync(0xFFFFFFFFu, my_tok, 8 * nt + g);
        const int head = __shfl_sync(0xFFFFFFFFu, my_head, 8 * nt + g);
        const uint16_t *src = p.q + tok * p.q_stride + static_cast<int64_t>(head) * D + t4 * (D / 4);
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) {
          const uint4 v = rl > 0 ? *reinterpret_cast<const uint4 *>(src + 8 * i) : make_uint4(0, 0, 0, 0);
          qf[nt][2 * i][0] = v.x, qf[nt][2 * i][1] = v.y, qf[nt][2 * i + 1][0] = v.z, qf[nt][2 * i + 1][1] = v.w;
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int there = __shfl_sync(0xFFFFFFFFu, my_lim, 8 * nt + 2 * t4 + c);
          lim[nt][c] = there > 0 ? there : limit;  // (a row that is not there needs no mask: its sums are not written)
          least = min(least, lim[nt][c]);
        }
      }
      if (first) fetch_first(w);
      first = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        uint32_t am = 0;
#pragma unroll
        for (int i = 0; i < KS * 2; ++i)
          am = max(am, max((qf[nt][i >> 1][i & 1] << 16) & 0x7FFF0000u, qf[nt][i >> 1][i & 1] & 0x7FFF0000u));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
        am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 2));
        // 2^sh brings the largest element to [2^14, 2^15) (bounded so that 2^sh and 2^-sh are normal)
        const int ex = static_cast<int>(am >> 23) - 127;
        const int sh = (am == 0 || ex >= 128) ? 0 : min(max(14 - ex, -113), 120);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
#pragma unroll
        for (int i = 0; i < KS * 2; ++i) {
          const uint32_t raw = qf[nt][i >> 1][i & 1];
          const uint32_t h = pack_half2(__uint_as_float(raw << 16) * up, __uint_as_float(raw & 0xFFFF0000u) * up);
          if (warp == 0) *reinterpret_cast<uint32_t *>(&S.q[8 * nt + g][8 * i + 2 * t4]) = h;
        }
        // (not below float32's normal numbers: a masked position is minus infinity times this)
        const float mine = fmaxf(
            p.softmax_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.17549435e-38f);
        rs[nt][0] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t4);      // lane 4 * (2 t4): column 2 t4
        rs[nt][1] = __shfl_sync(0xFFFFFFFFu, mine, 8 * t4 + 4);
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
      if (tid < D / kKv4Block) S.nan_at[tid] = 0x7FFFFFFF;
      __syncthreads();

      float o[KS][NT][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
      }
      for (int i = warp, h = NS; i < count; i += kWarps, h += 2) {
        int slot = arrived();
        if (slot < 0) break;
        const bool bad = S.bad[warp][slot];
        const typename Smem::Stage *T = &S.stage[warp][slot];
        const int key0 = (w.tile + i) * kTile;
        const bool edge = key0 + kTile > least;
        float s[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int ra = 16 * mt + key_of(g), rb = ra + 8;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
          constexpr int W = D / 32;  // words of a lane's codes of one key
          uint32_t ca[W], cb[W];
          if constexpr (W == 4) {
            const uint4 a = *reinterpret_cast<const uint4 *>(T->c + ra * (D / 2) + t4 * 16);
            const uint4 b = *reinterpret_cast<const uint4 *>(T->c + rb * (D / 2) + t4 * 16);
            ca[0] = a.x, ca[1] = a.y, ca[2] = a.z, ca[3] = a.w;
            cb[0] = b.x, cb[1] = b.y, cb[2] = b.z, cb[3] = b.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(T->c + ra * (D / 2) + t4 * 8);
            const uint2 b = *reinterpret_cast<const uint2 *>(T->c + rb * (D / 2) + t4 * 8);
            ca[0] = a.x, ca[1] = a.y;
            cb[0] = b.x, cb[1] = b.y;
          }
          const int blk = t4 * (D / 4) / kKv4Block;
          // 2^(byte - 127); a sum of them is infinite where a byte is 255 (NaN), which is looked at apart
          float fa = __uint_as_float(static_cast<uint32_t>(T->s[ra * (D / kKv4Block) + blk]) << 23);
          float fb = __uint_as_float(static_cast<uint32_t>(T->s[rb * (D / kKv4Block) + blk]) << 23);
          if (fa + fb == INFINITY) {
            if (fa == INFINITY) fa = __uint_as_float(0x7FC00000u);
            if (fb == INFINITY) fb = __uint_as_float(0x7FC00000u);
          }
          const uint32_t sa = pack_half2(fa, fa), sb = pack_half2(fb, fb);
#pragma unroll
          for (int c = 0; c < W; ++c) {
            uint32_t ha[4], hb[4];
            e2m1x8_to_half2(ca[c], ha);
            e2m1x8_to_half2(cb[c], hb);
            uint32_t qb[NT][4];  // steps 2 c and 2 c + 1, both halves
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) ldmatrix4(qb[nt], q_at + nt * static_cast<uint32_t>(8 * sizeof(S.q[0])) + 64 * c);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a0 = hmul2(ha[2 * k], sa), a2 = hmul2(ha[2 * k + 1], sa);
              const uint32_t a1 = hmul2(hb[2 * k], sb), a3 = hmul2(hb[2 * k + 1], sb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(s[mt][nt], a0, a1, a2, a3, qb[nt][2 * k], qb[nt][2 * k + 1]);
            }
          }
        }
        __syncwarp();
        fetch_half(w, count, h);
        // softmax: column c of tile nt is this lane's row pair; keys g and g + 8 of each 16
        if (bad) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = -INFINITY;
        } else if (edge) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const int ka = key0 + 16 * mt + key_of(g);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                if (ka >= lim[nt][c]) s[mt][nt][c] = -INFINITY;
                if (ka + 8 >= lim[nt][c]) s[mt][nt][2 + c] = -INFINITY;
              }
            }
          }
        }
        uint32_t pb[MT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float off[2];
          bool moved = false;
          float keep[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = s[0][nt][c];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][c], s[mt][nt][2 + c]));
#pragma unroll
            for (int o2 = 4; o2 < 32; o2 <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o2));
            const float now = fmaxf(m[nt][c], x * rs[nt][c]);
            keep[c] = now == -INFINITY ? 1.f : ex2_approx(m[nt][c] - now);
            moved |= now != m[nt][c];
            m[nt][c] = now;
            off[c] = now == -INFINITY ? 0.f : kPOff - now;
          }
          if (__any_sync(0xFFFFFFFFu, moved)) {
            l[nt][0] *= keep[0];
            l[nt][1] *= keep[1];
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[k][nt][0] *= keep[0], o[k][nt][1] *= keep[1];
              o[k][nt][2] *= keep[0], o[k][nt][3] *= keep[1];
            }
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const float p0 = ex2_approx(fmaf(s[mt][nt][0], rs[nt][0], off[0]));
            const float p1 = ex2_approx(fmaf(s[mt][nt][1], rs[nt][1], off[1]));
            const float p2 = ex2_approx(fmaf(s[mt][nt][2], rs[nt][0], off[0]));
            const float p3 = ex2_approx(fmaf(s[mt][nt][3], rs[nt][1], off[1]));
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            pb[mt][nt][0] = transpose8(pack_half2(p0, p1));
            pb[mt][nt][1] = transpose8(pack_half2(p2, p3));
          }
        }
        slot = arrived();
        if (slot < 0) break;
        T = &S.stage[warp][slot];
        // O^T += V^T P^T: a lane's channels are D/8 g .. + D/8 - 1, its keys 2 t4, 2 t4 + 1 and those + 8
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const int kA = 16 * mt + key_of(2 * t4), kB = 16 * mt + key_of(2 * t4 + 1);
          constexpr int W = D / 64;
          uint32_t c4[4][W];
          float sf[4];
          const int blk = g * (D / 8) / kKv4Block;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int key = ((q & 1) ? kB : kA) + (q >> 1) * 8;
            const uint8_t *src = T->c + key * (D / 2) + g * (D / 16);
            if constexpr (W == 2) {
              const uint2 v = *reinterpret_cast<const uint2 *>(src);
              c4[q][0] = v.x, c4[q][1] = v.y;
            } else {
              c4[q][0] = *reinterpret_cast<const uint32_t *>(src);
            }
            sf[q] = __uint_as_float(static_cast<uint32_t>(T->s[key * (D / kKv4Block) + blk]) << 23);
          }
          if (edge || bad) {
#pragma unroll
            for (int q = 0; q < 4; ++q)  // not a position of the unit
              if (bad || key0 + ((q & 1) ? kB : kA) + (q >> 1) * 8 >= limit) sf[q] = 0.f;
          }
          if ((sf[0] + sf[1]) + (sf[2] + sf[3]) == INFINITY) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (sf[q] == INFINITY) {
                atomicMin(&S.nan_at[blk], key0 + ((q & 1) ? kB : kA) + (q >> 1) * 8);
                sf[q] = 0.f;
              }
          }
          const uint32_t sAB = pack_half2(sf[0], sf[1]), sCD = pack_half2(sf[2], sf[3]);
          // Two keys' codes side by side in a byte before they are converted: 4 operations for 8 channels,
          // half of what permuting the converted pairs takes.
#pragma unroll
          for (int c = 0; c < W; ++c) {
            uint32_t lo[2][4], hi[2][4];  // [keys A, B / C, D][channel pair]: even and odd channels
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t x = c4[2 * q][c], y = c4[2 * q + 1][c];
              e2m1x8_to_half2((x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u), lo[q]);
              e2m1x8_to_half2((x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), hi[q]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a0 = hmul2(lo[0][k], sAB), a1 = hmul2(hi[0][k], sAB);
              const uint32_t a2 = hmul2(lo[1][k], sCD), a3 = hmul2(hi[1][k], sCD);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816(o[4 * c + k][nt], a0, a1, a2, a3, pb[mt][nt][0], pb[mt][nt][1]);
            }
          }
        }
        __syncwarp();
        fetch_half(w, count, h + 1);
      }
      // the next unit's first copies are under way while this one is joined
      Walk nx = w;
      const bool more = nx.next();
      if (more && !dead) fetch_first(nx);

      // ---- join the warps
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = l[nt][c];
#pragma unroll
          for (int o2 = 4; o2 < 32; o2 <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o2);
          const int r = 8 * nt + 2 * t4 + c;
          if (g == 0) S.ml[warp][r] = make_float2(m[nt][c], x);
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const int d = g * (D / 8) + 2 * k;
            *reinterpret_cast<float2 *>(&S.o[warp][r][d]) = make_float2(o[k][nt][c], o[k][nt][2 + c]);
          }
        }
      }
      __syncthreads();
      join_part<D, R>(P, S, w, stop);
      __syncthreads();
      if (!more) break;
      w = nx;
  }
  if (dead) {  // let the copies in flight land before the CTA leaves
    volatile int dummy = 0;
    for (; used != issued; ++used) mbar_wait(&S.full[warp][used % NS], (used / NS) & 1, &dummy);
  }
  if (S.abort_flag && lane == 0) report(p.d_status, DSV4_DEV_TIMEOUT);
}

// ---------------------------------------------------------------- few rows, long contexts: scores on the tensor cores

// The same slices, in tiles of 128 keys, for at most 8 rows of 128 channels. The codes of K are an operand of
// tcgen05.mma (kind::f8f6f4, e2m1) as they are: a block of 32 channels is one product of depth 32, keys on
// the 128-row side, whose sums the block's scale multiplies afterwards:
//   s_j = sum_b 2^k_jb (sum_c code_jc q_c)          8 x 4 scales a key in place of 128 conversions and products
// q enters as two e4m3 values, hi + lo / 32, that hold its 8 bits exactly but for elements 2^-14 below the row's
// largest, which are off by at most 2^-22 of that: columns 0-7 are the rows' hi and 8-15 their lo. What is
// missing is kept, and where it could move a score of the tile by more than kTcLoose, going by the keys' largest
// scale, its products with the keys are added in float32 (tc_missing), so that no channel drowns beside a larger one.
// On ordinary rows that never happens: the bound is some 2^-20 there.
// Warp 4 brings keys (TMA, which spreads the codes to the operand's layout) and values (bulk copies) into two stages
// each and issues the products; warps 0-3 take 32 keys of each tile, one per lane: scales, weights, and P to shared
// memory, from where it is the B operand of mma.sync with the values as in the kernel above.
// The reference of the weights is an integer (so that taking it off twice rounds alike), raised when a score exceeds
// it by more than 2^8; weights are held times 2^7.
// Measured: four sequences of 262144 positions 233 us (4.90 TB/s, 75% of the measured copy rate; 225 us without what a
// row's remainder and the rows without a finite score take); 194 us with the
// arithmetic left out, 195 us without the values' part of it, no less without the copies of the keys. What is left is
// that part, on three such warps a scheduler: its conversions some 33 us, the products with the scales 7 us, mma.sync
// nothing. The values' scales are converted once a warp and shared (each lane for itself: 240 us). Four CTAs an SM at
// 96 registers took 256 us against 247 us then, one wait for all of a tile's scores 249 us, and values brought to
// registers before the weights were no faster.
constexpr int kTcKeys = 128;
constexpr int kTcThreads = 32 * (kWarps + 1);
constexpr int kTcResident = 3;
constexpr int kTcCols = 128;       // TMEM columns: two tiles of 4 blocks x 16
constexpr float kTcOff = 7.f;      // weights are held times 2^7
constexpr float kTcRaise = 8.f;
constexpr float kTcNone = -kLeast;  // off of a row without a reference yet
constexpr float kTcLoose = 6.1e-5f; // log2 that a score may be off by: an eighth of the weights' rounding to fp16

struct alignas(1024) TcStepSmem {
  uint8_t k[2][kTcKeys * 128];     // codes, spread: 16 of them in each 16 bytes
  uint8_t q[16 * 128];             // e4m3: rows 0-7 hi, 8-15 lo
  struct alignas(128) Values {
    uint8_t c[kTcKeys * 64], ks[kTcKeys * 4], vs[kTcKeys * 4];
  } v[2];
  union {
    uint4 pw[kWarps][32];          // weights of a warp's keys, fp16
    int64_t prefix[kTcThreads + 1];  // before the first product
  };
  alignas(16) uint16_t sv[kWarps][4][4][8];  // scales of a warp's values, fp16, per block in the order of the products
  alignas(16) float o[kWarps][8][128 + 4];
  float2 ml[kWarps][8];
  float keep[kWarps][8];
  alignas(16) float rs[8];         // log2 score per product
  alignas(16) float missing[8];    // log2 that a score is off by at most, at a scale of 1
  alignas(16) int lim[8];
  int64_t index[8];
  int64_t warp_sums[kTcThreads / 32];
  uint64_t k_full[2], v_full[2], v_free[2], s_full[2], s_free[2], q_full;
  int bad[2];
  int nan_at[128 / kKv4Block];
  int abort_flag;
  uint32_t tmem_base;
};

__device__ __forceinline__ int tc_seen(const Walk &u) {
  return max(min(u.stop(), (u.unit_limit() + kTcKeys - 1) / kTcKeys) - u.tile, 0);
}

// Adds the products of a key (one per lane) with what hi + lo / 32 leaves out of each row, which lies where warp 0's sums
// will be: row tile r's channels 8 c .. 8 c + 7 at 16-byte word 16 r + c, bf16 (a remainder of 8 bits: exact).
__device__ __forceinline__ void tc_missing(const Kv4AttnLaunch &p, const TcStepSmem &S, int64_t row, uint32_t scales,
                                           uint64_t (&s)[4]) {
  const uint4 *rest = reinterpret_cast<const uint4 *>(S.o[0]);
  const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.cache.k_codes + row * 64);
#pragma unroll 1
  for (int c = 0; c < 16; ++c) {
    uint32_t h[4];
    e2m1x8_to_half2(codes[c], h);
    const uint32_t byte = scales >> (c / 4 * 8) & 255u;
    const float f = byte > 127u + kKv4ExpMax ? 0.f : __uint_as_float(byte << 23);  // (a NaN block)
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
      x[2 * i] = v.x * f, x[2 * i + 1] = v.y * f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 ra = rest[16 * (2 * k) + c], rb = rest[16 * (2 * k + 1) + c];
      const uint32_t a[4] = {ra.x, ra.y, ra.z, ra.w}, b[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[k] = fma_f32x2(pack_f32x2(x[2 * i], x[2 * i]), pack_f32x2(__uint_as_float(a[i] << 16), __uint_as_float(b[i] << 16)), s[k]);
        s[k] = fma_f32x2(pack_f32x2(x[2 * i + 1], x[2 * i + 1]),
                         pack_f32x2(__uint_as_float(a[i] & 0xFFFF0000u), __uint_as_float(b[i] & 0xFFFF0000u)), s[k]);
      }
    }
  }
}

// copies and products of the slice; w at its start
__device__ __forceinline__ void tc_feed(const AttnParams &P, const CUtensorMap &map, TcStepSmem &S, Walk &w, uint32_t tmem) {
  const Kv4AttnLaunch &p = P.a;
  const int lane = threadIdx.x & 31;
  struct Tile {
    int row;      // of the cache; negative: the page does not exist
    bool first;   // of its unit
  };
  int i = 0, count = tc_seen(w);
  bool fresh = true;
  auto settle = [&]() -> bool {  // the next unit with tiles, where this one has none left
    while (i >= count) {
      if (!w.next()) return false;
      i = 0;
      count = tc_seen(w);
      fresh = true;
    }
    return true;
  };
  auto look = [&]() -> Tile {
    const int t = w.tile + i;
    const int page = p.cache.block_table[static_cast<int64_t>(w.s) * p.cache.max_blocks + t / (DSV4_PAGE_POSITIONS / kTcKeys)];
    Tile c;
    c.first = fresh;
    if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.cache.num_pages)) {
      c.row = -1;
      if (lane == 0) report(p.d_status, DSV4_DEV_BAD_PAGE);
    } else {
      c.row = (page * p.Hk + w.kvh) * DSV4_PAGE_POSITIONS + t % (DSV4_PAGE_POSITIONS / kTcKeys) * kTcKeys;
    }
    fresh = false;
    ++i;
    return c;
  };
  bool dead = false;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_spin(bar, parity & 1, &S.abort_flag));
  };
  auto load_k = [&](uint32_t n, const Tile &c) {
    if (lane != 0) return;
    uint64_t *bar = &S.k_full[n & 1];
    if (c.row < 0) {
      mbar_arrive(bar);
    } else {  // (the transaction counts the packed bytes)
      mbar_arrive_expect_tx(bar, kTcKeys * 64);
      tma_load_2d(S.k[n & 1], &map, bar, 0, c.row);
    }
  };
  auto load_v = [&](uint32_t n, const Tile &c) {
    if (lane != 0) return;
    uint64_t *bar = &S.v_full[n & 1];
    S.bad[n & 1] = c.row < 0;
    if (c.row < 0) {
      mbar_arrive(bar);
    } else {
      TcStepSmem::Values &T = S.v[n & 1];
      const int64_t row = c.row;
      mbar_arrive_expect_tx(bar, kTcKeys * (64 + 4 + 4));
      bulk_load(T.ks, p.cache.k_scales + row * 4, kTcKeys * 4, bar);
      bulk_load(T.c, p.cache.v_codes + row * 64, kTcKeys * 64, bar);
      bulk_load(T.vs, p.cache.v_scales + row * 4, kTcKeys * 4, bar);
    }
  };
  constexpr uint32_t id = idesc_e2m1_e4m3(kTcKeys, 16);
  const uint64_t qd = sw128_desc(smem_u32(S.q), 16, 1024);
  uint32_t n = 0, loaded_k = 0, loaded_v = 0, units = 0;
  bool have = settle();
  Tile cur{}, nxt{};
  if (have) {
    cur = look();
    load_k(loaded_k++, cur);
  }
  for (; have; ++n) {
    const bool more = settle();
    if (more) {
      nxt = look();
      if (n >= 1) wait(&S.s_full[(n - 1) & 1], (n - 1) >> 1);  // its stage's products are done
      if (dead) break;
      load_k(loaded_k++, nxt);
    }
    if (n >= 2) wait(&S.v_free[n & 1], (n >> 1) - 1);
    if (dead) break;
    load_v(loaded_v++, cur);
    if (cur.first) wait(&S.q_full, units++);
    wait(&S.k_full[n & 1], n >> 1);
    if (n >= 2) wait(&S.s_free[n & 1], (n >> 1) - 1);
    if (dead) break;
    tc_fence_after();
    const uint64_t kd = sw128_desc(smem_u32(S.k[n & 1]), 16, 1024);
#pragma unroll
    for (int b = 0; b < 4; ++b)
      if (elect_one()) mma_e4m3(tmem + 64 * (n & 1) + 16 * b, kd + 2 * b, qd + 2 * b, id, 0);
    if (elect_one()) mma_commit(&S.s_full[n & 1]);
    cur = nxt;
    have = more;
  }
  if (dead) {  // let what is in flight land before the CTA leaves
    volatile int dummy = 0;
    for (uint32_t j = loaded_k < 2 ? 0 : loaded_k - 2; j < loaded_k; ++j) mbar_wait(&S.k_full[j & 1], (j >> 1) & 1, &dummy);
    for (uint32_t j = loaded_v < 2 ? 0 : loaded_v - 2; j < loaded_v; ++j) mbar_wait(&S.v_full[j & 1], (j >> 1) & 1, &dummy);
    for (uint32_t j = n < 2 ? 0 : n - 2; j < n; ++j) mbar_wait(&S.s_full[j & 1], (j >> 1) & 1, &dummy);
  }
}

// softmax and values of the slice, warps 0-3
__device__ __forceinline__ void tc_attend(const AttnParams &P, TcStepSmem &S, Walk &w, uint32_t tmem) {
  constexpr int D = 128, R = 8, KS = D / 16;
  const Kv4AttnLaunch &p = P.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t pw_at = smem_u32(&S.pw[warp][8 * (lane >> 3) + key_of(lane & 7)]);
  // where this lane's key's value scales go: halves [block][t4][16-key group][+ 8][first or second of the pair]
  const int lane_row = (0x1320 >> (4 * (lane & 3))) & 3;  // the inverse of key_of
  uint16_t *const sv_to = &S.sv[warp][0][0][0] + ((lane & 4) / 2 + (lane_row >> 1)) * 8 + (lane >> 4) * 4 + (lane >> 3 & 1) * 2 + (lane_row & 1);
  uint32_t n = 0;  // tiles of the CTA
  bool dead = false;
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_spin(bar, parity & 1, &S.abort_flag));
  };
  for (;;) {
    const int stop = w.stop(), limit = w.unit_limit(), count = tc_seen(w);
    {  // thread: channels 8 (tid % 16) .. of row tid / 16
      const int r = tid >> 4, c = tid & 15;
      const int64_t row = static_cast<int64_t>(w.rt) * R + r, G = w.ln.G;
      const bool there = row < static_cast<int64_t>(w.q.len) * G;
      const int64_t i = there ? quotient(row, G) : 0, tok = w.q.tok0 + i;
      const int64_t head = w.kvh * G + (row - i * G);
      uint4 v = make_uint4(0, 0, 0, 0);
      if (there) v = *reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride + head * D + 8 * c);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
      uint32_t am = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) am = max(am, max((x[k] << 16) & 0x7FFF0000u, x[k] & 0x7FFF0000u));
#pragma unroll
      for (int o2 = 1; o2 < 16; o2 <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o2));
      // 2^sh brings the largest element to [2^7, 2^8). A row with an infinity or NaN has no finite score: it goes in as
      // e4m3's NaN, which makes NaN of the scores of the positions that the row sees (masked ones are set afterwards).
      const int ex = static_cast<int>(am >> 23) - 127;
      const int sh = (am == 0 || ex >= 128) ? 0 : min(max(7 - ex, -120), 120);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
      uint32_t hi[4], lo[4], rest[4];
      float missing = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = __uint_as_float(x[k] << 16) * up, b = __uint_as_float(x[k] & 0xFFFF0000u) * up;
        float ha, hb;
        hi[k] = e4m3_pair(a, b, ha, hb);
        float la, lb;
        lo[k] = e4m3_pair((a - ha) * 32.f, (b - hb) * 32.f, la, lb);
        if (ex >= 128) hi[k] = lo[k] = 0x7F7Fu;
        const float ra = ex >= 128 ? 0.f : fmaf(la, -0.03125f, a - ha), rb = ex >= 128 ? 0.f : fmaf(lb, -0.03125f, b - hb);
        rest[k] = __byte_perm(__float_as_uint(ra), __float_as_uint(rb), 0x7632);
        missing += fabsf(ra) + fabsf(rb);
      }
#pragma unroll
      for (int o2 = 1; o2 < 16; o2 <<= 1) missing += __shfl_xor_sync(0xFFFFFFFFu, missing, o2);
      reinterpret_cast<uint4 *>(S.o[0])[tid] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
      const uint32_t at = sw128_offset(r, c >> 1) + 8 * (c & 1);
      *reinterpret_cast<uint2 *>(S.q + at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2 *>(S.q + 1024 + at) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
      if (c == 0) {
        S.lim[r] = there ? min(w.q.n, w.q.start + static_cast<int>(i) + 1) : 0;
        S.index[r] = tok * p.Hq + head;
        const float rs = fmaxf(p.softmax_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23),
                               1.17549435e-38f);
        S.rs[r] = rs;
        S.missing[r] = 6.f * missing * rs;  // (6: the largest code)
      }
      if (tid < D / kKv4Block) S.nan_at[tid] = 0x7FFFFFFF;
    }
    fence_proxy_async_smem();
    named_bar_sync(1, 32 * kWarps);
    if (count > 0 && lane == 0) mbar_arrive(&S.q_full);
    int least = limit;  // positions that every row sees
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int x = S.lim[r];
      if (x > 0) least = min(least, x);
    }
    // 2^(byte - 127) * missing is above kTcLoose where the byte is above 104 + 127 - wide: the sum of a scale byte (104 to
    // 140) less 104 and `wide` then has its upper bit. Four bytes at once.
    float missing = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) missing = fmaxf(missing, S.missing[r]);
    const int wide = min(max(104 + 127 - static_cast<int>(__float_as_uint(kTcLoose / missing) >> 23), 0), 128);
    const uint32_t wide4 = static_cast<uint32_t>(wide - 104) * 0x01010101u;
    float o[KS][4];
    uint64_t off[R / 2], l[R / 2];  // per pair of rows: kTcOff - reference; this lane's sums
#pragma unroll
    for (int k = 0; k < KS; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
#pragma unroll
    for (int k = 0; k < R / 2; ++k) off[k] = pack_f32x2(kTcNone, kTcNone), l[k] = 0;

    // The tiles from the i-th on: all (`exact`: with what the products leave out), or those before the first that needs that.
    // (As a branch in one loop it split a tile's code and took 3% of the time.)
    int i = 0;
    auto tiles = [&](auto exact) {
      for (; i < count; ++i, ++n) {
        const uint32_t slot = n & 1;
        wait(&S.v_full[slot], n >> 1);
        wait(&S.s_full[slot], n >> 1);
        if (dead) break;
        tc_fence_after();
        const TcStepSmem::Values &T = S.v[slot];
        const bool bad = S.bad[slot];
        const int key0 = (w.tile + i) * kTcKeys + 32 * warp;  // the warp's first key
        const bool edge = key0 + 32 > least;
        uint32_t kb = *reinterpret_cast<const uint32_t *>(T.ks + 4 * (32 * warp + lane));
        uint32_t vb = *reinterpret_cast<const uint32_t *>(T.vs + 4 * (32 * warp + lane));
        if ((edge || bad) && (bad || key0 + lane >= limit)) kb = 0x68686868u, vb = 0;  // not a position of the unit
        if (!decltype(exact)::value && __any_sync(0xFFFFFFFFu, (kb + wide4) & 0x80808080u)) break;
        if (vb & vb << 1 & 0x80808080u) {  // no scale but NaN's byte has its two upper bits
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if ((vb >> (8 * b) & 255u) == 255u) {
              atomicMin(&S.nan_at[b], key0 + lane);
              vb &= ~(255u << (8 * b));
            }
        }
        {
          auto power = [&](int b) { return __uint_as_float((vb >> (8 * b) & 255u) << 23); };
          const uint32_t h01 = pack_half2(power(0), power(1)), h23 = pack_half2(power(2), power(3));
          sv_to[0] = static_cast<uint16_t>(h01), sv_to[32] = static_cast<uint16_t>(h01 >> 16);
          sv_to[64] = static_cast<uint16_t>(h23), sv_to[96] = static_cast<uint16_t>(h23 >> 16);
        }
        const uint32_t s_at = tmem + 64 * slot + (static_cast<uint32_t>(32 * warp) << 16);
        uint64_t s[R / 2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[32];
          tmem_ld32(s_at + 32 * h, a);
          tmem_ld_wait();
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float f = __uint_as_float((kb >> (8 * (2 * h + b)) & 255u) << 23);
            const uint64_t f2 = pack_f32x2(f, f), part = pack_f32x2(0.03125f, 0.03125f);
#pragma unroll
            for (int k = 0; k < R / 2; ++k) {
              const uint64_t hi = pack_f32x2(__uint_as_float(a[16 * b + 2 * k]), __uint_as_float(a[16 * b + 2 * k + 1]));
              const uint64_t lo = pack_f32x2(__uint_as_float(a[16 * b + 8 + 2 * k]), __uint_as_float(a[16 * b + 9 + 2 * k]));
              const uint64_t x = fma_f32x2(lo, part, hi);
              s[k] = h + b == 0 ? mul_f32x2(f2, x) : fma_f32x2(f2, x, s[k]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.s_free[slot]);
        if constexpr (decltype(exact)::value) {
          if (!bad) {
            constexpr int kPer = DSV4_PAGE_POSITIONS / kTcKeys;  // tiles of a page
            const int t = w.tile + i, page = p.cache.block_table[static_cast<int64_t>(w.s) * p.cache.max_blocks + t / kPer];
            const int64_t head = static_cast<int64_t>(page) * p.Hk + w.kvh;
            tc_missing(p, S, head * DSV4_PAGE_POSITIONS + t % kPer * kTcKeys + 32 * warp + lane, kb, s);
          }
        }
        if (kb & kb << 1 & 0x80808080u) {  // a NaN block makes the key's scores NaN
          bool nan = false;
#pragma unroll
          for (int b = 0; b < 4; ++b) nan |= (kb >> (8 * b) & 255u) == 255u;
#pragma unroll
          for (int k = 0; k < R / 2; ++k)
            if (nan) s[k] = pack_f32x2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
        }
        if (edge || bad) {
#pragma unroll
          for (int k = 0; k < R / 2; ++k) {
            float a, b;
            unpack_f32x2(s[k], a, b);
            // (a row that is not there needs no mask, but for positions behind the last: its sums are not written)
            const int la = S.lim[2 * k], lb = S.lim[2 * k + 1];
            if (bad || key0 + lane >= (la > 0 ? la : limit)) a = -INFINITY;
            if (bad || key0 + lane >= (lb > 0 ? lb : limit)) b = -INFINITY;
            s[k] = pack_f32x2(a, b);
          }
        }
        auto rs = [&](int k) { return *reinterpret_cast<const uint64_t *>(&S.rs[2 * k]); };
        float y[R];
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < R / 2; ++k) {
          unpack_f32x2(fma_f32x2(s[k], rs(k), off[k]), y[2 * k], y[2 * k + 1]);
          most = fmaxf(most, fmaxf(y[2 * k], y[2 * k + 1]));
        }
        if (__any_sync(0xFFFFFFFFu, most > kTcOff + kTcRaise)) {
#pragma unroll
          for (int k = 0; k < R / 2; ++k) {
            float x[2], f[2], sums[2];
            unpack_f32x2(mul_f32x2(s[k], rs(k)), x[0], x[1]);
            unpack_f32x2(off[k], f[0], f[1]);
            unpack_f32x2(l[k], sums[0], sums[1]);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int o2 = 1; o2 < 32; o2 <<= 1) x[c] = fmaxf(x[c], __shfl_xor_sync(0xFFFFFFFFu, x[c], o2));
              const float was = f[c] == kTcNone ? -kTcNone : kTcOff - f[c], now = fmaxf(was, ceilf(x[c]));
              const float keep = now == was ? 1.f : ex2_approx(was - now);
              if (now != was) f[c] = kTcOff - now;
              sums[c] *= keep;
              if (lane == 0) S.keep[warp][2 * k + c] = keep;
            }
            off[k] = pack_f32x2(f[0], f[1]);
            l[k] = pack_f32x2(sums[0], sums[1]);
            unpack_f32x2(fma_f32x2(s[k], rs(k), off[k]), y[2 * k], y[2 * k + 1]);
          }
          __syncwarp();
          const float2 keep = *reinterpret_cast<const float2 *>(&S.keep[warp][2 * t4]);
#pragma unroll
          for (int k = 0; k < KS; ++k) o[k][0] *= keep.x, o[k][1] *= keep.y, o[k][2] *= keep.x, o[k][3] *= keep.y;
          __syncwarp();
        }
        uint32_t h[R / 2];
#pragma unroll
        for (int k = 0; k < R / 2; ++k) {
          const float a = ex2_approx(y[2 * k]), b = ex2_approx(y[2 * k + 1]);
          l[k] = add_f32x2(l[k], pack_f32x2(a, b));
          h[k] = pack_half2(a, b);
        }
        S.pw[warp][lane] = make_uint4(h[0], h[1], h[2], h[3]);
        __syncwarp();
        uint32_t pb[4];
        ldmatrix4_trans(pb, pw_at);
        const uint4 sv = *reinterpret_cast<const uint4 *>(S.sv[warp][g >> 1][t4]);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int kA = 16 * mt + key_of(2 * t4), kB = 16 * mt + key_of(2 * t4 + 1);  // of the warp's 32
          uint32_t c4[4][2];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int key = 32 * warp + ((q & 1) ? kB : kA) + (q >> 1) * 8;
            const uint2 v = *reinterpret_cast<const uint2 *>(T.c + key * 64 + g * 8);
            c4[q][0] = v.x, c4[q][1] = v.y;
          }
          const uint32_t sAB = mt == 0 ? sv.x : sv.z, sCD = mt == 0 ? sv.y : sv.w;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t lo[2][4], hi[2][4];  // as in the kernel above
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t x = c4[2 * q][c], z = c4[2 * q + 1][c];
              e2m1x8_to_half2((x & 0x0F0F0F0Fu) | (z << 4 & 0xF0F0F0F0u), lo[q]);
              e2m1x8_to_half2((x >> 4 & 0x0F0F0F0Fu) | (z & 0xF0F0F0F0u), hi[q]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma16816(o[4 * c + k], hmul2(lo[0][k], sAB), hmul2(hi[0][k], sAB), hmul2(lo[1][k], sCD), hmul2(hi[1][k], sCD),
                       pb[2 * mt], pb[2 * mt + 1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.v_free[slot]);
      }
    };
    tiles(std::false_type{});
    if (i < count && !dead) tiles(std::true_type{});
#pragma unroll
    for (int k = 0; k < R / 2; ++k) {
      float f[2], sums[2];
      unpack_f32x2(off[k], f[0], f[1]);
      unpack_f32x2(l[k], sums[0], sums[1]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int o2 = 1; o2 < 32; o2 <<= 1) sums[c] += __shfl_xor_sync(0xFFFFFFFFu, sums[c], o2);
        // as a reference for weights times 2^kPOff
        if (lane == 0) S.ml[warp][2 * k + c] = make_float2(f[c] == kTcNone ? -INFINITY : kPOff - f[c], sums[c]);
      }
    }
    named_bar_sync(1, 32 * kWarps);  // (all have read what the products leave out: warp 0's sums take its place)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int k = 0; k < KS; ++k)
        *reinterpret_cast<float2 *>(&S.o[warp][2 * t4 + c][16 * g + 2 * k]) = make_float2(o[k][c], o[k][2 + c]);
    named_bar_sync(1, 32 * kWarps);
    join_part<D, R>(P, S, w, stop);
    named_bar_sync(1, 32 * kWarps);
    if (!w.next()) break;
  }
}

__global__ void __launch_bounds__(kTcThreads, kTcResident)
    kv4_step_tc_kernel(const __grid_constant__ AttnParams P, const __grid_constant__ CUtensorMap map) {
  extern __shared__ uint8_t smem_raw[];
  TcStepSmem &S = *reinterpret_cast<TcStepSmem *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Kv4AttnLaunch &p = P.a;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 1);
      mbar_init(&S.v_full[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.v_free[i], kWarps);
      mbar_init(&S.s_free[i], kWarps);
    }
    mbar_init(&S.q_full, kWarps);
    S.abort_flag = 0;
    fence_mbar_init();
    prefetch_tensormap(&map);
  }
  pdl_wait();
  // (not before the wait: a kernel that this one waits for may want all of TMEM)
  if (warp == kWarps) {
    tmem_alloc(&S.tmem_base, kTcCols);
    tmem_relinquish();
    tc_fence_before();
  }
  const Line line{&p, P.group, 8, 3, P.key_log2};
  const int chunk = (p.B + kTcThreads - 1) / kTcThreads;
  const int64_t all = line_prefix(line, kTcThreads, chunk, S.prefix, S.warp_sums);
  tc_fence_after();
  pdl_launch_dependents();  // (the join follows in this call)
  const uint32_t tmem = __reduce_max_sync(0xFFFFFFFFu, S.tmem_base);
  const int ctas = slices(all, P.ctas, P.key_log2);
  if (static_cast<int>(blockIdx.x) < ctas) {
    Walk w;
    w.begin(line, S.prefix, kTcThreads, chunk, slice_at(all, ctas, blockIdx.x), slice_at(all, ctas, blockIdx.x + 1));
    fence_proxy_async_global();  // the cache's rows may come from the kernel before, by plain stores
    if (warp == kWarps) tc_feed(P, map, S, w, tmem);
    else tc_attend(P, S, w, tmem);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarps) tmem_dealloc(tmem, kTcCols);
  if (S.abort_flag && tid == 0) report(p.d_status, DSV4_DEV_TIMEOUT);
}

// Joins the parts of a unit that several slices share. All slices but the first of a unit start inside it: their
// CTAs here share its sums out, and the lanes of a CTA the parts of a sum, in an order that the number of slices fixes.
// (With one CTA joining a unit, a call for one sequence of 32000 positions, 74 slices to each of 8 units, took 35.4 us;
// so it takes 20.7 us. One of 131000: 59 us and 46 us. With eight loads at a time and 80 registers, not 64, 8 sequences
// of 32000 positions took 90 us in place of 81 us.)
constexpr int kCombineThreads = 128;
template <int D>
__global__ void __launch_bounds__(kCombineThreads, 8) kv4_combine_kernel(const __grid_constant__ AttnParams P, int R) {
  __shared__ int64_t prefix[kCombineThreads + 1], warp_sums[kCombineThreads / 32];
  const Kv4AttnLaunch &p = P.a;
  // (this grid starts once every CTA of the step kernel is past its own wait, so the lengths, which the
  // step kernel does not write, can be read before this one's)
  const Line line{&p, P.group, R, 31 - __clz(R), P.key_log2};
  const int chunk = (p.B + kCombineThreads - 1) / kCombineThreads;
  const int64_t all = line_prefix(line, kCombineThreads, chunk, prefix, warp_sums);
  const int ctas = slices(all, P.ctas, P.key_log2);
  const int c = static_cast<int>(blockIdx.x) + 1;
  Walk w;
  bool mine = c < ctas;
  int first = c, last = c;
  if (mine) {
    const int64_t from = slice_at(all, ctas, c);
    w.begin(line, prefix, kCombineThreads, chunk, from, from + 1);
    mine = w.tile != 0;
    auto slice_of = [&](int64_t x) {  // the slice that x lies in
      int k = min(static_cast<int>(static_cast<float>(x) / static_cast<float>(all) * ctas), ctas - 1);
      while (slice_at(all, ctas, k) > x) --k;
      while (slice_at(all, ctas, k + 1) <= x) ++k;
      return k;
    };
    if (mine) {
      first = slice_of(from - w.tile);
      last = slice_of(from - w.tile + w.tiles - 1);
    }
  }
  pdl_wait();  // (the last kernel of its call: it does not release the next call's kernels early)
  if (!mine) return;
  constexpr int V4 = D / 4, kAtOnce = 4;
  const int parts = last - first + 1, rank = c - first - 1;
  const int e0 = R * V4 * rank / (parts - 1), e1 = R * V4 * (rank + 1) / (parts - 1);
  int lanes = 1;  // of a sum
  while (lanes < 32 && 2 * lanes <= parts && kCombineThreads / (2 * lanes) >= e1 - e0) lanes *= 2;
  const int mine_at = threadIdx.x & (lanes - 1), lanes_log2 = 31 - __clz(lanes);
  for (int eb = e0; eb < e1; eb += kCombineThreads >> lanes_log2) {
    const int e = eb + static_cast<int>(threadIdx.x >> lanes_log2);
    const int r = e / V4, d = e % V4 * 4;
    const bool there = e < e1 && w.row_limit(r) > 0;
    float mx = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = first + mine_at; there && k0 <= last; k0 += kAtOnce * lanes) {  // four parts' loads at a time
      float2 ml[kAtOnce];
      float4 v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int k = k0 + i * lanes;
        const int64_t slot = 2 * k + (k == first);
        ml[i] = k <= last ? P.part_ml[slot * R + r] : make_float2(-INFINITY, 0.f);
        v[i] = k <= last ? *reinterpret_cast<const float4 *>(P.part_o + (slot * R + r) * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float now = mx;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) now = fmaxf(now, ml[i].x);
      const float keep = mx == -INFINITY && sum == 0.f ? 0.f : ex2_approx(mx - now);
      mx = now;
      sum *= keep, acc.x *= keep, acc.y *= keep, acc.z *= keep, acc.w *= keep;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const float f = ml[i].x == -INFINITY && ml[i].y == 0.f ? 0.f : ex2_approx(ml[i].x - mx);
        sum = fmaf(ml[i].y, f, sum);
        acc.x = fmaf(v[i].x, f, acc.x), acc.y = fmaf(v[i].y, f, acc.y);
        acc.z = fmaf(v[i].z, f, acc.z), acc.w = fmaf(v[i].w, f, acc.w);
      }
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const float mx2 = __shfl_xor_sync(0xFFFFFFFFu, mx, o), now = fmaxf(mx, mx2);
      const float f = mx == -INFINITY && sum == 0.f ? 0.f : ex2_approx(mx - now);
      auto add = [&](float x) {  // both sides' terms, each times its factor: the same sum on both
        x *= f;
        return x + __shfl_xor_sync(0xFFFFFFFFu, x, o);
      };
      sum = add(sum), acc.x = add(acc.x), acc.y = add(acc.y), acc.z = add(acc.z), acc.w = add(acc.w);
      mx = now;
    }
    if (!there || mine_at != 0) continue;
    const int64_t row = w.row_index(r);
    const float inv = row_inverse(mx, sum);
    *reinterpret_cast<uint2 *>(p.out + row * D + d) =
        make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    if (d == 0 && p.lse) p.lse[row] = row_lse(mx, sum, kPOff);
  }
}

// Whether the tensor-core form for 256-row blocks takes the call. What it costs goes by blocks of 256 rows in waves
// over the SMs, however few of their rows there are (1.66 us per 128 keys at 128 channels, 1.54 us at 64); the
// step form's cost by tiles of 16 rows over the whole card (2.9 ns per 64 keys, 1.9 ns): they meet where
// there are 283 (409) row tiles to a wave. Where the blocks' keys are split over CTAs a wave's tiles are that much
// shorter, so the tiles are counted as often. Measured beside that, at 8 key heads of 4 query heads each, step form and the other:
// 8 sequences of 32768 positions, 16 new tokens (256 row tiles, two splits) 392 us and 236 us, 32 (512) 764 us and
// 238 us; at 64 channels 246 us and 205 us, 476 us and 207 us. Short contexts, under a table of up to four pages, are
// latency: 8 sequences of 512 positions, 64 rows each 28.6 us and 14.2 us; one of 16 rows 11.6 us and 13.4 us, but 21 us
// and 18 us with the host's launches, of which this form makes one.
// One rule serves all sequences of a call: steps beside a prompt take blocks of 256 rows too (31 steps at 32768 positions and a
// piece of 2048 tokens of another, 64 query heads: 2855 us, as two calls 1926 us).
bool prompt_rows(const Kv4AttnLaunch &p, const Kv4PromptShape &g) {
  const int64_t group = p.Hq / p.Hk, rows = (p.max_new < p.T ? p.max_new : p.T) * group;
  if (rows <= 8) return false;
  auto row_blocks = [&](int64_t size) {  // of `size` rows: at most what the longest sequence has of each, and what all tokens make
    const int64_t by_max = p.B * ((rows + size - 1) / size), by_all = p.T * group / size + p.B;
    return p.Hk * (by_max < by_all ? by_max : by_all);
  };
  const int64_t sms = sm_count(), waves = (row_blocks(256) + sms - 1) / sms;
  if (p.cache.max_blocks <= 4 && waves <= 2) return true;
  return row_blocks(16) * (g.whole == 0 ? g.splits : 1) > (p.D == 128 ? 283 : 409) * waves;
}

// Rows of a tile: 16 read and convert a key once for what takes 8 twice (2.9 ns against 2 x 2.0 ns per 64 keys), but a
// warp's turn takes twice as long, which shows where there are few: with less than eight turns of 8 rows for
// each of the SMs' twelve warps, going by the longest context that the table holds, 8 it is (16 rows over 4096
// positions of one sequence 22 us against 29 us, over 32768 of eight 146 us against 114 us). Tiles of 32 rows at 64
// channels were slower yet: 43.5 us against 34.5 us for 13 sequences of 20 rows and up to 9001 tokens.
int64_t turns_of_8(const Kv4AttnLaunch &p) {
  const int64_t group = p.Hq / p.Hk, rows = (p.max_new < p.T ? p.max_new : p.T) * group;
  const int64_t by_max = p.B * ((rows + 7) / 8), by_all = p.T * group / 8 + p.B;
  return p.Hk * (by_max < by_all ? by_max : by_all) * p.cache.max_blocks * (DSV4_PAGE_POSITIONS / kTile);
}
int tile_rows(const Kv4AttnLaunch &p) {
  const int64_t rows = (p.max_new < p.T ? p.max_new : p.T) * (p.Hq / p.Hk);
  return rows <= 8 || turns_of_8(p) < int64_t(8) * 12 * sm_count() ? 8 : 16;
}

template <int D, int NT>
cudaError_t launch_step(AttnParams &P, cudaStream_t st) {
  const size_t smem = sizeof(AttnSmem<D, NT>) + 128;
  const cudaError_t e = launch_large<kv4_step_kernel<D, NT>>(dim3(P.ctas), dim3(kThreadsA), smem, st, P);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_combine_kernel<D>, dim3(P.ctas - 1), dim3(kCombineThreads), 0, st, 1, P, 8 * NT);
}

// The form with scores on the tensor cores takes calls of at least four of its tiles for each of its CTAs, going by the
// longest context that the table holds; with fewer its start and its longer turns show. At 8 key heads of 8 query
// heads each, the kernel above and this one: 8 sequences of 2000 positions (1024 tiles) 16.1 us and 21.4 us, one of
// 32000 (2000) 22.1 us and 26.0 us; 64 of 500 (2048) 30.1 us and 29.0 us, 8 of 8000 (4096) 32.0 us and 30.3 us, 8 of
// 32000 81.3 us and 73.0 us. All under tables as wide as the contexts: under a wider one the short ones take this form too (8 of 2000 under
// 512 pages 21.4 us).
// Its tensor map wants the codes at a multiple of 32 bytes and rows that an int counts.
bool tensor_scores(const Kv4AttnLaunch &p, int rows) {
  return p.D == 128 && rows == 8 && turns_of_8(p) >= int64_t(4) * (kTcKeys / kTile) * kTcResident * sm_count() &&
         static_cast<int64_t>(p.cache.num_pages) * p.Hk * DSV4_PAGE_POSITIONS <= 0x7FFFFFFF &&
         reinterpret_cast<uintptr_t>(p.cache.k_codes) % 32 == 0;
}

bool make_codes_map(CUtensorMap *map, const Kv4AttnLaunch &p) {
  auto fn = get_encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(p.cache.num_pages) * p.Hk * DSV4_PAGE_POSITIONS};  // codes
  const cuuint64_t strides[1] = {64};                                                                         // bytes
  const cuuint32_t box[2] = {128, kTcKeys}, steps[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, p.cache.k_codes, dims, strides, box, steps,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_tc_step(AttnParams &P, const CUtensorMap &map, cudaStream_t st) {
  const cudaError_t e =
      launch_large<kv4_step_tc_kernel>(dim3(P.ctas), dim3(kTcThreads), sizeof(TcStepSmem) + 1024, st, P, map);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv4_combine_kernel<128>, dim3(P.ctas - 1), dim3(kCombineThreads), 0, st, 1, P, 8);
}

}  // namespace

Kv4AttnPlan kv4_attention_plan(const Kv4AttnLaunch &p) {
  Kv4AttnPlan plan{};
  plan.shape = kv4_prompt_shape(p);
  if (prompt_rows(p, plan.shape)) {
    plan.form = DSV4_KV4_PROMPT;
    plan.rows = 256;
  } else {
    plan.rows = tile_rows(p);
    plan.form = tensor_scores(p, plan.rows) ? DSV4_KV4_STEP_TENSOR : DSV4_KV4_STEP;
  }
  return plan;
}

namespace {
size_t step_workspace_bytes(int D, int R) {
  const size_t rows = static_cast<size_t>(sm_count()) * resident_ctas(D, R / 8) * 2 * R;
  return align_up(rows * D * sizeof(float), 256) + align_up(rows * sizeof(float2), 256);
}
size_t prompt_workspace_bytes(int D, int64_t parts) { return align_up(kv4_prompt_workspace_bytes(D, parts) + 1, 256); }
}  // namespace

size_t kv4_attention_workspace_bytes(const Kv4AttnLaunch &p, const Kv4AttnPlan &plan) {
  return plan.form == DSV4_KV4_PROMPT ? prompt_workspace_bytes(p.D, kv4_prompt_parts(p, plan.shape))
                                      : step_workspace_bytes(p.D, plan.rows);
}

size_t kv4_attention_workspace_limit(const Kv4AttnLaunch &p) {
  size_t most = step_workspace_bytes(p.D, 8);
  if ((p.max_new < p.T ? p.max_new : p.T) * static_cast<int64_t>(p.Hq / p.Hk) > 8) {  // the other forms want more rows
    const size_t step = step_workspace_bytes(p.D, 16), prompt = prompt_workspace_bytes(p.D, kv4_prompt_most_parts(p));
    most = most > step ? most : step;
    most = most > prompt ? most : prompt;
  }
  return most;
}

cudaError_t launch_kv4_attention(const Kv4AttnLaunch &q, const Kv4AttnPlan &plan, void *ws, cudaStream_t st) {
  if (plan.form == DSV4_KV4_PROMPT) return launch_kv4_prompt(q, plan.shape, ws, st);
  AttnParams P{};
  P.a = q;
  const int R = plan.rows;
  const bool tc = plan.form == DSV4_KV4_STEP_TENSOR;
  P.ctas = sm_count() * (tc ? kTcResident : resident_ctas(q.D, R / 8));
  P.key_log2 = tc ? 7 : 6;
  P.group = q.Hq / q.Hk;
  P.part_o = static_cast<float *>(ws);
  P.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) +
                                         align_up(static_cast<size_t>(P.ctas) * 2 * R * q.D * sizeof(float), 256));
  if (tc) {
    CUtensorMap map;
    return make_codes_map(&map, q) ? launch_tc_step(P, map, st) : cudaErrorNotSupported;
  }
  if (q.D == 64) return R == 8 ? launch_step<64, 1>(P, st) : launch_step<64, 2>(P, st);
  return R == 8 ? launch_step<128, 1>(P, st) : launch_step<128, 2>(P, st);
}

}  // namespace dsv4
