// Attention over the 4-bit key/value cache, rows in tiles of 256: prompts and pieces of them.
//
// The same operation as kv4_attention.cu's step kernel (there the formulas), for calls whose
// sequences bring many rows (new tokens x query heads of a key/value head): bound by the tensor
// cores and by the exponentials, not by memory. A CTA takes 256 rows of one key/value head of one
// sequence, as two tiles of 128, and walks over the keys 128 at a time:
//   warps 0-3, 4-7   softmax of row tile 0 and 1, one row per thread
//   warps 8-11       codes -> fp16 K and V tiles in shared memory (128B swizzle, two stages)
//   warp 12          issues tcgen05.mma (kind::f16, M = 128):
//                    S = Q K^T (Q, K from shared memory, S in TMEM) and
//                    O += P V  (P in TMEM over S's columns, V from shared memory)
// TMEM is full: S (128 columns) and O (D) of both row tiles. The two tiles alternate, so that one
// tile's products run while the other's softmax does. The conversion of a K and V tile
// (exact, see kv4_attention.cu) is shared by both row tiles: 2 x 128 x D codes against 4 x 128 x 128 x D
// multiply-adds.
// Softmax: the reference R that weights are taken against is raised (and O scaled) only when a
// tile's maximum exceeds it by more than 2^8; weights are held times 2^7, at most 2^15 in fp16.
// With few blocks of rows the keys of a block are split over CTAs, which a second kernel joins.
// Measured: eight prompts of 4096 tokens, 32 heads over 8 of 128 channels, 1155 us (952 TFLOP/s); 2048 tokens behind
// 14336 442 us (1167 TFLOP/s; 457 us without the last wave shared out); a tile pair of 256 x 128 takes 1.85 us, 1342 TFLOP/s.
// A thread keeps its S row in 128 registers between the maximum and the weights (the warpgroups'
// registers are split 184, 184, 96, 48), and hands its weights over in halves of 64 keys.
#include "kv4_device.cuh"

namespace dsv4 {

namespace {

constexpr int kRows = 128;             // rows of a row tile
constexpr int kKeysLog2 = 7;
constexpr int kKeys = 1 << kKeysLog2;  // keys of a stage
constexpr int kPThreads = 512;         // 4 warpgroups
constexpr float kRaise = 8.f;          // log2 that a maximum may exceed the reference by
constexpr float kPOffP = 7.f;          // weights are held times 2^7

struct PromptParams {
  Kv4AttnLaunch a;
  int row_blocks;  // blocks of 256 rows along the grid
  int whole;       // units that one CTA takes whole; the keys of the others are shared by
  int splits;      // so many CTAs
  float4 *part_o;  // [unit - whole][split][row tile][D / 4][128 rows], unnormalised sums
  float2 *part_ml; // [unit - whole][split][row tile][128 rows]: reference (log2) and sum
};

template <int D>
struct alignas(1024) PromptSmem {
  static constexpr int kBlk = kKeys * 128;  // 128 rows x 64 channels
  uint8_t q[2][D / 64][kBlk];
  uint8_t k[2][D / 64][kBlk];
  uint8_t v[2][D / 64][kBlk];
  uint64_t q_full, k_full[2], v_full[2], kv_empty[2], s_full[2], p_full[2][2], o_done[2], mma_done;
  uint32_t tmem_base;
  int abort_flag;
  int bad[4];                  // the tile's page does not exist (tile index mod 4)
  int nan_at[D / kKv4Block];   // smallest position with a NaN value block
};

// tcgen05.mma kind::f16, A and B in shared memory (descriptors that share their high word) or A in TMEM
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc)
      : "memory");
}

// 32 lanes x 32 bits, 16 consecutive columns
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xFFFFFFFFu, x); }

// Registers of a warpgroup: the launch gives 512 threads x 128; softmax 2 x 184 + conversion 96 + products 48 = 4 x 128.
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// tiles of keys that each of `splits` CTAs takes of a unit's T
__device__ __forceinline__ int share_of(int T, int splits) { return (T + splits - 1) / splits; }

// the unit of a CTA: rows 256 rb .. of one key/value head of one sequence
struct PromptUnit {
  Seq q;
  int G, kvh;
  int64_t row0, rows;  // first row, rows of the sequence
  int j0;              // the CTA's first tile of keys
  __device__ __forceinline__ int limit(int64_t row) const {  // positions that the row sees (0: no such row)
    if (row >= rows) return 0;
    return min(q.n, q.start + static_cast<int>(row / G) + 1);
  }
  // tiles of keys that row tile t reads
  __device__ __forceinline__ int tiles(int t) const {
    const int64_t first = row0 + t * kRows;
    if (first >= rows) return 0;
    return (limit(min(first + kRows, rows) - 1) + kKeys - 1) / kKeys;
  }
};

template <int D>
__device__ void convert_role(const Kv4AttnLaunch &p, PromptSmem<D> &S, const PromptUnit &u, int s, int T, int count,
                             int events, bool &dead) {
  constexpr int W = D / 32;  // 16-byte pieces of a row's codes
  const int r = threadIdx.x - 256, lane = threadIdx.x & 31;
  const int32_t *table = p.cache.block_table + static_cast<int64_t>(s) * p.cache.max_blocks;
  uint4 kc[W], vc[W];
  uint32_t ks = 0, vs = 0;
  bool bad = false;
  auto load = [&](int j) {
    const int page = table[j / (DSV4_PAGE_POSITIONS / kKeys)];
    bad = page < 0 || page >= p.cache.num_pages;
    if (bad) {
      if (r == 0) report(p.d_status, DSV4_DEV_BAD_PAGE);
#pragma unroll
      for (int i = 0; i < W; ++i) kc[i] = vc[i] = make_uint4(0, 0, 0, 0);
      ks = vs = 0;
      return;
    }
    const int64_t row = (static_cast<int64_t>(page) * p.Hk + u.kvh) * DSV4_PAGE_POSITIONS +
                        j % (DSV4_PAGE_POSITIONS / kKeys) * kKeys + r;
    const uint4 *ksrc = reinterpret_cast<const uint4 *>(p.cache.k_codes + row * (D / 2));
    const uint4 *vsrc = reinterpret_cast<const uint4 *>(p.cache.v_codes + row * (D / 2));
#pragma unroll
    for (int i = 0; i < D / 32; ++i) kc[i] = ksrc[i], vc[i] = vsrc[i];
    if constexpr (D == 128) {
      ks = *reinterpret_cast<const uint32_t *>(p.cache.k_scales + row * 4);
      vs = *reinterpret_cast<const uint32_t *>(p.cache.v_scales + row * 4);
    } else {
      ks = *reinterpret_cast<const uint16_t *>(p.cache.k_scales + row * 2);
      vs = *reinterpret_cast<const uint16_t *>(p.cache.v_scales + row * 2);
    }
  };
  auto write = [&](uint8_t(&dst)[D / 64][PromptSmem<D>::kBlk], const uint4(&c)[W], uint32_t sc) {
#pragma unroll
    for (int i = 0; i < W; ++i) {  // piece i: channels 32 i .. 32 i + 31, one scale
      const float f = scale_value(sc >> (8 * i) & 255u);
      const uint32_t f2 = pack_half2(f, f);
      const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t h[4];
        e2m1x8_to_half2(w[k], h);
        *reinterpret_cast<uint4 *>(&dst[i / 2][sw128_offset(r, i % 2 * 4 + k)]) =
            make_uint4(hmul2(h[0], f2), hmul2(h[1], f2), hmul2(h[2], f2), hmul2(h[3], f2));
      }
    }
  };
  if (T > 0) load(u.j0);
  for (int j = 0; j < T; ++j, ++count) {
    uint4 k0[W], v0[W];
#pragma unroll
    for (int i = 0; i < W; ++i) k0[i] = kc[i], v0[i] = vc[i];
    const uint32_t ks0 = ks;
    uint32_t vs0 = vs;
    const bool bad0 = bad;
    if (j + 1 < T) load(u.j0 + j + 1);
    const int st = count & 1;
    if (dead) continue;
    // (K's stage is free: its last product came before event j - 2, which V of tile j - 1 waited for)
    write(S.k[st], k0, ks0);
    if (r == 0) S.bad[count & 3] = bad0;
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.k_full[st]);
    const int key = (u.j0 + j) * kKeys + r;
    if (key >= u.q.n) {
      vs0 = 0;  // not a position of the sequence: 2^-127, zero in fp16
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if ((vs0 >> (8 * i) & 255u) == 255u) {
          atomicMin(&S.nan_at[i], key);
          vs0 &= ~(255u << (8 * i));
        }
    }
    // events of a unit: 0 after S(0), j + 1 after PV(j) and S(j + 1); they take turns on two barriers, as one
    // may be through before its predecessor is asked for
    const int e = events + j - 1;
    const bool ok = j < 1 || mbar_spin(&S.kv_empty[e & 1], (e >> 1) & 1, &S.abort_flag);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      dead = true;
      continue;
    }
    write(S.v[st], v0, vs0);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.v_full[st]);
  }
}

// The products, in the order PV0 S0 PV1 S1 of each tile j (S of tile j + 1), so that one row tile's run
// beside the other's softmax. T0 and T1: tiles of the two row tiles; kv, done: tiles in the CTA's units
// before. The whole warp runs this, one lane issues. An issue waits for the tensor pipe and every
// hand-over costs some 150 cycles of it, so there are as few as the data needs: s_full also says
// that the product before it (O up to the last tile) is done, and one event per tile frees V of tile j
// and K of tile j + 1.
template <int D>
__device__ __forceinline__ void mma_role(PromptSmem<D> &S, uint32_t tmem, int T0, int T1, int kv, int (&done)[2], int units,
                                         bool &dead) {
  constexpr uint32_t id_s = idesc_f16(kRows, kKeys, 0, 0), id_o = idesc_f16(kRows, D, 0, 1);
  constexpr uint32_t kB = PromptSmem<D>::kBlk;
  const int T = max(T0, T1);
  auto wait = [&](uint64_t *bar, int phase) {
    if (!dead) dead = !__all_sync(0xFFFFFFFFu, mbar_spin(bar, static_cast<uint32_t>(phase & 1), &S.abort_flag));
    return !dead;
  };
  constexpr uint32_t kTileStep = (D / 64) * kB >> 4;  // descriptor units from one tile (q) or stage (k, v) to the next
  const uint64_t qd = sw128_desc(smem_u32(S.q[0][0]), 16, 1024), vd = sw128_desc(smem_u32(S.v[0][0]), kB, 1024);
  const uint32_t q_lo = static_cast<uint32_t>(qd), q_hi = static_cast<uint32_t>(qd >> 32);
  const uint32_t k_lo = static_cast<uint32_t>(sw128_desc(smem_u32(S.k[0][0]), 16, 1024));
  const uint32_t v_lo = static_cast<uint32_t>(vd), v_hi = static_cast<uint32_t>(vd >> 32);
  auto commit = [&](uint64_t *bar) {
    if (elect_one()) mma_commit(bar);
  };
  auto issue_s = [&](int t, int st) {
    tc_fence_after();
    const uint32_t a0 = q_lo + t * kTileStep, b0 = k_lo + st * kTileStep;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = (kk / 4) * (kB >> 4) + 2 * (kk & 3);
      if (elect_one()) mma_ss(tmem + 128u * t, a0 + off, b0 + off, q_hi, id_s, kk > 0 ? 1u : 0u);
    }
    commit(&S.s_full[t]);
  };
  auto issue_o = [&](int t, int st, int half, uint32_t acc) {
    tc_fence_after();
    const uint32_t d = tmem + 256u + static_cast<uint32_t>(D * t), a0 = tmem + 128u * t + 32u * half;
    const uint32_t b0 = v_lo + st * kTileStep + half * (kKeys / 2 * 128 >> 4);
#pragma unroll
    for (int i = 0; i < kKeys / 32; ++i)  // 16 keys: 8 columns of P, 2048 bytes of V
      if (elect_one()) mma_ts(d, a0 + 8u * i, b0 + i * (2048 >> 4), v_hi, id_o, i > 0 ? 1u : acc);
  };
  if (T == 0 || !wait(&S.q_full, units) || !wait(&S.k_full[kv & 1], kv / 2)) return;
  if (T0 > 0) issue_s(0, kv & 1);
  if (T1 > 0) issue_s(1, kv & 1);
  int e = kv + units;  // the unit's first event: each unit before had one more than tiles
  commit(&S.kv_empty[e & 1]);
  if (!wait(&S.v_full[kv & 1], kv / 2)) return;
  for (int j = 0; j < T; ++j) {
    const int st = (kv + j) & 1, nx = st ^ 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int Tt = t == 0 ? T0 : T1;
      if (j < Tt) {
        if (!wait(&S.p_full[t][0], done[t] + j)) return;
        issue_o(t, st, 0, j > 0 ? 1u : 0u);
        if (!wait(&S.p_full[t][1], done[t] + j)) return;
        issue_o(t, st, 1, 1u);
        if (j + 1 == Tt) commit(&S.o_done[t]);
      }
      if (t == 0 && j + 1 < T && !wait(&S.k_full[nx], (kv + j + 1) / 2)) return;
      if (j + 1 < Tt) issue_s(t, nx);
    }
    ++e;
    commit(&S.kv_empty[e & 1]);
    if (j + 1 < T && !wait(&S.v_full[nx], (kv + j + 1) / 2)) return;
  }
  done[0] += T0;
  done[1] += T1;
}

template <int D>
__device__ void softmax_role(const Kv4AttnLaunch &p, PromptSmem<D> &S, const PromptUnit &u, int seq, uint32_t tmem, int t,
                             int T, int kv, int &done, int &units, bool &dead, float4 *part_o, float2 *part_ml) {
  const int r = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(threadIdx.x & 96) << 16;
  const uint32_t s_at = tmem + 128u * t + lanes, o_at = tmem + 256u + static_cast<uint32_t>(D * t) + lanes;
  const int64_t row = u.row0 + t * kRows + r;
  const int lim = u.limit(row);
  const int64_t index = (u.q.tok0 + row / u.G) * p.Hq + u.kvh * u.G + row % u.G;  // of rows that exist
  // the query row: scaled by a power of two into fp16's range (see kv4_attention.cu)
  float rs;
  {
    uint4 raw[D / 8];
    const uint16_t *src = p.q + (u.q.tok0 + row / u.G) * p.q_stride + static_cast<int64_t>(u.kvh * u.G + row % u.G) * D;
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      raw[i] = lim > 0 ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) am = max(am, max((w[k] << 16) & 0x7FFF0000u, w[k] & 0x7FFF0000u));
    }
    const int ex = static_cast<int>(am >> 23) - 127;
    const int sh = (am == 0 || ex >= 128) ? 0 : min(max(14 - ex, -113), 120);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + sh) << 23);
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        h[k] = pack_half2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xFFFF0000u) * up);
      *reinterpret_cast<uint4 *>(&S.q[t][i / 8][sw128_offset(r, i % 8)]) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    // (not below float32's normal numbers: a masked position is minus infinity times this)
    rs = fmaxf(p.softmax_scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - sh) << 23), 1.17549435e-38f);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&S.q_full);

  float R = -INFINITY;
  uint64_t la = pack_f32x2(0.f, 0.f), lb = la;  // sums of the weights of every fourth pair of columns
  // positions that every row of the warp sees (rows that do not exist see none and are not asked)
  const int least = __reduce_min_sync(0xFFFFFFFFu, row < u.rows ? lim : 0x7FFFFFFF);
  for (int j = 0; j < T; ++j) {
    if (dead) break;
    const bool ok = mbar_spin(&S.s_full[t], (done + j) & 1, &S.abort_flag);
    if (!__all_sync(0xFFFFFFFFu, ok)) {
      dead = true;
      break;
    }
    tc_fence_after();
    const int key0 = (u.j0 + j) * kKeys;
    const bool edge = key0 + kKeys > least;
    const bool bad = S.bad[(kv + j) & 3];
    const int vis = bad ? 0 : lim - key0;  // columns that the row sees
    uint32_t a[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, a[c]);
    tmem_ld_wait();
    if (edge || bad) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (32 * c + i >= vis) a[c][i] = 0xFF800000u;
    }
    float mc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      mc[c] = __uint_as_float(a[c][0]);
#pragma unroll
      for (int i = 1; i < 31; i += 2)
        mc[c] = fmaxf(fmaxf(mc[c], __uint_as_float(a[c][i])), __uint_as_float(a[c][i + 1]));
      mc[c] = fmaxf(mc[c], __uint_as_float(a[c][31]));
    }
    const float mx = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
    const float z = mx * rs;
    const bool raise = z > R + kRaise || (R == -INFINITY && z > R);
    if (__any_sync(0xFFFFFFFFu, raise)) {
      const float f = raise ? ex2_approx(R - z) : 1.f;  // (R = -inf: zero)
      if (raise) R = z;
      la = mul_f32x2(la, pack_f32x2(f, f));
      lb = mul_f32x2(lb, pack_f32x2(f, f));
      if (j > 0) {  // (s_full of tile j: the products of tile j - 1 are in O)
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_at + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
          tmem_st32(o_at + c, o);
        }
      }
    }
    const float off = R == -INFINITY ? 0.f : kPOffP - R;
    const uint64_t rs2 = pack_f32x2(rs, rs), off2 = pack_f32x2(off, off);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float x0, x1;
        unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(a[c][2 * i]), __uint_as_float(a[c][2 * i + 1])), rs2, off2), x0, x1);
        x0 = ex2_approx(x0);
        x1 = ex2_approx(x1);
        if (i & 1) lb = add_f32x2(lb, pack_f32x2(x0, x1));
        else la = add_f32x2(la, pack_f32x2(x0, x1));
        w[i] = pack_half2(x0, x1);
      }
      tmem_st16(s_at + 16 * c, w);
      if (c & 1) {
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[t][c / 2]);
      }
    }
  }
  if (T > 0 && !dead) {
    const bool ok = mbar_spin(&S.o_done[t], units & 1, &S.abort_flag);
    if (__all_sync(0xFFFFFFFFu, ok)) {
      tc_fence_after();
      float l0, l1;
      unpack_f32x2(add_f32x2(la, lb), l0, l1);
      const float l = l0 + l1;
      if (R == -INFINITY && row_sees(p, seq, u.j0, u.j0 + T, kKeysLog2, lim)) R = kLeast;
      const float inv = row_inverse(R, l);
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_at + c, o);
        tmem_ld_wait();
        const float nan = S.nan_at[c / kKv4Block] < lim ? __uint_as_float(0x7FC00000u) : 1.f;
        if (part_o) {  // (a row's neighbours lie beside it, so that a warp's stores are whole lines)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part_o[(c / 4 + i) * kRows + r] =
                make_float4(__uint_as_float(o[4 * i]) * nan, __uint_as_float(o[4 * i + 1]) * nan,
                            __uint_as_float(o[4 * i + 2]) * nan, __uint_as_float(o[4 * i + 3]) * nan);
        } else if (lim > 0) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.out + index * D + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack_bf16(__uint_as_float(o[8 * i + 2 * k]) * inv * nan,
                                 __uint_as_float(o[8 * i + 2 * k + 1]) * inv * nan);
            dst[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      tc_fence_before();
      if (part_o) part_ml[r] = make_float2(R, l);
      else if (lim > 0 && p.lse) p.lse[index] = row_lse(R, l, kPOffP);
    } else {
      dead = true;
    }
  }
  done += T;
  if (T > 0) ++units;  // (units in which this row tile had rows)
}

template <int D>
__global__ void __launch_bounds__(kPThreads, 1) kv4_prompt_kernel(const __grid_constant__ PromptParams P) {
  extern __shared__ uint8_t smem_raw[];
  PromptSmem<D> &S = *reinterpret_cast<PromptSmem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Kv4AttnLaunch &p = P.a;
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  constexpr uint32_t kCols = 512;
  // Blocks of later rows (more keys) come first; the sequences and heads of one block of rows are neighbours.
  const int shared_at = static_cast<int>(blockIdx.x) - P.whole;  // this CTA among those that share
  // whether a join follows in this call (the last kernel of a call does not release the next call's early)
  const bool joined = static_cast<unsigned>(P.whole) < gridDim.x;
  const int splits = shared_at < 0 ? 1 : P.splits, split = shared_at < 0 ? 0 : shared_at % splits;
  const int unit = shared_at < 0 ? static_cast<int>(blockIdx.x) : P.whole + shared_at / splits;
  const int heads = p.B * p.Hk, first_rb = P.row_blocks - 1 - unit / heads, s = unit % heads / p.Hk, kvh = unit % heads % p.Hk;
  if (tid == 0) {
    mbar_init(&S.q_full, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], 4);
      mbar_init(&S.v_full[i], 4);
      mbar_init(&S.kv_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i][0], 4);
      mbar_init(&S.p_full[i][1], 4);
      mbar_init(&S.o_done[i], 1);
    }
    mbar_init(&S.mma_done, 1);
    S.abort_flag = 0;
    fence_mbar_init();
  }
  pdl_wait();
  PromptUnit u;
  u.G = p.Hq / p.Hk;
  u.kvh = kvh;
  const bool any = seq_info(p, s, &u.q, tid == 0);
  u.rows = any ? static_cast<int64_t>(u.q.len) * u.G : 0;
  u.row0 = static_cast<int64_t>(first_rb) * 2 * kRows;
  const int tiles = u.row0 < u.rows ? max(u.tiles(0), u.tiles(1)) : 0;
  if (split * share_of(tiles, splits) >= tiles) {  // (no such rows, or nothing left for this split)
    if (joined) pdl_launch_dependents();
    return;
  }
  if (warp == 12) {
    tmem_alloc(&S.tmem_base, kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (joined) pdl_launch_dependents();
  const uint32_t tmem = __reduce_max_sync(0xFFFFFFFFu, S.tmem_base);

  // Every role walks over the CTA's units (more than one only where a sequence brings more new
  // tokens than the call's max_new says) and meets the others before and after each.
  int kv = 0;
  bool dead = false, part = false;
  // (counts that steer loops pass through a warp reduction, whose result the compiler knows to be the
  // same in all lanes: the issuing warp's operands then stay in uniform registers)
  const int64_t blocks = (u.rows + 2 * kRows - 1) / (2 * kRows) - first_rb;
  // (the rows that max_new does not speak of have no place for parts: the first split takes them whole)
  const int turns = split > 0 ? 1 : uniform(static_cast<int>((blocks + P.row_blocks - 1) / P.row_blocks));
  auto units_loop = [&](auto &&role) {
    for (int turn = 0; turn < turns; ++turn) {
      u.row0 = (first_rb + static_cast<int64_t>(turn) * P.row_blocks) * 2 * kRows;
      int T0 = uniform(u.tiles(0)), T1 = uniform(u.tiles(1));
      u.j0 = 0;
      part = splits > 1 && turn == 0;
      if (part) {
        const int share = share_of(max(T0, T1), splits);
        u.j0 = split * share;
        T0 = min(max(T0 - u.j0, 0), share);
        T1 = min(max(T1 - u.j0, 0), share);
      }
      if (tid < D / kKv4Block) S.nan_at[tid] = 0x7FFFFFFF;
      __syncthreads();
      role(T0, T1);
      kv += max(T0, T1);
      __syncthreads();
    }
  };
  if (warp < 8) {
    more_registers<184>();
    int done = 0, n_units = 0;
    units_loop([&](int T0, int T1) {
      const int t = warp / 4;
      const int64_t slot = part ? (static_cast<int64_t>(unit - P.whole) * splits + split) * 2 + t : 0;
      softmax_role<D>(p, S, u, s, tmem, t, t == 0 ? T0 : T1, kv, done, n_units, dead,
                      part ? P.part_o + slot * (D / 4 * kRows) : nullptr, part ? P.part_ml + slot * kRows : nullptr);
    });
  } else if (warp < 12) {
    fewer_registers<96>();
    int events = 0;  // of kv_empty in the units before
    units_loop([&](int T0, int T1) {
      convert_role<D>(p, S, u, s, max(T0, T1), kv, events, dead);
      events += max(T0, T1) + 1;
    });
  } else {
    fewer_registers<48>();
    int n_units = 0, done[2] = {0, 0};
    units_loop([&](int T0, int T1) {
      if (warp == 12) mma_role<D>(S, tmem, T0, T1, kv, done, n_units, dead);
      ++n_units;
    });
  }
  if (warp == 12) {  // every product issued here ends before the TMEM is freed
    if (elect_one()) mma_commit(&S.mma_done);
    volatile int dummy = 0;
    mbar_wait(&S.mma_done, 0u, &dummy);
  }
  if (tid == 0 && S.abort_flag) report(p.d_status, DSV4_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

// Joins the splits of a unit: a block takes 32 channels of the 128 rows of a row tile, a thread a row.
template <int D>
__global__ void __launch_bounds__(kRows) kv4_prompt_combine_kernel(const __grid_constant__ PromptParams P) {
  const Kv4AttnLaunch &p = P.a;
  const int heads = p.B * p.Hk, t = blockIdx.x & 1, shared_at = static_cast<int>(blockIdx.x >> 1), r = threadIdx.x;
  const int unit = P.whole + shared_at, rb = P.row_blocks - 1 - unit / heads, s = unit % heads / p.Hk, c0 = blockIdx.y * 32;
  // (this grid starts once every CTA of the first kernel is past its own wait: the lengths can be read)
  PromptUnit u;
  u.G = p.Hq / p.Hk;
  u.kvh = unit % heads % p.Hk;
  const bool any = seq_info(p, s, &u.q, false);
  u.rows = any ? static_cast<int64_t>(u.q.len) * u.G : 0;
  u.row0 = static_cast<int64_t>(rb) * 2 * kRows;
  const int64_t row = u.row0 + t * kRows + r;
  int parts = 0;
  if (u.row0 < u.rows) {
    const int Tt = u.tiles(t), share = share_of(max(u.tiles(0), u.tiles(1)), P.splits);
    parts = (Tt + share - 1) / share;
  }
  pdl_wait();  // (the last kernel of its call: it does not release the next call's kernels early)
  if (row >= u.rows) return;
  const int64_t index = (u.q.tok0 + row / u.G) * p.Hq + u.kvh * u.G + row % u.G;
  const int64_t slot0 = static_cast<int64_t>(shared_at) * P.splits * 2 + t;
  float top = -INFINITY;
  for (int k = 0; k < parts; ++k) top = fmaxf(top, P.part_ml[(slot0 + 2 * k) * kRows + r].x);
  float sum = 0.f, acc[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const float2 ml = P.part_ml[(slot0 + 2 * k) * kRows + r];
    const float f = ml.x == -INFINITY && ml.y == 0.f ? 0.f : ex2_approx(ml.x - top);
    sum = fmaf(ml.y, f, sum);
    const float4 *src = P.part_o + (slot0 + 2 * k) * (D / 4 * kRows) + c0 / 4 * kRows + r;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 v = src[i * kRows];
      acc[4 * i] = fmaf(v.x, f, acc[4 * i]), acc[4 * i + 1] = fmaf(v.y, f, acc[4 * i + 1]);
      acc[4 * i + 2] = fmaf(v.z, f, acc[4 * i + 2]), acc[4 * i + 3] = fmaf(v.w, f, acc[4 * i + 3]);
    }
  }
  const float inv = row_inverse(top, sum);
  uint4 *dst = reinterpret_cast<uint4 *>(p.out + index * D + c0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    dst[i] = make_uint4(pack_bf16(acc[8 * i] * inv, acc[8 * i + 1] * inv), pack_bf16(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                        pack_bf16(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv), pack_bf16(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
  if (c0 == 0 && p.lse) p.lse[index] = row_lse(top, sum, kPOffP);
}

template <int D>
cudaError_t launch_typed(const PromptParams &P, cudaStream_t st) {
  const size_t smem = sizeof(PromptSmem<D>) + 1024;
  const unsigned shared = static_cast<unsigned>(P.row_blocks) * P.a.B * P.a.Hk - P.whole;
  const cudaError_t e = launch_large<kv4_prompt_kernel<D>>(dim3(P.whole + shared * P.splits), dim3(kPThreads), smem, st, P);
  if (e != cudaSuccess || shared == 0) return e;
  return launch_pdl(kv4_prompt_combine_kernel<D>, dim3(2 * shared, D / 32), dim3(kRows), 0, st, 1, P);
}

}  // namespace

// Blocks of 256 rows of the longest sequence, and how their keys are shared out. With at most half as many units (blocks x
// key heads x sequences) as SMs every unit's keys go to as many CTAs as fit one wave, four tiles of 128 keys each at least of the
// longest context that the table holds. With one to four waves of units the last, partial wave is shared by two to eight CTAs a
// unit where that shortens it by an eighth of a unit or more (2048 tokens behind 14336, 256 units on 148 SMs, the last 108 by
// four: see the measurement at the file's head).
Kv4PromptShape kv4_prompt_shape(const Kv4AttnLaunch &p) {
  Kv4PromptShape g;
  const int64_t heads = static_cast<int64_t>(p.B) * p.Hk;
  const int64_t most = p.max_new < p.T ? p.max_new : p.T;
  int64_t blocks = (most * (p.Hq / p.Hk) + 2 * kRows - 1) / (2 * kRows);
  const int64_t room = (int64_t(1) << 30) / heads;  // (a CTA walks on over rows beyond the grid)
  if (blocks > room) blocks = room;
  if (blocks < 1) blocks = 1;
  g.row_blocks = static_cast<int>(blocks);
  const int64_t units = blocks * heads, sms = sm_count();
  const int64_t tiles = static_cast<int64_t>(p.cache.max_blocks) * (DSV4_PAGE_POSITIONS / kKeys);
  g.whole = static_cast<int>(units);
  g.splits = 1;
  if (2 * units <= sms) {
    int64_t splits = sms / units;
    if (splits > tiles / 4) splits = tiles / 4;
    if (splits >= 2) g.whole = 0, g.splits = static_cast<int>(splits);
  } else if (units > sms && units <= 4 * sms && units % sms != 0) {
    const int64_t rest = units % sms;
    double best = 1.0 - 0.125;
    for (int k = 2; k <= 8 && k <= tiles / 8; ++k) {
      const double time = static_cast<double>((rest * k + sms - 1) / sms) / k;
      if (time < best) best = time, g.whole = static_cast<int>(units - rest), g.splits = k;
    }
  }
  return g;
}

// A call of no more units has as many parts at most: up to half the SMs' number of units, one wave; with more, as many
// waves as `splits` CTAs a unit may take to be an eighth of a unit shorter than one, ceil(7/8 splits) - 1.
int64_t kv4_prompt_most_parts(const Kv4AttnLaunch &p) {
  const int64_t tiles = static_cast<int64_t>(p.cache.max_blocks) * (DSV4_PAGE_POSITIONS / kKeys), sms = sm_count();
  const Kv4PromptShape g = kv4_prompt_shape(p);
  int64_t parts = tiles >= 8 ? sms : 0;
  if (static_cast<int64_t>(g.row_blocks) * p.B * p.Hk > sms)
    for (int k = 2; k <= 8 && k <= tiles / 8; ++k) parts = ((7 * k + 7) / 8 - 1) * sms;
  return parts;
}

size_t kv4_prompt_workspace_bytes(int dim, int64_t parts) {
  const size_t rows = static_cast<size_t>(parts) * 2 * kRows;
  return align_up(rows * dim * sizeof(float), 256) + align_up(rows * sizeof(float2), 256);
}

cudaError_t launch_kv4_prompt(const Kv4AttnLaunch &q, const Kv4PromptShape &g, void *ws, cudaStream_t st) {
  PromptParams P{};
  P.a = q;
  P.row_blocks = g.row_blocks;
  P.whole = g.whole;
  P.splits = g.splits;
  P.part_o = static_cast<float4 *>(ws);
  P.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(ws) + align_up(static_cast<size_t>(kv4_prompt_parts(q, g)) * 2 * kRows * q.D * sizeof(float), 256));
  return q.D == 64 ? launch_typed<64>(P, st) : launch_typed<128>(P, st);
}

}  // namespace dsv4
