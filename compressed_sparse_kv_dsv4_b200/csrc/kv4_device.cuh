// Device code that the attention kernels over the 4-bit key/value cache share.
#pragma once

#include "common.cuh"
#include "kv4.h"

namespace dsv4 {

// pairs of floats in one register pair, one instruction for both
__device__ __forceinline__ uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// mbar_wait for hand-overs that take a fraction of a microsecond: no sleep between probes (the probe
// itself holds the thread for a while), the abort flag and the clock only now and then.
__device__ __forceinline__ bool mbar_spin(uint64_t *bar, uint32_t parity, volatile int *abort) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    const uint64_t now = globaltimer();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitLimitNs) {
      *abort = 1;
      return false;
    }
  }
}

// One lane of the warp. Through elect.sync the compiler knows that a single thread is inside the branch
// and issues a product in few instructions; with "lane 0" as the condition (branch or predicate) an
// issue took 75 to 170 cycles beside busy warps, more than the 64 that the product itself takes, with
// elect.sync around each instruction 40 to 55.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

// new tokens and positions of sequence s; false (and d_status) where they make no sense
struct Seq {
  int tok0, len, start, n;  // first token, new tokens, first position, positions to read
};
__device__ __forceinline__ bool seq_info(const Kv4AttnLaunch &p, int s, Seq *q, bool tell) {
  const int64_t c0 = p.cu_seqlens[s], c1 = p.cu_seqlens[s + 1], st = p.start_pos[s];
  const int64_t cap = static_cast<int64_t>(p.cache.max_blocks) * DSV4_PAGE_POSITIONS;
  if (c0 < 0 || c1 < c0 || c1 > p.T || st < 0) {
    if (tell) report(p.d_status, DSV4_DEV_BAD_LENGTH);
    return false;
  }
  if (c1 == c0) return false;
  int64_t n = st + (c1 - c0);
  if (n > cap) {
    if (tell) report(p.d_status, DSV4_DEV_BAD_LENGTH);
    n = cap;
  }
  q->tok0 = static_cast<int>(c0);
  q->len = static_cast<int>(c1 - c0);
  q->start = static_cast<int>(st < cap ? st : cap);  // (a row behind the capacity sees what there is)
  q->n = static_cast<int>(n);
  return true;
}

// How a row's sums end. Its maximum (or reference) m is -infinity where the row saw no position, and
// kLeast where it saw some and all their scores are -infinity (scores beyond float32, an infinite query): no position
// gives zero and lse -infinity, the other NaN, as 0 / 0 does, so that neither passes for the other.
constexpr float kLeast = -3.402823466e38f;
__device__ __forceinline__ float row_inverse(float m, float sum) {
  return sum != 0.f ? 1.f / sum : (m == -INFINITY ? 0.f : __uint_as_float(0x7FC00000u));
}
__device__ __forceinline__ float row_lse(float m, float sum, float off) {  // weights are held times 2^off
  return sum != 0.f ? (m - off + log2f(sum)) * 0.6931471805599453f : (m == -INFINITY ? m : __uint_as_float(0x7FC00000u));
}
// Whether a row that sees positions below lim sees any of tiles first .. last - 1, of 2^keys_log2 keys (a tile lies on one
// page). For rows without a finite score only: the table is looked up again.
__device__ __forceinline__ bool row_sees(const Kv4AttnLaunch &p, int s, int first, int last, int keys_log2, int lim) {
  for (int i = first; i < last && i << keys_log2 < lim; ++i) {
    const int page = p.cache.block_table[static_cast<int64_t>(s) * p.cache.max_blocks + ((i << keys_log2) / DSV4_PAGE_POSITIONS)];
    if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.cache.num_pages)) return true;
  }
  return false;
}

// a byte of two e2m1 codes -> fp16 pair; four bytes at once
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// scale byte -> 2^(byte - 127) as float (255: NaN)
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b << 23 | (b == 255u ? 0x400000u : 0u));
}
// two floats as bf16x2 (lo in the low half), one conversion for both
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// two floats as e4m3 in the low half (lo in the low byte), and what they became
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi, float &was_lo, float &was_hi) {
  uint16_t d;
  uint32_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(d));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(was_lo), "=f"(was_hi)
      : "r"(h));
  return d;
}

}  // namespace dsv4
