// The 4-bit KV cache's tile format and the device code that its kernels share.
//
// A token's K (or V) row of a KV head is held in blocks of 16 channels, each
// with an E4M3 scale s and 16 E2M1 codes c: x ~ g * s * c, g the head's fp32
// scale.  E2M1 has 2 significant bits and E4M3 has 4, so s * c has at most 6
// and lies between 2^-10 and 2688: it is exact in fp16, and every kernel works
// on those exact halves (the head's g enters as one fp32 factor).
//
// Tokens are grouped in tiles of 16 (aligned at token 0 of the sequence); a
// page holds page_tokens / 16 tiles of every KV head, [Hkv][tile].  A tile is
// 18 * d contiguous bytes (16 tokens x 1.125 d), laid out so that a warp reads the
// A operands of mma.m16n8k16 straight out of it, with no shuffle or transpose:
//   [0, 8d)     K codes, words [b / 4][lane][b % 4] (b: block of 16 channels).
//               Word (b, lane), g = lane / 4, t = lane % 4, has four bytes of two
//               codes (even element in the low nibble):
//                 0: token g,     channels 16b + 2t, +1      (a0)
//                 1: token g + 8, the same channels          (a1)
//                 2: token g,     channels 16b + 2t + 8, +9  (a2)
//                 3: token g + 8, the same channels          (a3)
//   [8d, 16d)   V codes (V^T is the A operand), words [b / 4][lane][b % 4]:
//                 0: channel 16b + g,     tokens 2t, 2t + 1      (a0)
//                 1: channel 16b + g + 8, the same tokens        (a1)
//                 2: channel 16b + g,     tokens 2t + 8, 2t + 9  (a2)
//                 3: channel 16b + g + 8, the same tokens        (a3)
//   [16d, 17d)  K scales [g][b][token g, token g + 8]
//   [17d, 18d)  V scales [t][b][tokens 2t, 2t + 1, 2t + 8, 2t + 9]
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace attnq {

constexpr int kKv4Tile = 16;   // tokens of a tile
constexpr int kKv4Block = 16;  // channels of a scale

__host__ __device__ constexpr int kv4_tile_bytes(int d) { return 18 * d; }

// Word (b, lane) of the codes: index in words from the start of the K or V codes.
__host__ __device__ constexpr int kv4_code_word(int b, int lane) { return ((b >> 2) * 32 + lane) * 4 + (b & 3); }

// Where the tokens of the call's sequences are.
struct Kv4Map {
  uint8_t* pages;
  const int32_t* table;     // [B, max_pages]
  const int32_t* lens;      // [B]
  const int32_t* new_lens;  // [B] or null: T
  int B, max_pages, num_pages;
  int Hkv;
  int tpp_shift;            // log2 of the tiles per page
  int T;
  uint32_t* status;
};

inline Kv4Map kv4_map(const Kv4Args& a) {
  Kv4Map m{};
  m.pages = a.pages;
  m.table = a.table;
  m.lens = a.lens;
  m.new_lens = a.new_lens;
  m.B = a.B;
  m.max_pages = a.max_pages;
  m.num_pages = a.num_pages;
  m.Hkv = a.Hkv;
  for (int t = a.page_tokens / kKv4Tile; t > 1; t >>= 1) ++m.tpp_shift;
  m.T = a.T;
  m.status = a.status;
  return m;
}

__device__ __forceinline__ int kv4_len(const Kv4Map& m, int b) {
  const int cap = m.max_pages << (m.tpp_shift + 4);
  const int n = m.lens[b];
  if (n < 0 || n > cap) {
    atomicOr(m.status, DEV_PAGE);
    return n < 0 ? 0 : cap;
  }
  return n;
}

// New rows of sequence b.  Row t of n stands at place L - n + t.
__device__ __forceinline__ int kv4_new(const Kv4Map& m, int b) {
  if (!m.new_lens) return m.T;
  const int n = m.new_lens[b];
  if (n < 0 || n > m.T) {
    atomicOr(m.status, DEV_PAGE);
    return n < 0 ? 0 : m.T;
  }
  return n;
}

// Place of row 0 of the n new rows of sequence b, of length L as kv4_len gives it.  A length past the
// page table (reported there) moves no row: rows whose place it has no room for are dropped,
// and those before them do not land on other tokens.
__device__ __forceinline__ int kv4_first(const Kv4Map& m, int b, int L, int n) { return max(m.lens[b], L) - n; }

// Address of tile `tile` of sequence b, KV head h; null (and a status bit) for
// a page number outside the pool.
template <int D>
__device__ __forceinline__ uint8_t* kv4_tile_ptr(const Kv4Map& m, int b, int h, int tile) {
  const int page = m.table[int64_t(b) * m.max_pages + (tile >> m.tpp_shift)];
  if (uint32_t(page) >= uint32_t(m.num_pages)) {
    atomicOr(m.status, DEV_PAGE);
    return nullptr;
  }
  const int64_t t = ((int64_t(page) * m.Hkv + h) << m.tpp_shift) + (tile & ((1 << m.tpp_shift) - 1));
  return m.pages + t * kv4_tile_bytes(D);
}

// Eight E2M1 codes (four bytes of two) -> four f16x2, low nibble in the low half.
__device__ __forceinline__ void e2m1x8_to_h2x4(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two floats -> two E2M1 codes (round to nearest even, saturating to +-6), lo in the low nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\t"
      "mov.b32 %0, {b, 0, 0, 0};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 scales (lo | hi << 8) -> f16x2.
__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t v) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(v)));
  return h2;
}

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// D += A B, m16n8k16, fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of the warp's 8x8 matrix of halves (lane 4i + j holds row i, columns 2j, 2j + 1).
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t hmul2_lo(uint32_t a, uint32_t s2) {  // a * (low half of s2) in both halves
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s2)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_hi(uint32_t a, uint32_t s2) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s2)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The A operand of scores: 16 tokens x 16 channels of block b, exact halves.
// w: the lane's code word; s2: scales of (token g, token g + 8).
__device__ __forceinline__ void kv4_k_frag(uint32_t w, uint32_t s2, uint32_t (&a)[4]) {
  e2m1x8_to_h2x4(w, a);
  a[0] = hmul2_lo(a[0], s2);
  a[1] = hmul2_hi(a[1], s2);
  a[2] = hmul2_lo(a[2], s2);
  a[3] = hmul2_hi(a[3], s2);
}

// The A operand of P V: 16 channels of block b x 16 tokens, exact halves.
// s01, s89: scales of tokens (2t, 2t + 1) and (2t + 8, 2t + 9).
__device__ __forceinline__ void kv4_v_frag(uint32_t w, uint32_t s01, uint32_t s89, uint32_t (&a)[4]) {
  e2m1x8_to_h2x4(w, a);
  a[0] = hmul2_u(a[0], s01);
  a[1] = hmul2_u(a[1], s01);
  a[2] = hmul2_u(a[2], s89);
  a[3] = hmul2_u(a[3], s89);
}

// Sixteen consecutive elements as floats.
template <bool BF16>
__device__ __forceinline__ void kv4_load16(const void* src, float (&x)[16]) {
  if constexpr (BF16) {
    const uint4 a = __ldg(static_cast<const uint4*>(src)), b = __ldg(static_cast<const uint4*>(src) + 1);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(static_cast<const float4*>(src) + i);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  }
}

// x <- (signs * x) H / sqrt(d), the row's blocks on d / 16 neighbouring lanes:
// butterflies of stride 1, 2, ..., d / 2 (the first four inside a lane), then
// one multiplication by fl32(1 / sqrt d).
template <int D>
__device__ __forceinline__ void kv4_rotate16(float (&x)[16], const int8_t* signs, int blk, float inv_sqrt_d) {
  const uint4 sg = __ldg(reinterpret_cast<const uint4*>(signs) + blk);
  const uint32_t w[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
  for (int i = 0; i < 16; ++i)  // times -1 is the sign bit turned over
    x[i] = __uint_as_float(__float_as_uint(x[i]) ^ ((w[i >> 2] << (24 - 8 * (i & 3))) & 0x80000000u));
#pragma unroll
  for (int h = 1; h < 16; h *= 2)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & h)) {
        const float a = x[i], b = x[i + h];
        x[i] = __fadd_rn(a, b);
        x[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int o = 1; o < D / 16; o *= 2) {
    const float sgn = (blk & o) ? -1.0f : 1.0f;  // x + y on the lower lane, y - x on the upper: one rounding either way
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __fmaf_rn(x[i], sgn, __shfl_xor_sync(0xffffffffu, x[i], o));
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], inv_sqrt_d);
}

}  // namespace attnq
