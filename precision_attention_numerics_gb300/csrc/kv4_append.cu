// Writing tokens into the 4-bit KV cache, and reading them back as values.
//
// Per row of 16-channel blocks (K after k - mean and the rotation):
//   s = E4M3(amax / (6 g)),  code = E2M1(x / (g s))  (IEEE divisions; 0 where s = 0).
// A CTA owns one tile (16 tokens) of one KV head, so no two CTAs write the
// same word.  A lane holds one block of a row (16 values): the maximum and the first
// four butterfly stages stay inside it, the rest goes over the row's d / 16 lanes.
// The codes meet in shared memory, are turned into the tile's fragment order there with
// byte permutes, and leave as 16-byte stores; a tile that also holds tokens written
// before is merged word by word under a mask.
// Bound by instruction issue: about 90 warp instructions a K row and 40 a V row.
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "kv4.cuh"

namespace attnq {
namespace {

constexpr int kAppendThreads = 128;

struct AppendParams {
  Kv4Map map;
  Kv4Rows K, V;
  const float* k_mean;   // [B, Hkv, D] or null
  const int8_t* signs;   // null: no rotation
  const float* k_scale;  // [Hkv] or null
  const float* v_scale;
  float inv_sqrt_d;
};

// E2M1 codes of a block, nibble i = channel i, and its E4M3 scale.  Sets bad if a value is not finite.
__device__ __forceinline__ uint2 quantise16(const float (&x)[16], float g, uint32_t& s8, bool& bad) {
  // the largest magnitude (a NaN stays one: max.NaN, one instruction a value)
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(am) : "f"(fabsf(x[i])));
  bad |= !(am < INFINITY);
  s8 = cvt_e4m3x2(__fdiv_rn(am, __fmul_rn(6.0f, g)), 0.0f);
  const float den = __fmul_rn(g, e4m3x2_to_f2(uint16_t(s8)).x);
  uint32_t c[8];
  if ((__float_as_uint(g) & 0x007FFFFFu) == 0u && am <= __fmul_rn(den, 1048576.0f)) {
    // g is a power of two (1 mostly), so den has four significant bits, and the
    // code of fl32(x / den) comes without a division: let T be x / den rounded to three
    // bits after the leading one.  All points where E2M1 changes are such T, so only
    // the side of T matters; e = x - T den (one rounding, exact in sign) tells it, and
    // if e is not 0, x / den is further from T than half its last place: x - T den is at
    // least one last place of x, whose leading digits are at most 1.875.  So z = T + e / den is T
    // exactly when fl32(x / den) is, and on the same side otherwise.  Every step is finite up to
    // |x| = 2^20 den; a block with larger values is divided, where x / den may overflow to an
    // infinity of x's sign, which saturates.
    const float r = __fdiv_rn(1.0f, den);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float z[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float v = x[2 * i + e];
        const float T = __uint_as_float((__float_as_uint(__fmul_rn(v, r)) + 0x00080000u) & 0xFFF00000u);
        z[e] = __fmaf_rn(__fmaf_rn(-T, den, v), r, T);
      }
      c[i] = cvt_e2m1x2(z[0], z[1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = cvt_e2m1x2(__fdiv_rn(x[2 * i], den), __fdiv_rn(x[2 * i + 1], den));
  }
  if ((s8 & 0xFFu) == 0u) return make_uint2(0u, 0u);
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// Transposes the 4x4 bytes of (a, b, c, d): out[i] = byte i of each, a's lowest.
__device__ __forceinline__ void bytes_4x4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&out)[4]) {
  const uint32_t x0 = __byte_perm(a, b, 0x5140), x1 = __byte_perm(a, b, 0x7362);
  const uint32_t y0 = __byte_perm(c, d, 0x5140), y1 = __byte_perm(c, d, 0x7362);
  out[0] = __byte_perm(x0, y0, 0x5410);
  out[1] = __byte_perm(x0, y0, 0x7632);
  out[2] = __byte_perm(x1, y1, 0x5410);
  out[3] = __byte_perm(x1, y1, 0x7632);
}

// Mask of the bits of word i of a tile that belong to tokens lo .. hi - 1.
template <int D>
__device__ __forceinline__ uint32_t token_mask(int i, int lo, int hi) {
  constexpr int NB = D / kKv4Block;
  auto has = [&](int r) { return r >= lo && r < hi; };
  uint32_t m = 0;
  if (i < 2 * D) {
    const int g = (i >> 4) & 7;
    m = (has(g) ? 0x00FF00FFu : 0u) | (has(g + 8) ? 0xFF00FF00u : 0u);
  } else if (i < 4 * D) {
    const int t = (i >> 2) & 3;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (has(2 * t + (q & 1) + (q & 2 ? 8 : 0))) m |= 0x00000F0Fu << ((q & 1) * 4 + (q & 2) * 8);
  } else if (i < 4 * D + D / 4) {
    const int g = (i - 4 * D) / (NB / 2);
    m = (has(g) ? 0x00FF00FFu : 0u) | (has(g + 8) ? 0xFF00FF00u : 0u);
  } else {
    const int t = (i - 4 * D - D / 4) / NB;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (has(2 * t + (q & 1) + (q & 2 ? 8 : 0))) m |= 0xFFu << (8 * q);
  }
  return m;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAppendThreads) k_kv4_append(const AppendParams p) {
  constexpr int NB = D / kKv4Block;         // lanes of a row
  constexpr int RPP = 32 / NB, PASSES = 16 / RPP;  // rows a warp takes at a time; passes over a tile
  __shared__ uint2 s_code[2][16][NB];       // K and V codes, nibble i of a block = channel i
  __shared__ uint8_t s_scale[2][16][NB];
  __shared__ __align__(16) uint32_t s_tile[kv4_tile_bytes(D) / 4];
  const int h = blockIdx.y % p.map.Hkv, b = blockIdx.y / p.map.Hkv;
  const int L = kv4_len(p.map, b), n = kv4_new(p.map, b);
  const int first = kv4_first(p.map, b, L, n);  // place of row 0
  if (first >= L) return;
  const int tile = max(first, 0) / kKv4Tile + int(blockIdx.x);
  // places of this tile that the call writes: [lo, hi)
  const int lo = max(max(first, 0) - tile * kKv4Tile, 0), hi = min(L - tile * kKv4Tile, kKv4Tile);
  if (lo >= hi) return;
  uint8_t* dst = kv4_tile_ptr<D>(p.map, b, h, tile);
  if (!dst) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blk = lane % NB;
  // words that other tokens share are needed at the end: their loads are under way while the rows are made
  constexpr int WORDS = (kv4_tile_bytes(D) / 4 + kAppendThreads - 1) / kAppendThreads;
  const bool whole = lo == 0 && hi == kKv4Tile;
  uint32_t* out = reinterpret_cast<uint32_t*>(dst);
  uint32_t old[WORDS];
  if (!whole) {
#pragma unroll
    for (int q = 0; q < WORDS; ++q) {
      const int i = q * kAppendThreads + threadIdx.x;
      const uint32_t m = i < kv4_tile_bytes(D) / 4 ? token_mask<D>(i, lo, hi) : 0u;
      old[q] = m != 0u && m != 0xFFFFFFFFu ? out[i] : 0u;
    }
  }
  bool bad = false;
  for (int u = warp; u < 2 * PASSES; u += kAppendThreads / 32) {
    const bool is_v = u >= PASSES;
    const int r0 = (u % PASSES) * RPP, r = r0 + lane / NB;
    if (r0 + RPP <= lo || r0 >= hi) continue;
    float x[16] = {};
    if (r >= lo && r < hi) {
      const Kv4Rows& in = is_v ? p.V : p.K;
      const int64_t off = b * in.sb + h * in.sh + int64_t(tile * kKv4Tile + r - first) * in.st + blk * 16;
      kv4_load16<BF16>(static_cast<const uint8_t*>(in.ptr) + off * (BF16 ? 2 : 4), x);
    }
    float g = 1.0f;
    if (is_v) {
      if (p.v_scale) g = p.v_scale[h];
    } else {
      if (p.k_scale) g = p.k_scale[h];
      if (p.k_mean) {
        float mu[16];
        kv4_load16<false>(p.k_mean + (int64_t(b) * p.map.Hkv + h) * D + blk * 16, mu);
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __fsub_rn(x[i], mu[i]);
      }
      if (p.signs) kv4_rotate16<D>(x, p.signs, blk, p.inv_sqrt_d);
    }
    uint32_t s8;
    bool not_finite = false;
    s_code[is_v][r][blk] = quantise16(x, g, s8, not_finite);
    // a V block with a NaN holds zeros: rows that do not see its token have weight 0 for it, and 0 times a NaN scale
    // would reach them (their scores against a K block with one are masked)
    if (is_v && (s8 & 0x7Fu) == 0x7Fu) s8 = 0u;
    s_scale[is_v][r][blk] = uint8_t(s8);
    bad |= not_finite && r >= lo && r < hi;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.map.status, DEV_NONFINITE);
  __syncthreads();
  // rows that the call does not write left their shared memory undefined: masked below
  for (int i = threadIdx.x; i < 8 * NB + 4 * NB; i += kAppendThreads) {
    if (i < 8 * NB) {  // K words of (block, g): rows g and g + 8, t = 0 .. 3
      const int kb = i % NB, g = i / NB;
      const uint2 a = s_code[0][g][kb], c = s_code[0][g + 8][kb];
      uint32_t w[4];
      bytes_4x4(a.x, c.x, a.y, c.y, w);
#pragma unroll
      for (int t = 0; t < 4; ++t) s_tile[kv4_code_word(kb, g * 4 + t)] = w[t];
    } else {  // V words of (block, t): tokens 2t, 2t + 1, 2t + 8, 2t + 9, g = 0 .. 7
      const int vb = (i - 8 * NB) % NB, t = (i - 8 * NB) / NB;
      const uint2 k0 = s_code[1][2 * t][vb], k1 = s_code[1][2 * t + 1][vb];
      const uint2 k8 = s_code[1][2 * t + 8][vb], k9 = s_code[1][2 * t + 9][vb];
      auto even = [](uint32_t a, uint32_t c) { return (a & 0x0F0F0F0Fu) | (c << 4 & 0xF0F0F0F0u); };
      auto odd = [](uint32_t a, uint32_t c) { return (a >> 4 & 0x0F0F0F0Fu) | (c & 0xF0F0F0F0u); };
      uint32_t w[4];
      bytes_4x4(even(k0.x, k1.x), even(k0.y, k1.y), even(k8.x, k9.x), even(k8.y, k9.y), w);
#pragma unroll
      for (int q = 0; q < 4; ++q) s_tile[2 * D + kv4_code_word(vb, (2 * q) * 4 + t)] = w[q];
      bytes_4x4(odd(k0.x, k1.x), odd(k0.y, k1.y), odd(k8.x, k9.x), odd(k8.y, k9.y), w);
#pragma unroll
      for (int q = 0; q < 4; ++q) s_tile[2 * D + kv4_code_word(vb, (2 * q + 1) * 4 + t)] = w[q];
    }
  }
  uint8_t* tile8 = reinterpret_cast<uint8_t*>(s_tile);
  for (int i = threadIdx.x; i < 2 * 16 * NB; i += kAppendThreads) {
    const int r = (i / NB) & 15, sb = i % NB;
    if (i < 16 * NB) tile8[16 * D + (r & 7) * 2 * NB + 2 * sb + (r >> 3)] = s_scale[0][r][sb];
    else tile8[17 * D + ((r & 7) >> 1) * 4 * NB + 4 * sb + (r >> 3) * 2 + (r & 1)] = s_scale[1][r][sb];
  }
  __syncthreads();
  if (whole) {
    for (int i = threadIdx.x; i < kv4_tile_bytes(D) / 16; i += kAppendThreads)
      reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(s_tile)[i];
  } else {
#pragma unroll
    for (int q = 0; q < WORDS; ++q) {
      const int i = q * kAppendThreads + threadIdx.x;
      if (i >= kv4_tile_bytes(D) / 4) break;
      const uint32_t m = token_mask<D>(i, lo, hi);
      if (m) out[i] = (old[q] & ~m) | (s_tile[i] & m);
    }
  }
}

struct ReadParams {
  Kv4Map map;
  const float* k_scale;
  const float* v_scale;
  Kv4Rows K, V;  // outputs
};

// A warp takes K or V of one tile: the fragments' halves (V's transposed back with
// movmatrix) go through shared memory into whole rows, 16 bytes a lane.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) k_kv4_read(const ReadParams p) {
  constexpr int NB = D / kKv4Block, EB = BF16 ? 2 : 4, ROW = D * EB + 16;  // padded rows: no bank conflicts
  __shared__ __align__(16) uint8_t s_rows[4][16 * ROW];
  const int h = blockIdx.y % p.map.Hkv, b = blockIdx.y / p.map.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const bool is_v = warp & 1;
  const int L = kv4_len(p.map, b), n = kv4_new(p.map, b);
  const int first = kv4_first(p.map, b, L, n);  // place of row 0
  if (first >= L) return;
  const int tile = max(first, 0) / kKv4Tile + int(blockIdx.x) * 2 + (warp >> 1);
  const int lo = max(max(first, 0) - tile * kKv4Tile, 0), hi = min(L - tile * kKv4Tile, kKv4Tile);
  if (lo >= hi) return;
  const uint8_t* src = kv4_tile_ptr<D>(p.map, b, h, tile);
  if (!src) return;
  uint4 w4[NB / 4];
#pragma unroll
  for (int q = 0; q < NB / 4; ++q)
    w4[q] = __ldg(reinterpret_cast<const uint4*>(src + (is_v ? 8 * D : 0)) + q * 32 + lane);
  uint32_t sc[NB];  // K: of (token g, token g + 8); V: of the four tokens
  if (is_v) {
#pragma unroll
    for (int i = 0; i < NB; ++i) sc[i] = __ldg(reinterpret_cast<const uint32_t*>(src + 17 * D) + t * NB + i);
  } else {
#pragma unroll
    for (int i = 0; i < NB / 2; ++i) {
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * D) + g * (NB / 2) + i);
      sc[2 * i] = x;
      sc[2 * i + 1] = x >> 16;
    }
  }
  const float* gs = is_v ? p.v_scale : p.k_scale;
  const float gf = gs ? gs[h] : 1.0f;
  uint8_t* rows = s_rows[warp];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const uint32_t w = i % 4 == 0 ? w4[i / 4].x : i % 4 == 1 ? w4[i / 4].y : i % 4 == 2 ? w4[i / 4].z : w4[i / 4].w;
    uint32_t a[4];
    if (is_v) {
      uint32_t f[4];
      kv4_v_frag(w, e4m3x2_to_h2(sc[i]), e4m3x2_to_h2(sc[i] >> 16), f);
      a[0] = movmatrix_t(f[0]);
      a[1] = movmatrix_t(f[2]);
      a[2] = movmatrix_t(f[1]);
      a[3] = movmatrix_t(f[3]);
    } else {
      kv4_k_frag(w, e4m3x2_to_h2(sc[i]), a);
    }
    // a[x]: token g + 8 (x & 1), channels 16 i + 8 (x >> 1) + 2t, +1
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a[x]));
      const float v0 = __fmul_rn(f.x, gf), v1 = __fmul_rn(f.y, gf);  // code * s is exact: one rounding by g
      uint8_t* at = rows + (g + 8 * (x & 1)) * ROW + (16 * i + 8 * (x >> 1) + 2 * t) * EB;
      if constexpr (BF16) *reinterpret_cast<__nv_bfloat162*>(at) = __floats2bfloat162_rn(v0, v1);
      else *reinterpret_cast<float2*>(at) = make_float2(v0, v1);
    }
  }
  __syncwarp();
  const Kv4Rows& o = is_v ? p.V : p.K;
  constexpr int CH = D * EB / 16;  // 16-byte pieces of a row
  uint8_t* out = static_cast<uint8_t*>(const_cast<void*>(o.ptr)) + (b * o.sb + h * o.sh) * EB;
#pragma unroll
  for (int i = 0; i < 16 * CH / 32; ++i) {
    const int r = (i * 32 + lane) / CH, c = (i * 32 + lane) % CH;
    if (r >= lo && r < hi)
      *reinterpret_cast<uint4*>(out + int64_t(tile * kKv4Tile + r - first) * o.st * EB + c * 16) =
          *reinterpret_cast<const uint4*>(rows + r * ROW + c * 16);
  }
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4Args& a, const Kv4Rows& K, const Kv4Rows& V, int bf16, const float* k_mean,
                              cudaStream_t s) {
  AppendParams p{};
  p.map = kv4_map(a);
  p.K = K;
  p.V = V;
  p.k_mean = k_mean;
  p.signs = a.signs;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.inv_sqrt_d = a.d == 128 ? 0.08838834764831845f : 0.125f;
  const int tiles = (a.T + kKv4Tile - 2) / kKv4Tile + 1;  // that T tokens can touch
  const dim3 grid(tiles, a.B * a.Hkv);
  if (a.d == 128) {
    if (bf16) k_kv4_append<128, true><<<grid, kAppendThreads, 0, s>>>(p);
    else k_kv4_append<128, false><<<grid, kAppendThreads, 0, s>>>(p);
  } else {
    if (bf16) k_kv4_append<64, true><<<grid, kAppendThreads, 0, s>>>(p);
    else k_kv4_append<64, false><<<grid, kAppendThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_kv4_read(const Kv4Args& a, const Kv4Rows& K, const Kv4Rows& V, int bf16, cudaStream_t s) {
  ReadParams p{};
  p.map = kv4_map(a);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.K = K;
  p.V = V;
  const int tiles = (a.T + kKv4Tile - 2) / kKv4Tile + 1;
  const dim3 grid((tiles + 1) / 2, a.B * a.Hkv);
  if (a.d == 128) {
    if (bf16) k_kv4_read<128, true><<<grid, 128, 0, s>>>(p);
    else k_kv4_read<128, false><<<grid, 128, 0, s>>>(p);
  } else {
    if (bf16) k_kv4_read<64, true><<<grid, 128, 0, s>>>(p);
    else k_kv4_read<64, false><<<grid, 128, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace attnq
