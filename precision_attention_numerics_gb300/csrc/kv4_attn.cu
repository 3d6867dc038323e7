// Attention over the 4-bit KV cache, and the weights it gives each token.
//
// For query row r (query t of head h) and the tokens j it sees:
//   s_j = q_r . k_j,  m = max_j s_j c_r,  p_j = 2^(s_j c_r - m),  l = sum_j p_j,
//   O_r = g_v / l * sum_j p_j v_j,  lse_r = (m + log2 l) ln 2,
// with k_j, v_j the exact halves scale * code of the cache, c_r = scale log2 e g_k
// times the power of two that q_r was normalised by.
//
// The rows of all query heads of a KV head are taken together (row r = t G + head
// of the group), R = 8 NT of them at a time, and the products are transposed so
// that the tokens fill the 16-row side of mma.m16n8k16 and the few query rows
// its 8-column side: S^T = K Q^T, O^T += V^T P^T.  The cache's tiles hold the A
// operands of both in register order.  P goes from accumulator to B operand
// with movmatrix, inside the warp.
//
// Precision: K and V are exact in fp16, and unrotated bf16 queries down to 2^-31 of their row's largest
// element (within 2^-39 of it below); rotated or fp32 queries are split into two halves (hi + lo, 22 bits, the
// same 2^-39 at the least; QS), the second product added in the same accumulators.
// P is rounded to fp16 (2^-11 relative, an eighth of the bf16 output's rounding) for
// bf16 outputs and split in two for fp32 outputs
// (PS).  Scores, maxima, sums and outputs are fp32.
#include <cfloat>
#include <cmath>

#include "kv4_attn.cuh"

namespace attnq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kChunk = 32;  // tokens a warp takes at a time: two tiles
// What a segment's beginning and end cost, in chunks (with 4 the 64 segments of a batch with 20 rows
// each took 39.1 us, with 8 37.2, with 16 37.9), and the same of the tcgen05 kernel's chunks.  The
// weights of many rows cost more a chunk, so a beginning counts for fewer.
constexpr int kOverhead = 8, kPrefillOverhead = 4, kManyRowsOverhead = 4;
// P is held as 2^15 p: the row's maximum is 2^15 in fp16 (at most 65504), and
// weights keep all of fp16's bits down to 2^-29 of it and vanish below 2^-40, where a million
// of them add up to less than 2^-20.  l carries the same factor.
constexpr float kPBits = 15.0f;

// Query rows in B operand order, [row tile of 8][term][block][lane][2], and what goes with each row.
template <int D, int NT, bool QS>
struct QShared {
  static constexpr int R = 8 * NT, NB = D / kKv4Block;
  uint32_t frag[NT][QS ? 2 : 1][NB][32][2];
  float c[R];    // factor of the row's raw scores, log2 units
  int lim[R];    // tokens the row sees: j < lim (rows that are not there: all, their results go nowhere)
};

// Rows row0 .. row0 + R - 1 of (b, h), normalised to halves by a power of two
// each; run by `warps` warps.  A lane holds a block of 16 channels, d / 16 lanes a row.
// AT passes' loads are in flight at a time.
// PAIR (at most 4 rows): row i stands in columns i and i + 4 of the one row tile, with QS
// its low term in i + 4.
template <int D, bool QS, bool PAIR, int AT>
__device__ __forceinline__ void load_queries(const Kv4AttnParams& p, int b, int h, int L, int n, int row0, int R,
                                             uint32_t* frag, float* c, int* lim, int warp, int lane, int warps) {
  constexpr int NB = D / kKv4Block, RPP = 32 / NB, P = QS && !PAIR ? 2 : 1;
  const float gk = p.k_scale ? p.k_scale[h] : 1.0f;
  const int blk = lane % NB, step = warps * RPP;
  Kv4Raw16 raw[AT];
#pragma unroll 1
  for (int i0 = warp * RPP; i0 < R; i0 += AT * step) {
#pragma unroll
    for (int u = 0; u < AT; ++u) raw[u] = kv4_query_row(p, b, h, n, row0 + i0 + u * step + lane / NB, i0 + u * step < R, blk);
#pragma unroll
    for (int u = 0; u < AT; ++u) {
      const int i = i0 + u * step + lane / NB, row = row0 + i;
      float x[16], norm;
      kv4_unpack16(raw[u], p.q_bf16, x);
      const float down = kv4_normalise16<D>(p, x, blk, norm);
      uint32_t hi[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) hi[e] = pack_h2(x[2 * e] * down, x[2 * e + 1] * down);
      if (i >= R) continue;  // past the end, or a pass of 8 rows with d = 64 and 4 wanted
      uint2* dst = reinterpret_cast<uint2*>(frag) + ((i >> 3) * P * NB + blk) * 32 + (i & 7) * 4;
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[e] = make_uint2(hi[e], hi[e + 4]);
      if constexpr (QS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi[e]));
          hi[e] = pack_h2(x[2 * e] * down - f.x, x[2 * e + 1] * down - f.y);
        }
      }
      if constexpr (QS || PAIR) {
        uint2* second = dst + (PAIR ? 4 * 4 : NB * 32);
#pragma unroll
        for (int e = 0; e < 4; ++e) second[e] = make_uint2(hi[e], hi[e + 4]);
      }
      if (blk == 0) {
        const bool live = row < n * p.G;
        // at least the smallest normal number: a masked score, -infinity, times 0 would be NaN, and
        // |s| < 2^34, so the products below it are nothing beside 1 either way
        c[i] = fmaxf(live ? p.scale_log2e * gk * norm : 0.0f, FLT_MIN);
        lim[i] = live ? (p.causal ? min(max(L - n + row / p.G + 1, 0), L) : L) : 0x7FFFFFFF;
        if constexpr (PAIR) {
          c[i + 4] = c[i];
          lim[i + 4] = lim[i];
        }
      }
    }
  }
}

// S^T of U tiles: raw sums of 16 tokens x R rows each.  The query operands
// are read from shared memory once for all of them.
template <int D, int NT, bool QS, int U, typename Q>
__device__ __forceinline__ void tile_scores(const uint8_t* const (&tile)[U], const Q& sq, int lane,
                                            float (&s)[U][NT][4]) {
  constexpr int NB = D / kKv4Block;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[u][nt][i] = 0.0f;
#pragma unroll
  for (int q = 0; q < NB / 4; ++q) {
    uint32_t w[U][4], sc[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 w4 = reinterpret_cast<const uint4*>(tile[u])[q * 32 + lane];
      w[u][0] = w4.x;
      w[u][1] = w4.y;
      w[u][2] = w4.z;
      w[u][3] = w4.w;
      const uint2 s2 = reinterpret_cast<const uint2*>(tile[u] + 16 * D)[(lane >> 2) * (NB / 4) + q];
      sc[u][0] = s2.x;
      sc[u][1] = s2.y;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int blk = 4 * q + i;
      uint2 bq[QS ? 2 : 1][NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        bq[0][nt] = *reinterpret_cast<const uint2*>(sq.frag[nt][0][blk][lane]);
        if constexpr (QS) bq[1][nt] = *reinterpret_cast<const uint2*>(sq.frag[nt][1][blk][lane]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint32_t a[4];
        kv4_k_frag(w[u][i], e4m3x2_to_h2(sc[u][i >> 1] >> (16 * (i & 1))), a);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(s[u][nt], a, bq[0][nt].x, bq[0][nt].y);
          if constexpr (QS) mma_16816(s[u][nt], a, bq[1][nt].x, bq[1][nt].y);
        }
      }
    }
  }
}

// What bounds it: with up to 8 rows the instructions of turning 4 bits into operands (about 350 warp
// instructions a tile of 16 tokens, half of them conversions and scalings) beside the reads; 16 x
// 32768 tokens (32 on 8 heads, d 128) take 119 us, 5.1 TB/s, and 105 with the scalings cut out. With
// more rows products and softmax, and the latency of few warps.
//
// CTAs an SM holds, and the tiles in each warp's ring: the registers of NT row
// tiles allow 4, 3 or 2 CTAs of four warps (three CTAs of 24 rows spill: 37.8 us for 8 sequences
// of up to 8191 tokens and 20 rows, against 30.9 with two), and the ring takes the shared memory
// that is left (for 8 rows of d 128: 5 tiles a warp, 16 warps, so up to 110 KB of
// copies in flight per SM; 36 KB cover the memory latency at full bandwidth).
template <int D, int NT, bool QS>
struct Cfg {
  static constexpr int R = 8 * NT;
  static constexpr int CTAS = NT == 1 ? 4 : NT <= 2 ? 3 : 2;
  static constexpr int TB = kv4_tile_bytes(D);
  static constexpr int kFixed = int(sizeof(QShared<D, NT, QS>)) + kWarps * 16 * 16 + kWarps * R * 8 + 1024;
  static constexpr int NS0 = (232448 / CTAS - 1024 - kFixed) / (kWarps * TB);
  static constexpr int NS = NS0 > 12 ? 12 : NS0;
  static_assert(NS >= 4, "ring depth");
  // the joined sums of the warps take the ring's place
  static constexpr int kRing = kWarps * NS * TB, kSums = kWarps * R * D * 4;
  static constexpr int SMEM = kFixed + (kRing > kSums ? kRing : kSums);
  static_assert((SMEM + 1024) * CTAS <= 233472, "shared memory of an SM");
};

//
// PAIR: with at most 4 rows half of the row tile's columns are free, and the second
// terms take them instead of products of their own: low terms of Q in columns 4 to 7
// (the two halves of a score are added across lanes), low terms of P likewise (the two
// halves of an output are added at the end).  16 x 32768 tokens with rotated
// queries: 129 us with separate products, 117 without any second term.
//
// CL: a cluster of p.cl CTAs has a segment to itself and joins its rows over distributed
// shared memory; otherwise the chunks of all segments are dealt along the line.
template <int D, int NT, bool QS, bool PS, bool PAIR, bool CL>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT, QS>::CTAS) k_kv4_attn(const Kv4AttnParams p) {
  using C = Cfg<D, NT, QS>;
  static_assert(!PAIR || NT == 1, "one row tile");
  constexpr int R = C::R, NB = D / kKv4Block, NS = C::NS, TB = C::TB;
  extern __shared__ __align__(128) uint8_t smem[];
  auto& sq = *reinterpret_cast<QShared<D, NT, QS>*>(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + ((sizeof(QShared<D, NT, QS>) + 127) & ~size_t(127)));
  int* s_ok = reinterpret_cast<int*>(bars + kWarps * NS);                            // [warp][stage] tile readable
  float2* s_ml = reinterpret_cast<float2*>(s_ok + ((kWarps * NS + 3) & ~3));         // [warp][R]
  uint8_t* ring0 = smem + ((C::kFixed) & ~127);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = ring0 + warp * (NS * TB);
  uint64_t* full = bars + warp * NS;
  int* ok_flag = s_ok + warp * NS;
  float* s_o = reinterpret_cast<float*>(ring0);  // [warp][R][D], once the ring has been read
  if (lane < NS) mbar_init(full + lane, 1);
  fence_mbar_init();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  Kv4Line<R, kChunk> sg;
  // also orders the barriers' set-up
  int c1_cluster = 0;
  bool more;
  if constexpr (CL) {
    more = sg.begin_cluster(p, blockIdx.x, c1_cluster);
  } else {
    more = sg.template begin<kWarps>(p, blockIdx.x, kOverhead);
    if (threadIdx.x == 0) p.part_seg[blockIdx.x] = make_int4(0, -1, 0, 0);  // nothing to join, until the last segment
  }
  uint32_t st = 0, ph = 0;       // stage of this warp's next tile, and the parity of its barrier
  const int64_t page_bytes = (int64_t(p.map.Hkv) << p.map.tpp_shift) * TB;
  const int tpp_mask = (1 << p.map.tpp_shift) - 1;
  bool dead = false;
  __syncthreads();
  int slot = 0;
  while (more) {
    const int c0 = sg.c0, c1 = CL ? c1_cluster : sg.last_chunk();
    if (!CL && sg.nothing()) {
      more = sg.next(p, c1);
      continue;
    }
    const int c_end = min(c1, (sg.vis + kChunk - 1) / kChunk);
    const int mine = c_end - c0 - warp > 0 ? (c_end - c0 - warp + kWarps - 1) / kWarps : 0;  // this warp's chunks

    // Tile i of this warp's share is 2 (c0 + warp) + 8 (i / 2) + i % 2: copies go
    // NS tiles ahead.  A lane issues its own copy; pages are looked up one round
    // before they are needed.
    const int first_tile = 2 * (c0 + warp), tiles_seen = (sg.vis + kKv4Tile - 1) / kKv4Tile;
    const int32_t* pages_of = p.map.table + int64_t(sg.b) * p.map.max_pages;
    const uint8_t* head = p.map.pages + ((int64_t(sg.h) << p.map.tpp_shift)) * TB;
    auto page_of = [&](int tile) { return tile < tiles_seen ? pages_of[tile >> p.map.tpp_shift] : 0; };
    auto issue = [&](uint32_t stage, int tile, int page) {  // one lane
      const bool exists = tile < tiles_seen, good = exists && uint32_t(page) < uint32_t(p.map.num_pages);
      ok_flag[stage] = good;
      if (good) {
        mbar_arrive_expect_tx(full + stage, TB);
        bulk_load(ring + stage * TB, head + page * page_bytes + (tile & tpp_mask) * TB, TB, full + stage);
      } else {
        if (exists) atomicOr(p.map.status, DEV_PAGE);
        mbar_arrive(full + stage);
      }
    };
    int page_next = 0;
    int tile_next = first_tile + 2 * kWarps * ((NS + lane) >> 1) + ((NS + lane) & 1);  // lanes 0 and 1: their next tile
    if (!dead) {
      if (lane < NS && lane < 2 * mine) {
        const int tile = first_tile + 2 * kWarps * (lane >> 1) + (lane & 1);
        const uint32_t stage = st + lane;
        issue(stage < NS ? stage : stage - NS, tile, page_of(tile));
      }
      if (lane < 2) page_next = page_of(tile_next);
    }
    constexpr int kPasses = (R * NB / 32 + kWarps - 1) / kWarps;
    load_queries<D, QS, PAIR, kPasses>(p, sg.b, sg.h, sg.L, sg.n, sg.rg * R, PAIR ? 4 : R, &sq.frag[0][0][0][0][0], sq.c, sq.lim,
                              warp, lane, kWarps);
    __syncthreads();

    float m[NT][2], l[NT][2], c[NT][2];
    int lim[NT][2], lim_min = 0x7FFFFFFF;
    float o[NB][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        m[nt][x] = -INFINITY;
        l[nt][x] = 0.0f;
        c[nt][x] = sq.c[nt * 8 + 2 * t + x];
        lim[nt][x] = sq.lim[nt * 8 + 2 * t + x];
        lim_min = min(lim_min, lim[nt][x]);
      }
    lim_min = __reduce_min_sync(0xffffffffu, lim_min);
#pragma unroll
    for (int mb = 0; mb < NB; ++mb)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[mb][nt][i] = 0.0f;

    for (int it = 0; it < mine && !dead; ++it) {
      const int j0 = (c0 + warp + kWarps * it) * kChunk;
      float s[2][NT][4];
      const uint32_t st1 = st + 1 == NS ? 0 : st + 1, ph1 = st1 ? ph : ph ^ 1u;
      const bool in = kv4_wait(full + st, ph, p.wait_ns) && kv4_wait(full + st1, ph1, p.wait_ns);
      if (!__all_sync(0xffffffffu, in)) {
        // give up: report, and let the copies in flight land before the ring is reused
        dead = true;
        if (lane == 0) atomicOr(p.map.status, DEV_TIMEOUT);
        for (int i = 2 * it; i < 2 * it + NS && i < 2 * mine; ++i) {
          mbar_wait(full + st, ph, kKv4DrainNs);
          if (++st == NS) st = 0, ph ^= 1u;
        }
        break;
      }
      uint8_t* const tp[2] = {ring + st * TB, ring + st1 * TB};
      const bool there[2] = {ok_flag[st] != 0, ok_flag[st1] != 0};
      const bool whole = j0 + kChunk <= lim_min && there[0] && there[1];
      bool patched = false;
      if (!whole) {
        // Bytes of tokens past the end, or of a tile that is not there, are whatever
        // the memory held: their V scales become 0 (E2M1 codes are always finite).
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int left = there[u] ? sg.L - (j0 + u * kKv4Tile) : 0;
          if (left >= kKv4Tile) continue;
          patched = true;
          for (int i = lane; i < D; i += 32) {
            const int tok = 2 * (i / (4 * NB)) + (i & 1) + (i & 2 ? 8 : 0);
            if (tok >= left) tp[u][17 * D + i] = 0;
          }
        }
        __syncwarp();
      }
      const uint8_t* const tk[2] = {tp[0], tp[1]};
      tile_scores<D, NT, QS && !PAIR, 2>(tk, sq, lane, s);
      if constexpr (PAIR && QS) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[u][0][i] += __shfl_xor_sync(0xffffffffu, s[u][0][i], 2);
      }
      if (!whole) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!there[u] || j0 + u * kKv4Tile + g + 8 * (i >> 1) >= lim[nt][i & 1]) s[u][nt][i] = -INFINITY;
      }
      if constexpr (NT == 1) {
        const int W = PAIR || p.map.T * p.G <= 4 ? 16 : 32;  // up to 4 rows are in the first two lanes of four
        if (p.scores && (W == 32 || t < 2)) {
          float4* to = p.scores + ((int64_t(sg.b) * p.map.Hkv + sg.h) * (p.acc_ld / kKv4Tile) + (j0 / kKv4Tile)) * W +
                       (W == 16 ? g * 2 + t : lane);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (j0 + u * kKv4Tile < sg.L)
              to[u * W] = make_float4(s[u][0][0] * c[0][0], s[u][0][1] * c[0][1], s[u][0][2] * c[0][0], s[u][0][3] * c[0][1]);
        }
      } else if (p.scores) {
        const int n8 = (p.map.T * p.G + 7) >> 3;
        float4* to = p.scores + lane +
                     ((int64_t(sg.b) * p.map.Hkv + sg.h) * (p.acc_ld / kKv4Tile) + (j0 / kKv4Tile)) * n8 * 32;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (sg.rg * NT + nt < n8)
#pragma unroll
            for (int u = 0; u < 2; ++u)
              if (j0 + u * kKv4Tile < sg.L)
                to[(u * n8 + sg.rg * NT + nt) * 32] = make_float4(s[u][nt][0] * c[nt][0], s[u][nt][1] * c[nt][1],
                                                                  s[u][nt][2] * c[nt][0], s[u][nt][3] * c[nt][1]);
      }
      bool grew = false;
      float mnew[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float mx = fmaxf(fmaxf(s[0][nt][x], s[0][nt][x + 2]), fmaxf(s[1][nt][x], s[1][nt][x + 2]));
#pragma unroll
          for (int off = 4; off < 32; off *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          mnew[nt][x] = fmaxf(m[nt][x], mx == -INFINITY ? -INFINITY : mx * c[nt][x]);
          grew |= mnew[nt][x] != m[nt][x];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            // 0 the first time; 1 while nothing has been seen
            const float alpha = mnew[nt][x] == -INFINITY ? 1.0f : ex2(m[nt][x] - mnew[nt][x]);
            m[nt][x] = mnew[nt][x];
            l[nt][x] *= alpha;
#pragma unroll
            for (int mb = 0; mb < NB; ++mb) {
              o[mb][nt][x] *= alpha;
              o[mb][nt][x + 2] *= alpha;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          // a row that has seen nothing has only scores of -infinity: 2^(c s) = 0
          const float off = m[nt][x] == -INFINITY ? 0.0f : kPBits - m[nt][x];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int y = 0; y < 4; y += 2) {
              const float pv = ex2_ftz(fmaf(s[u][nt][x + y], c[nt][x], off));
              s[u][nt][x + y] = pv;
              l[nt][x] += pv;
            }
        }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = s[u][nt][2 * y], p1 = s[u][nt][2 * y + 1];
            uint32_t hi = pack_h2(p0, p1);
            if constexpr (PS && PAIR) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              const uint32_t lo = pack_h2(p0 - f.x, p1 - f.y);
              hi = t & 2 ? lo : hi;
            }
            ph[nt][y] = movmatrix_t(hi);
            if constexpr (PS && !PAIR) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
              pl[nt][y] = movmatrix_t(pack_h2(p0 - f.x, p1 - f.y));
            }
          }
        const uint4* vw = reinterpret_cast<const uint4*>(tp[u] + 8 * D);
        const uint4* vsc = reinterpret_cast<const uint4*>(tp[u] + 17 * D) + t * (NB / 4);
#pragma unroll
        for (int q = 0; q < NB / 4; ++q) {
          const uint4 w4 = vw[q * 32 + lane], s4 = vsc[q];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          const uint32_t sc[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a[4];
            kv4_v_frag(w[i], e4m3x2_to_h2(sc[i]), e4m3x2_to_h2(sc[i] >> 16), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816(o[4 * q + i][nt], a, ph[nt][0], ph[nt][1]);
              if constexpr (PS && !PAIR) mma_16816(o[4 * q + i][nt], a, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }
      if (patched) fence_proxy_async_smem();
      __syncwarp();  // the two stages have been read
      if (lane < 2 && 2 * it + NS + lane < 2 * mine) {
        issue(lane ? st1 : st, tile_next, page_next);
        tile_next += 2 * kWarps;
        page_next = page_of(tile_next);
      }
      st = st1 + 1 == NS ? 0 : st1 + 1;
      ph = st ? ph1 : ph1 ^ 1u;
      __syncwarp();
    }

    // join the warps: each scales its sums to the CTA's maximum
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int off = 4; off < 32; off *= 2) l[nt][x] += __shfl_xor_sync(0xffffffffu, l[nt][x], off);
        if (g == 0) s_ml[warp * R + nt * 8 + 2 * t + x] = make_float2(m[nt][x], l[nt][x]);
      }
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = nt * 8 + 2 * t + x;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w * R + r].x);
        const float f = m[nt][x] == -INFINITY ? 0.0f : ex2(m[nt][x] - mx);
#pragma unroll
        for (int mb = 0; mb < NB; ++mb) {
          s_o[(warp * R + r) * D + mb * 16 + g] = o[mb][nt][x] * f;
          s_o[(warp * R + r) * D + mb * 16 + g + 8] = o[mb][nt][x + 2] * f;
        }
      }
    __syncthreads();
    const bool entire = sg.entire(c1);
    for (int r = warp; r < R; r += kWarps) {
      const int row = sg.rg * R + r;
      if (row >= sg.n * p.G) break;
      float mx = -INFINITY, ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w * R + r].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * R + r];
        ls += ml.x == -INFINITY ? 0.0f : ml.y * ex2(ml.x - mx);
      }
      float x[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        x[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          x[e] += s_o[(w * R + r) * D + lane * (D / 32) + e];
          if constexpr (PS && PAIR) x[e] += s_o[(w * R + r + 4) * D + lane * (D / 32) + e];
        }
      }
      if constexpr (CL) {
        // for the cluster: this CTA's row in the place of its first warp's
        __syncwarp();
#pragma unroll
        for (int e = 0; e < D / 32; ++e) s_o[r * D + lane * (D / 32) + e] = x[e];
        if (lane == 0) s_ml[r] = make_float2(mx, ls);
      } else if (entire) {
        kv4_write_row<D>(p, sg.b, sg.h, row, lane, mx, ls, x, kPBits);
      } else {
        const int64_t to = (int64_t(blockIdx.x) * 2 + slot) * R + r;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) p.part_o[to * D + lane * (D / 32) + e] = x[e];
        if (lane == 0) p.part_ml[to] = make_float2(mx, ls);
      }
    }
    if constexpr (CL) {
      // Each CTA joins its share of the rows from all of them, over distributed shared memory.
      cluster_sync_all();
      const int rank = int(blockIdx.x) % p.cl;
      for (int r = rank + p.cl * warp; r < R; r += p.cl * kWarps) {
        const int row = sg.rg * R + r;
        if (row >= sg.n * p.G) break;
        float mx = -INFINITY, ls = 0.0f, x[D / 32] = {};
        for (int k = 0; k < p.cl; ++k) mx = fmaxf(mx, ld_cluster_f32(cluster_addr(&s_ml[r].x, k)));
        if (mx != -INFINITY)
          for (int k = 0; k < p.cl; ++k) {
            const float mk = ld_cluster_f32(cluster_addr(&s_ml[r].x, k)), lk = ld_cluster_f32(cluster_addr(&s_ml[r].y, k));
            const float f = mk == -INFINITY ? 0.0f : ex2(mk - mx);
            ls = fmaf(lk, f, ls);
#pragma unroll
            for (int e = 0; e < D / 32; ++e)
              x[e] = fmaf(ld_cluster_f32(cluster_addr(s_o + r * D + lane * (D / 32) + e, k)), f, x[e]);
          }
        kv4_write_row<D>(p, sg.b, sg.h, row, lane, mx, ls, x, kPBits);
      }
      cluster_sync_all();  // nobody leaves while its rows are read
      return;
    }
    const int4 record = sg.record(p, c1, slot);
    if (threadIdx.x == 0 && record.y >= 0) p.part_seg[blockIdx.x] = record;
    slot = 1;
    more = sg.next(p, c1);
    // the sums were plain stores where the next segment's copies will land
    fence_proxy_async_smem();
    __syncthreads();
  }
}

// acc_out[j] = acc_in[j] + sum over the rows that see j of exp(s_j - lse): the
// scores again, now that the rows' sums are known.  The chunks of all (sequence, KV
// head) are dealt as above; a warp turns the K half of two tiles into operands once and takes
// the rows past them, 8 at a time, so the sum has a fixed order.  n8 row tiles fit the shared
// memory; more rows take several passes, later ones adding to acc_out.
template <int D, bool QS>
struct WeightCfg {
  static constexpr int KB = 9 * D;              // K codes and scales of a tile
  static constexpr int NS = 8;                  // tiles in a warp's ring
  static constexpr int kTile8 = (QS ? 2 : 1) * (D / kKv4Block) * 256;  // bytes of 8 query rows
  static constexpr int kMax8 = 131072 / kTile8 < 32 ? 131072 / kTile8 : 32;
  static constexpr int smem(int n8) { return n8 * (kTile8 + 8 * 16) + kWarps * NS * (8 + 4) + kWarps * NS * KB + 256; }
  static constexpr int ctas(int n8) { return 232448 / (smem(n8) + 1024) < 4 ? 232448 / (smem(n8) + 1024) : 4; }
};

template <int D, bool QS>
__global__ void __launch_bounds__(kThreads, 4) k_kv4_weights(const Kv4AttnParams p, int n8) {
  using C = WeightCfg<D, QS>;
  constexpr int NB = D / kKv4Block, NS = C::NS, KB = C::KB, TB = kv4_tile_bytes(D), P = QS ? 2 : 1;
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring0 = smem;
  uint32_t* frag = reinterpret_cast<uint32_t*>(ring0 + kWarps * NS * KB);  // [n8][term][block][lane][2]
  uint64_t* bars = reinterpret_cast<uint64_t*>(frag + n8 * (C::kTile8 / 4));
  int* s_ok = reinterpret_cast<int*>(bars + kWarps * NS);
  float* s_c = reinterpret_cast<float*>(s_ok + kWarps * NS);
  float* s_bias = s_c + n8 * 8;
  int* s_lim = reinterpret_cast<int*>(s_bias + n8 * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = ring0 + warp * (NS * KB);
  uint64_t* full = bars + warp * NS;
  int* ok_flag = s_ok + warp * NS;
  if (lane < NS) mbar_init(full + lane, 1);
  fence_mbar_init();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  Kv4Line<kKv4AllRows, kChunk> sg;
  bool more = sg.template begin<kWarps>(p, blockIdx.x, kWarps);
  uint32_t st = 0, ph = 0;
  const int64_t page_bytes = (int64_t(p.map.Hkv) << p.map.tpp_shift) * TB;
  const int tpp_mask = (1 << p.map.tpp_shift) - 1;
  bool dead = false;
  while (more) {
    const int c0 = sg.c0, c1 = sg.last_chunk(), rows = sg.n * p.G;
    if (sg.nothing()) {
      more = sg.next(p, c1);
      continue;
    }
    const int tiles_seen = (sg.L + kKv4Tile - 1) / kKv4Tile;
    const int c_end = min(c1, (sg.L + kChunk - 1) / kChunk);
    const int mine = c_end - c0 - warp > 0 ? (c_end - c0 - warp + kWarps - 1) / kWarps : 0;
    const int32_t* pages_of = p.map.table + int64_t(sg.b) * p.map.max_pages;
    const uint8_t* head = p.map.pages + (int64_t(sg.h) << p.map.tpp_shift) * TB;
    const int64_t acc_at = (int64_t(sg.b) * p.map.Hkv + sg.h) * p.acc_ld;
    auto tile_of = [&](int i) { return 2 * (c0 + warp + kWarps * (i >> 1)) + (i & 1); };
    auto page_of = [&](int i) {
      const int tile = tile_of(i);
      return i < 2 * mine && tile < tiles_seen ? pages_of[tile >> p.map.tpp_shift] : 0;
    };
    auto issue = [&](uint32_t stage, int i, int page) {  // one lane
      const int tile = tile_of(i);
      const bool exists = tile < tiles_seen, good = exists && uint32_t(page) < uint32_t(p.map.num_pages);
      ok_flag[stage] = good;
      if (good) {
        const uint8_t* src = head + page * page_bytes + (tile & tpp_mask) * TB;
        mbar_arrive_expect_tx(full + stage, KB);
        bulk_load(ring + stage * KB, src, 8 * D, full + stage);
        bulk_load(ring + stage * KB + 8 * D, src + 16 * D, D, full + stage);
      } else {
        if (exists) atomicOr(p.map.status, DEV_PAGE);
        mbar_arrive(full + stage);
      }
    };
    for (int row0 = 0; row0 == 0 || row0 < rows; row0 += n8 * 8) {
      const int t8 = min(n8, (rows - row0 + 7) / 8);  // row tiles of this pass (0: no rows at all)
      int next_i = NS + lane, page_next = 0;
      if (!dead) {
        if (lane < NS && lane < 2 * mine) issue(st + lane < NS ? st + lane : st + lane - NS, lane, page_of(lane));
        if (lane < 2) page_next = page_of(next_i);
      }
      __syncthreads();  // the pass before has read its rows
      load_queries<D, QS, false, 4>(p, sg.b, sg.h, sg.L, sg.n, row0, t8 * 8, frag, s_c, s_lim, warp, lane, kWarps);
      for (int i = threadIdx.x; i < t8 * 8; i += kThreads) {
        const int row = row0 + i;
        float bias = -INFINITY;  // rows that are not there, or see nothing, weigh nothing
        if (row < rows) {
          const float l = p.lse2[sg.b * p.lse_sb + (sg.h * p.G + row % p.G) * p.lse_sh + row / p.G];
          if (l != -INFINITY) bias = -l;
        }
        s_bias[i] = bias;
      }
      __syncthreads();
      int lim_min = 0x7FFFFFFF;
      for (int i = lane; i < t8 * 8; i += 32) lim_min = min(lim_min, s_lim[i]);
      lim_min = __reduce_min_sync(0xffffffffu, lim_min);
      for (int it = 0; it < mine && !dead; ++it) {
        const int j0 = (c0 + warp + kWarps * it) * kChunk;
        // lane (g, t) ends with the sum of token j0 + 16 (t / 2) + 8 (t % 2) + g
        const int j = j0 + (t >> 1) * 16 + (t & 1) * 8 + g;
        float sum = 0.0f;
        if (j < sg.L) {
          if (row0 > 0) sum = p.acc_out[acc_at + j];
          else if (p.acc_in) sum = p.acc_in[acc_at + j];
        }
        const uint32_t st1 = st + 1 == NS ? 0 : st + 1, ph1 = st1 ? ph : ph ^ 1u;
        const bool in = kv4_wait(full + st, ph, p.wait_ns) && kv4_wait(full + st1, ph1, p.wait_ns);
        if (!__all_sync(0xffffffffu, in)) {
          dead = true;
          if (lane == 0) atomicOr(p.map.status, DEV_TIMEOUT);
          for (int i = 2 * it; i < 2 * it + NS && i < 2 * mine; ++i) {
            mbar_wait(full + st, ph, kKv4DrainNs);
            if (++st == NS) st = 0, ph ^= 1u;
          }
          break;
        }
        const bool there[2] = {ok_flag[st] != 0, ok_flag[st1] != 0};
        uint32_t a[2][NB][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint8_t* k = ring + (u ? st1 : st) * KB;
#pragma unroll
          for (int q = 0; q < NB / 4; ++q) {
            const uint4 w4 = reinterpret_cast<const uint4*>(k)[q * 32 + lane];
            const uint2 s2 = reinterpret_cast<const uint2*>(k + 8 * D)[g * (NB / 4) + q];
            const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w}, sc[2] = {s2.x, s2.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) kv4_k_frag(w[i], e4m3x2_to_h2(sc[i >> 1] >> (16 * (i & 1))), a[u][4 * q + i]);
          }
        }
        __syncwarp();  // the two stages have been read
        if (lane < 2 && next_i < 2 * mine) {
          issue(lane ? st1 : st, next_i, page_next);
          next_i += 2;
          page_next = page_of(next_i);
        }
        st = st1 + 1 == NS ? 0 : st1 + 1;
        ph = st ? ph1 : ph1 ^ 1u;
        const bool whole = j0 + kChunk <= lim_min && there[0] && there[1];
        float w[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        for (int nt = 0; nt < t8; ++nt) {
          const uint2* fb = reinterpret_cast<const uint2*>(frag) + nt * (P * NB * 32) + lane;
          float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint2 q0 = fb[b * 32];
            mma_16816(s[0], a[0][b], q0.x, q0.y);
            mma_16816(s[1], a[1][b], q0.x, q0.y);
            if constexpr (QS) {
              const uint2 q1 = fb[(NB + b) * 32];
              mma_16816(s[0], a[0][b], q1.x, q1.y);
              mma_16816(s[1], a[1][b], q1.x, q1.y);
            }
          }
          const float2 c = *reinterpret_cast<const float2*>(s_c + nt * 8 + 2 * t);
          const float2 bias = *reinterpret_cast<const float2*>(s_bias + nt * 8 + 2 * t);
          if (whole) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int y = 0; y < 2; ++y)
                w[u][y] += ex2_ftz(fmaf(s[u][2 * y], c.x, bias.x)) + ex2_ftz(fmaf(s[u][2 * y + 1], c.y, bias.y));
          } else {
            const int2 lim = *reinterpret_cast<const int2*>(s_lim + nt * 8 + 2 * t);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const int tok = j0 + 16 * u + 8 * y + g;
                if (there[u] && tok < lim.x) w[u][y] += ex2_ftz(fmaf(s[u][2 * y], c.x, bias.x));
                if (there[u] && tok < lim.y) w[u][y] += ex2_ftz(fmaf(s[u][2 * y + 1], c.y, bias.y));
              }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            w[u][y] += __shfl_xor_sync(0xffffffffu, w[u][y], 1);
            w[u][y] += __shfl_xor_sync(0xffffffffu, w[u][y], 2);
          }
        const float mine_w = t & 2 ? (t & 1 ? w[1][1] : w[1][0]) : (t & 1 ? w[0][1] : w[0][0]);
        if (j < sg.L) p.acc_out[acc_at + j] = sum + mine_w;
      }
    }
    more = sg.next(p, c1);
  }
}

// The same from the scores that k_kv4_attn has left: their bytes are read instead of K turned into operands
// and multiplied again.  With up to 8 rows a warp takes eight tiles, W lanes (16 for up to 4 rows,
// else 32) to a tile: 8 x 16384 tokens of 32 heads on 8 take 9 us (2 of them for the stores in
// k_kv4_attn), where reading K again took 31.  The kept scores have been rounded to fp32 (c s, log2 units, as
// the rows' maxima and log-sums are), where the kernel above has one fma: 2^-24 of the score.
// acc_in and the lengths are read before the wait for the kernels before: none of this call's writes them.
constexpr int kScoreTiles = 8;
template <int W>
__global__ void __launch_bounds__(kThreads) k_kv4_weigh_scores(const Kv4AttnParams p) {
  constexpr int PER = 32 / W, STEPS = kScoreTiles / PER;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane % W / (W / 8), t = lane % (W / 8);
  const int b = blockIdx.y / p.map.Hkv, h = blockIdx.y % p.map.Hkv;
  const int L = kv4_len(p.map, b), rows = kv4_new(p.map, b) * p.G;
  const int tile0 = (int(blockIdx.x) * kWarps + warp) * kScoreTiles;
  if (tile0 * kKv4Tile >= L) {
    // nothing to do, but the grid may not end before the kernels it depends on: the call's end is its end
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  const int64_t acc_at = int64_t(blockIdx.y) * p.acc_ld;
  const float4* from = p.scores + (int64_t(blockIdx.y) * (p.acc_ld / kKv4Tile) + tile0) * W + lane;
  float old[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int j = (tile0 + i * PER + lane / W) * kKv4Tile + g + 8 * t;  // lanes t < 2 end with token g + 8 t
    old[i] = p.acc_in && t < 2 && j < L ? p.acc_in[acc_at + j] : 0.0f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 s[STEPS];
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
    s[i] = (tile0 + i * PER + lane / W) * kKv4Tile < L && rows > 0 ? from[i * 32] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  bool live[2];
  float bias[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = 2 * t + x;
    const float l = row < rows ? p.lse2[b * p.lse_sb + (h * p.G + row % p.G) * p.lse_sh + row / p.G] : -INFINITY;
    live[x] = l != -INFINITY;  // rows that are not there, or see nothing, weigh nothing
    bias[x] = -l;
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    float w[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const float s0 = y ? s[i].z : s[i].x, s1 = y ? s[i].w : s[i].y;  // masked ones are -infinity
      w[y] = (live[0] ? ex2_ftz(s0 + bias[0]) : 0.0f) + (live[1] ? ex2_ftz(s1 + bias[1]) : 0.0f);
#pragma unroll
      for (int o = 1; o < W / 8; o *= 2) w[y] += __shfl_xor_sync(0xffffffffu, w[y], o);
    }
    const int j = (tile0 + i * PER + lane / W) * kKv4Tile + g + 8 * t;
    if (t < 2 && j < L) p.acc_out[acc_at + j] = old[i] + (t ? w[1] : w[0]);
  }
}

// More rows: a warp takes a tile past all of them, 8 rows at a time, so the sum has a fixed order.
// 2 x 32 queries of 12 heads on 2 over 4001 tokens: 3 us, where K took 33.  (Eight CTAs an SM leave
// registers for eight loads in flight a lane; without the bound the compiler took 32 and 2 us more.)
constexpr int kScoreRows = 512;  // rows whose sums are in shared memory at a time
__global__ void __launch_bounds__(kThreads, 8) k_kv4_weigh_many(const Kv4AttnParams p) {
  __shared__ float s_bias[kScoreRows];
  __shared__ int s_lim[kScoreRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.y / p.map.Hkv, h = blockIdx.y % p.map.Hkv;
  const int L = kv4_len(p.map, b), n = kv4_new(p.map, b), rows = n * p.G, n8 = (p.map.T * p.G + 7) >> 3;
  const int tile = int(blockIdx.x) * kWarps + warp;
  if (int(blockIdx.x) * kWarps * kKv4Tile >= L) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // as above
    return;
  }
  const float4* from = p.scores + (int64_t(blockIdx.y) * (p.acc_ld / kKv4Tile) + tile) * n8 * 32 + lane;
  const int j0 = tile * kKv4Tile + g, j = j0 + 8 * t;  // lanes t < 2 end with token j
  const bool mine = t < 2 && j < L;
  const int64_t acc_at = int64_t(blockIdx.y) * p.acc_ld + j;
  const float old = mine && p.acc_in ? p.acc_in[acc_at] : 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float w[2] = {0.0f, 0.0f};
  for (int row0 = 0; row0 < rows; row0 += kScoreRows) {
    const int here = min(rows - row0, kScoreRows), tiles = (here + 7) >> 3;
    __syncthreads();  // the rows before have been read
    for (int i = threadIdx.x; i < (tiles + 7) / 8 * 64; i += kThreads) {
      const int row = row0 + i;
      float bias = 0.0f;
      int lim = 0;  // rows that are not there, or see nothing, weigh nothing
      if (row < rows) {
        const float l = p.lse2[b * p.lse_sb + (h * p.G + row % p.G) * p.lse_sh + row / p.G];
        bias = -l;
        if (l != -INFINITY) lim = p.causal ? min(max(L - n + row / p.G + 1, 0), L) : L;
      }
      s_bias[i] = bias;
      s_lim[i] = lim;
    }
    __syncthreads();
    if (tile * kKv4Tile < L) {
#pragma unroll 1
      for (int i = 0; i < tiles; i += 8) {
        float4 s[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) s[q] = from[(row0 / 8 + min(i + q, tiles - 1)) * 32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float2 bias = *reinterpret_cast<const float2*>(s_bias + (i + q) * 8 + 2 * t);
          const int2 lim = *reinterpret_cast<const int2*>(s_lim + (i + q) * 8 + 2 * t);
          // scores past a row's limit may never have been written; past the last row tile no row sees anything
          w[0] += (j0 < lim.x ? ex2_ftz(s[q].x + bias.x) : 0.0f) + (j0 < lim.y ? ex2_ftz(s[q].y + bias.y) : 0.0f);
          w[1] += (j0 + 8 < lim.x ? ex2_ftz(s[q].z + bias.x) : 0.0f) + (j0 + 8 < lim.y ? ex2_ftz(s[q].w + bias.y) : 0.0f);
        }
      }
    }
  }
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    w[y] += __shfl_xor_sync(0xffffffffu, w[y], 1);
    w[y] += __shfl_xor_sync(0xffffffffu, w[y], 2);
  }
  if (mine) p.acc_out[acc_at] = old + (t ? w[1] : w[0]);
}

struct Plan {
  int R, n_cta, n_rg, cl;
};

// Row groups of 8, 16, 24 or 32 of the rows of a KV head, and as many CTAs as the GPU holds at once
// (or as there are chunks for their warps).
Plan plan_of(int B, int max_tokens, int Hkv, int64_t rows) {
  Plan pl{};
  pl.R = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 24 ? 24 : 32;
  const int64_t n_rg = (rows + pl.R - 1) / pl.R;
  const int64_t fill = int64_t(kKv4PlanSms) * (pl.R == 8 ? 4 : pl.R <= 16 ? 3 : 2);
  const int64_t chunks = int64_t(B) * Hkv * n_rg * ((max_tokens + kChunk - 1) / kChunk);
  const int64_t most = (chunks + kWarps - 1) / kWarps;
  pl.n_cta = int(fill < most ? fill : most);
  pl.n_rg = int(n_rg);
  // Up to 8 rows, short sequences in small batches: a cluster of CTAs to each segment, 16 chunks a CTA at the most,
  // joins its rows itself and saves the second launch (14 -> 10 us for one user's 1024 tokens).
  // Lengths are not known here, only what the page table can hold.
  const int64_t segs = int64_t(B) * Hkv * n_rg, longest = (max_tokens + kChunk - 1) / kChunk;
  int cl = 1;
  while (cl < 8 && cl * 4 * kWarps < longest) cl *= 2;
  if (pl.R == 8 && longest <= 32 * kWarps && segs * cl <= fill) pl.cl = cl;
  return pl;
}

// The tcgen05 kernel's, for bf16 outputs.
Plan prefill_plan(int B, int max_tokens, int Hq, int Hkv, int T) {
  Plan pl{};
  const int64_t rows = int64_t(T) * (Hq / Hkv);
  pl.R = kKv4PrefillRows;
  const int64_t chunks = int64_t(B) * Hkv * ((rows + pl.R - 1) / pl.R) * ((max_tokens + 127) / 128);
  pl.n_cta = int(chunks < kKv4PlanSms ? chunks : kKv4PlanSms);
  // 0: not for these sizes.  With 8 x 8 KV heads of 8192 tokens (d 128) the tcgen05 kernel takes
  // 70.6 us for 32 rows (the mma.sync kernel 50.1), 72.6 (80.5) for 48 and 101 (271) for 256; with fewer
  // chunks than the GPU has SMs, 8 KV heads of 2048 tokens, 25.0 (17.0), 25.2 (18.5) and 31.3 (29.2).
  if (rows <= 32 || (chunks < 2 * kKv4PlanSms && rows <= pl.R)) pl.n_cta = 0;
  return pl;
}

size_t plan_bytes(const Plan& pl, int d) {
  const size_t rows = size_t(pl.n_cta) * 2 * pl.R;
  return kv4_a256(rows * d * 4) + kv4_a256(rows * 8) + kv4_a256(size_t(pl.n_cta) * 16);
}

// Bytes for the parts of a call with either kernel (the output's type, which is not known here, chooses between
// them) or with fewer rows, whose smaller groups leave room for more CTAs: a call needs no more
// than one with more sequences, places or rows.
size_t parts_bytes(int B, int max_tokens, int Hq, int Hkv, int T, int d) {
  const int64_t rows = int64_t(T) * (Hq / Hkv);
  size_t most = plan_bytes(prefill_plan(B, max_tokens, Hq, Hkv, T), d);
  for (const int64_t n : {int64_t(8), int64_t(16), int64_t(24), int64_t(32), rows}) {
    const size_t x = plan_bytes(plan_of(B, max_tokens, Hkv, n < rows ? n : rows), d);
    most = x > most ? x : most;
  }
  return most;
}

// Bytes of the scores that k_kv4_attn leaves where there is room for them: up to half of the
// L2's 126 MB.  Past that they would travel to memory and back, and K is read again instead.
constexpr size_t kMaxScores = size_t(64) << 20;
size_t scores_bytes(int B, int64_t max_tokens, int Hq, int Hkv, int T) {
  const int64_t rows = int64_t(T) * (Hq / Hkv), most = int64_t(kMaxScores);
  const int64_t token = int64_t(B) * Hkv * (rows <= 4 ? 16 : (rows + 7) / 8 * 32);  // bytes of a token place
  return token <= most / max_tokens ? size_t(token * max_tokens) : kMaxScores + 1;
}

template <int D, bool QS>
cudaError_t run_weights(const Kv4AttnParams& q, int max_tokens, cudaStream_t s) {
  using C = WeightCfg<D, QS>;
  Kv4AttnParams p = q;
  const int64_t need8 = (int64_t(p.map.T) * p.G + 7) / 8;
  const int n8 = int(need8 < C::kMax8 ? need8 : C::kMax8);
  const int64_t chunks = int64_t(p.map.B) * p.map.Hkv * ((max_tokens + kChunk - 1) / kChunk);
  const int64_t most = (chunks + kWarps - 1) / kWarps, fill = int64_t(kKv4PlanSms) * C::ctas(n8);
  p.n_cta = int(fill < most ? fill : most);
  p.ov = n8 <= 2 ? kOverhead : kManyRowsOverhead;
  p.cl = 0;
  auto kern = k_kv4_weights<D, QS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = kv4_allow_smem(reinterpret_cast<const void*>(kern), C::smem(C::kMax8), done);
  if (e != cudaSuccess) return e;
  return kv4_launch_after(kern, dim3(p.n_cta), size_t(C::smem(n8)), s, p, n8);
}

template <int D, int NT, bool QS, bool PS, bool PAIR, bool CL>
cudaError_t launch_attn(const Kv4AttnParams& p, const Plan& pl, cudaStream_t s) {
  using C = Cfg<D, NT, QS>;
  auto kern = k_kv4_attn<D, NT, QS, PS, PAIR, CL>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv4_allow_smem(reinterpret_cast<const void*>(kern), C::SMEM, done);
  if (e != cudaSuccess) return e;
  if constexpr (CL)
    return kv4_launch_cluster(kern, dim3(unsigned(p.map.B) * p.map.Hkv * p.n_rg * p.cl), p.cl, C::SMEM, s, p);
  kern<<<pl.n_cta, kThreads, C::SMEM, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return kv4_launch_after(k_kv4_join<D, C::R>, dim3(pl.n_cta * (C::R / 4)), 0, s, p, kPBits);
}

template <int D, int NT, bool QS, bool PS, bool PAIR = false>
cudaError_t run(const Kv4AttnParams& p, const Plan& pl, int max_tokens, cudaStream_t s) {
  cudaError_t e;
  if constexpr (NT == 1)
    e = p.cl ? launch_attn<D, NT, QS, PS, PAIR, true>(p, pl, s) : launch_attn<D, NT, QS, PS, PAIR, false>(p, pl, s);
  else
    e = launch_attn<D, NT, QS, PS, PAIR, false>(p, pl, s);
  if (e != cudaSuccess || !p.acc_out) return e;
  if (p.scores && NT > 1) {
    const dim3 grid((max_tokens + kWarps * kKv4Tile - 1) / (kWarps * kKv4Tile), unsigned(p.map.B) * p.map.Hkv);
    return kv4_launch_after(k_kv4_weigh_many, grid, 0, s, p);
  }
  if (p.scores) {
    const dim3 grid((max_tokens + kWarps * kScoreTiles * kKv4Tile - 1) / (kWarps * kScoreTiles * kKv4Tile),
                    unsigned(p.map.B) * p.map.Hkv);
    return kv4_launch_after(p.map.T * p.G <= 4 ? k_kv4_weigh_scores<16> : k_kv4_weigh_scores<32>, grid, 0, s, p);
  }
  return run_weights<D, QS>(p, max_tokens, s);
}

template <int D, int NT>
cudaError_t run_nt(const Kv4AttnParams& p, const Plan& pl, int max_tokens, cudaStream_t s) {
  if constexpr (NT == 1) {
    if (int64_t(p.map.T) * p.G <= 4) {
      if (!p.q_bf16 || p.signs)
        return p.o_bf16 ? run<D, 1, true, false, true>(p, pl, max_tokens, s)
                        : run<D, 1, true, true, true>(p, pl, max_tokens, s);
      if (!p.o_bf16) return run<D, 1, false, true, true>(p, pl, max_tokens, s);
    }
  }
  if (!p.q_bf16 || p.signs)
    return p.o_bf16 ? run<D, NT, true, false>(p, pl, max_tokens, s) : run<D, NT, true, true>(p, pl, max_tokens, s);
  return p.o_bf16 ? run<D, NT, false, false>(p, pl, max_tokens, s) : run<D, NT, false, true>(p, pl, max_tokens, s);
}

template <int D>
cudaError_t run_d(const Kv4AttnParams& p, const Plan& pl, int max_tokens, cudaStream_t s) {
  if (pl.R == kKv4PrefillRows) {
    const bool inexact = !p.q_bf16 || p.signs;  // queries that one fp16 term rounds
    cudaError_t e = launch_kv4_prefill(p, D, inexact && (p.lse || p.acc_out), s);
    if (e != cudaSuccess || !p.acc_out) return e;
    return inexact ? run_weights<D, true>(p, max_tokens, s) : run_weights<D, false>(p, max_tokens, s);
  }
  if (pl.R == 8) return run_nt<D, 1>(p, pl, max_tokens, s);
  if (pl.R == 16) return run_nt<D, 2>(p, pl, max_tokens, s);
  if (pl.R == 24) return run_nt<D, 3>(p, pl, max_tokens, s);
  return run_nt<D, 4>(p, pl, max_tokens, s);
}

}  // namespace

// Without the scores this is what a call needs; with them, what serves it and every call of
// fewer sequences, places or rows at its best.
size_t kv4_attn_workspace_bytes(int B, int max_pages, int page_tokens, int Hq, int Hkv, int T, int d, bool with_scores) {
  const int max_tokens = max_pages * page_tokens;
  const size_t need = parts_bytes(B, max_tokens, Hq, Hkv, T, d) + kv4_a256(size_t(B) * Hq * T * 4);
  const size_t scores = scores_bytes(B, max_tokens, Hq, Hkv, T);
  return with_scores ? need + kv4_a256(scores < kMaxScores ? scores : kMaxScores) : need;
}

cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s) {
  const Kv4Args& kv = a.kv;
  const int max_tokens = kv.max_pages * kv.page_tokens;
  Plan pl = prefill_plan(kv.B, max_tokens, a.Hq, kv.Hkv, kv.T);
  const bool many = a.o_bf16 && pl.n_cta > 0;
  if (!many) pl = plan_of(kv.B, max_tokens, kv.Hkv, int64_t(kv.T) * (a.Hq / kv.Hkv));
  Kv4AttnParams p{};
  p.map = kv4_map(kv);
  p.Q = a.Q;
  p.O = a.O;
  p.q_bf16 = a.q_bf16;
  p.o_bf16 = a.o_bf16;
  p.G = a.Hq / kv.Hkv;
  p.n_cta = pl.n_cta;
  p.ov = many ? kPrefillOverhead : kOverhead;
  p.cl = pl.cl;
  p.n_rg = pl.n_rg;
  p.causal = a.causal;
  p.signs = kv.signs;
  p.k_scale = kv.k_scale;
  p.v_scale = kv.v_scale;
  p.inv_sqrt_d = kv.d == 128 ? 0.08838834764831845f : 0.125f;
  p.scale_log2e = float(double(a.scale) * 1.4426950408889634073599246810018921);
  const size_t rows = size_t(pl.n_cta) * 2 * pl.R;
  uint8_t* w = static_cast<uint8_t*>(a.ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += kv4_a256(rows * kv.d * 4);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += kv4_a256(rows * 8);
  p.part_seg = reinterpret_cast<int4*>(w);
  w += kv4_a256(size_t(pl.n_cta) * 16);
  uint8_t* tail = w + kv4_a256(size_t(kv.B) * a.Hq * kv.T * 4);
  const size_t scores = scores_bytes(kv.B, max_tokens, a.Hq, kv.Hkv, kv.T);
  const size_t room = a.ws_bytes - size_t(tail - static_cast<uint8_t*>(a.ws));
  p.scores = a.acc_out && !many && scores <= kMaxScores && scores <= room ? reinterpret_cast<float4*>(tail) : nullptr;
  p.lse = a.lse;
  p.lse2 = a.acc_out ? reinterpret_cast<float*>(w) : nullptr;
  p.lse_sb = int64_t(a.Hq) * kv.T;
  p.lse_sh = kv.T;
  p.acc_in = a.acc_in;
  p.acc_out = a.acc_out;
  p.acc_ld = max_tokens;
  p.wait_ns = kv.wait_ns;
  return kv.d == 128 ? run_d<128>(p, pl, max_tokens, s) : run_d<64>(p, pl, max_tokens, s);
}

}  // namespace attnq
