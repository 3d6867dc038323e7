// Attention over the 4-bit KV cache for many query rows (chunks of a prompt), on
// tcgen05 tensor cores: the mathematics of kv4_attn.cu, with products that are
// large enough to fill 128-row tiles.
//
// Work: a segment is 256 rows (query, head of the group) of a (sequence, KV head), two
// tiles of 128; a chunk is 128 tokens.  One CTA an SM; the chunks of all segments are
// dealt evenly (Kv4Line) and rows that several CTAs had are joined by k_kv4_join.
//
// CTA = 512 threads:
//   warps 0-3, 4-7  softmax, a thread half a row of both row tiles (TMEM lane = row); they also
//                   bring in, rotate and normalise the query rows of a segment
//   warps 8-11      turn 4-bit tiles into fp16: K as [token][channel] and V^T as
//                   [channel][token], 128-byte swizzled, the layout the MMA reads.  The
//                   cache's fragments are 8x8 matrices, so stmatrix stores them as
//                   they are.
//   warp 12         issues the MMAs (13 to 15 idle)
// TMEM columns: S_w at 128 w; O_w at 256 + D w.  P_w (fp16, twice 32 columns) takes the place of
// S_w's columns once they are read, and is the A operand of O_w += P_w V straight
// from there: no P in shared memory.
//
// Per row tile and chunk: S = Q K^T (behind O += P V of the chunk before, whose P lies in
// S's columns) -> row maximum (tcgen05.ld.red) -> P -> O += P V.  The two row tiles
// alternate on the tensor core.  O is rescaled only when a row's maximum has grown by more than
// 2^8 over the one in use: P is held as 2^(7 + s - m), so it stays below 2^15.
//
// A K or V tile is made once for 256 rows: about 8000 warp instructions a chunk, 2000 issue slots of
// an SM quadrant, of which the softmax has 1200 and the tiles 700, beside 2048 clocks of MMAs
// (4 x 128^3 products at 4096 multiply-adds a clock) and 2300 of shared memory (S reads 128 bytes
// a clock, all there is).  2 x 1024 rows of 32 heads on 16384 tokens (533 GFLOP) take 471 us,
// 1.13 PFLOP/s, about 3600 clocks a chunk.  Left are the chain S, softmax, P V of a row tile with the
// hand-overs between the roles, and what the two roles that give registers away spill (464 to 484 bytes
// of stores in the compiler's report); how much each costs has not been told apart.
//
// Precision: K, V and queries as in kv4_attn.cu, but rotated or fp32 queries are rounded to fp16
// once, 2^-11, unless lse or weights are asked for (QS: two terms; 2 x 1024 rotated rows as above take 626 us
// with them, 410 instead of 405 with d 64).  P, rounded to fp16 once, keeps all of its bits down to 2^-21 of the
// weight of the row's maximum and vanishes below 2^-32 of it (l still counts it): a step of 2^-24
// under P = 2^7, which is as high as the lag of 2^8 leaves.  bf16 outputs only.
//
// Every wait is bounded; on a timeout the CTA records DEV_TIMEOUT, every role leaves
// its loop, the MMAs in flight are drained (bounded again) and TMEM is freed.
#include <cfloat>

#include "kv4_attn.cuh"

namespace attnq {
namespace {

constexpr int kRows = 128;             // rows of a query tile
constexpr int kPre = 256;              // rows of a segment
constexpr int kTok = 128;              // tokens of a chunk
constexpr int kPreThreads = 512;
// launched at 128 registers a thread; 2 x 128 x 176 + 128 x 104 + 128 x 48 = 64,512 of 65,536
constexpr uint32_t kSoftRegs = 176, kTileRegs = 104, kMmaRegs = 48;
static_assert(256 * kSoftRegs + 128 * kTileRegs + 128 * kMmaRegs <= kPreThreads * 128, "register split");
constexpr float kPreBits = 7.0f;       // P = 2^(7 + s - m)
constexpr float kGrow = 8.0f;          // m is let lag by up to 2^8

template <int D, bool QS>
struct PreCfg {
  static constexpr int QT = kRows * D * 2;              // bytes of a query tile (one term)
  static constexpr int NQ = QS ? 4 : 2;
  static constexpr int KB = kTok * D * 2;               // bytes of a K (and of a V^T) tile
  static constexpr int TB = kv4_tile_bytes(D);
  // K and V^T stages, and 4-bit tiles in each tile warp's ring (two a chunk), that fit
  // (one K stage is enough: the next K is needed only after this chunk's S products, V beside them)
  static constexpr int NSK = 1, NSV = QS && D == 128 ? 1 : 2, RT = QS && D == 128 ? 3 : 6;
  static constexpr int NBARS = 1 + 2 * NSK + 2 * NSV + 6 + 1 + 4 * RT;
  static constexpr int SMEM = 1024 + NQ * QT + (NSK + NSV) * KB + 4 * RT * TB + 8 * NBARS + 16 + 4 * 8 + 4 * RT * 4 + 3 * kPre * 4;
  static_assert(SMEM <= 232448, "shared memory");
};

template <typename T>
__device__ __forceinline__ void swap2(T (&x)[2]) {
  const T t = x[0];
  x[0] = x[1];
  x[1] = t;
}

struct PreBars {
  uint64_t *q_full, *k_full, *k_empty, *v_full, *v_empty;
  uint64_t* s_full;   // [2] S_w in TMEM (commit)
  uint64_t* p_full;   // [2] P_w in TMEM, O_w rescaled (256 arrivals)
  uint64_t* o_done;   // [2] O_w += P_w V complete (commit)
  uint64_t* drain;
  uint64_t* raw;      // [4][RT] a 4-bit tile has landed in a tile warp's ring
};

// Bounded wait that also ends when another role has given up.  Plain polling: try_wait with a
// suspend-time hint wakes later, and every wait here is on the path (520 us with it, 461 without).
__device__ __forceinline__ bool pre_wait(uint64_t* bar, uint32_t parity, const Kv4AttnParams& p,
                                         volatile int* abort_flag) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (p.wait_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > p.wait_ns) break;
  }
  *abort_flag = 1;
  atomicOr(p.map.status, DEV_TIMEOUT);
  return false;
}
// The same for a whole warp, which leaves it converged.
__device__ __forceinline__ bool pre_wait_warp(uint64_t* bar, uint32_t parity, const Kv4AttnParams& p,
                                              volatile int* abort_flag) {
  return __all_sync(0xffffffffu, pre_wait(bar, parity, p, abort_flag));
}

__device__ __forceinline__ void stmatrix4(uint32_t addr, const uint32_t (&a)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a[0]), "r"(a[1]),
               "r"(a[2]), "r"(a[3])
               : "memory");
}

// Chunks of the segment that are this CTA's and that some row sees: [c0, end).
template <typename Seg>
__device__ __forceinline__ int chunks_here(const Seg& sg) {
  const int end = min(sg.last_chunk(), (sg.vis + kTok - 1) / kTok);
  return max(end - sg.c0, 0);
}

// ---- warps 8-11: 4-bit tiles -> fp16 operand tiles ---------------------------
// A warp makes tiles warp and warp + 4 of each chunk.  It copies its own 4-bit tiles RT ahead into
// its own ring (as the warps of kv4_attn.cu do).
template <int D, bool QS>
__device__ __forceinline__ void make_tiles(const Kv4AttnParams& p, Kv4Line<kPre, kTok> sg, uint8_t* sK, uint8_t* sV,
                                           uint8_t* s_raw, int* s_ok, uint8_t* s_there, const PreBars& br,
                                           volatile int* abort_flag) {
  using C = PreCfg<D, QS>;
  constexpr int NB = D / kKv4Block, TB = C::TB, RT = C::RT;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // stmatrix: lane l gives the address of row l % 8 of matrix l / 8 (matrix: + 8 rows for bit 0, + 8 columns for bit 1)
  const uint32_t mi = uint32_t(lane & 7), mx = uint32_t(lane >> 3);
  const uint32_t row_off = mi * 128u + (mx & 1u) * 1024u, swz = ((mx >> 1) ^ mi) << 4;
  uint8_t* ring = s_raw + warp * (RT * TB);
  int* ok_flag = s_ok + warp * RT;
  uint64_t* full = br.raw + warp * RT;
  const int64_t page_bytes = (int64_t(p.map.Hkv) << p.map.tpp_shift) * TB;
  const int mask = (1 << p.map.tpp_shift) - 1;
  uint32_t it = 0, st = 0, ph = 0;  // chunks of the segments before; ring stage of the next tile and its parity
  do {
    if (sg.nothing()) continue;
    const int todo = chunks_here(sg);
    const int32_t* pages_of = p.map.table + int64_t(sg.b) * p.map.max_pages;
    const uint8_t* head = p.map.pages + (int64_t(sg.h) << p.map.tpp_shift) * TB;
    const int c0 = sg.c0, L = sg.L, tiles = (L + kKv4Tile - 1) / kKv4Tile;
    auto tile_of = [&](int i) { return (c0 + (i >> 1)) * 8 + warp + 4 * (i & 1); };
    auto page_of = [&](int i) {
      const int tile = tile_of(i);
      return i < 2 * todo && tile < tiles ? pages_of[tile >> p.map.tpp_shift] : 0;
    };
    auto issue = [&](uint32_t stage, int i, int page) {  // one lane
      const int tile = tile_of(i);
      const bool exists = tile < tiles, good = exists && uint32_t(page) < uint32_t(p.map.num_pages);
      ok_flag[stage] = good;
      if (good) {
        mbar_arrive_expect_tx(full + stage, TB);
        bulk_load(ring + stage * TB, head + page * page_bytes + (tile & mask) * TB, TB, full + stage);
      } else {
        if (exists) atomicOr(p.map.status, DEV_PAGE);
        mbar_arrive(full + stage);
      }
    };
    int next_i = RT + lane, page_next = 0;  // lanes 0 and 1: their next tile
    if (lane < RT && lane < 2 * todo) {
      const uint32_t stage = st + lane;
      issue(stage < RT ? stage : stage - RT, lane, page_of(lane));
    }
    if (lane < 2) page_next = page_of(next_i);
    bool ok = true;
    int done = 0;  // chunks whose tiles have been given back to the ring
    // K of chunk k from the ring stages at (st, ph): wait for them and for the K stage's last readers
    auto make_k = [&](int k) -> bool {
      const uint32_t i = it + uint32_t(k), sk = i % C::NSK;
      const uint32_t stage[2] = {st, st + 1 == RT ? 0u : st + 1}, par[2] = {ph, st + 1 == RT ? ph ^ 1u : ph};
      if (!pre_wait_warp(full + stage[0], par[0], p, abort_flag) ||
          !pre_wait_warp(full + stage[1], par[1], p, abort_flag) ||
          !pre_wait_warp(br.k_empty + sk, ((i / C::NSK) & 1u) ^ 1u, p, abort_flag))
        return false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bool there = ok_flag[stage[u]] != 0;
        const int tile = warp + 4 * u;
        const uint8_t* raw = ring + stage[u] * TB;
        const uint32_t dst = smem_u32(sK) + sk * uint32_t(C::KB) + uint32_t(tile) * 2048u + row_off;
#pragma unroll
        for (int q = 0; q < NB / 4; ++q) {
          const uint4 w4 = reinterpret_cast<const uint4*>(raw)[q * 32 + lane];
          const uint2 s2 = reinterpret_cast<const uint2*>(raw + 16 * D)[g * (NB / 4) + q];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w}, sc[2] = {s2.x, s2.y};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t a[4];
            kv4_k_frag(w[x], e4m3x2_to_h2(sc[x >> 1] >> (16 * (x & 1))), a);
            stmatrix4(dst + uint32_t(q) * uint32_t(kTok * 128) + (swz ^ (uint32_t(x) << 5)), a);
          }
        }
        // the ring of four flags outlives its readers: S of the next chunk is issued when the softmax of this one
        // has handed P over, and it has to be done before K of the chunk after that is made here
        if (lane == 0) s_there[(i & 3u) * 8 + tile] = there;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(br.k_full + sk);
      return true;
    };
    // V of chunk k from the stages at (st, ph), which then take the next copies
    auto make_v = [&](int k) -> bool {
      const uint32_t sv = (it + uint32_t(k)) % C::NSV;
      const uint32_t st1 = st + 1 == RT ? 0u : st + 1, ph1 = st + 1 == RT ? ph ^ 1u : ph;
      if (!pre_wait_warp(br.v_empty + sv, (((it + uint32_t(k)) / C::NSV) & 1u) ^ 1u, p, abort_flag)) return false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tile = warp + 4 * u;
        const uint32_t stage = u ? st1 : st;
        const int left = ok_flag[stage] ? L - ((c0 + k) * 8 + tile) * kKv4Tile : 0;
        // tokens past the end, and tiles that are not there: whatever the memory held, scaled by 0
        uint32_t keep = 0xFFFFFFFFu;
        if (left < kKv4Tile) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (2 * t + (e & 1) + (e >> 1) * 8 >= left) keep &= ~(0xFFu << (8 * e));
        }
        const uint8_t* raw = ring + stage * TB;
        const uint32_t dst =
            smem_u32(sV) + sv * uint32_t(C::KB) + uint32_t(tile >> 2) * uint32_t(D * 128) + row_off;
        const uint32_t col = swz ^ (uint32_t(tile & 3) << 5);
#pragma unroll
        for (int q = 0; q < NB / 4; ++q) {
          const uint4 w4 = reinterpret_cast<const uint4*>(raw + 8 * D)[q * 32 + lane];
          const uint4 s4 = reinterpret_cast<const uint4*>(raw + 17 * D)[t * (NB / 4) + q];
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
          const uint32_t sc[4] = {s4.x & keep, s4.y & keep, s4.z & keep, s4.w & keep};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t a[4];
            kv4_v_frag(w[x], e4m3x2_to_h2(sc[x]), e4m3x2_to_h2(sc[x] >> 16), a);
            stmatrix4(dst + uint32_t(4 * q + x) * 2048u + col, a);
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(br.v_full + sv);
      if (lane < 2 && next_i < 2 * todo) {
        issue(lane ? st1 : st, next_i, page_next);
        next_i += 2;
        page_next = page_of(next_i);
      }
      st = st1 + 1 == RT ? 0u : st1 + 1;
      ph = st ? ph1 : ph1 ^ 1u;
      ++done;
      __syncwarp();
      return true;
    };
    for (int k = 0; ok && k < todo; ++k) ok = make_k(k) && make_v(k);
    if (!ok) {
      // let the copies in flight land before the CTA ends
      for (int i = 2 * done; i < 2 * done + RT && i < 2 * todo; ++i) {
        mbar_wait(full + st, ph, kKv4DrainNs);
        if (++st == RT) st = 0, ph ^= 1u;
      }
      return;
    }
    it += uint32_t(todo);
  } while (sg.next(p, sg.last_chunk()));
}

// ---- warp 12: the MMAs ---------------------------------------------------------
// One warp issues for both row tiles, in the order P V and next S of tile 0, P V and next S
// of tile 1.  Each tile's two products then run back to back and the other tile's
// softmax runs beside them; with a warp to each tile both softmaxes came to run at the
// same time and the tensor core waited for both.
template <int D, bool QS>
__device__ __forceinline__ void issue_mmas(const Kv4AttnParams& p, Kv4Line<kPre, kTok> sg, uint32_t tmem, uint8_t* sQ,
                                           uint8_t* sK, uint8_t* sV, const PreBars& br, volatile int* abort_flag) {
  using C = PreCfg<D, QS>;
  constexpr uint32_t idS = idesc_f16_f32(kRows, kTok), idO = idesc_f16_f32(kRows, D);
  const uint32_t hi = uint32_t(smem_desc(0, 16, 1024, 2) >> 32);
  const uint32_t lQ0 = uint32_t(smem_desc(smem_u32(sQ), 16, 1024, 2));
  const uint32_t lK0 = uint32_t(smem_desc(smem_u32(sK), 16, 1024, 2));
  const uint32_t lV0 = uint32_t(smem_desc(smem_u32(sV), 16, 1024, 2));
  uint32_t it = 0, n_seg = 0;  // chunks of the segments before, segments
  uint32_t par0 = 0, par1 = 0;  // parity of the next P of this row tile, and of the other
  bool ok = true, issued = false;
  do {
    if (sg.nothing()) continue;
    const int todo = chunks_here(sg);
    const int act = sg.rg * kPre + kRows < sg.n * p.G ? 2 : 1;  // row tiles that have rows
    if (todo == 0) continue;
    if (!(ok = pre_wait_warp(br.q_full, n_seg & 1u, p, abort_flag))) break;
    ++n_seg;
    // step (k, w): P V of chunk k and S of chunk k + 1 for row tile w, from k = -1 on.  The code stands
    // here once for all of them: unrolled by tile the kernel outgrew the instruction cache.
#pragma unroll 1
    for (int k = -1; ok && k < todo; ++k) {
      const uint32_t sv = (it + uint32_t(k)) % C::NSV, sk = (it + uint32_t(k + 1)) % C::NSK;
      if (k >= 0 && !(ok = pre_wait_warp(br.v_full + sv, ((it + uint32_t(k)) / C::NSV) & 1u, p, abort_flag))) break;
#pragma unroll 1
      for (int w = 0; w < act; ++w) {
        const uint32_t tS = tmem + uint32_t(w * kTok), tO = tmem + 256u + uint32_t(w * D);
        if (k >= 0) {
          if (!(ok = pre_wait_warp(br.p_full + w, par0, p, abort_flag))) break;
          par0 ^= 1u;
          tc_fence_after();
          const uint32_t lv = lV0 + sv * uint32_t(C::KB >> 4);
#pragma unroll
          for (int kk = 0; kk < kTok / 16; ++kk)
            // P of the second 64 tokens begins at column 64, where their S did
            mma_f16_ts_elect(tO, tS + uint32_t(8 * (kk & 3) + 64 * (kk >> 2)),
                             pack_desc(lv + uint32_t(kk >> 2) * uint32_t(D * 8) + uint32_t(2 * (kk & 3)), hi), idO,
                             (k > 0 || kk > 0) ? 1u : 0u);
          mma_commit_elect(br.o_done + w);
          if (w + 1 == act) mma_commit_elect(br.v_empty + sv);
        }
        if (k + 1 < todo) {
          if (w == 0 &&
              !(ok = pre_wait_warp(br.k_full + sk, ((it + uint32_t(k + 1)) / C::NSK) & 1u, p, abort_flag)))
            break;
          tc_fence_after();
          // the next S goes where P of this chunk lies: MMAs run in the order they are
          // issued, so P V has read it by then
          const uint32_t lq = lQ0 + uint32_t(w * ((C::NQ / 2) * C::QT >> 4)), lk = lK0 + sk * uint32_t(C::KB >> 4);
#pragma unroll
          for (int part = 0; part < (QS ? 2 : 1); ++part)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              // 16 channels are 32 bytes: four steps a 128-byte column block, then the next block
              const uint32_t cb = uint32_t(kk >> 2), sub = uint32_t(2 * (kk & 3));
              mma_f16_ss_elect(tS, pack_desc(lq + uint32_t(part * (C::QT >> 4)) + cb * uint32_t(kRows * 8) + sub, hi),
                               pack_desc(lk + cb * uint32_t(kTok * 8) + sub, hi), idS, (part > 0 || kk > 0) ? 1u : 0u);
            }
          issued = true;
          mma_commit_elect(br.s_full + w);
          if (w + 1 == act) mma_commit_elect(br.k_empty + sk);
        }
        if (act == 2) {
          const uint32_t x = par0;
          par0 = par1;
          par1 = x;
        }
      }
    }
    if (!ok) break;
    it += uint32_t(todo);
  } while (sg.next(p, sg.last_chunk()));
  if (!ok && issued) {
    mma_commit_elect(br.drain);
    mbar_wait(br.drain, 0, kKv4DrainNs);
    __syncwarp();
  }
}

// ---- warps 0-7: query rows, softmax, epilogue ----------------------------------
// A warpgroup has half of the columns of both row tiles: 64 of S (and of P, which takes the
// first 32 columns of that half), D / 2 of O.  Both work on one tile at a time, so a tile's softmax
// takes half as long and the other tile's products run beside it; a row's two halves
// exchange their maxima through shared memory.
template <int D, bool QS>
__device__ __forceinline__ void softmax_rows(const Kv4AttnParams& p, Kv4Line<kPre, kTok> sg, uint32_t tmem, uint8_t* sQ,
                                             const uint8_t* s_there, float* s_norm, float* s_max, const PreBars& br,
                                             volatile int* abort_flag) {
  using C = PreCfg<D, QS>;
  constexpr int NB = D / kKv4Block, RPP = 32 / NB, HC = kTok / 2, HD = D / 2;
  const int half = threadIdx.x >> 7, r = threadIdx.x & 127, lane = threadIdx.x & 31, wq = r >> 5;
  const uint32_t lane_off = uint32_t(wq * 32) << 16;
  uint32_t it = 0;               // chunks of the CTA
  uint32_t par[2] = {0u, 0u};    // parity of the next S of each row tile
  uint32_t flip = 0;             // buffer of the next exchange
  int slot = 0;
  // after a timeout the warps go on without waiting or computing, so that none
  // is left behind at a barrier that the two warpgroups share
  bool more = true, dead = false;
  while (more) {
    if (sg.nothing()) {
      more = sg.next(p, sg.last_chunk());
      continue;
    }
    const int todo = chunks_here(sg), c0 = sg.c0, c1 = sg.last_chunk();
    const int rows = sg.n * p.G;
    const int act = sg.rg * kPre + kRows < rows ? 2 : 1;  // row tiles that have rows
    // query rows of row tile `half`: a lane holds a block of 16 channels, NB lanes a row
    if (half < act && !dead) {
      uint8_t* my_q = sQ + half * (C::NQ / 2) * C::QT;
      constexpr int AT = 32 / RPP < 4 ? 32 / RPP : 4;  // passes whose loads are in flight at a time
      Kv4Raw16 raw[AT];
#pragma unroll 1
      for (int pass0 = 0; pass0 < 32 / RPP; pass0 += AT) {
        const int i0 = wq * 32 + pass0 * RPP + lane / NB, blk = lane % NB;
#pragma unroll
        for (int u = 0; u < AT; ++u)
          raw[u] = kv4_query_row(p, sg.b, sg.h, sg.n, sg.rg * kPre + half * kRows + i0 + u * RPP, true, blk);
#pragma unroll
        for (int u = 0; u < AT; ++u) {
          const int i = i0 + u * RPP;
          float x[16], norm;
          kv4_unpack16(raw[u], p.q_bf16, x);
          // by a power of two, as in kv4_attn.cu
          const float down = kv4_normalise16<D>(p, x, blk, norm);
          if (blk == 0) s_norm[half * kRows + i] = norm;
          uint32_t q[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = pack_h2(x[2 * e] * down, x[2 * e + 1] * down);
          // chunk c of 8 channels of row i: column block c / 8, swizzled by the row
          uint8_t* at = my_q + (blk >> 2) * (kRows * 128) + i * 128;
          const int c = 2 * (blk & 3), sw = i & 7;
          *reinterpret_cast<uint4*>(at + ((c ^ sw) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
          *reinterpret_cast<uint4*>(at + (((c + 1) ^ sw) << 4)) = make_uint4(q[4], q[5], q[6], q[7]);
          if constexpr (QS) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&q[e]));
              q[e] = pack_h2(x[2 * e] * down - f.x, x[2 * e + 1] * down - f.y);
            }
            at += C::QT;
            *reinterpret_cast<uint4*>(at + ((c ^ sw) << 4)) = make_uint4(q[0], q[1], q[2], q[3]);
            *reinterpret_cast<uint4*>(at + (((c + 1) ^ sw) << 4)) = make_uint4(q[4], q[5], q[6], q[7]);
          }
        }
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();  // O of the segment before has been read
    // a segment that sees no token has no MMAs: nothing would hold these warps back until
    // warp 12 has seen the phase, and two such segments would take the barrier past it
    if (todo > 0) mbar_arrive(br.q_full);
    named_bar_sync(1, 256);  // the other warps' norms
    float c[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int lim[2], lim_min[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int row = sg.rg * kPre + w * kRows + r;
      const bool live = row < rows;
      c[w] = w < act ? fmaxf(p.scale_log2e * (p.k_scale ? p.k_scale[sg.h] : 1.0f) * s_norm[w * kRows + r], FLT_MIN) : 1.0f;
      // tokens the row sees; rows that are not there see all, their results go nowhere
      lim[w] = live ? (p.causal ? min(max(sg.L - sg.n + row / p.G + 1, 0), sg.L) : sg.L) : 0x7FFFFFFF;
      lim_min[w] = __reduce_min_sync(0xffffffffu, lim[w]);
    }
    // One body for both row tiles, whose states change places after each step (unrolled by
    // tile the kernel outgrew the instruction cache): index 0 is the tile at hand.
    const int steps = todo * act;
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const int w = act == 2 ? step & 1 : 0, k = act == 2 ? step >> 1 : step;
      const uint32_t tS = tmem + lane_off + uint32_t(w * kTok + half * HC);
      const uint32_t tO = tmem + lane_off + 256u + uint32_t(w * D + half * HD);
      const int j0 = (c0 + k) * kTok + half * HC;
      if (!dead && !pre_wait_warp(br.s_full + w, par[0], p, abort_flag)) dead = true;
      par[0] ^= 1u;
      if (dead) {
        named_bar_sync(2 + wq, 64);  // the partner warp may be waiting for its exchange
        continue;
      }
      tc_fence_after();
      const uint32_t there =
          *reinterpret_cast<const uint32_t*>(s_there + ((it + uint32_t(k)) & 3u) * 8 + uint32_t(half * 4));
      const bool whole = j0 + HC <= lim_min[0] && there == 0x01010101u;
      const int left = lim[0] - j0;
      auto masked = [&](int j) { return j >= left || !((there >> (8 * (j >> 4))) & 1u); };
      float v[2][32], mx;
      if (whole) {
        // the maximum of each 32 columns comes with the load
        float hm[2];
        tmem_ld32f_max(tS, v[0], hm[0]);
        tmem_ld32f_max(tS + 32u, v[1], hm[1]);
        tmem_wait_ld();
        reg_fence32(v[0]);
        reg_fence32(v[1]);
        asm volatile("" : "+f"(hm[0]), "+f"(hm[1]));
        mx = fmaxf(hm[0], hm[1]);
      } else {
        tmem_ld32f(tS, v[0]);
        tmem_ld32f(tS + 32u, v[1]);
        tmem_wait_ld();
        reg_fence32(v[0]);
        reg_fence32(v[1]);
        mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < HC; ++j) {
          v[j >> 5][j & 31] = masked(j) ? -INFINITY : v[j >> 5][j & 31];
          mx = fmaxf(mx, v[j >> 5][j & 31]);
        }
      }
      // the row's other half: the same warp of the other warpgroup
      s_max[flip * kPre + half * kRows + r] = mx;
      named_bar_sync(2 + wq, 64);
      mx = fmaxf(mx, s_max[flip * kPre + (half ^ 1) * kRows + r]);
      flip ^= 1u;
      const float mt = mx == -INFINITY ? -INFINITY : mx * c[0];
      if (__any_sync(0xffffffffu, mt > m[0] + kGrow)) {  // -infinity + 8 is -infinity: the first tokens seen count as growth
        const float mnew = fmaxf(m[0], mt);
        const float alpha = mnew == -INFINITY ? 1.0f : ex2(m[0] - mnew);
        m[0] = mnew;
        l[0] *= alpha;
        // O += P V of the chunk before is complete: the commit of S covers what was issued before it
        if (k > 0) {
#pragma unroll 1
          for (int q = 0; q < HD / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(tO + uint32_t(32 * q), o);
            tmem_wait_ld();
            reg_fence32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + uint32_t(32 * q), o);
          }
        }
      }
      const float off = m[0] == -INFINITY ? 0.0f : kPreBits - m[0];
      const uint64_t c2 = pack2(c[0], c[0]), off2 = pack2(off, off);
      uint64_t ls[2] = {pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t pw[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          float a, b;
          unpack2(ffma2(pack2(v[q][2 * j], v[q][2 * j + 1]), c2, off2), a, b);
          a = ex2_ftz(a);
          b = ex2_ftz(b);
          ls[j & 1] = fadd2(ls[j & 1], pack2(a, b));
          pw[j] = pack_h2(a, b);
        }
        tmem_st16(tS + uint32_t(16 * q), pw);  // this half of S has been read
      }
      float a0, a1, b0, b1;
      unpack2(ls[0], a0, a1);
      unpack2(ls[1], b0, b1);
      l[0] += (a0 + a1) + (b0 + b1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(br.p_full + w);
      if (act == 2) {
        swap2(m);
        swap2(l);
        swap2(c);
        swap2(lim);
        swap2(lim_min);
        swap2(par);
      }
    }
    it += uint32_t(todo);
    // row sums of both halves
    named_bar_sync(1, 256);
    float* s_sum = s_max;
#pragma unroll
    for (int w = 0; w < 2; ++w) s_sum[(half * 2 + w) * kRows + r] = l[w];
    named_bar_sync(1, 256);
#pragma unroll
    for (int w = 0; w < 2; ++w) l[w] = s_sum[w * kRows + r] + s_sum[(2 + w) * kRows + r];
    const bool entire = sg.entire(c1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      if (w >= act) break;
      if (todo > 0 && !dead) {
        // (as many P V products as S: the last one's parity)
        if (!pre_wait_warp(br.o_done + w, par[w] ^ 1u, p, abort_flag)) dead = true;
        tc_fence_after();
      }
      if (dead) break;
      const int row = sg.rg * kPre + w * kRows + r;
      const bool live = row < rows;
      const int tq = row / p.G, head = sg.h * p.G + row % p.G;
      const float gv = p.v_scale ? p.v_scale[sg.h] : 1.0f;
      const float inv = l[w] > 0.0f ? __fdiv_rn(gv, l[w]) : 0.0f;
      const int64_t to = (int64_t(blockIdx.x) * 2 + slot) * kPre + w * kRows + r;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(const_cast<void*>(p.O.ptr)) + sg.b * p.O.sb +
                                            int64_t(head) * p.O.sh + int64_t(tq) * p.O.st + half * HD);
      float4* part = reinterpret_cast<float4*>(p.part_o + to * D + half * HD);
#pragma unroll 1
      for (int q = 0; q < HD / 32; ++q) {
        uint32_t o[32];
        if (todo > 0) {
          tmem_ld32(tmem + lane_off + 256u + uint32_t(w * D + half * HD + 32 * q), o);
          tmem_wait_ld();
          reg_fence32(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (!live) continue;
        if (entire) {
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[8 * v4 + 2 * e]) * inv,
                                                              __uint_as_float(o[8 * v4 + 2 * e + 1]) * inv);
              x[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            dst[4 * q + v4] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        } else {
#pragma unroll
          for (int v4 = 0; v4 < 8; ++v4)
            part[8 * q + v4] = make_float4(__uint_as_float(o[4 * v4]), __uint_as_float(o[4 * v4 + 1]),
                                           __uint_as_float(o[4 * v4 + 2]), __uint_as_float(o[4 * v4 + 3]));
        }
      }
      if (live && half == 0) {
        if (!entire) p.part_ml[to] = make_float2(m[w], l[w]);
        else kv4_write_lse(p, sg.b * p.lse_sb + head * p.lse_sh + tq, m[w], l[w], kPreBits);
      }
    }
    const int4 record = sg.record(p, c1, slot);
    if (record.y >= 0 && threadIdx.x == 0) p.part_seg[blockIdx.x] = record;
    more = sg.next(p, c1);
    slot = 1;
    named_bar_sync(1, 256);  // the norms and sums have been read
  }
}

template <int D, bool QS>
__global__ void __launch_bounds__(kPreThreads, 1) k_kv4_prefill(const Kv4AttnParams p) {
  using C = PreCfg<D, QS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = sm;                       // [row tile][term]
  uint8_t* sK = sQ + C::NQ * C::QT;       // [stage]
  uint8_t* sV = sK + C::NSK * C::KB;
  uint8_t* s_raw = sV + C::NSV * C::KB;   // [tile warp][ring]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_raw + 4 * C::RT * C::TB);
  PreBars br;
  br.q_full = bars;
  br.k_full = bars + 1;
  br.k_empty = br.k_full + C::NSK;
  br.v_full = br.k_empty + C::NSK;
  br.v_empty = br.v_full + C::NSV;
  br.s_full = br.v_empty + C::NSV;
  br.p_full = br.s_full + 2;
  br.o_done = br.p_full + 2;
  br.drain = br.o_done + 2;
  br.raw = br.drain + 1;
  uint8_t* s_there = reinterpret_cast<uint8_t*>(br.raw + 4 * C::RT);  // [4][8] tiles of a chunk that are there
  int* s_ok = reinterpret_cast<int*>(s_there + 32);                  // [tile warp][ring]
  float* s_norm = reinterpret_cast<float*>(s_ok + 4 * C::RT);
  float* s_max = s_norm + kPre;                                       // [2][2][row]
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_max + 2 * kPre);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    mbar_init(br.q_full, 256);
    for (int s = 0; s < C::NSK; ++s) {
      mbar_init(br.k_full + s, 4);
      mbar_init(br.k_empty + s, 1);
    }
    for (int s = 0; s < C::NSV; ++s) {
      mbar_init(br.v_full + s, 4);
      mbar_init(br.v_empty + s, 1);
    }
    for (int s = 0; s < 4 * C::RT; ++s) mbar_init(br.raw + s, 1);
    for (int w = 0; w < 2; ++w) {
      mbar_init(br.s_full + w, 1);
      mbar_init(br.p_full + w, 256);
      mbar_init(br.o_done + w, 1);
    }
    mbar_init(br.drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  Kv4Line<kPre, kTok> sg;
  const bool any = sg.template begin<kPreThreads / 32>(p, blockIdx.x, 2);
  // until the last segment is done (and if it never is) this CTA leaves nothing to join
  if (threadIdx.x == 0) p.part_seg[blockIdx.x] = make_int4(0, -1, 0, 0);
  if (!any) return;
  if (warp == 12) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if (warp < 8) {
    regs_increase<kSoftRegs>();
    softmax_rows<D, QS>(p, sg, tmem, sQ, s_there, s_norm, s_max, br, abort_flag);
  } else if (warp < 12) {
    regs_decrease<kTileRegs>();
    make_tiles<D, QS>(p, sg, sK, sV, s_raw, s_ok, s_there, br, abort_flag);
  } else {
    regs_decrease<kMmaRegs>();
    if (warp == 12) issue_mmas<D, QS>(p, sg, tmem, sQ, sK, sV, br, abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool QS>
cudaError_t run_prefill(const Kv4AttnParams& p, cudaStream_t s) {
  auto kern = k_kv4_prefill<D, QS>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = kv4_allow_smem(reinterpret_cast<const void*>(kern), PreCfg<D, QS>::SMEM, done);
  if (e != cudaSuccess) return e;
  kern<<<p.n_cta, kPreThreads, PreCfg<D, QS>::SMEM, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return kv4_launch_after(k_kv4_join<D, kPre>, dim3(p.n_cta * (kPre / 4)), 0, s, p, kPreBits);
}

}  // namespace

cudaError_t launch_kv4_prefill(const Kv4AttnParams& p, int d, bool two_terms, cudaStream_t s) {
  if (d == 128) return two_terms ? run_prefill<128, true>(p, s) : run_prefill<128, false>(p, s);
  return two_terms ? run_prefill<64, true>(p, s) : run_prefill<64, false>(p, s);
}

}  // namespace attnq
