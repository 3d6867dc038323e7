// Eviction from the 4-bit KV cache by accumulated attention weight: per
// (sequence, KV head) the first n_sink and the last n_recent tokens stay, and
// of those between them the ones with the largest weights, ties going to the
// lower place.  k_kv4_select finds the places, a block to a head; k_kv4_gather copies codes
// and scales into the new pages.
//
// Select: the k-th largest weight is found exactly, on the weights' bits.  Up to 32
// tokens a thread (32768) the keys stay in registers and the threshold is narrowed by
// counts of the keys at or above a candidate (about 12 of them): no atomics, and equal weights
// (a cache has thousands of zeros) cost nothing, where a histogram's atomics
// on one bin took most of 53 us.  8 x 8 heads of 32768 tokens take 31 us (37 with the threshold
// built bit by bit and the kept tokens marked one by one).  Of a CTA's 47,000 clocks there 11,000 go to loading the
// weights, 6,000 to their keys, 19,500 to the counts (1,560 each with 1024 threads an SM), 4,000 to marks and
// prefixes, 1,500 to placing the numbers and 4,000 to the stores.  Longer sequences take four histogram passes of 8
// bits over memory.  Two block-wide sums then place the kept tokens in order; their
// numbers go through shared memory, so that the stores are whole lines.
#include "internal.h"
#include "kv4.cuh"

namespace attnq {
namespace {

constexpr int kSelThreads = 1024;

struct EvictParams {
  Kv4Map map;           // source
  const float* acc;
  int64_t acc_ld;
  int budget, n_sink, n_recent;
  const int32_t* dst_table;
  int dst_pages;
  int32_t* new_lens;
  int32_t* kept;
  float* acc_out;
  int64_t acc_out_ld;
};

// Orders floats as unsigned integers; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive prefix of `v` over the block; `total` its sum.  `buf`: 33 words.
__device__ __forceinline__ int block_prefix(int v, int* buf, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int w = buf[lane];
    const int own = w;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    buf[lane] = w - own;
    if (lane == 31) buf[32] = w;
  }
  __syncthreads();
  total = buf[32];
  return buf[warp] + inc - v;
}

struct SelectRange {
  int L, lo, hi, k;  // k tokens wanted of [lo, hi)
  int32_t* kept;
  const float* acc;
  float* acc_out;
};

// What both forms begin with.  False: everything stays, and has been written.
__device__ __forceinline__ bool select_begin(const EvictParams& p, SelectRange& r) {
  const int bh = blockIdx.x, b = bh / p.map.Hkv;
  r.L = kv4_len(p.map, b);
  const int n = min(r.L, p.budget);
  r.kept = p.kept + int64_t(bh) * p.budget;
  r.acc = p.acc + int64_t(bh) * p.acc_ld;
  r.acc_out = p.acc_out ? p.acc_out + int64_t(bh) * p.acc_out_ld : nullptr;
  if (bh % p.map.Hkv == 0 && threadIdx.x == 0) p.new_lens[b] = n;
  for (int i = n + threadIdx.x; i < p.budget; i += kSelThreads) r.kept[i] = -1;
  if (r.L <= p.budget) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) {
      r.kept[i] = i;
      if (r.acc_out) r.acc_out[i] = r.acc[i];
    }
    return false;
  }
  r.lo = p.n_sink;
  r.hi = r.L - p.n_recent;
  r.k = p.budget - p.n_sink - p.n_recent;
  return true;
}

// Sum of v over the block.
__device__ __forceinline__ int block_sum(int v, int* buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, buf[threadIdx.x & 31]);
}

// Thread t holds the ITEMS tokens from t * ITEMS on, brought through shared
// memory (rows padded by one word) so that the loads are coalesced.
template <int ITEMS>
__global__ void __launch_bounds__(kSelThreads) k_kv4_select(const EvictParams p) {
  extern __shared__ float s_acc[];
  uint16_t* s_kept = reinterpret_cast<uint16_t*>(s_acc + (ITEMS + 1) * kSelThreads);
  __shared__ int buf[33];
  __shared__ uint32_t s_range[2];
  SelectRange r;
  if (!select_begin(p, r)) return;
  if (threadIdx.x == 0) {
    s_range[0] = 0xFFFFFFFFu;
    s_range[1] = 0u;
  }
  {
    constexpr int AT = ITEMS < 16 ? ITEMS : 16;  // loads in flight at a time
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < r.L; i0 += AT * kSelThreads) {
      float v[AT];
#pragma unroll
      for (int q = 0; q < AT; ++q) v[q] = i0 + q * kSelThreads < r.L ? r.acc[i0 + q * kSelThreads] : 0.0f;
#pragma unroll
      for (int q = 0; q < AT; ++q) {
        const int i = i0 + q * kSelThreads;
        if (i < r.L) s_acc[i + i / ITEMS] = v[q];
      }
    }
  }
  __syncthreads();
  const int base = threadIdx.x * ITEMS;
  // keys of the tokens that compete; 0, the key of a NaN, may stand for no token: it is never counted
  uint32_t key[ITEMS];
  uint32_t least = 0xFFFFFFFFu, most = 0u;
#pragma unroll
  for (int q = 0; q < ITEMS; ++q) {
    const int i = base + q;
    const bool in = i >= r.lo && i < r.hi;
    // NaN ranks below every number, above the places that do not compete
    key[q] = in ? max(weight_key(s_acc[i + threadIdx.x]), 1u) : 0u;
    if (in) least = min(least, key[q]);
    most = max(most, key[q]);
  }
  uint32_t thr = 0;
  int above = 0;  // keys > thr
  if (r.k > 0) {
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if ((threadIdx.x & 31) == 0) {
      atomicMin(&s_range[0], least);
      atomicMax(&s_range[1], most);
    }
    __syncthreads();
    // at_lo >= k keys are >= lo, at_hi < k are >= hi, until lo and hi are neighbours or at_lo is k: then
    // what stays is decided.  The candidate is where a straight line between the two counts meets
    // k, or the middle when the line has left more than a quarter of the interval; after two steps that
    // left lo in place its neighbour, in case lo is where the equal weights are.
    uint32_t lo = s_range[0], hi = s_range[1] + 1u;
    int at_lo = r.hi - r.lo, at_hi = 0, stuck = 0;
    bool middle = false;
    while (hi - lo > 1u && at_lo != r.k) {
      const uint32_t width = hi - lo;
      uint32_t cand;
      if (stuck == 2) cand = lo + 1u;
      else if (middle) cand = lo + width / 2u;
      else cand = lo + min(max(uint32_t(float(width) * __fdividef(float(at_lo - r.k), float(at_lo - at_hi))), 1u), width - 1u);
      int c = 0;
#pragma unroll
      for (int q = 0; q < ITEMS; ++q) c += key[q] >= cand;
      c = block_sum(c, buf);
      if (c >= r.k) {
        lo = cand;
        at_lo = c;
        stuck = 0;
      } else {
        hi = cand;
        at_hi = c;
        ++stuck;
      }
      middle = !middle && hi - lo > width / 4u;
    }
    // exactly k keys from lo on: all of them stay, and none that equals lo - 1 (at least 0) is wanted
    thr = at_lo == r.k ? lo - 1u : lo;
    above = at_lo == r.k ? r.k : at_hi;
  }
  const int need = r.k - above;  // tokens equal to thr that stay, the first ones
  // bit q: token base + q.  It stays outside [lo, hi), above thr, or as an early enough tie.
  uint32_t keep = 0, tie = 0;
#pragma unroll
  for (int q = 0; q < ITEMS; ++q) {
    if (key[q] > thr) keep |= 1u << q;
    if (key[q] == thr) tie |= 1u << q;
  }
  if (r.k == 0) keep = 0;
  const auto below = [&](int j) {  // bits of the tokens before j
    const int n = min(max(j - base, 0), ITEMS);
    return n == 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
  };
  const uint32_t in = below(r.hi) & ~below(r.lo);
  tie &= in;
  int total;
  int tie_at = 0;
  if (need > 0) tie_at = block_prefix(__popc(tie), buf, total);
  for (int drop = __popc(tie) - max(need - tie_at, 0); drop > 0; --drop) tie &= ~(0x80000000u >> __clz(tie));
  keep = (keep & in) | tie | (below(r.L) & ~in);
  int at = block_prefix(__popc(keep), buf, total);
  for (; keep; keep &= keep - 1) s_kept[at++] = uint16_t(base + __ffs(int(keep)) - 1);
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += kSelThreads) {
    const int j = s_kept[i];
    r.kept[i] = j;
    if (r.acc_out) r.acc_out[i] = s_acc[j + j / ITEMS];
  }
}

__global__ void __launch_bounds__(kSelThreads) k_kv4_select_long(const EvictParams p) {
  __shared__ int hist[256];
  __shared__ int buf[33];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  SelectRange r;
  if (!select_begin(p, r)) return;
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_need = r.k;
  }
  // after pass i the top 8 (i + 1) bits of the k-th largest key are known, and
  // s_need counts the wanted keys that share them
  for (int pass = 0; pass < 4 && r.k > 0; ++pass) {
    const int sh = 24 - 8 * pass;
    for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int i = r.lo + threadIdx.x; i < r.hi; i += kSelThreads) {
      const uint32_t key = weight_key(r.acc[i]);
      if (pass == 0 || (key >> (sh + 8)) == prefix) atomicAdd(&hist[(key >> sh) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      // lane i sums bins 255 - 8 i ... 248 - 8 i: lanes run from the largest keys down
      const int base = 255 - 8 * int(threadIdx.x);
      int sum = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) sum += hist[base - q];
      int inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (int(threadIdx.x) >= o) inc += y;
      }
      const int need = s_need;
      int above = inc - sum;
      __syncwarp();
      if (above < need && need <= inc) {
        int q = 0;
        while (above + hist[base - q] < need) above += hist[base - q++];
        s_prefix = (prefix << 8) | uint32_t(base - q);
        s_need = need - above;
      }
    }
    __syncthreads();
  }
  const uint32_t thr = s_prefix;
  const int need = s_need;  // tokens equal to thr that stay, the first ones
  int out = 0, ties = 0;
  for (int base = 0; base < r.L; base += kSelThreads) {
    const int i = base + threadIdx.x;
    const bool mid = i >= r.lo && i < r.hi;
    const float a = i < r.L ? r.acc[i] : 0.0f;
    const uint32_t key = weight_key(a);
    const bool tie = mid && r.k > 0 && key == thr;
    int tie_total;
    const int tie_at = ties + block_prefix(tie ? 1 : 0, buf, tie_total);
    const bool keep = i < r.L && (!mid || (r.k > 0 && (key > thr || (tie && tie_at < need))));
    int total;
    const int at = out + block_prefix(keep ? 1 : 0, buf, total);
    if (keep) {
      r.kept[at] = i;
      if (r.acc_out) r.acc_out[at] = a;
    }
    out += total;
    ties += tie_total;
  }
}

template <int D>
__global__ void __launch_bounds__(128) k_kv4_gather(const EvictParams p, const Kv4Map dst) {
  constexpr int NB = D / kKv4Block;
  __shared__ const uint8_t* s_src[16];
  __shared__ int s_row[16];
  const int bh = blockIdx.y, b = bh / p.map.Hkv, h = bh % p.map.Hkv, tile = blockIdx.x;
  const int n = min(kv4_len(p.map, b), p.budget);
  if (tile * kKv4Tile >= n) return;
  uint8_t* out8 = kv4_tile_ptr<D>(dst, b, h, tile);
  if (threadIdx.x < 16) {
    const int at = tile * kKv4Tile + threadIdx.x;
    const int j = at < n ? p.kept[int64_t(bh) * p.budget + at] : -1;
    s_src[threadIdx.x] = j >= 0 ? kv4_tile_ptr<D>(p.map, b, h, j / kKv4Tile) : nullptr;
    s_row[threadIdx.x] = j & 15;
  }
  __syncthreads();
  if (!out8) return;
  // A thread makes 16 bytes of K or of V: four blocks' words of one fragment lane, each
  // token's share picked from the same four words of its source tile.
  uint4* out = reinterpret_cast<uint4*>(out8);
  for (int i = threadIdx.x; i < D; i += 128) {
    const int q = (i % (D / 2)) / 32, ln = i & 31, g = ln >> 2, t = ln & 3;
    const bool is_v = i >= D / 2;
    const int parts = is_v ? 4 : 2;
    uint4 w[4];
    int sh[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int tok = is_v ? 2 * t + (x & 1) + (x & 2 ? 8 : 0) : g + 8 * (x & 1);
      const uint8_t* src = x < parts ? s_src[tok] : nullptr;
      const int r = s_row[tok];
      w[x] = make_uint4(0u, 0u, 0u, 0u);
      sh[x] = is_v ? 16 * (r >> 3) + 4 * (r & 1) : 8 * (r >> 3);
      if (src)
        w[x] = __ldg(reinterpret_cast<const uint4*>(src + (is_v ? 8 * D : 0)) + q * 32 +
                     (is_v ? g * 4 + ((r & 7) >> 1) : (r & 7) * 4 + t));
    }
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const uint32_t m = is_v ? 0x00000F0Fu : 0x00FF00FFu;
      const int to = is_v ? (x & 1) * 4 + (x & 2) * 8 : 8 * (x & 1);
      v.x |= (w[x].x >> sh[x] & m) << to;
      v.y |= (w[x].y >> sh[x] & m) << to;
      v.z |= (w[x].z >> sh[x] & m) << to;
      v.w |= (w[x].w >> sh[x] & m) << to;
    }
    out[i] = v;
  }
  for (int i = threadIdx.x; i < D; i += 128) {
    // scales byte by byte: K [g][block][half], V [t][block][token of the four]
    const int kt = i / (2 * NB) + 8 * (i & 1), kb = (i % (2 * NB)) >> 1;
    const uint8_t* src = s_src[kt];
    out8[16 * D + i] = src ? src[16 * D + (s_row[kt] & 7) * 2 * NB + 2 * kb + (s_row[kt] >> 3)] : uint8_t(0);
    const int q = i & 3, vb = (i >> 2) % NB, vt = 2 * (i / (4 * NB)) + (q & 1) + (q & 2 ? 8 : 0);
    src = s_src[vt];
    const int r = s_row[vt];
    out8[17 * D + i] =
        src ? src[17 * D + ((r & 7) >> 1) * 4 * NB + 4 * vb + (r >> 3) * 2 + (r & 1)] : uint8_t(0);
  }
}

}  // namespace

cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s) {
  EvictParams p{};
  p.map = kv4_map(a.kv);
  p.acc = a.acc;
  p.acc_ld = int64_t(a.kv.max_pages) * a.kv.page_tokens;
  p.budget = a.budget;
  p.n_sink = a.n_sink;
  p.n_recent = a.n_recent;
  p.dst_table = a.dst_table;
  p.dst_pages = a.dst_pages;
  p.new_lens = a.new_lens;
  p.kept = a.kept;
  p.acc_out = a.acc_out;
  p.acc_out_ld = int64_t(a.dst_pages) * a.kv.page_tokens;
  const int64_t max_tokens = p.acc_ld;
  const int heads = a.kv.B * a.kv.Hkv;
  cudaError_t e;
  if (max_tokens <= 4 * kSelThreads) {
    k_kv4_select<4><<<heads, kSelThreads, 4 * (4 * kSelThreads + kSelThreads) + 2 * 4 * kSelThreads, s>>>(p);
    e = cudaGetLastError();
  } else if (max_tokens <= 32 * kSelThreads) {
    constexpr int smem = 4 * (32 * kSelThreads + kSelThreads) + 2 * 32 * kSelThreads;
    e = cudaFuncSetAttribute(k_kv4_select<32>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    k_kv4_select<32><<<heads, kSelThreads, smem, s>>>(p);
    e = cudaGetLastError();
  } else {
    k_kv4_select_long<<<heads, kSelThreads, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  Kv4Map dst = p.map;
  dst.table = a.dst_table;
  dst.max_pages = a.dst_pages;
  const dim3 grid((a.budget + kKv4Tile - 1) / kKv4Tile, a.kv.B * a.kv.Hkv);
  if (a.kv.d == 128) k_kv4_gather<128><<<grid, 128, 0, s>>>(p, dst);
  else k_kv4_gather<64><<<grid, 128, 0, s>>>(p, dst);
  return cudaGetLastError();
}

}  // namespace attnq
