// What the two attention kernels over the 4-bit KV cache share: their arguments,
// the way their work is dealt to CTAs, and the join of rows that several CTAs had.
#pragma once

#include <cuda_bf16.h>

#include <atomic>

#include "kv4.cuh"

namespace attnq {

constexpr int kKv4PlanSms = 152;  // SMs the grids are planned for (the workspace size is asked for without a device)
constexpr uint64_t kKv4DrainNs = 1000000000ull;  // bound on waiting for copies in flight after a timeout

struct Kv4AttnParams {
  Kv4Map map;
  Kv4Rows Q, O;
  int q_bf16, o_bf16;
  int G;
  int causal;
  const int8_t* signs;
  const float* k_scale;
  const float* v_scale;
  float inv_sqrt_d;
  float scale_log2e;
  float* lse;      // ln of the rows' sums, or null
  float* lse2;     // log2 of them for the weights (as ln they would be rounded twice more), null without weights
  int64_t lse_sb, lse_sh;
  int n_cta;       // CTAs the chunks are dealt to
  int ov;          // what beginning a segment costs, in chunks
  int cl, n_rg;    // cl > 0: a cluster of cl CTAs a segment instead of the line; row groups of T rows
  float* part_o;   // [CTA][2][R][D]: sums of the CTA's first and last segment
  float2* part_ml; // [CTA][2][R]: their maxima and row sums
  int4* part_seg;  // [CTA]: the segment that begins in this CTA and ends in a later one
  const float* acc_in;
  float* acc_out;
  int64_t acc_ld;
  float4* scores;  // every score of the call, [b, h][tile][8 rows][lane], or null
  uint64_t wait_ns;
};

// A block of 16 channels of a query row, as loaded: 32 bytes of bf16 or 64 of fp32.
struct Kv4Raw16 {
  uint4 w[4];
};
__device__ __forceinline__ Kv4Raw16 kv4_query_row(const Kv4AttnParams& p, int b, int h, int n, int row, bool wanted,
                                                  int blk) {
  Kv4Raw16 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = make_uint4(0u, 0u, 0u, 0u);
  if (wanted && row < n * p.G) {
    const int64_t off = b * p.Q.sb + int64_t(h * p.G + row % p.G) * p.Q.sh + int64_t(row / p.G) * p.Q.st + blk * 16;
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.Q.ptr) + off * (p.q_bf16 ? 2 : 4));
    r.w[0] = __ldg(src);
    r.w[1] = __ldg(src + 1);
    if (!p.q_bf16) {
      r.w[2] = __ldg(src + 2);
      r.w[3] = __ldg(src + 3);
    }
  }
  return r;
}
__device__ __forceinline__ void kv4_unpack16(const Kv4Raw16& r, bool bf16, float (&x)[16]) {
  const uint32_t w[16] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w,
                          r.w[2].x, r.w[2].y, r.w[2].z, r.w[2].w, r.w[3].x, r.w[3].y, r.w[3].z, r.w[3].w};
  if (bf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i]);
  }
}
// Rotates the row (on d / 16 neighbouring lanes) and returns 2^(14 - e) for 2^e <= its largest magnitude <
// 2^(e + 1); norm = 2^(e - 14), the exponent held to what both powers can express.  The row's largest
// element then lies in [2^14, 2^15), as high as fp16 lets it: a bf16 element is exact down to 2^-31 of it (its
// last bit at fp16's last, 2^-24) and off by at most 2^-39 of it below.  (With the largest in [1, 2) elements
// lost bits from 2^-17 on.)  The raw scores stay below 2^15 * 2688 * 128 < 2^34.
template <int D>
__device__ __forceinline__ float kv4_normalise16(const Kv4AttnParams& p, float (&x)[16], int blk, float& norm) {
  if (p.signs) kv4_rotate16<D>(x, p.signs, blk, p.inv_sqrt_d);
  uint32_t am = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) am = max(am, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int o = 1; o < D / kKv4Block; o *= 2) am = max(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (am >= 0x7F800000u && blk == 0) atomicOr(p.map.status, DEV_NONFINITE);
  const int e14 = max(int(am >> 23) - 127 - 14, -126);
  norm = __uint_as_float(uint32_t(127 + e14) << 23);
  return __uint_as_float(uint32_t(127 - e14) << 23);
}

// Work is counted in chunks of C tokens of a segment (sequence, KV head, group of R rows),
// segments in that order.  All chunks of the call form one line, and CTA i takes the
// i-th of n_cta equal pieces, so the load is even however ragged the lengths are.
// The lengths are read here, on the device.  A segment has the chunks that some row
// of its group sees (one at least: rows that see nothing are still written), and on the
// line p.ov more behind them, which nobody works on: a CTA that crosses from one segment
// into the next loads queries and joins warps twice, and gets that much less to do.
// R = kKv4AllRows: one group of all rows, which sees every token.
constexpr int kKv4AllRows = 0;
template <int R, int C>
struct Kv4Line {
  int64_t at, end, per;  // this CTA's chunks of the line, and a full piece
  int b, h, rg, L, n, groups;
  int vis;               // tokens that some row of the group sees
  int real, chunks, c0;  // chunks of the segment, places it has on the line, and the first that is this CTA's

  static __device__ __forceinline__ int groups_of(const Kv4AttnParams& p, int n) {
    return R == kKv4AllRows ? 1 : (n * p.G + R - 1) / R;
  }
  static __device__ __forceinline__ int vis_of(const Kv4AttnParams& p, int L, int n, int rg) {
    if (R == kKv4AllRows) return L;
    const int t_last = min((rg * R + R - 1) / p.G, n - 1);
    return p.causal ? min(max(L - n + t_last + 1, 0), L) : L;
  }
  static __device__ __forceinline__ int real_of(int vis) { return max(1, (vis + C - 1) / C); }
  static __device__ __forceinline__ int chunks_of(const Kv4AttnParams& p, int vis) { return real_of(vis) + p.ov; }
  // Chunks of one KV head of a sequence.
  static __device__ __forceinline__ int64_t head_work(const Kv4AttnParams& p, int L, int n) {
    const int groups = groups_of(p, n);
    if (!p.causal) return int64_t(groups) * chunks_of(p, L);
    int64_t sum = 0;
    for (int rg = 0; rg < groups; ++rg) sum += chunks_of(p, vis_of(p, L, n, rg));
    return sum;
  }

  __device__ __forceinline__ void load_seq(const Kv4AttnParams& p) {
    L = kv4_len(p.map, b);
    n = kv4_new(p.map, b);
    groups = groups_of(p, n);
  }
  __device__ __forceinline__ void load_seg(const Kv4AttnParams& p) {
    vis = vis_of(p, L, n, rg);
    real = real_of(vis);
    chunks = real + p.ov;
  }

  // Run by the whole block (WARPS warps): where this CTA's piece begins.  False: it has none.
  template <int WARPS>
  __device__ __forceinline__ bool begin(const Kv4AttnParams& p, int cta, int least) {
    __shared__ int64_t s_warp[WARPS];
    __shared__ int64_t s_before;
    __shared__ int s_b;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int each = (p.map.B + WARPS * 32 - 1) / (WARPS * 32);
    const int b0 = min(int(threadIdx.x) * each, p.map.B), b1 = min(b0 + each, p.map.B);
    int64_t sum = 0;
    for (int i = b0; i < b1; ++i) sum += head_work(p, kv4_len(p.map, i), kv4_new(p.map, i)) * p.map.Hkv;
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) base += s_warp[w];
      total += s_warp[w];
    }
    per = max((total + p.n_cta - 1) / p.n_cta, int64_t(least));
    at = cta * per;
    end = min(at + per, total);
    int64_t before = base + inc - sum;  // chunks before sequence b0
    if (at >= before && at < before + sum)
      for (int i = b0; i < b1; ++i) {
        const int64_t w = head_work(p, kv4_len(p.map, i), kv4_new(p.map, i)) * p.map.Hkv;
        if (at >= before && at < before + w) {
          s_b = i;
          s_before = before;
        }
        before += w;
      }
    __syncthreads();
    if (at >= end) return false;
    b = s_b;
    load_seq(p);
    const int64_t work = max(head_work(p, L, n), int64_t(1));
    int64_t rem = at - s_before;
    h = int(rem / work);
    rem %= work;
    if (!p.causal) {
      rg = int(rem / chunks_of(p, L));
      rem %= chunks_of(p, L);
      load_seg(p);
    } else {
      for (rg = 0; load_seg(p), rem >= chunks && rg < groups; ++rg) rem -= chunks;
    }
    c0 = int(rem);
    return h < p.map.Hkv && rg < groups;
  }

  // The segment of this CTA's cluster, and this CTA's share of its chunks.  False: it has no rows.
  __device__ __forceinline__ bool begin_cluster(const Kv4AttnParams& p, int cta, int& c1) {
    const int seg = cta / p.cl, rank = cta % p.cl;
    rg = seg % p.n_rg;
    h = (seg / p.n_rg) % p.map.Hkv;
    b = seg / (p.n_rg * p.map.Hkv);
    load_seq(p);
    if (rg >= groups) return false;
    load_seg(p);
    c0 = real * rank / p.cl;
    c1 = real * (rank + 1) / p.cl;
    return true;
  }

  // Chunks of the current segment up to c1 are done: the next segment, or false.
  __device__ __forceinline__ bool next(const Kv4AttnParams& p, int c1) {
    at += c1 - c0;
    c0 = 0;
    if (at >= end) return false;
    if (++rg == groups) {
      rg = 0;
      if (++h == p.map.Hkv) {
        h = 0;
        do {
          if (++b >= p.map.B) return false;
          load_seq(p);
        } while (groups == 0);
      }
    }
    load_seg(p);
    return true;
  }
  // The end of the current segment's places on the line that are this CTA's.
  __device__ __forceinline__ int last_chunk() const { return int(min(int64_t(chunks), c0 + (end - at))); }
  // Only the empty places of the current segment are this CTA's: nothing to do or to write.
  __device__ __forceinline__ bool nothing() const { return c0 >= real; }
  // No other CTA has a part of the current segment, of which this one has up to c1.
  __device__ __forceinline__ bool entire(int c1) const { return c0 == 0 && c1 >= real; }
  // What the join has to know of the segment that ends at c1: y < 0 for one
  // that does not begin here and end later; else slot, (b, h), group, parts.
  __device__ __forceinline__ int4 record(const Kv4AttnParams& p, int c1, int slot) const {
    if (c0 != 0 || c1 >= real) return make_int4(0, -1, 0, 0);
    return make_int4(slot, b * p.map.Hkv + h, rg, int(1 + (real - c1 + per - 1) / per));
  }
};

// The log-sum of a row of maximum mx (log2 units) and sum l, which holds 2^p_bits; -infinity when it saw no token.
__device__ __forceinline__ void kv4_write_lse(const Kv4AttnParams& p, int64_t at, float mx, float l, float p_bits) {
  if (!p.lse && !p.lse2) return;
  const float l2 = l > 0.0f ? mx + (log2f(l) - p_bits) : -INFINITY;
  if (p.lse) p.lse[at] = l2 * 0.69314718055994531f;
  if (p.lse2) p.lse2[at] = l2;
}

// Row `row` of (b, h): O = g_v x / l (0 when the row saw no token) and lse.
template <int D>
__device__ __forceinline__ void kv4_write_row(const Kv4AttnParams& p, int b, int h, int row, int lane, float mx, float l,
                                              const float (&x)[D / 32], float p_bits) {
  constexpr int E = D / 32;
  const float gv = p.v_scale ? p.v_scale[h] : 1.0f;
  const float inv = l > 0.0f ? __fdiv_rn(gv, l) : 0.0f;
  const int t = row / p.G, head = h * p.G + row % p.G;
  uint8_t* dst = static_cast<uint8_t*>(const_cast<void*>(p.O.ptr)) +
                 (b * p.O.sb + head * p.O.sh + t * p.O.st) * (p.o_bf16 ? 2 : 4);
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    if (p.o_bf16)
      reinterpret_cast<__nv_bfloat162*>(dst)[(lane * E + e) / 2] = __floats2bfloat162_rn(x[e] * inv, x[e + 1] * inv);
    else
      reinterpret_cast<float2*>(dst)[(lane * E + e) / 2] = make_float2(x[e] * inv, x[e + 1] * inv);
  }
  if (lane == 0) kv4_write_lse(p, b * p.lse_sb + head * p.lse_sh + t, mx, l, p_bits);
}

// Joins the parts of a segment that several CTAs had, in their order: block
// (CTA, rows) looks after the segment that begins in that CTA.  A warp takes a row.
template <int D, int R>
__global__ void __launch_bounds__(128) k_kv4_join(const Kv4AttnParams p, float p_bits) {
  constexpr int E = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x / (R / 4), r = blockIdx.x % (R / 4) * 4 + warp;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 seg = p.part_seg[cta];
  if (seg.y < 0) return;
  const int b = seg.y / p.map.Hkv, h = seg.y % p.map.Hkv, n = kv4_new(p.map, b);
  const int row = seg.z * R + r;
  if (row >= n * p.G) return;
  float mx = -INFINITY, l = 0.0f, x[E] = {};
  // the first part is in its CTA's slot seg.x, the others in the first slots of theirs
  auto part = [&](int i) { return (int64_t(cta + i) * 2 + (i == 0 ? seg.x : 0)) * R + r; };
  // 32 parts at a time, a lane to each part's maximum and sum, and the parts' rows
  // eight loads at a time: one after another their latencies add up (30 us for 32 parts)
  for (int i = 0; i < seg.w; i += 32) {
    const int parts = min(seg.w - i, 32);
    const float2 ml = lane < parts ? p.part_ml[part(i + lane)] : make_float2(-INFINITY, 0.0f);
    float mc = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) mc = fmaxf(mc, __shfl_xor_sync(0xffffffffu, mc, o));
    if (mc == -INFINITY) continue;
    const float mnew = fmaxf(mx, mc), alpha = ex2(mx - mnew);
    mx = mnew;
    const float f = ml.x == -INFINITY ? 0.0f : ex2(ml.x - mx);
    float ls = ml.y * f;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) ls += __shfl_xor_sync(0xffffffffu, ls, o);
    l = fmaf(l, alpha, ls);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= alpha;
    for (int k = 0; k < parts; k += 8) {
      float y[8][E];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float* src = p.part_o + part(i + min(k + q, parts - 1)) * D + lane * E;
        if constexpr (E == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          y[q][0] = v.x;
          y[q][1] = v.y;
          y[q][2] = v.z;
          y[q][3] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          y[q][0] = v.x;
          y[q][1] = v.y;
        }
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float fq = __shfl_sync(0xffffffffu, f, k + q);  // 0 from the lanes past the last part
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = fmaf(y[q][e], fq, x[e]);
      }
    }
  }
  kv4_write_row<D>(p, b, h, row, lane, mx, l, x, p_bits);
}

// Launch with programmatic stream serialisation: the kernel may start while the
// one before it drains, and waits for it with griddepcontrol.wait, in every CTA and on every
// way out: what comes next in the stream waits for this grid alone.
template <typename... Args>
cudaError_t kv4_launch_after(void (*kern)(Args...), dim3 grid, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Launch with clusters of `cl` CTAs.
template <typename... Args>
cudaError_t kv4_launch_cluster(void (*kern)(Args...), dim3 grid, int cl, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = unsigned(cl);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The tcgen05 kernel for many query rows (256 to a segment), and its join.
cudaError_t launch_kv4_prefill(const Kv4AttnParams& p, int d, bool two_terms, cudaStream_t s);
constexpr int kKv4PrefillRows = 256;

// Bounded wait; a limit of 0 means not to wait at all.
__device__ __forceinline__ bool kv4_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_test_wait(bar, parity)) return true;
  return limit_ns && mbar_wait(bar, parity, limit_ns);
}

// Lets `kern` use `bytes` of dynamic shared memory.  `done` belongs to the kernel (a static of
// the caller): a bit per device on which this has been set, since the call costs a microsecond
// and the kernel keeps the setting.
inline cudaError_t kv4_allow_smem(const void* kern, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (done.load(std::memory_order_relaxed) >> dev & 1u) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return e;
}

inline size_t kv4_a256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace attnq
