// Launchers shared between the kernel translation units and the C-ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace attnq {

// ---- prepare -------------------------------------------------------------
// Tokens per scale tile of the per-tile Q/K scales (tiles aligned at token 0).
constexpr int kScaleTile = 128;

struct PrepareArgs {
  int B, Hq, Hkv, N, d;
  int P;              // tokens the mean key and the slice scales are taken over (1..N)
  int bf16;           // input element type: 1 bf16, 0 fp32
  int rotate, center, vt;
  int tiles;          // per-tile Q/K scales
  int i8;             // Q and K as INT8 codes held in bf16 (V stays E4M3)
  const int8_t* signs;
  const void* Q;
  const void* K;
  const void* V;
  uint8_t* q8;
  uint8_t* k8;
  uint8_t* v8;
  float* q_ds;
  float* k_ds;
  float* v_ds;
  float* k_mean;      // optional
  int64_t ldv;        // row length of transposed V
  // workspace carve-up
  uint32_t* amax_bits;  // [nslices]
  uint32_t* a_done;     // [nslices] warp-tiles whose amax is in amax_bits
  uint32_t* m_done;     // [B*Hkv] mean-key chunks summed
  uint32_t* mu_ready;   // [B*Hkv] mean key published
  uint32_t* ctl;        // [4] ticket, abort, number of entries
  uint32_t* entries;    // [3*nslices] work list: kind << 30 | slice
  float* mean_part;     // [B*Hkv*nchunks*d]
  float* mu;            // [B*Hkv*d]
  uint32_t* status;
  int num_sms;
  uint64_t wait_ns;
};

size_t prepare_workspace_bytes(int B, int Hq, int Hkv, int N, int d, int center);
// Size of the fixed scratch array behind attnq_prepare_static (ATTNQ_STATIC_SCRATCH_BYTES).
constexpr size_t kStaticScratchBytes = size_t(4) << 20;
// Device address of that array on the current device (looked up once per device).
cudaError_t static_scratch_address(void** out);
void carve_prepare_workspace(PrepareArgs& a, void* ws);
cudaError_t launch_prepare(const PrepareArgs& a, cudaStream_t s);

// ---- attention forward (tcgen05) -----------------------------------------
struct FwdArgs {
  int B, Hq, Hkv, N, d, T;
  int causal, reverse;
  int rotate;
  int tiles;          // per-tile Q/K scales
  int i8;             // q8, k8: INT8 codes held in bf16 (S = Q K^T as kind::f16)
  float S;
  const uint8_t* q8;
  const uint8_t* k8;
  const uint8_t* v8t;
  int64_t ldv;
  const float* q_ds;
  const float* k_ds;
  const float* v_ds;
  void* O;
  int out_bf16;
  unsigned long long* underflow;
  int k_sink;
  uint32_t* status;
  uint64_t wait_ns;
  int num_sms;
};
cudaError_t launch_fwd(const FwdArgs& a, cudaStream_t s);

// ---- P-only forward (SIMT fp32) -------------------------------------------
struct PonlyArgs {
  int B, Hq, Hkv, N, d, T;
  int causal, reverse;
  float S;
  const float* Q;
  const float* K;
  const float* V;
  float* O;
  unsigned long long* underflow;
  int k_sink;
};
cudaError_t launch_ponly(const PonlyArgs& a, cudaStream_t s);

// ---- per-head error ----------------------------------------------------------
struct ErrArgs {
  int n_heads;
  int64_t per_head;
  const void* O;
  int o_bf16;
  const double* O_ref;
  double* err;
};
cudaError_t launch_err(const ErrArgs& a, cudaStream_t s);

// ---- FP64 reference attention ----------------------------------------------
struct RefArgs {
  int B, Hq, Hkv, N, d;
  int bf16, causal;
  const void* Q;
  const void* K;
  const void* V;
  double* O_ref;
};
cudaError_t launch_ref_attn(const RefArgs& a, cudaStream_t s);

// ---- 4-bit paged KV cache --------------------------------------------------
struct Kv4Args {
  int num_pages, page_tokens, Hkv, d;
  const int8_t* signs;    // null: no rotation
  const float* k_scale;   // [Hkv] or null (1)
  const float* v_scale;
  uint8_t* pages;
  int B, max_pages;
  const int32_t* table;
  const int32_t* lens;
  const int32_t* new_lens;  // null: T of every sequence
  int T;
  uint32_t* status;
  uint64_t wait_ns;
};
// Rows of d contiguous elements at ptr + (b * sb + h * sh + t * st) elements.
struct Kv4Rows {
  const void* ptr;
  int64_t sb, sh, st;
};
cudaError_t launch_kv4_append(const Kv4Args& a, const Kv4Rows& K, const Kv4Rows& V, int bf16, const float* k_mean,
                              cudaStream_t s);
cudaError_t launch_kv4_read(const Kv4Args& a, const Kv4Rows& K, const Kv4Rows& V, int bf16, cudaStream_t s);

struct Kv4AttnArgs {
  Kv4Args kv;
  int Hq;
  Kv4Rows Q, O;
  int q_bf16, o_bf16;
  float scale;
  int causal;
  float* lse;            // [B, Hq, T] or null
  const float* acc_in;   // [B, Hkv, max_pages * page_tokens] or null (zeros)
  float* acc_out;        // null: no weights
  void* ws;
  size_t ws_bytes;
};
size_t kv4_attn_workspace_bytes(int B, int max_pages, int page_tokens, int Hq, int Hkv, int T, int d, bool with_scores);
cudaError_t launch_kv4_attn(const Kv4AttnArgs& a, cudaStream_t s);

struct Kv4EvictArgs {
  Kv4Args kv;
  const float* acc;      // [B, Hkv, max_pages * page_tokens]
  int budget, n_sink, n_recent;
  const int32_t* dst_table;  // [B, dst_pages]
  int dst_pages;
  int32_t* new_lens;     // [B]
  int32_t* kept;         // [B, Hkv, budget]
  float* acc_out;        // [B, Hkv, dst_pages * page_tokens] or null
};
cudaError_t launch_kv4_evict(const Kv4EvictArgs& a, cudaStream_t s);

// ---- driver entry point for tensor maps ------------------------------------
CUresult encode_tiled_3d(CUtensorMap* map, const void* base, uint64_t dim0, uint64_t dim1, uint64_t dim2,
                         uint64_t stride1_bytes, uint64_t stride2_bytes, uint32_t box0, uint32_t box1,
                         CUtensorMapSwizzle swizzle);

}  // namespace attnq
