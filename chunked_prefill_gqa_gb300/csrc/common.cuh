// common.cuh -- definitions shared by the CUDA translation units of
// libattnprefill.so: problem constants, the launch-parameter block, the
// device error word protocol and the host-side launcher declarations.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/attn_prefill.h"

namespace attn {

constexpr int kHQ = ATTN_HQ;            // query heads
constexpr int kHKV = ATTN_HKV;          // KV heads
constexpr int kGroup = kHQ / kHKV;      // query heads per KV head (4)
constexpr int kD = ATTN_D;              // head dimension
constexpr float kScale = 0.125f;        // 1 / sqrt(64), exact in fp32
constexpr float kLog2e = 1.4426950408889634f;

// Device error codes written into the error word (first writer wins).
constexpr unsigned kDevErrTimeout = 1u;
constexpr unsigned kDevErrBounds = 2u;

// Everything a kernel needs about one call.
struct Problem {
  const float* q;   // [C][32][64]
  const float* k;   // [P+C][8][64]
  const float* v;   // [P+C][8][64]
  float* out;       // [C][32][64]
  int C;            // chunk rows
  int P;            // cached prefix length
  unsigned* err;    // device error word
};

__device__ __forceinline__ void record_error(unsigned* err, unsigned code) {
  atomicCAS(err, 0u, code);
}

// Visible keys of chunk rows [t0, t0 + rows) clipped to the chunk: the unit's
// key range is [0, P + min(t0 + rows, C)).
__host__ __device__ __forceinline__ int unit_keys(int P, int C, int t0, int rows) {
  const int end = t0 + rows < C ? t0 + rows : C;
  return P + end;
}

// Host launchers, one per kernel family (defined in their own .cu files).
cudaError_t launch_reference(const Problem& p, cudaStream_t stream);
cudaError_t launch_ffma(const Problem& p, cudaStream_t stream);
int launch_tc(const Problem& p, cudaStream_t stream);             // returns an ATTN_* code
int launch_tc_fault_test(const Problem& p, cudaStream_t stream);  // skips a load, 20 ms waits
// Decode (decode.cu): how many split blocks the current device holds at once
// (first call per device sets the kernel up); split count and segment length
// for B sequences of at most max_context keys; workspace bytes for the
// partials; launch. The int results are ATTN_* codes.
int decode_slots(int* slots);
int decode_splits(int B, int max_context, int splits_hint, int slots, int* split_len);
size_t decode_workspace_bytes(int B, int splits);
// fault != 0 (failure-path test): the first tile of every block is never
// loaded and every wait is limited to 20 ms (2 s otherwise).
int launch_decode(const float* q, const float* k_pages, const float* v_pages, const int* table,
                  const int* ctx_lens, float* out, float* parts, int B, int max_blocks, int num_pages,
                  int max_context, int split_len, int splits, unsigned* err, cudaStream_t stream, int fault = 0);
// Three-kernel score-matrix attention (naive.cu): workspace bytes, the row
// limit of its grids, and one launcher per kernel.
size_t naive_workspace_bytes(int C, int P);
int naive_max_rows();
cudaError_t launch_naive_scores(const float* q, const float* k, float* S, int C, int P, cudaStream_t stream);
cudaError_t launch_naive_softmax(float* S, int C, int P, cudaStream_t stream);
cudaError_t launch_naive_weighted_sum(const float* S, const float* v, float* out, int C, int P,
                                      cudaStream_t stream);
// The fixed partials scratch of attn_decode_paged_noalloc (decode.cu) and its
// device address on the current device (looked up on the first call).
constexpr size_t kDecodeScratchBytes = size_t(4) << 20;
cudaError_t decode_scratch(float** ptr);
// BF16 K/V cache (tc_bf16.cu): p.k / p.v point at [P + C][8][64] bf16 caches.
int launch_tc_bf16(const Problem& p, cudaStream_t stream);
// fp32 K/V cache through the same kernel, K/V split into bf16 pairs in place.
int launch_tc_bf16x3(const Problem& p, cudaStream_t stream);
// Paged K/V: p.k / p.v point at [num_pages * 16][8][64] page pools.
int launch_tc_paged(const Problem& p, const int* table, int num_pages, cudaStream_t stream);

// A refused launch is reported by its own call: the runtime would also hand it to the
// next one that asks for the last error.
inline cudaError_t launched(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

#ifdef __CUDACC__
// A launch that may be prepared while the kernel before it in the stream still runs
// (programmatic dependent launch); every thread of the kernel calls follow() before it
// reads or writes anything that another launch may touch.
template <typename... P, typename... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, dim3 block, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}
// Waits for the grid before this one to end, its writes visible; and lets the next
// one be prepared.
__device__ __forceinline__ void follow() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}
// What such a kernel reads may be written while it is already there, up to follow():
// a plain load, which stays behind it, never one by the read-only path.
template <typename T>
__device__ __forceinline__ T fetch(const T* p) {
  return *p;
}
#endif

// Rows between the projections and attention (rows.cu): norm, rotation and the
// store into a contiguous destination (table == nullptr) or a paged cache.
struct RowCall {
  const void *q, *k, *v;  // q and v may be nullptr
  long long q_stride, k_stride, v_stride;
  int in_type, out_type;  // ATTN_F32 or ATTN_BF16: of q, k, v; of k_out, v_out
  const float *q_weight, *k_weight;
  float eps;
  const float* cos_sin;
  const int* positions;
  int num_positions, pairing;
  float* q_out;
  void *k_out, *v_out;
  const int *table, *ctx_lens, *row_start;
  int B, N, max_blocks, num_pages;
  // Several positions a row (num_axes > 0): axis x of row n at positions[x * pos_stride +
  // n], and the axis of frequency i in bits 2 i and 2 i + 1.
  int num_axes;
  long long pos_stride;
  unsigned long long axis_of;
};
cudaError_t launch_rows(const RowCall& c, unsigned* err, cudaStream_t stream);
cudaError_t launch_rope_table(const double* inv_freq, float* table, int num_positions, cudaStream_t stream);
cudaError_t launch_compact(void* k_pages, void* v_pages, int type, const int* table, const int* ctx_lens,
                           const int* keep, const int* counts, int B, int max_keep, int max_rows, int max_blocks,
                           int num_pages, unsigned* err, cudaStream_t stream);

// Attention of drafted rows over a paged cache (tree.cu): how a call is cut into
// key segments, the workspace of its partials, launch. int results are ATTN_* codes.
struct TreePlan {
  int variant;  // which kernel of the page type
  int splits, split_len;
  bool cluster;  // the segments of a unit are one cluster: no partials in memory
};
struct TreeCall {
  const float* q;
  const void *k_pages, *v_pages;
  int type;  // ATTN_F32 or ATTN_BF16 pages
  const int *table, *ctx_lens, *row_start;
  const long long* masks;
  float *out, *parts;
  int B, N, max_rows, max_blocks, num_pages, max_context;
  TreePlan plan;
  int withheld;  // failure test: segments whose first tile is never loaded, and every wait limited to 20 ms
};
// room: bytes of workspace that a choice of segments (splits_hint 0) may take.
int tree_plan(bool bf16, int B, int N, int max_rows, int max_context, int splits_hint, size_t room, TreePlan* plan);
size_t tree_workspace_bytes(int N, const TreePlan& plan);
int launch_tree(const TreeCall& c, unsigned* err, cudaStream_t stream);

// A decode step that also adds what each cached token was given to its weight
// (decode_weigh.cu): workspace bytes, launch.
struct DecodeWeighCall {
  const float* q;
  const void *k_pages, *v_pages;
  int type;  // ATTN_F32 or ATTN_BF16 pages
  float* weights;
  const int *table, *ctx_lens, *weighed_lens;  // weighed_lens may be nullptr
  float* out;
  void* workspace;
  int B, max_blocks, num_pages, max_context;
  float decay;
  int withheld;  // failure test: segments that never get their first keys, and every wait limited to 20 ms
};
int decode_weigh_workspace_bytes(int B, int max_context, size_t* bytes);
int launch_decode_weigh(const DecodeWeighCall& c, unsigned* err, cudaStream_t stream);

// The same weights from a window of rows, without their attention (weigh.cu).
struct WeighCall {
  const float* q;
  const void* k_pages;
  int type;
  float* weights;
  const int *table, *ctx_lens, *row_start, *weighed_lens;
  void* workspace;
  int B, N, max_rows, max_blocks, num_pages, max_context;
  float decay;
  int withheld;  // as above
};
int weigh_workspace_bytes(int B, int N, int max_rows, int max_context, size_t* bytes);
int launch_weigh(const WeighCall& c, unsigned* err, cudaStream_t stream);

// Tokens of least weight leave a cache (evict.cu).
struct EvictCall {
  void *k_pages, *v_pages;
  int type;
  float* weights;
  const int *table, *ctx_lens, *keep_lens;
  void* workspace;
  int B, max_blocks, num_pages, max_context, first, last;
};
size_t evict_workspace_bytes(int B, int max_context);
int launch_evict(const EvictCall& c, unsigned* err, cudaStream_t stream);

// Tensor-pipe rate measurement (peak.cu): `ctas` CTAs each issue `iters`
// dense M = 128, N = n MMAs (kind::tf32, or kind::f16 with bf16 operands).
int launch_tensor_peak(int bf16, int n, int iters, int ctas, unsigned* err, cudaStream_t stream);

}  // namespace attn
