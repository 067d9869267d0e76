// tree.cuh -- what the drafted-tree attention kernels share: the parameters of a
// launch, a sequence's checked lengths, and the split of an fp32 pair into bf16
// terms.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace attn {

constexpr float kTreeC = kScale * kLog2e;  // scores in log2 units
constexpr float kTreeStale = 8.f;          // log2: how far a score may pass its row's reference maximum

struct TreeArgs {
  const float* q;            // [N][32][64]
  const void *k_pages, *v_pages;  // [num_pages][16][8][64]
  const int* table;          // [B][max_blocks]
  const int* ctx_lens;       // [B]
  const int* row_start;      // [B + 1]
  const long long* masks;    // [N], or nullptr: a chain (row i sees rows 0 .. i)
  float* out;                // [N][32][64]
  float* parts;              // [N][32][splits][64], then [N][32][splits][2] (log2 maximum, sum)
  int B, N, max_rows, max_blocks, num_pages, max_context, split_len, splits;
  unsigned* err;
  unsigned long long timeout_ns;
};

// One sequence of the batch, its lengths checked.
struct Seq {
  int ctx, first, rows, keys;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const TreeArgs& a, int b) {
  Seq s;
  s.ctx = __ldg(a.ctx_lens + b);
  s.first = __ldg(a.row_start + b);
  const int end = __ldg(a.row_start + b + 1);
  s.ok = true;
  const int room = min((long long)a.max_blocks * ATTN_PAGE, (long long)ATTN_MAX_TOKENS);
  if (s.ctx < 0 || s.ctx > a.max_context) {
    s.ok = false;
    s.ctx = s.ctx < 0 ? 0 : a.max_context;
  }
  if (s.first < 0 || end < s.first || end > a.N || (long long)end - s.first > a.max_rows) {
    s.ok = false;
    s.first = min(max(s.first, 0), a.N);
    s.rows = min(min(max(end, s.first), a.N) - s.first, a.max_rows);
  } else {
    s.rows = end - s.first;
  }
  if (s.ctx + s.rows > room) {
    s.ok = false;
    s.ctx = min(s.ctx, room);
  }
  s.keys = min(s.ctx + s.rows, room);
  return s;
}

// Three bf16 terms of a pair: two truncated, the last rounded to nearest: 24
// bits, all of an fp32 value whose last term does not underflow.
__device__ __forceinline__ void split3(float x, float y, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  t0 = tc::pack_bf16_trunc(x, y);
  float rx, ry;
  tc::fma2(rx, ry, tc::bf16_trunc(x), tc::bf16_trunc(y), -1.f, -1.f, x, y);  // exact
  t1 = tc::pack_bf16_trunc(rx, ry);
  tc::fma2(rx, ry, tc::bf16_trunc(rx), tc::bf16_trunc(ry), -1.f, -1.f, rx, ry);
  t2 = tc::pack_bf16_rn(rx, ry);
}

// ---- pieces of the tcgen05 kernels
constexpr float kUnseen = -3e38f;  // reference of a row that has seen no key: any score passes it

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// All softmax threads of the block meet; returns how many warps failed a wait,
// and in `over` how many saw a score that moves a reference. (A hardware
// barrier: it can hang only if a warp stays away, so none ever does. A warp
// whose wait failed still meets, and all leave together.)
__device__ __forceinline__ int meet(int threads, bool mine_over, bool failed, int lane, int* over) {
  int count;
  const int p = lane == 0 ? failed : mine_over;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.s32 p, %1, 0;\n\tbarrier.cta.red.popc.aligned.u32 %0, 1, %2, p;\n\t}"
      : "=r"(count)
      : "r"(p), "r"(threads)
      : "memory");
  *over = count / 31;
  return count % 31;
}
__device__ __forceinline__ void meet(int threads) {
  asm volatile("barrier.cta.sync.aligned 1, %0;" ::"r"(threads) : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

struct Wait {
  unsigned* err;
  unsigned long long timeout_ns;
  volatile int* abort_flag;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (true) {
#pragma unroll 1
      for (int i = 0; i < 32; ++i)
        if (tc::mbar_try_wait(bar, parity)) return true;
      if (*abort_flag) return false;
      if (tc::globaltimer_ns() - t0 > timeout_ns) {
        record_error(err, kDevErrTimeout);
        *abort_flag = 1;
        return false;
      }
    }
  }
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, (*this)(bar, parity));
  }
};

// A kernel of the family: drafted rows a block takes, threads, shared memory,
// resident blocks of an SM.
struct TreeVariant {
  void (*kernel)(CUtensorMap, CUtensorMap, TreeArgs);
  int tokens, threads;
  uint32_t smem;
  int blocks;
  bool v_atom32;  // fp32 V in the 128-byte swizzle of 32-byte chunks
  int regs;       // registers a thread at least at launch (what its register split adds up to)
};
TreeVariant tree_tc_variant(bool bf16, int which);  // 0, 1, 2: 4, 8, 16 drafted rows a block
TreeVariant tree_wide_variant(bool bf16);           // 32 drafted rows a block

}  // namespace attn
