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
  int cluster;               // the segments of a unit are one cluster and merge in shared memory
  unsigned* err;
  unsigned long long timeout_ns;
};

// A failure test's waits are limited to 20 ms, and by as many nanoseconds more as there
// are segments that never get their first tile. Its kernels are instantiations of their
// own (kFault), so that the others hold nothing of it.
constexpr unsigned long long kTimeoutNs = 2000000000ull, kFaultNs = 20000000ull;
template <bool kFault>
__device__ __forceinline__ bool withheld(const TreeArgs& a, int segment, int tile) {
  return kFault && tile == 0 && segment < (int)(a.timeout_ns - kFaultNs);
}

// One sequence of the batch, its lengths checked.
struct Seq {
  int ctx, first, rows, keys;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const TreeArgs& a, int b) {
  Seq s;
  s.ctx = fetch(a.ctx_lens + b);
  s.first = fetch(a.row_start + b);
  const int end = fetch(a.row_start + b + 1);
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

// Keys of a segment. Where the segments of a unit are one cluster, which holds its
// SMs until the last of them ends, a sequence's own keys are cut evenly (48
// sequences of 1 to 4096 tokens: five rows on bf16 pages 72 to 59 us, one row on
// fp32 pages 132 to 105); otherwise the call's length counts, and blocks past a
// short sequence's end leave at once. (So a call whose bound is far above its lengths
// and whose segments merge through memory leaves most of its blocks without keys.)
__device__ __forceinline__ int segment_len(const TreeArgs& a, const Seq& s) {
  if (!a.cluster) return a.split_len;
  return ((s.keys + a.splits - 1) / a.splits + 127) / 128 * 128;
}

// The first tf32 term of an fp32 operand, rounded to nearest: half the remainder of a
// truncation, and of either sign, so that what the products drop does not lean one
// way. A finite value that would round to infinity takes the largest tf32 number
// instead, with all of the rest in its second term, x - hi. (Of an infinity that rest
// is infinite, of a NaN NaN.)
__device__ __forceinline__ float tf32_near(float x) {
  float y;
  asm("min.xorsign.abs.f32 %0, %1, %2;"
      : "=f"(y)
      : "f"(__uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u)), "f"(__uint_as_float(0x7f7fe000u)));
  return y;
}

// Three bf16 terms of a pair, each rounded to nearest: 24 bits, all of an fp32
// value whose last term does not underflow. The remainders, exact, come from
// fused products of bf16 operands into fp32 (t * -1 + x), one instruction where
// unpacking the term first takes two. (For probabilities, which stay below 2^8: a
// value next to fp32's largest would round to infinity.)
__device__ __forceinline__ void split3(float x, float y, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  asm("{\n\t.reg .b16 l, h, m;\n\t.reg .f32 rx, ry;\n\t"
      "mov.b16 m, 0xBF80;\n\t"  // -1
      "cvt.rn.bf16x2.f32 %0, %4, %3;\n\tmov.b32 {l, h}, %0;\n\t"
      "fma.rn.f32.bf16 rx, l, m, %3;\n\tfma.rn.f32.bf16 ry, h, m, %4;\n\t"
      "cvt.rn.bf16x2.f32 %1, ry, rx;\n\tmov.b32 {l, h}, %1;\n\t"
      "fma.rn.f32.bf16 rx, l, m, rx;\n\tfma.rn.f32.bf16 ry, h, m, ry;\n\t"
      "cvt.rn.bf16x2.f32 %2, ry, rx;\n\t}"
      : "=&r"(t0), "=&r"(t1), "=r"(t2)
      : "f"(x), "f"(y));
}

// The same with the first terms cut off instead of rounded, one byte permutation for
// a conversion: the remainder is exact either way, the other two terms hold 16 bits
// of it, 24 in all, and every finite value has finite terms, as a query needs. (Also
// p of tree_wide, whose softmax is what takes the time: 16 rows of 16 sequences of
// 16384 tokens 131 to 128 us.)
__device__ __forceinline__ void split3_cut(float x, float y, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
  asm("{\n\t.reg .b16 l, h, m;\n\t.reg .f32 rx, ry;\n\t"
      "mov.b16 m, 0xBF80;\n\t"  // -1
      "prmt.b32 %0, %5, %6, 0x7632;\n\tmov.b32 {l, h}, %0;\n\t"
      "fma.rn.f32.bf16 rx, l, m, %3;\n\tfma.rn.f32.bf16 ry, h, m, %4;\n\t"
      "cvt.rn.bf16x2.f32 %1, ry, rx;\n\tmov.b32 {l, h}, %1;\n\t"
      "fma.rn.f32.bf16 rx, l, m, rx;\n\tfma.rn.f32.bf16 ry, h, m, ry;\n\t"
      "cvt.rn.bf16x2.f32 %2, ry, rx;\n\t}"
      : "=&r"(t0), "=&r"(t1), "=r"(t2)
      : "f"(x), "f"(y), "r"(__float_as_uint(x)), "r"(__float_as_uint(y)));
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

// Waits up to timeout_ns, or until another warp of the block has given up. A block in
// which a wait ran out winds down: every warp leaves its loop at its next wait, all of
// them meet, and only then, with the abort flag final, do the warps that started
// copies and products wait for those still in flight. (One that looked earlier could
// have started its last and left while another warp still waited for it.)
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

// The segments of a unit as one cluster of blocks, up to kMaxCluster of them:
// each leaves its rows ([4 nrows][stride], 64 used) and their (log2 maximum, sum)
// in its own shared memory, and after a barrier of the cluster every block merges
// and writes its share of the rows. No partial goes through memory, and no second
// kernel waits for the first. Every block of a cluster comes here, also one
// without keys or with a failed wait (its sums are then empty): none may leave
// while another reads its shared memory. Called by the first `threads` threads
// of every block; the others have left.
constexpr int kMaxCluster = 8;

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

__device__ __forceinline__ void cluster_merge(const TreeArgs& a, int first_row, int nrows, int head,
                                              const float* rows, int stride, const float2* ml, int tid,
                                              int threads) {
  __syncwarp();
  tc::cluster_sync_all();
  // A thread an element (4 dims of a row), all segments' loads on their way at once,
  // a warp's from one block's shared memory each. (A lane a segment, in pieces of 64
  // bytes a block, took 17.2 us where this takes 12.7: 32 drafted rows, 1000 tokens,
  // eight segments; 9.4 and 9.0 with 8 rows.)
  const int elements = nrows * kGroup * 16;
  for (int e = blockIdx.x * threads + tid; e < elements; e += a.splits * threads) {
    const int r = e >> 4, d = (e & 15) * 4;
    float2 p[kMaxCluster];
    float4 y[kMaxCluster];
    float m = -INFINITY;
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      p[s] = make_float2(-INFINITY, 0.f);
      if (s < a.splits) {
        p[s] = ld_cluster2(tc::mapa_shared(tc::smem_u32(ml + r), s));
        y[s] = ld_cluster4(tc::mapa_shared(tc::smem_u32(rows + r * stride + d), s));
      }
      m = fmaxf(m, p[s].x);
    }
    float den = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int s = 0; s < kMaxCluster; ++s) {
      const float w = p[s].x == -INFINITY ? 0.f : ex2(p[s].x - m);
      den = fmaf(w, p[s].y, den);
      if (w != 0.f)  // an empty segment's rows have no weight, whatever they hold
        x = make_float4(fmaf(w, y[s].x, x.x), fmaf(w, y[s].y, x.y), fmaf(w, y[s].z, x.z), fmaf(w, y[s].w, x.w));
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;  // no key: zeros
    *reinterpret_cast<float4*>(a.out + ((size_t)(first_row + (r >> 2)) * kHQ + head * kGroup + (r & 3)) * kD + d) =
        make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  }
  __syncwarp();
  tc::cluster_sync_all();
}

// Waits for the copies of the last `stages` of `issued` tiles to land.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int issued, uint64_t timeout_ns) {
#pragma unroll 1
  for (int i = max(0, issued - stages); i < issued; ++i) tc::mbar_wait(&full[i % stages], (i / stages) & 1, timeout_ns);
}
// Waits for every product the warp has issued; the whole warp comes here.
__device__ __forceinline__ void drain_products(uint64_t* bar, uint64_t timeout_ns) {
  if (elect()) {
    tc::mma_commit(bar);
    tc::mbar_wait(bar, 0, timeout_ns);
  }
  __syncwarp();
}

// A kernel of the family: drafted rows a block takes, threads, shared memory,
// resident blocks of an SM; and in the time of 128 keys, what a block costs besides
// its keys and what the second kernel does that merges segments through memory.
struct TreeVariant {
  void (*kernel)(CUtensorMap, CUtensorMap, TreeArgs);
  void (*fault)(CUtensorMap, CUtensorMap, TreeArgs);  // the failure test's
  int tokens, threads;
  uint32_t smem;
  int blocks;
  bool v_atom32;  // fp32 V in the 128-byte swizzle of 32-byte chunks
  int regs;       // registers a thread at least at launch (what its register split adds up to)
  int fixed, merge;
};
TreeVariant tree_tc_variant(int tokens);   // bf16 pages, 4 or 8 drafted rows a block
TreeVariant tree_wide_variant(bool bf16);  // 32 drafted rows a block

}  // namespace attn
