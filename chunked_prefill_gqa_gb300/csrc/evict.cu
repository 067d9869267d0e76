// evict.cu -- tokens of least weight leave a paged cache, per key/value head.
//
// Of a sequence's ctx tokens new = min(ctx, keep) stay. The first `first` and the last
// `last` of them stay whatever their weight; of the middle those m = new - first - last
// with the largest weights, the lower token among equal ones. The key rows carry their
// rotation, and attention does not go by their order, so nothing but the gaps has to
// close: with edge = new - last,
//   the i-th middle token below edge that leaves   <- the i-th middle one from edge on that stays
//   tokens edge .. new - 1                         <- tokens ctx - last .. ctx - 1, in their order
// (both lists rising; they are as long as each other, since m middle tokens stay and edge
// - first = m places are below edge). A cache cut from n to n / 2 tokens so moves about n /
// 4 rows a head instead of n / 2 kept in order.
//
// Two launches. select_kernel: a cluster of blocks per (sequence, head) finds the m-th
// largest weight by its digits (11, 11 and 10 bits of the weights mapped to ordered
// integers, a histogram in shared memory, the cluster's added up through distributed
// shared memory), then walks its tokens once more and writes both lists. move_kernel moves
// the rows: sources at or past new are written by nobody, so those go in any order; what
// lies between edge and new is read (as sources of holes) before one block per (sequence,
// head) writes the last ones there, batch by batch.
#include <cstdint>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPerThread = kBins / kThreads;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 40960;  // tokens of a block whose keys stay in shared memory (160 KB)

struct EvictArgs {
  void *k_pages, *v_pages;
  float* weights;             // [num_pages][8][16]
  const int *table, *ctx_lens, *keep_lens;
  int *counts, *holes, *movers;  // [B][8]; [B][8][cap] each
  int B, max_blocks, num_pages, max_context, first, last, cap, cached;
  unsigned* err;
};

// A sequence's lengths: what stays, and where the last tokens go. live: something leaves.
struct Cut {
  int ctx, now, edge, end;  // tokens before and after; places of the last ones; end of the middle
  bool ok, live;
};
__device__ __forceinline__ Cut load_cut(const EvictArgs& a, int b) {
  Cut c;
  c.ctx = fetch(a.ctx_lens + b);
  const int keep = fetch(a.keep_lens + b);
  c.ok = c.ctx >= 0 && c.ctx <= a.max_context && (long long)c.ctx <= (long long)a.max_blocks * ATTN_PAGE && keep >= 0;
  c.live = c.ok && keep < c.ctx;
  if (c.live && (long long)a.first + a.last > keep) c.ok = c.live = false;
  c.now = c.live ? keep : c.ctx;
  c.edge = c.now - a.last;
  c.end = c.ctx - a.last;
  return c;
}

// Weights as integers of the same order: NaN lowest, both zeros equal.
__device__ __forceinline__ uint32_t ordered(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : u & 0x80000000u ? ~u : u | 0x80000000u;
}

struct Shared {
  uint32_t hist[2][kBins];
  uint32_t warp_sums[kWarps];
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t totals[4];  // this block's: above, equal, and both below edge
  uint32_t bin, need;
  int bad;
};

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::mapa_shared(tc::smem_u32(p), rank)) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a) {
  extern __shared__ uint32_t cache[];
  __shared__ Shared sh;
  follow();
  const int rank = blockIdx.x, ranks = gridDim.x, head = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Cut cut = load_cut(a, b);
  int* const count = a.counts + b * kHKV + head;
  if (!cut.live) {  // for every block of the cluster
    if (rank == 0 && tid == 0) {
      if (!cut.ok) record_error(a.err, kDevErrBounds);
      *count = -1;
    }
    return;
  }
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  // This block's tokens: whole pages, the sequence's own length cut evenly.
  const int span = ((cut.ctx + ATTN_PAGE - 1) / ATTN_PAGE + ranks - 1) / ranks * ATTN_PAGE;
  const int t0 = min((long long)rank * span, (long long)cut.ctx), t1 = min((long long)t0 + span, (long long)cut.ctx);
  if (tid == 0) sh.bad = 0;
  for (int i = tid; i < kBins; i += kThreads) sh.hist[0][i] = 0;
  __syncthreads();
  auto key_of = [&](int t) -> uint32_t {
    const int page = fetch(trow + t / ATTN_PAGE);
    if (page < 0 || page >= a.num_pages) {
      sh.bad = 1;
      return 0;
    }
    return ordered(fetch(a.weights + ((size_t)page * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE));
  };
  if (a.cached)
    for (int t = t0 + tid; t < t1; t += kThreads) cache[t - t0] = key_of(t);
  const auto key_at = [&](int t) -> uint32_t { return a.cached ? cache[t - t0] : key_of(t); };
  const int lo = max(t0, a.first), hi = min(t1, cut.end);  // the middle's part of them
  const uint32_t m = cut.now - a.first - a.last;

  // The m-th largest key, digit by digit from the top.
  uint32_t prefix = 0, need = m;
  int shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3 && m > 0; ++pass) {
    const int bits = pass == 2 ? 10 : 11, above = shift;
    shift -= bits;
    uint32_t* const hist = sh.hist[pass & 1];
    __syncthreads();
    for (int t = lo + tid; t - lane < hi; t += kThreads) {
      uint32_t key = 0;
      bool in = t < hi;
      if (in) {
        key = key_at(t);
        in = pass == 0 || key >> above == prefix;
      }
      const uint32_t digit = key >> shift & ((1u << bits) - 1);
      // Equal digits of a whole warp (weights of zero, above all) count at once.
      const unsigned some = __ballot_sync(kFull, in);
      if (!some) continue;
      const uint32_t one = __shfl_sync(kFull, digit, __ffs(some) - 1);
      if (__ballot_sync(kFull, in && digit == one) == some) {
        if (lane == 0) atomicAdd(hist + one, __popc(some));
      } else if (in) {
        atomicAdd(hist + digit, 1u);
      }
    }
    if (ranks > 1) tc::cluster_sync_all();
    else __syncthreads();
    // Thread i owns bins kBins - 1 - 4 i and the three below: counts from the top.
    uint32_t n[kPerThread], sum = 0;
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      const uint32_t* at = hist + (kBins - 1 - (tid * kPerThread + j));
      n[j] = ranks > 1 ? 0 : *at;
      if (ranks > 1)
        for (int r = 0; r < ranks; ++r) n[j] += ld_cluster(at, r);
      sum += n[j];
    }
    uint32_t up = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t x = __shfl_up_sync(kFull, up, off);
      if (lane >= off) up += x;
    }
    if (lane == 31) sh.warp_sums[warp] = up;
    for (int i = tid; i < kBins; i += kThreads) sh.hist[(pass + 1) & 1][i] = 0;  // read by nobody since the last meeting
    __syncthreads();
    uint32_t before = up - sum;
    for (int w = 0; w < warp; ++w) before += sh.warp_sums[w];
#pragma unroll
    for (int j = 0; j < kPerThread; ++j) {
      if (before < need && need <= before + n[j]) {
        sh.bin = kBins - 1 - (tid * kPerThread + j);
        sh.need = need - before;
      }
      before += n[j];
    }
    __syncthreads();
    prefix = prefix << bits | sh.bin;
    need = sh.need;
  }
  // Stays: key > top, or one of the first `need` equal to it.
  const uint32_t top = m > 0 ? prefix : kFull;

  // A warp's tokens are consecutive, so that ranks follow from counts.
  const int per = ((max(hi - lo, 0) + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int w0 = lo + warp * per, w1 = min(w0 + per, hi);
  uint32_t gt = 0, eq = 0, gt_in = 0, eq_in = 0;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint32_t key = t < w1 ? key_at(t) : 0;
    const bool g = t < w1 && key > top, e = t < w1 && key == top;
    gt += __popc(__ballot_sync(kFull, g));
    eq += __popc(__ballot_sync(kFull, e));
    gt_in += __popc(__ballot_sync(kFull, g && t < cut.edge));
    eq_in += __popc(__ballot_sync(kFull, e && t < cut.edge));
  }
  if (!a.cached)  // the pages of what stays in any case count too
    for (int t = t0 + tid; t < t1; t += kThreads)
      if (t < lo || t >= hi) key_of(t);
  if (tid < 4) sh.totals[tid] = 0;
  __syncthreads();
  if (lane == 0) {
    sh.warp_gt[warp] = gt;
    sh.warp_eq[warp] = eq;
    atomicAdd(sh.totals + 0, gt);
    atomicAdd(sh.totals + 1, eq);
    atomicAdd(sh.totals + 2, gt_in);
    atomicAdd(sh.totals + 3, eq_in);
  }
  if (ranks > 1) tc::cluster_sync_all();
  else __syncthreads();
  uint32_t gt_before = 0, eq_before = 0, in_gt = 0, in_eq = 0;
  int bad = 0;
  for (int r = 0; r < ranks; ++r) {
    if (r < rank) {
      gt_before += ld_cluster(sh.totals + 0, r);
      eq_before += ld_cluster(sh.totals + 1, r);
    }
    in_gt += ld_cluster(sh.totals + 2, r);
    in_eq += ld_cluster(sh.totals + 3, r);
    bad |= (int)ld_cluster(reinterpret_cast<const uint32_t*>(&sh.bad), r);
  }
  if (ranks > 1) tc::cluster_sync_all();  // nobody's shared memory is read past here
  if (bad) {  // of every block of every head of the sequence
    if (rank == 0 && tid == 0) {
      record_error(a.err, kDevErrBounds);
      *count = -1;
    }
    return;
  }
  const uint32_t kept_in = in_gt + min(in_eq, need);  // middle tokens that stay below edge
  if (rank == 0 && tid == 0) *count = (int)(m - kept_in);
  for (int w = 0; w < warp; ++w) gt_before += sh.warp_gt[w], eq_before += sh.warp_eq[w];
  const size_t base = ((size_t)b * kHKV + head) * a.cap;
  const unsigned below = (1u << lane) - 1;
  for (int t = w0 + lane; t - lane < w1; t += 32) {
    const uint32_t key = t < w1 ? key_at(t) : 0;
    const bool g = t < w1 && key > top, e = t < w1 && key == top;
    const unsigned gs = __ballot_sync(kFull, g), es = __ballot_sync(kFull, e);
    const uint32_t g_rank = gt_before + __popc(gs & below), e_rank = eq_before + __popc(es & below);
    if (t < w1) {
      const uint32_t kept_before = g_rank + min(e_rank, need);
      const bool stays = g || (e && e_rank < need);
      if (t < cut.edge && !stays) a.holes[base + (t - a.first) - kept_before] = t;
      if (t >= cut.edge && stays) a.movers[base + kept_before - kept_in] = t;
    }
    gt_before += __popc(gs);
    eq_before += __popc(es);
  }
}

// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 128, kMoveWarps = kMoveThreads / 32;

// kVecs: 16-byte words of a head's row (8 or 16).
template <int kVecs>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a) {
  follow();
  const int head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31;
  const int pairs = fetch(a.counts + b * kHKV + head);
  if (pairs < 0) return;
  const Cut cut = load_cut(a, b);
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  const size_t base = ((size_t)b * kHKV + head) * a.cap;
  uint4* const kp = static_cast<uint4*>(a.k_pages);
  uint4* const vp = static_cast<uint4*>(a.v_pages);
  // The row of the pool, in heads' rows, that holds token t of this head; and its weight.
  const auto row_of = [&](int t) { return (fetch(trow + t / ATTN_PAGE) * ATTN_PAGE + t % ATTN_PAGE) * kHKV + head; };
  const auto weight_of = [&](int t) {
    return a.weights + ((size_t)fetch(trow + t / ATTN_PAGE) * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE;
  };
  // A warp moves 32 pairs: a lane looks one up, then the rows go several at once.
  constexpr int kAtOnce = 32 / kVecs;  // rows of one pool that a warp's load covers
  const auto fill = [&](int i, bool near) {
    int src = 0, dst = 0;
    bool in = i + lane < pairs;
    if (in) {
      const int from = fetch(a.movers + base + i + lane);
      in = (from < cut.now) == near;
      if (in) {
        const int to = fetch(a.holes + base + i + lane);
        src = row_of(from), dst = row_of(to);
        *weight_of(to) = *weight_of(from);
      }
    }
    const unsigned some = __ballot_sync(kFull, in);
    if (!some) return;
    constexpr int kUnroll = 4;
#pragma unroll 1
    for (int p = 0; p < 32; p += kAtOnce * kUnroll) {
      uint4 x[kUnroll], y[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kAtOnce + lane / kVecs;
        const int s = __shfl_sync(kFull, src, q);
        if (some >> q & 1) {
          x[u] = kp[(size_t)s * kVecs + lane % kVecs];
          y[u] = vp[(size_t)s * kVecs + lane % kVecs];
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kAtOnce + lane / kVecs;
        const int d = __shfl_sync(kFull, dst, q);
        if (some >> q & 1) {
          kp[(size_t)d * kVecs + lane % kVecs] = x[u];
          vp[(size_t)d * kVecs + lane % kVecs] = y[u];
        }
      }
    }
  };
  if (blockIdx.x > 0) {
    for (int i = ((blockIdx.x - 1) * kMoveWarps + (tid >> 5)) * 32; i < pairs; i += (gridDim.x - 1) * kMoveThreads) fill(i, false);
    return;
  }
  // What leaves the places of the last ones, then those: in rising batches, each read
  // before it is written (a source is never below its destination).
  for (int i = (tid >> 5) * 32; i < pairs && i <= a.last; i += kMoveThreads) fill(i, true);
  const int shift = cut.ctx - cut.now;
  constexpr int kRows = 4 * kMoveThreads / kVecs;  // of a batch
  for (int i0 = 0; i0 < a.last; i0 += kRows) {
    uint4 x[4], y[4];
    float w = 0.f;
    const bool weigh = tid < kRows && i0 + tid < a.last;
    if (weigh) w = *weight_of(cut.edge + shift + i0 + tid);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + (tid + u * kMoveThreads) / kVecs;
      if (i < a.last) {
        const size_t s = (size_t)row_of(cut.edge + shift + i) * kVecs + tid % kVecs;
        x[u] = kp[s];
        y[u] = vp[s];
      }
    }
    __syncthreads();
    if (weigh) *weight_of(cut.edge + i0 + tid) = w;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + (tid + u * kMoveThreads) / kVecs;
      if (i < a.last) {
        const size_t d = (size_t)row_of(cut.edge + i) * kVecs + tid % kVecs;
        kp[d] = x[u];
        vp[d] = y[u];
      }
    }
    __syncthreads();
  }
}

int list_cap(int max_context) { return max_context / 2 + 1; }

}  // namespace

size_t evict_workspace_bytes(int B, int max_context) {
  return ((size_t)B * kHKV * sizeof(int) + 15) / 16 * 16 + 2 * (size_t)B * kHKV * list_cap(max_context) * sizeof(int);
}

cudaError_t launch_evict(const EvictCall& c, int sms, unsigned* err, cudaStream_t stream) {
  EvictArgs a{};
  a.k_pages = c.k_pages;
  a.v_pages = c.v_pages;
  a.weights = c.weights;
  a.table = c.table;
  a.ctx_lens = c.ctx_lens;
  a.keep_lens = c.keep_lens;
  a.B = c.B;
  a.max_blocks = c.max_blocks;
  a.num_pages = c.num_pages;
  a.max_context = c.max_context;
  a.first = c.first;
  a.last = c.last;
  a.cap = list_cap(c.max_context);
  a.counts = static_cast<int*>(c.workspace);
  a.holes = a.counts + ((size_t)c.B * kHKV + 3) / 4 * 4;
  a.movers = a.holes + (size_t)c.B * kHKV * a.cap;
  a.err = err;

  // Blocks of a cluster: as many as have a place on two blocks an SM, with 1024 tokens each
  // at least; and so many that a block's keys fit its shared memory, if they can.
  int ranks = 1;
  while (ranks < kMaxCluster && ((long long)c.B * kHKV * 2 * ranks <= 2 * sms ? c.max_context / (2 * ranks) >= 1024
                                                                              : c.max_context / ranks > kMaxCached))
    ranks *= 2;
  const int span = ((c.max_context + ATTN_PAGE - 1) / ATTN_PAGE + ranks - 1) / ranks * ATTN_PAGE;
  a.cached = span <= kMaxCached;
  const size_t smem = a.cached ? (size_t)span * sizeof(uint32_t) : 0;
  if (smem > 24576) {  // past 48 KB with the block's own
    const cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCached * 4);
    if (e != cudaSuccess) return launched(e);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, kHKV, c.B);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = launched(cudaLaunchKernelEx(&cfg, select_kernel, a));
  if (e != cudaSuccess) return e;
  // Blocks for the pairs: one for 128 of them, at most 32 resident rounds of all SMs.
  const long long most = 32LL * 16 * sms / ((long long)c.B * kHKV);
  long long blocks = (a.cap + kMoveThreads - 1) / kMoveThreads;
  if (blocks > most) blocks = most < 1 ? 1 : most;
  const dim3 grid((unsigned)blocks + 1, kHKV, c.B);
  return launch_following(c.type == ATTN_BF16 ? move_kernel<8> : move_kernel<16>, grid, dim3(kMoveThreads), stream, a);
}

}  // namespace attn
