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
// Up to kSmall tokens a block does both steps from registers and shared memory, in one launch
// (small_kernel). Longer contexts take two. select_kernel: a cluster of blocks per (sequence,
// head) finds the m-th largest weight by its digits (12, 10 and 10 bits of the weights mapped to
// ordered integers, a histogram in shared memory, the cluster's added up through distributed
// shared memory), then walks its tokens once more and writes both lists. move_kernel moves the
// rows: sources at or past new are written by nobody, so those go in any order; what lies between
// edge and new is read (as sources of holes) before one block per (sequence, head) writes the
// last ones there, batch by batch.
//
// Bound by the moves' latency and bytes: 16 sequences of 16384 tokens to half (bf16 pages) read and
// write 287 MB in 80 us, the copy that restores their weights among them: select 21, move 50 (their
// floor 43 together). Rows of 128 bytes at random places move at 5.5 TB/s.
#include <cstddef>
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
// Digits of 12, 10 and 10 bits: with three bits of the fraction in the first one, the weights of
// a warp (within a few powers of two) seldom meet in a bin.
constexpr int kBins = 4096, kFirst = 20, kDigit = 10;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 40960;  // tokens of a block whose keys stay in shared memory: 160 KB of its 227, with Shared's 57
struct EvictArgs {
  void *k_pages, *v_pages;
  float* weights;             // [num_pages][8][16]
  const int *table, *ctx_lens, *keep_lens;
  int2* counts;               // [B][8]: pairs of a hole and its mover (-1: nothing to do); those whose mover lies below new
  int *holes, *movers;        // [B][8][cap] each: slots of the pool, page * 16 + slot
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

constexpr int kListed = 2048;  // keys of the first digit's bin that a block keeps apart

template <int kThreads>
struct alignas(16) Shared {  // the keys follow
  static constexpr int kWarps = kThreads / 32;
  uint32_t hist[2][kBins];     // these two in vectors of 16 bytes
  uint32_t slice[kBins / 2];   // the cluster's counts of this block's share of the bins
  uint32_t in_slice[3];        // and their sum, in each pass
  uint32_t keys[kListed], places[kListed];  // and their tokens, from the block's first on
  uint32_t listed;
  uint32_t warp_sums[kWarps];
  uint32_t warp_gt[kWarps], warp_eq[kWarps];
  uint32_t totals[8];  // this block's keys above and equal to the m-th: all, below edge, below new; bad
  uint32_t others[kMaxCluster][8];      // the cluster's
  uint32_t bin, need, whole;
  int bad;
};

__device__ __forceinline__ uint32_t ld_cluster(const uint32_t* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::mapa_shared(tc::smem_u32(p), rank)) : "memory");
  return v;
}

__device__ __forceinline__ uint4 ld_cluster4u(const uint32_t* p, int rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(tc::mapa_shared(tc::smem_u32(p), rank)) : "memory");
  return v;
}

// The lowest n of a quad's four bits.
__device__ __forceinline__ uint32_t lowest(int n) { return (1u << min(max(n, 0), 4)) - 1; }

// Of four bits, how many are set up to each, in a byte each (the last one: in all). POPC would
// take four times as long.
__device__ __forceinline__ uint32_t running(uint32_t bits) { return ((bits * 0x00204081u) & 0x01010101u) * 0x01010101u; }

// The bin of a digit that holds the cluster's need-th key from the top, how many of the bin's
// are needed, and whether that is all of them. Zeroes the other histogram, which nobody has
// read since the last meeting. A cluster's blocks add up a share of the bins each, and then look at
// the one share that the key is in. (Every block adding up all: eight times the distant reads, one
// sequence of 20000 tokens 51 us for the call, 27 this way.)
template <int kThreads>
__device__ __forceinline__ void choose(Shared<kThreads>& sh, int ranks, int rank, int pass, uint32_t need) {
  constexpr int kWarps = kThreads / 32, kPerThread = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* const hist = sh.hist[pass & 1];
  uint32_t n[kPerThread] = {}, sum = 0, passed = 0;
  int base = 0, per = kPerThread, low = kBins - kPerThread * (tid + 1);  // this thread's bins, from low on; the last thread's are the lowest
  if (ranks > 1) {
    tc::cluster_sync_all();
    const int share = kBins / ranks;  // block r has bins share * r and on
    if (4 * tid < share) {
      uint4 all = make_uint4(0, 0, 0, 0);
      for (int r = 0; r < ranks; ++r) {
        const uint4 x = ld_cluster4u(hist + rank * share + 4 * tid, r);
        all.x += x.x, all.y += x.y, all.z += x.z, all.w += x.w;
      }
      *reinterpret_cast<uint4*>(sh.slice + 4 * tid) = all;
      atomicAdd(sh.in_slice + pass, all.x + all.y + all.z + all.w);
    }
    __syncwarp();
    tc::cluster_sync_all();
    int owner = ranks - 1;
    for (; owner > 0; --owner) {
      const uint32_t in = ld_cluster(sh.in_slice + pass, owner);
      if (need <= passed + in) break;
      passed += in;
    }
    per = share >= kThreads ? share / kThreads : 1;
    low = share - per * (tid + 1);
    base = share * owner;
#pragma unroll
    for (int j = 0; j < kPerThread / 2; ++j)
      if (j < per && low >= 0) n[j] = ld_cluster(sh.slice + low + j, owner);
  } else {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPerThread; j += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(hist + low + j);
      n[j] = x.x, n[j + 1] = x.y, n[j + 2] = x.z, n[j + 3] = x.w;
    }
  }
#pragma unroll
  for (int j = 0; j < kPerThread; ++j) sum += n[j];
  uint32_t up = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(kFull, up, off);
    if (lane >= off) up += x;
  }
  if (lane == 31) sh.warp_sums[warp] = up;
#pragma unroll
  for (int i = 0; i < kBins / 4; i += kThreads)
    reinterpret_cast<uint4*>(sh.hist[(pass + 1) & 1])[i + tid] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  uint32_t before = passed + up - sum;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += w < warp ? sh.warp_sums[w] : 0;
#pragma unroll
  for (int j = kPerThread - 1; j >= 0; --j) {
    if (before < need && need <= before + n[j]) {
      sh.bin = base + low + j;
      sh.need = need - before;
      sh.whole = need == before + n[j];
    }
    before += n[j];
  }
  __syncthreads();
}

// Four tokens' keys, a quarter of a page, are looked at together. (16 sequences of 16384 tokens:
// 20 us; 32 with every digit counted over all keys, 250 instructions for each 32 of them.)
template <int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(const EvictArgs a) {
  constexpr int kWarps = kThreads / 32, kPerThread = kBins / kThreads;
  extern __shared__ __align__(16) uint8_t select_smem[];
  Shared<kThreads>& sh = *reinterpret_cast<Shared<kThreads>*>(select_smem);
  uint4* const cache = reinterpret_cast<uint4*>(select_smem + sizeof(Shared<kThreads>));  // the keys, if they fit
  const int rank = blockIdx.x, ranks = gridDim.x, head = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins / 4; i += kThreads) reinterpret_cast<uint4*>(sh.hist[0])[i] = make_uint4(0, 0, 0, 0);
  if (tid < 8) sh.totals[tid] = 0;
  if (tid < 3) sh.in_slice[tid] = 0;
  if (tid == 0) sh.bad = 0, sh.listed = 0;
  follow();
  const Cut cut = load_cut(a, b);
  int2* const count = a.counts + b * kHKV + head;
  if (!cut.live) {  // for every block of the cluster
    if (rank == 0 && tid == 0) {
      if (!cut.ok) record_error(a.err, kDevErrBounds);
      *count = make_int2(-1, 0);
    }
    return;
  }
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  // This block's tokens: whole pages, the sequence's own length cut evenly.
  const int span = ((cut.ctx + ATTN_PAGE - 1) / ATTN_PAGE + ranks - 1) / ranks * ATTN_PAGE;
  const int t0 = min((long long)rank * span, (long long)cut.ctx), t1 = min((long long)t0 + span, (long long)cut.ctx);
  const int quads = (t1 - t0 + 3) / 4;
  const int lo = max(t0, a.first), hi = min(t1, cut.end);  // the middle's part of the tokens
  const uint32_t m = cut.now - a.first - a.last;
  __syncthreads();
  const auto page_of = [&](int quad) {
    const int page = fetch(trow + (t0 + 4 * quad) / ATTN_PAGE);
    if (page >= 0 && page < a.num_pages) return page;
    sh.bad = 1;
    return -1;
  };
  const auto keys_at = [&](int quad, int page) {  // slots past the last token of a page may hold anything
    if (page < 0) return make_uint4(0, 0, 0, 0);
    const float4 w = fetch(reinterpret_cast<const float4*>(a.weights + ((size_t)page * kHKV + head) * ATTN_PAGE) + (t0 / 4 + quad) % 4);
    return make_uint4(ordered(w.x), ordered(w.y), ordered(w.z), ordered(w.w));
  };
  const auto quad_at = [&](int quad) -> uint4 {
    return a.cached ? cache[quad] : keys_at(quad, page_of(quad));
  };
  const auto middle = [&](int t) { return lowest(hi - t) & ~lowest(lo - t); };  // of a quad's tokens
  // Of a quad, the keys above and equal to a border.
  const auto above_equal = [&](uint4 k, int t, uint32_t border, uint32_t* g, uint32_t* e) {
    const uint32_t in = middle(t);
    *g = in & ((uint32_t)(k.x > border) | (uint32_t)(k.y > border) << 1 | (uint32_t)(k.z > border) << 2 | (uint32_t)(k.w > border) << 3);
    *e = in & ((uint32_t)(k.x == border) | (uint32_t)(k.y == border) << 1 | (uint32_t)(k.z == border) << 2 | (uint32_t)(k.w == border) << 3);
  };
  // All keys once, with the first digit's histogram; several quads' lookups on their way at once.
  constexpr int kAhead = 4;
  for (int q0 = tid; q0 < quads; q0 += kAhead * kThreads) {
    int page[kAhead];
    uint4 key[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) page[i] = q0 + i * kThreads < quads ? page_of(q0 + i * kThreads) : -1;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) key[i] = keys_at(q0 + i * kThreads, page[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int q = q0 + i * kThreads, t = t0 + 4 * q;
      if (q >= quads) break;
      if (a.cached) cache[q] = key[i];
      const uint32_t in = middle(t);
      if (in & 1) atomicAdd(sh.hist[0] + (key[i].x >> kFirst), 1u);
      if (in & 2) atomicAdd(sh.hist[0] + (key[i].y >> kFirst), 1u);
      if (in & 4) atomicAdd(sh.hist[0] + (key[i].z >> kFirst), 1u);
      if (in & 8) atomicAdd(sh.hist[0] + (key[i].w >> kFirst), 1u);
    }
  }

  // Stays: key > top, or one of the first `need` equal to it. A warp's quads are consecutive, so
  // that ranks follow from counts.
  uint32_t top = kFull, need = 0;
  const int per = (quads + 32 * kWarps - 1) / (32 * kWarps) * 32;
  const int w0 = min(warp * per, quads), w1 = min(w0 + per, quads);
  uint32_t c[6] = {};  // as totals, of this thread
  const auto tally = [&](int i, uint32_t bits, int t) {  // of tokens t .. t + 3, to c[i], c[i + 2] and c[i + 4]
    const uint32_t n = running(bits) >> 24;
    c[i] += n;
    c[i + 2] += t + 4 <= cut.edge ? n : t >= cut.edge ? 0 : running(bits & lowest(cut.edge - t)) >> 24;
    c[i + 4] += t + 4 <= cut.now ? n : t >= cut.now ? 0 : running(bits & lowest(cut.now - t)) >> 24;
  };
  bool listed = false;
  if (m > 0) {
    choose<kThreads>(sh, ranks, rank, 0, m);
    uint32_t prefix = sh.bin;
    need = sh.need;
    // Keys above the bin are counted, those in it (a few in a hundred) listed: the other
    // digits and what goes by them look at the list alone, if it holds them all.
    for (int q = w0 + lane; q < w1; q += 32) {
      const uint4 key = quad_at(q);
      const int t = t0 + 4 * q;
      uint32_t g, e;
      above_equal(make_uint4(key.x >> kFirst, key.y >> kFirst, key.z >> kFirst, key.w >> kFirst), t, prefix, &g, &e);
      tally(0, g, t);
      while (e) {
        const int j = __ffs(e) - 1;
        e &= e - 1;
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kListed) sh.keys[at] = j == 0 ? key.x : j == 1 ? key.y : j == 2 ? key.z : key.w, sh.places[at] = t + j - t0;
      }
    }
    uint32_t gt = __reduce_add_sync(kFull, c[0]);
    if (lane == 0) sh.warp_gt[warp] = gt, sh.warp_eq[warp] = 0;
    bool whole = sh.whole;
    __syncthreads();
    listed = sh.listed <= kListed;
    const int entries = sh.listed;
    int shift = kFirst;
#pragma unroll 1
    for (int pass = 1; pass < 3 && !whole; ++pass) {
      const int above = shift;
      shift -= kDigit;
      const auto count_digit = [&](uint32_t key, bool in) {
        if (in && key >> above == prefix) atomicAdd(sh.hist[pass & 1] + (key >> shift & ((1u << kDigit) - 1)), 1u);
      };
      if (listed) {
        for (int i = tid; i < entries; i += kThreads) count_digit(sh.keys[i], true);
      } else {
        for (int q = tid; q < quads; q += kThreads) {
          const uint4 key = quad_at(q);
          const uint32_t in = middle(t0 + 4 * q);
          count_digit(key.x, in & 1);
          count_digit(key.y, in & 2);
          count_digit(key.z, in & 4);
          count_digit(key.w, in & 8);
        }
      }
      choose<kThreads>(sh, ranks, rank, pass, need);
      prefix = prefix << kDigit | sh.bin;
      need = sh.need;
      whole = sh.whole;
    }
    // Where all of the last bin stay (never all tokens: prefix is not 0 then) any above its border do.
    top = prefix << shift;
    if (whole) --top, need = 0;
    if (listed) {
      for (int i = tid; i < entries; i += kThreads) {
        const int place = sh.places[i];
        const uint32_t g = sh.keys[i] > top, e = sh.keys[i] == top;
        tally(0, g, t0 + place);
        tally(1, e, t0 + place);
        if (g) atomicAdd(&sh.warp_gt[place / 4 / per], 1u);
        if (e) atomicAdd(&sh.warp_eq[place / 4 / per], 1u);
      }
    }
  }
  if (!listed) {
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = 0;
    for (int q = w0 + lane; q < w1; q += 32) {
      uint32_t g, e;
      above_equal(quad_at(q), t0 + 4 * q, top, &g, &e);
      tally(0, g, t0 + 4 * q);
      tally(1, e, t0 + 4 * q);
    }
    const uint32_t gt = __reduce_add_sync(kFull, c[0]), eq = __reduce_add_sync(kFull, c[1]);
    if (lane == 0) sh.warp_gt[warp] = gt, sh.warp_eq[warp] = eq;
  }
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const uint32_t sum = __reduce_add_sync(kFull, c[i]);
    if (lane == i && sum) atomicAdd(sh.totals + i, sum);
  }
  __syncthreads();
  if (tid == 0) sh.totals[6] = sh.bad;
  if (ranks > 1) tc::cluster_sync_all();
  else __syncthreads();
  if (tid < 8 * ranks) sh.others[tid >> 3][tid & 7] = ld_cluster(sh.totals + (tid & 7), tid >> 3);
  if (ranks > 1) {
    __syncwarp();
    tc::cluster_arrive();  // nobody's shared memory is read past here
  }
  __syncthreads();
  uint32_t gt_before = 0, eq_before = 0, in_gt = 0, in_eq = 0, now_gt = 0, now_eq = 0;
  int bad = 0;
  for (int r = 0; r < ranks; ++r) {
    const uint32_t* const x = sh.others[r];
    if (r < rank) gt_before += x[0], eq_before += x[1];
    in_gt += x[2], in_eq += x[3], now_gt += x[4], now_eq += x[5];
    bad |= (int)x[6];
  }
  const uint32_t kept_in = in_gt + min(in_eq, need);  // middle tokens that stay below edge
  if (rank == 0 && tid == 0) {
    if (bad) record_error(a.err, kDevErrBounds);
    *count = bad ? make_int2(-1, 0) : make_int2((int)(m - kept_in), (int)(now_gt + min(now_eq, need) - kept_in));
  }
  if (!bad) {  // else of every block of every head of the sequence
#pragma unroll
    for (int w = 0; w < kWarps; ++w) gt_before += w < warp ? sh.warp_gt[w] : 0, eq_before += w < warp ? sh.warp_eq[w] : 0;
    const size_t base = ((size_t)b * kHKV + head) * a.cap;
    int page = w0 + lane < w1 ? fetch(trow + (t0 + 4 * (w0 + lane)) / ATTN_PAGE) : 0;
    for (int q = w0 + lane; q - lane < w1; q += 32) {
      const int t = t0 + 4 * q, slot = page * ATTN_PAGE + t % ATTN_PAGE;
      if (q + 32 < w1) page = fetch(trow + (t + 128) / ATTN_PAGE);
      uint32_t g = 0, e = 0, in = 0;
      if (q < w1) {
        above_equal(quad_at(q), t, top, &g, &e);
        in = middle(t);
      }
      // Keys above in the upper half, equal ones (few, as a rule none) in the lower.
      const uint32_t eqs = running(e), own = (running(g) >> 24) << 16 | eqs >> 24;
      uint32_t up = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, up, off);
        if (lane >= off) up += x;
      }
      const uint32_t all = __shfl_sync(kFull, up, 31);
      const uint32_t g_rank = gt_before + ((up - own) >> 16), e_rank = eq_before + ((up - own) & 0xffffu);
      uint32_t stays = g;
      if (e)  // the first `need` of them
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((e >> j & 1) && e_rank + (eqs >> 8 * j & 255u) <= need) stays |= 1u << j;
      const uint32_t kept_before = g_rank + min(e_rank, need), kept = running(stays) << 8;  // up to each token, without it
      const uint32_t ahead = lowest(cut.edge - t), out = in & ~stays & ahead, move = stays & ~ahead;
      int* const hole = a.holes + base + (t - a.first) - (int)kept_before;
      int* const mover = a.movers + base + (int)(kept_before - kept_in);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = kept >> 8 * j & 255u;
        if (out >> j & 1) hole[j - n] = slot + j;
        if (move >> j & 1) mover[n] = slot + j;
      }
      gt_before += all >> 16;
      eq_before += all & 0xffffu;
    }
  }
  if (ranks > 1) {
    __syncwarp();
    tc::cluster_wait();
  }
}

// ---------------------------------------------------------------------------
// Where a head's rows and weights lie. A slot is page * 16 + its place there.
template <int kVecs>  // 16-byte words of a head's row (8 or 16)
struct Rows {
  uint4 *k, *v;
  float* weights;
  const int* trow;
  int head;
  __device__ __forceinline__ Rows(const EvictArgs& a, int b, int h)
      : k(static_cast<uint4*>(a.k_pages)), v(static_cast<uint4*>(a.v_pages)), weights(a.weights),
        trow(a.table + (size_t)b * a.max_blocks), head(h) {}
  __device__ __forceinline__ int slot(int t) const { return fetch(trow + t / ATTN_PAGE) * ATTN_PAGE + t % ATTN_PAGE; }
  __device__ __forceinline__ size_t row(int slot) const { return ((size_t)slot * kHKV + head) * kVecs; }
  __device__ __forceinline__ float* weight(int slot) const {
    return weights + ((size_t)(slot / ATTN_PAGE) * kHKV + head) * ATTN_PAGE + slot % ATTN_PAGE;
  }

  // A warp moves the pairs i .. i + kMost - 1 below end: a lane looks one up, then the rows go, all
  // of kStep pairs at once.
  static constexpr int kAtOnce = 32 / kVecs, kUnroll = 4, kStep = kAtOnce * kUnroll;  // kAtOnce: rows that a warp's load covers
  template <int kMost>
  __device__ __forceinline__ void fill(const int* holes, const int* movers, int i, int end, int lane) const {
    int src = 0, dst = 0;
    if (lane < kMost && i + lane < end) {
      src = fetch(movers + i + lane);
      dst = fetch(holes + i + lane);
      *weight(dst) = *weight(src);
    }
    const int pairs = min(end - i, kMost);
#pragma unroll 1
    for (int p = 0; p < pairs; p += kStep) {
      uint4 x[kUnroll], y[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kAtOnce + lane / kVecs;
        const size_t s = row(__shfl_sync(kFull, src, q)) + lane % kVecs;
        if (q < pairs) x[u] = k[s], y[u] = v[s];
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int q = p + u * kAtOnce + lane / kVecs;
        const size_t d = row(__shfl_sync(kFull, dst, q)) + lane % kVecs;
        if (q < pairs) k[d] = x[u], v[d] = y[u];
      }
    }
  }

  // A block moves the last tokens to their places, in rising batches, each read before it is
  // written (a source is never below its destination). What leaves those places has left them
  // by the first batch's barrier.
  template <int kThreads>
  __device__ __forceinline__ void follow_up(const Cut& cut, int last, int tid) const {
    const int shift = cut.ctx - cut.now;
    constexpr int kRows = 4 * kThreads / kVecs;  // of a batch
    for (int i0 = 0; i0 < last; i0 += kRows) {
      uint4 x[4], y[4];
      float w = 0.f;
      const bool weigh = tid < kRows && i0 + tid < last;
      if (weigh) w = *weight(slot(cut.edge + shift + i0 + tid));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + (tid + u * kThreads) / kVecs;
        if (i < last) {
          const size_t s = row(slot(cut.edge + shift + i)) + tid % kVecs;
          x[u] = k[s], y[u] = v[s];
        }
      }
      __syncthreads();
      if (weigh) *weight(slot(cut.edge + i0 + tid)) = w;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + (tid + u * kThreads) / kVecs;
        if (i < last) {
          const size_t d = row(slot(cut.edge + i)) + tid % kVecs;
          k[d] = x[u], v[d] = y[u];
        }
      }
      __syncthreads();
    }
  }
};

constexpr int kMoveThreads = 128, kMoveWarps = kMoveThreads / 32;

template <int kVecs>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const EvictArgs a) {
  // Lengths are there before the selection that this follows has ended: that grid has waited
  // for whatever came before.
  const int head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Cut cut = load_cut(a, b);
  follow();
  const int2 counts = fetch(a.counts + b * kHKV + head);
  const int pairs = counts.x, near = counts.y;
  if (pairs < 0) return;
  const Rows<kVecs> rows(a, b, head);
  const int* const holes = a.holes + ((size_t)b * kHKV + head) * a.cap;
  const int* const movers = a.movers + ((size_t)b * kHKV + head) * a.cap;
  if (blockIdx.x > 0) {
    for (int i = near + ((blockIdx.x - 1) * kMoveWarps + warp) * 32; i < pairs; i += (gridDim.x - 1) * kMoveThreads)
      rows.template fill<32>(holes, movers, i, pairs, lane);
    return;
  }
  // What leaves the places of the last ones, then those.
  for (int i = warp * Rows<kVecs>::kStep; i < near; i += kMoveWarps * Rows<kVecs>::kStep) rows.template fill<Rows<kVecs>::kStep>(holes, movers, i, near, lane);
  rows.template follow_up<kMoveThreads>(cut, a.last, tid);
}

// ---------------------------------------------------------------------------
// Both steps in one launch, for contexts of up to kSmall tokens: a thread has two quads' keys in
// registers, the first digit's bin settles all but a few keys, whose ranks are counted among
// themselves (or, of many equal ones, by further digits), and what stays is a bit a token. A
// cluster's blocks all find the same lists, in shared memory, and share the moves.
// (With the copy that restores its weights, one sequence of 1000 tokens: 9.6 us in a graph, of which the
// copy is 1.0; call by call 12.2, as two launches 14.4. One of 4000, bf16 pages: 14.3 and 17.8; 64 of 4000: 76 and 85.)
constexpr int kSmall = 4096, kSmallThreads = 512, kQuads = kSmall / 4 / kSmallThreads, kWords = kSmall / 32;
constexpr int kRanked = 256;  // listed keys whose ranks are counted

struct alignas(16) Small {
  Shared<kSmallThreads> sh;
  uint32_t stays[kWords], equal[kWords];
  int hole_at[kWords], mover_at[kWords];  // places in the lists of a word's first
  int holes[kSmall / 2 + 1], movers[kSmall / 2 + 1];
  int pairs, near;
};

template <int kVecs>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint8_t small_smem[];
  Small& sm = *reinterpret_cast<Small*>(small_smem);
  Shared<kSmallThreads>& sh = sm.sh;
  const int rank = blockIdx.x, ranks = gridDim.x, head = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins / 4; i += kSmallThreads) reinterpret_cast<uint4*>(sh.hist[0])[i] = make_uint4(0, 0, 0, 0);
  if (tid < kWords) sm.stays[tid] = sm.equal[tid] = 0;
  if (tid == 0) sh.bad = 0, sh.listed = 0;
  follow();
  const Cut cut = load_cut(a, b);
  if (!cut.live) {  // for every block of the cluster
    if (!cut.ok && rank == 0 && head == 0 && tid == 0) record_error(a.err, kDevErrBounds);
    return;
  }
  const Rows<kVecs> rows(a, b, head);
  const uint32_t m = cut.now - a.first - a.last;
  const auto middle = [&](int t) { return lowest(cut.end - t) & ~lowest(a.first - t); };  // of a quad's tokens
  __syncthreads();
  int page[kQuads];
  uint4 key[kQuads];
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int t = 4 * (tid + i * kSmallThreads);
    page[i] = t < cut.ctx ? fetch(rows.trow + t / ATTN_PAGE) : 0;
    if (page[i] < 0 || page[i] >= a.num_pages) sh.bad = 1, page[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int t = 4 * (tid + i * kSmallThreads);
    key[i] = make_uint4(0, 0, 0, 0);
    if (t >= cut.ctx) continue;
    const float4 w = fetch(reinterpret_cast<const float4*>(a.weights + ((size_t)page[i] * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE));
    key[i] = make_uint4(ordered(w.x), ordered(w.y), ordered(w.z), ordered(w.w));
    const uint32_t in = middle(t);
    if (in & 1) atomicAdd(sh.hist[0] + (key[i].x >> kFirst), 1u);
    if (in & 2) atomicAdd(sh.hist[0] + (key[i].y >> kFirst), 1u);
    if (in & 4) atomicAdd(sh.hist[0] + (key[i].z >> kFirst), 1u);
    if (in & 8) atomicAdd(sh.hist[0] + (key[i].w >> kFirst), 1u);
  }
  if (ranks > 1) {
    __syncwarp();
    tc::cluster_arrive();  // this block has read the weights, which are moved too
  }
  if (m > 0) {
    choose<kSmallThreads>(sh, 1, 0, 0, m);
    uint32_t prefix = sh.bin, need = sh.need;
    bool whole = sh.whole;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int t = 4 * (tid + i * kSmallThreads);
      const uint32_t in = middle(t), k[4] = {key[i].x, key[i].y, key[i].z, key[i].w};
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (!(in >> j & 1)) continue;
        const uint32_t bin = k[j] >> kFirst;
        if (bin > prefix || (whole && bin == prefix)) bits |= 1u << j;
        else if (bin == prefix) {
          const uint32_t at = atomicAdd(&sh.listed, 1u);
          if (at < kListed) sh.keys[at] = k[j], sh.places[at] = t + j;
        }
      }
      bits <<= 4 * (lane & 7);
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) bits |= __shfl_xor_sync(kFull, bits, off);
      if ((lane & 7) == 0) sm.stays[t / 32] = bits;
    }
    __syncthreads();
    const int entries = sh.listed;
    if (!whole && entries <= kRanked) {
      // The rank of each among them, equal ones by their token.
      for (int i = tid; i < entries; i += kSmallThreads) {
        const uint32_t mine = sh.keys[i], place = sh.places[i];
        uint32_t rank = 0;
#pragma unroll 8
        for (int j = 0; j < entries; ++j) rank += sh.keys[j] > mine || (sh.keys[j] == mine && sh.places[j] < place);
        if (rank < need) atomicOr(sm.stays + place / 32, 1u << (place & 31));
      }
    } else if (!whole) {
      // The other digits, over all keys (they may be too many for the list).
      int shift = kFirst;
#pragma unroll 1
      for (int pass = 1; pass < 3 && !whole; ++pass) {
        const int above = shift;
        shift -= kDigit;
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          const uint32_t in = middle(4 * (tid + i * kSmallThreads)), k[4] = {key[i].x, key[i].y, key[i].z, key[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((in >> j & 1) && k[j] >> above == prefix) atomicAdd(sh.hist[pass & 1] + (k[j] >> shift & ((1u << kDigit) - 1)), 1u);
        }
        choose<kSmallThreads>(sh, 1, 0, pass, need);
        prefix = prefix << kDigit | sh.bin;
        need = sh.need;
        whole = sh.whole;
      }
      // Those above stay, and of the equal ones the first `need` (all, where the last bin is).
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int t = 4 * (tid + i * kSmallThreads);
        const uint32_t in = middle(t), k[4] = {key[i].x, key[i].y, key[i].z, key[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (!(in >> j & 1) || k[j] >> kFirst != prefix >> (kFirst - shift)) continue;
          const uint32_t digits = k[j] >> shift;
          if (digits > prefix || (whole && digits == prefix)) atomicOr(sm.stays + (t + j) / 32, 1u << ((t + j) & 31));
          else if (digits == prefix) atomicOr(sm.equal + (t + j) / 32, 1u << ((t + j) & 31));
        }
      }
      __syncthreads();
      if (!whole && warp == 0) {
        uint32_t before = 0;
        for (int w0 = 0; w0 < kWords; w0 += 32) {
          const uint32_t e = sm.equal[w0 + lane];
          uint32_t up = __popc(e);
          const uint32_t own = up;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const uint32_t x = __shfl_up_sync(kFull, up, off);
            if (lane >= off) up += x;
          }
          uint32_t left = need > before + up - own ? need - (before + up - own) : 0, keep = 0, rest = e;
          for (; left > 0 && rest; --left, rest &= rest - 1) keep |= rest & -rest;
          sm.stays[w0 + lane] |= keep;
          before += __shfl_sync(kFull, up, 31);
        }
      }
    }
  }
  __syncthreads();
  if (ranks > 1) {
    __syncwarp();
    tc::cluster_wait();
  }
  if (sh.bad) {  // seen by the blocks of all heads: nothing of the sequence is moved
    if (rank == 0 && head == 0 && tid == 0) record_error(a.err, kDevErrBounds);
    return;
  }
  // The lists: warp 0 counts what leaves below edge and what stays from there on, word by word.
  const auto below = [&](int n) { return n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1; };
  const auto split = [&](int word, uint32_t* out, uint32_t* move) {
    const int t = 32 * word;
    const uint32_t in = below(cut.end - t) & ~below(a.first - t), ahead = below(cut.edge - t);
    *out = in & ~sm.stays[word] & ahead;
    *move = sm.stays[word] & ~ahead;
  };
  if (warp == 0) {
    int holes = 0, movers = 0, near = 0;
    for (int w0 = 0; w0 * 32 < cut.end; w0 += 32) {
      uint32_t out, move;
      split(w0 + lane, &out, &move);
      const uint32_t own = __popc(out) << 16 | __popc(move);  // 1024 at most
      uint32_t up = own;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t x = __shfl_up_sync(kFull, up, off);
        if (lane >= off) up += x;
      }
      sm.hole_at[w0 + lane] = holes + (int)((up - own) >> 16);
      sm.mover_at[w0 + lane] = movers + (int)((up - own) & 0xffffu);
      const uint32_t all = __shfl_sync(kFull, up, 31);
      holes += (int)(all >> 16);
      movers += (int)(all & 0xffffu);
      near += (int)__reduce_add_sync(kFull, __popc(move & below(cut.now - 32 * (w0 + lane))));
    }
    if (lane == 0) sm.pairs = movers, sm.near = near;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuads; ++i) {
    const int t = 4 * (tid + i * kSmallThreads);
    if (t >= cut.end) continue;
    uint32_t out, move;
    split(t / 32, &out, &move);
    const uint32_t before = (1u << (t & 31)) - 1;
    int hole = sm.hole_at[t / 32] + __popc(out & before), mover = sm.mover_at[t / 32] + __popc(move & before);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int slot = page[i] * ATTN_PAGE + (t + j) % ATTN_PAGE;
      if (out >> (t + j & 31) & 1) sm.holes[hole++] = slot;
      if (move >> (t + j & 31) & 1) sm.movers[mover++] = slot;
    }
  }
  __syncthreads();
  // The first block moves what lies where the last ones go, then those; all share the others.
  constexpr int kStep = Rows<kVecs>::kStep, kWarps = kSmallThreads / 32;
  const int near = sm.near, pairs = sm.pairs;
  if (rank == 0)
    for (int i = warp * kStep; i < near; i += kWarps * kStep) rows.template fill<kStep>(sm.holes, sm.movers, i, near, lane);
  // (from the last block and warp on, which have no near ones)
  for (int i = near + ((ranks - 1 - rank) + (kWarps - 1 - warp) * ranks) * kStep; i < pairs; i += kWarps * kStep * ranks)
    rows.template fill<kStep>(sm.holes, sm.movers, i, pairs, lane);
  if (rank == 0) rows.template follow_up<kSmallThreads>(cut, a.last, tid);
}

static_assert(offsetof(Shared<512>, slice) % 16 == 0 && offsetof(Shared<1024>, slice) % 16 == 0 && offsetof(Small, sh) % 16 == 0,
              "histograms in vectors of 16 bytes");
static_assert(sizeof(Shared<512>) % 16 == 0 && sizeof(Shared<1024>) % 16 == 0, "the keys start on 16 bytes");
static_assert(sizeof(Shared<1024>) + (size_t)kMaxCached * sizeof(uint32_t) <= 232448, "exceeds the 227 KB per-block shared memory limit");

// Once per device: the shared-memory opt-in, how many SMs there are, and how many clusters
// of each size whose blocks have an SM each.
struct Device {
  bool ready = false;
  int sms = 0, clusters[kMaxCluster + 1] = {};
};
int device(Device** out) {
  constexpr int kMaxDev = 64;
  constexpr int kAll = 232448;
  static std::mutex mu;
  static Device devs[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return ATTN_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  Device& d = devs[dev];
  if (!d.ready) {
    const auto room = [](auto kernel) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAll) == cudaSuccess;
    };
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || !room(select_kernel<512>) ||
        !room(select_kernel<1024>) || !room(small_kernel<8>) || !room(small_kernel<16>)) {
      (void)cudaGetLastError();
      return ATTN_ECUDA;
    }
    for (int size = 1; size <= kMaxCluster; size *= 2) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(size, kHKV);
      cfg.blockDim = dim3(1024);
      cfg.dynamicSmemBytes = kAll;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = size;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&d.clusters[size], select_kernel<1024>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        d.clusters[size] = 0;
      }
    }
    d.ready = true;
  }
  *out = &d;
  return ATTN_OK;
}

int list_cap(int max_context) { return max_context / 2 + 1; }

}  // namespace

size_t evict_workspace_bytes(int B, int max_context) {
  if (max_context <= kSmall) return 0;
  return (size_t)B * kHKV * sizeof(int2) + 2 * (size_t)B * kHKV * list_cap(max_context) * sizeof(int);
}

int launch_evict(const EvictCall& c, unsigned* err, cudaStream_t stream) {
  Device* d = nullptr;
  const int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const int sms = d->sms;
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
  a.counts = static_cast<int2*>(c.workspace);
  a.holes = reinterpret_cast<int*>(a.counts + (size_t)c.B * kHKV);
  a.movers = a.holes + (size_t)c.B * kHKV * a.cap;
  a.err = err;

  if (c.max_context <= kSmall) {
    // Blocks to share the moves: as many as have an SM each, with 128 tokens at least.
    int ranks = 1;
    while (ranks < kMaxCluster && (long long)c.B * kHKV * 2 * ranks <= sms && c.max_context / (2 * ranks) >= 128) ranks *= 2;
    const auto kernel = c.type == ATTN_BF16 ? small_kernel<8> : small_kernel<16>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, kHKV, c.B);
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = sizeof(Small);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return launched(cudaLaunchKernelEx(&cfg, kernel, a)) == cudaSuccess ? ATTN_OK : ATTN_ELAUNCH;
  }

  // Blocks of a cluster: as many as have an SM each at once, with 1024 tokens at least; and so many that
  // a block's keys fit its shared memory, if they can.
  int ranks = 1;
  while (ranks < kMaxCluster && (c.B * kHKV <= d->clusters[2 * ranks] ? c.max_context / (2 * ranks) >= 1024
                                                                      : c.max_context / ranks > kMaxCached))
    ranks *= 2;
  const int span = ((c.max_context + ATTN_PAGE - 1) / ATTN_PAGE + ranks - 1) / ranks * ATTN_PAGE;
  a.cached = span <= kMaxCached;
  // Threads by a block's tokens. Blocks of 512 share an SM, and one counts while the other waits
  // (40 sequences of 6000 tokens: 82 us for the call, 96 with 1024; 30 of 10000: 91 and 102);
  // with 1024 more is under way where an SM holds one or two such blocks' keys (60 of up to
  // 14000: 165 and 157; 16 of 16384: 92 and 81).
  const bool wide = span > 12288;
  const size_t keys = a.cached ? (size_t)span * sizeof(uint32_t) : 0;
  const auto kernel = wide ? select_kernel<1024> : select_kernel<512>;
  const size_t smem = (wide ? sizeof(Shared<1024>) : sizeof(Shared<512>)) + keys;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks, kHKV, c.B);
  cfg.blockDim = dim3(wide ? 1024 : 512);
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
  if (launched(cudaLaunchKernelEx(&cfg, kernel, a)) != cudaSuccess) return ATTN_ELAUNCH;
  // Blocks for the pairs: one for 128 of them, at most 32 resident rounds of all SMs.
  const long long most = 32LL * 16 * sms / ((long long)c.B * kHKV);
  long long blocks = (a.cap + kMoveThreads - 1) / kMoveThreads;
  if (blocks > most) blocks = most < 1 ? 1 : most;
  const dim3 grid((unsigned)blocks + 1, kHKV, c.B);
  return launch_following(c.type == ATTN_BF16 ? move_kernel<8> : move_kernel<16>, grid, dim3(kMoveThreads), stream, a) == cudaSuccess
             ? ATTN_OK : ATTN_ELAUNCH;
}

}  // namespace attn
