// tree.cu -- attention of drafted tokens over a paged cache: each of B
// sequences has up to 64 drafted rows whose keys and values already lie in its
// cache behind the ctx_b accepted tokens, and row i sees all of those and the
// drafted rows j whose bit is set in its mask (itself and its ancestors in the
// tree of drafts):
//   K_i = {0 .. ctx-1} u {ctx + j : bit j of mask_i, j < T}
//   out_i = sum_{j in K_i} softmax_j(q_i . k_j / 8) v_j,   zeros for an empty K_i
//
// Three kernels compute it, all in one pass over the cache with all four query
// heads of a KV head at once, in fp32 precision on both page types:
//   bf16 pages, up to 8 drafted rows: tree_tc.cu (keys on the M side of tcgen05)
//   more rows, and fp32 pages from 5 on: tree_wide.cu (rows on the M side)
//   fp32 pages, up to 4 rows: the kernel here
// (small calls with more rows take several blocks of the first and last kind)
// This file also holds what they share on the host: how a call is cut into key
// segments, the launch, and the merge of segments that are not one cluster, with
// the split-K rule m = max m_s, out = sum e^(m_s - m) O_s / sum e^(m_s - m) l_s.
//
// The kernel here: a block owns (key segment, KV head, sequence) and 16 query
// rows, 4 drafted tokens, an m-tile of mma.sync (16 rows x 8 keys, so few rows
// waste little, where a tcgen05 tile would be mostly padding and fp32 pages would
// have to be split in shared memory first). Its warps share nothing until the
// end: each walks its own 16-token pages through its own ring of TMA boxes, with
// its own running maximum, sum and accumulator. Each operand is two tf32 terms
// x = hi + lo (hi = x rounded to 11 bits), hi hi + hi lo + lo hi, split in
// registers. The reference maximum of a row moves only when a score passes it by
// 2^8 (p stays below 2^8, far from fp32's range), so in the steady state a page
// costs one vote instead of a reduction over lanes and a rescaled accumulator.
// Bound: HBM, and the two blocks that 16 sequences of 16384 tokens leave each of 128
// SMs: 1.07 GB in 205 us, 5.2 TB/s (4 rows: 206; the mma.sync pipe is 46% active; 201
// with first terms that round to infinity past 2^128 - 2^115).
#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"
#include "tree.cuh"

namespace attn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kC = kTreeC, kStale = kTreeStale;
constexpr int kMaxSplits = 64;

constexpr int kWarps = 4;
constexpr int kStages = 3;                       // pages of a warp in flight: 96 KB a block, two blocks an SM
constexpr int kRows = 16, kTokens = kRows / kGroup;  // query rows, drafted rows
constexpr int kRowStride = kD + 4;
constexpr uint32_t kBox = ATTN_PAGE * 128;       // 32 dims of 16 tokens
constexpr uint32_t kStage = 4 * kBox;            // a page of K, then of V
constexpr int kSteps = 8;                        // k-steps of q . k
constexpr uint32_t kSmemQ = kWarps * kStages * kStage;          // q's fragments, later the warps' maxima and sums
constexpr uint32_t kSmemRows = kSmemQ + kSteps * 2 * 512;       // [16][kRowStride], for a cluster's merge
constexpr uint32_t kSmemEnds = kSmemRows + kRows * kRowStride * 4;
constexpr uint32_t kSmemMask = kSmemEnds + kRows * 8;
constexpr uint32_t kSmemBar = kSmemMask + 4 * 8;
constexpr uint32_t kSmemAlloc = kSmemBar + kWarps * kStages * 8 + 1024;
constexpr int kBlocks = 2;
static_assert(kBlocks * (kSmemAlloc + 1024) <= 233472, "shared memory of an SM");
static_assert(kRows * kD * 4 <= kStages * kStage, "a warp's accumulator fits its own ring");

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The tf32 terms of an operand of any size: hi by tf32_near, lo the exact rest, of
// which the tensor core reads the upper 11 bits. p stays below 2^8 and needs no limit.
__device__ __forceinline__ uint32_t hi_of(float x) { return __float_as_uint(tf32_near(x)); }
__device__ __forceinline__ uint32_t lo_of(float x) { return __float_as_uint(x - tf32_near(x)); }
__device__ __forceinline__ uint32_t hi_of_p(float x) { return (__float_as_uint(x) + 0x1000u) & 0xffffe000u; }
__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// The tensor core's own accumulation does not round to nearest: over a long key
// range its error would all lean one way. Each page's product starts at zero
// and is added here, rounded to nearest; a score's small terms have a chain of
// their own for the same reason.
__device__ __forceinline__ void add4(float (&o)[4], const float (&x)[4]) {
  tc::add2(o[0], o[1], o[0], o[1], x[0], x[1]);
  tc::add2(o[2], o[3], o[2], o[3], x[2], x[3]);
}

// Inside an 8-row group the order of keys, and inside a 32-dim group the order
// of 16-byte chunks, is free as long as both sides of a product use one order.
// This one (0 4 1 5 2 6 3 7 backwards: bit 0 to bit 2) makes every 128-bit load
// of a fragment touch all eight chunk positions of the swizzle once.
__device__ __forceinline__ int turn(int n) { return (n >> 1) | ((n & 1) << 2); }

template <bool kFault>
__global__ void __launch_bounds__(32 * kWarps, kBlocks)
tree_narrow_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const TreeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* const bars = reinterpret_cast<uint64_t*>(smem + kSmemBar);
  uint64_t* const full = bars + warp * kStages;
  if (lane == 0) {
    if (warp < 2) tc::tma_prefetch_desc(warp ? &mv : &mk);
    for (int i = 0; i < kStages; ++i) tc::mbar_init(&full[i], 1);
    tc::fence_mbar_init();
  }
  follow();
  const int g = lane >> 2, c = lane & 3;  // fragment row (or key), fragment column
  const int s = blockIdx.x, head = blockIdx.y % kHKV, rt = blockIdx.y / kHKV, b = blockIdx.z;

  // The table's first entries are on their way while the lengths are, as of a
  // sequence as long as the call allows: an entry past the sequence is read and not
  // used.
  const int first_page = s * (a.split_len / ATTN_PAGE) + warp + lane * kWarps;
  const int first_entries = first_page < a.max_blocks ? fetch(a.table + (size_t)b * a.max_blocks + first_page) : 0;
  const Seq seq = load_seq(a, b);
  const int i0 = rt * kTokens;  // the block's first drafted row
  const int nrows = min(kTokens, seq.rows - i0);
  const int len = segment_len(a, seq), k0 = s * len;
  const int k1 = min(k0 + len, seq.keys);
  if (!seq.ok && s == 0 && tid == 0) record_error(a.err, kDevErrBounds);
  if (nrows <= 0) return;
  if (k0 >= k1 && !a.cluster) {
    // Past the sequence: the merge counts its segments from the lengths. A
    // sequence without any key (only a refused one) gets zeros.
    if (s == 0)
      for (int e = tid; e < nrows * kGroup * kD; e += 32 * kWarps)
        a.out[((size_t)(seq.first + i0 + e / (kGroup * kD)) * kHQ + head * kGroup) * kD + e % (kGroup * kD)] = 0.f;
    return;
  }
  const bool whole = !a.cluster && seq.keys <= a.split_len;  // one segment: the output is written here

  unsigned long long* masks = reinterpret_cast<unsigned long long*>(smem + kSmemMask);
  uint8_t* const ring = smem + warp * (kStages * kStage);
  if (tid < kTokens)
    masks[tid] = tid >= nrows ? 0ull
                 : a.masks    ? (unsigned long long)fetch(a.masks + seq.first + i0 + tid)
                              : ~0ull >> (63 - (i0 + tid));
  __syncwarp();

  // This warp's pages: pages warp, warp + kWarps, ... of the segment. Lane l
  // holds the table entry of its l-th page from the last multiple of 32.
  const int npages = max(0, (k1 - k0 + ATTN_PAGE - 1) / ATTN_PAGE);
  const int mine = warp < npages ? (npages - warp + kWarps - 1) / kWarps : 0;
  const int* trow = a.table + (size_t)b * a.max_blocks + k0 / ATTN_PAGE + warp;
  int entries = 0;
  auto issue = [&](int n) {
    if ((n & 31) == 0)
      entries = n == 0 && len == a.split_len ? first_entries
                : n + lane < mine            ? fetch(trow + (size_t)(n + lane) * kWarps)
                                             : 0;
    int page = __shfl_sync(kFull, entries, n & 31);
    if (lane == 0) {
      if (page < 0 || page >= a.num_pages) {  // reads as zeros: past the pool's end
        record_error(a.err, kDevErrBounds);
        page = a.num_pages;
      }
      const int st = n % kStages;
      uint8_t* dst = ring + st * kStage;
      tc::mbar_arrive_expect_tx(&full[st], kStage);
      if (withheld<kFault>(a, s, n)) return;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        tc::tma_load_2d(dst + x * kBox, &mk, &full[st], head * kD + x * 32, page * ATTN_PAGE);
        tc::tma_load_2d(dst + (2 + x) * kBox, &mv, &full[st], head * kD + x * 32, page * ATTN_PAGE);
      }
    }
  };
  int issued = 0;
  for (; issued < kStages && issued < mine; ++issued) issue(issued);

  // q's fragments, split into their terms once for the block, in the order the
  // lanes read them; then in registers.
  uint4* const qs = reinterpret_cast<uint4*>(smem + kSmemQ);
  {
    const int j = warp;  // 16 dims
    float x[2][4];       // rows g and g + 8, dims 4c .. 4c + 3
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 2 * h + (g >> 2);
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < nrows)
        u = fetch(reinterpret_cast<const float4*>(a.q + ((size_t)(seq.first + i0 + i) * kHQ + head * kGroup + (g & 3)) * kD +
                                                  16 * j + 4 * c));
      x[h][0] = u.x, x[h][1] = u.y, x[h][2] = u.z, x[h][3] = u.w;
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // k-step 2 j + u: k = c is dim 4c + 2u, k = c + 4 the next
      uint4* dst = qs + ((2 * j + u) * 2) * 32 + lane;
      dst[0] = make_uint4(hi_of(x[0][2 * u]), hi_of(x[1][2 * u]), hi_of(x[0][2 * u + 1]), hi_of(x[1][2 * u + 1]));
      dst[32] = make_uint4(lo_of(x[0][2 * u]), lo_of(x[1][2 * u]), lo_of(x[0][2 * u + 1]), lo_of(x[1][2 * u + 1]));
    }
  }
  __syncthreads();
  uint4 qreg[2 * kSteps];
#pragma unroll
  for (int e = 0; e < 2 * kSteps; ++e) qreg[e] = qs[e * 32 + lane];
  auto qfrag = [&](int step, int term, uint32_t (&r)[4]) {
    const uint4 v = qreg[step * 2 + term];
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  };

  // State of this warp's partial: rows g and g + 8. The sums are this lane's
  // columns' alone until the end.
  float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
  for (int u = 0; u < 8; ++u) o[u][0] = o[u][1] = o[u][2] = o[u][3] = 0.f;

  bool failed = false;
  int n = 0;
  for (; n < mine; ++n) {
    const int st = n % kStages;
    if (!__all_sync(kFull, tc::mbar_wait(&full[st], (n / kStages) & 1, a.timeout_ns))) {
      failed = true;
      break;
    }
    const uint8_t* kt = ring + st * kStage;
    const uint8_t* vt = kt + 2 * kBox;
    const int t0 = k0 + (warp + n * kWarps) * ATTN_PAGE;
    const bool tail = t0 + ATTN_PAGE > seq.ctx;  // holds drafted keys, or slots past them

    // Scores: sc[nt], columns 2c and 2c + 1 of 8-key group nt. Column n is key
    // turn(n) of the group.
    float sc[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
      float low[4] = {0.f, 0.f, 0.f, 0.f};  // the small terms' own chain
      const int r = nt * 8 + turn(g);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(kt + (j >> 1) * kBox + r * 128 +
                                                          ((((j & 1) * 4 + c) ^ (r & 7)) << 4));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float e0 = u ? x.z : x.x, e1 = u ? x.w : x.y;
          uint32_t qh[4], ql[4];
          qfrag(2 * j + u, 0, qh);
          qfrag(2 * j + u, 1, ql);
          mma_tf32(low, ql, hi_of(e0), hi_of(e1));
          mma_tf32(low, qh, lo_of(e0), lo_of(e1));
          mma_tf32(sc[nt], qh, hi_of(e0), hi_of(e1));
        }
      }
      add4(sc[nt], low);
    }

    if (tail) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = t0 + nt * 8 + turn(2 * c + (e & 1));
          const int at = pos - seq.ctx;
          const bool seen = pos < k1 && (at < 0 || (masks[2 * (e >> 1) + (g >> 2)] >> at & 1));
          if (!seen) sc[nt][e] = -INFINITY;
        }
    }

    // Does a score pass its row's reference by more than 2^8? (Any score does
    // while the reference is -inf.)
    bool over = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float most = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
      over |= most * kC > top[h] + kStale;
    }
    if (__any_sync(kFull, over)) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float most = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
        most = fmaxf(most, __shfl_xor_sync(kFull, most, 1));
        most = fmaxf(most, __shfl_xor_sync(kFull, most, 2));
        const float next = fmaxf(top[h], most * kC);
        const float alpha = next == -INFINITY ? 1.f : ex2(top[h] - next);
        top[h] = next;
        sum[h] *= alpha;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          o[u][2 * h] *= alpha;
          o[u][2 * h + 1] *= alpha;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float ref = top[h] == -INFINITY ? 0.f : top[h];  // a row that has seen no key yet
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 2 * h; e < 2 * h + 2; ++e) {
          sc[nt][e] = ex2(fmaf(sc[nt][e], kC, -ref));
          sum[h] += sc[nt][e];
        }
    }

    // Drafted values that are not finite reach only the rows that see them; a
    // product with a zero probability would spread NaN. They are taken out of
    // the operand and added row by row. Slots past the last key count as zeros.
    bool odd = false;
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      float va[2][2][4];  // keys c and c + 4 of each group, dims 32 hh + 4 turn(g) ..
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = nt * 8 + c + 4 * y;
          const float4 x = *reinterpret_cast<const float4*>(vt + hh * kBox + r * 128 + ((turn(g) ^ (r & 7)) << 4));
          va[nt][y][0] = x.x, va[nt][y][1] = x.y, va[nt][y][2] = x.z, va[nt][y][3] = x.w;
          if (tail) {
            const int pos = t0 + r;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              if (pos >= k1) va[nt][y][u] = 0.f;
              if (pos >= seq.ctx && !finite(va[nt][y][u])) {
                odd = true;
                va[nt][y][u] = 0.f;
              }
            }
          }
        }
      uint32_t ph[2][4], pl[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // a0 a1: column 2c (key c), rows g, g + 8; a2 a3: column 2c + 1 (key c + 4)
          const float p = sc[nt][(e & 1) * 2 + (e >> 1)];
          ph[nt][e] = hi_of_p(p);
          pl[nt][e] = __float_as_uint(p - __uint_as_float(ph[nt][e]));
        }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          mma_tf32(x, pl[nt], hi_of(va[nt][0][u]), hi_of(va[nt][1][u]));
          mma_tf32(x, ph[nt], lo_of(va[nt][0][u]), lo_of(va[nt][1][u]));
        }
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) mma_tf32(x, ph[nt], hi_of(va[nt][0][u]), hi_of(va[nt][1][u]));
        add4(o[hh * 4 + u], x);
      }
    }
    if (tail && __any_sync(kFull, odd)) {
#pragma unroll 1
      for (int key = 0; key < ATTN_PAGE; ++key) {
        const int at = t0 + key - seq.ctx;
        if (at < 0 || t0 + key >= k1) continue;
        const int from = (lane & ~3) | (key & 3);  // the lane of this row's columns of keys c and c + 4
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = __shfl_sync(kFull, key < 8 ? sc[0][2 * h] : sc[1][2 * h], from);
          const float p1 = __shfl_sync(kFull, key < 8 ? sc[0][2 * h + 1] : sc[1][2 * h + 1], from);
          const float p = (key & 4) ? p1 : p0;
          const bool seen = masks[2 * h + (g >> 2)] >> at & 1;
#pragma unroll
          for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int chunk = c + 4 * e;  // turn(2c + e)
              const float v = *reinterpret_cast<const float*>(vt + (u >> 2) * kBox + key * 128 +
                                                              ((chunk ^ (key & 7)) << 4) + (u & 3) * 4);
              if (seen && !finite(v)) o[u][2 * h + e] += p * v;
            }
        }
      }
    }
    __syncwarp();  // the stage is read: refill it
    if (issued < mine) issue(issued++);
  }

  if (failed) {
    // A page did not land in time: record it, give the copies still in flight
    // a bounded wait before the block's shared memory is released.
    if (lane == 0) record_error(a.err, kDevErrTimeout);
    for (int i = n; i < issued; ++i) tc::mbar_wait(&full[i % kStages], (i / kStages) & 1, a.timeout_ns);
  }

  // The warp's partial: sums over its lanes, the accumulator into its own ring
  // (every copy into it has landed and been read), row-major with the 16-byte
  // chunks of a row turned by the row.
  float* const acc = reinterpret_cast<float*>(ring);
  auto acc_at = [](int row, int d) { return row * kD + ((((d >> 2) ^ row) & 7) | ((d >> 2) & 8)) * 4 + (d & 3); };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 8 * h + g;
    sum[h] += __shfl_xor_sync(kFull, sum[h], 1);
    sum[h] += __shfl_xor_sync(kFull, sum[h], 2);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float4*>(acc + acc_at(row, 32 * hh + 16 * e + 4 * c)) =
            make_float4(o[4 * hh][2 * h + e], o[4 * hh + 1][2 * h + e], o[4 * hh + 2][2 * h + e],
                        o[4 * hh + 3][2 * h + e]);
  }
  const bool any_failed = __syncthreads_or(failed);  // and q's fragments are no longer read
  float2* const ml = reinterpret_cast<float2*>(smem + kSmemQ);  // [warp][row]
  if (c == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) ml[warp * kRows + 8 * h + g] = make_float2(top[h], sum[h]);
  }
  __syncthreads();
  float* const rows = reinterpret_cast<float*>(smem + kSmemRows);
  float2* const ends = reinterpret_cast<float2*>(smem + kSmemEnds);
  for (int e = tid; e < nrows * kGroup * 16; e += 32 * kWarps) {  // (row, 16-byte chunk)
    const int row = e >> 4, d = (e & 15) * 4;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, ml[w * kRows + row].x);
    float den = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 p = ml[w * kRows + row];
      // A warp that saw no key of the row has no weight; a sum that is NaN (a
      // row whose scores are) stays NaN.
      const float wt = p.x == -INFINITY ? 0.f : ex2(p.x - m);
      den = fmaf(wt, p.y, den);
      if (wt == 0.f) continue;
      const float4 y =
          *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * (kStages * kStage)) + acc_at(row, d));
      x.x = fmaf(wt, y.x, x.x);
      x.y = fmaf(wt, y.y, x.y);
      x.z = fmaf(wt, y.z, x.z);
      x.w = fmaf(wt, y.w, x.w);
    }
    const size_t at = (size_t)(seq.first + i0 + row / kGroup) * kHQ + head * kGroup + row % kGroup;
    // after a failed wait the segment counts as empty
    const float2 end = any_failed ? make_float2(-INFINITY, 0.f) : make_float2(m, den);
    if (a.cluster) {
      *reinterpret_cast<float4*>(rows + row * kRowStride + d) = x;
      if (d == 0) ends[row] = end;
    } else if (whole) {
      if (any_failed) continue;  // left unwritten
      const float inv = den == 0.f ? 0.f : 1.f / den;  // no key: zeros
      *reinterpret_cast<float4*>(a.out + at * kD + d) = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    } else {
      *reinterpret_cast<float4*>(a.parts + (at * a.splits + s) * kD + d) = x;
      if (d == 0) reinterpret_cast<float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD)[at * a.splits + s] = end;
    }
  }
  if (a.cluster) cluster_merge(a, seq.first + i0, nrows, head, rows, kRowStride, ends, tid, 32 * kWarps);
}

// Merge of segments that are not one cluster: a warp per (drafted row, query
// head), two dims a lane. Lane s holds segment s's maximum and sum, 32 segments at
// a time; eight segments' rows are on their way at once.
constexpr int kMergeWarps = 8;
__global__ void __launch_bounds__(32 * kMergeWarps)
tree_merge_kernel(const TreeArgs a) {
  constexpr int kAhead = 8;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const int i = blockIdx.x / (kHQ / kMergeWarps);
  const int h = (blockIdx.x % (kHQ / kMergeWarps)) * kMergeWarps + (threadIdx.x >> 5);
  follow();  // the lengths too may come from a kernel that only the one before has waited for
  const Seq seq = load_seq(a, b);
  if (i >= seq.rows || seq.keys <= a.split_len) return;
  const int active = (seq.keys + a.split_len - 1) / a.split_len;
  const size_t at = (size_t)(seq.first + i) * kHQ + h;
  const float2* mls = reinterpret_cast<const float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD) + at * a.splits;
  const float2* rows = reinterpret_cast<const float2*>(a.parts + at * a.splits * kD) + lane;
  float2 p[kMaxSplits / 32];
  float m = -INFINITY;
#pragma unroll
  for (int k = 0; k < kMaxSplits / 32; ++k) {
    p[k] = make_float2(-INFINITY, 0.f);
    if (k * 32 + lane < active) p[k] = mls[k * 32 + lane];
    m = fmaxf(m, p[k].x);
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
  float den = 0.f;
  float2 x = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kMaxSplits / 32; ++k) {
    const float w = p[k].x == -INFINITY ? 0.f : ex2(p[k].x - m);
    const int most = min(32, active - k * 32);
    den = fmaf(w, p[k].y, den);
    for (int t = 0; t < most; t += kAhead) {
      float2 y[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (t + u < most) y[u] = rows[(k * 32 + t + u) * (kD / 2)];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const float wt = __shfl_sync(kFull, w, (t + u) & 31);
        if (t + u < most && wt != 0.f) {  // an empty segment's row has no weight, whatever it holds
          x.x = fmaf(wt, y[u].x, x.x);
          x.y = fmaf(wt, y[u].y, x.y);
        }
      }
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) den += __shfl_xor_sync(kFull, den, off);
  const float inv = den == 0.f ? 0.f : 1.f / den;  // no key: zeros
  *reinterpret_cast<float2*>(a.out + at * kD + 2 * lane) = make_float2(x.x * inv, x.y * inv);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// A page pool [num_pages * 16][8][64]; a box is the 16 rows of a page.
int encode_pool(const void* base, int num_pages, bool bf16, bool atom32, CUtensorMap* map) {
  return encode_rows_map(base, bf16, (long long)num_pages * ATTN_PAGE, ATTN_PAGE,
                         atom32 ? CU_TENSOR_MAP_SWIZZLE_128B_ATOM_32B : CU_TENSOR_MAP_SWIZZLE_128B, map);
}

// Variants by page type and the drafted rows of a block. Long calls take the least
// that holds their rows. Measured on 16 sequences of 16384 tokens, in graphs: bf16
// pages, 8 rows, tree_tc 99 us and tree_wide 129; 16 rows, 184 (as two tiles of 8) and
// 129. fp32 pages, 4 rows, the kernel here 205 us and tree_wide 216; 8 rows, 395 and 216.
// A small call is another matter: where a block for every 128 keys of every tile of
// few rows has its place at once, reading a page for each of those tiles costs less
// than the longer way through a wide block: one sequence of 1000 tokens with 8 rows
// on fp32 pages 7.6 and 9.0 us, with 16 8.2 and 9.4; with 16 rows on bf16 pages 8.3
// and 8.6. With four sequences more blocks than places: 11.5 and 10.9, 17.3 and 11.4,
// 10.1 and 10.0. On bf16 pages a third more blocks than places still pay (384 of 304:
// eight sequences of 300 tokens with 16 rows 7.6 and 8.7, one of 2000 with 24 10.0 and
// 10.5; 576: two of 1000 with 32 11.8 and 10.7); on fp32 pages it depends (384: four
// of 300 with 16 rows 9.1 and 9.4, sixteen of 60 11.5 and 8.1).
using Variant = TreeVariant;
const Variant kNarrow = {tree_narrow_kernel<false>, tree_narrow_kernel<true>, kTokens, 32 * kWarps, kSmemAlloc, kBlocks, false, 0, 2, 1};
constexpr int kCount[2] = {2, 3};
const Variant kVariants[2][3] = {{kNarrow, tree_wide_variant(false)},
                                 {tree_tc_variant(4), tree_tc_variant(8), tree_wide_variant(true)}};

// Per device and variant: how many blocks fit at once, and how many clusters of
// each size.
struct TreeDevice {
  bool ready = false;
  int slots[2][3] = {};
  int clusters[2][3][kMaxCluster + 1] = {};
};
int set_up(const Variant& x, decltype(x.kernel) kernel) {
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)x.smem) != cudaSuccess)
    return ATTN_ECUDA;
  if (x.regs) {  // a split that adds up to more than the launch has would wait forever
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess) return ATTN_ECUDA;
    if (fa.numRegs < x.regs) return ATTN_ELAUNCH;
  }
  return ATTN_OK;
}
int tree_device(TreeDevice** out) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static TreeDevice devs[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return ATTN_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  TreeDevice& d = devs[dev];
  if (!d.ready) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return ATTN_ECUDA;
    for (int t = 0; t < 2; ++t)
      for (int v = 0; v < kCount[t]; ++v) {
        const Variant& x = kVariants[t][v];
        if (const int rc = set_up(x, x.kernel); rc != ATTN_OK) return rc;
        // The occupancy queries count one block an SM for any kernel that uses
        // tensor memory; with half an SM's shared and tensor memory two run
        // (measured: 256 blocks of tree_tc take the time of 128).
        int counted = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&counted, x.kernel, x.threads, x.smem) != cudaSuccess)
          return ATTN_ECUDA;
        const int more = counted > 0 && counted < x.blocks ? x.blocks / counted : 1;
        d.slots[t][v] = sms * x.blocks;
        for (int size = 2; size <= kMaxCluster; ++size) {
          cudaLaunchConfig_t cfg = {};
          cfg.gridDim = dim3(size, kHKV);
          cfg.blockDim = dim3(x.threads);
          cfg.dynamicSmemBytes = x.smem;
          cudaLaunchAttribute attr[1];
          attr[0].id = cudaLaunchAttributeClusterDimension;
          attr[0].val.clusterDim.x = size;
          attr[0].val.clusterDim.y = 1;
          attr[0].val.clusterDim.z = 1;
          cfg.attrs = attr;
          cfg.numAttrs = 1;
          int n = 0;
          if (cudaOccupancyMaxActiveClusters(&n, x.kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            n = 0;  // no such clusters: segments merge through memory
          }
          d.clusters[t][v][size] = n * more;
        }
      }
    d.ready = true;
  }
  *out = &d;
  return ATTN_OK;
}

}  // namespace

int tree_plan(bool bf16, int B, int N, int max_rows, int max_context, int splits_hint, size_t room, TreePlan* plan) {
  TreeDevice* d = nullptr;
  const int rc = tree_device(&d);
  if (rc != ATTN_OK) return rc;
  auto small = [&](int v) {  // a block for every 128 keys of every row tile, nearly all at once
    const int tokens = kVariants[bf16][v].tokens, slots = d->slots[bf16][v];
    return (long long)B * ((max_context + max_rows + 127) / 128) * kHKV * ((max_rows + tokens - 1) / tokens) <=
           (bf16 ? slots + slots / 3 : slots);
  };
  int v = 0;
  if (bf16)
    v = max_rows <= kVariants[1][0].tokens ? 0 : max_rows <= kVariants[1][1].tokens || small(1) ? 1 : 2;
  else
    v = max_rows <= kTokens || small(0) ? 0 : 1;
  plan->variant = v;
  const int* const clusters = d->clusters[bf16][v];
  const int keys = max_context + max_rows;
  auto cut = [&](int n) {  // into n segments, or as many of whole 128 keys as that leaves
    const int per = (keys + n - 1) / n;
    plan->split_len = (per + 127) / 128 * 128;
    plan->splits = (keys + plan->split_len - 1) / plan->split_len;
    plan->cluster = plan->splits > 1 && plan->splits <= kMaxCluster && clusters[plan->splits] > 0;
  };
  int n = splits_hint < kMaxSplits ? splits_hint : kMaxSplits;
  if (n <= 0) {
    // The segments that take the least time, counted in tiles of 128 keys: rounds
    // of resident blocks, each as long as its tiles and what a block costs besides
    // them, and the merge: one in a cluster; through memory a second kernel and what
    // the partials take. One row on fp32 pages, 300 tokens: three segments
    // 5.8 us, one 8.4; sixteen such sequences: three 12.3, one 8.8. 2000 tokens: 16
    // segments 7.3 us, eight 8.6; 4000: 24 9.3, eight 13.0. Only what the workspace
    // holds counts: fewer sequences may want more segments, and a buffer that was
    // enough for the batch before is enough for every one, if not for the best cut.
    const Variant& x = kVariants[bf16][v];
    const int slots = d->slots[bf16][v];
    const long long units = (long long)B * kHKV * ((max_rows + x.tokens - 1) / x.tokens);
    const int tiles = (keys + 127) / 128;
    const int limit = tiles < kMaxSplits ? tiles : kMaxSplits;
    long long best = 0;
    n = 1;
    for (int s = 1; s <= limit; ++s) {
      if ((size_t)N * kHQ * s * (kD + 2) * sizeof(float) > room) {  // unless a cluster, or fewer once cut
        cut(s);
        if (tree_workspace_bytes(N, *plan) > room) continue;  // never of one segment
      }
      const bool cluster = s > 1 && s <= kMaxCluster && clusters[s] > 0;
      const long long rounds = cluster ? (units + clusters[s] - 1) / clusters[s] : (units * s + slots - 1) / slots;
      const long long merge = s == 1 ? 0 : cluster ? 1 : x.merge + (long long)B * max_rows * s / 440;
      const long long cost = rounds * ((tiles + s - 1) / s + x.fixed) + merge;
      if (s == 1 || cost < best) {
        best = cost;
        n = s;
      }
    }
  }
  cut(n);
  return ATTN_OK;
}

size_t tree_workspace_bytes(int N, const TreePlan& plan) {
  return plan.splits <= 1 || plan.cluster ? 0 : (size_t)N * kHQ * plan.splits * (kD + 2) * sizeof(float);
}

int launch_tree(const TreeCall& c, unsigned* err, cudaStream_t stream) {
  TreeDevice* d = nullptr;
  int rc = tree_device(&d);
  if (rc != ATTN_OK) return rc;
  const bool bf16 = c.type == ATTN_BF16;
  const Variant& x = kVariants[bf16][c.plan.variant];
  if (c.withheld && (rc = set_up(x, x.fault)) != ATTN_OK) return rc;
  alignas(64) CUtensorMap mk, mv;
  if ((rc = encode_pool(c.k_pages, c.num_pages, bf16, false, &mk)) != ATTN_OK ||
      (rc = encode_pool(c.v_pages, c.num_pages, bf16, x.v_atom32, &mv)) != ATTN_OK)
    return rc;
  const TreePlan& p = c.plan;
  const TreeArgs a{c.q, c.k_pages, c.v_pages, c.table, c.ctx_lens, c.row_start, c.masks, c.out, c.parts,
                   c.B, c.N, c.max_rows, c.max_blocks, c.num_pages, c.max_context, p.split_len, p.splits,
                   p.cluster, err, c.withheld ? kFaultNs + c.withheld : kTimeoutNs};
  const int row_tiles = (c.max_rows + x.tokens - 1) / x.tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.splits, kHKV * row_tiles, c.B);
  cfg.blockDim = dim3(x.threads);
  cfg.dynamicSmemBytes = x.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (p.cluster) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  if (launched(cudaLaunchKernelEx(&cfg, c.withheld ? x.fault : x.kernel, mk, mv, a)) != cudaSuccess) return ATTN_ELAUNCH;
  if (p.splits > 1 && !p.cluster) {
    // The merge's blocks start as this grid's last ones run (programmatic
    // dependent launch) and wait for its end.
    cudaLaunchConfig_t mcfg = {};
    mcfg.gridDim = dim3(c.max_rows * (kHQ / kMergeWarps), c.B);
    mcfg.blockDim = dim3(32 * kMergeWarps);
    mcfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    mcfg.attrs = attr;
    mcfg.numAttrs = 1;
    if (launched(cudaLaunchKernelEx(&mcfg, tree_merge_kernel, a)) != cudaSuccess) return ATTN_ELAUNCH;
  }
  return ATTN_OK;
}

}  // namespace attn
