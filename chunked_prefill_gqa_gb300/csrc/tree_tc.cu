// tree_tc.cu -- the drafted-tree attention of tree.cu on the tcgen05 tensor
// cores, for bf16 pages.
//
// The few query rows of a (sequence, KV head) are the N side of both products
// and the keys the M side, so a tile is always 128 full keys whatever the
// number of rows, and the three bf16 terms of q (and of the probabilities) that
// keep them in fp32 precision cost narrow instructions, or stack along N:
//   S^T [128 keys][R] = K [128][64] . (q3, q2, q1)^T         12 MMAs of N = R
//   O^T [64 dims][3 R] += V^T [64][128] . [p1 | p2 | p3]      8 MMAs of N = 3 R
// with R = 4 x the drafted rows of a block (16 or 32 columns). K is a
// K-major operand as it lies in the page, V^T an MN-major one, also as it lies;
// nothing of the cache is converted or transposed. p goes through shared memory,
// written by the thread that owns its key: one row of N per key, which is an
// MN-major operand again. The accumulators are in tensor memory: S^T in lanes =
// keys, O^T (M = 64) in lanes 0-15 of each lane quarter.
//
// A thread owns one key and 16 columns, so the softmax over keys runs across
// threads. It needs no maximum in the steady state: a row's reference moves only
// when a score passes it by 2^8, which each thread checks on its own values; one
// barrier with a vote per tile decides. Sums stay per thread until the end. The
// tensor core's accumulation does not round to nearest, and over a long key
// range that error would lean one way: every 4 tiles (and when a reference
// moves, which then costs nothing more) O is added to fp32 sums in shared
// memory and starts anew.
//
// Roles: the softmax warps; one warp for TMA (16-token pages through the block
// table, 8 boxes each of K and V a tile); one thread for the MMAs. S(n+1) is
// issued as soon as S(n) has been read into registers, so it runs under the
// softmax of tile n, and PV(n) under the first half of that of tile n + 1.
//
// Bound: HBM up to 4 rows; with 8 also the softmax's own instructions. 16 sequences of
// 16384 tokens (537 MB): 1 to 4 rows 87 us (6.2 TB/s), 8 rows 99 us (5.4 TB/s; issue
// slots 51% used, tensor pipe 36%), two blocks an SM in both.
#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tree.cuh"

namespace attn {
namespace {

using namespace tc;

constexpr int kKeys = 128;                          // keys of a tile: M of S^T
constexpr int kPages = kKeys / ATTN_PAGE;
constexpr uint32_t kOperand = kKeys * kD * 2;       // 16 KB: a tile of K, of V, or an N atom of p
constexpr uint32_t kStageBytes = 2 * kOperand;
constexpr uint32_t kBox = ATTN_PAGE * 128;

constexpr int kCols = 16;                           // columns of a softmax thread
constexpr int kFlush = 4;                           // tiles between two flushes of O

constexpr int kStages = 2;
constexpr int kRowStride = kD + 4;                  // floats, for rows written a row a thread

template <int R>
struct Lay {
  static constexpr int kParts = R / kCols;          // warps on one lane quarter
  static constexpr int kSoft = 4 * kParts;          // softmax warps
  static constexpr int kTmaWarp = kSoft, kMmaWarp = kSoft + 1;
  static constexpr int kThreads = 32 * (kSoft + 2);
  static constexpr int kBlocks = 2;                 // per SM
  static constexpr int kN = 3 * R;
  static constexpr uint32_t kColS = 0, kColO = 2 * R;                // two S buffers, then O's three terms
  static constexpr uint32_t kTmem = R == 32 ? 256 : 128;
  static constexpr uint32_t kSmemQ = kStages * kStageBytes;          // [3 R rows][128 bytes]
  static constexpr uint32_t kSmemP = kSmemQ + kN * 128;
  // O so far, [R][64] fp32, in the bytes that the last atom of p leaves free in
  // each of its 128 rows (2 R of 128: just as many), so that two blocks fit an SM.
  static constexpr uint32_t kFree = 2 * R;
  static constexpr uint32_t kSmemAcc = kSmemP + ((kN + 63) / 64 - 1) * kOperand;
  static constexpr uint32_t kSmemMask = kSmemAcc + kOperand;
  static_assert(kKeys * kFree == R * kD * 4 && (kN % 64) * 2 + kFree <= 128 && kSmemP % 1024 == 0, "acc");
  static constexpr uint32_t kSmemMax = kSmemMask + (R / 4) * 8;      // [4 quarters][R], then [R] for the end
  static constexpr uint32_t kSmemEnds = kSmemMax + 5 * R * 4;        // [R] (log2 maximum, sum)
  static constexpr uint32_t kSmemBar = kSmemEnds + R * 8;
  static constexpr int kNumBars = 4 * kStages + 7;
  static constexpr uint32_t kSmemWords = kSmemBar + kNumBars * 8;    // TMEM address, abort flag, odd rows (2), fresh (2), issued (2)
  static constexpr uint32_t kSmemAlloc = kSmemWords + 32 + 1024;
  static_assert(kBlocks * (kSmemAlloc + 1024) <= 233472, "shared memory of an SM");
  static_assert(kColO + kN <= kTmem && kBlocks * kTmem <= 512, "TMEM layout");
  static_assert(R * kRowStride * 4 <= kStages * kStageBytes, "the rows fit the ring");
};

// kind::f16, bf16 operands, fp32 accumulate; A K-major (S) or MN-major (PV).
__host__ __device__ constexpr uint32_t idesc_tree(int M, int N, bool mn_major) {
  return idesc_bf16(M, N, mn_major) | (mn_major ? 1u << 15 : 0u);
}

__device__ __forceinline__ float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Where column j of dim d is kept.
template <int R>
__device__ __forceinline__ float* acc_at(uint8_t* smem, int j, int d) {
  constexpr uint32_t kFree = Lay<R>::kFree;
  const uint32_t at = (uint32_t)(j * kD + d) * 4u;
  return reinterpret_cast<float*>(smem + Lay<R>::kSmemAcc + sw128(at / kFree * 128u + 128u - kFree + at % kFree));
}

template <int R, bool kFault>
__global__ void __launch_bounds__(Lay<R>::kThreads, Lay<R>::kBlocks)
tree_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const TreeArgs a) {
  using L = Lay<R>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: descriptors in uniform registers
  if (warp == L::kTmaWarp && lane < 2) tma_prefetch_desc(lane ? &mv : &mk);
  follow();
  const int s = blockIdx.x, head = blockIdx.y % kHKV, rt = blockIdx.y / kHKV, b = blockIdx.z;

  // The table's first entries are on their way while the lengths are, as of a
  // sequence as long as the call allows: an entry past the sequence is read and not
  // used.
  const int first_page = s * (a.split_len / ATTN_PAGE) + lane;
  int first_entries = -1;
  if (warp == L::kTmaWarp && first_page < a.max_blocks)
    first_entries = fetch(a.table + (size_t)b * a.max_blocks + first_page);
  const Seq seq = load_seq(a, b);
  const int i0 = rt * (R / 4);  // the block's first drafted row
  const int nrows = min(R / 4, seq.rows - i0);
  const int len = segment_len(a, seq), k0 = s * len;
  const int k1 = min(k0 + len, seq.keys);
  if (!seq.ok && s == 0 && tid == 0) record_error(a.err, kDevErrBounds);
  if (nrows <= 0) return;
  if (k0 >= k1 && !a.cluster) {
    // Past the sequence: the merge counts its segments from the lengths. A
    // sequence without any key (only a refused one) gets zeros.
    if (s == 0)
      for (int e = tid; e < nrows * kGroup * kD; e += L::kThreads)
        a.out[((size_t)(seq.first + i0 + e / (kGroup * kD)) * kHQ + head * kGroup) * kD + e % (kGroup * kD)] = 0.f;
    return;
  }
  const bool whole = !a.cluster && seq.keys <= a.split_len;  // one segment: the output is written here
  const int ntiles = max(0, (k1 - k0 + kKeys - 1) / kKeys);

  uint64_t* const kfull = reinterpret_cast<uint64_t*>(smem + L::kSmemBar);  // [stage] K landed
  uint64_t* const vfull = kfull + kStages;                                  // [stage] V landed
  uint64_t* const kempty = vfull + kStages;                                 // [stage] S done with K
  uint64_t* const vempty = kempty + kStages;                                // [stage] PV done with V
  uint64_t* const sfull = vempty + kStages;                                // [2] S written
  uint64_t* const sread = sfull + 2;                                       // [2] S read into registers
  uint64_t* const pfull = sread + 2;                                       // p written (and O rescaled)
  uint64_t* const odone = pfull + 1;                                       // PV complete
  uint64_t* const drain = odone + 1;                                       // MMAs in flight on abort
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + L::kSmemWords);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);
  uint32_t* const odd = words + 2;                 // [2] drafted rows whose value is not finite
  volatile uint32_t* const fresh = words + 4;      // [2] tile n starts O anew, at n % 2
  volatile uint32_t* const issued = words + 6;     // [2] tiles of K and of V loaded
  unsigned long long* const masks = reinterpret_cast<unsigned long long*>(smem + L::kSmemMask);
  float2* const ends = reinterpret_cast<float2*>(smem + L::kSmemEnds);
  const Wait wait{a.err, a.timeout_ns, abort_flag};

  const int* const trow = a.table + (size_t)b * a.max_blocks;

  // ---- bf16 pages: one warp, TMA boxes of a page each; 8 lanes load the 8 pages
  // of a tile of K, or of V. Lane l holds the table's entry of page l of a group
  // of four tiles, for V's group and for the next.
  int entries = -1, entries_next = -1, group = 0, ahead = 0;
  auto entry_at = [&](int g) -> int {
    const int t = k0 + g * 4 * kKeys + lane * ATTN_PAGE;
    return t < k1 ? fetch(trow + t / ATTN_PAGE) : -1;
  };
  auto load = [&](const CUtensorMap* map, uint64_t* full, uint32_t operand, int n) {
    const int st = n % kStages;
    int page = __shfl_sync(0xffffffffu, (n >> 2) == group ? entries : entries_next, (n & 3) * kPages + (lane & 7));
    const bool has = lane < kPages && k0 + n * kKeys + lane * ATTN_PAGE < k1;
    if (has && (page < 0 || page >= a.num_pages)) {
      record_error(a.err, kDevErrBounds);
      page = a.num_pages;  // past the pool's end: reads as zeros
    }
    const unsigned boxes = __popc(__ballot_sync(0xffffffffu, has));
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[st], boxes * kBox);
      issued[operand != 0] = n + 1;
    }
    __syncwarp();
    if (has && !(operand == 0 && withheld<kFault>(a, s, n)))
      tma_load_2d(smem + st * kStageBytes + operand + lane * kBox, map, &full[st], head * kD, page * ATTN_PAGE);
  };
  auto load_next = [&]() -> bool {  // K(ahead + 1), whose stage is free earlier, then V(ahead)
    const int n = ahead;
    if (n + 1 < ntiles) {
      if (n + 1 >= kStages && !wait.warp(&kempty[(n + 1) % kStages], ((n + 1) / kStages - 1) & 1)) return false;
      load(&mk, kfull, 0, n + 1);
    }
    if (n >= kStages && !wait.warp(&vempty[n % kStages], (n / kStages - 1) & 1)) return false;
    load(&mv, vfull, kOperand, n);
    ++ahead;
    if ((ahead >> 2) != group) {
      group = ahead >> 2;
      entries = entries_next;
      entries_next = entry_at(group + 1);
    }
    return true;
  };

  if (warp == L::kTmaWarp) {
    for (int i = lane; i < L::kNumBars; i += 32)
      mbar_init(&kfull[i], &kfull[i] >= sread && &kfull[i] < odone ? L::kSoft : 1);  // sread and pfull: every softmax warp
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      odd[0] = odd[1] = 0;
      issued[0] = issued[1] = 0;
    }
    __syncwarp();
    // The first tile is on its way before the block has met.
    entries = len == a.split_len ? first_entries : entry_at(0);
    entries_next = entry_at(1);
    if (ntiles > 0) load(&mk, kfull, 0, 0);
  } else if (warp == L::kMmaWarp) {
    tmem_alloc(words, L::kTmem);
    tmem_relinquish();
  } else {
    // q's terms: row t R + r of 128 bytes holds term t of row r.
    for (int e = tid; e < R * 8; e += 32 * L::kSoft) {  // (row, 8 dims)
      const int r = e >> 3, c8 = e & 7, i = r >> 2;
      float x[8];
      if (i < nrows) {
        const float4* src = reinterpret_cast<const float4*>(
            a.q + ((size_t)(seq.first + i0 + i) * kHQ + head * kGroup + (r & 3)) * kD + c8 * 8);
        const float4 u = fetch(src), v = fetch(src + 1);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = 0.f;
      }
      uint32_t w[3][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) split3_cut(x[2 * k], x[2 * k + 1], w[0][k], w[1][k], w[2][k]);
#pragma unroll
      for (int t = 0; t < 3; ++t)
        *reinterpret_cast<uint4*>(smem + L::kSmemQ + sw128((uint32_t)(t * R + r) * 128u + c8 * 16u)) =
            make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
    }
    for (int i = tid; i < R / 4; i += 32 * L::kSoft)
      masks[i] = i >= nrows ? 0ull
                 : a.masks  ? (unsigned long long)fetch(a.masks + seq.first + i0 + i)
                            : ~0ull >> (63 - (i0 + i));
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = words[0];

  if (warp == L::kTmaWarp) {
    while (ahead < ntiles && load_next()) {
    }
    __syncwarp();
  } else if (warp == L::kMmaWarp) {
    constexpr uint32_t kIdS = idesc_tree(128, R, false), kIdPV = idesc_tree(64, L::kN, true);
    const uint32_t base = smem_u32(smem);
    const uint64_t qd = sdesc_sw128(base + L::kSmemQ), pd = sdesc_sw128_mn(base + L::kSmemP, kOperand);
    auto issue_s = [&](int n) -> bool {
      const int st = n % kStages;
      if (!wait.warp(&kfull[st], (n / kStages) & 1)) return false;
      if (n > 1 && !wait.warp(&sread[n & 1], ((n >> 1) - 1) & 1)) return false;  // S(n - 2) is in registers
      tc_fence_after();
      const uint64_t kd = sdesc_sw128(base + st * kStageBytes);
      const uint32_t dst = tmem + L::kColS + (n & 1) * R;
      if (elect()) {
        // The smallest term first: only the last four accumulations are at the
        // score's own size.
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            mma_f16_ss(dst, kd + x * 2, qd + t * (R * 8) + x * 2, kIdS, t < 2 || x > 0);
        mma_commit(&sfull[n & 1]);
        mma_commit(&kempty[st]);
      }
      __syncwarp();
      return true;
    };
    bool ok = ntiles == 0 || issue_s(0);
    for (int n = 0; ok && n < ntiles; ++n) {
      if (n + 1 < ntiles && !(ok = issue_s(n + 1))) break;
      const int st = n % kStages;
      if (!(ok = wait.warp(pfull, n & 1) && wait.warp(&vfull[st], (n / kStages) & 1))) break;
      tc_fence_after();
      const uint64_t vd = sdesc_sw128_mn(base + st * kStageBytes + kOperand);
      const uint32_t old = n > 0 && !fresh[n & 1];
      if (elect()) {
#pragma unroll
        for (int x = 0; x < 8; ++x)  // 16 keys a step: 2048 bytes of rows
          mma_f16_ss(tmem + L::kColO, vd + x * 128, pd + x * 128, kIdPV, x > 0 ? 1u : old);
        mma_commit(&vempty[st]);
        mma_commit(odone);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------- softmax
    const int quarter = warp & 3, part = warp >> 2;
    const int key = quarter * 32 + lane;       // this thread's key of a tile
    const int col0 = part * kCols;             // its first column
    const uint32_t lane_tmem = tmem + ((uint32_t)(quarter * 32) << 16);
    constexpr int kMeet = 32 * L::kSoft;
    float* const maxima = reinterpret_cast<float*>(smem + L::kSmemMax);
    const int d = quarter * 16 + lane;         // lanes 0-15 hold the dims of O^T
    float sum[kCols], neg[kCols];  // this key's share of the sums; minus the references
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
      sum[j] = 0.f;
      neg[j] = -kUnseen;
    }
    float ref = kUnseen;  // lane j (and 16 + j): the reference of column col0 + j
    bool failed = false, kept = false;  // kept: acc holds something
    // Eight columns of O^T at this thread's dim, from tensor memory: the three
    // terms added, the smallest first.
    auto read_o = [&](int h, float (&o)[8]) {
      float o1[8];
      tmem_ld8(lane_tmem + L::kColO + 2 * R + col0 + h, o);
      tmem_ld8(lane_tmem + L::kColO + R + col0 + h, o1);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += o1[j];
      tmem_ld8(lane_tmem + L::kColO + col0 + h, o1);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += o1[j];
    };

    int n = 0;
    for (; n < ntiles; ++n) {
      failed |= !wait.warp(&sfull[n & 1], (n >> 1) & 1);
      tc_fence_after();
      const uint32_t s_tmem = lane_tmem + L::kColS + (n & 1) * R + col0;
      float x[kCols];
      tmem_ld16(s_tmem, x);
      tmem_wait_ld();
      const int pos = k0 + n * kKeys + key;
      const int at = pos - seq.ctx;  // >= 0: a drafted row, or a slot past the last
      const bool tail = k0 + (n + 1) * kKeys > seq.ctx;
      uint32_t hidden = 0;  // columns that do not see this key
      if (tail) {
        if (at >= 0) {
          const bool past = pos >= k1;
          hidden = past ? ~0u : 0u;
          if (!past)
#pragma unroll
            for (int i = 0; i < kCols / 4; ++i)
              if (!(masks[col0 / 4 + i] >> at & 1)) hidden |= 15u << (4 * i);
          {
            // The value row of this key: zeros past the last key (its slot may hold
            // anything), and no infinity or NaN of a drafted row into a product
            // with the zero probability of a row that does not see it.
            if (!wait(&vfull[n % kStages], (n / kStages) & 1)) failed = true;
            uint8_t* v = smem + (n % kStages) * kStageBytes + kOperand;
            for (int c8 = part; c8 < 8; c8 += L::kParts) {
              uint4* p = reinterpret_cast<uint4*>(v + sw128((uint32_t)key * 128u + c8 * 16u));
              uint4 u = past ? make_uint4(0, 0, 0, 0) : *p;
              uint32_t* w = reinterpret_cast<uint32_t*>(&u);
              bool bad = past;
  #pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((w[k] & 0x7f80u) == 0x7f80u) w[k] &= 0xffff0000u, bad = true;
                if ((w[k] & 0x7f800000u) == 0x7f800000u) w[k] &= 0xffffu, bad = true;
              }
              if (bad) *p = u;
              if (bad && !past) atomicOr(odd + (at >> 5), 1u << (at & 31));
            }
          }
        }
        failed = __any_sync(0xffffffffu, failed);
      }
      // Scores relative to the references, in log2 units. Does one pass 2^8?
      auto relative = [&]() -> float {
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < kCols; j += 2) {
          fma2(x[j], x[j + 1], x[j], x[j + 1], kTreeC, kTreeC, neg[j], neg[j + 1]);
          if (tail) {
            if (hidden >> j & 1) x[j] = -INFINITY;
            if (hidden >> (j + 1) & 1) x[j + 1] = -INFINITY;
          }
          most = max3(most, x[j], x[j + 1]);
        }
        return most;
      };
      int over = 1;  // of the first tile it is known
      if (n > 0) {
        const float most = relative();
        if (meet(kMeet, __any_sync(0xffffffffu, most > kTreeStale), failed, lane, &over)) {
          failed = true;
          break;
        }
        if (over) {
          tmem_ld16(s_tmem, x);  // the scores again
          tmem_wait_ld();
        }
      }
      float alpha = 1.f;
      if (over) {
        float mine = -INFINITY;
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const float m = warp_max(hidden >> j & 1 ? -INFINITY : x[j]);
          if ((lane & 15) == j) mine = m;
        }
        const int c = col0 + (lane & 15);
        if (lane < kCols) maxima[quarter * R + c] = mine;
        meet(kMeet);
        mine = fmaxf(fmaxf(maxima[c], maxima[R + c]), fmaxf(maxima[2 * R + c], maxima[3 * R + c]));
        const float next = fmaxf(ref, mine * kTreeC);
        alpha = ex2(ref - next);
        ref = next;
#pragma unroll
        for (int j = 0; j < kCols; ++j) neg[j] = -__shfl_sync(0xffffffffu, next, j);
        if (n > 0) {
#pragma unroll
          for (int j = 0; j < kCols; ++j) sum[j] *= __shfl_sync(0xffffffffu, alpha, j);
        }
        relative();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sread[n & 1]);
      uint32_t w[3][kCols / 2];
#pragma unroll
      for (int j = 0; j < kCols; j += 2) {
        const float p0 = ex2(x[j]), p1 = ex2(x[j + 1]);
        add2(sum[j], sum[j + 1], sum[j], sum[j + 1], p0, p1);
        split3(p0, p1, w[0][j / 2], w[1][j / 2], w[2][j / 2]);
      }
      // PV(n-1) has read p, and its O is complete.
      if (n > 0) {
        failed |= !wait.warp(odone, (n - 1) & 1);
        if (over || n % kFlush == 0) {
          // O moves to fp32 sums that round to nearest, with the references' change.
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < kCols; h += 8) {
            float o[8];
            read_o(h, o);
            if (kept && lane < 16) {
              float old[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) old[j] = *acc_at<R>(smem, col0 + h + j, d);
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] += old[j];
            }
            if (over) {
#pragma unroll
              for (int j = 0; j < 8; ++j) o[j] *= __shfl_sync(0xffffffffu, alpha, h + j);
            }
            if (lane < 16) {
#pragma unroll
              for (int j = 0; j < 8; ++j) *acc_at<R>(smem, col0 + h + j, d) = o[j];
            }
          }
          kept = true;
        }
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) {
        const int c = t * R + col0;  // 64 columns an atom, 8 a 16-byte chunk
        uint8_t* row = smem + L::kSmemP + (c >> 6) * kOperand;
#pragma unroll
        for (int k = 0; k < kCols / 8; ++k)
          *reinterpret_cast<uint4*>(row + sw128((uint32_t)key * 128u + ((c & 63) / 8 + k) * 16u)) =
              make_uint4(w[t][4 * k], w[t][4 * k + 1], w[t][4 * k + 2], w[t][4 * k + 3]);
      }
      if (tid == 0) fresh[n & 1] = over || n % kFlush == 0;
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
    }

    // ------------------------------------------------------------ epilogue
    {
      // Sums over the warp's keys: halving the columns a lane holds each round,
      // lanes j and 16 + j end with column col0 + j.
#pragma unroll
      for (int w = 8; w >= 1; w >>= 1)
#pragma unroll
        for (int j = 0; j < w; ++j) {
          const bool up = lane & w;
          const float give = up ? sum[j] : sum[j + w], keep = up ? sum[j + w] : sum[j];
          sum[j] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
      const float l = sum[0] + __shfl_xor_sync(0xffffffffu, sum[0], 16);
      const int c = col0 + (lane & 15);
      int over;
      if (!failed && ntiles > 0) failed = !wait.warp(odone, (ntiles - 1) & 1);
      // The maxima of the last tile may still be read: meet before they become sums.
      if (meet(kMeet, false, failed, lane, &over)) goto done;
      if (lane < kCols) maxima[quarter * R + c] = l;
      tc_fence_after();
      float o[kCols];
#pragma unroll
      for (int h = 0; h < kCols; h += 8) read_o(h, reinterpret_cast<float (&)[8]>(o[h]));
      if (kept && lane < 16) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) o[j] += *acc_at<R>(smem, col0 + j, d);
      }
      unsigned long long rest = ((unsigned long long)odd[1] << 32) | odd[0];
      while (rest) {  // drafted values that are not finite reach the rows that see them
        const int j0 = __ffsll((long long)rest) - 1;
        rest &= rest - 1;
        const int page = fetch(trow + (seq.ctx + j0) / ATTN_PAGE);
        if (lane < 16 && page >= 0 && page < a.num_pages) {
          const size_t at = (((size_t)page * ATTN_PAGE + (seq.ctx + j0) % ATTN_PAGE) * kHKV + head) * kD + d;
          const float v = __uint_as_float((uint32_t)fetch(static_cast<const uint16_t*>(a.v_pages) + at) << 16);
          if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u)
#pragma unroll
            for (int j = 0; j < kCols; ++j)
              if (masks[(col0 + j) >> 2] >> j0 & 1) o[j] += v;
        }
      }
      // Rows to shared memory, so that they leave in 16-byte pieces. (p's atoms
      // are free, and so is what the tiles occupied.)
      float* const rows = reinterpret_cast<float*>(smem);  // [R][kRowStride]
      if (lane < 16) {
#pragma unroll
        for (int j = 0; j < kCols; ++j) rows[(col0 + j) * kRowStride + d] = ntiles > 0 ? o[j] : 0.f;
      }
      if (quarter == 0 && lane < kCols) maxima[4 * R + c] = ref;
      meet(kMeet);
      const size_t at0 = (size_t)(seq.first + i0) * kHQ + head * kGroup;  // row r: + (r / 4) * 32 + r % 4
      float2* const mls = reinterpret_cast<float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD);
#pragma unroll 1
      for (int e = tid; e < nrows * kGroup * 16; e += kMeet) {  // (row, 4 dims)
        const int r = e >> 4, d4 = (e & 15) * 4;
        const float sl = (maxima[r] + maxima[R + r]) + (maxima[2 * R + r] + maxima[3 * R + r]);
        if (a.cluster) {
          if (d4 == 0) ends[r] = make_float2(maxima[4 * R + r] == kUnseen ? -INFINITY : maxima[4 * R + r], sl);
          continue;
        }
        float4 y = *reinterpret_cast<const float4*>(rows + r * kRowStride + d4);
        const size_t at = at0 + (r >> 2) * kHQ + (r & 3);
        if (whole) {
          const float inv = sl == 0.f ? 0.f : 1.f / sl;  // no key: zeros
          y = make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
          *reinterpret_cast<float4*>(a.out + at * kD + d4) = y;
        } else {
          *reinterpret_cast<float4*>(a.parts + (at * a.splits + s) * kD + d4) = y;
          if (d4 == 0) {
            const float m = maxima[4 * R + r];
            mls[at * a.splits + s] = make_float2(m == kUnseen ? -INFINITY : m, sl);
          }
        }
      }
    }
  done:;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (warp == L::kTmaWarp) {  // before the block's shared memory is released
      drain_copies(kfull, kStages, issued[0], a.timeout_ns);
      drain_copies(vfull, kStages, issued[1], a.timeout_ns);
    } else if (warp == L::kMmaWarp) {
      drain_products(drain, a.timeout_ns);
    } else if (!whole) {  // after a failed wait the segment counts as empty
      float2* const mls = reinterpret_cast<float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD);
      for (int r = tid; r < nrows * kGroup; r += 32 * L::kSoft) {
        if (a.cluster) ends[r] = make_float2(-INFINITY, 0.f);
        else
          mls[((size_t)(seq.first + i0 + (r >> 2)) * kHQ + head * kGroup + (r & 3)) * a.splits + s] =
              make_float2(-INFINITY, 0.f);
      }
    }
    __syncthreads();
  }
  if (warp == L::kMmaWarp) tmem_dealloc(tmem, L::kTmem);
  if (a.cluster && warp < L::kSoft)
    cluster_merge(a, seq.first + i0, nrows, head, reinterpret_cast<const float*>(smem), kRowStride, ends, tid,
                  32 * L::kSoft);
}

}  // namespace

template <int R>
TreeVariant variant() {
  using L = Lay<R>;
  return {tree_tc_kernel<R, false>, tree_tc_kernel<R, true>, R / 4, L::kThreads, L::kSmemAlloc, L::kBlocks, false, 0, 5,
          2};
}

TreeVariant tree_tc_variant(int tokens) { return tokens == 4 ? variant<16>() : variant<32>(); }

}  // namespace attn
