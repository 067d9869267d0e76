// tree_wide.cu -- the drafted-tree attention of tree.cu for wide trees, on the
// tcgen05 tensor cores with the query rows on the M side: 32 drafted rows x the
// 4 query heads of a KV head fill the 128 lanes of tensor memory, a thread owns
// one row, and nothing of the softmax crosses threads.
//
// Tiles of 64 keys go in turn to two softmax groups of four warps (tile n to
// group n % 2), each with its own reference maximum, sum and accumulator, so one
// group's softmax runs under the other's products; the two partials merge at the
// end like two segments. The
// tensor core's accumulation does not round to nearest: O of a tile starts at
// zero, and the row's thread adds it to fp32 registers, rounded to nearest. A
// reference that moves therefore costs a product in registers and no trip to
// tensor memory.
//
//   bf16 pages (K and V as stored, q and p in three bf16 terms):
//     S  = (q3, q2, q1) K^T        3 x 4 MMAs of 128 x 64 x 16
//     O  = (p3, p2, p1) V          3 x 4 MMAs of 128 x 64 x 16
//   fp32 pages (x = hi + lo, hi a tf32 value; of K and V four converter warps round
//   it in place in each landed tile and write lo next to it):
//     S  = q_lo K + q_hi K_lo + q_hi K       3 x 8 MMAs of 128 x 64 x 8
//     O  = p_lo V + p_hi V_lo + p_hi V       3 x 8 MMAs of 128 x 64 x 8
// q and p are tensor-memory operands (p overwrites the S it came from), K a
// K-major and V an MN-major shared-memory operand as TMA lays them down.
//
// Roles: warps 0-3 and 4-7 softmax; (fp32) 8-11 converters; one warp each for the
// TMA of K and of V (16-token pages through the block table); one each to issue
// the products S and O.
//
// Bound: the tensor pipe, at 31.5 cycles an MMA, on as many SMs as there are blocks.
// 16 sequences of 16384 tokens are 128 blocks of 152 places: 32 rows on bf16 pages 140
// us (537 MB, 3.8 TB/s; 206 GFLOP of term products, 1.47 PFLOP/s; pipe active 77% on
// those SMs, the softmax of a tile as long as its products), 16 rows on fp32 pages 221
// us (4.9 TB/s; pipe active 95%, half of its lanes without rows). 64 rows of one
// sequence of 131071 tokens on bf16 pages: 144 blocks, 132 us. Those are short bursts:
// back to back for long they meet the power limit and take 154, 235 and 144 us, and up
// to 4 % more on another card. (Registers are full: the bf16 kernel, at 168, stores 36
// bytes a thread to local memory and loads 68, the fp32 one, launched with 128, 12 and
// 20.) A grid of one block an SM that shares all tiles evenly, units cut where a
// block's share ends, was built on an earlier form and ran 252 and 157 us for its 254
// and 146: what a second unit costs a block (q again, an empty pipeline, two partials
// through memory) is what the idle SMs gave. 16 rows on all 128 lanes, p's hi on one
// half and its lo on the other, two products instead of three for fp32 pages: 227 us,
// the softmax done twice.
#include <cuda.h>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tree.cuh"

namespace attn {
namespace {

using namespace tc;

constexpr int kRows = 32;                  // drafted rows of a block
constexpr int kKeys = 64;                  // keys of a tile
constexpr int kPages = kKeys / ATTN_PAGE;
constexpr int kSoft = 8;                   // softmax warps, two groups of four
constexpr uint32_t kHalf = kKeys * 128;    // 64 rows of 128 bytes
constexpr int kRowStride = kD + 4;         // floats, for rows written a row a thread

template <bool kF32>
struct Wide {
  static constexpr int kConvWarp = kSoft, kConvWarps = kF32 ? 4 : 0;
  static constexpr int kKWarp = kSoft + kConvWarps, kVWarp = kKWarp + 1, kQkWarp = kKWarp + 2, kPvWarp = kKWarp + 3;
  static constexpr int kThreads = 32 * (kPvWarp + 1);
  static constexpr uint32_t kOperand = kF32 ? 2 * kHalf : kHalf;     // a tile of K or V as stored
  static constexpr uint32_t kStageBytes = (kF32 ? 4 : 2) * kOperand; // K (K lo) V (V lo)
  static constexpr uint32_t kV = (kF32 ? 2 : 1) * kOperand;
  static constexpr int kStages = kF32 ? 3 : 8;
  // Tensor memory: q's terms, then three buffers of S (p overwrites it; with fp32
  // pages its lo part lies beside them, a buffer a group), so S(n + 2) runs ahead of
  // PV(n) and a group finds it ready; then O, one a group, or with fp32 pages one
  // that a group reads as soon as it is complete, before the other's product.
  static constexpr int kBufs = 3, kOs = kF32 ? 1 : 2;
  static constexpr uint32_t kColQ = 0, kColS = kF32 ? 128 : 96, kBufCols = kF32 ? 64 : 96;
  static constexpr uint32_t kColLo = kColS + kBufs * kBufCols;
  static constexpr uint32_t kColO = kColLo + (kF32 ? 2 * kKeys : 0);
  static constexpr uint32_t kSmemMask = kStages * kStageBytes;
  static constexpr uint32_t kSmemMl = kSmemMask + kRows * 8;         // [2 groups][128 rows] (reference, sum)
  static constexpr uint32_t kSmemEnds = kSmemMl + 2 * 128 * 8;       // [128 rows] the same of both groups together
  static constexpr uint32_t kSmemBar = kSmemEnds + 128 * 8;
  // In the ring once it is idle: the groups' exchange, then the block's rows.
  static constexpr uint32_t kSmemRows = 2 * 128 * 32 * 4;
  static constexpr int kNumBars = 6 * kStages + 2 * kBufs + 4 + 6;
  static constexpr uint32_t kSmemWords = kSmemBar + kNumBars * 8;    // TMEM address, abort flag, odd rows (2), issued (2)
  static constexpr uint32_t kSmemAlloc = kSmemWords + 24 + 1024;
  static_assert(kSmemAlloc <= 232448, "exceeds the 227 KB per-block shared memory limit");
  static_assert(kColO + kOs * kD <= 512, "TMEM layout");
  static_assert(kSmemRows + 128 * kRowStride * 4 <= kStages * kStageBytes, "the exchange and the rows fit the ring");
};

template <bool kF32, bool kFault>
__global__ void __launch_bounds__(Wide<kF32>::kThreads, 1)
tree_wide_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const TreeArgs a) {
  using L = Wide<kF32>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (warp == L::kKWarp && lane == 0) tma_prefetch_desc(&mk);
  if (warp == L::kVWarp && lane == 0) tma_prefetch_desc(&mv);
  follow();
  const int s = blockIdx.x, head = blockIdx.y % kHKV, rt = blockIdx.y / kHKV, b = blockIdx.z;

  // The table's first entries are on their way while the lengths are, as of a
  // sequence as long as the call allows: an entry past the sequence is read and not
  // used.
  const int first_page = s * (a.split_len / ATTN_PAGE) + lane;
  int first_entries = -1;
  if ((warp == L::kKWarp || warp == L::kVWarp) && first_page < a.max_blocks) first_entries = fetch(a.table + (size_t)b * a.max_blocks + first_page);
  const Seq seq = load_seq(a, b);
  const int i0 = rt * kRows;  // the block's first drafted row
  const int nrows = min(kRows, seq.rows - i0);
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
  const int quarters = (nrows * kGroup + 31) / 32;  // lane quarters that hold rows

  uint64_t* const kfull = reinterpret_cast<uint64_t*>(smem + L::kSmemBar);  // [stage] K landed
  uint64_t* const vfull = kfull + kStages;                                  // [stage] V landed
  uint64_t* const kready = vfull + kStages;                                 // [stage] K lo written (fp32)
  uint64_t* const vready = kready + kStages;                                // [stage] V lo written (fp32)
  uint64_t* const kempty = vready + kStages;                                // [stage] S done with K
  uint64_t* const vempty = kempty + kStages;                                // [stage] PV done with V
  uint64_t* const sfull = vempty + kStages;                                 // [buffer] S written
  uint64_t* const sfree = sfull + L::kBufs;                                 // [buffer] PV done with its p
  uint64_t* const pfull = sfree + L::kBufs;                                        // [group] p written, O read
  uint64_t* const odone = pfull + 2;                                        // [group] PV complete
  uint64_t* const qready = odone + 2;                                       // q's terms in tensor memory
  uint64_t* const drain = qready + 1;                                       // [2] MMAs in flight on abort
  uint64_t* const oread = drain + 2;                                        // (fp32) O read
  uint64_t* const pissued = oread + 1;                                      // (fp32) [2] O of the group's tile issued
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + L::kSmemWords);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);
  uint32_t* const odd = words + 2;  // [2] drafted rows whose value is not finite
  volatile uint32_t* const issued = words + 4;  // [2] tiles of K and of V loaded
  unsigned long long* const masks = reinterpret_cast<unsigned long long*>(smem + L::kSmemMask);
  float2* const ends = reinterpret_cast<float2*>(smem + L::kSmemEnds);
  const Wait wait{a.err, a.timeout_ns, abort_flag};

  // The TMA warps, one for K and one for V (a box of 16 rows costs its warp about
  // 100 cycles): lanes load the four pages of a tile, for fp32 in two halves of 32
  // dims. Lane l holds the table's entry of page l of a group of eight tiles.
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  int entries = -1, entries_next = -1;
  auto entry_at = [&](int g) -> int {
    const int t = k0 + g * 8 * kKeys + lane * ATTN_PAGE;
    return t < k1 ? fetch(trow + t / ATTN_PAGE) : -1;
  };
  auto load = [&](const CUtensorMap* map, uint64_t* full, uint32_t operand, int n) {
    const int st = n % kStages, p = lane & (kPages - 1), half = lane / kPages;
    int page = __shfl_sync(0xffffffffu, entries, (n & 7) * kPages + p);
    const int pages = min(kPages, (k1 - k0 - n * kKeys + ATTN_PAGE - 1) / ATTN_PAGE);
    const bool has = half < (kF32 ? 2 : 1) && p < pages;
    if (has && (page < 0 || page >= a.num_pages)) {
      record_error(a.err, kDevErrBounds);
      page = a.num_pages;  // past the pool's end: reads as zeros
    }
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[st], pages * (kF32 ? 2 : 1) * (ATTN_PAGE * 128));
      issued[operand != 0] = n + 1;
    }
    __syncwarp();
    if (has && !(operand == 0 && withheld<kFault>(a, s, n)))
      tma_load_2d(smem + st * L::kStageBytes + operand + half * kHalf + p * (ATTN_PAGE * 128), map, &full[st],
                  head * kD + half * 32, page * ATTN_PAGE);
    if ((n & 7) == 7) {
      entries = entries_next;
      entries_next = entry_at((n >> 3) + 2);
    }
  };

  if (warp == L::kKWarp) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      const int kind = i / kStages;  // kfull, vfull, kready, vready, kempty, vempty, then the single ones
      mbar_init(&kfull[i], kind < 6 ? ((kind & ~1) == 2 && kF32 ? L::kConvWarps : 1)
                           : (&kfull[i] >= pfull && &kfull[i] < odone) || &kfull[i] == oread ? quarters
                           : &kfull[i] == qready                     ? kSoft
                                                                     : 1);
    }
    fence_mbar_init();
    if (lane == 0) {
      *abort_flag = 0;
      odd[0] = odd[1] = 0;
      issued[0] = issued[1] = 0;
    }
    __syncwarp();
    // The first tiles are on their way before the block has met.
    entries = len == a.split_len ? first_entries : entry_at(0);
    entries_next = entry_at(1);
    if (ntiles > 0) load(&mk, kfull, 0, 0);
  } else if (warp == L::kVWarp) {
    entries = len == a.split_len ? first_entries : entry_at(0);
    entries_next = entry_at(1);
  } else if (warp == L::kQkWarp) {
    tmem_alloc(words, 512);
    tmem_relinquish();
  } else if (warp < kSoft) {
    if (tid < kRows) {
      unsigned long long m = 0;
      if (tid < nrows)
        m = (a.masks ? (unsigned long long)fetch(a.masks + seq.first + i0 + tid) : ~0ull >> (63 - (i0 + tid))) &
            (~0ull >> (64 - seq.rows));  // bits past the sequence's rows see nothing
      masks[tid] = m;
    }
  }
  // A softmax thread's 32 dims (32 g ..) of its row of q are on their way before the
  // block has met.
  float x[32];
  if (warp < kSoft) {
    const int row = (warp & 3) * 32 + lane, i = row >> 2;
    const float* src =
        a.q + ((size_t)(seq.first + i0 + i) * kHQ + head * kGroup + (row & 3)) * kD + (warp >> 2) * 32;
#pragma unroll
    for (int k = 0; k < 32; k += 4) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < nrows) v = fetch(reinterpret_cast<const float4*>(src + k));
      x[k] = v.x, x[k + 1] = v.y, x[k + 2] = v.z, x[k + 3] = v.w;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = words[0];

  if (warp >= kSoft) {
    // fp32: the loaders give registers to the softmax warps (launched with 128
    // each: 8 warps x 168 + 4 x 88 + 4 x 80 = 16 x 126).
    if constexpr (kF32) {
      if (warp < L::kKWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
      else asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    }
    if (warp == L::kKWarp || warp == L::kVWarp) {
      const bool is_k = warp == L::kKWarp;
      uint64_t* const full = is_k ? kfull : vfull;
      uint64_t* const empty = is_k ? kempty : vempty;
      int n = is_k ? 1 : 0;
      for (; n < ntiles; ++n) {
        if (n >= kStages && !wait.warp(&empty[n % kStages], (n / kStages - 1) & 1)) break;
        load(is_k ? &mk : &mv, full, is_k ? 0 : L::kV, n);
      }
    } else if (warp == L::kQkWarp || warp == L::kPvWarp) {
      // Two issuers, so that one's waits and issue run under the other's. With fp32
      // pages S of a tile is issued after O of the one two before: in the pipe
      // behind it, or both would end late, and one group's softmax runs under both
      // (16 rows of 16 sequences of 16384 tokens: 219 us, and 238 in no order).
      const uint32_t base = smem_u32(smem);
      const bool qk = warp == L::kQkWarp;
      uint64_t* const go = (kF32 ? kready : kfull) + (qk ? 0 : kStages);  // K, or V, ready
      if (qk) {
        bool ok = ntiles == 0 || wait.warp(qready, 0);
        for (int n = 0; ok && n < ntiles; ++n) {
          const int st = n % kStages, buf = n % L::kBufs;
          if (!(ok = wait.warp(&go[st], (n / kStages) & 1) &&
                     (n < L::kBufs || wait.warp(&sfree[buf], (n / L::kBufs - 1) & 1)) &&
                     (!kF32 || n < 2 || wait.warp(&pissued[n & 1], ((n >> 1) - 1) & 1))))
            break;
          tc_fence_after();
          const uint64_t kd = sdesc_sw128(base + st * L::kStageBytes);
          const uint32_t d = tmem + L::kColS + buf * L::kBufCols, q = tmem + L::kColQ;
          if (elect()) {
            if constexpr (kF32) {
              constexpr uint32_t id = idesc_tf32(128, kKeys);
              constexpr uint64_t lo = L::kOperand >> 4;
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma_tf32_ts(d, q + 64 + x * 8, kd + (x >> 2) * (kHalf >> 4) + (x & 3) * 2, id, x > 0);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma_tf32_ts(d, q + x * 8, kd + lo + (x >> 2) * (kHalf >> 4) + (x & 3) * 2, id, 1);
#pragma unroll
              for (int x = 0; x < 8; ++x)
                mma_tf32_ts(d, q + x * 8, kd + (x >> 2) * (kHalf >> 4) + (x & 3) * 2, id, 1);
            } else {
              constexpr uint32_t id = idesc_bf16(128, kKeys, false);
#pragma unroll
              for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_f16_ts(d, q + t * 32 + x * 8, kd + x * 2, id, t < 2 || x > 0);
            }
            mma_commit(&sfull[buf]);
            mma_commit(&kempty[st]);
          }
          __syncwarp();
        }
      } else {
        for (int n = 0; n < ntiles; ++n) {
          const int st = n % kStages, g = n & 1, buf = n % L::kBufs;
          if (!wait.warp(&go[st], (n / kStages) & 1) || !wait.warp(&pfull[g], (n >> 1) & 1)) break;
          if (kF32 && n > 0 && !wait.warp(oread, (n - 1) & 1)) break;
          tc_fence_after();
          const uint32_t d = tmem + L::kColO + g % L::kOs * kD, p = tmem + L::kColS + buf * L::kBufCols;
          const uint32_t p_lo = tmem + L::kColLo + g * kKeys;
          const uint32_t vb = base + st * L::kStageBytes + L::kV;
          if (elect()) {
            if constexpr (kF32) {
              constexpr uint32_t id = idesc_tf32(128, kD, true);
              const uint64_t vd = sdesc_sw128a32_mn(vb, kHalf);
              constexpr uint64_t lo = L::kOperand >> 4;
#pragma unroll
              for (int x = 0; x < 8; ++x) mma_tf32_ts(d, p_lo + x * 8, vd + x * 64, id, x > 0);
#pragma unroll
              for (int x = 0; x < 8; ++x) mma_tf32_ts(d, p + x * 8, vd + lo + x * 64, id, 1);
#pragma unroll
              for (int x = 0; x < 8; ++x) mma_tf32_ts(d, p + x * 8, vd + x * 64, id, 1);
            } else {
              constexpr uint32_t id = idesc_bf16(128, kD, true);
              const uint64_t vd = sdesc_sw128_mn(vb);
#pragma unroll
              for (int t = 2; t >= 0; --t)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  mma_f16_ts(d, p + t * 32 + x * 8, vd + x * 128, id, t < 2 || x > 0);
            }
            mma_commit(&odone[g]);
            mma_commit(&sfree[buf]);
            mma_commit(&vempty[st]);
            if (kF32) mbar_arrive(&pissued[g]);
          }
          __syncwarp();
        }
      }
    } else if (kF32 && warp < L::kKWarp) {
      // hi(x), rounded to nearest, in place and lo = x - hi(x) at the same offset of
      // the next region, element by element. (Left as it landed, x would reach the
      // tensor core truncated: a remainder of twice the size and of x's own sign.)
      const int ctid = tid - 32 * L::kConvWarp;
      auto split = [&](uint8_t* at, float4 x) {
        const float4 h = make_float4(tf32_near(x.x), tf32_near(x.y), tf32_near(x.z), tf32_near(x.w));
        *reinterpret_cast<float4*>(at) = h;
        *reinterpret_cast<float4*>(at + L::kOperand) = make_float4(x.x - h.x, x.y - h.y, x.z - h.z, x.w - h.w);
      };
      auto convert_k = [&](int n) -> bool {
        const int st = n % kStages;
        uint8_t* const stage = smem + st * L::kStageBytes;
        if (!wait.warp(&kfull[st], (n / kStages) & 1)) return false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(stage + (ctid + (4 * h + i) * 128) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) split(stage + (ctid + (4 * h + i) * 128) * 16, x[i]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[st]);
        return true;
      };
      // K of the next tile first: its stage is free before V's, and the scores that
      // wait for it are what the softmax waits for.
      bool ok = ntiles == 0 || convert_k(0);
      for (int n = 0; ok && n < ntiles; ++n) {
        if (n + 1 < ntiles && !(ok = convert_k(n + 1))) break;
        const int st = n % kStages;
        uint8_t* const stage = smem + st * L::kStageBytes;
        if (!(ok = wait.warp(&vfull[st], (n / kStages) & 1))) break;
        const bool tail = k0 + (n + 1) * kKeys > seq.ctx;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const float4*>(stage + L::kV + (ctid + (4 * h + i) * 128) * 16);
          if (tail) {
            // Slots past the last key count as zeros, and no infinity or NaN of
            // a drafted row meets the zero probability of a row that does not
            // see it.
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int unit = ctid + (4 * h + i) * 128, pos = k0 + n * kKeys + ((unit >> 3) & (kKeys - 1));
              const int at = pos - seq.ctx;
              float* y = reinterpret_cast<float*>(&x[i]);
              bool bad = false;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (pos >= k1 || (at >= 0 && (__float_as_uint(y[k]) & 0x7f800000u) == 0x7f800000u)) {
                  y[k] = 0.f;
                  bad = true;
                }
              if (bad) *reinterpret_cast<float4*>(stage + L::kV + unit * 16) = x[i];
              if (bad && pos < k1) atomicOr(odd + (at >> 5), 1u << (at & 31));
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) split(stage + L::kV + (ctid + (4 * h + i) * 128) * 16, x[i]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&vready[st]);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- softmax
    if constexpr (kF32) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    constexpr int kMeet = 32 * kSoft;
    const int quarter = warp & 3, g = warp >> 2;
    const int row = quarter * 32 + lane;
    const bool active = quarter < quarters;
    const uint32_t lane_tmem = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t o_tmem = lane_tmem + L::kColO + g % L::kOs * kD;
    float ref = kUnseen, l0 = 0.f, l1 = 0.f;
    float o[kD];
#pragma unroll
    for (int i = 0; i < kD; ++i) o[i] = 0.f;
    bool failed = false;

    if (!active && ntiles > 0) {
      // Lanes without rows: zeros in q and p, or the tensor cores would spend power
      // on whatever tensor memory holds (16 rows of 16 sequences of 16384 tokens, a
      // thousand calls in a row: fp32 pages 272 to 255 us, bf16 150 to 137).
      float zero[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) zero[i] = 0.f;
      for (int c = g * 32; c < (int)L::kColO; c += 64) tmem_st32(lane_tmem + c, zero);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
    }
    if (active && ntiles > 0) {
      {  // q in its terms
        if constexpr (kF32) {
          float hi[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            hi[k] = tf32_near(x[k]);
            x[k] -= hi[k];
          }
          tmem_st32(lane_tmem + L::kColQ + g * 32, hi);
          tmem_st32(lane_tmem + L::kColQ + 64 + g * 32, x);
        } else {
          uint32_t w[3][16];
#pragma unroll
          for (int k = 0; k < 16; ++k) split3_cut(x[2 * k], x[2 * k + 1], w[0][k], w[1][k], w[2][k]);
#pragma unroll
          for (int t = 0; t < 3; ++t) tmem_st16(lane_tmem + L::kColQ + t * 32 + g * 16, w[t]);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(qready);
      }
      const unsigned long long mask = masks[row >> 2];

      // O of the group's previous tile, once it is complete, joins the row's sums.
      auto add_o = [&](int k) {
        failed |= !wait.warp(&odone[g], k & 1);
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < kD; h += 32) {
          float t[32];
          tmem_ld32(o_tmem + h, t);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) add2(o[h + i], o[h + i + 1], o[h + i], o[h + i + 1], t[i], t[i + 1]);
        }
        if (kF32) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(oread);
        }
      };

      int k = 0;  // the group's k-th tile
      for (int n = g; n < ntiles; n += 2, ++k) {
        // fp32: at once, the other group's product waits for it.
        if (kF32 && k > 0) add_o(k - 1);
        const int buf = n % L::kBufs;
        const uint32_t s_tmem = lane_tmem + L::kColS + buf * L::kBufCols;
        failed |= !wait.warp(&sfull[buf], (n / L::kBufs) & 1);
        tc_fence_after();
        float x[kKeys];
        tmem_ld32(s_tmem, *reinterpret_cast<float(*)[32]>(&x[0]));
        tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(&x[32]));
        tmem_wait_ld();
        const int t0 = k0 + n * kKeys;
        if (t0 + kKeys > seq.ctx) {  // drafted keys, or slots past the last
          const int at = t0 - seq.ctx;
          unsigned long long see = at >= 0 ? mask >> at : -at >= 64 ? ~0ull : (mask << -at) | (~0ull >> (64 + at));
          if (k1 - t0 < kKeys) see &= ~0ull >> (64 - (k1 - t0));
#pragma unroll
          for (int i = 0; i < kKeys; ++i)
            if (!(see >> i & 1)) x[i] = -INFINITY;
          if constexpr (!kF32) {
            // The tile's value rows: zeros past the last key, and no infinity or
            // NaN of a drafted row into a product with the zero probability of a
            // row that does not see it. The group's threads share the rows.
            failed |= !wait.warp(&vfull[n % kStages], (n / kStages) & 1);
            uint8_t* v = smem + (n % kStages) * L::kStageBytes + L::kV;
            for (int e = row; e < kKeys * 8; e += 32 * quarters) {
              const int key = e >> 3, pos = t0 + key;
              if (pos < seq.ctx) continue;
              uint4* p = reinterpret_cast<uint4*>(v + sw128((uint32_t)key * 128u + (e & 7) * 16u));
              uint4 u = pos >= k1 ? make_uint4(0, 0, 0, 0) : *p;
              uint32_t* w = reinterpret_cast<uint32_t*>(&u);
              bool bad = pos >= k1;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if ((w[j] & 0x7f80u) == 0x7f80u) w[j] &= 0xffff0000u, bad = true;
                if ((w[j] & 0x7f800000u) == 0x7f800000u) w[j] &= 0xffffu, bad = true;
              }
              if (bad) *p = u;
              if (bad && pos < k1) atomicOr(odd + ((pos - seq.ctx) >> 5), 1u << ((pos - seq.ctx) & 31));
            }
            fence_proxy_async_smem();
          }
        }
        // The row's reference moves when a score passes it by 2^8.
        float top[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {  // four chains
          top[c] = fmaxf(x[c], x[c + 4]);
#pragma unroll
          for (int i = 8; i < kKeys; i += 8) top[c] = max3(top[c], x[i + c], x[i + c + 4]);
        }
        const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]) * kTreeC;
        float alpha = 1.f;
        if (most > ref + kTreeStale) {
          alpha = ex2(ref - most);
          ref = most;
        }
        l0 *= alpha;
        l1 *= alpha;
        const float neg = -ref;
#pragma unroll
        for (int h = 0; h < kKeys; h += 32) {
          float* const y = x + h;
          if constexpr (kF32) {
            float lo[32];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              fma2(y[i], y[i + 1], y[i], y[i + 1], kTreeC, kTreeC, neg, neg);
              y[i] = ex2(y[i]);
              y[i + 1] = ex2(y[i + 1]);
              add2(l0, l1, l0, l1, y[i], y[i + 1]);
              // p hi is what the tensor core reads of p
              fma2(lo[i], lo[i + 1], tf32_hi(y[i]), tf32_hi(y[i + 1]), -1.f, -1.f, y[i], y[i + 1]);
            }
            tmem_st32(s_tmem + h, *reinterpret_cast<float(*)[32]>(y));
            tmem_st32(lane_tmem + L::kColLo + g * kKeys + h, lo);
          } else {
            uint32_t w[3][16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              fma2(y[i], y[i + 1], y[i], y[i + 1], kTreeC, kTreeC, neg, neg);
              y[i] = ex2(y[i]);
              y[i + 1] = ex2(y[i + 1]);
              add2(l0, l1, l0, l1, y[i], y[i + 1]);
              split3_cut(y[i], y[i + 1], w[0][i / 2], w[1][i / 2], w[2][i / 2]);
            }
#pragma unroll
            for (int t = 0; t < 3; ++t) tmem_st16(s_tmem + t * 32 + h / 2, w[t]);
          }
        }
        if (!kF32 && k > 0) add_o(k - 1);
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int i = 0; i < kD; ++i) o[i] *= alpha;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[g]);
      }
      if (k > 0) add_o(k - 1);
    }

    // ------------------------------------------------------------ epilogue
    // The groups exchange halves of their rows (dims 32 (1 - g) .. of this
    // thread's) through the ring, which is idle once both have seen their last
    // O, and each writes its half.
    {
      float l = l0 + l1;
      int over;
      if (meet(kMeet, false, failed, lane, &over)) goto done;
      unsigned long long rest = ((unsigned long long)odd[1] << 32) | odd[0];
      const unsigned long long mask = masks[row >> 2];
      while (rest && g == 0) {  // drafted values that are not finite reach the rows that see them
        const int j0 = __ffsll((long long)rest) - 1;
        rest &= rest - 1;
        const int page = fetch(trow + (seq.ctx + j0) / ATTN_PAGE);
        if (!(mask >> j0 & 1) || page < 0 || page >= a.num_pages) continue;
        const size_t at = (((size_t)page * ATTN_PAGE + (seq.ctx + j0) % ATTN_PAGE) * kHKV + head) * kD;
#pragma unroll
        for (int i = 0; i < kD; ++i) {
          const float v = kF32 ? fetch(static_cast<const float*>(a.v_pages) + at + i)
                               : __uint_as_float((uint32_t)fetch(static_cast<const uint16_t*>(a.v_pages) + at + i) << 16);
          if ((__float_as_uint(v) & 0x7f800000u) == 0x7f800000u) o[i] += v;
        }
      }
      float2* const ml = reinterpret_cast<float2*>(smem + L::kSmemMl);
      uint8_t* const give = smem + ((1 - g) * 128 + row) * 128, * const take = smem + (g * 128 + row) * 128;
      ml[g * 128 + row] = make_float2(ref, l);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = 4 * i;  // the other group's half
        *reinterpret_cast<float4*>(give + ((i ^ (row & 7)) << 4)) =
            g == 0 ? make_float4(o[32 + d], o[33 + d], o[34 + d], o[35 + d]) : make_float4(o[d], o[d + 1], o[d + 2], o[d + 3]);
      }
      meet(kMeet);
      const float2 other = ml[(1 - g) * 128 + row];
      const float m = fmaxf(ref, other.x);
      const float w0 = ex2(ref - m), w1 = ex2(other.x - m);  // an unseen group's sums are zeros
      l = fmaf(w0, l, w1 * other.y);
      const bool mine = active && (row >> 2) < nrows;
      const size_t at = (size_t)(seq.first + i0 + (row >> 2)) * kHQ + head * kGroup + (row & 3);
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;  // no key: zeros
      float* const dst = (a.cluster ? reinterpret_cast<float*>(smem + L::kSmemRows) + row * kRowStride
                          : whole   ? a.out + at * kD
                                    : a.parts + (at * a.splits + s) * kD) + g * 32;
      if (mine) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(take + ((i ^ (row & 7)) << 4));
          const int d = 4 * i;
          const float a0 = g ? o[32 + d] : o[d], a1 = g ? o[33 + d] : o[d + 1], a2 = g ? o[34 + d] : o[d + 2],
                      a3 = g ? o[35 + d] : o[d + 3];
          *reinterpret_cast<float4*>(dst + d) =
              make_float4(fmaf(w0, a0, w1 * y.x) * inv, fmaf(w0, a1, w1 * y.y) * inv, fmaf(w0, a2, w1 * y.z) * inv,
                          fmaf(w0, a3, w1 * y.w) * inv);
        }
        if (a.cluster && g == 0) ends[row] = make_float2(m == kUnseen ? -INFINITY : m, l);
        if (!a.cluster && !whole && g == 0) {
          float2* const mls = reinterpret_cast<float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD);
          mls[at * a.splits + s] = make_float2(m == kUnseen ? -INFINITY : m, l);
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
    if (warp == L::kKWarp || warp == L::kVWarp) {  // before the block's memory is released
      const bool is_v = warp == L::kVWarp;
      drain_copies(is_v ? vfull : kfull, kStages, issued[is_v], a.timeout_ns);
    } else if (warp == L::kQkWarp || warp == L::kPvWarp) {
      drain_products(&drain[warp == L::kPvWarp], a.timeout_ns);
    } else if (warp < kSoft && !whole) {  // after a failed wait the segment counts as empty
      float2* const mls = reinterpret_cast<float2*>(a.parts + (size_t)a.N * kHQ * a.splits * kD);
      for (int r = tid; r < nrows * kGroup; r += 32 * kSoft) {
        if (a.cluster) ends[r] = make_float2(-INFINITY, 0.f);
        else
          mls[((size_t)(seq.first + i0 + (r >> 2)) * kHQ + head * kGroup + (r & 3)) * a.splits + s] =
              make_float2(-INFINITY, 0.f);
      }
    }
    __syncthreads();
  }
  if (warp == L::kQkWarp) tmem_dealloc(tmem, 512);
  // (The softmax warps: with fp32 pages the others have given their registers away.)
  if (a.cluster && warp < kSoft)
    cluster_merge(a, seq.first + i0, nrows, head, reinterpret_cast<const float*>(smem + L::kSmemRows), kRowStride, ends,
                  tid, 32 * kSoft);
}

}  // namespace

TreeVariant tree_wide_variant(bool bf16) {
  if (bf16)
    return {tree_wide_kernel<false, false>, tree_wide_kernel<false, true>, kRows, Wide<false>::kThreads,
            Wide<false>::kSmemAlloc, 1, false, 0, 6, 2};
  return {tree_wide_kernel<true, false>, tree_wide_kernel<true, true>, kRows, Wide<true>::kThreads,
          Wide<true>::kSmemAlloc, 1, true, 126, 6, 2};
}

}  // namespace attn
