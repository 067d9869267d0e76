// weigh.cu -- what a window of rows gives to every cached token, without the rows'
// attention: the weights by which a prompt's cache is cut down.
//   s_rhj = q_rh . k_j / 8,  p_rhj = softmax over the tokens j that row r sees,
//   W[j][g] = (decay W[j][g], or 0 for a token without a weight yet) + sum of p_rhj over rows r
//             and the 4 heads h of g; row i of a sequence sees its tokens j <= context + i
//
// p needs its row's sum over all keys first, and a window's scores (up to 8 KB a token) cost
// more to keep than to compute again: two passes over K with their operands exchanged. A
// block has the 128 (row, head) pairs of 32 rows and a KV head and streams tiles of 128 keys:
//   rows pass  S [rows][keys], q in tensor memory: a thread owns a row, its maximum and sum
//              never cross threads
//   keys pass  S [keys][rows], K in tensor memory: a thread owns a key and adds up its p's
// The rows pass leaves (reference, sum) of every row and segment of keys; the keys pass merges
// them and has the tensor core subtract them too, by one more K step (1 .. 1) . (reference and
// log2 of the sum, in three terms each), so that what a thread reads is log2 p and all it does
// is 2^x and an addition. (Read from shared memory, 8 bytes a column and thread, they took as
// long as the products.) q is scaled by log2(e) / 8 before it is split. Windows of more than 32
// rows: more blocks in the rows pass, one row tile after another in the keys pass, whose
// block adds to weights that it alone writes. Windows of up to 32 rows over so few keys that all
// products stay in tensor memory need no second pass: weights_of_products().
//   bf16 pages: K as stored, q in three bf16 terms: 3 x 4 MMAs of 128 x 128 x 16 a tile
//   fp32 pages: q K_lo + q_lo K + q K, tf32 terms: 3 x 8 of 128 x 128 x 8
// (K is read truncated; K_lo is the remainder rounded to tf32, q's first term rounded too.) By
// key, windows of fewer rows take fewer columns. Fewer terms were measured and not kept: with two
// bf16 terms in both passes 64 rows of 131071 tokens (bf16 pages) took 119 us for 144, 32 rows of
// 16 sequences of 16384 (fp32) 205 for 278, but weights were off by 2e-6 to 4e-6 where a plain
// fp32 computation is by 5e-7; in the rows pass alone, as much.
//
// Bound by the products and by shared memory, neither full: those fp32 windows take 274 us in short
// runs (2070 MHz) and 309 in long ones, which meet the power limit (1630 MHz). Their 206 GFLOP of
// tf32 terms are 174 us at the rate of a dense loop, K's bytes, read twice, 83. In a short run the
// tensor pipe is active for 70 % of the cycles and shared memory's data path for 65 (35 the products'
// operand there, 30 the warps' loads and stores), K's landings not counted. The 64 rows on bf16
// pages take 140 and 159 us, 112 of bf16 terms at the rate of a library product.
//
// Roles: three groups of four warps take the tiles in turn; four warps that write K_lo (fp32,
// rows) or move K to tensor memory (keys); one warp for TMA (16-token pages through the block
// table), one to issue the products.
#include <cuda.h>

#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"
#include "tree.cuh"
#include "weigh_tiles.cuh"

namespace attn {
namespace {

using namespace tc;

using weigh_tiles::kKeys;
using weigh_tiles::kRows;
constexpr int kPages = kKeys / ATTN_PAGE;
constexpr int kGroups = 3, kSoft = 4 * kGroups;  // warps that read S
constexpr int kChunk = 64;                 // columns of S that a thread has in registers
constexpr int kTmaWarps = 2;               // tiles in turn: a box of 16 rows costs its warp about 100 cycles
constexpr uint32_t kHalf = 128 * 128;      // 128 rows of 128 bytes
constexpr uint32_t kBox = ATTN_PAGE * 128;
constexpr int kMaxSplits = 64;
constexpr float kNothing = 1e30f;          // reference of a row that gives nothing
constexpr unsigned kFull = 0xffffffffu;

struct WeighArgs {
  const float* q;          // [N][32][64]
  float* weights;          // [num_pages][8][16]
  const int *table, *ctx_lens, *row_start, *weighed_lens;
  float2* stats;           // [N][32][splits]: log2 maximum, sum (kUnseen and 0 of a segment without keys)
  int B, N, max_rows, max_blocks, num_pages, max_context;
  int row_tiles, splits;   // of the rows pass
  int key_splits;          // of the keys pass
  float decay;
  int withheld;            // failure test: segments whose first tile is never loaded
  unsigned* err;
  unsigned long long timeout_ns;
};

template <bool kF32, bool kByKey>
struct Lay {
  static constexpr bool kDirect = !kF32 && !kByKey;  // the tensor core reads K as it landed
  static constexpr bool kSlotted = kByKey;           // K goes on to slots in tensor memory
  static constexpr uint32_t kRaw = kF32 ? 2 * kHalf : kHalf;          // a tile of K as it lands
  static constexpr uint32_t kOperand = kRaw;                          // an operand of 128 rows
  static constexpr uint32_t kStageBytes = kRaw + (kF32 && !kByKey ? kOperand : 0);  // K (, K lo)
  static constexpr int kStages = kF32 ? 3 : 8;
  static constexpr int kTerms = kF32 ? 2 : 3;               // of q
  static constexpr int kSlots = 3;
  static constexpr uint32_t kSmemQ = kStages * kStageBytes;           // keys pass: q's terms
  static constexpr uint32_t kSmemRef = kSmemQ + (kByKey ? kTerms * kOperand : 0);                    // and the references' tile
  static constexpr uint32_t kSmemEnds = kSmemRef + (kByKey ? kHalf : 0);         // rows pass: [groups][128] (reference, sum)
  static constexpr uint32_t kSmemEnd = kSmemEnds + (kByKey ? 0 : kGroups * 128 * 8);
  // Tensor memory. Rows: q's terms, then S. Keys: K (fp32: its lo and itself, one after the other), ones, S.
  static constexpr int kParts = kF32 && kByKey ? 2 : 1;
  static constexpr uint32_t kSlotCols = kF32 ? 64 : 32;
  static constexpr uint32_t kColK = 0, kColOnes = kSlots * kSlotCols;
  static constexpr uint32_t kColQ = 0, kTermCols = kF32 ? 64 : 32, kColS = kByKey ? kColOnes + 16 : kTerms * kTermCols;
  static constexpr int kBufs = kF32 && kByKey ? 2 : 3;
  static constexpr int kNumBars = 3 * kStages + 2 * kSlots + kGroups + kBufs + 2;
  static_assert(kColS + kBufs * kKeys <= 512, "TMEM layout");
};

// Warps: those that read S, four that pass K on, TMA, products. (The first four of them have
// nothing to do where the tensor core reads K as it landed.)
constexpr int kConvWarp = kSoft, kTmaWarp = kConvWarp + 4, kMmaWarp = kTmaWarp + kTmaWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);

// A kernel runs one pass, or both (kFused) one after the other over the same segment of keys:
// the passes' operands lie in the same bytes, their barriers beside each other. kOnce: the
// rows pass alone, whose products stay in tensor memory until the sums are known.
constexpr int kRowsPass = 0, kKeysPass = 1, kFused = 2, kOnce = 3;
constexpr int kHeld = 3;        // tiles of S that a block's tensor memory holds
constexpr int kFusedTiles = 2;  // row tiles of a fused window, whose sums stay in shared memory
template <bool kF32, int kPass>
struct Kernel {
  using R = Lay<kF32, false>;
  using K = Lay<kF32, true>;
  static constexpr bool kRows = kPass != kKeysPass, kKeys = kPass == kKeysPass || kPass == kFused;
  static constexpr uint32_t kEnd = !kKeys ? R::kSmemEnd : kPass == kKeysPass ? K::kSmemEnd
                                   : R::kSmemEnd > K::kSmemEnd ? R::kSmemEnd : K::kSmemEnd;
  static constexpr uint32_t kSmemKept = kEnd;  // one launch: [row tiles][128] (reference, sum) of this block's keys
  static constexpr uint32_t kSmemBarR = kSmemKept + (kPass == kFused ? kFusedTiles * 128 * 8 : kPass == kOnce ? 128 * 8 : 0);
  static constexpr uint32_t kSmemBarK = kSmemBarR + (kRows ? R::kNumBars * 8 : 0);
  static constexpr uint32_t kSmemWords = kSmemBarK + (kKeys ? K::kNumBars * 8 : 0);  // TMEM address, abort flag
  static constexpr uint32_t kSmemAlloc = kSmemWords + 16 + 1024;
  static_assert(kSmemAlloc <= 232448, "exceeds the 227 KB per-block shared memory limit");
};

// The lengths of a sequence, checked as those of drafted rows are.
__device__ __forceinline__ Seq load_window(const WeighArgs& a, int b) {
  TreeArgs t;
  t.ctx_lens = a.ctx_lens;
  t.row_start = a.row_start;
  t.max_blocks = a.max_blocks;
  t.max_context = a.max_context;
  t.N = a.N;
  t.max_rows = a.max_rows;
  return load_seq(t, b);
}

// Three terms of x that the tensor core takes exactly: bf16, or tf32 (of fp32 pages).
template <bool kF32>
__device__ __forceinline__ void three_terms(float x, float (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = kF32 ? tf32_hi(x) : bf16_trunc(x);
    x -= t[i];
  }
}

// tcgen05.st of 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&u)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
               "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

// What a block works on.
struct Work {
  uint8_t* smem;
  uint32_t tmem;
  Seq seq;
  int head, b, s;    // s: its segment
  int k0, k1;        // of these keys
  int rt0, rt1;      // and row tiles
  int ranks;         // fused: segments, the blocks of the cluster
  float2* kept;      // fused: [row tiles][128], the rows' (reference, sum) over this block's keys
  volatile int* abort_flag;
  // Keys that some row of row tile rt sees, and the tiles that hold them.
  __device__ __forceinline__ int visible(int rt) const { return weigh_tiles::visible(seq.ctx, seq.rows, k1, rt); }
  // Columns of S by key: the row tile's (row, head) pairs, in steps of 32.
  __device__ __forceinline__ int cols(int rt) const { return (min(seq.rows - rt * kRows, kRows) * kGroup + 31) / 32 * 32; }
  __device__ __forceinline__ int tiles(int rt) const { return weigh_tiles::tiles(seq.ctx, seq.rows, k0, k1, rt); }
};

// A pass's barriers.
template <class L>
struct Bars {
  uint64_t *kfull, *kready, *kempty, *tfull, *tempty, *sfull, *sfree, *qready, *drain;
  __device__ __forceinline__ explicit Bars(uint64_t* at) {
    kfull = at;                       // [stage] K landed
    kready = kfull + L::kStages;      // [stage] K lo written (tf32, rows)
    kempty = kready + L::kStages;     // [stage] K read
    tfull = kempty + L::kStages;      // [slot] K written there
    tempty = tfull + L::kSlots;       // [slot] products done with it
    // A group's next S: a barrier a group, since the buffers go round in another time; the group
    // has waited for its tile before the buffer's next product, and so its own, is issued.
    sfull = tempty + L::kSlots;       // [group] S written
    sfree = sfull + kGroups;          // [buffer] S read
    qready = sfree + L::kBufs;        // q's terms of a row tile written
    drain = qready + 1;
  }
  __device__ __forceinline__ void init(int lane) const {
    for (int i = lane; i < L::kNumBars; i += 32) {
      uint64_t* const bar = &kfull[i];
      const bool by_four = (bar >= kready && bar < kempty) || (L::kSlotted && bar >= kempty && bar < tempty) || (bar >= sfree && bar < qready);
      mbar_init(bar, by_four ? 4 : bar == qready ? kSoft : 1);
    }
  }
};

// One pass of the block, every warp in its role. All warps meet at the end; after a wait that
// ran out those that started copies and products have waited for them.
//
// It begins at the first row tile that sees a key of the segment, in every role. `qready` has one
// phase a row tile, told apart by its parity alone, and what keeps the warps that write q from
// completing two of them before the issuing warp has looked is that they wait for S of the tile
// between: each row tile that is gone through has one.
template <bool kF32, bool kByKey>
__device__ __forceinline__ void run_pass(const CUtensorMap& mk, const WeighArgs& a, const Work& x_, uint64_t* bars) {
  using L = Lay<kF32, kByKey>;
  constexpr int kStages = L::kStages;
  uint8_t* const smem = x_.smem;
  const Seq& seq = x_.seq;
  const int head = x_.head, b = x_.b, s = x_.s, k0 = x_.k0, k1 = x_.k1, rt1 = x_.rt1;
  const int rt0 = weigh_tiles::first_seeing(seq.ctx, k0, k1, x_.rt0, rt1);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  const auto visible = [&](int rt) { return x_.visible(rt); };
  const auto tiles = [&](int rt) { return x_.tiles(rt); };
  const Bars<L> bar_(bars);
  uint64_t *const kfull = bar_.kfull, *const kready = bar_.kready, *const kempty = bar_.kempty, *const tfull = bar_.tfull,
           *const tempty = bar_.tempty, *const sfull = bar_.sfull, *const sfree = bar_.sfree, *const qready = bar_.qready,
           *const drain = bar_.drain;
  volatile int* const abort_flag = x_.abort_flag;
  const Wait wait{a.err, a.timeout_ns, abort_flag};
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  const uint32_t tmem = x_.tmem;
  int last = -1;  // the last tile that a TMA warp has asked for

  if (warp >= kTmaWarp && warp < kMmaWarp) {
    const int mine = warp - kTmaWarp;  // this warp's tiles: every second one
    int it = 0;
    bool ok = true;
    for (int rt = rt0; ok && rt < rt1; ++rt) {
      const int end = visible(rt), count = tiles(rt);
      // Lane l holds the table's entry of page l of a group of four tiles.
      const auto entry_at = [&](int g) -> int {
        const int t = k0 + g * 4 * kKeys + lane * ATTN_PAGE;
        return t < end ? fetch(trow + t / ATTN_PAGE) : -1;
      };
      int entries = entry_at(0), entries_next = entry_at(1);
      for (int n = 0; n < count; ++n, ++it) {
        if ((it & (kTmaWarps - 1)) == mine) {
          const int st = it % kStages;
          if (it >= kStages && !(ok = wait.warp(&kempty[st], (it / kStages - 1) & 1))) break;
          const int p = lane & (kPages - 1), half = lane / kPages;
          int page = __shfl_sync(kFull, entries, (n & 3) * kPages + p);
          const int pages = min(kPages, (end - k0 - n * kKeys + ATTN_PAGE - 1) / ATTN_PAGE);
          const bool has = half < (kF32 ? 2 : 1) && p < pages;
          if (has && (page < 0 || page >= a.num_pages)) {
            record_error(a.err, kDevErrBounds);
            page = a.num_pages;  // past the pool's end: reads as zeros
          }
          if (lane == 0) mbar_arrive_expect_tx(&kfull[st], pages * (kF32 ? 2 : 1) * kBox);
          last = it;
          __syncwarp();
          if (has && !(it == 0 && s < a.withheld))
            tma_load_2d(smem + st * L::kStageBytes + half * kHalf + p * kBox, &mk, &kfull[st], head * kD + half * 32,
                        page * ATTN_PAGE);
        }
        if ((n & 3) == 3) {
          entries = entries_next;
          entries_next = entry_at((n >> 2) + 2);
        }
      }
    }
  } else if (warp == kMmaWarp) {
    const uint32_t base = smem_u32(smem);
    int it = 0;
    bool ok = true;
    for (int rt = rt0; ok && rt < rt1; ++rt) {
      const int count = tiles(rt), cols = kByKey ? x_.cols(rt) : kKeys;
      ok = wait.warp(qready, (rt - rt0) & 1);
      for (int n = 0; ok && n < count; ++n, ++it) {
        const int buf = it % L::kBufs;
        const uint32_t d = tmem + L::kColS + buf * kKeys;
        if (it >= L::kBufs && !(ok = wait.warp(&sfree[buf], (it / L::kBufs - 1) & 1))) break;
        const uint32_t id = kF32 ? idesc_tf32(128, cols) : idesc_bf16(128, cols, false);
        constexpr uint64_t lo = L::kOperand >> 4;
        if constexpr (!kByKey) {
          const int st = it % kStages;
          if (!(ok = wait.warp(kF32 ? &kready[st] : &kfull[st], (it / kStages) & 1))) break;
          tc_fence_after();
          const uint64_t kd = sdesc_sw128(base + st * L::kStageBytes);
          const uint32_t q = tmem + L::kColQ;
          if (elect()) {
            if constexpr (kF32) {  // the small products first, as by key
              const auto product = [&](uint32_t qt, uint64_t kt, bool first) {
#pragma unroll
                for (int x = 0; x < 8; ++x) mma_tf32_ts(d, qt + x * 8, kt + (x >> 2) * (kHalf >> 4) + (x & 3) * 2, id, !first || x > 0);
              };
              product(q, kd + lo, true);
              product(q + 64, kd, false);
              product(q, kd, false);
            } else {
#pragma unroll
              for (int t = L::kTerms - 1; t >= 0; --t)
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_f16_ts(d, q + t * 32 + x * 8, kd + x * 2, id, t < L::kTerms - 1 || x > 0);
            }
            mma_commit(&sfull[it % kGroups]);
            mma_commit(&kempty[st]);
          }
          __syncwarp();
        } else {
          const uint64_t qd = sdesc_sw128(base + L::kSmemQ), rd = sdesc_sw128(base + L::kSmemRef);
#pragma unroll 1
          for (int h = 0; ok && h < L::kParts; ++h) {
            const int part = it * L::kParts + h, slot = part % L::kSlots;
            if (!(ok = wait.warp(&tfull[slot], (part / L::kSlots) & 1))) break;
            tc_fence_after();
            const uint32_t k = tmem + L::kColK + slot * L::kSlotCols;
            if (elect()) {
              if constexpr (kF32) {  // K lo, then K
                const auto product = [&](uint64_t qt, bool first) {
#pragma unroll
                  for (int x = 0; x < 8; ++x) mma_tf32_ts(d, k + x * 8, qt + (x >> 2) * (kHalf >> 4) + (x & 3) * 2, id, !first || x > 0);
                };
                if (h == 1) product(qd + lo, false);
                product(qd, h == 0);
              } else {
#pragma unroll
                for (int t = L::kTerms - 1; t >= 0; --t)
#pragma unroll
                  for (int x = 0; x < 4; ++x) mma_f16_ts(d, k + x * 8, qd + t * lo + x * 2, id, t < L::kTerms - 1 || x > 0);
              }
              mma_commit(&tempty[slot]);
              if (h == L::kParts - 1) {
                if constexpr (kF32) mma_tf32_ts(d, tmem + L::kColOnes, rd, id, 1);
                else mma_f16_ts(d, tmem + L::kColOnes, rd, id, 1);
                mma_commit(&sfull[it % kGroups]);
              }
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp >= kConvWarp && warp < kTmaWarp) {
    const int ctid = tid - 32 * kConvWarp;
    int total = 0;
    for (int rt = rt0; !L::kDirect && rt < rt1; ++rt) total += tiles(rt);
    for (int it = 0; it < total; ++it) {
      const int st = it % kStages;
      uint8_t* const stage = smem + st * L::kStageBytes;
      if (!wait.warp(&kfull[st], (it / kStages) & 1)) break;
      if constexpr (!kByKey) {
        // K lo, at the same offset of the next region.
#pragma unroll 2
        for (int h = 0; h < 4; ++h) {
          float4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(stage + (ctid + (4 * h + i) * 128) * 16);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(stage + (ctid + (4 * h + i) * 128) * 16 + L::kOperand) =
                make_float4(tf32_near(x[i].x - tf32_hi(x[i].x)), tf32_near(x[i].y - tf32_hi(x[i].y)),
                            tf32_near(x[i].z - tf32_hi(x[i].z)), tf32_near(x[i].w - tf32_hi(x[i].w)));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&kready[st]);
      } else {
        // A thread's key, row ctid of the tile, to its lane of tensor memory.
        bool ok = true;
#pragma unroll
        for (int h = 0; ok && h < L::kParts; ++h) {
          const int part = it * L::kParts + h, slot = part % L::kSlots;
          if (part >= L::kSlots && !(ok = wait.warp(&tempty[slot], (part / L::kSlots - 1) & 1))) break;
          tc_fence_after();
          const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + L::kColK + slot * L::kSlotCols;
#pragma unroll
          for (int half = 0; half < (kF32 ? 2 : 1); ++half) {
            float x[32];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(x + 4 * i) =
                  *reinterpret_cast<const float4*>(stage + half * kHalf + sw128((uint32_t)ctid * 128u + i * 16u));
            if (kF32 && h == 0) {  // K lo first
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = tf32_near(x[i] - tf32_hi(x[i]));
            }
            tmem_st32(at + half * 32, x);
          }
          if (h == L::kParts - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&kempty[st]);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tfull[slot]);
        }
        if (!ok) break;
      }
    }
  } else if (warp < kSoft) {
    constexpr int kMeet = 32 * kSoft;
    const int quarter = warp & 3, g = warp >> 2, row = quarter * 32 + lane;  // lane of tensor memory
    const uint32_t lane_tmem = tmem + ((uint32_t)(quarter * 32) << 16);
    bool failed = false;
    float ref = kUnseen, l0 = 0.f, l1 = 0.f;
    const int weighed = kByKey ? (a.weighed_lens ? fetch(a.weighed_lens + b) : seq.ctx) : 0;
    int done = 0;  // tiles of the row tiles before
    // What the rows pass leaves of a row tile, by the threads of one group.
    const auto leave = [&](int rt, float2 all) {
      if (x_.kept) x_.kept[rt * 128 + row] = all;
      else if (rt * kRows + (row >> 2) < seq.rows)
        a.stats[((size_t)(seq.first + rt * kRows + (row >> 2)) * kHQ + head * kGroup + (row & 3)) * a.splits + s] = all;
    };
    if (!kByKey && g == 0)
      for (int rt = x_.rt0; rt < rt0; ++rt) leave(rt, make_float2(kUnseen, 0.f));
    for (int rt = rt0; rt < rt1; ++rt) {
      const int i0 = rt * kRows, nrows = min(kRows, seq.rows - i0);
      const bool in = (row >> 2) < nrows;
      const size_t pair = (size_t)(seq.first + i0 + (row >> 2)) * kHQ + head * kGroup + (row & 3);
      if (rt > rt0) {  // what the tile before needs is still in use; its weights are written
        int over;
        if (meet(kMeet, false, failed, lane, &over)) {
          for (int x = rt; !kByKey && g == 0 && x < rt1; ++x) leave(x, make_float2(kUnseen, 0.f));
          break;
        }
      }
      // q in its terms; rows past the last are zeros.
#pragma unroll 1
      for (int c = g; g < 2 && c < 4; c += 2) {  // 16 dims at a time, by the first two groups
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (in) v = fetch(reinterpret_cast<const float4*>(a.q + pair * kD + c * 16 + i));
          x[i] = v.x * kTreeC, x[i + 1] = v.y * kTreeC, x[i + 2] = v.z * kTreeC, x[i + 3] = v.w * kTreeC;
        }
        if constexpr (!kByKey && kF32) {
          uint32_t w[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float h = tf32_near(x[i]);
            w[0][i] = __float_as_uint(h), w[1][i] = __float_as_uint(tf32_near(x[i] - h));
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) tmem_st16(lane_tmem + L::kColQ + t * 64 + c * 16, w[t]);
        } else if constexpr (!kByKey) {
          uint32_t w[3][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) split3_cut(x[2 * i], x[2 * i + 1], w[0][i], w[1][i], w[2][i]);
#pragma unroll
          for (int t = 0; t < L::kTerms; ++t) tmem_st8(lane_tmem + L::kColQ + t * 32 + c * 8, w[t]);
        } else if constexpr (kF32) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            uint8_t* const at = smem + L::kSmemQ + (c >> 1) * kHalf + sw128((uint32_t)row * 128u + (c & 1) * 64u + i * 4u);
            const float4 h = make_float4(tf32_near(x[i]), tf32_near(x[i + 1]), tf32_near(x[i + 2]), tf32_near(x[i + 3]));
            *reinterpret_cast<float4*>(at) = h;
            *reinterpret_cast<float4*>(at + L::kOperand) = make_float4(tf32_near(x[i] - h.x), tf32_near(x[i + 1] - h.y), tf32_near(x[i + 2] - h.z), tf32_near(x[i + 3] - h.w));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            uint32_t w[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) split3_cut(x[i + 2 * j], x[i + 2 * j + 1], w[0][j], w[1][j], w[2][j]);
            uint8_t* const at = smem + L::kSmemQ + sw128((uint32_t)row * 128u + c * 32u + i * 2u);
#pragma unroll
            for (int t = 0; t < L::kTerms; ++t) *reinterpret_cast<uint4*>(at + t * L::kOperand) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
          }
        }
      }
      if (kByKey && g == kGroups - 1) {
        // The row's reference and the logarithm of its sum over all keys, from the segments.
        float top = kUnseen, sum = 0.f;
        if (in && x_.kept) {  // the cluster's
          float2 p[kMaxCluster];
#pragma unroll
          for (int i = 0; i < kMaxCluster; ++i) {
            p[i] = make_float2(kUnseen, 0.f);
            if (i < x_.ranks) p[i] = ld_cluster2(mapa_shared(smem_u32(x_.kept + rt * 128 + row), i));
            top = fmaxf(top, p[i].x);
          }
#pragma unroll
          for (int i = 0; i < kMaxCluster; ++i) sum = fmaf(ex2(p[i].x - top), p[i].y, sum);
        } else if (in) {
          const float2* const st = a.stats + pair * a.splits;
#pragma unroll 4
          for (int i = 0; i < a.splits; ++i) top = fmaxf(top, fetch(st + i).x);
#pragma unroll 4
          for (int i = 0; i < a.splits; ++i) {
            const float2 p = fetch(st + i);
            sum = fmaf(ex2(p.x - top), p.y, sum);
          }
        }
        // A row whose scores are all -inf, or none: 2^x is 0 whatever x is.
        float t[6];
        three_terms<kF32>(sum == 0.f ? -kNothing : -top, *reinterpret_cast<float(*)[3]>(t));
        three_terms<kF32>(sum == 0.f ? 0.f : -log2f(sum), *reinterpret_cast<float(*)[3]>(t + 3));
        uint4 u0, u1 = make_uint4(0, 0, 0, 0);
        if constexpr (kF32) {
          u0 = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3]));
          u1.x = __float_as_uint(t[4]), u1.y = __float_as_uint(t[5]);
        } else {
          u0 = make_uint4(pack_bf16_trunc(t[0], t[1]), pack_bf16_trunc(t[2], t[3]), pack_bf16_trunc(t[4], t[5]), 0u);
        }
        *reinterpret_cast<uint4*>(smem + L::kSmemRef + sw128((uint32_t)row * 128u)) = u0;
        *reinterpret_cast<uint4*>(smem + L::kSmemRef + sw128((uint32_t)row * 128u + 16u)) = u1;
        if (rt == rt0) {
          constexpr uint32_t kOne = kF32 ? 0x3f800000u : 0x3f803f80u;
          const uint32_t ones[8] = {kOne, kOne, kOne, kOne, kOne, kOne, kOne, kOne};
          tmem_st8(lane_tmem + L::kColOnes, ones);
        }
      }
      if (kByKey) fence_proxy_async_smem();
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(qready);
      const int count = tiles(rt);
      const int cols = x_.cols(rt);
      const int first = (g + kGroups - done % kGroups) % kGroups;  // the group's first tile
      // By key: the page of a thread's key, looked up a tile ahead.
      const int seen = visible(rt);
      const auto page_at = [&](int n) {
        const int t = k0 + n * kKeys + row;
        return kByKey && t < seen ? fetch(trow + t / ATTN_PAGE) : -1;
      };
      int page_next = page_at(first);
      for (int n = first; n < count; n += kGroups) {
        const int it = done + n, buf = it % L::kBufs, t0 = k0 + n * kKeys;
        const uint32_t s_tmem = lane_tmem + L::kColS + buf * kKeys;
        if constexpr (kByKey) {
          const int t = t0 + row, page = page_next;
          page_next = page_at(n + kGroups);
          // The key's weight so far, on its way while the products run. Row tile (t - context) /
          // 32 is the first that sees a token of the rows themselves, 0 any other.
          float* w = nullptr;
          float old = 0.f;
          if (page >= 0 && page < a.num_pages) {
            w = a.weights + ((size_t)page * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE;
            if (rt > max(0, t - seq.ctx) / kRows) old = *w;
            else if (a.decay != 0.f && t < weighed) old = a.decay * *w;
          }
          failed |= !wait.warp(&sfull[g], (it / kGroups) & 1);
          tc_fence_after();
          float sum0 = 0.f, sum1 = 0.f;
          const int late = t - seq.ctx - i0;  // rows before it do not see the key
          const auto add = [&](int h, float* x, auto width) {
            constexpr int kWidth = decltype(width)::value;
            if (t0 + kKeys > seq.ctx + i0) {
#pragma unroll
              for (int i = 0; i < kWidth; ++i)
                if ((h + i) / 4 < late) x[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < kWidth; i += 2) add2(sum0, sum1, sum0, sum1, ex2(x[i]), ex2(x[i + 1]));
          };
          const auto read = [&] {  // the buffer is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[buf]);
          };
          if (cols == kKeys) {
#pragma unroll
            for (int h = 0; h < 128; h += kChunk) {
              float x[kChunk];
#pragma unroll
              for (int i = 0; i < kChunk; i += 32) tmem_ld32(s_tmem + h + i, *reinterpret_cast<float(*)[32]>(&x[i]));
              tmem_wait_ld();
              if (h == 128 - kChunk) read();
              add(h, x, std::integral_constant<int, kChunk>());
            }
          } else {
#pragma unroll 1
            for (int h = 0; h < cols; h += 32) {
              float x[32];
              tmem_ld32(s_tmem + h, x);
              tmem_wait_ld();
              if (h == cols - 32) read();
              add(h, x, std::integral_constant<int, 32>());
            }
          }
          if (w && !failed) *w = old + (sum0 + sum1);
        } else {
          failed |= !wait.warp(&sfull[g], (it / kGroups) & 1);
          tc_fence_after();
          if (quarter * 8 >= nrows) {  // no row in this warp's lanes
            __syncwarp();
            if (lane == 0) mbar_arrive(&sfree[buf]);
            continue;
          }
          const int limit = min(seq.ctx + i0 + (row >> 2) + 1, k1) - t0;  // keys of the tile that the row sees
#pragma unroll
          for (int h = 0; h < 128; h += kChunk) {
            float x[kChunk];
#pragma unroll
            for (int i = 0; i < kChunk; i += 32) tmem_ld32(s_tmem + h + i, *reinterpret_cast<float(*)[32]>(&x[i]));
            tmem_wait_ld();
            if (h == 128 - kChunk) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sfree[buf]);
            }
            if (t0 + kKeys > min(seq.ctx + i0, k1)) {
#pragma unroll
              for (int i = 0; i < kChunk; ++i)
                if (h + i >= limit) x[i] = -INFINITY;
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              top[c] = fmaxf(x[c], x[c + 4]);
#pragma unroll
              for (int i = 8; i < kChunk; i += 8) top[c] = max3(top[c], x[i + c], x[i + c + 4]);
            }
            const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]);
            if (most > ref + kTreeStale) {
              const float alpha = ex2(ref - most);
              ref = most;
              l0 *= alpha;
              l1 *= alpha;
            }
            const float neg = -ref;
#pragma unroll
            for (int i = 0; i < kChunk; i += 2) {
              add2(x[i], x[i + 1], x[i], x[i + 1], neg, neg);
              add2(l0, l1, l0, l1, ex2(x[i]), ex2(x[i + 1]));
            }
          }
        }
      }
      done += count;
      if constexpr (!kByKey) {  // the groups' sums
        float2* const ends = reinterpret_cast<float2*>(smem + L::kSmemEnds);
        if (g > 0) ends[g * 128 + row] = make_float2(ref, l0 + l1);
        int over;
        const bool lost = meet(kMeet, false, failed, lane, &over);
        if (g == 0) {
          float top = ref;
#pragma unroll
          for (int x = 1; x < kGroups; ++x) top = fmaxf(top, ends[x * 128 + row].x);
          float sum = ex2(ref - top) * (l0 + l1);
#pragma unroll
          for (int x = 1; x < kGroups; ++x) sum = fmaf(ex2(ends[x * 128 + row].x - top), ends[x * 128 + row].y, sum);
          leave(rt, lost ? make_float2(kUnseen, 0.f) : make_float2(top, sum));
        }
        ref = kUnseen, l0 = l1 = 0.f;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (warp >= kTmaWarp && warp < kMmaWarp)  // its copies still in flight
      for (int i = last; i >= 0 && i > last - kStages; i -= kTmaWarps) mbar_wait(&kfull[i % kStages], (i / kStages) & 1, a.timeout_ns);
    if (warp == kMmaWarp) drain_products(drain, a.timeout_ns);
    __syncthreads();
  }
}

// The weights from a rows pass whose tiles all have a buffer of S of their own: p by row as the
// pass had it, and its sums over the rows, 32 keys at a time, by exchanging halves of them
// between the lanes (31 shuffles) and adding the quarters up in shared memory. It spares the second
// load of K and its products, for more work a key than the keys pass has.
template <bool kF32>
__device__ __forceinline__ void weights_of_products(const WeighArgs& a, const Work& x) {
  using L = Lay<kF32, false>;
  static_assert(kHeld == L::kBufs && kHeld == kGroups, "a buffer and a group for each tile");
  const int lane = threadIdx.x & 31, warp = __shfl_sync(kFull, threadIdx.x >> 5, 0);
  const int quarter = warp & 3, g = warp >> 2, row = quarter * 32 + lane, count = x.tiles(0);
  const bool soft = warp < kSoft, lost = *x.abort_flag;
  float* const sums = reinterpret_cast<float*>(x.smem);  // [tiles][quarters][128], where K was
  // A thread's key, of tile g, and its weight so far.
  const int t = x.k0 + g * kKeys + row;
  float* w = nullptr;
  float old = 0.f;
  if (soft && t < x.visible(0)) {
    const int page = fetch(a.table + (size_t)x.b * a.max_blocks + t / ATTN_PAGE);
    if (page >= 0 && page < a.num_pages) {
      w = a.weights + ((size_t)page * kHKV + x.head) * ATTN_PAGE + t % ATTN_PAGE;
      if (a.decay != 0.f && t < (a.weighed_lens ? fetch(a.weighed_lens + x.b) : x.seq.ctx)) old = a.decay * *w;
    }
  }
  __syncwarp();
  cluster_sync_all();  // the rows' sums are written
  float top = kUnseen, sum = 0.f;
  const bool in = soft && (row >> 2) < x.seq.rows;
  if (in) {
    float2 p[kMaxCluster];
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      p[i] = make_float2(kUnseen, 0.f);
      if (i < x.ranks) p[i] = ld_cluster2(mapa_shared(smem_u32(x.kept + row), i));
      top = fmaxf(top, p[i].x);
    }
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) sum = fmaf(ex2(p[i].x - top), p[i].y, sum);
  }
  __syncwarp();
  cluster_arrive();  // and read
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int quarters = (x.seq.rows + 7) / 8;
  if (soft && !lost) {
    if (quarter < quarters) {
#pragma unroll 1
      for (int i = g; i < 4 * count; i += kGroups) {  // tile i / 4, its columns 32 (i % 4) and on
        const int n = i >> 2, c = (i & 3) * 32;
        const int limit = min(x.seq.ctx + (row >> 2) + 1, x.k1) - x.k0 - n * kKeys - c;  // of the columns, those that the row sees
        float p[32];
        tmem_ld32(x.tmem + ((uint32_t)(quarter * 32) << 16) + L::kColS + n * kKeys + c, p);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j) p[j] = inv == 0.f || j >= limit ? 0.f : ex2(p[j] - top) * inv;
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1)
#pragma unroll
          for (int j = 0; j < off; ++j) {
            const bool upper = lane & off;
            p[j] = (upper ? p[j + off] : p[j]) + __shfl_xor_sync(kFull, upper ? p[j] : p[j + off], off);
          }
        sums[(n * 4 + quarter) * kKeys + c + lane] = p[0];
      }
    }
    meet(32 * kSoft);
    if (w) {
      float all = 0.f;
      for (int i = 0; i < quarters; ++i) all += sums[(g * 4 + i) * kKeys + row];
      *w = old + all;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(x.tmem, 512);
  __syncwarp();
  cluster_wait();
}

template <bool kF32, int kPass>
__global__ void __launch_bounds__(kThreads, 1) weigh_kernel(const __grid_constant__ CUtensorMap mk, const WeighArgs a) {
  using K = Kernel<kF32, kPass>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  if (warp == kTmaWarp && lane == 0) tma_prefetch_desc(&mk);
  follow();
  // Rows pass: the row tiles of a segment are neighbours in the grid and read its keys at
  // about the same time, all but one from L2.
  const int row_tiles = kPass == kRowsPass ? a.row_tiles : 1, splits = kPass == kKeysPass ? a.key_splits : a.splits;
  Work x;
  x.smem = smem;
  x.s = blockIdx.x / row_tiles;
  x.head = blockIdx.y;
  x.b = blockIdx.z;
  x.seq = load_window(a, x.b);
  if (!x.seq.ok && K::kRows && blockIdx.x == 0 && x.head == 0 && tid == 0) record_error(a.err, kDevErrBounds);
  // The rows of this block: a tile of 32 of them, or all tiles one after another.
  x.rt0 = kPass == kRowsPass ? blockIdx.x % row_tiles : 0;
  x.rt1 = kPass == kRowsPass ? x.rt0 + 1 : (x.seq.rows + kRows - 1) / kRows;
  if (x.seq.rows - x.rt0 * kRows <= 0) return;  // of a cluster all blocks
  // The sequence's own keys, cut evenly into segments of whole tiles.
  weigh_tiles::segment(x.seq.keys, splits, x.s, &x.k0, &x.k1);
  if (kPass == kKeysPass && x.k0 >= x.k1) return;
  x.ranks = splits;
  x.kept = kPass == kFused || kPass == kOnce ? reinterpret_cast<float2*>(smem + K::kSmemKept) : nullptr;
  uint64_t* const rbars = reinterpret_cast<uint64_t*>(smem + K::kSmemBarR);
  uint64_t* const kbars = reinterpret_cast<uint64_t*>(smem + K::kSmemBarK);
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + K::kSmemWords);
  x.abort_flag = reinterpret_cast<volatile int*>(words + 1);

  if (warp == kTmaWarp) {
    if constexpr (K::kRows) Bars<typename K::R>(rbars).init(lane);
    if constexpr (K::kKeys) Bars<typename K::K>(kbars).init(lane);
    fence_mbar_init();
    if (lane == 0) *x.abort_flag = 0;
  } else if (warp == kMmaWarp) {
    tmem_alloc(words, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  x.tmem = words[0];

  if constexpr (K::kRows) run_pass<kF32, false>(mk, a, x, rbars);
  if constexpr (kPass == kOnce) {
    weights_of_products<kF32>(a, x);
    return;
  }
  if constexpr (kPass == kFused) cluster_sync_all();  // the rows' sums are written
  if constexpr (K::kKeys) {
    if (!*x.abort_flag) run_pass<kF32, true>(mk, a, x, kbars);
  }
  if (warp == kMmaWarp) tmem_dealloc(x.tmem, 512);
  if constexpr (kPass == kFused) {
    __syncwarp();
    cluster_sync_all();  // and read by all
  }
}

struct Device {
  bool ready = false;
  int sms = 0;
  int clusters[kMaxCluster + 1] = {};  // of each size, that the device holds at once
};
// A kernel of the call and its shared memory.
struct Choice {
  void (*kernel)(CUtensorMap, WeighArgs);
  uint32_t smem;
};
template <bool kF32>
Choice choice(int pass) {
  if (pass == kRowsPass) return {weigh_kernel<kF32, kRowsPass>, Kernel<kF32, kRowsPass>::kSmemAlloc};
  if (pass == kKeysPass) return {weigh_kernel<kF32, kKeysPass>, Kernel<kF32, kKeysPass>::kSmemAlloc};
  if (pass == kOnce) return {weigh_kernel<kF32, kOnce>, Kernel<kF32, kOnce>::kSmemAlloc};
  return {weigh_kernel<kF32, kFused>, Kernel<kF32, kFused>::kSmemAlloc};
}

int device(Device** out) {
  constexpr int kMaxDev = 64;
  static std::mutex mu;
  static Device devs[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDev) return ATTN_ECUDA;
  std::lock_guard<std::mutex> lock(mu);
  Device& d = devs[dev];
  if (!d.ready) {
    bool ok = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess;
    for (int i = 0; i < 8; ++i) {
      const Choice p = i & 1 ? choice<true>(i >> 1) : choice<false>(i >> 1);
      ok = ok && cudaFuncSetAttribute(p.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem) == cudaSuccess;
    }
    if (!ok) {
      (void)cudaGetLastError();
      return ATTN_ECUDA;
    }
    d.clusters[1] = d.sms;
    const Choice k = choice<true>(kFused);  // all have an SM to themselves
    for (int size = 2; size <= kMaxCluster; ++size) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(size, kHKV);
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = k.smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = size;
      attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      if (cudaOccupancyMaxActiveClusters(&d.clusters[size], k.kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();
        d.clusters[size] = 0;
      }
    }
    d.ready = true;
  }
  *out = &d;
  return ATTN_OK;
}

// Segments of the keys for `units` blocks each: the number whose rounds of one block an SM
// take the least time, a block costing its tiles (each of them `passes` times) and as long
// as four tiles besides.
int segments(long long units, int max_keys, int passes, int sms, double* least) {
  const int tiles = (max_keys + kKeys - 1) / kKeys;
  int best = 1;
  *least = 1e300;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    const long long rounds = (units * s + sms - 1) / sms;
    const double time = (double)rounds * ((double)((tiles + s - 1) / s) * passes + 4.0 * passes);
    if (time < *least * 0.999) *least = time, best = s;
  }
  return best;
}

// How a call runs. Once, where a window's 32 rows and the keys of each block of one round of
// clusters fit tensor memory (8 rows at 1000, fp32 pages: 8.5 us, 9.8 with both passes; 32 rows at
// 2900: 13.0, 15.8 as two launches). Else as one launch, with the rows' sums in shared memory, or as
// two launches with the sums through memory. One launch where a block has a sequence's keys alone
// (44 sequences of 5 rows at 320 to 3213, bf16 pages: 71 us, and 79 as two) or a cluster's blocks
// exchange their sums and all have an SM at once; not in several rounds of clusters (8 windows of
// 64 rows at 16384, bf16 pages: 217 us in clusters of seven, 126; 2 of 16 rows at 2000: 10.4 us in
// clusters of seven, and 17 of eight, of which the device does not hold the 16 at once).
struct Plan {
  bool fused, once;
  int splits, key_splits;
};
Plan plan(int B, int max_rows, int max_keys, const Device& d) {
  const int tiles = (max_rows + kRows - 1) / kRows, sms = d.sms;
  double rows = 0, keys = 0;
  Plan p{};
  p.splits = segments((long long)B * kHKV * tiles, max_keys, 1, sms, &rows);
  p.key_splits = segments((long long)B * kHKV, max_keys, tiles, sms, &keys);
  if (tiles > kFusedTiles) return p;
  const int key_tiles = (max_keys + kKeys - 1) / kKeys;
  double least = rows + keys;
  for (int s = 1; s <= kMaxCluster && s <= key_tiles; ++s) {
    const bool one_round = (long long)B * kHKV <= d.clusters[s];
    if (s > 1 && !one_round) continue;
    const int each = (key_tiles + s - 1) / s;
    if (tiles == 1 && one_round && each <= kHeld) {
      if (!p.once || each < (key_tiles + p.splits - 1) / p.splits) p.once = true, p.splits = s;
      continue;
    }
    const long long rounds = ((long long)B * kHKV * s + sms - 1) / sms;
    const double time = (double)rounds * (2.0 * tiles * each + 4.0 + 2.0 * tiles);
    if (!p.once && time < least * 0.999) least = time, p.fused = true, p.splits = s;
  }
  p.fused &= !p.once;
  return p;
}

int max_keys(int max_context, int max_rows) {
  return max_context > ATTN_MAX_TOKENS - max_rows ? ATTN_MAX_TOKENS : max_context + max_rows;
}

}  // namespace

int weigh_workspace_bytes(int B, int N, int max_rows, int max_context, size_t* bytes) {
  Device* d = nullptr;
  const int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const Plan p = plan(B, max_rows, max_keys(max_context, max_rows), *d);
  *bytes = p.fused || p.once ? 0 : (size_t)N * kHQ * p.splits * sizeof(float2);
  return ATTN_OK;
}

int launch_weigh(const WeighCall& c, unsigned* err, cudaStream_t stream) {
  Device* d = nullptr;
  int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const bool bf16 = c.type == ATTN_BF16;
  alignas(64) CUtensorMap mk;
  if ((rc = encode_rows_map(c.k_pages, bf16, (long long)c.num_pages * ATTN_PAGE, ATTN_PAGE, CU_TENSOR_MAP_SWIZZLE_128B,
                            &mk)) != ATTN_OK)
    return rc;
  const Plan p = plan(c.B, c.max_rows, max_keys(c.max_context, c.max_rows), *d);
  WeighArgs a{};
  a.q = c.q;
  a.weights = c.weights;
  a.table = c.table;
  a.ctx_lens = c.ctx_lens;
  a.row_start = c.row_start;
  a.weighed_lens = c.weighed_lens;
  a.stats = static_cast<float2*>(c.workspace);
  a.B = c.B;
  a.N = c.N;
  a.max_rows = c.max_rows;
  a.max_blocks = c.max_blocks;
  a.num_pages = c.num_pages;
  a.max_context = c.max_context;
  a.row_tiles = (c.max_rows + kRows - 1) / kRows;
  a.splits = p.splits;
  a.key_splits = p.key_splits;
  a.decay = c.decay;
  a.err = err;
  a.withheld = c.withheld;
  a.timeout_ns = c.withheld ? kFaultNs : kTimeoutNs;
  const int first = p.once ? kOnce : p.fused ? kFused : kRowsPass, last = p.once ? kOnce : p.fused ? kFused : kKeysPass;
  for (int pass = first; pass <= last; ++pass) {
    const Choice k = bf16 ? choice<false>(pass) : choice<true>(pass);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(pass == kRowsPass ? a.splits * a.row_tiles : pass == kKeysPass ? a.key_splits : a.splits, kHKV, c.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = k.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.splits;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pass >= kFused ? 2 : 1;
    if (launched(cudaLaunchKernelEx(&cfg, k.kernel, mk, a)) != cudaSuccess) return ATTN_ELAUNCH;
  }
  return ATTN_OK;
}

}  // namespace attn
