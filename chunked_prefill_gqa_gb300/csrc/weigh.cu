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
// block adds to weights that it alone writes.
//   bf16 pages: K as stored, q in three bf16 terms: 3 x 4 MMAs of 128 x 128 x 16 a tile
//   fp32 pages: q_lo K + q K_lo + q K, tf32 terms, in halves of 32 dims: 3 x 8 of 128 x 128 x 8
// (K is read truncated; K_lo is the remainder rounded to tf32, q's first term rounded too.)
//
// Roles: three groups of four warps take the tiles in turn; four warps that write K_lo (fp32,
// rows) or move K to tensor memory (keys); one warp for TMA (16-token pages through the block
// table), one to issue the products.
#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"
#include "tree.cuh"

namespace attn {
namespace {

using namespace tc;

constexpr int kRows = 32;                  // rows of a block: 128 (row, head) pairs
constexpr int kKeys = 128;                 // keys of a tile
constexpr int kPages = kKeys / ATTN_PAGE;
constexpr int kGroups = 3, kSoft = 4 * kGroups;  // warps that read S
constexpr int kChunk = 64;                 // columns of S that a thread has in registers
constexpr int kTmaWarps = 2;               // tiles in turn: a box of 16 rows costs its warp about 100 cycles
constexpr uint32_t kHalf = 128 * 128;      // 128 rows of 128 bytes
constexpr uint32_t kBox = ATTN_PAGE * 128;
constexpr int kMaxSplits = 64;
constexpr int kWideRows = 8;               // windows from which on operands have two bf16 terms
constexpr float kNothing = 1e30f;          // reference of a row that gives nothing
constexpr unsigned kFull = 0xffffffffu;

struct WeighArgs {
  const float* q;          // [N][32][64]
  float* weights;          // [num_pages][8][16]
  const int *table, *ctx_lens, *row_start, *weighed_lens;
  float2* stats;           // [N][32][splits]: log2 maximum, sum (both 0 of a segment without keys)
  int B, N, max_rows, max_blocks, num_pages, max_context;
  int row_tiles, splits;   // of the rows pass
  int key_splits;          // of the keys pass
  float decay;
  unsigned* err;
  unsigned long long timeout_ns;
};

template <bool kF32, bool kByKey, bool kWide>
struct Lay {
  static constexpr bool kTf32 = kF32 && !kWide;  // else bf16 operands
  static constexpr bool kDirect = !kF32 && !kByKey;  // the tensor core reads K as it landed
  static constexpr bool kSlotted = kByKey || (kF32 && kWide);  // K goes on to slots, in tensor memory (keys) or shared (rows)
  static constexpr int kConvWarp = kSoft, kConvWarps = kDirect ? 0 : 4;
  static constexpr int kTmaWarp = kSoft + kConvWarps, kMmaWarp = kTmaWarp + kTmaWarps;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr uint32_t kRaw = kF32 ? 2 * kHalf : kHalf;          // a tile of K as it lands
  static constexpr uint32_t kOperand = kTf32 ? 2 * kHalf : kHalf;     // an operand of 128 rows
  static constexpr uint32_t kStageBytes = kRaw + (kTf32 && !kByKey ? kOperand : 0);  // K (, K lo)
  static constexpr int kStages = kTf32 ? 3 : kF32 ? 4 : 8;
  static constexpr int kTerms = kTf32 || kWide ? 2 : 3;               // of q
  static constexpr int kSlots = kF32 && kWide && !kByKey ? 2 : 3;
  static constexpr uint32_t kSmemSlots = kStages * kStageBytes;       // rows pass of wide windows: K's two terms
  static constexpr uint32_t kSmemQ = kSmemSlots + (kSlotted && !kByKey ? kSlots * 2 * kOperand : 0);  // keys pass: q's terms
  static constexpr uint32_t kSmemRef = kSmemQ + (kByKey ? kTerms * kOperand : 0);                    // and the references' tile
  static constexpr uint32_t kSmemEnds = kSmemRef + (kByKey ? kHalf : 0);         // rows pass: [groups][128] (reference, sum)
  static constexpr uint32_t kSmemBar = kSmemEnds + kGroups * 128 * 8;
  // Tensor memory. Rows: q's terms, then S. Keys: parts of K (tf32: halves, hi and lo), ones, S.
  static constexpr int kParts = kTf32 && kByKey ? 2 : 1;
  static constexpr uint32_t kSlotCols = kF32 ? 64 : 32;
  static constexpr uint32_t kColK = 0, kColOnes = kSlots * kSlotCols;
  static constexpr uint32_t kColQ = 0, kTermCols = kTf32 ? 64 : 32, kColS = kByKey ? kColOnes + 16 : kTerms * kTermCols;
  static constexpr int kBufs = kF32 && kByKey ? 2 : 3;
  static constexpr int kNumBars = 3 * kStages + 2 * kSlots + kGroups + kBufs + 2;
  static constexpr uint32_t kSmemWords = kSmemBar + kNumBars * 8;     // TMEM address, abort flag
  static constexpr uint32_t kSmemAlloc = kSmemWords + 16 + 1024;
  static_assert(kSmemAlloc <= 232448, "exceeds the 227 KB per-block shared memory limit");
  static_assert(kColS + kBufs * kKeys <= 512, "TMEM layout");
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
template <bool kTf32>
__device__ __forceinline__ void three_terms(float x, float (&t)[3]) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    t[i] = kTf32 ? tf32_hi(x) : bf16_trunc(x);
    x -= t[i];
  }
}

// Two bf16 terms of a pair, each rounded to nearest: 16 bits and a sign, 2^-18 of x left out.
// (A finite value that would round to infinity takes the largest bf16 number.)
__device__ __forceinline__ void split2(float x, float y, uint32_t& t0, uint32_t& t1) {
  const float most = __uint_as_float(0x7f7f0000u);
  float cx, cy, hx, hy;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(cx) : "f"(x), "f"(most));
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(cy) : "f"(y), "f"(most));
  t0 = pack_bf16_rn_keep(cx, cy, hx, hy);
  t1 = pack_bf16_rn(x - hx, y - hy);
}

// tcgen05.st of 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&u)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(u[0]), "r"(u[1]),
               "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
               : "memory");
}

template <bool kF32, bool kByKey, bool kWide>
__global__ void __launch_bounds__(Lay<kF32, kByKey, kWide>::kThreads, 1)
weigh_kernel(const __grid_constant__ CUtensorMap mk, const WeighArgs a) {
  using L = Lay<kF32, kByKey, kWide>;
  constexpr int kStages = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(kFull, tid >> 5, 0);
  if (warp == L::kTmaWarp && lane == 0) tma_prefetch_desc(&mk);
  follow();
  // Rows pass: the row tiles of a segment are neighbours in the grid and read its keys at
  // about the same time, all but one from L2.
  const int row_tiles = kByKey ? 1 : a.row_tiles;
  const int s = blockIdx.x / row_tiles, head = blockIdx.y, b = blockIdx.z;
  const Seq seq = load_window(a, b);
  if (!seq.ok && !kByKey && blockIdx.x == 0 && head == 0 && tid == 0) record_error(a.err, kDevErrBounds);
  // The rows of this block: a tile of 32 of them, or by key all tiles one after another.
  const int rt0 = kByKey ? 0 : blockIdx.x % row_tiles, rt1 = kByKey ? (seq.rows + kRows - 1) / kRows : rt0 + 1;
  if (seq.rows - rt0 * kRows <= 0) return;
  // The sequence's own keys, cut evenly into segments of whole tiles.
  const int splits = kByKey ? a.key_splits : a.splits;
  const int len = ((seq.keys + splits - 1) / splits + kKeys - 1) / kKeys * kKeys;
  const int k0 = min((long long)s * len, (long long)seq.keys), k1 = min((long long)k0 + len, (long long)seq.keys);
  // Keys that some row of row tile rt sees, and the tiles that hold them.
  const auto visible = [&](int rt) { return min(k1, seq.ctx + min(seq.rows, (rt + 1) * kRows)); };
  const auto tiles = [&](int rt) { return max(0, (visible(rt) - k0 + kKeys - 1) / kKeys); };
  if (kByKey && k0 >= k1) return;

  uint64_t* const kfull = reinterpret_cast<uint64_t*>(smem + L::kSmemBar);  // [stage] K landed
  uint64_t* const kready = kfull + kStages;                                 // [stage] K lo written (tf32, rows)
  uint64_t* const kempty = kready + kStages;                                // [stage] K read
  uint64_t* const tfull = kempty + kStages;                                 // [slot] K written there
  uint64_t* const tempty = tfull + L::kSlots;                               // [slot] products done with it
  // A group's next S: a barrier a group, since the buffers go round in another time; the group
  // has waited for its tile before the buffer's next product, and so its own, is issued.
  uint64_t* const sfull = tempty + L::kSlots;                               // [group] S written
  uint64_t* const sfree = sfull + kGroups;                                  // [buffer] S read
  uint64_t* const qready = sfree + L::kBufs;                                // q's terms of a row tile written
  uint64_t* const drain = qready + 1;
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + L::kSmemWords);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(words + 1);
  const Wait wait{a.err, a.timeout_ns, abort_flag};
  const int* const trow = a.table + (size_t)b * a.max_blocks;

  if (warp == L::kTmaWarp) {
    for (int i = lane; i < L::kNumBars; i += 32) {
      uint64_t* const bar = &kfull[i];
      const bool by_four = (bar >= kready && bar < kempty) || (L::kSlotted && bar >= kempty && bar < tempty) || (bar >= sfree && bar < qready);
      mbar_init(bar, by_four ? 4 : bar == qready ? kSoft : 1);
    }
    fence_mbar_init();
    if (lane == 0) *abort_flag = 0;
  } else if (warp == L::kMmaWarp) {
    tmem_alloc(words, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = words[0];
  int last = -1;  // the last tile that a TMA warp has asked for

  if (warp >= L::kTmaWarp && warp < L::kMmaWarp) {
    const int mine = warp - L::kTmaWarp;  // this warp's tiles: every second one
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
          if (has)
            tma_load_2d(smem + st * L::kStageBytes + half * kHalf + p * kBox, &mk, &kfull[st], head * kD + half * 32,
                        page * ATTN_PAGE);
        }
        if ((n & 3) == 3) {
          entries = entries_next;
          entries_next = entry_at((n >> 2) + 2);
        }
      }
    }
  } else if (warp == L::kMmaWarp) {
    const uint32_t base = smem_u32(smem);
    int it = 0;
    bool ok = true;
    for (int rt = rt0; ok && rt < rt1; ++rt) {
      const int count = tiles(rt);
      ok = wait.warp(qready, (rt - rt0) & 1);
      for (int n = 0; ok && n < count; ++n, ++it) {
        const int buf = it % L::kBufs;
        const uint32_t d = tmem + L::kColS + buf * kKeys;
        if (it >= L::kBufs && !(ok = wait.warp(&sfree[buf], (it / L::kBufs - 1) & 1))) break;
        constexpr uint32_t id = L::kTf32 ? idesc_tf32(128, 128) : idesc_bf16(128, 128, false);
        constexpr uint64_t lo = L::kOperand >> 4;
        if constexpr (!kByKey) {
          const int st = it % kStages, slot = it % L::kSlots;
          if (!(ok = L::kSlotted ? wait.warp(&tfull[slot], (it / L::kSlots) & 1)
                                 : wait.warp(kF32 ? &kready[st] : &kfull[st], (it / kStages) & 1)))
            break;
          tc_fence_after();
          const uint64_t kd = sdesc_sw128(base + (L::kSlotted ? L::kSmemSlots + slot * 2 * L::kOperand : st * L::kStageBytes));
          const uint32_t q = tmem + L::kColQ;
          if (elect()) {
            if constexpr (L::kTf32) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint64_t kh = kd + h * (kHalf >> 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, q + 64 + h * 32 + x * 8, kh + x * 2, id, h + x > 0);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, q + h * 32 + x * 8, kh + lo + x * 2, id, 1);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, q + h * 32 + x * 8, kh + x * 2, id, 1);
              }
            } else {
              if constexpr (kF32) {
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_f16_ts(d, q + x * 8, kd + lo + x * 2, id, x > 0);
              }
#pragma unroll
              for (int t = L::kTerms - 1; t >= 0; --t)
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_f16_ts(d, q + t * 32 + x * 8, kd + x * 2, id, kF32 || t < L::kTerms - 1 || x > 0);
            }
            mma_commit(&sfull[it % kGroups]);
            mma_commit(L::kSlotted ? &tempty[slot] : &kempty[st]);
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
              if constexpr (L::kTf32) {
                const uint64_t qh = qd + h * (kHalf >> 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, k + x * 8, qh + lo + x * 2, id, h + x > 0);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, k + 32 + x * 8, qh + x * 2, id, 1);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma_tf32_ts(d, k + x * 8, qh + x * 2, id, 1);
              } else {
                if constexpr (kF32) {
#pragma unroll
                  for (int x = 0; x < 4; ++x) mma_f16_ts(d, k + 32 + x * 8, qd + x * 2, id, x > 0);
                }
#pragma unroll
                for (int t = L::kTerms - 1; t >= 0; --t)
#pragma unroll
                  for (int x = 0; x < 4; ++x)
                    mma_f16_ts(d, k + x * 8, qd + t * lo + x * 2, id, kF32 || t < L::kTerms - 1 || x > 0);
              }
              mma_commit(&tempty[slot]);
              if (h == L::kParts - 1) {
                if constexpr (L::kTf32) mma_tf32_ts(d, tmem + L::kColOnes, rd, id, 1);
                else mma_f16_ts(d, tmem + L::kColOnes, rd, id, 1);
                mma_commit(&sfull[it % kGroups]);
              }
            }
            __syncwarp();
          }
        }
      }
    }
  } else if (warp >= L::kConvWarp && warp < L::kTmaWarp) {
    const int ctid = tid - 32 * L::kConvWarp;
    int total = 0;
    for (int rt = rt0; rt < rt1; ++rt) total += tiles(rt);
    for (int it = 0; it < total; ++it) {
      const int st = it % kStages;
      uint8_t* const stage = smem + st * L::kStageBytes;
      if (!wait.warp(&kfull[st], (it / kStages) & 1)) break;
      if constexpr (kF32 && kWide && !kByKey) {
        // K's two terms, a tile of bf16 each. A thread takes 8 dims (two 16-byte words of fp32,
        // one of bf16) of a key.
        const int slot = it % L::kSlots;
        if (it >= L::kSlots && !wait.warp(&tempty[slot], (it / L::kSlots - 1) & 1)) break;
        uint8_t* const to = smem + L::kSmemSlots + slot * 2 * L::kOperand;
        const uint32_t oct = ctid & 7, odd = oct >> 2;  // half a row apart, words of the other parity first: no bank twice
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
          float4 x[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t key = (uint32_t)(ctid >> 3) + 16u * (h + j);
            x[j][0] = *reinterpret_cast<const float4*>(stage + odd * kHalf + sw128(key * 128u + ((oct & 3) * 2 + odd) * 16u));
            x[j][1] = *reinterpret_cast<const float4*>(stage + odd * kHalf + sw128(key * 128u + ((oct & 3) * 2 + 1 - odd) * 16u));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t key = (uint32_t)(ctid >> 3) + 16u * (h + j);
            const float4 u = odd ? x[j][1] : x[j][0], v = odd ? x[j][0] : x[j][1];
            uint4 w0, w1;
            split2(u.x, u.y, w0.x, w1.x);
            split2(u.z, u.w, w0.y, w1.y);
            split2(v.x, v.y, w0.z, w1.z);
            split2(v.z, v.w, w0.w, w1.w);
            uint8_t* const at = to + sw128(key * 128u + oct * 16u);
            *reinterpret_cast<uint4*>(at) = w0;
            *reinterpret_cast<uint4*>(at + L::kOperand) = w1;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&kempty[st]);
          mbar_arrive(&tfull[slot]);
        }
      } else if constexpr (!kByKey) {
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
          float x[32];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(x + 4 * i) =
                *reinterpret_cast<const float4*>(stage + h * kHalf + sw128((uint32_t)ctid * 128u + i * 16u));
          if (h == L::kParts - 1 && !(kF32 && kWide)) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&kempty[st]);
          }
          if (part >= L::kSlots && !(ok = wait.warp(&tempty[slot], (part / L::kSlots - 1) & 1))) break;
          tc_fence_after();
          const uint32_t at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + L::kColK + slot * L::kSlotCols;
          if constexpr (kF32 && kWide) {
            // Two bf16 terms of the 32 dims; the other half of the row follows.
            uint32_t w0[16], w1[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], w0[i], w1[i]);
            tmem_st16(at, w0);
            tmem_st16(at + 32, w1);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(x + 4 * i) =
                  *reinterpret_cast<const float4*>(stage + kHalf + sw128((uint32_t)ctid * 128u + i * 16u));
            __syncwarp();
            if (lane == 0) mbar_arrive(&kempty[st]);
#pragma unroll
            for (int i = 0; i < 16; ++i) split2(x[2 * i], x[2 * i + 1], w0[i], w1[i]);
            tmem_st16(at + 16, w0);
            tmem_st16(at + 48, w1);
          } else {
            tmem_st32(at, x);
            if constexpr (kF32) {
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] = tf32_near(x[i] - tf32_hi(x[i]));
              tmem_st32(at + 32, x);
            }
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
    for (int rt = rt0; rt < rt1; ++rt) {
      const int i0 = rt * kRows, nrows = min(kRows, seq.rows - i0);
      const bool in = (row >> 2) < nrows;
      const size_t pair = (size_t)(seq.first + i0 + (row >> 2)) * kHQ + head * kGroup + (row & 3);
      if (rt > rt0) {  // what the tile before needs is still in use; its weights are written
        int over;
        if (meet(kMeet, false, failed, lane, &over)) break;
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
        if constexpr (!kByKey && L::kTf32) {
          uint32_t w[2][16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float h = tf32_near(x[i]);
            w[0][i] = __float_as_uint(h), w[1][i] = __float_as_uint(x[i] - h);
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) tmem_st16(lane_tmem + L::kColQ + t * 64 + c * 16, w[t]);
        } else if constexpr (!kByKey) {
          uint32_t w[3][8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (kWide) split2(x[2 * i], x[2 * i + 1], w[0][i], w[1][i]);
            else split3_cut(x[2 * i], x[2 * i + 1], w[0][i], w[1][i], w[2][i]);
          }
#pragma unroll
          for (int t = 0; t < L::kTerms; ++t) tmem_st8(lane_tmem + L::kColQ + t * 32 + c * 8, w[t]);
        } else if constexpr (L::kTf32) {
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            uint8_t* const at = smem + L::kSmemQ + (c >> 1) * kHalf + sw128((uint32_t)row * 128u + (c & 1) * 64u + i * 4u);
            const float4 h = make_float4(tf32_near(x[i]), tf32_near(x[i + 1]), tf32_near(x[i + 2]), tf32_near(x[i + 3]));
            *reinterpret_cast<float4*>(at) = h;
            *reinterpret_cast<float4*>(at + L::kOperand) = make_float4(x[i] - h.x, x[i + 1] - h.y, x[i + 2] - h.z, x[i + 3] - h.w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; i += 8) {
            uint32_t w[3][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if (kWide) split2(x[i + 2 * j], x[i + 2 * j + 1], w[0][j], w[1][j]);
              else split3_cut(x[i + 2 * j], x[i + 2 * j + 1], w[0][j], w[1][j], w[2][j]);
            }
            uint8_t* const at = smem + L::kSmemQ + sw128((uint32_t)row * 128u + c * 32u + i * 2u);
#pragma unroll
            for (int t = 0; t < L::kTerms; ++t) *reinterpret_cast<uint4*>(at + t * L::kOperand) = make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
          }
        }
      }
              if (kByKey && g == kGroups - 1) {
                // The row's reference and the logarithm of its sum over all keys, from the segments.
                float top = kUnseen, sum = 0.f;
                if (in) {
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
                three_terms<L::kTf32>(sum == 0.f ? -kNothing : -top, *reinterpret_cast<float(*)[3]>(t));
                three_terms<L::kTf32>(sum == 0.f ? 0.f : -log2f(sum), *reinterpret_cast<float(*)[3]>(t + 3));
                uint4 u0, u1 = make_uint4(0, 0, 0, 0);
                if constexpr (L::kTf32) {
                  u0 = make_uint4(__float_as_uint(t[0]), __float_as_uint(t[1]), __float_as_uint(t[2]), __float_as_uint(t[3]));
                  u1.x = __float_as_uint(t[4]), u1.y = __float_as_uint(t[5]);
                } else {
                  u0 = make_uint4(pack_bf16_trunc(t[0], t[1]), pack_bf16_trunc(t[2], t[3]), pack_bf16_trunc(t[4], t[5]), 0u);
                }
                *reinterpret_cast<uint4*>(smem + L::kSmemRef + sw128((uint32_t)row * 128u)) = u0;
                *reinterpret_cast<uint4*>(smem + L::kSmemRef + sw128((uint32_t)row * 128u + 16u)) = u1;
                if (rt == rt0) {
                  constexpr uint32_t kOne = L::kTf32 ? 0x3f800000u : 0x3f803f80u;
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
      for (int n = (g + kGroups - done % kGroups) % kGroups; n < count; n += kGroups) {
        const int it = done + n, buf = it % L::kBufs, t0 = k0 + n * kKeys;
        const uint32_t s_tmem = lane_tmem + L::kColS + buf * kKeys;
        if constexpr (kByKey) {
          const int t = t0 + row;
          // The key's weight so far, on its way while the products run. Row tile (t - context) /
          // 32 is the first that sees a token of the rows themselves, 0 any other.
          float* w = nullptr;
          float old = 0.f;
          if (t < visible(rt)) {
            const int page = fetch(trow + t / ATTN_PAGE);
            if (page >= 0 && page < a.num_pages) {
              w = a.weights + ((size_t)page * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE;
              if (rt > max(0, t - seq.ctx) / kRows) old = *w;
              else if (a.decay != 0.f && t < weighed) old = a.decay * *w;
            }
          }
          failed |= !wait.warp(&sfull[g], (it / kGroups) & 1);
          tc_fence_after();
          float sum0 = 0.f, sum1 = 0.f;
          const int late = t - seq.ctx - i0;  // rows before it do not see the key
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
            if (t0 + kKeys > seq.ctx + i0) {
#pragma unroll
              for (int i = 0; i < kChunk; ++i)
                if ((h + i) / 4 < late) x[i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < kChunk; i += 2) add2(sum0, sum1, sum0, sum1, ex2(x[i]), ex2(x[i + 1]));
          }
          if (w && !failed) *w = old + (sum0 + sum1);
        } else {
          failed |= !wait.warp(&sfull[g], (it / kGroups) & 1);
          tc_fence_after();
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
    }
    if constexpr (!kByKey) {
      float2* const ends = reinterpret_cast<float2*>(smem + L::kSmemEnds);
      if (g > 0) ends[g * 128 + row] = make_float2(ref, l0 + l1);
      int over;
      const bool lost = meet(kMeet, false, failed, lane, &over);
      const int i = rt0 * kRows + (row >> 2);
      if (g == 0 && i < seq.rows) {
        float top = ref;
#pragma unroll
        for (int x = 1; x < kGroups; ++x) top = fmaxf(top, ends[x * 128 + row].x);
        float sum = ex2(ref - top) * (l0 + l1);
#pragma unroll
        for (int x = 1; x < kGroups; ++x) sum = fmaf(ex2(ends[x * 128 + row].x - top), ends[x * 128 + row].y, sum);
        a.stats[((size_t)(seq.first + i) * kHQ + head * kGroup + (row & 3)) * a.splits + s] =
            lost ? make_float2(kUnseen, 0.f) : make_float2(top, sum);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (warp >= L::kTmaWarp && warp < L::kMmaWarp)  // its copies still in flight
      for (int i = last; i >= 0 && i > last - kStages; i -= kTmaWarps) mbar_wait(&kfull[i % kStages], (i / kStages) & 1, a.timeout_ns);
    if (warp == L::kMmaWarp) drain_products(drain, a.timeout_ns);
    __syncthreads();
  }
  if (warp == L::kMmaWarp) tmem_dealloc(tmem, 512);
}

struct Device {
  bool ready = false;
  int sms = 0;
};
// A pass of the call: its kernel, threads and shared memory.
struct Pass {
  void (*kernel)(CUtensorMap, WeighArgs);
  int threads;
  uint32_t smem;
};
template <bool kF32, bool kWide>
Pass pass_of(bool by_key) {
  if (by_key) return {weigh_kernel<kF32, true, kWide>, Lay<kF32, true, kWide>::kThreads, Lay<kF32, true, kWide>::kSmemAlloc};
  return {weigh_kernel<kF32, false, kWide>, Lay<kF32, false, kWide>::kThreads, Lay<kF32, false, kWide>::kSmemAlloc};
}
Pass pass_of(bool f32, bool wide, bool by_key) {
  return f32 ? (wide ? pass_of<true, true>(by_key) : pass_of<true, false>(by_key))
             : (wide ? pass_of<false, true>(by_key) : pass_of<false, false>(by_key));
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
      const Pass p = pass_of(i & 1, i & 2, i & 4);
      ok = ok && cudaFuncSetAttribute(p.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)p.smem) == cudaSuccess;
    }
    if (!ok) {
      (void)cudaGetLastError();
      return ATTN_ECUDA;
    }
    d.ready = true;
  }
  *out = &d;
  return ATTN_OK;
}

// Segments of the keys for `units` blocks each: the number whose rounds of one block an SM
// take the least time, a block costing its tiles (each of them `passes` times) and as long
// as four tiles besides.
int plan(long long units, int max_keys, int passes, int sms) {
  const int tiles = (max_keys + kKeys - 1) / kKeys;
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    const long long rounds = (units * s + sms - 1) / sms;
    const double time = (double)rounds * ((double)((tiles + s - 1) / s) * passes + 4.0 * passes);
    if (time < least * 0.999) least = time, best = s;
  }
  return best;
}

int max_keys(int max_context, int max_rows) {
  return max_context > ATTN_MAX_TOKENS - max_rows ? ATTN_MAX_TOKENS : max_context + max_rows;
}

}  // namespace

int weigh_workspace_bytes(int B, int N, int max_rows, int max_context, size_t* bytes) {
  Device* d = nullptr;
  const int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const int tiles = (max_rows + kRows - 1) / kRows;
  *bytes = (size_t)N * kHQ * plan((long long)B * kHKV * tiles, max_keys(max_context, max_rows), 1, d->sms) * sizeof(float2);
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
  const int tiles = (c.max_rows + kRows - 1) / kRows;
  const int keys = max_keys(c.max_context, c.max_rows);
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
  a.row_tiles = tiles;
  a.splits = plan((long long)c.B * kHKV * tiles, keys, 1, d->sms);
  a.key_splits = plan((long long)c.B * kHKV, keys, tiles, d->sms);
  a.decay = c.decay;
  a.err = err;
  a.timeout_ns = kTimeoutNs;
  for (int by_key = 0; by_key < 2; ++by_key) {
    const Pass p = pass_of(!bf16, c.max_rows >= kWideRows, by_key);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(by_key ? a.key_splits : a.splits * tiles, kHKV, c.B);
    cfg.blockDim = dim3(p.threads);
    cfg.dynamicSmemBytes = p.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (launched(cudaLaunchKernelEx(&cfg, p.kernel, mk, a)) != cudaSuccess) return ATTN_ELAUNCH;
  }
  return ATTN_OK;
}

}  // namespace attn
