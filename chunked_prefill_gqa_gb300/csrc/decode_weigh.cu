// decode_weigh.cu -- attention of one new token a sequence over its paged cache that
// also adds what every cached token was given to that token's weight:
//   s_hj = q_h . k_j / 8,  p_hj = softmax_j(s_hj),  out_h = sum_j p_hj v_j
//   W[j][g] = (decay W[j][g], or 0 for a token without a weight yet) + sum of p_hj, the 4 heads h of g
//
// p needs the maximum and sum over all keys, which are known at the end. So the kernel that
// reads K and V once keeps the scores (16 bytes a token and KV head, where K and V are 256 or
// 512), and the weights are added from them afterwards. Two forms:
//   cluster  up to eight segments of a (sequence, KV head) are one cluster of blocks. Each
//            keeps its scores in shared memory (up to 2448 tokens), they exchange maxima and
//            sums through distributed shared memory, and each adds its own tokens' weights:
//            one launch, nothing through memory but what the call is about
//   memory   longer contexts: scores and partials in the workspace, a second kernel merges
// (Clusters whose scores wait in tensor memory, 8192 tokens a block, were built: 16 sequences of
// 16384 tokens, bf16 pages, 98 us for 101, lengths of 1600 to 16384 63 for 60.)
//
// A block owns (segment, KV head, sequence), each of its warps (eight, four on fp32 pages) every
// eighth (fourth) 16-token page, which arrives by TMA in a ring of the warp's own; warps meet only
// at the end. A page is exactly the 16 rows of mma.sync, keys on the M side, and the 8
// columns of N hold the four query heads in two terms each, so a thread ends with the
// scores of two keys and one head, already summed over the terms:
//   bf16 pages: S^T = K (q1 | q2) + K (q3 | 0), O^T += V^T (p1 | p2) + V^T (p3 | 0)
//   fp32 pages: S^T = (K hi + K lo)(q hi | q lo), O^T += (V hi + V lo)(p hi | p lo), tf32 terms
// K and V of bf16 pages are used as stored; the three bf16 (two tf32) terms keep q and p in
// fp32 precision. A page's products start at zero and join the fp32 sums rounded to
// nearest. A head's reference maximum moves when a score passes it by 2^8.
//
// (Two pages at a time a warp, with twice the registers, made no difference; eight warps for four,
// each with half the ring: 104 to 102 us for 16 sequences of 16384 tokens, bf16 pages.)
// Bound by reading K and V: those 16 sequences (554 MB) 102 us, 5.4 TB/s; one
// of 131071 (bf16, 277 MB) 52 us; 48 of 410 to 4096 (fp32, 453 MB) 82 us, 5.5 TB/s; one of 1000
// (fp32, 4 MB), cluster form, 6.0 us, of which 2.5 are an empty call.
#include <cuda.h>

#include <mutex>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "tensor_map.cuh"
#include "tree.cuh"

namespace attn {
namespace {

using namespace tc;

constexpr int kPartFloats = kGroup * kD + 2 * kGroup;  // O of 4 heads, then their log2 maxima and sums
constexpr float kFailed = -1.f;                        // sum of a segment whose tiles never came
constexpr unsigned kFull = 0xffffffffu;
constexpr int kMaxSplits = 64;                         // a lane of the merge has two segments
constexpr uint32_t kBox = ATTN_PAGE * 128;             // 16 rows of 128 bytes
constexpr int kMaxKept = 2448;                         // tokens of a segment whose scores a block keeps

template <bool kF32, bool kCluster>
struct Pages {
  static constexpr int kWarps = kF32 ? 4 : 8, kThreads = 32 * kWarps;
  static constexpr uint32_t kOperand = kF32 ? 2 * kBox : kBox;  // a page of K or V of a head; fp32 in halves of 32 dims
  static constexpr uint32_t kStageBytes = 2 * kOperand;
  static constexpr int kStages = kCluster ? 2 : 3;  // 64 or 96 KB a block, two blocks an SM
  static constexpr uint32_t kRing = kStages * kStageBytes;
  static constexpr uint32_t kSmemAcc = kWarps * kRing;                        // [warps][4][64] floats
  static constexpr uint32_t kSmemMl = kSmemAcc + kWarps * kGroup * kD * 4;    // [warps][4] (maximum, sum), then [4] of all
  static constexpr uint32_t kSmemOut = kSmemMl + (kWarps + 1) * kGroup * 8;   // cluster: [4][64] floats, [4] (maximum, sum)
  static constexpr uint32_t kSmemBar = kSmemOut + (kCluster ? kGroup * kD * 4 + kGroup * 8 : 0);
  static constexpr uint32_t kSmemScores = (kSmemBar + kWarps * kStages * 8 + 15) / 16 * 16;  // cluster: float4 a token
  static constexpr uint32_t kSmemAlloc = kSmemScores + 1024;                  // and the scores
  static_assert(2 * (kSmemAlloc + 1024 + (kCluster ? kMaxKept * 16 : 0)) <= 233472, "shared memory of an SM");
};

struct DecodeWeighArgs {
  const float* q;          // [B][32][64]
  float* weights;          // [num_pages][8][16]
  const int *table, *ctx_lens, *weighed_lens;
  float* out;              // [B][32][64]
  float4* scores;          // [B][8][stride]: log2 scores of a token, four heads
  float* parts;            // [B][8][splits][kPartFloats], with more than one segment
  int B, max_blocks, num_pages, max_context, splits;
  long long stride;        // tokens: max_context rounded up to a page
  float decay;
  int withheld;            // failure test: segments whose first pages are never loaded
  unsigned* err;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ int checked_ctx(const DecodeWeighArgs& a, int b, bool tell) {
  const int ctx = fetch(a.ctx_lens + b);
  const int most = min((long long)a.max_context, (long long)a.max_blocks * ATTN_PAGE);
  if (ctx >= 0 && ctx <= most) return ctx;
  if (tell) record_error(a.err, kDevErrBounds);
  return ctx < 0 ? 0 : most;
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], float a0, float a1, float a2, float a3, float b0, float b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(__float_as_uint(a0)), "r"(__float_as_uint(a1)), "r"(__float_as_uint(a2)), "r"(__float_as_uint(a3)),
        "r"(__float_as_uint(b0)), "r"(__float_as_uint(b1)));
}
template <bool kTrans>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// A score that waits in L2 for the second kernel, while 16 times as many bytes of K and V go
// through (16 sequences of 16384 tokens on bf16 pages: 110 to 108 us).
__device__ __forceinline__ void store_kept(float* p, float x, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(p), "f"(x), "l"(policy) : "memory");
}

// What a (sequence, head)'s four query heads have in common over all keys.
struct Heads {
  float top[kGroup], inv[kGroup];  // log2 maximum, inverse sum (0: all scores -inf, which give nothing)
};
__device__ __forceinline__ float given(float4 s, const Heads& x) {
  const float g0 = x.inv[0] == 0.f ? 0.f : ex2(s.x - x.top[0]) * x.inv[0];
  const float g1 = x.inv[1] == 0.f ? 0.f : ex2(s.y - x.top[1]) * x.inv[1];
  const float g2 = x.inv[2] == 0.f ? 0.f : ex2(s.z - x.top[2]) * x.inv[2];
  const float g3 = x.inv[3] == 0.f ? 0.f : ex2(s.w - x.top[3]) * x.inv[3];
  return (g0 + g1) + (g2 + g3);
}

// Tokens first + t, first + t + kThreads, ... of (b, head) with their scores (of first on),
// places and old weights, all on their way before any is used (while partial sums are merged).
template <int kThreads, int kTokens>
struct Tokens {
  float4 s[kTokens];
  float* w[kTokens];  // nullptr: no such token, or on a page that is none (recorded where its keys were read)
  float old[kTokens];
  __device__ __forceinline__ void load(const DecodeWeighArgs& a, const float4* scores, int b, int head, int first, int t, int count,
                                       int weighed) {
    int page[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int at = t + i * kThreads;
      page[i] = at < count ? fetch(a.table + (size_t)b * a.max_blocks + (first + at) / ATTN_PAGE) : -1;
      if (at < count) s[i] = fetch(scores + at);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const int at = first + t + i * kThreads;
      w[i] = page[i] >= 0 && page[i] < a.num_pages
                 ? a.weights + ((size_t)page[i] * kHKV + head) * ATTN_PAGE + at % ATTN_PAGE : nullptr;
      old[i] = w[i] && a.decay != 0.f && at < weighed ? a.decay * *w[i] : 0.f;
    }
  }
  __device__ __forceinline__ void store(const Heads& x, int i) const {
    if (w[i]) *w[i] = old[i] + given(s[i], x);
  }
};

template <bool kF32, bool kCluster>
__global__ void __launch_bounds__(Pages<kF32, kCluster>::kThreads, 2)
decode_weigh_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const DecodeWeighArgs a) {
  using L = Pages<kF32, kCluster>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int c = lane & 3, r = lane >> 2;  // of the fragments: column pair (the thread's head), row
  const int s = blockIdx.x, head = blockIdx.y, b = blockIdx.z;
  if (tid < 2) tma_prefetch_desc(tid ? &mv : &mk);
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + L::kSmemBar) + warp * L::kStages;
  if (lane < L::kStages) mbar_init(&full[lane], 1);
  fence_mbar_init();
  __syncwarp();
  follow();

  uint64_t policy = 0;
  if (!kCluster) asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  const int ctx = checked_ctx(a, b, s == 0 && head == 0 && tid == 0);
  const int pages = (ctx + ATTN_PAGE - 1) / ATTN_PAGE, per = (pages + a.splits - 1) / a.splits;
  const int p0 = s * per, p1 = min(p0 + per, pages);  // the segment's pages
  const int count = max(0, (p1 - p0 - warp + kWarps - 1) / kWarps);  // this warp's: p0 + warp, then every kWarps-th
  uint8_t* const ring = smem + warp * L::kRing;
  // Of the segment's first token on.
  float4* const scores = kCluster ? reinterpret_cast<float4*>(smem + L::kSmemScores)
                                  : a.scores + ((size_t)b * kHKV + head) * a.stride + (size_t)p0 * ATTN_PAGE;

  // Lane l holds the table's entry of the warp's page l of a group of 32.
  const int* const trow = a.table + (size_t)b * a.max_blocks;
  const auto entry_at = [&](int n) -> int { return n < count ? fetch(trow + p0 + warp + kWarps * n) : -1; };
  int entries = entry_at(lane), entries_next = entry_at(32 + lane);
  const int never = s < a.withheld ? 0 : -1;
  const auto issue = [&](int n) {
    const int st = n % L::kStages;
    int page = __shfl_sync(kFull, entries, n & 31);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], L::kStageBytes);
    __syncwarp();
    if (lane < (kF32 ? 4 : 2) && n != never) {
      if (page < 0 || page >= a.num_pages) {
        record_error(a.err, kDevErrBounds);
        page = a.num_pages;  // past the pool's end: zeros
      }
      const int half = kF32 ? lane & 1 : 0;
      const bool v = lane >= (kF32 ? 2 : 1);
      tma_load_2d(ring + st * L::kStageBytes + lane * kBox, v ? &mv : &mk, &full[st], head * kD + half * 32, page * ATTN_PAGE);
    }
    if ((n & 31) == 31) {
      entries = entries_next;
      entries_next = entry_at((n >> 5) * 32 + 64 + lane);
    }
  };
  for (int n = 0; n < min(count, L::kStages); ++n) issue(n);

  // q in its terms: column r of N is head r / 2, term r % 2.
  const float* const q = a.q + ((size_t)b * kHQ + head * kGroup + (r >> 1)) * kD;
  const bool second = r & 1;
  uint32_t qa[8], qb[8];   // bf16: k-step x in 2 x, 2 x + 1; terms 1 and 2, term 3 and zeros
  float qf[16];            // fp32: k-step x in 2 x, 2 x + 1
  if constexpr (kF32) {
    // Which dim a k index stands for is free as long as q and K agree: thread c takes dims 16 i
    // + 4 c .. + 3 as k = c and c + 4 of steps 2 i and 2 i + 1, one 16-byte load.
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = fetch(reinterpret_cast<const float4*>(q + 16 * i + 4 * c));
      const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float h = tf32_near(y[j]);
        qf[4 * i + j] = second ? y[j] - h : h;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 x = fetch(reinterpret_cast<const float2*>(q + 8 * i + 2 * c));
      uint32_t t0, t1, t2;
      split3_cut(x.x, x.y, t0, t1, t2);
      qa[i] = second ? t1 : t0;
      qb[i] = second ? 0u : t2;
    }
  }

  float ref = kUnseen, l = 0.f, o[8];  // of head c; o: dims by the V fragment's rows
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  bool failed = false;
  int n = 0;
#pragma unroll 1
  for (; n < count; ++n) {
    const int st = n % L::kStages;
    if (!__all_sync(kFull, mbar_wait(&full[st], (n / L::kStages) & 1, a.timeout_ns))) {
      failed = true;
      break;
    }
    uint8_t* const kt = ring + st * L::kStageBytes;
    uint8_t* const vt = kt + L::kOperand;
    const int t0 = (p0 + warp + kWarps * n) * ATTN_PAGE;
    const int valid = ctx - t0;  // keys of the page, 16 or more but for the sequence's last
    if (valid < ATTN_PAGE) {
      // What lies behind the last token may be NaN and gets no weight: zeros. (The warp's
      // last page: nothing is loaded over it.)
      for (int e = lane; e < (ATTN_PAGE - valid) * 8; e += 32) {
        uint8_t* const at = vt + (valid + e / 8) * 128 + (e & 7) * 16;
        *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
        if (kF32) *reinterpret_cast<uint4*>(at + kBox) = make_uint4(0, 0, 0, 0);
      }
      __syncwarp();
    }
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    int key0;  // the thread's keys: key0 and key0 + 8
    if constexpr (kF32) {
      // Fragment row r is key (r / 2) + 4 (r % 2): two neighbouring rows of one load phase
      // then lie in different halves of the swizzled banks.
      key0 = (r >> 1) | ((r & 1) << 2);
      float4 k0[4], k1[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t at = (i >> 1) * kBox + key0 * 128 + ((((i & 1) * 4 + c) ^ (key0 & 7)) << 4);
        k0[i] = *reinterpret_cast<const float4*>(kt + at);
        k1[i] = *reinterpret_cast<const float4*>(kt + at + 8 * 128);
      }
#pragma unroll
      for (int part = 1; part >= 0; --part)  // the small products first
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u[4] = {k0[i].x, k0[i].y, k0[i].z, k0[i].w}, w[4] = {k1[i].x, k1[i].y, k1[i].z, k1[i].w};
          float f[4], g[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            f[j] = tf32_near(u[j]);
            g[j] = tf32_near(w[j]);
            if (part) f[j] = u[j] - f[j], g[j] = w[j] - g[j];
          }
          mma_tf32(x, f[0], g[0], f[1], g[1], qf[4 * i], qf[4 * i + 1]);
          mma_tf32(x, f[2], g[2], f[3], g[3], qf[4 * i + 2], qf[4 * i + 3]);
        }
    } else {
      key0 = r;
      const int key = (lane & 7) + (lane & 8);
      uint32_t k[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ldmatrix4<false>(k[i], smem_u32(kt) + key * 128 + (((2 * i + (lane >> 4)) ^ (key & 7)) << 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_bf16(x, k[i], qb[2 * i], qb[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_bf16(x, k[i], qa[2 * i], qa[2 * i + 1]);
    }
    const float s0 = key0 < valid ? (x[0] + x[1]) * kTreeC : -INFINITY;
    const float s1 = key0 + 8 < valid ? (x[2] + x[3]) * kTreeC : -INFINITY;
    float* const keep = reinterpret_cast<float*>(scores + (t0 - p0 * ATTN_PAGE) + key0) + c;
    if constexpr (kCluster) {
      keep[0] = s0;
      keep[8 * 4] = s1;
    } else {
      store_kept(keep, s0, policy);
      store_kept(keep + 8 * 4, s1, policy);
    }
    if (__any_sync(kFull, fmaxf(s0, s1) > ref + kTreeStale)) {
      float most = fmaxf(s0, s1);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(kFull, most, off));
      if (most > ref + kTreeStale) {
        const float alpha = ex2(ref - most);
        ref = most;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= alpha;
      }
    }
    const float e0 = ex2(s0 - ref), e1 = ex2(s1 - ref);
    l += e0 + e1;
    // p as the B operand: this thread's column r is head r / 2, term r % 2.
    if constexpr (kF32) {
      // k index -> key: step t, k = j (+ 4): key 8 t + 2 j (+ 1), as V's rows are read below.
      const int from = ((c & 1) * 4 + (c >> 1)) * 4 + (r >> 1);  // fragment row of key 2 c, its head
      const float p[4] = {__shfl_sync(kFull, e0, from), __shfl_sync(kFull, e0, from + 8),
                          __shfl_sync(kFull, e1, from), __shfl_sync(kFull, e1, from + 8)};
      float pt[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float h = tf32_hi(p[j]);
        pt[j] = second ? p[j] - h : h;
      }
      // Thread (r, c) takes four dims 4 r .. of each half of a key's row: m-tile x has dim 4 r
      // + x in fragment row r, 32 + 4 r + x in row r + 8. Keys 2 c (+ 1): conflict-free.
      float d[4][4];
#pragma unroll
      for (int m = 0; m < 4; ++m) d[m][0] = d[m][1] = d[m][2] = d[m][3] = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        float v[2][2][4];  // [key][half][dim]
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int key = 8 * t + 2 * c + k;
          const uint32_t at = key * 128 + ((r ^ (key & 7)) << 4);
          *reinterpret_cast<float4*>(v[k][0]) = *reinterpret_cast<const float4*>(vt + at);
          *reinterpret_cast<float4*>(v[k][1]) = *reinterpret_cast<const float4*>(vt + kBox + at);
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float h00 = tf32_near(v[0][0][m]), h01 = tf32_near(v[0][1][m]), h10 = tf32_near(v[1][0][m]),
                      h11 = tf32_near(v[1][1][m]);
          mma_tf32(d[m], v[0][0][m] - h00, v[0][1][m] - h01, v[1][0][m] - h10, v[1][1][m] - h11, pt[2 * t], pt[2 * t + 1]);
          mma_tf32(d[m], h00, h01, h10, h11, pt[2 * t], pt[2 * t + 1]);
        }
      }
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        o[2 * m] += d[m][0] + d[m][1];
        o[2 * m + 1] += d[m][2] + d[m][3];
      }
    } else {
      const int from = 8 * c + (r >> 1);  // key 2 c
      uint32_t t0_, t1_, t2_, u0, u1, u2;
      split3(__shfl_sync(kFull, e0, from), __shfl_sync(kFull, e0, from + 4), t0_, t1_, t2_);
      split3(__shfl_sync(kFull, e1, from), __shfl_sync(kFull, e1, from + 4), u0, u1, u2);
      const uint32_t ba0 = second ? t1_ : t0_, ba1 = second ? u1 : u0, bb0 = second ? 0u : t2_, bb1 = second ? 0u : u2;
      const int key = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        uint32_t v[4];
        ldmatrix4<true>(v, smem_u32(vt) + key * 128 + (((2 * m + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_bf16(d, v, bb0, bb1);
        mma_bf16(d, v, ba0, ba1);
        o[2 * m] += d[0] + d[1];
        o[2 * m + 1] += d[2] + d[3];
      }
    }
    __syncwarp();  // the stage has been read by every lane
    if (n + L::kStages < count) issue(n + L::kStages);
  }
  if (failed) {  // what is still in flight lands before the block's memory is released
    if (lane == 0) record_error(a.err, kDevErrTimeout);
    for (int i = n; i < min(count, n + L::kStages); ++i) mbar_wait(&full[i % L::kStages], (i / L::kStages) & 1, a.timeout_ns);
  }
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);

  // The warps' sums.
  float* const acc = reinterpret_cast<float*>(smem + L::kSmemAcc);
  float2* const ml = reinterpret_cast<float2*>(smem + L::kSmemMl);
  if (r == 0) ml[warp * kGroup + c] = make_float2(ref, l);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int d0 = kF32 ? 4 * r + m : 16 * m + r, d1 = kF32 ? 32 + 4 * r + m : 16 * m + r + 8;
    acc[(warp * kGroup + c) * kD + d0] = o[2 * m];
    acc[(warp * kGroup + c) * kD + d1] = o[2 * m + 1];
  }
  const bool lost = __syncthreads_or(failed);
  const int h = warp % kGroup;  // (with eight warps, two do the same and one writes)
  const bool writer = warp < kGroup;
  float top = kUnseen;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * kGroup + h].x);
  float sum = 0.f;
  float2 y = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float2 p = ml[w * kGroup + h], v = *reinterpret_cast<const float2*>(acc + (w * kGroup + h) * kD + 2 * lane);
    const float f = ex2(p.x - top);  // (a warp without keys: sums of zero)
    sum = fmaf(f, p.y, sum);
    y.x = fmaf(f, v.x, y.x);
    y.y = fmaf(f, v.y, y.y);
  }
  const int first = p0 * ATTN_PAGE, end = min(p1 * ATTN_PAGE, ctx);  // the segment's tokens
  const int weighed = a.weighed_lens ? fetch(a.weighed_lens + b) : ctx - 1;
  Heads heads;
  float2* const all = ml + kWarps * kGroup;
  if constexpr (kCluster) {
    // Every block's sums to all: lane x of warp h looks at head h of block x.
    float* const mine = reinterpret_cast<float*>(smem + L::kSmemOut);
    float2* const ends = reinterpret_cast<float2*>(mine + kGroup * kD);
    if (writer) *reinterpret_cast<float2*>(mine + h * kD + 2 * lane) = y;
    if (writer && lane == 0) ends[h] = make_float2(top, lost ? kFailed : sum);
    Tokens<kThreads, 4> x;  // its first tokens' places and weights meanwhile
    x.load(a, scores, b, head, first, tid, end - first, weighed);
    __syncwarp();
    cluster_sync_all();
    float2 p = make_float2(kUnseen, 0.f);
    if (lane < a.splits) p = ld_cluster2(mapa_shared(smem_u32(ends + h), lane));
    const bool none = p.y == kFailed;
    if (none) p = make_float2(kUnseen, 0.f);
    float m = p.x;
#pragma unroll
    for (int off = 1; off < kMaxCluster; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
    m = __shfl_sync(kFull, m, 0);
    const float f = ex2(p.x - m);
    float total = f * p.y;
#pragma unroll
    for (int off = 1; off < kMaxCluster; off <<= 1) total += __shfl_xor_sync(kFull, total, off);
    total = __shfl_sync(kFull, total, 0);
    const float inv = total == 0.f ? 0.f : 1.f / total;  // no key: zeros
    // Block s writes every a.splits-th pair of dims.
    const unsigned gone = __ballot_sync(kFull, none);
    const bool writes = writer && tid % a.splits == s;
    float2 z = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      const float w = __shfl_sync(kFull, f, i);
      if (!writes || i >= a.splits || (gone >> i & 1)) continue;
      const float2 v = ld_cluster2(mapa_shared(smem_u32(mine + h * kD + 2 * lane), i));
      z.x = fmaf(w, v.x, z.x);
      z.y = fmaf(w, v.y, z.y);
    }
    if (writes)
      *reinterpret_cast<float2*>(a.out + ((size_t)b * kHQ + head * kGroup + h) * kD + 2 * lane) = make_float2(z.x * inv, z.y * inv);
    if (writer && lane == 0) all[h] = make_float2(m, inv);
    __syncwarp();
    cluster_arrive();  // the others' shared memory has been read
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGroup; ++i) heads.top[i] = all[i].x, heads.inv[i] = all[i].y;
    if (!lost) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x.store(heads, i);
      for (int t = tid + 4 * kThreads; t < end - first; t += 4 * kThreads) {
        x.load(a, scores, b, head, first, t, end - first, weighed);
#pragma unroll
        for (int i = 0; i < 4; ++i) x.store(heads, i);
      }
    }
    __syncwarp();
    cluster_wait();
    return;
  }
  if (a.splits > 1) {
    float* const part = a.parts + (((size_t)b * kHKV + head) * a.splits + s) * kPartFloats;
    if (writer) *reinterpret_cast<float2*>(part + h * kD + 2 * lane) = y;
    if (writer && lane == 0) {
      part[kGroup * kD + h] = top;
      part[kGroup * kD + kGroup + h] = lost ? kFailed : sum;
    }
    return;
  }
  if (lost) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // no key: zeros
  if (writer) *reinterpret_cast<float2*>(a.out + ((size_t)b * kHQ + head * kGroup + h) * kD + 2 * lane) = make_float2(y.x * inv, y.y * inv);
  if (writer && lane == 0) all[h] = make_float2(top, inv);
  __syncthreads();  // and the block's scores are visible to it
#pragma unroll
  for (int i = 0; i < kGroup; ++i) heads.top[i] = all[i].x, heads.inv[i] = all[i].y;
  for (int t = tid; t < ctx; t += 2 * kThreads) {
    Tokens<kThreads, 2> x;
    x.load(a, scores, b, head, 0, t, ctx, weighed);
#pragma unroll
    for (int i = 0; i < 2; ++i) x.store(heads, i);
  }
}

// Merges the segments of (sequence, head): the last block of a row of the grid writes the
// output, each of the others adds the weights of a stretch of tokens, whose scores arrive as one
// copy (held in registers they would leave an SM half of its blocks).
constexpr int kPerThread = 8, kMergeThreads = 32 * kGroup, kStretch = kPerThread * kMergeThreads;
__global__ void __launch_bounds__(kMergeThreads, 12) decode_weigh_merge_kernel(const DecodeWeighArgs a) {
  __shared__ __align__(16) float4 scores[kStretch];
  __shared__ uint64_t full;
  __shared__ Heads heads;
  __shared__ unsigned lost[2];
  const int head = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, h = tid >> 5;
  if (tid == 0) {
    mbar_init(&full, 1);
    fence_mbar_init();
  }
  __syncthreads();
  // Before the wait for the grid that reads K and V: what that grid only reads or does not
  // touch. It is there, because this one is launched when all blocks of that one have passed
  // their own wait for whatever came before.
  const int ctx = checked_ctx(a, b, false);
  const bool output = blockIdx.x == gridDim.x - 1;
  const long long first = (long long)blockIdx.x * kStretch;
  const int count = output || first >= ctx ? 0 : (int)min((long long)kStretch, ctx - first);
  const int weighed = a.weighed_lens ? fetch(a.weighed_lens + b) : ctx - 1;
  int slot[kPerThread];   // of the weights' pool, in heads' rows of a page; negative: no such token, or no such page
  float old[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int t = (int)first + i * kMergeThreads + tid;
    slot[i] = i * kMergeThreads + tid < count ? fetch(a.table + (size_t)b * a.max_blocks + t / ATTN_PAGE) : -1;
    if (slot[i] >= a.num_pages) slot[i] = -1;  // recorded where its keys were read
  }
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int t = (int)first + i * kMergeThreads + tid;
    if (slot[i] >= 0) slot[i] = (slot[i] * kHKV + head) * ATTN_PAGE + t % ATTN_PAGE;  // 2^27 at most
    old[i] = slot[i] >= 0 && a.decay != 0.f && t < weighed ? a.decay * fetch(a.weights + slot[i]) : 0.f;
  }
  follow();
  if (!output && count == 0) return;
  const float* const part = a.parts + ((size_t)b * kHKV + head) * a.splits * kPartFloats;
  if (!output && tid == 0) {
    const uint32_t bytes = (count + ATTN_PAGE - 1) / ATTN_PAGE * ATTN_PAGE * (uint32_t)sizeof(float4);  // scores of whole pages are there
    mbar_arrive_expect_tx(&full, bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(scores)),
                 "l"(a.scores + ((size_t)b * kHKV + head) * a.stride + first), "r"(bytes), "r"(smem_u32(&full))
                 : "memory");
  }
  // Warp h: head h, a lane two segments (at most 64 of them).
  float m[2] = {kUnseen, kUnseen}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < a.splits) {
      m[i] = fetch(part + (size_t)(lane + 32 * i) * kPartFloats + kGroup * kD + h);
      sum[i] = fetch(part + (size_t)(lane + 32 * i) * kPartFloats + kGroup * kD + kGroup + h);
    }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const unsigned gone = __ballot_sync(kFull, sum[i] == kFailed);
    if (tid == 0) lost[i] = gone;  // all heads of a segment alike
    if (sum[i] == kFailed) m[i] = kUnseen, sum[i] = 0.f;
  }
  float top = fmaxf(m[0], m[1]);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
  const float f0 = ex2(m[0] - top), f1 = ex2(m[1] - top);
  float total = fmaf(f0, sum[0], f1 * sum[1]);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) total += __shfl_xor_sync(kFull, total, off);
  const float inv = total == 0.f ? 0.f : 1.f / total;
  if (lane == 0) heads.top[h] = top, heads.inv[h] = inv;
  __syncthreads();
  const unsigned long long gone = (unsigned long long)lost[1] << 32 | lost[0];
  if (output) {  // two dims of head h a lane
    float2 y = make_float2(0.f, 0.f);
    for (int s = 0; s < a.splits; s += 8) {
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (s + i < a.splits) v[i] = fetch(reinterpret_cast<const float2*>(part + (size_t)(s + i) * kPartFloats + h * kD + 2 * lane));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = __shfl_sync(kFull, s < 32 ? f0 : f1, (s + i) & 31);
        if (s + i >= a.splits || (gone >> (s + i) & 1)) continue;
        y.x = fmaf(f, v[i].x, y.x);
        y.y = fmaf(f, v[i].y, y.y);
      }
    }
    *reinterpret_cast<float2*>(a.out + ((size_t)b * kHQ + head * kGroup + h) * kD + 2 * lane) = make_float2(y.x * inv, y.y * inv);
    return;
  }
  if (__syncthreads_or(!mbar_wait(&full, 0, a.timeout_ns))) {  // nothing was copied: the weights stay
    if (tid == 0) record_error(a.err, kDevErrTimeout);
    return;
  }
  const int per = ((ctx + ATTN_PAGE - 1) / ATTN_PAGE + a.splits - 1) / a.splits * ATTN_PAGE;
  const Heads all = heads;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    if (slot[i] >= 0 && !(gone && gone >> (((int)first + i * kMergeThreads + tid) / per) & 1))
      a.weights[slot[i]] = old[i] + given(scores[i * kMergeThreads + tid], all);
}

struct Device {
  bool ready = false;
  int sms = 0;
  int clusters[kMaxCluster + 1] = {};  // of each size, that the device holds at once on either page type
};
// A call's kernel, the shared memory that it takes, scores apart, and its threads.
struct Choice {
  void (*kernel)(CUtensorMap, CUtensorMap, DecodeWeighArgs);
  size_t smem;
  int threads;
};
template <bool kF32, bool kCluster>
Choice choice() {
  using L = Pages<kF32, kCluster>;
  return {decode_weigh_kernel<kF32, kCluster>, L::kSmemAlloc, L::kThreads};
}
Choice choice(bool f32, bool cluster) {
  return f32 ? cluster ? choice<true, true>() : choice<true, false>() : cluster ? choice<false, true>() : choice<false, false>();
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
    for (int i = 0; i < 4; ++i) {
      const bool cluster = i & 1;
      const Choice x = choice(i >> 1, cluster);
      ok = ok && cudaFuncSetAttribute(x.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)(x.smem + (cluster ? kMaxKept * sizeof(float4) : 0))) == cudaSuccess;
    }
    if (!ok) {
      (void)cudaGetLastError();
      return ATTN_ECUDA;
    }
    for (int size = 1; size <= kMaxCluster; ++size) {
      d.clusters[size] = 1 << 30;
      for (int f32 = 0; f32 < 2; ++f32) {
        const Choice x = choice(f32, true);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size, kHKV);
        cfg.blockDim = dim3(x.threads);
        cfg.dynamicSmemBytes = x.smem + kMaxKept * sizeof(float4);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = size;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, x.kernel, &cfg) != cudaSuccess) {
          (void)cudaGetLastError();
          n = 0;
        }
        if (n < d.clusters[size]) d.clusters[size] = n;
      }
    }
    d.ready = true;
  }
  *out = &d;
  return ATTN_OK;
}

long long score_stride(int max_context) { return ((long long)max_context + ATTN_PAGE - 1) / ATTN_PAGE * ATTN_PAGE; }

// How a call is cut: as clusters where the device holds them all at once and a
// segment's scores fit, of as many segments as that allows (one sequence of 1000 tokens 6.0
// us, through memory 8.0); else through memory. (More rounds of clusters were slower: they hold
// their places until the last of them ends. 16 sequences of 16384 tokens on bf16 pages 132 us,
// 110 through memory; 48 of 1 to 4096 on fp32 pages 91 and 85. Of three blocks and more the last few
// that the device is said to hold wait as well: 12 sequences of 4000 in 96 clusters of three, of
// 97, 32 us, in clusters of two 24; 7 in 56 of five, of 58, 21.5, of four 15.7.) There, segments as decode has
// them, two blocks an SM and several rounds, but for
//   one or two sequences: a block an SM, since all begin and end together and a second one only adds
//     its own start (131071 tokens, bf16 pages: 52 us in 19 segments, 55 in 38; 30000: 16.6 and 18.7)
//   more than 1536 tokens: two segments at least, since a block that has a sequence alone adds its
//     weights at the end by itself (32 sequences of 8192, bf16 pages: 101 us, 112 in one segment;
//     64 of up to 2000, fp32: 59 and 69; 64 of 1000, bf16: 34 and 30)
struct Plan {
  bool cluster;
  int splits, kept;  // kept: tokens of a segment at most (cluster)
};
Plan plan(int B, int max_context, const Device& d) {
  const long long pages = score_stride(max_context) / ATTN_PAGE;
  for (int s = kMaxCluster; s >= 1; --s) {
    const long long per = (pages + s - 1) / s;
    if (per * ATTN_PAGE > kMaxKept) break;
    if (B * kHKV > (s > 2 ? d.clusters[s] * 19 / 20 : d.clusters[s]) || (s > 1 && per < 4)) continue;  // four pages at least
    return Plan{true, s, (int)per * ATTN_PAGE};
  }
  const int each = d.sms / (B * kHKV);
  if (each >= 9) return Plan{false, each < kMaxSplits ? each : kMaxSplits, 0};  // 19584 tokens and more
  int len = 0;
  const int splits = decode_splits(B, max_context, 0, 2 * d.sms, &len);
  return Plan{false, splits == 1 && max_context > 1536 ? 2 : splits, 0};
}

}  // namespace

int decode_weigh_workspace_bytes(int B, int max_context, size_t* bytes) {
  Device* d = nullptr;
  const int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const Plan p = plan(B, max_context, *d);
  *bytes = p.cluster ? 0
                     : (size_t)B * kHKV * ((size_t)score_stride(max_context) * sizeof(float4) +
                                                   (p.splits > 1 ? p.splits * kPartFloats * sizeof(float) : 0));
  return ATTN_OK;
}

int launch_decode_weigh(const DecodeWeighCall& c, unsigned* err, cudaStream_t stream) {
  Device* d = nullptr;
  int rc = device(&d);
  if (rc != ATTN_OK) return rc;
  const bool bf16 = c.type == ATTN_BF16;
  alignas(64) CUtensorMap mk, mv;
  const long long rows = (long long)c.num_pages * ATTN_PAGE;
  if ((rc = encode_rows_map(c.k_pages, bf16, rows, ATTN_PAGE, CU_TENSOR_MAP_SWIZZLE_128B, &mk)) != ATTN_OK ||
      (rc = encode_rows_map(c.v_pages, bf16, rows, ATTN_PAGE, CU_TENSOR_MAP_SWIZZLE_128B, &mv)) != ATTN_OK)
    return rc;
  const Plan p = plan(c.B, c.max_context, *d);
  DecodeWeighArgs a{};
  a.q = c.q;
  a.weights = c.weights;
  a.table = c.table;
  a.ctx_lens = c.ctx_lens;
  a.weighed_lens = c.weighed_lens;
  a.out = c.out;
  a.B = c.B;
  a.max_blocks = c.max_blocks;
  a.num_pages = c.num_pages;
  a.max_context = c.max_context;
  a.splits = p.splits;
  a.stride = score_stride(c.max_context);
  if (!p.cluster) {
    a.scores = static_cast<float4*>(c.workspace);
    a.parts = reinterpret_cast<float*>(a.scores + (size_t)c.B * kHKV * a.stride);
  }
  a.decay = c.decay;
  a.err = err;
  a.withheld = c.withheld;
  a.timeout_ns = c.withheld ? kFaultNs : kTimeoutNs;
  const Choice k = choice(!bf16, p.cluster);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.splits, kHKV, c.B);
  cfg.blockDim = dim3(k.threads);
  cfg.dynamicSmemBytes = k.smem + p.kept * sizeof(float4);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 2 : 1;
  if (launched(cudaLaunchKernelEx(&cfg, k.kernel, mk, mv, a)) != cudaSuccess) return ATTN_ELAUNCH;
  if (!p.cluster && a.splits > 1) {
    const unsigned stretches = (c.max_context + kStretch - 1) / kStretch;
    if (launch_following(decode_weigh_merge_kernel, dim3(stretches + 1, kHKV, c.B), dim3(kMergeThreads), stream, a) != cudaSuccess)
      return ATTN_ELAUNCH;
  }
  return ATTN_OK;
}

}  // namespace attn
