// rows.cu -- what happens to a row's query, key and value heads between the
// projections and the attention kernels: the per-head RMS norm, the position
// rotation, the store into a contiguous or a paged cache, and the moves that
// keep an accepted path of drafted rows.
//
// Norm and rotation of one head x [64] with weight w, at a row with angles
// t_0 .. t_31 (cos and sin from the caller's table):
//   y[d] = x[d] w[d] / sqrt(sum_e x[e]^2 / 64 + eps)
//   (y[a], y[b]) -> (y[a] cos t_i - y[b] sin t_i, y[b] cos t_i + y[a] sin t_i)
// with (a, b) = (i, i + 32) (halves) or (2 i, 2 i + 1) (neighbours). All of it
// in fp32, rounded once when the destination is bf16.
//
// A row is 48 heads at most (32 query, 8 key, 8 value). A warp owns 8 heads of
// one row: 16 lanes hold a head, four consecutive dims each, so a head's loads
// and stores are 16 bytes a lane (8 from or to bf16), the sum of squares is
// four shuffles, a halves pair sits eight lanes away and a neighbours pair in
// the lane itself. The cos and sin of a row are read once per warp. Nothing is
// staged in shared memory: every byte is used once, so the bound is memory, and
// for a few rows the launch and a chain of dependent loads (the row's sequence, its
// context, its page or angles). Measured in graphs, inputs in HBM: 8192 fp32 rows
// appended with their queries 31.6 us, normed and rotated alone 26.5; 2048 bf16 rows
// 7.8 and 7.0; 16 rows 2.2 and 2.1, of which 1.4 are a launch. The 8192 rows read 101
// MB and write 101, of which half is still in the 129 MB L2 when the kernel ends: DRAM
// moves 152 MB, 4.8 TB/s, 60% of its peak, with 63% of the warps' places filled.
#include <cstdint>
#include <cuda_bf16.h>

#include "common.cuh"

namespace attn {
namespace {

// 12 blocks of 4 warps an SM (40 registers a thread, at which the paged forms store 32
// bytes to local memory and load 16, 8 and 4 with bf16 rows): a chunk's rows wait for the
// lookups of where they go, so as many warps as fit wait at once, with bf16 heads
// held as loaded until then, and each lookup starts as soon as it can. (2048 bf16 rows
// appended with their queries: 7.8 us; 8.9 with a context, a page, a position and its
// angles each after the other; 10.5 with 44 registers and heads widened as they land.)
constexpr int kRowWarps = 4, kRowBlocks = 12;
constexpr int kHeadsPerWarp = 8;
constexpr int kQChunks = kHQ / kHeadsPerWarp;  // 4 warps for a row's queries, one for its keys, one for its values
constexpr unsigned kFull = 0xffffffffu;

template <bool kBf16>
struct Elem {
  using type = float;
};
template <>
struct Elem<true> {
  using type = __nv_bfloat16;
};

// Four consecutive values, and what they are in fp32. Plain loads: a call may run
// in place.
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ uint2 load4(const __nv_bfloat16* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ float4 widen(float4 v) { return v; }
__device__ __forceinline__ float4 widen(uint2 u) {
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  // one rounding to nearest even, the cache's precision
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const unsigned*>(&a), *reinterpret_cast<const unsigned*>(&b));
}

struct Angles {
  float4 c, s;  // this lane's cosines and sines (neighbours: .x and .y only)
};

__device__ __forceinline__ float4 norm_rotate(float4 x, const float4& w, bool normed, const Angles& a, bool rotated,
                                              int pairing, float eps) {
  if (normed) {
    float ss = fmaf(x.x, x.x, fmaf(x.y, x.y, fmaf(x.z, x.z, x.w * x.w)));
#pragma unroll
    for (int off = 8; off >= 1; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
    const float r = rsqrtf(fmaf(ss, 1.f / kD, eps));
    x = make_float4(x.x * r * w.x, x.y * r * w.y, x.z * r * w.z, x.w * r * w.w);
  }
  if (!rotated) return x;
  if (pairing == ATTN_ROPE_PAIRS)
    return make_float4(x.x * a.c.x - x.y * a.s.x, fmaf(x.y, a.c.x, x.x * a.s.x), x.z * a.c.y - x.w * a.s.y,
                       fmaf(x.w, a.c.y, x.z * a.s.y));
  float4 o;  // the other half of the pair
  o.x = __shfl_xor_sync(kFull, x.x, 8);
  o.y = __shfl_xor_sync(kFull, x.y, 8);
  o.z = __shfl_xor_sync(kFull, x.z, 8);
  o.w = __shfl_xor_sync(kFull, x.w, 8);
  // a.s carries the sign: -sin in the first half, +sin in the second
  return make_float4(fmaf(o.x, a.s.x, x.x * a.c.x), fmaf(o.y, a.s.y, x.y * a.c.y), fmaf(o.z, a.s.z, x.z * a.c.z),
                     fmaf(o.w, a.s.w, x.w * a.c.w));
}

// The sequence whose rows hold row n: the last b with row_start[b] <= n, found
// by the warp 32 entries at a time (two rounds up to 1024 sequences, where a
// binary search would wait for ten loads one after another). B when the row
// lies behind the last sequence, -1 when before the first.
__device__ __forceinline__ int find_sequence(const int* row_start, int B, int n, int lane, int* first) {
  int lo = 0, hi = B + 1;  // entries lo .. hi - 1 are left; entry lo <= n once a round has passed
  int base = 0;
  while (true) {
    const int step = (hi - lo + 31) / 32;
    const long long at = (long long)lo + (long long)lane * step;
    const int v = at < hi ? fetch(row_start + at) : 0x7fffffff;
    const unsigned le = __ballot_sync(kFull, at < hi && v <= n);
    if (le == 0) return -1;
    const int last = 31 - __clz(le);
    base = __shfl_sync(kFull, v, last);
    lo += last * step;
    if (step == 1) break;
    hi = min(lo + step, hi);
  }
  *first = base;
  return lo;
}

struct RowArgs {
  const void *q, *k, *v;  // [N] rows of 32, 8 and 8 heads; q and v may be absent
  long long q_stride, k_stride, v_stride;  // elements between rows
  const float *q_weight, *k_weight;        // [64] each, or nullptr: not normed
  float eps;
  const float* cos_sin;  // [num_positions][64], or nullptr: not rotated
  const int* positions;  // [N], or nullptr: consecutive after the sequence's context
  int num_positions, pairing;
  // Several positions a row: axis x of row n at positions[x * pos_stride + n], and two
  // bits of axis_of for each frequency. grouped: a lane's frequencies share an axis.
  long long pos_stride;
  unsigned long long axis_of;
  int num_axes;
  bool grouped;
  float* q_out;          // [N][32][64]
  void *k_out, *v_out;   // contiguous: k_out [N][8][64]; paged: the page pools
  const int *table, *ctx_lens, *row_start;  // paged
  int B, N, max_blocks, num_pages;
  int q_chunks, chunks;  // warps per row: for the queries, and in all
  unsigned* err;
};

// This lane's cosines and sines where each frequency goes by one of several positions:
// lane x holds the row's position on axis x, checked by axis_position(). Where a lane's
// frequencies (four of a halves pairing, two of a neighbours one) share an axis they come
// as one vector each; otherwise one by one, from table rows that L1 holds (2048 rows of
// bf16 into a paged cache, with queries: 7.98 us grouped, 8.20 one by one).
__device__ __forceinline__ Angles axis_angles(const RowArgs& a, int position, int sub) {
  const bool pairs = a.pairing == ATTN_ROPE_PAIRS;
  const int f0 = pairs ? 2 * sub : (4 * sub) & 31;
  float c[4] = {}, s[4] = {};
  if (a.grouped) {
    const int p = __shfl_sync(kFull, position, (int)(a.axis_of >> (2 * f0)) & 3);
    const float* row = a.cos_sin + (size_t)p * kD + f0;
    if (pairs) {
      const float2 x = fetch(reinterpret_cast<const float2*>(row)), y = fetch(reinterpret_cast<const float2*>(row + kD / 2));
      c[0] = x.x, c[1] = x.y, s[0] = y.x, s[1] = y.y;
    } else {
      const float4 x = fetch(reinterpret_cast<const float4*>(row)), y = fetch(reinterpret_cast<const float4*>(row + kD / 2));
      c[0] = x.x, c[1] = x.y, c[2] = x.z, c[3] = x.w, s[0] = y.x, s[1] = y.y, s[2] = y.z, s[3] = y.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int f = pairs ? f0 + (j & 1) : f0 + j;
      const int p = __shfl_sync(kFull, position, (int)(a.axis_of >> (2 * f)) & 3);
      if (j < 2 || !pairs) {
        const float* row = a.cos_sin + (size_t)p * kD + f;
        c[j] = fetch(row), s[j] = fetch(row + kD / 2);
      }
    }
  }
  const float sign = !pairs && sub < 8 ? -1.f : 1.f;
  return Angles{make_float4(c[0], c[1], c[2], c[3]), make_float4(sign * s[0], sign * s[1], sign * s[2], sign * s[3])};
}

template <bool kInBf16, bool kOutBf16, bool kPaged, bool kAxes>
__global__ void __launch_bounds__(32 * kRowWarps, kRowBlocks)
rows_kernel(const RowArgs a) {
  follow();
  using In = typename Elem<kInBf16>::type;
  using Out = typename Elem<kOutBf16>::type;
  const unsigned item = blockIdx.x * kRowWarps + (threadIdx.x >> 5);  // 6 x ATTN_MAX_TOKENS at most
  const int lane = threadIdx.x & 31, sub = lane & 15, d = 4 * sub;
  const int n = (int)(item / (unsigned)a.chunks), chunk = (int)(item % (unsigned)a.chunks);
  if (n >= a.N) return;

  const bool is_q = chunk < a.q_chunks, is_k = chunk == a.q_chunks;
  // The eight heads' loads do not depend on where they go: issue them first.
  const In* src = is_q ? static_cast<const In*>(a.q) + (size_t)n * a.q_stride + chunk * kHeadsPerWarp * kD
                  : is_k ? static_cast<const In*>(a.k) + (size_t)n * a.k_stride
                         : static_cast<const In*>(a.v) + (size_t)n * a.v_stride;
  src += (lane >> 4) * kD + d;
  decltype(load4(src)) raw[kHeadsPerWarp / 2];
#pragma unroll
  for (int i = 0; i < kHeadsPerWarp / 2; ++i) raw[i] = load4(src + 2 * i * kD);

  // Then what the lookups need, as much of it at once as there is.
  int position = 0;
  if constexpr (kAxes) {
    if (lane < a.num_axes) position = fetch(a.positions + lane * a.pos_stride + n);
  } else {
    position = a.positions ? fetch(a.positions + n) : 0;
  }
  int slot = n;  // row of the destination
  int page = 0;
  if (kPaged) {
    int ctx = lane < a.B ? fetch(a.ctx_lens + lane) : 0;  // of the first 32 sequences
    int first = 0;
    const int b = find_sequence(a.row_start, a.B, n, lane, &first);
    if (b < 0 || b >= a.B) return;  // a row of no sequence: left as it is
    ctx = b < 32 ? __shfl_sync(kFull, ctx, b) : fetch(a.ctx_lens + b);
    const long long row = (long long)n - first, token = ctx + row;
    page = -1;
    if (!is_q && token >= row && token < (long long)a.max_blocks * ATTN_PAGE) {
      page = fetch(a.table + (size_t)b * a.max_blocks + token / ATTN_PAGE);
      slot = (int)token % ATTN_PAGE;
    }
    if (!kAxes && !a.positions) position = (int)min(max(token, -1ll), (long long)ATTN_MAX_TOKENS);
  }

  float4 x[kHeadsPerWarp / 2];
  if (is_q || is_k) {
    const float* weight = is_q ? a.q_weight : a.k_weight;
    const float4 w = weight ? fetch(reinterpret_cast<const float4*>(weight + d)) : make_float4(1.f, 1.f, 1.f, 1.f);
    Angles t{};
    if constexpr (kAxes) {
      if (position < 0 || position >= a.num_positions) {  // lanes without an axis hold 0
        record_error(a.err, kDevErrBounds);
        position = position < 0 ? 0 : a.num_positions - 1;
      }
      t = axis_angles(a, position, sub);
    } else if (a.cos_sin) {
      if (position < 0 || position >= a.num_positions) {
        if (lane == 0) record_error(a.err, kDevErrBounds);
        position = position < 0 ? 0 : a.num_positions - 1;
      }
      const float* row = a.cos_sin + (size_t)position * kD;
      if (a.pairing == ATTN_ROPE_PAIRS) {
        const float2 c = fetch(reinterpret_cast<const float2*>(row + 2 * sub));
        const float2 s = fetch(reinterpret_cast<const float2*>(row + kD / 2 + 2 * sub));
        t.c = make_float4(c.x, c.y, 0.f, 0.f);
        t.s = make_float4(s.x, s.y, 0.f, 0.f);
      } else {
        t.c = fetch(reinterpret_cast<const float4*>(row + (d & 31)));
        t.s = fetch(reinterpret_cast<const float4*>(row + kD / 2 + (d & 31)));
        if (sub < 8) t.s = make_float4(-t.s.x, -t.s.y, -t.s.z, -t.s.w);
      }
    }
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp / 2; ++i)
      x[i] = norm_rotate(widen(raw[i]), w, weight != nullptr, t, kAxes || a.cos_sin != nullptr, a.pairing, a.eps);
  } else {
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp / 2; ++i) x[i] = widen(raw[i]);
  }

  if (is_q) {
    float* dst = a.q_out + ((size_t)n * kHQ + chunk * kHeadsPerWarp + (lane >> 4)) * kD + d;
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp / 2; ++i) store4(dst + 2 * i * kD, x[i]);
  } else {
    if (kPaged) {
      if (page < 0 || page >= a.num_pages) {
        if (lane == 0) record_error(a.err, kDevErrBounds);
        return;
      }
      slot += page * ATTN_PAGE;
    }
    Out* dst = static_cast<Out*>(is_k ? a.k_out : a.v_out) + ((size_t)slot * kHKV + (lane >> 4)) * kD + d;
#pragma unroll
    for (int i = 0; i < kHeadsPerWarp / 2; ++i) store4(dst + 2 * i * kD, x[i]);
  }
}

template <bool kPaged, bool kAxes>
cudaError_t launch_rows_as(const RowArgs& a, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  const unsigned blocks = (unsigned)(((long long)a.N * a.chunks + kRowWarps - 1) / kRowWarps);
  return launch_following(
      in_bf16 ? (out_bf16 ? rows_kernel<true, true, kPaged, kAxes> : rows_kernel<true, false, kPaged, kAxes>)
              : (out_bf16 ? rows_kernel<false, true, kPaged, kAxes> : rows_kernel<false, false, kPaged, kAxes>),
      dim3(blocks), dim3(32 * kRowWarps), stream, a);
}

// ---------------------------------------------------------------------------
// The angle table: cos and sin of position x frequency, in double (at position
// 2^24 the fp32 product would be off by a radian), rounded once to fp32.
struct Frequencies {
  double f[kD / 2];
};
__global__ void rope_table_kernel(const __grid_constant__ Frequencies inv, float* table, long long n) {
  const long long at = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (at >= n) return;
  const long long pos = at / (kD / 2);
  const int i = (int)(at % (kD / 2));
  double s, c;
  sincos((double)pos * inv.f[i], &s, &c);
  table[pos * kD + i] = (float)c;
  table[pos * kD + kD / 2 + i] = (float)s;
}

// ---------------------------------------------------------------------------
// Keeping an accepted path. Block (b, pool): row keep[b][i] of the drafted rows
// moves to row i, for K (pool 0) or V (pool 1). A thread owns 16 bytes of up to 16
// rows (of one to four groups of threads, by maxKeep), and all rows are in registers
// before any is stored, so the moves run in place whatever overlaps. At most 64 rows
// of 2 or 4 KB a sequence: the launch and three dependent loads (list, table, rows)
// are nearly all of it. 64 rows of 64 sequences 2.8 us in a graph; with one group,
// eight rows at a time, and the list read after its length 6.2.
constexpr int kKeepRows = 16, kKeepGroups = ATTN_TREE_ROWS / kKeepRows;

__global__ void __launch_bounds__(128 * kKeepGroups)
compact_kernel(uint4* k_pages, uint4* v_pages, int row_vecs, const int* table, const int* ctx_lens,
               const int* keep, const int* counts, int max_keep, int max_rows, int max_blocks, int num_pages,
               unsigned* err) {
  __shared__ int from[ATTN_TREE_ROWS], to[ATTN_TREE_ROWS];  // rows of the pool
  follow();
  const int b = blockIdx.x, tid = threadIdx.x;
  const int count = fetch(counts + b);
  const int ctx = fetch(ctx_lens + b);
  const int r = tid < max_keep ? fetch(keep + (size_t)b * max_keep + tid) : 0;
  const int before = tid > 0 && tid < max_keep ? fetch(keep + (size_t)b * max_keep + tid - 1) : -1;
  bool bad = count < 0 || count > max_keep || count > max_rows || ctx < 0;
  if (!bad && tid < count) {
    const long long src = (long long)ctx + r, dst = (long long)ctx + tid;
    if (r <= before || r >= max_rows || src >= (long long)max_blocks * ATTN_PAGE) {
      bad = true;
    } else {
      const int ps = fetch(table + (size_t)b * max_blocks + src / ATTN_PAGE);
      const int pd = fetch(table + (size_t)b * max_blocks + dst / ATTN_PAGE);
      bad = ps < 0 || ps >= num_pages || pd < 0 || pd >= num_pages;
      from[tid] = ps * ATTN_PAGE + (int)src % ATTN_PAGE;
      to[tid] = pd * ATTN_PAGE + (int)dst % ATTN_PAGE;
    }
  }
  if (__syncthreads_or(bad)) {  // nothing of this sequence is moved
    if (tid == 0) record_error(err, kDevErrBounds);
    return;
  }
  const int group = tid / row_vecs, groups = blockDim.x / row_vecs;
  uint4* pool = (blockIdx.y ? v_pages : k_pages) + tid % row_vecs;
  uint4 x[kKeepRows];
#pragma unroll
  for (int k = 0; k < kKeepRows; ++k) {
    const int i = k * groups + group;
    if (i < count && from[i] != to[i]) x[k] = pool[(size_t)from[i] * row_vecs];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kKeepRows; ++k) {
    const int i = k * groups + group;
    if (i < count && from[i] != to[i]) pool[(size_t)to[i] * row_vecs] = x[k];
  }
}

}  // namespace

cudaError_t launch_rows(const RowCall& c, unsigned* err, cudaStream_t stream) {
  RowArgs a{};
  a.q = c.q;
  a.k = c.k;
  a.v = c.v;
  a.q_stride = c.q_stride;
  a.k_stride = c.k_stride;
  a.v_stride = c.v_stride;
  a.q_weight = c.q_weight;
  a.k_weight = c.k_weight;
  a.eps = c.eps;
  a.cos_sin = c.cos_sin;
  a.positions = c.positions;
  a.num_positions = c.num_positions;
  a.pairing = c.pairing;
  a.q_out = c.q_out;
  a.k_out = c.k_out;
  a.v_out = c.v_out;
  a.table = c.table;
  a.ctx_lens = c.ctx_lens;
  a.row_start = c.row_start;
  a.B = c.B;
  a.N = c.N;
  a.max_blocks = c.max_blocks;
  a.num_pages = c.num_pages;
  a.q_chunks = c.q ? kQChunks : 0;
  a.chunks = a.q_chunks + (c.k ? 1 : 0) + (c.v ? 1 : 0);
  a.err = err;
  const bool in = c.in_type == ATTN_BF16, out = c.out_type == ATTN_BF16;
  if (c.num_axes == 0) return c.table ? launch_rows_as<true, false>(a, in, out, stream) : launch_rows_as<false, false>(a, in, out, stream);
  a.num_axes = c.num_axes;
  a.pos_stride = c.pos_stride;
  a.axis_of = c.axis_of;
  const int per_lane = c.pairing == ATTN_ROPE_PAIRS ? 2 : 4;
  a.grouped = true;
  for (int f = 1; f < kD / 2; ++f)
    if (f % per_lane && ((c.axis_of >> (2 * f)) & 3) != ((c.axis_of >> (2 * f - 2)) & 3)) a.grouped = false;
  return c.table ? launch_rows_as<true, true>(a, in, out, stream) : launch_rows_as<false, true>(a, in, out, stream);
}

cudaError_t launch_rope_table(const double* inv_freq, float* table, int num_positions, cudaStream_t stream) {
  Frequencies f;
  for (int i = 0; i < kD / 2; ++i) f.f[i] = inv_freq[i];
  const long long n = (long long)num_positions * (kD / 2);
  rope_table_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(f, table, n);
  return cudaGetLastError();
}

cudaError_t launch_compact(void* k_pages, void* v_pages, int type, const int* table, const int* ctx_lens,
                           const int* keep, const int* counts, int B, int max_keep, int max_rows, int max_blocks,
                           int num_pages, unsigned* err, cudaStream_t stream) {
  const int vecs = kHKV * kD * (type == ATTN_BF16 ? 2 : 4) / 16;  // 16-byte words of a token's row: 64 or 128
  const int groups = (max_keep + kKeepRows - 1) / kKeepRows;
  return launch_following(compact_kernel, dim3(B, 2), dim3(vecs * groups), stream, static_cast<uint4*>(k_pages),
                          static_cast<uint4*>(v_pages), vecs, table, ctx_lens, keep, counts, max_keep, max_rows,
                          max_blocks, num_pages, err);
}

}  // namespace attn
