// Linear attention with a decay L = exp(log_decay[h]) per head, CUDA-core kernels: fp32 prompts and
// gradients (the bf16 ones are in decay_bf16.cuh), the scan that joins segments, the single-token
// step, and the sum over query heads that share a key/value head.
//
// One form serves the prompt and its gradients.  A pass reads rows a, b, c and writes
//     out_i = sp * sum_{j in past(i)} L^|i-j| (a_i . b_j) c_j  +  si * L^(t_i + e) a_i^T S ,
//     S    <- L^n S + sd * sum_j L^(n - t_j - e) b_j c_j^T              (over the n rows of a range)
// where past(i) is j <= i and t_i = i - (first row of the range) forward in time, j >= i and
// t_i = (last row) - i backward.  With the rows q, k, v, dO and the state S:
//     prompt  out: a = q,  b = k,  c = v   forward,  e = 1, S from S_0
//     dQ         : a = dO, b = v,  c = k   forward,  e = 1, S^T
//     dK         : a = v,  b = dO, c = q   backward, e = 0, dS^T   (from the final state's gradient)
//     dV         : a = k,  b = q,  c = dO  backward, e = 0, dS
// e says on which side of a range's border the state stands: S_0 has decayed once when row 0 reads
// it, the gradient of the last state reaches the last row undecayed.
//
// States in the workspace are stored by column quads: elements (r, 4c .. 4c+3) at float4 c * D + r,
// so that the kernels' threads, one row each, read and write neighbouring float4s (by rows, a state
// took a row-pass CTA 3.8 us to read and a states CTA 2.9 us to write).
//
// Sequences are cut into segments of whole chunks (Cut).  Three launches: the sum of every segment's
// own rows (decay_states), its exclusive prefix in time order (decay_scan), and the rows of every
// segment, chunk after chunk with the state carried along (decay_rows).  Every exponent above is
// >= 0, so no power grows for L <= 1 and none is divided by; L = 0 (log_decay = -inf) leaves each
// row its own term.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sm100.cuh"

namespace rehyat {
namespace decay {

constexpr int kMaxD = 128;
constexpr int kC = 64;           // rows of one chunk of the CUDA-core kernels
constexpr int kThreads = 256;

// Rows of a [B, heads, N, D] tensor with strides in elements; head h of the pass reads head
// h / group (query heads that share a key/value head).
struct Rows {
  const void* p;
  long long sb, sh, sn;
  int group;
};

// How sequences are cut: into segments of `chunks` chunks of `chunk` rows, segment s of sequence b in
// slot b * per_seq + s.  With `search` (ragged batches) the segments are instead the shortest that
// fit all sequences' valid rows into the slots, one sequence's behind the other's.  One CTA for each
// slot and head.
struct Cut {
  int chunk, chunks, per_seq, slots, search;
};

struct Pass {
  Rows a, b, c;
  void* out;                 // row type, or fp32 where the group sum follows
  long long ob, oh, on;      // its strides
  const float* log_decay;    // [H]
  const int* lengths;        // [B] or null: rows at and past a sequence's length are padding
  float* states;             // [slots][H] each segment's own sum, then the state before it
  int B, H, N, D;
  Cut cut;
  int reverse, e;
  int carried;               // rows: segments have a state before them (else zero)
  int transposed;            // rows: the pass's state is the transpose of `states`
  int exact;                 // states: the last state is given out (bf16: two-part products)
  int out_f32;               // rows: fp32 output for the group sum
  float sp, si, sd;
};
struct Passes {  // of one launch: blockIdx.z
  Pass p[3];
};

// log2 of the decay, bounded below so that 0 * log2(0) stays 0 (2^-1000 is 0 in fp32); NaN stays.
__device__ __forceinline__ float log2_decay(const float* g, int h) {
  const float x = g[h] * 1.4426950408889634f;
  return x < -1000.f ? -1000.f : x;
}
__device__ __forceinline__ int length_of(const int* lengths, int b, int N) {
  return lengths ? min(max(lengths[b], 0), N) : N;
}

__device__ __forceinline__ int chunks_of(const int* lengths, int b, int N, int chunk) {
  return (length_of(lengths, b, N) + chunk - 1) / chunk;
}
// A ragged batch's cut, by one warp (all lanes; at most kMaxSearch sequences): the fewest chunks a
// segment with which the sequences' segments fit into the slots, by bisection between the mean and
// the longest.  A lane holds every 32nd sequence.  (By the whole block, with a barrier for each sum,
// it took 5 us of every launch.)
constexpr int kMaxSearch = 256;
struct Search {
  int n[kMaxSearch / 32];  // chunks of sequences lane, lane + 32, ...
  int per;

  __device__ __forceinline__ Search(const Cut& cut, const int* lengths, int B, int N) {
    const int lane = threadIdx.x & 31;
    unsigned total = 0;
#pragma unroll
    for (int k = 0; k < kMaxSearch / 32; ++k) {
      const int b = lane + 32 * k;
      n[k] = b < B ? chunks_of(lengths, b, N, cut.chunk) : 0;
      total += n[k];
    }
    total = __reduce_add_sync(0xffffffffu, total);
    int lo = max((int)((total + cut.slots - 1) / cut.slots), 1);
    int hi = max(cut.chunks * cut.per_seq, lo);
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      unsigned used = 0;
#pragma unroll
      for (int k = 0; k < kMaxSearch / 32; ++k)
        if (32 * k < B) used += (unsigned)(n[k] + mid - 1) / (unsigned)mid;
      if ((int)__reduce_add_sync(0xffffffffu, used) <= cut.slots)
        hi = mid;
      else
        lo = mid + 1;
    }
    per = lo;
  }
  // Slots of the sequences before b, and in all (b >= the batch).
  __device__ __forceinline__ int slots_before(int b) const {
    unsigned used = 0;
#pragma unroll
    for (int k = 0; k < kMaxSearch / 32; ++k)
      if ((int)(threadIdx.x & 31) + 32 * k < b) used += (unsigned)(n[k] + per - 1) / (unsigned)per;
    return (int)__reduce_add_sync(0xffffffffu, used);
  }
};

// Segment of this CTA (head blockIdx.x, slot blockIdx.y): valid rows [begin, end) of sequence b; none
// if begin >= end.  All threads of the block call it.
struct Segment {
  int b, h, begin, end;
  bool last;  // in time
};
__device__ __forceinline__ Segment find_segment(const Pass& p) {
  __shared__ int found[3];
  const int slot = blockIdx.y;
  int b, s, per = p.cut.chunks;
  if (!p.cut.search) {
    b = slot / p.cut.per_seq;
    s = slot - b * p.cut.per_seq;
  } else {
    if (threadIdx.x < 32) {
      const Search f(p.cut, p.lengths, p.B, p.N);
      if (threadIdx.x == 0) found[0] = -1;
      __syncwarp();
      int base = 0;  // slots of the sequences before: 32 sequences a turn
#pragma unroll
      for (int k = 0; k < kMaxSearch / 32; ++k) {
        const int n = (f.n[k] + f.per - 1) / f.per;
        int end = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, end, m);
          if ((int)threadIdx.x >= m) end += y;
        }
        end += base;
        if (end - n <= slot && slot < end) {
          found[0] = threadIdx.x + 32 * k;
          found[1] = slot - (end - n);
        }
        base = __shfl_sync(0xffffffffu, end, 31);
        if (base > slot) break;
      }
      if (threadIdx.x == 0) found[2] = f.per;
    }
    __syncthreads();
    b = found[0];
    s = found[1];
    per = found[2];
    if (b < 0) return Segment{0, (int)blockIdx.x, 0, 0, false};
  }
  const int len = length_of(p.lengths, b, p.N), rows = per * p.cut.chunk;
  Segment g{b, (int)blockIdx.x, s * rows, 0, false};
  g.end = min(len, g.begin + rows);
  g.last = p.reverse ? s == 0 : g.end == len;
  return g;
}
// This CTA's state in the workspace.
__device__ __forceinline__ float* state_of(const Pass& p) {
  return p.states + ((size_t)blockIdx.y * p.H + blockIdx.x) * p.D * p.D;
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(sm100::pack_bf16x2(v.x, v.y), sm100::pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ float4 fma4(float s, float4 v, float4 acc) {
  return make_float4(fmaf(s, v.x, acc.x), fmaf(s, v.y, acc.y), fmaf(s, v.z, acc.z),
                     fmaf(s, v.w, acc.w));
}
__device__ __forceinline__ float4 mul4(float s, float4 v) {
  return make_float4(s * v.x, s * v.y, s * v.z, s * v.w);
}

// ---- fp32 rows on the CUDA cores ----
// kDp: D rounded up to 32, with n = kDp / 32.  256 threads form 16 x 16 groups; a thread's columns are
// the pairs 2 (tid % 16) + 32 u, u < n, so a half warp's eight-byte reads are one 128-byte row, and
// products are taken two columns at a time.  Tiles have rows of kDp + 4, so that threads on different
// rows reach different banks.
__host__ __device__ constexpr int padded(int D) { return (D + 31) / 32 * 32; }
__host__ __device__ constexpr int rows_smem_floats(int Dp) {
  return 3 * kC * (Dp + 4) + kC * (kC + 4) + Dp * (Dp + 4) + 2 * kC;
}
__host__ __device__ constexpr int states_smem_floats(int Dp) { return 2 * kC * (Dp + 4) + kC; }

__device__ __forceinline__ uint64_t pair_at(const float* p) {
  return *reinterpret_cast<const uint64_t*>(p);
}
__device__ __forceinline__ uint64_t twice(float x) { return sm100::f2_pack(x, x); }

// Rows [r0, r0 + kC) of one head into shared memory, columns [D, kDp) and rows at or past `end` as
// zeros whatever the tensor holds there.
template <int kDp, int kFrom = kThreads>
__device__ __forceinline__ void load_rows(float* dst, const Rows& t, int b, int h, int r0, int end,
                                          int D) {
  const float* src = static_cast<const float*>(t.p) + b * t.sb + (h / t.group) * t.sh;
  constexpr int v4 = kDp / 4;
#pragma unroll
  for (int i0 = 0; i0 < kC * v4; i0 += kFrom) {
    const int i = i0 + threadIdx.x, r = i / v4, c = (i % v4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < end && c < D) x = load4<float>(src + (long long)(r0 + r) * t.sn + c);
    *reinterpret_cast<float4*>(dst + r * (kDp + 4) + c) = x;
  }
}

// acc += sum over `rows` rows r of (w[r] x[r][i]) y[r][j] for the thread's 2n x 2n elements: rows
// i = 2 (tid / 16) + 32 u and the one after, columns likewise by tid % 16.
template <int kDp>
__device__ __forceinline__ void outer_add(uint64_t (&acc)[kDp / 16][kDp / 32], const float* x,
                                          const float* y, const float* w, int rows) {
  constexpr int n = kDp / 32, ld = kDp + 4;
  const int t = threadIdx.x % kThreads, i0 = (t / 16) * 2, j0 = (t % 16) * 2;
#pragma unroll 2
  for (int r = 0; r < rows; ++r) {
    const uint64_t wr = twice(w[r]);
    uint64_t yv[n];
#pragma unroll
    for (int u = 0; u < n; ++u) yv[u] = sm100::f2_mul(wr, pair_at(y + r * ld + j0 + 32 * u));
#pragma unroll
    for (int u = 0; u < n; ++u) {
      const float2 xv = *reinterpret_cast<const float2*>(x + r * ld + i0 + 32 * u);
#pragma unroll
      for (int v = 0; v < n; ++v) {
        acc[2 * u][v] = sm100::f2_fma(twice(xv.x), yv[v], acc[2 * u][v]);
        acc[2 * u + 1][v] = sm100::f2_fma(twice(xv.y), yv[v], acc[2 * u + 1][v]);
      }
    }
  }
}

// Each segment's own sum: sd * sum_j L^(n - t_j - e) b_j c_j^T over its n valid rows.
// grid (H, slots, passes), block 256.
template <int kDp>
__global__ void __launch_bounds__(kThreads, kDp <= 64 ? 2 : 1)
    decay_states_kernel(const __grid_constant__ Passes all) {
  extern __shared__ __align__(16) float smf[];
  sm100::grid_dep_signal();
  const Pass& p = all.p[blockIdx.z];
  const Segment seg = find_segment(p);
  const int b = seg.b, h = seg.h, r_begin = seg.begin, r_end = seg.end;
  if (r_begin >= r_end || (seg.last && !p.exact)) return;  // nothing reads its sum
  constexpr int n = kDp / 32, ld = kDp + 4;
  const int tid = threadIdx.x;
  float* sb = smf;
  float* sc = sb + kC * ld;
  float* sw = sc + kC * ld;
  const float g2 = log2_decay(p.log_decay, h);
  uint64_t acc[2 * n][n];
#pragma unroll
  for (int i = 0; i < 2 * n; ++i)
#pragma unroll
    for (int v = 0; v < n; ++v) acc[i][v] = 0ull;
  for (int r0 = r_begin; r0 < r_end; r0 += kC) {
    __syncthreads();
    load_rows<kDp>(sb, p.b, b, h, r0, r_end, p.D);
    load_rows<kDp>(sc, p.c, b, h, r0, r_end, p.D);
    if (tid < kC) {
      const int r = r0 + tid;
      sw[tid] = p.sd * exp2f(g2 * (float)(p.reverse ? r - r_begin + 1 - p.e : r_end - p.e - r));
    }
    __syncthreads();
    outer_add<kDp>(acc, sb, sc, sw, min(kC, r_end - r0));
  }
  float* dst = state_of(p);
  const int i0 = (tid / 16) * 2, j0 = (tid % 16) * 2;
#pragma unroll
  for (int i = 0; i < 2 * n; ++i)
#pragma unroll
    for (int v = 0; v < n; ++v) {
      const int r = i0 + 32 * (i / 2) + (i & 1), c = j0 + 32 * v;
      if (r < p.D && c < p.D)
        *reinterpret_cast<uint64_t*>(dst + (c & ~3) * p.D + r * 4 + (c & 3)) = acc[i][v];
    }
}

// The state before each segment in time order, written over the segment's own sum, and the state
// after the last: state_{s+1} = L^(rows of s) state_s + delta_s.  S0 and last are stored by rows and
// may be the same buffer (each element is read before it is written, by one thread).
struct Scan {
  float* states;
  const float* S0;
  float* last;
  int reverse;
};
struct Scans {
  Scan s[2];
  const float* log_decay;
  const int* lengths;
  int B, H, N, D;
  Cut cut;
};
// grid (ceil(D*D/4 / 256), B*H, scans), block 256.
__global__ void __launch_bounds__(256, 4) decay_scan_kernel(const __grid_constant__ Scans a) {
  sm100::grid_dep_signal();
  const float* S0 = a.s[blockIdx.z].S0;
  float* last = a.s[blockIdx.z].last;
  const int reverse = a.s[blockIdx.z].reverse, H = a.H, D = a.D;
  const int bh = blockIdx.y, b = bh / H, h = bh - b * H;
  const int n4 = D * D / 4, i = blockIdx.x * 256 + threadIdx.x;
  const int at = (i % D) * (D / 4) + i / D;  // of a state stored by rows
  const float g2 = log2_decay(a.log_decay, h);
  const int n = length_of(a.lengths, b, a.N);
  int per = a.cut.chunks, slot = b * a.cut.per_seq;
  if (a.cut.search) {
    __shared__ int found[2];
    if (threadIdx.x < 32) {
      const Search f(a.cut, a.lengths, a.B, a.N);
      const int before = f.slots_before(b);
      if (threadIdx.x == 0) {
        found[0] = f.per;
        found[1] = before;
      }
    }
    __syncthreads();
    per = found[0];
    slot = found[1];
  }
  const int seg_rows = per * a.cut.chunk, nseg = (n + seg_rows - 1) / seg_rows;
  sm100::grid_dep_wait();
  if (i >= n4) return;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (S0) acc = reinterpret_cast<const float4*>(S0)[(size_t)bh * n4 + at];
  float4* d = reinterpret_cast<float4*>(a.s[blockIdx.z].states) + ((size_t)slot * H + h) * n4 + i;
  const size_t stride = (size_t)H * n4;
  const int steps = last ? nseg : nseg - 1;  // the last segment's sum is only in the last state
  // eight segments' sums are loaded before any is written over, so their latencies overlap
  for (int t0 = 0; t0 < nseg; t0 += 8) {
    float4 add[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = t0 + u, s = reverse ? nseg - 1 - t : t;
      add[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t < steps) add[u] = d[s * stride];
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int t = t0 + u, s = reverse ? nseg - 1 - t : t;
      if (t >= nseg) break;
      d[s * stride] = acc;
      if (t < steps) acc = fma4(exp2f(g2 * (float)min(n - s * seg_rows, seg_rows)), acc, add[u]);
    }
  }
  if (last) reinterpret_cast<float4*>(last)[(size_t)bh * n4 + at] = acc;
}

// Zeros in the output rows of whole chunks of padding, by `n` threads of each CTA, this one the t-th.
// A pair's padding is dealt out in sixteen parts, one CTA after the other: left to one CTA, the
// padding of an empty sequence took as long as the rows of the others.  kBytes: of an element.
template <int kBytes>
__device__ __forceinline__ void zero_padding(const Pass& p, int t, int n) {
  if (!p.lengths) return;
  constexpr int kParts = 16;
  const int vec = p.D * kBytes / 16;
  for (int u = blockIdx.y * gridDim.x + blockIdx.x; u < p.B * p.H * kParts;
       u += gridDim.x * gridDim.y) {
    const int bh = u / kParts, part = u % kParts, b = bh / p.H, h = bh - b * p.H;
    const int z0 = chunks_of(p.lengths, b, p.N, p.cut.chunk) * p.cut.chunk;
    if (z0 >= p.N) continue;
    const int rows = (p.N - z0 + kParts - 1) / kParts, r0 = z0 + part * rows;
    uint8_t* out = static_cast<uint8_t*>(p.out) + (b * p.ob + h * p.oh + r0 * p.on) * kBytes;
    const int items = max(0, min(rows, p.N - r0)) * vec;
    for (int i = t; i < items; i += n) {
      const int r = i / vec;
      *reinterpret_cast<uint4*>(out + r * p.on * kBytes + (i - r * vec) * 16) =
          make_uint4(0, 0, 0, 0);
    }
  }
}

// The rows of one segment: chunks of kC in time order.  Bound by the fp32 pipes and shared memory
// alike: about kC D (1.1 kC + 2 D) multiply-adds a chunk, 56 % of the fp32 rate with 60 % of the
// shared-memory cycles at D = 128.  Half of the warps form scores and outputs, the other half the
// state, which they hold in registers and copy out between chunks (gradients of 4 sequences, 6 heads
// over 3, 1,151 rows, D = 128: 250 us, 281 with eight warps going through all of it in turn).
// Narrow heads run two CTAs an SM on 64 registers a thread, wide ones one on 128.
// grid (H, slots, passes), block 512.
constexpr int kRowThreads = 2 * kThreads;
template <int kN>
struct Blocks {
  static constexpr int value = kN;
};
template <int kDp>
__global__ void __launch_bounds__(kRowThreads, kDp <= 64 ? 2 : 1)
    decay_rows_kernel(const __grid_constant__ Passes all) {
  extern __shared__ __align__(16) float smf[];
  const Pass& p = all.p[blockIdx.z];
  const Segment seg = find_segment(p);
  const int b = seg.b, h = seg.h, r_begin = seg.begin, r_end = seg.end;
  zero_padding<4>(p, threadIdx.x, kRowThreads);
  constexpr int n = kDp / 32, ld = kDp + 4, ldp = kC + 4, kScoreSteps = kDp <= 64 ? 1 : 4;
  float* sa = smf;
  float* sb = sa + kC * ld;
  float* sc = sb + kC * ld;
  float* sp = sc + kC * ld;
  float* ss = sp + kC * ldp;
  float* spow = ss + kDp * ld;  // sp L^d
  float* sw = spow + kC;        // weights of b's rows
  const int tid = threadIdx.x, warp = (tid >> 5) & 7;
  const bool states = tid >= kThreads;
  const float g2 = log2_decay(p.log_decay, h);
  if (tid < kC) spow[tid] = p.sp * exp2f(g2 * (float)tid);

  sm100::grid_dep_wait();  // the states come from the launch before
  if (r_begin >= r_end) return;
  for (int i = tid; i < kDp * (kDp / 4); i += kRowThreads) {
    const int r = i % kDp, c = (i / kDp) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p.carried && r < p.D && c < p.D) {
      const float* src = state_of(p);
      if (p.transposed) {
        const float* col = src + (r >> 2) * 4 * p.D + c * 4 + (r & 3);
        x = make_float4(col[0], col[4], col[8], col[12]);
      } else {
        x = load4<float>(src + c * p.D + r * 4);
      }
    }
    *reinterpret_cast<float4*>(ss + r * ld + c) = x;
  }
  const int nc = (r_end - r_begin + kC - 1) / kC;
  auto chunk = [&](int ci) { return r_begin + (p.reverse ? nc - 1 - ci : ci) * kC; };
  auto load = [&](int r0) {
    load_rows<kDp, kRowThreads>(sa, p.a, b, h, r0, r_end, p.D);
    load_rows<kDp, kRowThreads>(sb, p.b, b, h, r0, r_end, p.D);
    load_rows<kDp, kRowThreads>(sc, p.c, b, h, r0, r_end, p.D);
    if (tid < kC) {
      const int rows = min(r_end - r0, kC);
      sw[tid] = p.sd * exp2f(g2 * (float)(p.reverse ? tid + 1 - p.e : rows - p.e - tid));
    }
  };
  load(chunk(0));
  __syncthreads();
  auto both = [] { sm100::named_bar_sync(1, kRowThreads); };  // of both halves, from either's code
  if (states) {  // S = L^rows S + sd * sum L^(rows - t - e) b c^T
    const int i2 = ((tid - kThreads) / 16) * 2, j2 = (tid % 16) * 2;
    uint64_t acc[2 * n][n];
    auto at = [&](int i, int v) {
      return reinterpret_cast<uint64_t*>(ss + (i2 + 32 * (i / 2) + (i & 1)) * ld + j2 + 32 * v);
    };
#pragma unroll
    for (int i = 0; i < 2 * n; ++i)
#pragma unroll
      for (int v = 0; v < n; ++v) acc[i][v] = *at(i, v);
    for (int ci = 0; ci < nc; ++ci) {
      const int rows = min(r_end - chunk(ci), kC);
      const bool more = ci + 1 < nc;
      if (more) {
        const uint64_t keep = twice(exp2f(g2 * (float)rows));
#pragma unroll
        for (int i = 0; i < 2 * n; ++i)
#pragma unroll
          for (int v = 0; v < n; ++v) acc[i][v] = sm100::f2_mul(keep, acc[i][v]);
        outer_add<kDp>(acc, sb, sc, sw, rows);
      }
      both();  // the chunk is used up
      if (!more) break;
#pragma unroll
      for (int i = 0; i < 2 * n; ++i)
#pragma unroll
        for (int v = 0; v < n; ++v) *at(i, v) = acc[i][v];
      load(chunk(ci + 1));
      both();
    }
    return;
  }
  float* out = static_cast<float*>(p.out) + b * p.ob + h * p.oh;
  // Eight rows a warp, of which a thread has rows i4 .. i4 + 3 and column pairs from j2.  The cost of a
  // warp's past grows with its rows, so the two warps of a scheduler (w, w + 4) get rows that
  // even out.
  const int eight = (warp < 4 ? warp : 11 - warp) * 8;
  const int i4 = eight + ((tid / 16) & 1) * 4, j2 = (tid % 16) * 2;
  // P = sp * L^|i-j| (a_i . b_j) over the past of i, 4 x kBlocks a thread (columns 16 apart)
  auto scores = [&](auto blocks, int rows) {
    constexpr int kBlocks = decltype(blocks)::value;
    const int j0 = tid % 16 + (p.reverse ? kC - 16 * kBlocks : 0);
    float acc[4][kBlocks] = {};
#pragma unroll kScoreSteps
    for (int k = 0; k < kDp; k += 4) {
      float4 x[4], y[kBlocks];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const float4*>(sa + (i4 + u) * ld + k);
#pragma unroll
      for (int w = 0; w < kBlocks; ++w)
        y[w] = *reinterpret_cast<const float4*>(sb + (j0 + 16 * w) * ld + k);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < kBlocks; ++w)
          acc[u][w] = fmaf(x[u].x, y[w].x, fmaf(x[u].y, y[w].y,
                      fmaf(x[u].z, y[w].z, fmaf(x[u].w, y[w].w, acc[u][w]))));
    }
    __syncwarp();  // a warp's rows of P are its own: it has read the last chunk's
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int w = 0; w < kBlocks; ++w) {
        const int i = i4 + u, j = j0 + 16 * w, d = p.reverse ? j - i : i - j;
        sp[i * ldp + j] = d >= 0 && j < rows ? spow[max(d, 0)] * acc[u][w] : 0.f;
      }
  };
  for (int ci = 0; ci < nc; ++ci) {
    const int r0 = chunk(ci), rows = min(r_end - r0, kC);  // valid rows
    const int past = p.reverse ? 4 - eight / 16 : eight / 16 + 1;  // blocks of 16 columns
    switch (past) {
      case 1: scores(Blocks<1>{}, rows); break;
      case 2: scores(Blocks<2>{}, rows); break;
      case 3: scores(Blocks<3>{}, rows); break;
      default: scores(Blocks<4>{}, rows); break;
    }
    __syncwarp();
    // out = si * L^(t + e) a^T S + P c
    uint64_t acc[4][n];
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < n; ++v) acc[u][v] = 0ull;
    auto add = [&](const float* xr, int ldx, const float* y, int k0, int k1) {
#pragma unroll 2
      for (int k = k0; k < k1; k += 4) {
        float4 x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const float4*>(xr + (i4 + u) * ldx + k);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint64_t yv[n];
#pragma unroll
          for (int v = 0; v < n; ++v) yv[v] = pair_at(y + (k + w) * ld + j2 + 32 * v);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float xv = w == 0 ? x[u].x : w == 1 ? x[u].y : w == 2 ? x[u].z : x[u].w;
#pragma unroll
            for (int v = 0; v < n; ++v) acc[u][v] = sm100::f2_fma(twice(xv), yv[v], acc[u][v]);
          }
        }
      }
    };
    add(sa, ld, ss, 0, kDp);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = p.reverse ? rows - 1 - (i4 + u) : i4 + u;
      const uint64_t f = twice(p.si * exp2f(g2 * (float)(max(t, 0) + p.e)));
#pragma unroll
      for (int v = 0; v < n; ++v) acc[u][v] = sm100::f2_mul(f, acc[u][v]);
    }
    // a warp's eight rows have no past beyond their last (first, backward in time)
    add(sp, ldp, sc, p.reverse ? eight : 0, p.reverse ? kC : eight + 8);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = i4 + u;
      if (r0 + r >= p.N) continue;
      float* dst = out + (long long)(r0 + r) * p.on;
#pragma unroll
      for (int v = 0; v < n; ++v)
        if (j2 + 32 * v < p.D)
          *reinterpret_cast<uint64_t*>(dst + j2 + 32 * v) = r < rows ? acc[u][v] : 0ull;
    }
    both();  // the chunk is used up
    if (ci + 1 == nc) break;
    load(chunk(ci + 1));
    both();
  }
}

// out[b, kv head, row] = sum over its `group` query heads of part [B][Hk * group][N][D] (fp32),
// in head order, for two tensors.  grid (blocks over rows * D / 4, B*Hk, 2), block 256.
struct GroupSum {
  const float* part[2];
  void* out[2];
  long long ob[2], oh[2], on[2];
  int Hk, group, N, D;
};
template <typename T>
__global__ void __launch_bounds__(256) decay_group_sum_kernel(const __grid_constant__ GroupSum a) {
  const int w = blockIdx.z, bk = blockIdx.y, b = bk / a.Hk, hk = bk - b * a.Hk;
  const int v4 = a.D / 4;
  const long long total = (long long)a.N * v4;
  const float4* src = reinterpret_cast<const float4*>(a.part[w]) + (long long)bk * a.group * total;
  T* out = static_cast<T*>(a.out[w]) + b * a.ob[w] + hk * a.oh[w];
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int u = 0; u < a.group; ++u) acc = fma4(1.f, src[u * total + i], acc);
    const long long r = i / v4;
    store4(out + r * a.on[w] + (i - r * v4) * 4, acc);
  }
}

// ---------------------------------------------------------------------------------------------
// One token: S <- L S + k v^T, o = scale * q S.
// ---------------------------------------------------------------------------------------------
struct StepParams {
  Rows q, k, v;            // sn unused (one row); k and v grouped
  void* out;
  long long ob, oh;
  const float* log_decay;
  float* state;            // [pool][H][D][D]
  const int* slots;        // [B] or null (sequence b's state is b)
  int B, H, D, pool;
  float scale;
};

// The state is read and written once (8 D^2 bytes a head and sequence), which bounds the step.  A
// CTA owns kStepCols columns of one state: eight lanes cover a row's 128 bytes, 16 rows a pass, so
// all its loads are in flight at once and no CTA waits on another.  States are read and written
// evict-first: a large batch's are gone from L2 by its next step (192 x 12 states of 64 KB: 53.7 us,
// 5.6 TB/s, against 55.3).  Wider column shares (64, 128) were no faster.
// A slot that a batch lists more than once is stepped in batch order: the CTA of its first entry
// holds the state in registers and takes the later entries' tokens too.  A negative slot is an
// idle entry (zeros out).  A slot past the pool is reported through the device error word.
// grid (ceil(D / kStepCols), H, B), block 128.
constexpr int kStepCols = 32, kStepThreads = 128;

template <typename T, int kPasses>
__global__ void __launch_bounds__(kStepThreads) decay_step_kernel(const StepParams p) {
  __shared__ float sq[kMaxD], sk[kMaxD];
  __shared__ float red[kStepThreads / 32][kStepCols];
  __shared__ int next_sh;
  const int tid = threadIdx.x, lane8 = tid & 7, row0 = tid >> 3;
  const int col = blockIdx.x * kStepCols + lane8 * 4;
  const int h = blockIdx.y;
  int b = blockIdx.z;
  const int D = p.D;
  const bool col_ok = col < D;
  const int slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.pool) {
    if (slot >= p.pool && tid == 0 && atomicCAS(&sm100::g_device_error, 0, 2) == 0) {
      sm100::g_bounds_info[0] = 50;
      sm100::g_bounds_info[1] = slot;
      sm100::g_bounds_info[2] = p.pool;
    }
    if (row0 == 0 && col_ok)
      store4(static_cast<T*>(p.out) + b * p.ob + h * p.oh + col, make_float4(0.f, 0.f, 0.f, 0.f));
    return;
  }
  float* S = p.state + ((size_t)slot * p.H + h) * D * D + col;
  float4 s[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + 16 * i;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < D && col_ok) s[i] = __ldcs(reinterpret_cast<const float4*>(S + (size_t)r * D));
  }
  if (p.slots) {  // an earlier entry of the same slot takes this one too
    bool earlier = false;
    for (int j = tid; j < b; j += kStepThreads) earlier |= p.slots[j] == slot;
    if (__syncthreads_or(earlier)) return;
  }
  const float L = expf(p.log_decay[h]);
  while (true) {
    if (tid < D / 4) {
      const T* q = static_cast<const T*>(p.q.p) + b * p.q.sb + (h / p.q.group) * p.q.sh + tid * 4;
      *reinterpret_cast<float4*>(sq + tid * 4) = load4<T>(q);
    } else if (tid >= 64 && tid < 64 + D / 4) {
      const int c = (tid - 64) * 4;
      const T* k = static_cast<const T*>(p.k.p) + b * p.k.sb + (h / p.k.group) * p.k.sh + c;
      *reinterpret_cast<float4*>(sk + c) = load4<T>(k);
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col_ok)
      v = load4<T>(static_cast<const T*>(p.v.p) + b * p.v.sb + (h / p.v.group) * p.v.sh + col);
    if (tid == 0) next_sh = p.B;
    __syncthreads();
    if (p.slots)
      for (int j = b + 1 + tid; j < p.B; j += kStepThreads)
        if (p.slots[j] == slot) {
          atomicMin(&next_sh, j);
          break;
        }
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = row0 + 16 * i;
      if (r < D) {
        s[i] = fma4(sk[r], v, mul4(L, s[i]));
        o = fma4(sq[r], s[i], o);
      }
    }
#pragma unroll
    for (int m = 8; m < 32; m <<= 1) {
      o.x += __shfl_xor_sync(0xffffffffu, o.x, m);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, m);
      o.z += __shfl_xor_sync(0xffffffffu, o.z, m);
      o.w += __shfl_xor_sync(0xffffffffu, o.w, m);
    }
    if ((tid & 31) < 8) *reinterpret_cast<float4*>(&red[tid >> 5][lane8 * 4]) = o;
    __syncthreads();
    if (tid < 8 && col_ok) {
      float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kStepThreads / 32; ++w)
        t = fma4(1.f, *reinterpret_cast<const float4*>(&red[w][tid * 4]), t);
      store4(static_cast<T*>(p.out) + b * p.ob + h * p.oh + col, mul4(p.scale, t));
    }
    b = next_sh;
    if (b >= p.B) break;
    __syncthreads();  // red, sq, sk and next_sh are written again
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = row0 + 16 * i;
    if (r < D && col_ok) __stcs(reinterpret_cast<float4*>(S + (size_t)r * D), s[i]);
  }
}

}  // namespace decay
}  // namespace rehyat
