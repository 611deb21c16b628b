// Linear attention with a decay per head on the tensor cores (bf16, D <= 128): the two passes of
// decay.cuh over 128-row chunks.
//
// A chunk of the row pass moves 128 KB of HBM (a, b, c in, out) for four 128^3 products: 3.0 us of one
// SM's share of the measured copy rate, against 1.1 us of the tensor pipe at 1.9 GHz.  The 480x832 5 s
// prompt (12 heads, 32,760 rows, D = 128; 402 MB): rows 74-79 us, 5.1 to 5.4 TB/s or 0.78 to 0.83 of the
// copy rate, 3.5-3.7 us a chunk.  So HBM bounds it first, with each CTA's start and the chain from one
// chunk to the next on top: of the cycles, shared memory is busy in 64 % (products 27, warps 21, copies
// 16) and the tensor pipe in 31 %.  What a prompt takes beyond that is the states pass, 46 us (4.4 TB/s,
// k and v read a first time), and the scan.  Long runs are held at 1.45-1.65 GHz by the board's power
// limit.
// Not faster: the outputs on eight warps of their own (setmaxnreg shares), runs of chunks that cross
// from one head into the next, L2 eviction hints, waits by test_wait or with nanosleep.
// One CTA per SM, two (rows) or three (states) stages of whole chunks, one warp for each thing that
// waits, short loops (straight-line code of every role at once overran the instruction cache).
//
// Rounded to bf16: the weighted scores P, the weighted rows b of the carried state, the state the
// rows read, and the output; sums, states and powers are fp32.  Where the last state is given out, the
// states pass multiplies each weighted row in two bf16 parts (16 mantissa bits), so that state and those
// between segments are fp32 sums of terms good to 2^-16; where only the row pass reads them, in one.
//
// Narrow heads (D < 128) run on the same tiles: columns at and past D load as zeros (the tensor map
// ends there) and are not stored, and the products' depth and width stop at D rounded up to 16.
#pragma once

#include "decay.cuh"
#include "sm100_rows.cuh"

namespace rehyat {
namespace decay {
namespace tc {

using namespace sm100;

constexpr int kRows = 128;  // rows of a chunk
constexpr uint32_t kTile = kRows * 128 * 2;

__device__ __forceinline__ uint64_t kmajor_desc(uint32_t tile, int kk) {
  return sdesc_sw128(tile + (kk >> 2) * (kRows * 128) + (kk & 3) * 32, 16, 1024);
}
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t tile, int kk) {
  return sdesc_sw128(tile + kk * 16 * 128, kRows * 128, 1024);
}
__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}
__device__ __forceinline__ void load_tile(int site, uint8_t* dst, const CUtensorMap* m,
                                          uint64_t* bar, int row, int h, int b, const Pass& p,
                                          int heads) {
  tma_load_4d_chk(site, dst, m, bar, 0, row, h, b, p.N, heads, p.B);
  tma_load_4d_chk(site, dst + kRows * 128, m, bar, 64, row, h, b, p.N, heads, p.B);
}
__device__ __forceinline__ uint64_t f2_bits(uint32_t lo, uint32_t hi) {
  return f2_pack(__uint_as_float(lo), __uint_as_float(hi));
}
__device__ __forceinline__ uint32_t f2_bf16(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return pack_bf16x2(a, b);
}
// Eight bf16 values times w, rounded to bf16; with kTwo what the rounding left in a second part.
template <bool kTwo>
__device__ __forceinline__ uint4 scale8(uint4 x, float w, uint4& lo) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t hi[4], rest[4] = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a bf16 is the upper half of an fp32
    const uint64_t f = f2_mul(f2_bits(in[i] << 16, in[i] & 0xffff0000u), f2_pack(w, w));
    hi[i] = f2_bf16(f);
    if (kTwo)
      rest[i] = f2_bf16(f2_fma(f2_bits(hi[i] << 16, hi[i] & 0xffff0000u), f2_pack(-1.f, -1.f), f));
  }
  lo = make_uint4(rest[0], rest[1], rest[2], rest[3]);
  return make_uint4(hi[0], hi[1], hi[2], hi[3]);
}
// A weight w > 0 in two bf16 parts, hi + lo, good to 2^-16 of w.  hi is cut, so lo has its sign, and
// lo is never zero: an infinity times the parts stays one.
struct Weight {
  __nv_bfloat162 hi, lo;
  __device__ __forceinline__ explicit Weight(float w) {
    const float h = __uint_as_float(__float_as_uint(w) & 0xffff0000u);
    hi = __float2bfloat162_rn(h);
    lo = __float2bfloat162_rn(fmaxf(w - h, 1.17549435e-38f));
  }
};
// Eight bf16 values times a weight, rounded to bf16 once: the small part's product is added to the
// large one's before that is rounded.
__device__ __forceinline__ uint4 mul8(uint4 x, const Weight& w) {
  __nv_bfloat162* v = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __hfma2(v[i], w.hi, __hmul2(v[i], w.lo));
  return x;
}
// Weights L^m of n rows, m from 1 - e to n - e, are taken relative to L^middle, which a sum over the
// rows is multiplied by in fp32.  Rounding x w to bf16 gives x for every w just below 1: where the
// decay is slow, all rows would be rounded up together and their sum come out up to 0.1 % too large
// (measured 0.08 % at log_decay = -1.2e-5; 0.002 % with w on both sides of 1).  A span beyond two
// halvings crosses enough steps of the type to average out by itself, and is left alone so that no
// power grows beyond 2.
__device__ __forceinline__ float middle(float g2, int n, int e) {
  return fabsf(g2) * (float)(n + 1) <= 2.f ? 0.5f * (float)(n + 1) - (float)e : 0.f;
}

// ---------------------------------------------------------------------------------------------
// States: sd * sum_j L^(n - t_j - e) b_j c_j^T over a segment.
// ---------------------------------------------------------------------------------------------
constexpr int kStStages = 3;
constexpr int kStHalf = 256;                   // warps 0-7 weigh rows 0-63 of a chunk, 8-15 the rest
constexpr int kStIn = 16, kStMma = 17;         // copies, products
constexpr int kStThreads = 2 * kStHalf + 64;
constexpr uint32_t kStOffLo = kStStages * 2 * kTile;
constexpr uint32_t kStSmem = kStOffLo + kTile + 1024;
static_assert(kStSmem + 1024 <= 232448, "shared memory over the limit");

// Every weight is taken to the segment's end (or its middle, see above), so chunks add up without
// rescaling, in any order; what all share, that power and sd, multiplies the sum.
// They run in the order opposite to the row pass that follows: what was read last (and may still be
// in L2) is read first there.  The two halves of a chunk have their own warps and barriers, so one
// is weighed while the other is multiplied.
// kTwo: weighted rows in two bf16 parts, for a last state good to fp32; without, in one, for sums
// that only the row pass reads (it rounds the state to bf16 anyway).
// The tensor core's own accumulation truncates, which shows in fp32 sums over thousands of rows
// (8.6e-6 of the state after 12,600 rows).  So every kFlush chunks the sum goes on in the other of
// two accumulators, and kLate chunks later, when its products are long complete, the first is added
// to registers; it is written again only after both halves have weighed a later chunk.
constexpr int kFlush = 8, kLate = 2;
template <bool kTwo>
__device__ __forceinline__ void states_of_segment(const CUtensorMap& tmB, const CUtensorMap& tmC,
                                                  const Pass& p, const Segment& seg) {
  enum {
    kFull = 0, kEmpty = kFull + kStStages, kReady = kEmpty + kStStages,  // kReady: [half][stage]
    kLoFree = kReady + 2 * kStStages, kSummed = kLoFree + 2, kDone, kNum
  };
  const int b = seg.b, h = seg.h, r_begin = seg.begin, r_end = seg.end;
  const int nc = (r_end - r_begin + kRows - 1) / kRows;
  if (nc <= 0 || (seg.last && !p.exact)) return;  // nothing reads its sum
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ __align__(8) uint64_t bars[kNum];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  volatile int* abort_flag = &abort_sh;
  if (warp == kStIn) {
    tmem_alloc(&tmem_sh, 256);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kNum; ++i)
      mbar_init(&bars[i], i >= kReady && i < kLoFree ? kStHalf : 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  auto wait = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(&bars[bar], parity, abort_flag));
  };
  auto chunk_row = [&](int i) { return r_begin + (p.reverse ? i : nc - 1 - i) * kRows; };

  if (warp == kStIn) {  // ---- copies ----
    const int hb = h / p.b.group, hc = h / p.c.group;
    bool ok = true;
    int issued = 0;
    for (int i = 0; i < nc; ++i) {
      const int s = i % kStStages;
      if (i >= kStStages) ok = wait(kEmpty + s, (i / kStStages - 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        uint8_t* dst = sm + s * 2 * kTile;
        mbar_arrive_expect_tx(&bars[kFull + s], 2 * kTile);
        load_tile(51, dst, &tmB, &bars[kFull + s], chunk_row(i), hb, b, p, p.H / p.b.group);
        load_tile(52, dst + kTile, &tmC, &bars[kFull + s], chunk_row(i), hc, b, p, p.H / p.c.group);
      }
      __syncwarp();
      ++issued;
    }
    if (!ok)
      for (int i = max(0, issued - kStStages); i < issued; ++i)
        mbar_wait_drain(&bars[kFull + i % kStStages], (i / kStStages) & 1);
    __syncwarp();
  } else if (warp == kStMma) {  // ---- products: b^T c, both parts of b ----
    const int w = (p.D + 15) / 16 * 16;
    const uint32_t id = idesc_bf16(128, w, true, true);
    const uint32_t sm0 = smem_u32(sm), lo = sm0 + kStOffLo, leader = elect_lane();
    bool ok = true;
    for (int i = 0; i < nc && ok; ++i) {
      const int s = i % kStStages;
      const uint32_t sum = tmem + ((i / kFlush) & 1) * 128;
      for (int half = 0; half < 2 && ok; ++half) {
        ok = wait(kReady + half * kStStages + s, (i / kStStages) & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t hi = sm0 + s * 2 * kTile, c = hi + kTile;
#pragma unroll
        for (int k4 = 0; k4 < 4; ++k4) {
          const int kk = half * 4 + k4;
          mma_ss_by(leader, sum, mnmajor_desc(hi, kk), mnmajor_desc(c, kk), id,
                    (i % kFlush > 0 || kk > 0) ? 1u : 0u);
          if (kTwo)
            mma_ss_by(leader, sum, mnmajor_desc(lo, kk), mnmajor_desc(c, kk), id, 1u);
        }
        if (kTwo) mma_commit_by(leader, &bars[kLoFree + half]);
        if (half) mma_commit_by(leader, &bars[kEmpty + s]);
        if (half && (i + 1) % kFlush == 0) mma_commit_by(leader, &bars[kSummed]);
        __syncwarp();
      }
    }
    mma_commit_by(leader, &bars[kDone]);
    __syncwarp();
    mbar_wait_drain(&bars[kDone], 0);
    __syncwarp();
  } else {  // ---- weights: a row of a half chunk, 32 columns a thread ----
    const int half = warp >> 3, r = half * 64 + (tid & 63), c0 = ((tid >> 6) & 3) * 32;
    const float g2 = log2_decay(p.log_decay, h), mid = middle(g2, r_end - r_begin, p.e);
    // the sum: row (TMEM lane) rs, columns cs .. cs + 31
    const int rs = tid & 127, cs = (tid >> 7) * 32;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float sum[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) sum[j] = 0.f;
    auto flush = [&](int group) {
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(tmem + lanes + (group & 1) * 128 + cs, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) sum[j] += __uint_as_float(v[j]);
      tc_fence_before();
    };
    bool ok = true;
    for (int i = 0; i < nc; ++i) {
      const int s = i % kStStages;
      const int row = chunk_row(i) + r;
      const bool valid = row < r_end;
      const int m = p.reverse ? row - r_begin + 1 - p.e : r_end - p.e - row;
      const float w = valid ? exp2f(g2 * ((float)m - mid)) : 0.f;
      ok = wait(kFull + s, (i / kStStages) & 1);
      if (!ok) break;
      uint8_t* hi = sm + s * 2 * kTile;
      uint8_t* lo = sm + kStOffLo;
      uint4 x[4], rest[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = *reinterpret_cast<uint4*>(hi + sw128_offset(r, c0 + j * 8, kRows));
        if (!valid) x[j] = make_uint4(0, 0, 0, 0);  // padding may hold anything
        x[j] = scale8<kTwo>(x[j], w, rest[j]);
      }
      if (kTwo && i > 0) ok = wait(kLoFree + half, (i - 1) & 1);
      if (ok && i > kFlush && i % kFlush == kLate) {
        ok = wait(kSummed, (i / kFlush - 1) & 1);
        if (ok) flush(i / kFlush - 1);
      }
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t off = sw128_offset(r, c0 + j * 8, kRows);
        *reinterpret_cast<uint4*>(hi + off) = x[j];
        if (kTwo) *reinterpret_cast<uint4*>(lo + off) = rest[j];
        if (!valid) *reinterpret_cast<uint4*>(hi + kTile + off) = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      mbar_arrive(&bars[kReady + half * kStStages + s]);
    }
    if (ok) ok = wait(kDone, 0);
    if (ok) {
      const int group = (nc - 1) / kFlush;
      if (group > 0 && (nc - 1) % kFlush < kLate) flush(group - 1);
      flush(group);
      float* dst = state_of(p) + rs * 4;
      const float all = p.sd * exp2f(g2 * mid);
#pragma unroll
      for (int j = 0; j < 32; ++j) sum[j] *= all;
      if (rs < p.D) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (cs + j * 4 < p.D)
            *reinterpret_cast<float4*>(dst + (cs + j * 4) * p.D) =
                make_float4(sum[j * 4], sum[j * 4 + 1], sum[j * 4 + 2], sum[j * 4 + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kStIn) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// The passes of one launch, one after the other (blockIdx.z): a pass fills the SMs that the one
// before leaves idle at its end.  Interleaving them, so that passes over the same rows run side by
// side, was slower (480x832 5 s gradients 385 us against 316).
struct StatesArgs {
  Pass p[2];
  CUtensorMap b[2], c[2];
};
// grid (H, slots, passes), block 576.
__global__ void __launch_bounds__(kStThreads, 1)
    decay_states_bf16_kernel(const __grid_constant__ StatesArgs a) {
  grid_dep_signal();
  const int w = blockIdx.z;
  const Segment seg = find_segment(a.p[w]);
  if (a.p[w].exact)
    states_of_segment<true>(a.b[w], a.c[w], a.p[w], seg);
  else
    states_of_segment<false>(a.b[w], a.c[w], a.p[w], seg);
}

// ---------------------------------------------------------------------------------------------
// Rows.
// ---------------------------------------------------------------------------------------------
// warps 0-7: scores and outputs, 8-15: weights and the state (of each, four warps take columns 0-63
// and four 64-127), 16: copies in, 17: products, 18: copies out.
constexpr int kRwThreads = 608;
constexpr int kRwIn = 16, kRwMma = 17, kRwOut = 18;
constexpr uint32_t kRwStage = 3 * kTile;
constexpr uint32_t kRwOffS = 2 * kRwStage;
constexpr uint32_t kRwSmem = kRwOffS + kTile + 1024;
static_assert(kRwSmem + 2048 <= 232448 + 512, "shared memory over the limit");
// TMEM columns: scores a b^T (P over them), P c, a S, the chunk's own b^T c
constexpr uint32_t kColP = 0, kColIn = 128, kColSt = 256, kColAdd = 384;

// No barrier completes a phase ahead of a thread that has yet to wait for the one before: each is
// either armed by that thread's own earlier step or, like kStaged, has one for each stage.
// A chunk i, chunk after chunk in time order:
//   scores = a b^T -> P = sp L^|i-j| scores on the past, bf16, into TMEM     (warps 0-7)
//   b weighted in place (after the scores have read it)                       (warps 8-15)
//   add = b^T c;  in = P c;  st = a S                                         (warp 17)
//   out = in + si L^(t+e) st -> over c's tile -> global                       (warps 0-7, 18)
// (over c's, which the next product needs last: over a's, the next load of a came 1,100 clk late)
//   S = L^rows S + sd add, in registers (half a row a thread), bf16 copy for a S (warps 8-15)
template <bool kReverse, bool kOutF32>
__device__ __forceinline__ void rows_of_segment(const CUtensorMap& tmA, const CUtensorMap& tmB,
                                                const CUtensorMap& tmC, const CUtensorMap& tmOut,
                                                const Pass& p, const Segment& seg) {
  enum {
    kAFull = 0, kBFull = 2, kCFull = 4, kAEmpty = 6, kBEmpty = 8, kCEmpty = 10, kScores = 12,
    kPReady, kBReady, kOFull, kAddFull, kStaged, kDone = kStaged + 2, kNum
  };
  const int b = seg.b, h = seg.h, r_begin = seg.begin, r_end = seg.end;
  const int nc = (r_end - r_begin + kRows - 1) / kRows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (nc <= 0) {
    zero_padding<kOutF32 ? 4 : 2>(p, tid, kRwThreads);
    grid_dep_wait();
    return;
  }
  auto chunk_row = [&](int i) { return r_begin + (kReverse ? nc - 1 - i : i) * kRows; };

  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  __shared__ __align__(8) uint64_t bars[kNum];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ float diag_sh[64];  // sp L^(i - 31), zeros below 31: the past of a 32 x 32 block
  volatile int* abort_flag = &abort_sh;
  if (tid < 64) {
    const float g2 = log2_decay(p.log_decay, h);
    diag_sh[tid] = tid < 31 ? 0.f : p.sp * ex2(g2 * (float)(tid - 31));
  }
  if (warp == kRwIn) {
    tmem_alloc(&tmem_sh, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < kNum; ++i) {
      const bool many = i == kPReady || i == kBReady || i == kStaged || i == kStaged + 1;
      mbar_init(&bars[i], many ? 256 : 1);
    }
    abort_sh = 0;
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  const bool carried = p.carried;  // chunk 0 has a state to read
  auto wait = [&](int bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(&bars[bar], parity, abort_flag));
  };

  if (warp == kRwIn) {  // ---- copies in ----
    const int hb = h / p.b.group, hc = h / p.c.group, ha = h / p.a.group;
    if (lane == 0) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
      tma_prefetch_desc(&tmC);
    }
    __syncwarp();
    bool ok = true;
    int n_a = 0, n_b = 0, n_c = 0;
    auto load = [&](int i, int full, int empty, int slot, const CUtensorMap* m, int head, int heads,
                    int& n) {
      const int s = i & 1;
      if (i >= 2) ok = wait(empty + s, ((i >> 1) - 1) & 1);
      if (!ok) return;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[full + s], kTile);
        load_tile(53 + slot, sm + s * kRwStage + slot * kTile, m, &bars[full + s], chunk_row(i), head,
                  b, p, heads);
      }
      __syncwarp();
      ++n;
    };
    for (int i = 0; i < nc && ok; ++i) {
      load(i, kBFull, kBEmpty, 1, &tmB, hb, p.H / p.b.group, n_b);  // in the order they come free
      if (ok) load(i, kAFull, kAEmpty, 0, &tmA, ha, p.H / p.a.group, n_a);
      if (ok) load(i, kCFull, kCEmpty, 2, &tmC, hc, p.H / p.c.group, n_c);
    }
    if (!ok) {
      auto drain = [&](int full, int n) {
        for (int i = max(0, n - 2); i < n; ++i) mbar_wait_drain(&bars[full + (i & 1)], (i >> 1) & 1);
      };
      drain(kAFull, n_a);
      drain(kBFull, n_b);
      drain(kCFull, n_c);
    }
    __syncwarp();
  } else if (warp == kRwMma) {  // ---- products ----
    const int kd = (p.D + 15) / 16, w = kd * 16;
    const uint32_t id_p = idesc_bf16(128, 128, false, false);  // a (K-major) x b (K-major)
    const uint32_t id_o = idesc_bf16(128, w, false, true);     // P or a x c or S (N-major)
    const uint32_t id_s = idesc_bf16(128, w, true, true);      // b^T x c
    const uint32_t sm0 = smem_u32(sm), sS = sm0 + kRwOffS, leader = elect_lane();
    auto tile = [&](int i, int slot) { return sm0 + (i & 1) * kRwStage + slot * kTile; };
    auto scores = [&](int i) {
      bool ok = wait(kAFull + (i & 1), (i >> 1) & 1) && wait(kBFull + (i & 1), (i >> 1) & 1);
      if (!ok) return false;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        if (kk < kd)
          mma_ss_by(leader, tmem + kColP, kmajor_desc(tile(i, 0), kk), kmajor_desc(tile(i, 1), kk),
                    id_p, kk > 0 ? 1u : 0u);
      mma_commit_by(leader, &bars[kScores]);
      __syncwarp();
      return true;
    };
    bool ok = scores(0);
    for (int i = 0; i < nc && ok; ++i) {
      const int s = i & 1;
      const bool last = i + 1 == nc, reads_state = i > 0 || carried;
      // the threads that arrive on kBReady have read chunk i - 1's sum out of TMEM and published
      // the state before; those of kPReady have read chunk i - 1's outputs
      ok = wait(kCFull + s, (i >> 1) & 1) && wait(kBReady, i & 1);
      if (!ok) break;
      tc_fence_after();
      if (!last) {
#pragma unroll
        for (int kk = 0; kk < kRows / 16; ++kk)
          mma_ss_by(leader, tmem + kColAdd, mnmajor_desc(tile(i, 1), kk),
                    mnmajor_desc(tile(i, 2), kk), id_s, kk > 0 ? 1u : 0u);
        mma_commit_by(leader, &bars[kAddFull]);
      }
      mma_commit_by(leader, &bars[kBEmpty + s]);
      __syncwarp();
      ok = wait(kPReady, i & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < kRows / 16; ++kk)
        mma_ts_by(leader, tmem + kColIn, tmem + kColP + (kk >> 2) * 64 + (kk & 3) * 8,
                  mnmajor_desc(tile(i, 2), kk), id_o, kk > 0 ? 1u : 0u);
      if (reads_state) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk < kd)
            mma_ss_by(leader, tmem + kColSt, kmajor_desc(tile(i, 0), kk), mnmajor_desc(sS, kk), id_o,
                      kk > 0 ? 1u : 0u);
      }
      mma_commit_by(leader, &bars[kOFull]);
      mma_commit_by(leader, &bars[kAEmpty + s]);
      __syncwarp();
      if (!last) ok = scores(i + 1);
    }
    mma_commit_by(leader, &bars[kDone]);
    __syncwarp();
    mbar_wait_drain(&bars[kDone], 0);
    __syncwarp();
  } else if (warp == kRwOut) {  // ---- copies out; c's tile is free once the output has left it ----
    bool ok = true;
    for (int i = 0; i < nc && ok; ++i) {
      ok = wait(kStaged + (i & 1), (i >> 1) & 1);
      if (!ok) break;
      if (lane == 0) {
        if (!kOutF32) {
          const uint8_t* src = sm + (i & 1) * kRwStage + 2 * kTile;
          tma_store_4d_chk(56, &tmOut, src, 0, chunk_row(i), h, b, p.N, p.H, p.B);
          if (p.D > 64)
            tma_store_4d_chk(56, &tmOut, src + kRows * 128, 64, chunk_row(i), h, b, p.N, p.H, p.B);
          bulk_commit_group();
          bulk_wait_read_all();
        }
        mbar_arrive(&bars[kCEmpty + (i & 1)]);
      }
      __syncwarp();
    }
    if (!kOutF32 && lane == 0) bulk_wait_all();
    __syncwarp();
  } else if (warp < 8) {  // ---- scores and outputs: row r of the chunk = TMEM lane ----
    const int r = tid & 127, half = warp >> 2, rw = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(rw * 32) << 16;
    const float g2 = log2_decay(p.log_decay, h);
    // L^|i-j| off the diagonal 32 x 32 blocks = (power of the row to the near edge of 16 columns)
    // x (power within them), both exponents >= 0; on the diagonal one power an element
    uint64_t within[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      within[j] = f2_pack(ex2(g2 * (float)(kReverse ? 2 * j : 15 - 2 * j)),
                          ex2(g2 * (float)(kReverse ? 2 * j + 1 : 14 - 2 * j)));
    bool ok = true;
    for (int i = 0; i < nc; ++i) {
      const int row0 = chunk_row(i), rows = min(kRows, r_end - row0);
      ok = wait(kScores, i & 1);
      if (!ok) break;
      tc_fence_after();
      // 32 columns a turn; a warp's P (64 columns' bf16 pairs: 32 TMEM columns) lies over its own
      // half of the scores, behind the columns already read
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        const int jb = half * 2 + q;
        uint32_t pk[16];
        if (kReverse ? jb < rw : jb > rw) {  // no past here
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = 0u;
        } else {
          uint32_t v[32];
          tmem_ld32(tmem + lanes + kColP + jb * 32, v);
          if (rows == kRows && jb == rw) {
            // the powers of the diagonal block by lane - column; above it they are zeros
            const float* w = diag_sh + (kReverse ? 31 - lane : lane + 31);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pk[j] = f2_bf16(f2_mul(f2_pack(w[kReverse ? 2 * j : -2 * j],
                                             w[kReverse ? 2 * j + 1 : -2 * j - 1]),
                                     f2_bits(v[2 * j], v[2 * j + 1])));
          } else if (jb == rw || (kReverse && rows < kRows)) {
            // a chunk with padding, whose scores may hold anything: one power and mask an element
            const int d0 = kReverse ? jb * 32 - r : r - jb * 32;
            const int stop = rows - jb * 32;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              float f[2];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const int c = 2 * j + u, d = kReverse ? d0 + c : d0 - c;
                const float x = p.sp * ex2(g2 * (float)d) * __uint_as_float(v[c]);
                f[u] = d >= 0 && (!kReverse || c < stop) ? x : 0.f;
              }
              pk[j] = pack_bf16x2(f[0], f[1]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c0 = jb * 32 + e * 16;
              const float edge = p.sp * ex2(g2 * (float)(kReverse ? c0 - r : r - c0 - 15));
              const uint64_t edge2 = f2_pack(edge, edge);
#pragma unroll
              for (int j = 0; j < 8; ++j)
                pk[e * 8 + j] = f2_bf16(f2_mul(f2_mul(edge2, within[j]),
                                               f2_bits(v[e * 16 + 2 * j], v[e * 16 + 2 * j + 1])));
            }
          }
        }
        tmem_st16(tmem + lanes + kColP + half * 64 + q * 16, pk);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&bars[kPReady]);

      const bool reads_state = i > 0 || carried;
      const int t = kReverse ? rows - 1 - r : r;
      const bool valid = r < rows;
      const float f = p.si * ex2(g2 * (float)(max(t, 0) + p.e));
      const uint64_t f2 = f2_pack(f, f);
      ok = wait(kOFull, i & 1);
      if (!ok) break;
      tc_fence_after();
      uint8_t* stage = sm + (i & 1) * kRwStage + 2 * kTile;
      float* of = kOutF32 ? static_cast<float*>(p.out) + b * p.ob + h * p.oh + (row0 + r) * p.on
                          : nullptr;
      const int c_end = min(half * 64 + 64, p.D);
#pragma unroll 1
      for (int c0 = half * 64; c0 < c_end; c0 += 32) {
        uint64_t o[16];
        if (reads_state) {
          uint32_t v[32], w[32];
          tmem_ld32_pair(tmem + lanes + kColIn + c0, tmem + lanes + kColSt + c0, v, w);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            o[j] = f2_fma(f2, f2_bits(w[2 * j], w[2 * j + 1]), f2_bits(v[2 * j], v[2 * j + 1]));
        } else {
          uint32_t v[32];
          tmem_ld32(tmem + lanes + kColIn + c0, v);
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = f2_bits(v[2 * j], v[2 * j + 1]);
        }
        if (!valid)
#pragma unroll
          for (int j = 0; j < 16; ++j) o[j] = 0ull;
        if (kOutF32) {
          if (row0 + r < p.N)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c0 + j * 4 < p.D) {
                float4 x;
                f2_unpack(o[2 * j], x.x, x.y);
                f2_unpack(o[2 * j + 1], x.z, x.w);
                *reinterpret_cast<float4*>(of + c0 + j * 4) = x;
              }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(stage + sw128_offset(r, c0 + j * 8, kRows)) =
                make_uint4(f2_bf16(o[4 * j]), f2_bf16(o[4 * j + 1]), f2_bf16(o[4 * j + 2]),
                           f2_bf16(o[4 * j + 3]));
        }
      }
      tc_fence_before();
      fence_async_smem();
      mbar_arrive(&bars[kStaged + (i & 1)]);
    }
  } else {  // ---- weights and the state: row r of b's tile, and row r of S = TMEM lane ----
    const int r = tid & 127, c0 = ((warp - 8) >> 2) * 64;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float g2 = log2_decay(p.log_decay, h);
    uint8_t* sS = sm + kRwOffS;
    uint64_t S[32];  // pairs of columns
#pragma unroll
    for (int j = 0; j < 32; ++j) S[j] = 0ull;
    auto publish = [&]() {  // bf16 copy of S for the next chunk's a S
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(sS + sw128_offset(r, c0 + j * 8, kRows)) = make_uint4(
            f2_bf16(S[j * 4]), f2_bf16(S[j * 4 + 1]), f2_bf16(S[j * 4 + 2]), f2_bf16(S[j * 4 + 3]));
    };
    zero_padding<kOutF32 ? 4 : 2>(p, tid - 256, 256);  // nothing else to do yet
    grid_dep_wait();  // the states come from the launch before
    if (carried && r < p.D) {
      const float* src = state_of(p);
      // loads in batches, before any is used
      if (p.transposed) {
        const float* col = src + (r >> 2) * 4 * p.D + c0 * 4 + (r & 3);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float x[16];
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[j] = c0 + q * 16 + j < p.D ? col[(q * 16 + j) * 4] : 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) S[q * 8 + j] = f2_pack(x[2 * j], x[2 * j + 1]);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float4 x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = c0 + q * 32 + j * 4;
            x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < p.D) x[j] = *reinterpret_cast<const float4*>(src + c * p.D + r * 4);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            S[q * 16 + j * 2] = f2_pack(x[j].x, x[j].y);
            S[q * 16 + j * 2 + 1] = f2_pack(x[j].z, x[j].w);
          }
        }
      }
    }
    publish();
    bool ok = true;
    for (int i = 0; i < nc; ++i) {
      const int s = i & 1;
      const bool last = i + 1 == nc;
      const int rows = min(kRows, r_end - chunk_row(i));
      const int t = kReverse ? rows - 1 - r : r;
      const bool valid = r < rows;
      // x w is rounded to bf16 once, on the way through the carried state (with the state's copy and
      // the output three roundings: 2^-8 / sqrt(3) * sqrt(3) = 3.9e-3 at most in the mean square)
      const float mid = middle(g2, rows, p.e);
      const Weight w(valid ? ex2(g2 * ((float)(rows - t - p.e) - mid)) : 0.f);
      const float all = p.sd * ex2(g2 * mid);
      uint8_t* tb = sm + s * kRwStage + kTile;
      ok = wait(kScores, i & 1) && wait(kCFull + s, (i >> 1) & 1);
      if (!ok) break;
      if (!last) {
#pragma unroll 1
        for (int c = c0; c < c0 + 64; c += 16) {
          uint4* q0 = reinterpret_cast<uint4*>(tb + sw128_offset(r, c, kRows));
          uint4* q1 = reinterpret_cast<uint4*>(tb + sw128_offset(r, c + 8, kRows));
          uint4 x = *q0, y = *q1;
          if (!valid) x = y = make_uint4(0, 0, 0, 0);
          *q0 = mul8(x, w);
          *q1 = mul8(y, w);
        }
      }
      if (!valid)  // padding may hold anything, and P's zeros must not meet it
#pragma unroll 1
        for (int c = c0; c < c0 + 64; c += 8)
          *reinterpret_cast<uint4*>(tb + kTile + sw128_offset(r, c, kRows)) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
      mbar_arrive(&bars[kBReady]);
      if (last) break;
      const float keep = ex2(g2 * (float)rows);
      const uint64_t keep2 = f2_pack(keep, keep), all2 = f2_pack(all, all);
      // also waits until a S of this chunk has read the copy
      ok = wait(kAddFull, i & 1) && wait(kOFull, i & 1);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t v[16];
        tmem_ld16(tmem + lanes + kColAdd + c0 + q * 16, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          S[q * 8 + j] = f2_fma(keep2, S[q * 8 + j],
                                f2_mul(all2, f2_bits(v[2 * j], v[2 * j + 1])));
      }
      tc_fence_before();
      publish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kRwIn) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct RowsArgs {
  Pass p[3];
  CUtensorMap a[3], b[3], c[3], out[3];
};
// grid (H, slots, passes), block 608.
__global__ void __launch_bounds__(kRwThreads, 1)
    decay_rows_bf16_kernel(const __grid_constant__ RowsArgs a) {
  const int w = blockIdx.z;
  const Pass& p = a.p[w];
  const Segment seg = find_segment(p);
  if (!p.reverse)
    rows_of_segment<false, false>(a.a[w], a.b[w], a.c[w], a.out[w], p, seg);
  else if (!p.out_f32)
    rows_of_segment<true, false>(a.a[w], a.b[w], a.c[w], a.out[w], p, seg);
  else
    rows_of_segment<true, true>(a.a[w], a.b[w], a.c[w], a.out[w], p, seg);
}

}  // namespace tc
}  // namespace decay
}  // namespace rehyat
