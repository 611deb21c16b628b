// Rotary positions: pair p of a head's first R dimensions turns by the angle pos * freq[p],
//     (x1, x2) -> scale * (x1 cos a - x2 sin a, x2 cos a + x1 sin a),
// with (x1, x2) = (x[p], x[p + R/2]) (halves) or (x[2p], x[2p + 1]) (interleaved); dimensions R
// and up are copied.  The gradient is the same turn by -a.
//
// Angles: a float holds pos * freq only to 2^-24 of its value, which at position 10^6 is 0.06
// radians.  So a frequency is kept as a 64-bit fraction of a turn, within 2 units of 2^-64, and
// pos * freq modulo one turn is an integer product that wraps: off by at most 2 |pos| 2^-64 turns
// (7.5e-7 radians at position 2^40; a fraction of fp64's 53 bits was 8.9e-5 off there).  Of the
// wrapped turn the nearest quarter is taken off, so what becomes a float is at most an eighth of a
// turn: 2.3e-8 radians, a quarter of what a whole turn's float loses.  sincospif gives its sine and
// cosine, and the quarter turns them.
//
// Bound by memory: every row is read and written once.  A thread owns eight pairs of one token:
// it forms their sines and cosines once, in registers, and applies them to every head of both
// tensors, two 16-byte loads and stores (bf16) a head, so the trigonometry is a 1/(H + Hk) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "decay.cuh"

namespace rehyat {
namespace rotary {

constexpr int kThreads = 128;
constexpr int kPairs = 8;   // pairs a thread turns
constexpr int kMaxAxes = 4;

struct Tensor {
  const void* x;
  void* y;
  long long xb, xh, xn, yb, yh, yn;  // strides in elements
  int heads;
};

struct Params {
  Tensor t[2];
  int B, n, D, R;
  int interleaved;
  int copy_tail;               // dimensions R .. D-1 are copied (out of place)
  const double* freq;          // [R/2] radians per position
  const unsigned char* axis;   // [R/2] or null (all 0)
  const void* pos;             // int32 or int64, or null
  int pos64, axes;
  long long pa, pb, pn;        // strides of pos: axis, sequence, token
  int add_index;               // position = pos + token index
  long long start;             // added to every position
  float scale;
  float sign;                  // -1: the gradient
  int heads_per_block;
};

// x modulo 1 in units of 2^-64, nearest: x - rint(x) is exact, and so is its product.
__device__ __forceinline__ unsigned long long fraction64(double x) {
  return static_cast<unsigned long long>(__double2ll_rn((x - rint(x)) * 18446744073709551616.0));
}
// freq / (2 pi) modulo one turn.  The constant and its product with freq are both sums of two doubles,
// good to 2^-105 of freq: a fraction's own 64 bits decide.
__device__ __forceinline__ unsigned long long turn_fraction(double freq) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double hi = freq * kHi, lo = fma(freq, kHi, -hi) + freq * kLo;
  return fraction64(hi) + fraction64(lo);
}
__device__ __forceinline__ long long position(const Params& p, int axis, int b, int i) {
  long long x = p.start + (p.add_index ? i : 0);
  if (p.pos) {
    const long long at = axis * p.pa + b * p.pb + i * p.pn;
    x += p.pos64 ? static_cast<const long long*>(p.pos)[at]
                 : (long long)static_cast<const int*>(p.pos)[at];
  }
  return x;
}
__device__ __forceinline__ void turn(const Params& p, int pair, int b, int i, float& c, float& s) {
  const int axis = p.axis ? min((int)p.axis[pair], p.axes - 1) : 0;
  const unsigned long long a = static_cast<unsigned long long>(position(p, axis, b, i)) *
                               turn_fraction(p.freq[pair]);
  const unsigned quarter = (unsigned)((a + (1ull << 61)) >> 62);
  // what is left, in [-1/8, 1/8] turns: its upper half, in units of 2^-31 half turns
  const int rest = (int)((a - ((unsigned long long)quarter << 62)) >> 32);
  float cr, sr;
  sincospif((float)rest * (1.f / 2147483648.f), &sr, &cr);
  c = quarter & 1 ? sr : cr;
  s = quarter & 1 ? cr : sr;
  if (quarter == 1 || quarter == 2) c = -c;
  if (quarter >= 2) s = -s;
  c *= p.scale;
  s *= p.scale * p.sign;
}

// Eight values of a row, as they lie in memory.
template <typename T>
struct Eight {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const;
  __device__ __forceinline__ void set(const float (&v)[8]);
};
template <>
__device__ __forceinline__ void Eight<float>::get(float (&v)[8]) const {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ void Eight<float>::set(const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    u[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                      __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
}
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::get(float (&v)[8]) const {
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::set(const float (&v)[8]) {
  using sm100::pack_bf16x2;
  u[0] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Heads [h0, h1) of the two tensors counted one after the other.
// grid (ceil(tokens * units / kThreads), head blocks), block kThreads.  A token has R/16 units of
// eight pairs and, out of place, (D - R)/16 units that copy sixteen dimensions.
// Needs R % 16 == 0, D % 16 == 0 and 16-byte aligned rows.
template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const Params p) {
  const int turning = p.R / 16, units = turning + (p.copy_tail ? (p.D - p.R) / 16 : 0);
  const long long g = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long token = g / units;
  const int u = (int)(g - token * units);
  if (token >= (long long)p.B * p.n) return;
  const int b = (int)(token / p.n), i = (int)(token - (long long)b * p.n);
  const bool turns = u < turning;
  float c[kPairs], s[kPairs];
  if (turns) {
#pragma unroll
    for (int k = 0; k < kPairs; ++k) turn(p, u * kPairs + k, b, i, c[k], s[k]);
  }
  const int d0 = turns ? (kInterleaved ? u * 16 : u * 8) : p.R + (u - turning) * 16;
  const int d1 = turns && !kInterleaved ? d0 + p.R / 2 : d0 + 8;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.t[0].heads + p.t[1].heads);
  // a batch of heads is loaded before any is stored (the output may be the input, so the compiler
  // would not move a load past a store): eight 16-byte loads of a thread in flight
  constexpr int kBatch = 8 / (int)sizeof(T);
  for (int hb = h0; hb < h1; hb += kBatch) {
    Eight<T> a[kBatch], z[kBatch];
    T* y[kBatch];
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      const int hh = hb + m, w = hh >= p.t[0].heads;
      const Tensor& t = p.t[w];
      const int h = hh - (w ? p.t[0].heads : 0);
      y[m] = static_cast<T*>(t.y) + b * t.yb + h * t.yh + i * t.yn;
      if (hh < h1) {
        const T* x = static_cast<const T*>(t.x) + b * t.xb + h * t.xh + i * t.xn;
        a[m].load(x + d0);
        z[m].load(x + d1);
      }
    }
#pragma unroll
    for (int m = 0; m < kBatch; ++m) {
      if (hb + m >= h1) break;
      if (turns) {
        float v0[8], v1[8], o0[8], o1[8];
        a[m].get(v0);
        z[m].get(v1);
        if (kInterleaved) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o0[2 * k] = v0[2 * k] * c[k] - v0[2 * k + 1] * s[k];
            o0[2 * k + 1] = v0[2 * k + 1] * c[k] + v0[2 * k] * s[k];
            o1[2 * k] = v1[2 * k] * c[4 + k] - v1[2 * k + 1] * s[4 + k];
            o1[2 * k + 1] = v1[2 * k + 1] * c[4 + k] + v1[2 * k] * s[4 + k];
          }
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            o0[k] = v0[k] * c[k] - v1[k] * s[k];
            o1[k] = v1[k] * c[k] + v0[k] * s[k];
          }
        }
        a[m].set(o0);
        z[m].set(o1);
      }
      a[m].store(y[m] + d0);
      z[m].store(y[m] + d1);
    }
  }
}

// The same for every even R, every D and strides that are not whole vectors: a thread turns one
// pair, or copies one dimension past R, of every head.
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_any_kernel(const Params p) {
  const int turning = p.R / 2, units = turning + (p.copy_tail ? p.D - p.R : 0);
  const long long g = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long token = g / units;
  const int u = (int)(g - token * units);
  if (token >= (long long)p.B * p.n) return;
  const int b = (int)(token / p.n), i = (int)(token - (long long)b * p.n);
  const bool turns = u < turning;
  float c = 0.f, s = 0.f;
  if (turns) turn(p, u, b, i, c, s);
  const int d0 = turns ? (p.interleaved ? 2 * u : u) : p.R + u - turning;
  const int d1 = turns ? (p.interleaved ? 2 * u + 1 : u + p.R / 2) : d0;
  const int h0 = blockIdx.y * p.heads_per_block;
  const int h1 = min(h0 + p.heads_per_block, p.t[0].heads + p.t[1].heads);
  for (int hh = h0; hh < h1; ++hh) {
    const int w = hh >= p.t[0].heads;
    const Tensor& t = p.t[w];
    const int h = hh - (w ? p.t[0].heads : 0);
    const T* x = static_cast<const T*>(t.x) + b * t.xb + h * t.xh + i * t.xn;
    T* y = static_cast<T*>(t.y) + b * t.yb + h * t.yh + i * t.yn;
    const float v0 = (float)x[d0], v1 = (float)x[d1];
    if (turns) {
      y[d0] = (T)(v0 * c - v1 * s);
      y[d1] = (T)(v1 * c + v0 * s);
    } else {
      y[d0] = x[d0];
    }
  }
}

}  // namespace rotary
}  // namespace rehyat
