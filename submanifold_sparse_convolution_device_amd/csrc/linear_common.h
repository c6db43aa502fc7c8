// Shared device code of the row products (linear_kernels.h, linear.hip):
// groups of rows, activations and the epilogue of 8 columns.
#pragma once

#include <hip/hip_runtime.h>

#include "attention_common.h"
#include "internal.h"

namespace spconv {
namespace lin {

// ---- Groups of packed rows ----
// Group e holds the rows [cu[e], cu[e + 1]).  The offsets cut all rows into
// segments: 0 (before the first offset) and groups + 1 (after the last) belong
// to no group, segment s to group s - 1.  Offsets are clamped to the rows
// there are, so no access leaves the tensors whatever they hold.
//
// Segment s starts at slot floor(bound(s) / unit) + s, which leaves it at least
// ceil(rows / unit) slots and at least one, with no pass over the lengths
// before: a grid of rows / unit + groups + 2 workgroups covers every segment.
__device__ __forceinline__ int segment_start(const ProductArgs& a, int s) {
  return fast_div(attn::bound(a.cu, a.groups, a.rows, s), a.by_unit) + s;
}

struct Segment {
  int seg;
  int group;   // -1: rows of no group
  int lo, hi;  // this slot's rows
  bool first;  // the segment's first slot
};

// The rows of a slot (all lanes of a wavefront call it together).  The search
// narrows 64-fold a round: one round of loads up to 62 groups.
__device__ __forceinline__ Segment find_segment(const ProductArgs& a, int slot) {
  Segment g;
  const int unit = a.by_unit.d;
  if (a.cu == nullptr) {
    g.seg = g.group = 0;
    g.lo = slot * unit;
    g.hi = min(a.rows, g.lo + min(unit, a.rows));
    g.first = slot == 0;
    return g;
  }
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.groups + 2;
  while (hi - lo > 1) {
    const int step = (hi - lo + 63) >> 6;
    const int at = lo + lane * step;
    const bool before = at < hi && segment_start(a, at) <= slot;
    const int c = max(static_cast<int>(__builtin_popcountll(__ballot(before))), 1);
    lo += (c - 1) * step;
    hi = min(lo + step, hi);
  }
  const int s = __builtin_amdgcn_readfirstlane(lo);
  const int r0 = attn::bound(a.cu, a.groups, a.rows, s), r1 = attn::bound(a.cu, a.groups, a.rows, s + 1);
  const int64_t nth = max(slot - (fast_div(r0, a.by_unit) + s), 0);  // (below 0 with decreasing offsets alone)
  const int64_t from = r0 + nth * unit;
  g.seg = s;
  g.group = s == 0 || s == a.groups + 1 ? -1 : s - 1;
  g.lo = static_cast<int>(min(from, static_cast<int64_t>(max(r1, r0))));
  g.hi = static_cast<int>(min(from + unit, static_cast<int64_t>(max(r1, r0))));
  g.first = nth == 0;
  return g;
}

// ---- Workgroup shapes of the tiled products ----
// BM x BN tiles by WR x WC wavefronts, BK contracted values a step.
// STAGES: LDS buffers.
template <int BM_, int BN_, int WR_, int WC_, int BK_, int STAGES_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WR = WR_, WC = WC_, BK = BK_, STAGES = STAGES_;
  static constexpr int NT = 64 * WR * WC, TM = BM / WR, TN = BN / WC;
};
// Narrow: few columns, or too few tiles to fill the chip; Half (f32): 64
// columns a tile for up to as many, and by rows also in Narrow's place where
// its tiles fill the CUs twice or the contraction is long; Medium; Large:
// whole large products.
template <class T>
struct Shapes;
template <class T>
struct Shapes16 {
  typedef Shape<128, 64, 4, 1, 64, 2> Narrow;
  typedef Narrow Half;
  typedef Shape<128, 128, 2, 2, 64, 2> Medium;
  typedef Shape<256, 256, 2, 4, 64, 2> Large;
};
template <>
struct Shapes<float> {
  typedef Shape<128, 32, 4, 1, 32, 1> Narrow;
  typedef Shape<128, 64, 4, 1, 32, 1> Half;
  typedef Shape<128, 128, 2, 2, 32, 1> Medium;
  typedef Medium Large;
};
template <>
struct Shapes<_Float16> : Shapes16<_Float16> {};
template <>
struct Shapes<__bf16> : Shapes16<__bf16> {};

// ---- Activations ----
enum Act { kIdentity = 0, kRelu = 1, kSilu = 2, kGelu = 3 };

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + attn::fast_exp2(z * -attn::kLog2e));
}

// The normal distribution's lower tail at -a, a >= 0, as t (c1 + c2 t + ...
// + c6 t^5) e with t = 1 / (1 + 0.31 a) and e = exp(-a^2 / 2).  The
// coefficients are a fit to erfcx of the smallest relative error, 4.7e-6 for
// a up to 13.5: a hundredth of fp16's rounding, a 400th of bf16's.  (One
// coefficient fewer leaves 2.9e-5.)
__device__ __forceinline__ float tail(float a, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, a, 1.f));
  float p = -0.073935856f;
  p = __builtin_fmaf(p, t, 0.180469782f);
  p = __builtin_fmaf(p, t, 0.0157236098f);
  p = __builtin_fmaf(p, t, 0.133440446f);
  p = __builtin_fmaf(p, t, 0.120438788f);
  p = __builtin_fmaf(p, t, 0.123860916f);
  return p * t * e;
}

// act(z) and its derivative, of N values with one branch.  fp32 takes the
// library's functions, whose errors are of fp32's size relative to the value:
// erfc, as 1 + erf loses the lower tail, all of it from z = -5.6 (100,003 rows
// 128 -> 256 with gelu 87 us, by erf 75).  What the argument's rounding makes
// of the tail, z^2 / 2^24 of it, a rounding of z makes too.  16-bit types take
// the unit's exponential and reciprocal.  An infinite z gives the limit, as a
// stored product past fp16's range needs it: a factor z beside one that is 0
// there is held finite, and a NaN stays one through the other.
__device__ __forceinline__ float held(float z) { return __builtin_amdgcn_fmed3f(z, -1e30f, 1e30f); }
// z from `low` up; an infinity stays one, as a residual is added to it.  In one
// instruction: a maximum takes two, the first for NaN, and the compiler makes
// one of a median with an infinity that it sees (400,000 rows 256 -> 1024 with
// gelu: 441 us, hidden 428).
__device__ __forceinline__ float from(float low, float z) {
  float top = __builtin_inff();
  asm("" : "+s"(top));
  return __builtin_amdgcn_fmed3f(z, low, top);
}

template <class T>
__device__ __forceinline__ float relu(float z) {
  return z <= 0.f ? 0.f : z;  // (a NaN stays)
}
template <class T>
__device__ __forceinline__ float silu(float z) {
  // (to -inf the value is -0; held on that side alone)
  if constexpr (sizeof(T) == 4) return fmaxf(z, -1e30f) / (1.f + expf(-z));
  return from(-1e30f, z) * sigmoid(z);
}
template <class T>
__device__ __forceinline__ float gelu(float z) {
  if constexpr (sizeof(T) == 4) return 0.5f * fmaxf(z, -1e30f) * erfcf(z * -0.70710678f);
  // z - z t above 0, z t below (a NaN comes from the second part)
  return from(0.f, z) - __builtin_amdgcn_fmed3f(fabsf(z), 0.f, 1e30f) * tail(fabsf(z), attn::fast_exp2(z * (z * (-0.5f * attn::kLog2e))));
}
template <class T>
__device__ __forceinline__ float silu_slope(float z) {
  const float s = sizeof(T) == 4 ? 1.f / (1.f + expf(-z)) : sigmoid(z);
  return s * (1.f + held(z) * (1.f - s));
}
template <class T>
__device__ __forceinline__ float gelu_slope(float z) {
  constexpr float inv_root = 0.3989422804014327f;  // 1 / sqrt(2 pi)
  if constexpr (sizeof(T) == 4) return 0.5f * erfcf(z * -0.70710678f) + held(z) * inv_root * expf(-0.5f * z * z);
  const float e = attn::fast_exp2(z * (z * (-0.5f * attn::kLog2e)));
  const float t = tail(fabsf(z), e);
  return (z < 0.f ? t : 1.f - t) + held(z) * inv_root * e;
}
// f(i) for i < N, 4 at a time: the registers of all N together do not fit.
template <int N, class F>
__device__ __forceinline__ void by_fours(F&& f) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    f(i);
    if (i % 4 == 3) __builtin_amdgcn_sched_barrier(0);
  }
}
template <class T, int N>
__device__ __forceinline__ void activate(int act, float (&v)[N]) {
  if (act == kRelu) {
    by_fours<N>([&](int i) { v[i] = relu<T>(v[i]); });
  } else if (act == kSilu) {
    by_fours<N>([&](int i) { v[i] = silu<T>(v[i]); });
  } else if (act == kGelu) {
    by_fours<N>([&](int i) { v[i] = gelu<T>(v[i]); });
  }
}
// v times the slope at z(i).
template <class T, int N, class Z>
__device__ __forceinline__ void times_slope(int act, Z&& z, float (&v)[N]) {
  if (act == kRelu) {
    by_fours<N>([&](int i) { v[i] *= z(i) > 0.f ? 1.f : 0.f; });
  } else if (act == kSilu) {
    by_fours<N>([&](int i) { v[i] *= silu_slope<T>(z(i)); });
  } else if (act == kGelu) {
    by_fours<N>([&](int i) { v[i] *= gelu_slope<T>(z(i)); });
  }
}

// ---- 8 columns of a row ----
template <class T>
__device__ __forceinline__ void unpack8(const attn::Raw<T>& r, float (&v)[8]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(__builtin_bit_cast(vec, r.v[i / E])[i % E]);
}
template <class T>
__device__ __forceinline__ float element(const attn::Raw<T>& r, int i) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(E)));
  return static_cast<float>(__builtin_bit_cast(vec, r.v[i / E])[i % E]);
}
// 16-byte accesses (p is aligned).
template <class T>
__device__ __forceinline__ attn::Raw<T> load_raw8(const T* p) {
  return attn::load_piece<T>(p, true);
}
template <class T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
  for (int i = 0; i < 8; i += E) {
    vec x;
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = static_cast<T>(v[i + j]);
    *reinterpret_cast<uint4*>(p + i) = __builtin_bit_cast(uint4, x);
  }
}
// A piece whose first `cols` values exist (whole 16 bytes of them), zeros for
// the others and for a row that does not (on).
template <class T>
__device__ __forceinline__ attn::Raw<T> load_piece_of(const T* p, bool on, int cols) {
  attn::Raw<T> r;
#pragma unroll
  for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h)
    r.v[h] = on && 4 * h < cols ? reinterpret_cast<const uint4*>(p)[h] : make_uint4(0, 0, 0, 0);
  return r;
}
// The first `there` of 8, one by one unless all are there and aligned.
template <class T>
__device__ __forceinline__ void load_some8(const T* p, int there, bool whole, float (&v)[8]) {
  if (whole) {
    unpack8<T>(load_raw8<T>(p), v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < there ? static_cast<float>(p[i]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void store_some8(T* p, int there, bool whole, const float (&v)[8]) {
  if (whole) {
    store8<T>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < there) p[i] = static_cast<T>(v[i]);
  }
}

// The sums (with the bias) of N values of a row or of several to the output,
// in fp32 until each output is rounded once.  By rows: the stored product
// (pre), activation, residual; by rows T: times the slope of the activation
// before.  side(i) is the residual's or before's value.  Rows of no group come
// with sums of zero.
template <class T, int FORM, int N, class Side, class Store>
__device__ __forceinline__ void finish(const ProductArgs& a, bool in_group, bool sides, Side&& side, float (&v)[N], Store&& store) {
  if constexpr (FORM == kByRows) {
    if (a.pre != nullptr) store(static_cast<T*>(a.pre), a.pre_row, v);
    if (in_group) {
      activate<T, N>(a.act, v);
      if (sides) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += side(i);
      }
    }
  } else {
    if (sides) times_slope<T, N>(a.act, side, v);
  }
  store(static_cast<T*>(a.out), a.out_row, v);
}

// Where a row's part of `side` begins.
template <class T>
__device__ __forceinline__ const T* side_row(const ProductArgs& a, int64_t row) {
  return static_cast<const T*>(a.side) + row * a.side_row;
}

}  // namespace lin
}  // namespace spconv
