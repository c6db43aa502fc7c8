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
    g.group = 0;
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
  const int64_t nth = slot - (fast_div(r0, a.by_unit) + s);
  const int64_t from = r0 + nth * unit;
  g.group = s == 0 || s == a.groups + 1 ? -1 : s - 1;
  g.lo = static_cast<int>(min(from, static_cast<int64_t>(max(r1, r0))));
  g.hi = static_cast<int>(min(from + unit, static_cast<int64_t>(max(r1, r0))));
  g.first = nth == 0;
  return g;
}

// ---- Activations ----
enum Act { kIdentity = 0, kRelu = 1, kSilu = 2, kGelu = 3 };

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + attn::fast_exp2(z * -attn::kLog2e));
}

// The normal distribution's lower tail at -a, a >= 0, as t (c1 + c2 t + ...
// + c6 t^5) e with t = 1 / (1 + 0.3 a) and e = exp(-a^2 / 2).  The
// coefficients are a fit to erfcx of the smallest relative error, 7.6e-6 for
// a up to 13.5: a 64th of fp16's rounding, a 500th of bf16's.
__device__ __forceinline__ float tail(float a, float e) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.f));
  float p = -0.07751068f;
  p = __builtin_fmaf(p, t, 0.21727989f);
  p = __builtin_fmaf(p, t, -0.01836866f);
  p = __builtin_fmaf(p, t, 0.14496221f);
  p = __builtin_fmaf(p, t, 0.1135486f);
  p = __builtin_fmaf(p, t, 0.12009241f);
  return p * t * e;
}

// act(z) and its derivative.  fp32 takes the library's functions, whose errors
// are of fp32's size; 16-bit types the unit's exponential and reciprocal.
template <class T>
__device__ __forceinline__ float activate(int act, float z) {
  if (act == kRelu) return z <= 0.f ? 0.f : z;  // (a NaN stays)
  if (act == kSilu) {
    if constexpr (sizeof(T) == 4) return z / (1.f + expf(-z));
    return z * sigmoid(z);
  }
  if (act == kGelu) {
    if constexpr (sizeof(T) == 4) return 0.5f * z * (1.f + erff(z * 0.70710678f));
    const float t = tail(fabsf(z), attn::fast_exp2(z * z * (-0.5f * attn::kLog2e)));
    return z * (z < 0.f ? t : 1.f - t);
  }
  return z;
}
template <class T>
__device__ __forceinline__ float slope(int act, float z) {
  if (act == kRelu) return z > 0.f ? 1.f : 0.f;
  if (act == kSilu) {
    float s;
    if constexpr (sizeof(T) == 4) {
      s = 1.f / (1.f + expf(-z));
    } else {
      s = sigmoid(z);
    }
    return s * (1.f + z * (1.f - s));
  }
  if (act == kGelu) {
    constexpr float inv_root = 0.3989422804014327f;  // 1 / sqrt(2 pi)
    if constexpr (sizeof(T) == 4) return 0.5f * (1.f + erff(z * 0.70710678f)) + z * inv_root * expf(-0.5f * z * z);
    const float e = attn::fast_exp2(z * z * (-0.5f * attn::kLog2e));
    const float t = tail(fabsf(z), e);
    return (z < 0.f ? t : 1.f - t) + z * inv_root * e;
  }
  return 1.f;
}

// ---- 8 columns of a row ----
// `there` of them exist; wide: all do and the address is 16-byte aligned.
template <class T>
__device__ __forceinline__ void load8(const T* p, int there, bool wide, float (&v)[8]) {
  if (wide && there == 8) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      const vec x = __builtin_bit_cast(vec, *reinterpret_cast<const uint4*>(p + i));
#pragma unroll
      for (int j = 0; j < E; ++j) v[i + j] = static_cast<float>(x[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < there ? static_cast<float>(p[i]) : 0.f;
  }
}
template <class T>
__device__ __forceinline__ void unpack8(const attn::Raw<T>& r, float (&v)[8]) {
  constexpr int E = 16 / static_cast<int>(sizeof(T));
  typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(__builtin_bit_cast(vec, r.v[i / E])[i % E]);
}
template <class T>
__device__ __forceinline__ void store8(T* p, int there, bool wide, const float (&v)[8]) {
  if (wide && there == 8) {
    constexpr int E = 16 / static_cast<int>(sizeof(T));
    typedef T vec __attribute__((ext_vector_type(E)));
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      vec x;
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = static_cast<T>(v[i + j]);
      *reinterpret_cast<uint4*>(p + i) = __builtin_bit_cast(uint4, x);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < there) p[i] = static_cast<T>(v[i]);
  }
}

// The sums of 8 columns to the output: bias, the stored product (pre),
// activation or the slope of the activation before, residual; fp32 until here,
// each output rounded once.
template <class T>
__device__ __forceinline__ void finish8(const ProductArgs& a, int64_t row, int col, int there, bool in_group, const float (&bias)[8], float (&v)[8]) {
  if (!in_group) {  // rows of no group
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    if (a.pre != nullptr) store8<T>(static_cast<T*>(a.pre) + row * a.pre_row + col, there, a.wide & kWidePre, v);
    store8<T>(static_cast<T*>(a.out) + row * a.out_row + col, there, a.wide & kWideOut, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  if (a.pre != nullptr) store8<T>(static_cast<T*>(a.pre) + row * a.pre_row + col, there, a.wide & kWidePre, v);
  if (a.before != nullptr) {
    float z[8];
    load8<T>(static_cast<const T*>(a.before) + row * a.before_row + col, there, a.wide & kWideBefore, z);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= slope<T>(a.act, z[i]);
  } else if (a.act != kIdentity) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = activate<T>(a.act, v[i]);
  }
  if (a.residual != nullptr) {
    float r[8];
    load8<T>(static_cast<const T*>(a.residual) + row * a.residual_row + col, there, a.wide & kWideResidual, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += r[i];
  }
  store8<T>(static_cast<T*>(a.out) + row * a.out_row + col, there, a.wide & kWideOut, v);
}

}  // namespace lin
}  // namespace spconv
