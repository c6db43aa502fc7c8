// RMS norm of every head of the queries and keys with the position rotation
// in the same pass, its gradient, and the table of the rotation.
//
//   r = 1 / sqrt(mean_j x_j^2 + eps),  y_j = x_j r w_j   (w NULL: y = x)
//   pair p < R / 2 of the first R elements turns by the angle whose cosine
//   and sine are table[position of axis p / n][p mod n], n = R / (2 axes):
//   (y_a, y_b) -> (y_a c - y_b s, y_a s + y_b c), where (a, b) = (2p, 2p + 1)
//   (interleaved) or (p, p + R / 2).
// Gradient: g is the output's gradient turned back,
//   dw_j = sum over rows and heads of g_j x_j r,
//   dx_j = r (g_j w_j - x_j r^2 mean_i(g_i w_i x_i)).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"

namespace spconv {
namespace {

// Elements per lane: one 16-byte piece.
template <class T>
constexpr int kE = 16 / static_cast<int>(sizeof(T));

template <class T>
__device__ __forceinline__ void load_piece(const T* p, float (&v)[kE<T>]) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  const vec t = *reinterpret_cast<const vec*>(p);
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) v[u] = static_cast<float>(t[u]);
}
template <class T>
__device__ __forceinline__ void store_piece(T* p, const float (&v)[kE<T>]) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  vec t;
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) t[u] = static_cast<T>(v[u]);
  *reinterpret_cast<vec*>(p) = t;
}

// Sum over the LPR lanes of a row (an aligned power of two of them).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPR; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Cosine and sine of the angles that turn this lane's elements e0 .. e0 + E - 1
// (of each pair the lane's member).  A position outside the table turns by NaN.
template <class T>
__device__ __forceinline__ void load_turns(const NormRotaryArgs& a, int row, int e0, bool on, float (&c)[kE<T>],
                                           float (&s)[kE<T>]) {
  const int n = a.rotary / (2 * max(a.axes, 1)), half = a.rotary / 2;
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) {
    const int e = e0 + u;
    c[u] = 1.f;
    s[u] = 0.f;
    if (!on || e >= a.rotary) continue;
    const int p = a.interleaved ? e >> 1 : e < half ? e : e - half;
    const int axis = p / n;
    const int pos = a.positions[row * a.pos_row + axis];
    const bool in = static_cast<uint32_t>(pos) < static_cast<uint32_t>(a.extent);
    const float2 t = *reinterpret_cast<const float2*>(a.table + (static_cast<int64_t>(in ? pos : 0) * n + (p - axis * n)) * 2);
    c[u] = in ? t.x : __builtin_nanf("");
    s[u] = in ? t.y : __builtin_nanf("");
  }
}

// The turned elements; `sign` -1 turns back.  stage: the row's LDS (half
// layout only), where each lane finds its pairs' other members.
template <class T>
__device__ __forceinline__ void turn(const NormRotaryArgs& a, float* stage, int e0, float sign, float (&y)[kE<T>],
                                     const float (&c)[kE<T>], const float (&s)[kE<T>]) {
  constexpr int E = kE<T>;
  if (a.rotary == 0) return;
  if (a.interleaved) {
#pragma unroll
    for (int u = 0; u < E; u += 2) {
      const float x0 = y[u], x1 = y[u + 1];
      y[u] = x0 * c[u] - sign * x1 * s[u];
      y[u + 1] = sign * x0 * s[u] + x1 * c[u];
    }
    return;
  }
  const int half = a.rotary / 2;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < E; ++u) stage[e0 + u] = y[u];
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int u = 0; u < E; ++u) {
    const int e = e0 + u;
    if (e < a.rotary) {
      const float other = stage[e < half ? e + half : e - half];
      y[u] = y[u] * c[u] + (e < half ? -sign : sign) * other * s[u];
    }
  }
  __builtin_amdgcn_wave_barrier();
}

constexpr int kWaves = 4;

template <class T, int LPR>
__global__ __launch_bounds__(64 * kWaves) void k_norm_rotary(NormRotaryArgs a, int heads_per_block) {
  constexpr int E = kE<T>, RPW = 64 / LPR;
  __shared__ float stage[kWaves * 64 * E];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LPR, e0 = sub * E;
  const int row = (blockIdx.x * kWaves + wave) * RPW + lane / LPR;
  if (row >= a.rows) return;
  float* mine = stage + (wave * RPW + lane / LPR) * LPR * E;
  const bool on = e0 < a.dim;
  float c[E], s[E];
  load_turns<T>(a, row, e0, on, c, s);
  const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, a.t[0].heads + a.t[1].heads);
  for (int h = h0; h < h1; ++h) {
    const bool second = h >= a.t[0].heads;
    const NormRotaryTensor& t = a.t[second ? 1 : 0];
    const int head = second ? h - a.t[0].heads : h;
    float x[E] = {};
    if (on) load_piece<T>(static_cast<const T*>(t.x) + row * t.x_row + head * t.x_head + e0, x);
    if (t.weight != nullptr) {
      float sq = 0.f;
#pragma unroll
      for (int u = 0; u < E; ++u) sq = __builtin_fmaf(x[u], x[u], sq);
      const float r = 1.f / sqrtf(row_sum<LPR>(sq) / static_cast<float>(a.dim) + a.eps);
      float w[E] = {};
      if (on) load_piece<T>(static_cast<const T*>(t.weight) + e0, w);
#pragma unroll
      for (int u = 0; u < E; ++u) x[u] = x[u] * r * w[u];
    }
    turn<T>(a, mine, e0, 1.f, x, c, s);
    if (on) store_piece<T>(static_cast<T*>(t.y) + row * t.y_row + head * t.y_head + e0, x);
  }
}

// Partial weight gradients: [2][blocks][dim] fp32 sums, one per workgroup.
template <class T, int LPR>
__global__ __launch_bounds__(64 * kWaves) void k_norm_rotary_backward(NormRotaryArgs a, float* part) {
  constexpr int E = kE<T>, RPW = 64 / LPR;
  __shared__ float stage[kWaves * 64 * E];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane % LPR, e0 = sub * E;
  float* mine = stage + (wave * RPW + lane / LPR) * LPR * E;
  const bool on = e0 < a.dim;
  float dw[2][E] = {};
  const int step = gridDim.x * kWaves * RPW;
  const int rows_up = (a.rows + RPW - 1) / RPW * RPW;
  for (int row = (blockIdx.x * kWaves + wave) * RPW + lane / LPR; row < rows_up; row += step) {
    if (row >= a.rows) continue;
    float c[E], s[E];
    load_turns<T>(a, row, e0, on, c, s);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const NormRotaryTensor& t = a.t[k];
      for (int head = 0; head < t.heads; ++head) {
        float x[E] = {}, g[E] = {};
        if (on) {
          load_piece<T>(static_cast<const T*>(t.x) + row * t.x_row + head * t.x_head + e0, x);
          load_piece<T>(static_cast<const T*>(t.grad) + row * t.g_row + head * t.g_head + e0, g);
        }
        turn<T>(a, mine, e0, -1.f, g, c, s);
        if (t.weight != nullptr) {
          float w[E] = {}, sq = 0.f, gx = 0.f;
          if (on) load_piece<T>(static_cast<const T*>(t.weight) + e0, w);
#pragma unroll
          for (int u = 0; u < E; ++u) sq = __builtin_fmaf(x[u], x[u], sq);
          const float r = 1.f / sqrtf(row_sum<LPR>(sq) / static_cast<float>(a.dim) + a.eps);
#pragma unroll
          for (int u = 0; u < E; ++u) {
            dw[k][u] = __builtin_fmaf(g[u] * x[u], r, dw[k][u]);
            g[u] *= w[u];
            gx = __builtin_fmaf(g[u], x[u], gx);
          }
          const float m = row_sum<LPR>(gx) / static_cast<float>(a.dim) * r * r;
#pragma unroll
          for (int u = 0; u < E; ++u) g[u] = r * (g[u] - x[u] * m);
        }
        if (on) store_piece<T>(static_cast<T*>(t.grad_x) + row * t.gx_row + head * t.gx_head + e0, g);
      }
    }
  }
  // The workgroup's sums, in a fixed order: over the rows of a wave, then over the waves.
  for (int k = 0; k < 2; ++k) {
    if (a.t[k].weight == nullptr || a.t[k].heads == 0) continue;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < E; ++u) mine[e0 + u] = dw[k][u];
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += 64 * kWaves) {
      float sum = 0.f;
      for (int q = 0; q < kWaves * RPW; ++q) sum += stage[q * LPR * E + d];
      part[(static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * a.dim + d] = sum;
    }
  }
}

// dw[d] = sum over the blocks' partial sums, in a fixed order.
__global__ __launch_bounds__(256) void k_norm_weight_sum(const float* part, int blocks, int dim, float* dq, float* dk) {
  __shared__ float stage[256];
  const int d = blockIdx.x;
  float* dst = blockIdx.y ? dk : dq;
  if (dst == nullptr) return;
  const float* src = part + static_cast<int64_t>(blockIdx.y) * blocks * dim + d;
  float sum = 0.f;
  for (int b = threadIdx.x; b < blocks; b += 256) sum += src[static_cast<int64_t>(b) * dim];
  stage[threadIdx.x] = sum;
  __syncthreads();
  for (int w = 128; w > 0; w /= 2) {
    if (static_cast<int>(threadIdx.x) < w) stage[threadIdx.x] += stage[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) dst[d] = stage[0];
}

__global__ __launch_bounds__(256) void k_rotary_table(float* table, int extent, int pairs, double base, double scale) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (id >= static_cast<int64_t>(extent) * pairs) return;
  const int i = static_cast<int>(id % pairs);
  const double angle = static_cast<double>(id / pairs) * scale * pow(base, -static_cast<double>(i) / pairs);
  table[2 * id] = static_cast<float>(cos(angle));
  table[2 * id + 1] = static_cast<float>(sin(angle));
}

int backward_blocks(const NormRotaryArgs& a, int rows_per_block) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((a.rows + rows_per_block - 1) / rows_per_block, 1024)));
}

int lanes_per_row(const NormRotaryArgs& a) {
  const int pieces = a.dim * (a.dtype == 0 ? 4 : 2) / 16;
  int l = 1;
  while (l < pieces) l *= 2;
  return l;
}

template <class F>
hipError_t dispatch(const NormRotaryArgs& a, F&& f) {
  auto by_lanes = [&](auto t) -> hipError_t {
    switch (lanes_per_row(a)) {  // dim is at most 128
      case 1: return f(t, std::integral_constant<int, 1>{});
      case 2: return f(t, std::integral_constant<int, 2>{});
      case 4: return f(t, std::integral_constant<int, 4>{});
      case 8: return f(t, std::integral_constant<int, 8>{});
      case 32:
        if constexpr (sizeof(t) == 4) return f(t, std::integral_constant<int, 32>{});
        break;
      default: break;
    }
    return f(t, std::integral_constant<int, 16>{});
  };
  if (a.dtype == 0) return by_lanes(0.f);
  if (a.dtype == 1) return by_lanes(static_cast<_Float16>(0));
  return by_lanes(static_cast<__bf16>(0.f));
}

}  // namespace

hipError_t launch_norm_rotary(const NormRotaryArgs& a, hipStream_t stream) {
  const int heads = a.t[0].heads + a.t[1].heads;
  if (a.rows == 0 || heads == 0) return hipSuccess;
  return dispatch(a, [&](auto t, auto lanes) -> hipError_t {
    typedef decltype(t) T;
    constexpr int LPR = decltype(lanes)::value, rows = kWaves * 64 / LPR;
    const int64_t blocks = (a.rows + rows - 1) / rows;
    // heads share a row's turns; few rows spread their heads over workgroups
    int hpb = heads;
    while (hpb > 1 && blocks * ((heads + hpb - 1) / hpb) < 512) hpb = (hpb + 1) / 2;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + hpb - 1) / hpb));
    k_norm_rotary<T, LPR><<<grid, 64 * kWaves, 0, stream>>>(a, hpb);
    return hipGetLastError();
  });
}

size_t norm_rotary_backward_workspace_bytes(const NormRotaryArgs& a) {
  return static_cast<size_t>(2) * 1024 * a.dim * sizeof(float);
}

hipError_t launch_norm_rotary_backward(const NormRotaryArgs& a, void* workspace, hipStream_t stream) {
  const int heads = a.t[0].heads + a.t[1].heads;
  if (heads == 0) return hipSuccess;
  return dispatch(a, [&](auto t, auto lanes) -> hipError_t {
    typedef decltype(t) T;
    constexpr int LPR = decltype(lanes)::value, rows = kWaves * 64 / LPR;
    const int blocks = backward_blocks(a, rows);
    float* part = static_cast<float*>(workspace);
    k_norm_rotary_backward<T, LPR><<<blocks, 64 * kWaves, 0, stream>>>(a, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float* dq = a.t[0].heads > 0 && a.t[0].weight != nullptr ? a.t[0].grad_weight : nullptr;
    float* dk = a.t[1].heads > 0 && a.t[1].weight != nullptr ? a.t[1].grad_weight : nullptr;
    if (dq == nullptr && dk == nullptr) return hipSuccess;
    k_norm_weight_sum<<<dim3(a.dim, 2), 256, 0, stream>>>(part, blocks, a.dim, dq, dk);
    return hipGetLastError();
  });
}

hipError_t launch_rotary_table(float* table, int32_t extent, int32_t pairs, double base, double scale,
                               hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(extent) * pairs;
  if (n == 0) return hipSuccess;
  k_rotary_table<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(table, extent, pairs, base, scale);
  return hipGetLastError();
}

}  // namespace spconv
