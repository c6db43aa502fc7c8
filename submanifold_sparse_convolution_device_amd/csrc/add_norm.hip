// The residual's addition and the RMS norm of whole rows in one pass, and its
// gradient.
//
//   h = x + residual (rounded to the type, as it is stored),
//   r = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j r w_j
// Gradient, g the gradient of y and d that of h (from what else reads h):
//   dw_j = sum over rows of g_j h_j r,
//   dx_j = d_j + r (g_j w_j - h_j r^2 mean_i(g_i w_i h_i)),
// the same for x and for the residual.
//
// Bound by HBM: every value is read once and written once, a row stays in
// registers between its sum and its use.  A row is LANES lanes of P pieces of
// 16 bytes each, a power of two of lanes so that a wavefront's rows follow one
// another; rows longer than a wavefront's registers go by workgroups, whose
// wavefronts add their sums in LDS.  24,001 rows of 4096 in bf16: 130 us (6.0
// TB/s), their gradient 149 (5.3 TB/s); 800,000 rows of 256: 283 us (5.8 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"

namespace spconv {
namespace {

template <class T>
constexpr int kE = 16 / static_cast<int>(sizeof(T));  // elements of a piece

template <class T>
__device__ __forceinline__ void unpack(uint4 p, float* v) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  const vec t = __builtin_bit_cast(vec, p);
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) v[u] = static_cast<float>(t[u]);
}
template <class T>
__device__ __forceinline__ uint4 pack(const float* v) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  vec t;
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) t[u] = static_cast<T>(v[u]);
  return __builtin_bit_cast(uint4, t);
}

constexpr int kThreads = 256;

// Sum over the lanes of a row; `turn` alternates the LDS of consecutive sums.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float (&lds)[2][4], int turn) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) v += __shfl_xor(v, d);
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = v;
    __syncthreads();
    v = (lds[turn][0] + lds[turn][1]) + (lds[turn][2] + lds[turn][3]);
  }
  return v;
}

// 1 / sqrt(mean + eps) of a row's sum of squares.  The unit's reciprocal root
// is off by up to a unit of 2^-23, a root and a division by two roundings; the
// step of Newton's method with its remainder in twice the precision leaves
// one.  (r is a factor of a whole row: its error does not average out in what
// sums over the row.)  Zeros, infinities and values below the normal range
// have no remainder to work with.
__device__ __forceinline__ float row_scale(float sq, const AddNormArgs& a) {
  const float x = sq / static_cast<float>(a.channels) + a.eps;
  if (!(x >= 1e-37f && x < 1e37f)) return 1.f / sqrtf(x);
  const float r = __builtin_amdgcn_rsqf(x);
  const float p = x * r, rest = __builtin_fmaf(x, r, -p);  // x r = p + rest
  const float e = __builtin_fmaf(-p, r, 1.f) - rest * r;   // 1 - x r^2
  return __builtin_fmaf(0.5f * r, e, r);
}

template <class T, int LANES, int P>
__global__ __launch_bounds__(kThreads) void k_add_norm(AddNormArgs a) {
  constexpr int E = kE<T>, RPB = kThreads / LANES;
  __shared__ float sums[2][4];
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + threadIdx.x / LANES;
  const bool there = row < a.rows;
  uint4 xr[P], rr[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = (i * LANES + lane) * E;
    xr[i] = rr[i] = make_uint4(0, 0, 0, 0);
    if (there && e < a.channels) {
      xr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + row * a.x_row + e);
      if (a.residual != nullptr) rr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.residual) + row * a.residual_row + e);
    }
  }
  float h[P][E], sq = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    unpack<T>(xr[i], h[i]);
    if (a.residual != nullptr) {
      float r[E];
      unpack<T>(rr[i], r);
#pragma unroll
      for (int u = 0; u < E; ++u) h[i][u] += r[u];
      const uint4 stored = pack<T>(h[i]);  // the norm is of the sum as it is stored
      unpack<T>(stored, h[i]);
      const int e = (i * LANES + lane) * E;
      if (there && e < a.channels) *reinterpret_cast<uint4*>(static_cast<T*>(a.h) + row * a.h_row + e) = stored;
    }
#pragma unroll
    for (int u = 0; u < E; ++u) sq = __builtin_fmaf(h[i][u], h[i][u], sq);
  }
  const float r = row_scale(row_sum<LANES>(sq, sums, 0), a);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = (i * LANES + lane) * E;
    if (!there || e >= a.channels) continue;
    float w[E];
    unpack<T>(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.weight) + e), w);
#pragma unroll
    for (int u = 0; u < E; ++u) h[i][u] = h[i][u] * r * w[u];
    *reinterpret_cast<uint4*>(static_cast<T*>(a.y) + row * a.y_row + e) = pack<T>(h[i]);
  }
}

// The gradient: a workgroup walks the rows by the grid's step and keeps its
// sums of the weight's gradient in registers; part[block][channels] takes
// them, the block's rows in a fixed order.
template <class T, int LANES, int P>
__global__ __launch_bounds__(kThreads) void k_add_norm_backward(AddNormArgs a, float* part) {
  constexpr int E = kE<T>, RPB = kThreads / LANES;
  __shared__ float sums[2][4];
  __shared__ float stage[LANES < kThreads ? kThreads * P * E : 1];
  const int lane = threadIdx.x % LANES;
  float w[P][E], dw[P][E] = {};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = (i * LANES + lane) * E;
    unpack<T>(e < a.channels ? *reinterpret_cast<const uint4*>(static_cast<const T*>(a.weight) + e) : make_uint4(0, 0, 0, 0), w[i]);
  }
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPB; base < a.rows; base += static_cast<int64_t>(gridDim.x) * RPB) {
    const int64_t row = base + threadIdx.x / LANES;
    const bool there = row < a.rows;
    uint4 hr[P], gr[P], dr[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = (i * LANES + lane) * E;
      hr[i] = gr[i] = dr[i] = make_uint4(0, 0, 0, 0);
      if (there && e < a.channels) {
        hr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.h) + row * a.h_row + e);
        gr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.grad_y) + row * a.grad_y_row + e);
        if (a.grad_h != nullptr) dr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.grad_h) + row * a.grad_h_row + e);
      }
    }
    float sq = 0.f, th = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float h[E], g[E];
      unpack<T>(hr[i], h);
      unpack<T>(gr[i], g);
#pragma unroll
      for (int u = 0; u < E; ++u) {
        sq = __builtin_fmaf(h[u], h[u], sq);
        th = __builtin_fmaf(g[u] * w[i][u], h[u], th);
      }
    }
    sq = row_sum<LANES>(sq, sums, turn);
    if constexpr (LANES > 64) turn ^= 1;
    th = row_sum<LANES>(th, sums, turn);
    if constexpr (LANES > 64) turn ^= 1;
    const float r = row_scale(sq, a);
    const float m = th / static_cast<float>(a.channels) * r * r;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = (i * LANES + lane) * E;
      float h[E], g[E], d[E];
      unpack<T>(hr[i], h);
      unpack<T>(gr[i], g);
      unpack<T>(dr[i], d);
#pragma unroll
      for (int u = 0; u < E; ++u) {
        dw[i][u] = there ? __builtin_fmaf(g[u] * h[u], r, dw[i][u]) : dw[i][u];
        d[u] += r * (g[u] * w[i][u] - h[u] * m);
      }
      if (there && e < a.channels) *reinterpret_cast<uint4*>(static_cast<T*>(a.grad) + row * a.grad_row + e) = pack<T>(d);
    }
  }
  if (a.grad_weight == nullptr) return;
  float* dst = part + static_cast<int64_t>(blockIdx.x) * a.channels;
  if constexpr (LANES == kThreads) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int e = (i * LANES + lane) * E;
      if (e >= a.channels) continue;
#pragma unroll
      for (int u = 0; u < E; u += 4) *reinterpret_cast<float4*>(dst + e + u) = make_float4(dw[i][u], dw[i][u + 1], dw[i][u + 2], dw[i][u + 3]);
    }
  } else {
    constexpr int COLS = LANES * P * E;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int u = 0; u < E; ++u) stage[(threadIdx.x / LANES) * COLS + (i * LANES + lane) * E + u] = dw[i][u];
    __syncthreads();
    for (int c = threadIdx.x; c < a.channels; c += kThreads) {
      double v = 0;
#pragma unroll 8
      for (int q = 0; q < RPB; ++q) v += stage[q * COLS + c];
      dst[c] = static_cast<float>(v);
    }
  }
}

// dw[c] = sum over the blocks' partial sums, in a fixed order: 32 columns by
// 32 shares of the blocks a workgroup.  In 64 bits, as the sums of a block's
// rows above: in fp32 these chains, whose sums are the largest, left more than
// all additions before (100,003 rows of 96 in f32: 1.7e-7 of the gradient's
// norm, 0.8e-7 so).
__global__ __launch_bounds__(1024) void k_add_norm_weight_sum(const float* part, int blocks, int channels, float* dw) {
  __shared__ double stage[32][33];
  const int x = threadIdx.x & 31, q = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  double v = 0;
  if (c < channels) {
#pragma unroll 8
    for (int b = q; b < blocks; b += 32) v += part[static_cast<int64_t>(b) * channels + c];
  }
  stage[q][x] = v;
  __syncthreads();
  if (q == 0 && c < channels) {
    double sum = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += stage[i][x];
    dw[c] = static_cast<float>(sum);
  }
}

// Calls f(type, lanes of a row, pieces of a lane): up to 4 pieces a lane (8
// for the longest rows, of 32 KB), the fewest lanes that hold the row (from 8,
// so that a row's access is 128 bytes).
template <class F>
hipError_t dispatch(const AddNormArgs& a, F&& f) {
  auto by_size = [&](auto t) -> hipError_t {
    const int pieces = a.channels / kE<decltype(t)>;
    auto by_pieces = [&](auto lanes) -> hipError_t {
      constexpr int L = decltype(lanes)::value;
      if (pieces <= L) return f(t, lanes, std::integral_constant<int, 1>{});
      if (pieces <= 2 * L) return f(t, lanes, std::integral_constant<int, 2>{});
      if constexpr (L == 256) {
        if (pieces > 4 * L) return f(t, lanes, std::integral_constant<int, 8>{});
      }
      return f(t, lanes, std::integral_constant<int, 4>{});
    };
    if (pieces <= 16) return by_pieces(std::integral_constant<int, 8>{});
    if (pieces <= 32) return by_pieces(std::integral_constant<int, 16>{});
    if (pieces <= 256) return by_pieces(std::integral_constant<int, 64>{});
    return by_pieces(std::integral_constant<int, 256>{});
  };
  if (a.dtype == 0) return by_size(0.f);
  if (a.dtype == 1) return by_size(static_cast<_Float16>(0));
  return by_size(static_cast<__bf16>(0.f));
}

// Workgroups of the gradient: two for each CU, whose loads keep the memory
// busy, where a lane has two pieces or more of each tensor, else four (24,001
// rows of 4096 in bf16: 149 us with 512, 168 with 1024, 172 with 2048;
// 3,000,000 rows of 32 in f16: 212, 153, 183).
constexpr int64_t kBackwardBlocks = 1024;
constexpr int64_t backward_blocks(int pieces) { return pieces > 1 ? 512 : kBackwardBlocks; }

}  // namespace

uint64_t add_norm_work_items(const AddNormArgs& a) {
  uint64_t items = 0;
  (void)dispatch(a, [&](auto, auto lanes, auto) -> hipError_t {
    constexpr int rpb = kThreads / decltype(lanes)::value;
    items = (static_cast<uint64_t>(a.rows) + rpb - 1) / rpb * kThreads;
    return hipSuccess;
  });
  return items;
}

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return dispatch(a, [&](auto t, auto lanes, auto pieces) -> hipError_t {
    constexpr int rpb = kThreads / decltype(lanes)::value;
    k_add_norm<decltype(t), decltype(lanes)::value, decltype(pieces)::value>
        <<<static_cast<unsigned>((static_cast<int64_t>(a.rows) + rpb - 1) / rpb), kThreads, 0, stream>>>(a);
    return hipGetLastError();
  });
}

size_t add_norm_backward_workspace_bytes(const AddNormArgs& a) {
  return static_cast<size_t>(kBackwardBlocks) * a.channels * sizeof(float);
}

hipError_t launch_add_norm_backward(const AddNormArgs& a, void* workspace, hipStream_t stream) {
  return dispatch(a, [&](auto t, auto lanes, auto pieces) -> hipError_t {
    constexpr int rpb = kThreads / decltype(lanes)::value;
    // (one block at least: no rows give zero sums)
    const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((static_cast<int64_t>(a.rows) + rpb - 1) / rpb, backward_blocks(decltype(pieces)::value)));
    float* part = static_cast<float*>(workspace);
    k_add_norm_backward<decltype(t), decltype(lanes)::value, decltype(pieces)::value><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(a, part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.grad_weight == nullptr) return e;
    k_add_norm_weight_sum<<<static_cast<unsigned>((a.channels + 31) / 32), 1024, 0, stream>>>(part, static_cast<int>(blocks), a.channels, a.grad_weight);
    return hipGetLastError();
  });
}

}  // namespace spconv
