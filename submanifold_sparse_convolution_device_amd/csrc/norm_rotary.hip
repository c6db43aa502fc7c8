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
//
// Bound by HBM: each value is read once and written once.  A (row, head) unit
// is LPR lanes of one 16-byte piece each, and the units of a tensor run over
// the lanes in memory order (heads within rows), so a wavefront's access is
// one contiguous run as long as the heads are.  Measured: 800k rows of 16
// heads of 32, bf16, three axes: 313 us, 5.2 TB/s, the rate of a large copy;
// one lane group per row that walks its heads, whose accesses are 64-byte
// pieces, takes 486 us.  The gradient reads two tensors and writes one: 120k
// rows of 20 heads of 128, bf16, 380 us (4.8 TB/s).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"

namespace spconv {
namespace {

// Elements per lane: one 16-byte piece.
template <class T>
constexpr int kE = 16 / static_cast<int>(sizeof(T));

template <class T>
__device__ __forceinline__ void unpack(uint4 p, float (&v)[kE<T>]) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  const vec t = __builtin_bit_cast(vec, p);
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) v[u] = static_cast<float>(t[u]);
}
template <class T>
__device__ __forceinline__ uint4 pack(const float (&v)[kE<T>]) {
  typedef T vec __attribute__((ext_vector_type(kE<T>)));
  vec t;
#pragma unroll
  for (int u = 0; u < kE<T>; ++u) t[u] = static_cast<T>(v[u]);
  return __builtin_bit_cast(uint4, t);
}

// Sum over the LPR lanes of a unit (an aligned power of two of them).
template <int LPR>
__device__ __forceinline__ float unit_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPR; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// How a kernel rotates.  The wide forms read the angles of neighbouring pairs
// together: 16 bytes at a time, which needs the pairs of a piece (interleaved)
// or of 4 elements (halves) to lie within one axis.
enum Turn { kNone, kInterleaved, kInterleavedWide, kHalves, kHalvesWide };

// Cosine and sine of the angles of the pairs that this lane's elements
// e0 .. e0 + E - 1 belong to: E / 2 pairs when interleaved, else E.  A
// position outside the table turns by NaN.  Elements past R are copied: the
// other member that their pair lacks counts as a zero (an infinity of their
// own would make NaN of the factor 0), signed so that even their zeros keep
// their signs: y x 1 + (-0) = y.
template <class T, Turn TURN>
struct Angles {
  static constexpr int E = kE<T>;
  static constexpr int N = TURN == kInterleaved || TURN == kInterleavedWide ? E / 2 : E;
  float c[N], s[N];

  __device__ __forceinline__ void load(const NormRotaryArgs& a, int row, int e0) {
    if constexpr (TURN == kNone) return;
    const int half = a.rotary / 2, n = half / a.axes;
    constexpr int G = TURN == kInterleavedWide ? N : TURN == kHalvesWide ? 4 : 1;  // pairs read together
#pragma unroll
    for (int u = 0; u < N; u += G) {
      const int e = TURN == kInterleaved || TURN == kInterleavedWide ? e0 + 2 * u : e0 + u;
      const bool on = e < a.rotary;
      int p = TURN == kInterleaved || TURN == kInterleavedWide ? e >> 1 : e < half ? e : e - half;
      p = on ? p : 0;
      const int axis = (p >= n) + (p >= 2 * n) + (p >= 3 * n);  // at most 4 axes
      const int pos = a.positions[row * a.pos_row + axis];
      const bool in = static_cast<uint32_t>(pos) < static_cast<uint32_t>(a.extent);
      const float* t = a.table + (static_cast<int64_t>(in ? pos : 0) * n + (p - axis * n)) * 2;
      float v[2 * G];
      if constexpr (G == 1) {
        const float2 x = *reinterpret_cast<const float2*>(t);
        v[0] = x.x;
        v[1] = x.y;
      } else {
#pragma unroll
        for (int q = 0; q < G / 2; ++q) {
          const float4 x = reinterpret_cast<const float4*>(t)[q];
          v[4 * q] = x.x;
          v[4 * q + 1] = x.y;
          v[4 * q + 2] = x.z;
          v[4 * q + 3] = x.w;
        }
      }
#pragma unroll
      for (int q = 0; q < G; ++q) {
        c[u + q] = !on ? 1.f : in ? v[2 * q] : __builtin_nanf("");
        s[u + q] = !on ? -0.f : in ? v[2 * q + 1] : __builtin_nanf("");
      }
    }
  }

  // Turns y forward (SIGN 1) or back (-1).  stage: the unit's LDS, where each
  // lane finds its pairs' other members (halves only); zero: the place of
  // four zeros from there (lack).
  template <int SIGN>
  __device__ __forceinline__ void turn(const NormRotaryArgs& a, float* stage, int zero, int e0, float (&y)[E]) const {
    if constexpr (TURN == kNone) return;
    if constexpr (TURN == kInterleaved || TURN == kInterleavedWide) {
      // Pieces of 8 past R skip the turn (frames of 16 heads of 32, bf16: 317 us,
      // 321 by selects alone); for those of 4 selects alone are faster (57.5
      // against 58.3 us for 30k rows of 9 heads of 40 with the gradient).
      if (E == 8 && e0 >= a.rotary) return;
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const float x0 = y[2 * u], x1 = y[2 * u + 1], sn = SIGN > 0 ? s[u] : -s[u];
        const bool on = (TURN == kInterleavedWide && E == 8) || e0 + 2 * u < a.rotary;  // (a wide piece lies on one side)
        y[2 * u] = on ? x0 * c[u] - x1 * sn : x0;
        y[2 * u + 1] = on ? x0 * sn + x1 * c[u] : x1;
      }
    } else {
      const int half = a.rotary / 2;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < E; u += 4) *reinterpret_cast<float4*>(stage + e0 + u) = make_float4(y[u], y[u + 1], y[u + 2], y[u + 3]);
      __builtin_amdgcn_wave_barrier();
      constexpr int G = TURN == kHalvesWide ? 4 : 1;
#pragma unroll
      for (int u = 0; u < E; u += G) {
        const int e = e0 + u;
        const bool low = e < half;
        const int at = e >= a.rotary ? zero : low ? e + half : e - half;
        float o[G];
        if constexpr (G == 4) {
          const float4 x = *reinterpret_cast<const float4*>(stage + at);
          o[0] = x.x;
          o[1] = x.y;
          o[2] = x.z;
          o[3] = x.w;
        } else {
          o[0] = stage[at];
        }
#pragma unroll
        for (int q = 0; q < G; ++q) {
          const float sn = low == (SIGN > 0) ? -s[u + q] : s[u + q];
          y[u + q] = y[u + q] * c[u + q] + o[q] * sn;
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
};

// What stands for the missing member in a pass of that sign.
constexpr float lack(int sign) { return sign > 0 ? 0.f : -0.f; }

constexpr int kWaves = 4;
// Units per lane in flight: their loads are issued together.
constexpr int kUnits = 4;

template <class T, int LPR, Turn TURN>
__global__ __launch_bounds__(64 * kWaves) void k_norm_rotary(NormRotaryArgs a, int first_blocks) {
  constexpr int E = kE<T>, UPW = 64 / LPR, UPB = kWaves * UPW;  // units per wavefront and block pass
  __shared__ float4 stage[TURN >= kHalves ? kWaves * 64 * E / 4 + kWaves : 1];
  const bool second = static_cast<int>(blockIdx.x) >= first_blocks;
  const NormRotaryTensor& t = a.t[second ? 1 : 0];
  const int block = second ? blockIdx.x - first_blocks : blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = lane % LPR * E;
  float* mine = reinterpret_cast<float*>(stage) + (TURN >= kHalves ? (wave * 64 + lane / LPR * LPR) * E : 0);
  const int zero = kWaves * 64 * E + 4 * wave - (wave * 64 + lane / LPR * LPR) * E;  // a wave's own
  if (TURN >= kHalves && lane < 4) mine[zero + lane] = lack(1);
  const bool on = e0 < a.dim;
  const int units = a.rows * t.heads;
  const int u0 = block * (UPB * kUnits) + wave * UPW + lane / LPR;

  uint4 raw[kUnits];
  int row[kUnits], head[kUnits];
  bool ok[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    // (the last blocks' sums stay below 2^31: units is bounded on the host)
    const int u = u0 + i * UPB;
    ok[i] = u < units;
    row[i] = fast_div(ok[i] ? u : 0, t.by_heads);
    head[i] = (ok[i] ? u : 0) - row[i] * t.heads;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (ok[i] && on) raw[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(t.x) + row[i] * t.x_row + head[i] * t.x_head + e0);
  }
  Angles<T, TURN> ang[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) ang[i].load(a, row[i], e0);
  float w[E];
  if (t.weight != nullptr) unpack<T>(on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(t.weight) + e0) : make_uint4(0, 0, 0, 0), w);
  const float inv_dim = 1.f / static_cast<float>(a.dim);
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    float x[E];
    unpack<T>(raw[i], x);
    if (t.weight != nullptr) {
      float sq = 0.f;
#pragma unroll
      for (int u = 0; u < E; ++u) sq = __builtin_fmaf(x[u], x[u], sq);
      const float r = 1.f / sqrtf(unit_sum<LPR>(sq) * inv_dim + a.eps);
#pragma unroll
      for (int u = 0; u < E; ++u) x[u] = x[u] * r * w[u];
    }
    ang[i].template turn<1>(a, mine, zero, e0, x);
    if (ok[i] && on) *reinterpret_cast<uint4*>(static_cast<T*>(t.y) + row[i] * t.y_row + head[i] * t.y_head + e0) = pack<T>(x);
  }
}

// The gradient: a workgroup walks the units of one tensor by the grid's step
// and keeps its sums of the weight gradient in registers; part[block][dim]
// takes them.
template <class T, int LPR, Turn TURN>
__global__ __launch_bounds__(64 * kWaves) void k_norm_rotary_backward(NormRotaryArgs a, int first_blocks, float* part) {
  constexpr int E = kE<T>, UPW = 64 / LPR, UPB = kWaves * UPW, U = 2;
  __shared__ float4 stage[kWaves * 64 * E / 4 + kWaves];
  const bool second = static_cast<int>(blockIdx.x) >= first_blocks;
  const NormRotaryTensor& t = a.t[second ? 1 : 0];
  const int block = second ? blockIdx.x - first_blocks : blockIdx.x;
  const int blocks = second ? gridDim.x - first_blocks : first_blocks;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e0 = lane % LPR * E;
  float* mine = reinterpret_cast<float*>(stage) + (wave * 64 + lane / LPR * LPR) * E;
  const int zero = kWaves * 64 * E + 4 * wave - (wave * 64 + lane / LPR * LPR) * E;  // a wave's own
  if (TURN >= kHalves && lane < 4) mine[zero + lane] = lack(-1);
  const bool on = e0 < a.dim;
  const int units = a.rows * t.heads;
  const int64_t step = static_cast<int64_t>(blocks) * (UPB * U);
  float w[E], dw[E] = {};
  if (t.weight != nullptr) unpack<T>(on ? *reinterpret_cast<const uint4*>(static_cast<const T*>(t.weight) + e0) : make_uint4(0, 0, 0, 0), w);
  const float inv_dim = 1.f / static_cast<float>(a.dim);
  for (int64_t base = static_cast<int64_t>(block) * (UPB * U); base < units; base += step) {
    uint4 xr[U], gr[U];
    int row[U], head[U];
    bool ok[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t u = base + i * UPB + wave * UPW + lane / LPR;
      ok[i] = u < units;
      row[i] = fast_div(ok[i] ? static_cast<int>(u) : 0, t.by_heads);
      head[i] = (ok[i] ? static_cast<int>(u) : 0) - row[i] * t.heads;
      xr[i] = gr[i] = make_uint4(0, 0, 0, 0);
      if (ok[i] && on) {
        gr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(t.grad) + row[i] * t.g_row + head[i] * t.g_head + e0);
        if (t.weight != nullptr)
          xr[i] = *reinterpret_cast<const uint4*>(static_cast<const T*>(t.x) + row[i] * t.x_row + head[i] * t.x_head + e0);
      }
    }
    Angles<T, TURN> ang[U];
#pragma unroll
    for (int i = 0; i < U; ++i) ang[i].load(a, row[i], e0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float x[E], g[E];
      unpack<T>(gr[i], g);
      ang[i].template turn<-1>(a, mine, zero, e0, g);
      if (t.weight != nullptr) {
        unpack<T>(xr[i], x);
        float sq = 0.f, gx = 0.f, gw[E];
#pragma unroll
        for (int u = 0; u < E; ++u) {
          sq = __builtin_fmaf(x[u], x[u], sq);
          gw[u] = g[u] * w[u];
          gx = __builtin_fmaf(gw[u], x[u], gx);
        }
        const float r = 1.f / sqrtf(unit_sum<LPR>(sq) * inv_dim + a.eps);
        const float m = unit_sum<LPR>(gx) * inv_dim * r * r;
#pragma unroll
        for (int u = 0; u < E; ++u) {
          // a lane without a unit has no share (its angle is some row's)
          dw[u] = ok[i] ? __builtin_fmaf(g[u] * x[u], r, dw[u]) : dw[u];
          g[u] = r * (gw[u] - x[u] * m);
        }
      }
      if (ok[i] && on) *reinterpret_cast<uint4*>(static_cast<T*>(t.grad_x) + row[i] * t.gx_row + head[i] * t.gx_head + e0) = pack<T>(g);
    }
  }
  if (t.weight == nullptr || t.grad_weight == nullptr) return;
  // The workgroup's sums, in the order of its units' lanes.
  __syncthreads();
#pragma unroll
  for (int u = 0; u < E; ++u) mine[e0 + u] = dw[u];
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(stage);
  for (int d = threadIdx.x; d < a.dim; d += 64 * kWaves) {
    float sum = 0.f;
#pragma unroll 8
    for (int q = 0; q < UPB; ++q) sum += all[q * LPR * E + d];
    part[static_cast<int64_t>(blockIdx.x) * a.dim + d] = sum;
  }
}

// dw[d] = sum over the blocks' partial sums, in a fixed order.
__global__ __launch_bounds__(256) void k_norm_weight_sum(const float* part, int first_blocks, int blocks, int dim, float* dq,
                                                         float* dk) {
  __shared__ float stage[256];
  const int d = blockIdx.x;
  float* dst = blockIdx.y ? dk : dq;
  if (dst == nullptr) return;
  const int b0 = blockIdx.y ? first_blocks : 0, b1 = blockIdx.y ? blocks : first_blocks;
  float sum = 0.f;
  for (int b = b0 + threadIdx.x; b < b1; b += 256) sum += part[static_cast<int64_t>(b) * dim + d];
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

int lanes_per_unit(const NormRotaryArgs& a) {
  const int pieces = a.dim * (a.dtype == 0 ? 4 : 2) / 16;
  int l = 1;
  while (l < pieces) l *= 2;
  return l;
}

// Calls f(type, lanes per unit, turn) as compile-time values.
template <class F>
hipError_t dispatch(const NormRotaryArgs& a, F&& f) {
  const int pairs = a.rotary / (2 * a.axes);  // of one axis
  // the wide reads are 16 bytes: an even number of pairs keeps the table's rows on them
  const bool aligned = (reinterpret_cast<uintptr_t>(a.table) & 15u) == 0;
  auto by_turn = [&](auto t, auto l) -> hipError_t {
    constexpr int group = kE<decltype(t)> / 2;
    if (a.rotary == 0) return f(t, l, std::integral_constant<Turn, kNone>{});
    if (a.interleaved) {
      if (aligned && pairs % group == 0) return f(t, l, std::integral_constant<Turn, kInterleavedWide>{});
      return f(t, l, std::integral_constant<Turn, kInterleaved>{});
    }
    if (aligned && pairs % 4 == 0) return f(t, l, std::integral_constant<Turn, kHalvesWide>{});
    return f(t, l, std::integral_constant<Turn, kHalves>{});
  };
  auto by_lanes = [&](auto t) -> hipError_t {
    switch (lanes_per_unit(a)) {
      case 1: return by_turn(t, std::integral_constant<int, 1>{});
      case 2: return by_turn(t, std::integral_constant<int, 2>{});
      case 4: return by_turn(t, std::integral_constant<int, 4>{});
      case 8: return by_turn(t, std::integral_constant<int, 8>{});
      case 32:
        if constexpr (sizeof(t) == 4) return by_turn(t, std::integral_constant<int, 32>{});
        break;
      default: break;
    }
    return by_turn(t, std::integral_constant<int, 16>{});
  };
  if (a.dtype == 0) return by_lanes(0.f);
  if (a.dtype == 1) return by_lanes(static_cast<_Float16>(0));
  return by_lanes(static_cast<__bf16>(0.f));
}

// Blocks of the gradient's kernel for one tensor: enough to fill the chip,
// few enough that their partial weight gradients stay small.
constexpr int64_t kBackwardBlocks = 2048;
int64_t blocks_for(const NormRotaryArgs& a, const NormRotaryTensor& t, int64_t units_per_block) {
  return (static_cast<int64_t>(a.rows) * t.heads + units_per_block - 1) / units_per_block;
}

}  // namespace

uint64_t norm_rotary_work_items(const NormRotaryArgs& a) {
  const int64_t upb = kWaves * 64 / lanes_per_unit(a) * kUnits;
  return static_cast<uint64_t>(blocks_for(a, a.t[0], upb) + blocks_for(a, a.t[1], upb)) * (64 * kWaves);
}

hipError_t launch_norm_rotary(const NormRotaryArgs& a, hipStream_t stream) {
  if (a.rows == 0 || a.t[0].heads + a.t[1].heads == 0) return hipSuccess;
  return dispatch(a, [&](auto t, auto lanes, auto turn) -> hipError_t {
    typedef decltype(t) T;
    constexpr int LPR = decltype(lanes)::value;
    constexpr Turn TURN = decltype(turn)::value;
    constexpr int upb = kWaves * 64 / LPR * kUnits;
    const int64_t b0 = blocks_for(a, a.t[0], upb), b1 = blocks_for(a, a.t[1], upb);
    k_norm_rotary<T, LPR, TURN><<<static_cast<unsigned>(b0 + b1), 64 * kWaves, 0, stream>>>(a, static_cast<int>(b0));
    return hipGetLastError();
  });
}

size_t norm_rotary_backward_workspace_bytes(const NormRotaryArgs& a) {
  return static_cast<size_t>(2 * kBackwardBlocks) * a.dim * sizeof(float);
}

hipError_t launch_norm_rotary_backward(const NormRotaryArgs& a, void* workspace, hipStream_t stream) {
  if (a.t[0].heads + a.t[1].heads == 0) return hipSuccess;
  return dispatch(a, [&](auto t, auto lanes, auto turn) -> hipError_t {
    typedef decltype(t) T;
    constexpr int LPR = decltype(lanes)::value;
    constexpr Turn TURN = decltype(turn)::value;
    constexpr int upb = kWaves * 64 / LPR * 2;
    auto blocks = [&](const NormRotaryTensor& x) -> int64_t {
      if (x.heads == 0) return 0;
      return std::max<int64_t>(1, std::min(blocks_for(a, x, upb), kBackwardBlocks));  // one at least: no rows give zero sums
    };
    const int64_t b0 = blocks(a.t[0]), b1 = blocks(a.t[1]);
    float* part = static_cast<float*>(workspace);
    k_norm_rotary_backward<T, LPR, TURN><<<static_cast<unsigned>(b0 + b1), 64 * kWaves, 0, stream>>>(a, static_cast<int>(b0), part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    float* dq = b0 > 0 && a.t[0].weight != nullptr ? a.t[0].grad_weight : nullptr;
    float* dk = b1 > 0 && a.t[1].weight != nullptr ? a.t[1].grad_weight : nullptr;
    if (dq == nullptr && dk == nullptr) return hipSuccess;
    k_norm_weight_sum<<<dim3(a.dim, 2), 256, 0, stream>>>(part, static_cast<int>(b0), static_cast<int>(b0 + b1), a.dim, dq, dk);
    return hipGetLastError();
  });
}

hipError_t launch_rotary_table(float* table, int32_t extent, int32_t pairs, double base, double scale,
                               hipStream_t stream) {
  const int64_t n = static_cast<int64_t>(extent) * pairs;
  k_rotary_table<<<static_cast<unsigned>((n + 255) / 256), 256, 0, stream>>>(table, extent, pairs, base, scale);
  return hipGetLastError();
}

}  // namespace spconv
