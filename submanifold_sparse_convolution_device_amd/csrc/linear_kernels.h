// The matrix products of packed rows, for one type (linear_f32.hip,
// linear_f16.hip and linear_bf16.hip hold an instance each).
//
//   by rows:    out[m][n] = sum_k a[m][k] b[k][n]      b rows along k (the weights as they lie)
//   by rows T:  out[m][n] = sum_k a[m][k] b[n][k]      b rows along n (the same weights, transposed)
//   over rows:  out[m][n] = sum_r a[r][m] b[r][n]      both rows along the contraction
//
// A workgroup computes a BM x BN tile of one group of rows, or of one part of
// its contraction; its wavefronts WR x WC share it in tiles of 32 x 32
// products.  Per step of BK contracted values it loads its part of both
// operands in 16-byte pieces (rows, columns and contracted values that do not
// exist come back as zeros from the buffer's bounds check), and puts them into
// LDS as they lie in memory: an operand whose rows run along the contraction
// is read with the transposing LDS read, the other one piece by piece.  The
// next step's loads are in flight during this step's products.  fp32 operands
// go into LDS as three bf16 planes (attention_common.h).
//
// Where sums are long the matrix cores are busy in 53% of the cycles, LDS in
// 33%, at a clock of about 2 GHz: 8192 x 4096 x 4096 at 1.0 to 1.1 PFLOP/s (f16:
// 273 us by rows, 268 transposed, 279 over rows).  The library's products there
// take 0.72 to 0.89 of the time by rows and transposed and 0.91 to 1.04 over
// rows, so the clock alone is not what bounds these; the operands' way through
// registers into LDS between the products may be.  Writing the next step's
// tiles between the products rather than after them took 291 us to 275 by rows;
// two steps of loads in flight, halves of a workgroup in opposite phases and the
// epilogue between the next tile's products were no faster or slower.
//
// The products run as C^T = B^T A^T, so a lane holds 4 neighbouring columns of
// one row; the sums pass through the wavefront's own LDS into whole rows, 8
// columns a lane, for the epilogue (finish) and 16-byte accesses.
#pragma once

#include <algorithm>
#include <type_traits>

#include "linear_common.h"

namespace spconv {
namespace lin {

using attn::Frag;
using attn::Raw;
using attn::floatx16;
using attn::kPlanes;

// Orders a wavefront's own LDS accesses.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// One operand's part of a step: ROWS rows of PPR pieces, by NT threads.
template <class T, int ROWS, int PPR, int NT>
struct Stage {
  static constexpr int kCount = (ROWS * PPR + NT - 1) / NT;
  static constexpr bool kWhole = ROWS * PPR % NT == 0;
  static_assert(NT % PPR == 0 && ((PPR & (PPR - 1)) == 0) && PPR >= 4, "a thread's pieces share a column");
  Raw<T> r[kCount];

  // base: the first piece; rows_left rows and cols_left columns (whole
  // 16-byte pieces) exist from there.
  __device__ __forceinline__ void load(const T* base, int64_t stride, int rows_left, int cols_left, int tid) {
    const uint32_t row_bytes = static_cast<uint32_t>(stride) * sizeof(T);  // (at most 2^22: 2^30 for a tile)
    const int rows = min(max(rows_left, 0), ROWS);
    const int bytes = rows > 0 && cols_left > 0 ? (rows - 1) * static_cast<int>(row_bytes) + min(cols_left, PPR * 8) * static_cast<int>(sizeof(T)) : 0;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, bytes, attn::kBufferWord3);
    const int piece = tid % PPR, row = tid / PPR;
#pragma unroll
    for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) {
      const bool on = piece * 8 + h * 4 < cols_left;
      const uint32_t v0 = on ? row * row_bytes + (piece * 8 * sizeof(T) + 16 * h) : attn::kNowhere;
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const uint32_t v = v0 + static_cast<uint32_t>(i * (NT / PPR)) * row_bytes;
        r[i].v[h] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, static_cast<int>(kWhole || row + i * (NT / PPR) < ROWS ? v : attn::kNowhere), 0, 0));
      }
    }
  }

  // The place of a piece: its index XOR-ed with a function of the row.
  // ALONG: the contraction runs along a row, and 16 lanes read one piece of 16
  // rows; else 16 lanes read 4 rows x 32 bytes (transposed).
  template <bool ALONG>
  __device__ static __forceinline__ int at(int row, int piece) {
    if constexpr (ALONG) {
      return row * PPR + (piece ^ (PPR >= 16 ? row & 15 : PPR == 8 ? row >> 1 & 7 : row >> 2 & 3));
    } else if constexpr (PPR >= 16) {
      return row * PPR + (piece ^ ((row & 3) << 2 ^ (row & 2)));
    } else if constexpr (PPR == 8) {
      return row * PPR + (piece ^ (row & 3) << 1);
    } else {
      return row * PPR + (piece ^ (row & 2));
    }
  }

  template <bool ALONG>
  __device__ __forceinline__ void store(uint4* lds, int tid) const {
    const int piece = tid % PPR, row = tid / PPR;
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      const Frag<T> f = attn::to_frag<T>(r[i]);
      const int w = row + i * (NT / PPR);
      if (kWhole || w < ROWS) {
#pragma unroll
        for (int p = 0; p < kPlanes<T>; ++p) lds[p * ROWS * PPR + at<ALONG>(w, piece)] = f.v[p];
      }
    }
  }

  // The operand of 32 rows (columns, where the contraction runs along the
  // tile's rows) from x0 and 16 contracted values from 16 t.
  template <bool ALONG>
  __device__ static __forceinline__ Frag<T> frag(const uint4* lds, int x0, int t, int lane) {
    Frag<T> f;
    if constexpr (ALONG) {
      const int place = at<true>(x0 + (lane & 31), 2 * t + (lane >> 5));
#pragma unroll
      for (int p = 0; p < kPlanes<T>; ++p) f.v[p] = lds[p * ROWS * PPR + place];
    } else {
      // lane g of 16 addresses 4 columns of row g / 4, and receives column g of the four rows
      const int g = lane & 15, row = 16 * t + 8 * (lane >> 5) + (g >> 2), col = x0 + 16 * (lane >> 4 & 1) + 4 * (g & 3);
#pragma unroll
      for (int p = 0; p < kPlanes<T>; ++p) {
        uint2 half[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const char* src = reinterpret_cast<const char*>(lds + p * ROWS * PPR + at<false>(row + 4 * u, col / 8)) + (col & 4) * 2;
          half[u] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((attn::lds_s16x4*)src));
        }
        f.v[p] = make_uint4(half[0].x, half[0].y, half[1].x, half[1].y);
      }
    }
    return f;
  }
};

template <class T, class S, int FORM>
struct Kernel {
  static constexpr bool kAlongA = FORM != kOverRows, kAlongB = FORM == kByRowsT;
  static constexpr int kRowsA = kAlongA ? S::BM : S::BK, kPprA = (kAlongA ? S::BK : S::BM) / 8;
  static constexpr int kRowsB = kAlongB ? S::BN : S::BK, kPprB = (kAlongB ? S::BK : S::BN) / 8;
  typedef Stage<T, kRowsA, kPprA, S::NT> A;
  typedef Stage<T, kRowsB, kPprB, S::NT> B;
  static constexpr int kPiecesA = kRowsA * kPprA * kPlanes<T>, kPieces = kPiecesA + kRowsB * kPprB * kPlanes<T>;
  static constexpr int kOutStride = S::TN + 4;  // floats of a staged row of sums
  static constexpr int kOutPieces = S::WR * S::WC * 32 * kOutStride / 4;
  static constexpr int kLds = std::max(kPieces * S::STAGES, std::max(kOutPieces, S::NT * 2));
};

template <class T, class S, int FORM>
__global__ __launch_bounds__(S::NT) void k_product(ProductArgs a) {
  typedef Kernel<T, S, FORM> K;
  __shared__ uint4 lds[K::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;

  // Consecutive workgroups go to the 8 XCDs in turn; each XCD takes a
  // consecutive eighth of the tiles, so that tiles that share rows or weights
  // share its L2.  Over groups, whose lengths may differ by any factor, an
  // eighth of them could be nearly all of the work: there every group's sums
  // are spread over the XCDs, by their tiles or by the group's parts.
  const int total = gridDim.x, eighth = total / 8, over = total % 8;
  const int xcd = blockIdx.x % 8;
  int at = blockIdx.x / 8 + xcd * eighth + min(xcd, over);
  int slot, m0, n0, k0 = 0, k1, split = 0;
  if constexpr (FORM == kOverRows) {
    int tile;
    if (a.cu == nullptr) {
      slot = at / a.tiles;
      tile = at - slot * a.tiles;
    } else {
      const int j = blockIdx.x / 8, run = a.by_tiles ? (a.tiles + 7) / 8 : a.tiles, nth = j / run;
      slot = a.by_tiles ? nth : 8 * nth + xcd;
      tile = j - nth * run + (a.by_tiles ? xcd * run : 0);
      if (slot >= a.slots || tile >= a.tiles) return;
    }
    m0 = tile / a.tiles_n * S::BM;
    n0 = tile % a.tiles_n * S::BN;
  } else {
    // 4 slots by all columns at a time: what runs together shares both sides
    const int per = a.slots * a.tiles;
    split = at / per;
    at -= split * per;
    const int band = at / (4 * a.tiles), high = min(4, a.slots - 4 * band);
    at -= band * 4 * a.tiles;
    slot = 4 * band + at % high;
    n0 = at / high * S::BN;
    m0 = 0;
    k0 = split * a.k_split;
  }
  const Segment seg = find_segment(a, slot);
  const int rows = seg.hi - seg.lo;
  if constexpr (FORM == kOverRows) {
    // (a part without rows is written only where it is the whole sum)
    if (seg.group < 0 || (rows <= 0 && (a.part != nullptr || !seg.first))) return;
    k1 = max(rows, 0);
  } else {
    if (rows <= 0 || (seg.group < 0 && a.part != nullptr)) return;
    k1 = seg.group < 0 ? 0 : min(a.k, k0 + a.k_split);
  }

  // The bias of this lane's columns, on its way during the products.
  constexpr int LPR = S::TN / 8, RPP = 64 / LPR;  // lanes of a row, rows of a pass of the epilogue
  const int col = n0 + wc * S::TN + lane % LPR * 8;
  float bias[8] = {};
  if (FORM == kByRows && a.whole && a.part == nullptr && a.bias != nullptr && seg.group >= 0 && col < a.n)
    unpack8<T>(load_raw8<T>(static_cast<const T*>(a.bias) + static_cast<int64_t>(seg.group) * a.n + col), bias);

  const T* A0 = static_cast<const T*>(a.a) + static_cast<int64_t>(seg.lo) * a.a_row;
  const T* B0 = static_cast<const T*>(a.b) + (FORM == kOverRows ? static_cast<int64_t>(seg.lo) * a.b_row : static_cast<int64_t>(max(seg.group, 0)) * a.b_group);
  typename K::A sa;
  typename K::B sb;
  auto fetch = [&](int k) {
    if constexpr (FORM == kOverRows) {
      sa.load(A0 + static_cast<int64_t>(k) * a.a_row + m0, a.a_row, k1 - k, a.a_cols - m0, tid);
      sb.load(B0 + static_cast<int64_t>(k) * a.b_row + n0, a.b_row, k1 - k, a.b_cols - n0, tid);
    } else {
      sa.load(A0 + k, a.a_row, rows, a.a_cols - k, tid);
      if constexpr (FORM == kByRows) {
        sb.load(B0 + static_cast<int64_t>(k) * a.b_row + n0, a.b_row, a.k - k, a.b_cols - n0, tid);
      } else {
        sb.load(B0 + static_cast<int64_t>(n0) * a.b_row + k, a.b_row, a.n - n0, a.b_cols - k, tid);
      }
    }
  };
  float column[8] = {};  // over rows: this thread's share of the sums of 8 columns of b
  const bool sums = FORM == kOverRows && m0 == 0 && (a.sums != nullptr || a.sums_part != nullptr);
  auto put_a = [&](uint4* to) { sa.template store<K::kAlongA>(to, tid); };
  auto put_b = [&](uint4* to) {
    if constexpr (FORM == kOverRows) {
      if (sums) {
#pragma unroll
        for (int i = 0; i < K::B::kCount; ++i) {
          float v[8];
          unpack8<T>(sb.r[i], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) column[j] += v[j];
        }
      }
    }
    sb.template store<K::kAlongB>(to + K::kPiecesA, tid);
  };

  constexpr int RB = S::TM / 32, CB = S::TN / 32, STEPS = S::BK / 16;
  floatx16 acc[RB][CB] = {};
  // The products of a step; between(t) runs before those of 16 values t.
  auto multiply = [&](const uint4* from, auto&& between) {
    Frag<T> fa[STEPS][RB], fb[STEPS][CB];
    auto read = [&](int t) {
#pragma unroll
      for (int i = 0; i < RB; ++i) fa[t][i] = K::A::template frag<K::kAlongA>(from, wr * S::TM + 32 * i, t, lane);
#pragma unroll
      for (int j = 0; j < CB; ++j) fb[t][j] = K::B::template frag<K::kAlongB>(from + K::kPiecesA, wc * S::TN + 32 * j, t, lane);
    };
    // (over rows, with the column sums, two sets of operands do not fit beside large tiles)
    constexpr bool TWO = FORM != kOverRows || RB * CB <= 4;
    if (TWO) read(0);
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      if (!TWO) read(t);
      else if (t + 1 < STEPS) read(t + 1);
      between(t);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < CB; ++j) acc[i][j] = attn::mma_frag<T>(fb[t][j], fa[t][i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
    attn::settle();
  };

  if (k0 < k1) {
    fetch(k0);
    if constexpr (S::STAGES == 2) {
      // One barrier a step: it ends the writes of this step's buffer and the
      // reads of the other one, which is filled between this step's products.
      put_a(lds);
      put_b(lds);
      int buf = 0;
      for (int k = k0; k < k1; k += S::BK) {
        __syncthreads();
        const bool more = k + S::BK < k1;
        if (more) fetch(k + S::BK);
        __builtin_amdgcn_sched_barrier(0);
        uint4* other = lds + (buf ^ 1) * K::kPieces;
        multiply(lds + buf * K::kPieces, [&](int t) {
          if (t == STEPS - 2 && more) put_a(other);
          if (t == STEPS - 1 && more) put_b(other);
        });
        buf ^= 1;
      }
    } else {
      for (int k = k0; k < k1; k += S::BK) {
        __syncthreads();
        put_a(lds);
        put_b(lds);
        __syncthreads();
        if (k + S::BK < k1) fetch(k + S::BK);
        __builtin_amdgcn_sched_barrier(0);
        multiply(lds, [](int) {});
      }
    }
  }

  if constexpr (FORM == kOverRows) {
    if (sums) {
      // the threads of one column piece, in the order of their rows
      constexpr int PPR = K::kPprB, GROUPS = S::NT / PPR;
      float* stage = reinterpret_cast<float*>(lds);
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) stage[(tid / PPR) * (PPR * 8) + tid % PPR * 8 + j] = column[j];
      __syncthreads();
      for (int c = tid; c < S::BN; c += S::NT) {
        float v = 0.f;
#pragma unroll 8
        for (int q = 0; q < GROUPS; ++q) v += stage[q * (PPR * 8) + c];
        if (n0 + c < a.n) {
          if (a.part != nullptr) a.sums_part[static_cast<int64_t>(slot) * a.n_part + n0 + c] = v;
          else a.sums[static_cast<int64_t>(seg.group) * a.n + n0 + c] = v;
        }
      }
    }
  }
  __syncthreads();

  // The sums, 32 rows at a time.
  float* stage = reinterpret_cast<float*>(lds) + wave * 32 * K::kOutStride;
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    constexpr int PASSES = 32 / RPP;
    const int mi = wr * S::TM + 32 * i;  // first row in the tile
    const int64_t first = FORM == kOverRows ? static_cast<int64_t>(seg.group) * a.m + m0 + mi : static_cast<int64_t>(seg.lo) + mi;  // of out
    const int limit = (FORM == kOverRows ? a.m - m0 : rows) - mi;  // rows there are
    Raw<T> side[PASSES];
    const bool sides = FORM != kOverRows && a.whole && a.part == nullptr && a.side != nullptr && seg.group >= 0;
    if (sides) {
#pragma unroll
      for (int q = 0; q < PASSES; ++q) {
        const int r = q * RPP + lane / LPR;
        side[q] = attn::load_piece<T>(side_row<T>(a, first + r) + col, r < limit && col < a.n);
      }
    }
    wave_order();
#pragma unroll
    for (int j = 0; j < CB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<float4*>(stage + (lane & 31) * K::kOutStride + 32 * j + 8 * q + 4 * (lane >> 5)) =
            make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    wave_order();
    if (a.part != nullptr || a.whole) {
#pragma unroll
      for (int q = 0; q < PASSES; ++q) {
        const int r = q * RPP + lane / LPR;
        float v[8];
        const float4 lo = *reinterpret_cast<const float4*>(stage + r * K::kOutStride + lane % LPR * 8);
        const float4 hi = *reinterpret_cast<const float4*>(stage + r * K::kOutStride + lane % LPR * 8 + 4);
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
        if (r >= limit || col >= a.n) continue;
        if (a.part != nullptr) {
          const int64_t row = FORM == kOverRows ? static_cast<int64_t>(slot) * a.m + m0 + mi + r : static_cast<int64_t>(split) * a.rows + first + r;
          store8<float>(a.part + row * a.n_part + col, v);
        } else if constexpr (FORM == kOverRows) {
          store8<float>(static_cast<float*>(a.out) + (first + r) * a.n + col, v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += bias[j];
          finish<T, FORM, 8>(a, seg.group >= 0, sides, [&](int j) { return element<T>(side[q], j); }, v, [&](T* to, int64_t stride, const float (&x)[8]) { store8<T>(to + (first + r) * stride + col, x); });
        }
      }
    } else {
      // Rows without 16-byte places: a lane a column, so that stores follow
      // one another.
      constexpr int LANES = S::TN < 64 ? S::TN : 64, ROWS = 64 / LANES;
#pragma unroll 1
      for (int c0 = 0; c0 < S::TN; c0 += LANES) {
        const int c = c0 + lane % LANES, at = n0 + wc * S::TN + c;
        if (at >= a.n) continue;
        float b = 0.f;
        if (FORM == kByRows && a.bias != nullptr && seg.group >= 0) b = static_cast<float>(static_cast<const T*>(a.bias)[static_cast<int64_t>(seg.group) * a.n + at]);
#pragma unroll 4
        for (int r = lane / LANES; r < min(32, limit); r += ROWS) {
          float v[1] = {stage[r * K::kOutStride + c] + b};
          if constexpr (FORM == kOverRows) {
            static_cast<float*>(a.out)[(first + r) * a.n + at] = v[0];
          } else {
            const bool beside = a.side != nullptr && seg.group >= 0;
            const float z = beside ? static_cast<float>(side_row<T>(a, first + r)[at]) : 0.f;
            finish<T, FORM, 1>(a, seg.group >= 0, beside, [&](int) { return z; }, v, [&](T* to, int64_t stride, const float (&x)[1]) { to[(first + r) * stride + at] = static_cast<T>(x[0]); });
          }
        }
      }
    }
  }
}

// ---- Weights in registers ----
// By rows with a short contraction (16 KS values at most): a workgroup of
// WR x WC wavefronts keeps its columns of the weights in registers, 32 a
// wavefront, and walks a run of slots of BM rows, RW blocks of 32 a wavefront.
// A tile's rows are loaded one tile ahead and pass through LDS, where the WC wavefronts of the
// same rows read them; the weights are read once, and a tile ends in one
// barrier.  The sums go to memory straight from the registers: an exchange
// between the halves of a wavefront gives each lane 8 neighbouring columns of
// a row.  OCC: wavefronts on a SIMD.
//
// Bound by memory and, with an activation, by the vector units: 400,000 rows
// 256 -> 1024 in bf16 are 1.02 GB, 293 to 327 us (3.1 to 3.5 TB/s); gelu's 15
// vector instructions an element beside the products make it 416 us.
template <int KS_, int WR_, int WC_, int RW_, int OCC_>
struct StreamShape {
  static constexpr int KS = KS_, WR = WR_, WC = WC_, RW = RW_, OCC = OCC_;
  static constexpr int NT = 64 * WR * WC, BM = 32 * WR * RW, BN = 32 * WC;
  static constexpr int PER_CU = OCC * 4 / (WR * WC);
};

template <class T, class S, int FORM>
__global__ __launch_bounds__(S::NT, S::OCC) void k_stream(ProductArgs a, int chunks, int per) {
  constexpr int KS = S::KS, WC = S::WC, RW = S::RW;
  typedef Stage<T, S::BM, 2 * KS, S::NT> A;
  typedef Stage<T, 16, 4, 64> W;  // 16 contracted values by 32 columns, a wavefront's own
  constexpr int PIECES = S::BM * 2 * KS * kPlanes<T>;
  __shared__ uint4 lds[2 * PIECES];
  __shared__ uint4 weights_lds[FORM == kByRows ? S::NT * kPlanes<T> : 1];  // a wavefront's own
  __shared__ float4 bias_lds[S::BN / 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / WC, wc = wave % WC, half = lane >> 5;
  // The workgroups of one run of slots, one for each tile of columns, follow
  // one another on one XCD, whose L2 then serves all but the first.
  const int xcd = blockIdx.x % 8, j = blockIdx.x / 8;
  const int chunk = j / a.tiles * 8 + xcd, n0 = j % a.tiles * S::BN;
  if (chunk >= chunks) return;
  const int n_wave = n0 + wc * 32;

  // The walk over the slots: segment, its bounds and first slot, the next one's.
  struct Walk {
    int slot, seg, r0, r1, first, next;
  };
  const int end = min((chunk + 1) * per, a.slots);
  auto group_of = [&](const Walk& w) { return a.cu == nullptr ? 0 : w.seg == 0 || w.seg == a.groups + 1 ? -1 : w.seg - 1; };
  auto rows_of = [&](const Walk& w) { return w.slot < end ? min(w.r1 - w.r0 - (w.slot - w.first) * S::BM, S::BM) : 0; };
  auto settle_walk = [&](Walk& w) {  // on to a slot with rows, or the end
    if (a.cu == nullptr) return;
    while (w.slot < end) {
      while (w.slot >= w.next) {
        ++w.seg;
        w.r0 = w.r1;
        w.first = w.next;
        w.r1 = max(__builtin_amdgcn_readfirstlane(attn::bound(a.cu, a.groups, a.rows, w.seg + 1)), w.r0);
        w.next = w.seg > a.groups ? end : fast_div(w.r1, a.by_unit) + w.seg + 1;
      }
      if (rows_of(w) > 0) return;
      ++w.slot;
    }
  };
  Walk cur;
  cur.slot = chunk * per;
  if (a.cu == nullptr) {
    cur.seg = 0, cur.r0 = 0, cur.r1 = a.rows, cur.first = 0, cur.next = a.slots;
  } else {
    const Segment g = find_segment(a, min(cur.slot, a.slots - 1));
    cur.seg = g.seg;
    cur.r0 = __builtin_amdgcn_readfirstlane(attn::bound(a.cu, a.groups, a.rows, g.seg));
    cur.r1 = max(__builtin_amdgcn_readfirstlane(attn::bound(a.cu, a.groups, a.rows, g.seg + 1)), cur.r0);
    cur.first = min(fast_div(cur.r0, a.by_unit) + g.seg, cur.slot);
    cur.next = g.seg > a.groups ? end : fast_div(cur.r1, a.by_unit) + g.seg + 1;
  }
  settle_walk(cur);
  if (cur.slot >= end) return;

  A sa;
  auto fetch = [&](const Walk& w) {
    const int rows = group_of(w) < 0 ? 0 : rows_of(w);
    const int64_t lo = w.r0 + static_cast<int64_t>(w.slot - w.first) * S::BM;
    sa.load(static_cast<const T*>(a.a) + lo * a.a_row, a.a_row, rows, a.a_cols, tid);
  };
  fetch(cur);
  int group = -2, buf = 0;
  Frag<T> fb[KS];
  auto load_weights = [&](int g) {
    const T* B = static_cast<const T*>(a.b) + static_cast<int64_t>(g) * a.b_group;
    if constexpr (FORM == kByRows) {
      uint4* mine = weights_lds + wave * 64 * kPlanes<T>;
      constexpr int STEP = sizeof(T) == 4 ? 4 : 8;  // loads in flight
#pragma unroll
      for (int t0 = 0; t0 < KS; t0 += STEP) {
        W w[STEP];
#pragma unroll
        for (int t = 0; t < STEP && t0 + t < KS; ++t)
          w[t].load(B + static_cast<int64_t>(16 * (t0 + t)) * a.b_row + n_wave, a.b_row, a.k - 16 * (t0 + t), a.b_cols - n_wave, lane);
#pragma unroll
        for (int t = 0; t < STEP && t0 + t < KS; ++t) {
          wave_order();
          w[t].template store<false>(mine, lane);
          wave_order();
          fb[t0 + t] = W::template frag<false>(mine, 0, 0, lane);
        }
      }
      __syncthreads();  // (the last tile's products have read the last group's bias)
      for (int c = tid; c < S::BN; c += S::NT)
        reinterpret_cast<float*>(bias_lds)[c] =
            a.bias != nullptr && n0 + c < a.n ? static_cast<float>(static_cast<const T*>(a.bias)[static_cast<int64_t>(g) * a.n + n0 + c]) : 0.f;
    } else {
      const int n = n_wave + (lane & 31);
#pragma unroll
      for (int t = 0; t < KS; ++t)
        fb[t] = attn::to_frag<T>(load_piece_of<T>(B + static_cast<int64_t>(n) * a.b_row + 16 * t + 8 * half, n < a.n, a.b_cols - 16 * t - 8 * half));
    }
  };
  // A wavefront's tile: its sums, and where they go.
  floatx16 acc[RW] = {};
  Raw<T> side[RW][2];
  int64_t row = 0;  // of this lane's first block
  int left = 0;     // rows from there on
  bool in_group = false, sides = false;
  auto multiply = [&](const Walk& w, int g) {
    row = w.r0 + static_cast<int64_t>(w.slot - w.first) * S::BM + wr * (32 * RW) + (lane & 31);
    left = rows_of(w) - wr * (32 * RW) - (lane & 31);
    in_group = g >= 0;
    sides = a.side != nullptr && in_group;
    if (sides) {
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int col = n_wave + 16 * p + 8 * half;
          side[i][p] = attn::load_piece<T>(side_row<T>(a, row + 32 * i) + col, 32 * i < left && col < a.n);
        }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (FORM == kByRows && a.bias != nullptr && in_group) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 b = bias_lds[wc * 8 + 2 * q + half];
#pragma unroll
        for (int i = 0; i < RW; ++i) acc[i][4 * q] = b.x, acc[i][4 * q + 1] = b.y, acc[i][4 * q + 2] = b.z, acc[i][4 * q + 3] = b.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < RW; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][e] = 0.f;
    }
    if (in_group) {
      constexpr int AHEAD = RW == 2 ? 2 : 3;  // operands on their way from LDS
      Frag<T> fa[KS][RW];
      auto read = [&](int t) {
#pragma unroll
        for (int i = 0; i < RW; ++i) fa[t][i] = A::template frag<true>(lds + buf * PIECES, (wr * RW + i) * 32, t, lane);
      };
#pragma unroll
      for (int t = 0; t < AHEAD; ++t) read(t);
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        if (t + AHEAD < KS) read(t + AHEAD);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < RW; ++i) acc[i] = attn::mma_frag<T>(fb[t], fa[t][i], acc[i]);
      }
    }
    attn::settle();
  };
  auto emit = [&]() {
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      float v[16];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = acc[i][8 * p + e], y = acc[i][8 * p + 4 + e];  // scalars first: a bit cast of a vector's element reads element 0
          const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y), false, false);
          const uint32_t r0 = r[0], r1 = r[1];
          v[8 * p + e] = __builtin_bit_cast(float, r0);
          v[8 * p + 4 + e] = __builtin_bit_cast(float, r1);
        }
      finish<T, FORM, 16>(a, in_group, sides, [&](int e) { return element<T>(side[i][e / 8], e % 8); }, v, [&](T* to, int64_t stride, const float (&x)[16]) {
        T* dst = to + (row + 32 * i) * stride + n_wave + 8 * half;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float u[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) u[e] = x[8 * b + e];
          if (32 * i < left && n_wave + 16 * b + 8 * half < a.n) store8<T>(dst + 16 * b, u);
        }
      });
    }
  };
  sa.template store<true>(lds, tid);
  while (true) {
    const int g = group_of(cur);
    if (g != group) {
      group = g;
      if (g >= 0) load_weights(g);
    }
    Walk nxt = cur;
    ++nxt.slot;
    settle_walk(nxt);
    __syncthreads();
    const bool more = nxt.slot < end;
    if (more) fetch(nxt);
    __builtin_amdgcn_sched_barrier(0);
    multiply(cur, g);
    // The next tile goes into LDS before this one's values leave: the wait for
    // its loads is then none for the stores.
    if (more) sa.template store<true>(lds + (buf ^ 1) * PIECES, tid);
    __builtin_amdgcn_sched_barrier(0);
    emit();
    if (!more) return;
    cur = nxt;
    buf ^= 1;
  }
}

// ---- Few rows ----
// By rows with up to 128 rows of a group on average (a group may have any
// number): a workgroup computes 32 rows by 32 CB columns, and its 4 or 8
// wavefronts take chunks of KC contracted values in turn,
// each by itself: both operands pass through the wavefront's own LDS, so that
// its loads are of whole lines, with the next chunk's in flight during a
// chunk (bf16, transposed: 128 groups of 20 rows 1024 -> 1024 46 us, 70 with
// operands straight from memory, a line's quarter a lane; 8 groups of 80 rows
// 11.7 and 18.9).  fp32 rows come straight, as their planes would take more of
// LDS than the loads gain (32 groups of 20 rows 512 -> 256 13.4 us by LDS,
// 11.3).  No wavefront waits for another before the sums of all of them are
// joined in LDS.  Bound by the weights' way from memory: 5 rows 2048 -> 8192
// in bf16 are 34 MB, 7.5 us (4.5 TB/s).
template <class T, int CB, int WAVES_, int FORM>
struct Few {
  static constexpr int KC = sizeof(T) == 4 ? 32 : 64, WAVES = WAVES_;
  typedef std::conditional_t<FORM == kByRows, Stage<T, KC, 4 * CB, 64>, Stage<T, 32 * CB, KC / 8, 64>> W;
  typedef Stage<T, 32, KC / 8, 64> A;
  static constexpr bool kStageRows = sizeof(T) == 2;
  static constexpr int kMineW = KC * 4 * CB * kPlanes<T>;                    // a wavefront's weights
  static constexpr int kMine = kMineW + (kStageRows ? 32 * KC / 8 : 0);  // and its rows
  static constexpr int kStride = 32 * CB + 4;                                   // floats of a row of sums
  static constexpr int kLds = std::max(WAVES * kMine, WAVES * 32 * kStride / 4);
};

template <class T, int CB, int WAVES, int FORM>
__global__ __launch_bounds__(64 * WAVES) void k_few(ProductArgs a) {
  typedef Few<T, CB, WAVES, FORM> F;
  constexpr int KC = F::KC, STEPS = KC / 16;
  __shared__ uint4 lds[F::kLds];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = lane >> 5;
  // a consecutive eighth of the tiles for each XCD (as in k_product): neighbouring columns share lines
  const int eighth = gridDim.x / 8, over = gridDim.x % 8, xcd = blockIdx.x % 8;
  int at = blockIdx.x / 8 + xcd * eighth + min(xcd, over);
  const int per = a.slots * a.tiles, split = at / per;
  at -= split * per;
  const int slot = at / a.tiles, n0 = (at - slot * a.tiles) * (32 * CB);
  const Segment seg = find_segment(a, slot);
  const int rows = seg.hi - seg.lo;
  if (rows <= 0 || (seg.group < 0 && a.part != nullptr)) return;
  const int k0 = split * a.k_split, k1 = seg.group < 0 ? k0 : min(a.k, k0 + a.k_split);
  const int a_end = k1 == a.k ? a.a_cols : k1, b_end = k1 == a.k ? a.b_cols : k1;  // (whole pieces)

  const T* A0 = static_cast<const T*>(a.a) + static_cast<int64_t>(seg.lo) * a.a_row;
  const T* B0 = static_cast<const T*>(a.b) + static_cast<int64_t>(max(seg.group, 0)) * a.b_group;
  const bool row_there = (lane & 31) < rows;
  Raw<T> ra[F::kStageRows ? 1 : STEPS];
  typename F::A rows_stage;
  typename F::W w;
  auto fetch = [&](int k) {
    if constexpr (F::kStageRows) {
      rows_stage.load(A0 + k, a.a_row, rows, a_end - k, lane);
    } else {
#pragma unroll
      for (int t = 0; t < STEPS; ++t)
        ra[t] = load_piece_of<T>(A0 + (lane & 31) * a.a_row + k + 16 * t + 8 * half, row_there, a_end - (k + 16 * t + 8 * half));
    }
    if constexpr (FORM == kByRows) {
      w.load(B0 + static_cast<int64_t>(k) * a.b_row + n0, a.b_row, k1 - k, a.b_cols - n0, lane);
    } else {
      w.load(B0 + static_cast<int64_t>(n0) * a.b_row + k, a.b_row, a.n - n0, b_end - k, lane);
    }
  };
  floatx16 acc[CB] = {};
  uint4* mine = lds + wave * F::kMine;
  int k = k0 + wave * KC;
  if (k < k1) fetch(k);
  while (k < k1) {
    Frag<T> fa[STEPS], fb[STEPS][CB];
    wave_order();
    w.template store<FORM != kByRows>(mine, lane);
    if constexpr (F::kStageRows) rows_stage.template store<true>(mine + F::kMineW, lane);
    wave_order();
#pragma unroll
    for (int t = 0; t < STEPS; ++t) {
      if constexpr (F::kStageRows) fa[t] = F::A::template frag<true>(mine + F::kMineW, 0, t, lane);
      else fa[t] = attn::to_frag<T>(ra[t]);
    }
#pragma unroll
    for (int t = 0; t < STEPS; ++t)
#pragma unroll
      for (int c = 0; c < CB; ++c) fb[t][c] = F::W::template frag<FORM != kByRows>(mine, 32 * c, t, lane);
    k += KC * F::WAVES;
    if (k < k1) fetch(k);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < STEPS; ++t)
#pragma unroll
      for (int c = 0; c < CB; ++c) acc[c] = attn::mma_frag<T>(fb[t][c], fa[t], acc[c]);
    attn::settle();
  }
  attn::settle();
  __syncthreads();
  float* stage = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int c = 0; c < CB; ++c)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *reinterpret_cast<float4*>(stage + (wave * 32 + (lane & 31)) * F::kStride + 32 * c + 8 * q + 4 * half) =
          make_float4(acc[c][4 * q], acc[c][4 * q + 1], acc[c][4 * q + 2], acc[c][4 * q + 3]);
  __syncthreads();
  // 8 columns of a row a thread, the wavefronts' sums in their order
  static_assert(64 * WAVES >= 128 * CB, "a thread a piece");
  if (tid >= 128 * CB) return;
  const int r = tid / (4 * CB), c = tid % (4 * CB) * 8, col = n0 + c, there = min(a.n - col, 8);
  if (r >= rows || there <= 0) return;
  const int64_t row = static_cast<int64_t>(seg.lo) + r;
  const bool in_group = seg.group >= 0, sides = a.part == nullptr && a.side != nullptr && in_group;
  float v[8] = {}, z[8] = {}, bias[8] = {};
  if (FORM == kByRows && a.part == nullptr && a.bias != nullptr && in_group)
    load_some8<T>(static_cast<const T*>(a.bias) + static_cast<int64_t>(seg.group) * a.n + col, there, a.whole, bias);
  if (sides) load_some8<T>(side_row<T>(a, row) + col, there, a.whole, z);
#pragma unroll
  for (int q = 0; q < F::WAVES; ++q) {
    const float4 lo = *reinterpret_cast<const float4*>(stage + (q * 32 + r) * F::kStride + c), hi = *reinterpret_cast<const float4*>(stage + (q * 32 + r) * F::kStride + c + 4);
    v[0] += lo.x, v[1] += lo.y, v[2] += lo.z, v[3] += lo.w, v[4] += hi.x, v[5] += hi.y, v[6] += hi.z, v[7] += hi.w;
  }
  if (a.part != nullptr) {
    store8<float>(a.part + (static_cast<int64_t>(split) * a.rows + row) * a.n_part + col, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] += bias[i];
  finish<T, FORM, 8>(a, in_group, sides, [&](int i) { return z[i]; }, v, [&](T* to, int64_t stride, const float (&x)[8]) { store_some8<T>(to + row * stride + col, there, a.whole, x); });
}

// ---- Launches ----
template <class T, class S, int FORM>
hipError_t launch_shape(const ProductArgs& a, hipStream_t stream) {
  const int64_t blocks = product_blocks(a, static_cast<ProductForm>(FORM));
  if (blocks == 0) return hipSuccess;
  k_product<T, S, FORM><<<static_cast<unsigned>(blocks), S::NT, 0, stream>>>(a);
  return hipGetLastError();
}

// Runs of slots: as many workgroups as run at once, a whole number of runs for
// each XCD.
template <class T, class S, int FORM>
hipError_t launch_stream(ProductArgs a, hipStream_t stream) {
  a.by_unit = make_fast_div(S::BM);
  a.slots = a.cu == nullptr ? (a.rows + S::BM - 1) / S::BM : a.rows / S::BM + a.groups + 2;
  a.tiles = a.tiles_n = (a.n + S::BN - 1) / S::BN;
  int chunks = std::max(8, 256 * S::PER_CU / a.tiles / 8 * 8);
  chunks = std::min(chunks, a.slots);
  const int per = (a.slots + chunks - 1) / chunks;
  chunks = (a.slots + per - 1) / per;
  const int64_t blocks = static_cast<int64_t>((chunks + 7) / 8 * 8) * a.tiles;
  k_stream<T, S, FORM><<<static_cast<unsigned>(blocks), S::NT, 0, stream>>>(a, chunks, per);
  return hipGetLastError();
}
// The shape by the columns there are, so that few are computed in vain
// (400,000 rows in bf16, 256 -> 64: 44 us by 64 columns, 52 by 128; 256 ->
// 128: 61 by 128, 80 by 256), then by the registers that the weights leave:
// two row blocks a wavefront for the longest contraction, with two wavefronts
// on a SIMD (256 -> 1024: 327 us, by one block 365).  f32, as three planes,
// has registers for 128 columns (200,000 rows 128 -> 256: 94 us, by 64 125).
template <class T, int FORM>
hipError_t launch_stream_sized(const ProductArgs& a, hipStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    if (a.k <= 64) return launch_stream<T, StreamShape<4, 1, 4, 1, 3>, FORM>(a, stream);
    return launch_stream<T, StreamShape<8, 1, 4, 1, 2>, FORM>(a, stream);
  } else {
    auto by_columns = [&](auto ks) -> hipError_t {
      constexpr int KS = decltype(ks)::value;
      if (a.n <= 64) return launch_stream<T, StreamShape<KS, 4, 2, 1, 4>, FORM>(a, stream);
      if (a.n <= 128) return launch_stream<T, StreamShape<KS, 2, 4, 1, 4>, FORM>(a, stream);
      return launch_stream<T, StreamShape<KS, 1, 8, 1, 4>, FORM>(a, stream);
    };
    if (a.k <= 64) return by_columns(std::integral_constant<int, 4>{});
    if (a.k <= 128) return by_columns(std::integral_constant<int, 8>{});
    if (a.n <= 64) return launch_stream<T, StreamShape<16, 4, 2, 1, 2>, FORM>(a, stream);
    if (a.n <= 128) return launch_stream<T, StreamShape<16, 2, 4, 1, 2>, FORM>(a, stream);
    return launch_stream<T, StreamShape<16, 1, 8, 2, 2>, FORM>(a, stream);
  }
}

template <class T>
hipError_t launch_typed(const ProductArgs& a, ProductForm form, ProductShape shape, hipStream_t stream) {
  auto by_form = [&](auto s) -> hipError_t {
    typedef decltype(s) S;
    if (form == kByRows) return launch_shape<T, S, kByRows>(a, stream);
    if (form == kByRowsT) return launch_shape<T, S, kByRowsT>(a, stream);
    return launch_shape<T, S, kOverRows>(a, stream);
  };
  if (shape == kStreamShape) return form == kByRows ? launch_stream_sized<T, kByRows>(a, stream) : launch_stream_sized<T, kByRowsT>(a, stream);
  if (shape == kFewShape || shape == kFewWideShape || shape == kFewShortShape) {
    auto few = [&](auto cb, auto waves) -> hipError_t {
      constexpr int CB = decltype(cb)::value, WAVES = decltype(waves)::value;
      const int64_t blocks = product_blocks(a, form);
      if (form == kByRows) k_few<T, CB, WAVES, kByRows><<<static_cast<unsigned>(blocks), 64 * WAVES, 0, stream>>>(a);
      else k_few<T, CB, WAVES, kByRowsT><<<static_cast<unsigned>(blocks), 64 * WAVES, 0, stream>>>(a);
      return hipGetLastError();
    };
    typedef std::integral_constant<int, 1> One;
    typedef std::integral_constant<int, 2> Two;
    if (shape == kFewShortShape) return form == kByRows ? few(Two{}, std::integral_constant<int, 4>{}) : few(One{}, std::integral_constant<int, 4>{});
    if (shape == kFewShape) return few(One{}, std::integral_constant<int, 8>{});
    return few(Two{}, std::integral_constant<int, 8>{});
  }
  if (shape == kNarrowShape) return by_form(typename Shapes<T>::Narrow{});
  if (shape == kHalfShape) return by_form(typename Shapes<T>::Half{});
  if (shape == kMediumShape) return by_form(typename Shapes<T>::Medium{});
  return by_form(typename Shapes<T>::Large{});
}

}  // namespace lin
}  // namespace spconv
