// Gradients of softmax attention over packed sequences.
//
//   P_ij = exp(s_ij - lse_i),  D_i = dO_i . O_i,
//   dS_ij = P_ij (dO_i . v_j - D_i),
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i,
// the sums over i running over every query head that shares the key's head.
//
// Two kernels, one with a tile of queries resident that walks the keys (dq),
// one with a tile of keys resident that walks the queries (dk, dv).  The
// scores and dO V^T are computed in both, 14 products of d per pair instead
// of 10, and in exchange every sum has one owner: no atomics, the same bits
// on every run.
//
// Bound, as the forward, by the vector unit and its overlap with the matrix
// unit for long sequences (causal f16, 14.6k rows, 8 heads of 64 over 2: 134
// and 184 us for the 10 products' 0.12 TFLOP), and by the latency of each
// workgroup's few dependent loads for short ones (1200 windows of up to 343
// rows, 8 heads of 32, bf16: 227 and 305 us; the bytes alone would take 125 and
// 124).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "attention_common.h"

namespace spconv {
namespace {

using namespace attn;

// fp16 operands of the gradients' products.  dS is as small as the output's
// gradient times a probability, far below what fp16 holds, so each column
// (lane) of a dS tile is scaled by a power of two that keeps its largest
// value near 2^14, and the sums follow when the scale drops.  P^T takes the
// fixed scale 2^14 (it is at most 1).  bf16 and fp32 need neither.
template <class T>
constexpr float kShift = __is_same(T, _Float16) ? 14.f : 0.f;

template <class T, int DB>
__device__ __forceinline__ void rescale(float (&ds)[16], float& factor, floatx16 (&acc)[DB]) {
  if constexpr (__is_same(T, _Float16)) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(ds[i]));
    top = halves_max(top);
    if (__any(top * factor > 32768.f)) {
      // 2^(14 - exponent of top), never above the factor so far
      const int e = static_cast<int>((__builtin_bit_cast(uint32_t, top) >> 23) & 255) - 127;
      const float now = fminf(factor, __builtin_ldexpf(1.f, 14 - e));
      const float drop = now / factor;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[db][i] *= drop;
      factor = now;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) ds[i] *= factor;
  }
}
constexpr float kFirstFactor = 1.2676506002282294e30f;  // 2^100

// D comes from the output as it was rounded, and where a row sees few keys
// the dO v and D of its dS nearly cancel: the 16-bit gradients of q and k were
// 2.1 times as far from 64 bits as results that are rounded once at 3 keys, 1.6
// at 16 and 1.5 at 40 (all where values are nearly equal); from 100 on it is
// the 1.45 that the rounded dS itself makes.  Waves whose rows see at most so
// many keys together take D = sum_j P_ij dP_ij in a walk of their own before,
// straight from memory.  It takes 260 instead of 231 us in 4000 windows of up
// to 64 rows, 8 heads of 32, with the other two kernels; windows of up to 343
// rows and long causal sequences show nothing of it.
constexpr int kFewKeys = 64;

// Rows per LDS tile of the side that a workgroup walks, and tiles of its two
// tensors in LDS (two: one read, one filled; a lone wave stages through one).
template <class T, int DP, int WAVES>
constexpr int kWalk = sizeof(T) == 4 ? 32 : DP == 32 ? (WAVES == 4 ? 128 : 64) : DP == 64 && WAVES > 1 ? 64 : 32;
template <int WAVES>
constexpr int kBuffers = WAVES == 1 ? 1 : 2;

// (A lone wave at heads of up to 128 needs 340 registers: 355 us for 2000
// windows of up to 32 rows, 8 heads; held to 256 it spills and takes 385.)
template <class T, int DP, int DQ, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 && (DP < 128 || WAVES > 1) ? 2 : 1) void k_attention_dq(AttentionArgs a, int slots, int run, int nsplit, const int32_t* order,
                                                                                    float2* stats, float* part) {
  typedef Tile<T, DP> TL;
  constexpr int BN = kWalk<T, DP, WAVES>, BUFS = kBuffers<WAVES>, PPR = TL::PPR, DB = DP / 32, NT = 64 * WAVES;
  constexpr int BM = 32 * WAVES, KS = DQ / (2 * kPiece), NL = (BN * PPR + NT - 1) / NT;
  __shared__ uint4 ks[BUFS][kPlanes<T> * BN * PPR], vs[BUFS][kPlanes<T> * BN * PPR];
  __shared__ int scrubbed[BUFS][WAVES];  // whether the wave found infinities or NaN in its part of an edge tile's keys
  __shared__ uint32_t bad_keys[BUFS][BN / 32];  // and then, which keys hold them

  const int split = static_cast<int>(blockIdx.x) & (nsplit - 1), id = static_cast<int>(blockIdx.x) >> __builtin_ctz(nsplit);
  const Place at_block = place_of(a, id, run);
  if (at_block.slot >= slots) return;
  const int kvh = at_block.kvh;
  const Span sp = find_span(a, false, a.group, tile_shift(WAVES),
                            order != nullptr ? order[at_block.slot] : a.right >= 0 ? slots - 1 - at_block.slot : at_block.slot, slots);
  if (!sp.any) return;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = sp.nq * a.group;
  const int shift = sp.nk - sp.nq;

  const int wr0 = sp.r0 + 32 * wave;
  const int r = wr0 + (lane & 31);
  const bool has_row = r < rows;
  const int tok = div_group(a, has_row ? r : 0);
  const int head = kvh * a.group + (has_row ? r - tok * a.group : 0);
  const int64_t row_out = static_cast<int64_t>(sp.q0 + tok) * a.heads + head;
  Frag<T> qf[KS], gf[KS];
  Raw<T> go[KS], ov[KS];
  {
    const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(sp.q0 + tok) * a.q_row + static_cast<int64_t>(head) * a.q_head;
    const T* gsrc = static_cast<const T*>(a.grad_out) + static_cast<int64_t>(sp.q0 + tok) * a.go_row + static_cast<int64_t>(head) * a.go_head;
    const T* osrc = static_cast<const T*>(a.out) + row_out * a.dim;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const int e = (2 * t + half) * kPiece;
      const bool ok = has_row && e < a.dim;
      go[t] = load_piece(gsrc + e, ok);
      ov[t] = load_piece(osrc + e, ok);
      qf[t] = to_frag<T>(load_piece(src + e, ok));
    }
  }
  const int place = tok + shift;
  const int lane_lo = a.left >= 0 ? place - a.left : 0;
  const int lane_hi = a.right >= 0 ? min(place + a.right + 1, sp.nk) : sp.nk;
  const KeyRange wg = key_range(a, sp.nk, div_group(a, sp.r0) + shift, div_group(a, min(sp.r0 + BM, rows) - 1) + shift);
  const bool wave_on = wr0 < rows;
  const int wp0 = div_group(a, wave_on ? wr0 : 0) + shift, wp1 = div_group(a, wave_on ? min(wr0 + 32, rows) - 1 : 0) + shift;
  const KeyRange wv = key_range(a, sp.nk, wp0, wp1);
  const int full_lo = a.left >= 0 ? wp1 - a.left : 0;
  const int full_hi = a.right >= 0 ? min(wp0 + a.right + 1, sp.nk) : sp.nk;

  const int blocks = wg.hi > wg.lo ? (wg.hi - wg.lo + BN - 1) / BN : 0;
  const Share mine = share_of(blocks, split, nsplit);
  const int jb0 = mine.first, jb1 = mine.end;

  const T* kbase = static_cast<const T*>(a.k) + static_cast<int64_t>(kvh) * a.k_head + static_cast<int64_t>(sp.k0) * a.k_row;
  const T* vbase = static_cast<const T*>(a.v) + static_cast<int64_t>(kvh) * a.v_head + static_cast<int64_t>(sp.k0) * a.v_row;
  const uint32_t kb = static_cast<uint32_t>(a.k_row * sizeof(T)), vb = static_cast<uint32_t>(a.v_row * sizeof(T));
  Raw<T> kr[NL], vr[NL];
  uint32_t koff[NL], voff[NL];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
    const int slot = tid + n * NT, row = slot / PPR, piece = slot % PPR;
    const bool on = row < BN && piece * kPiece < a.dim;
    koff[n] = on ? row * kb + piece * kPieceBytes<T> : kNowhere;
    voff[n] = on ? row * vb + piece * kPieceBytes<T> : kNowhere;
  }
  auto load = [&](int jb) {
    const int j0 = wg.lo + jb * BN;
    const auto kbuf = rows_buffer(kbase + j0 * a.k_row, sp.nk - j0, kb), vbuf = rows_buffer(vbase + j0 * a.v_row, sp.nk - j0, vb);
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      kr[n] = load_piece<T>(kbuf, koff[n]);
      vr[n] = load_piece<T>(vbuf, voff[n]);
    }
  };

  // The first tile's loads are on their way while D is made (heads of up to
  // 64: the registers of larger ones do not hold both).
  constexpr bool kEarly = DP <= 64 && sizeof(T) == 2;
  if (kEarly && jb0 < jb1) load(jb0);

  float dot = 0.f;
#pragma unroll
  for (int t = 0; t < KS; ++t) {
    gf[t] = to_frag<T>(go[t]);
    typedef T part_t __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
    for (int w = 0; w < static_cast<int>(sizeof(T) / 2); ++w) {
      const part_t o = __builtin_bit_cast(part_t, ov[t].v[w]), g = __builtin_bit_cast(part_t, go[t].v[w]);
#pragma unroll
      for (int u = 0; u < static_cast<int>(16 / sizeof(T)); ++u) dot = __builtin_fmaf(to_f32(g[u]), to_f32(o[u]), dot);
    }
  }
  dot = halves_sum(dot);
  // exp(s - lse) as exp2(s c - lse2); a row without keys, or past the end, has P = 0
  float lse2 = INFINITY;
  if (has_row) {
    const float v = a.lse[row_out];
    lse2 = v == -INFINITY ? INFINITY : log2_units(v) - kShift<T>;
  }
  const float c = a.scale * kLog2e;
  if constexpr (sizeof(T) == 2) {
    if (wave_on && wv.hi > wv.lo && wv.hi - wv.lo <= kFewKeys) {
      float sum = 0.f;
#pragma unroll 1
      for (int j0 = wv.lo; j0 < wv.hi; j0 += 32) {
        const auto kbuf = rows_buffer(kbase + j0 * a.k_row, sp.nk - j0, kb), vbuf = rows_buffer(vbase + j0 * a.v_row, sp.nk - j0, vb);
        Raw<T> kp[KS], vp[KS];
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const int piece = 2 * t + half;
          const bool on = piece * kPiece < a.dim;
          kp[t] = load_piece<T>(kbuf, on ? (lane & 31) * kb + piece * kPieceBytes<T> : kNowhere);
          vp[t] = load_piece<T>(vbuf, on ? (lane & 31) * vb + piece * kPieceBytes<T> : kNowhere);
        }
        floatx16 s(0.f), dp(0.f);
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          s = mma_frag<T>(to_frag<T>(kp[t]), qf[t], s);
          dp = mma_frag<T>(to_frag<T>(vp[t]), gf[t], dp);
        }
        settle();
        const int first = lane_lo - j0 - 4 * half, end = lane_hi - j0 - 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = fast_exp2(__builtin_fmaf(s[i], c, -lse2)) * dp[i];
          sum += c_row(i) >= first && c_row(i) < end ? x : 0.f;
        }
      }
      sum = halves_sum(sum) * (__is_same(T, _Float16) ? 6.103515625e-05f : 1.f);  // P's shift
      dot = fabsf(dot) < INFINITY ? sum : dot;
    }
  }
  // The statistics for the other kernel, in the order in which it walks the
  // rows; a D that is not finite makes NaN of both.
  if (has_row && half == 0 && split == 0)
    stats[static_cast<int64_t>(kvh) * a.total_q * a.group + static_cast<int64_t>(sp.q0) * a.group + r] = make_float2(__builtin_fmaf(0.f, dot, lse2), dot);

  floatx16 acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) acc[db] = floatx16(0.f);
  float factor = kFirstFactor;

  // Edge tiles hold keys that some row of the workgroup does not see: these go
  // into LDS with their infinities and NaN as zeros.  A row that sees such a
  // key has a NaN lse, or a score of -inf with it: its dS is set to 0 in the
  // loop, and what 0 or NaN times the key gives follows after the loop.  What
  // lies past the sequence's end is zero as loaded, unless the rows repeat one.
  const int edge_end = a.k_row != 0 ? INT_MAX : sp.nk;
  const int edge_hi = a.right >= 0 ? min(div_group(a, sp.r0) + shift + a.right + 1, edge_end) : edge_end;
  const int edge_lo = a.left >= 0 ? div_group(a, min(sp.r0 + BM, rows) - 1) + shift - a.left : 0;
  auto is_edge = [&](int jb) { return wg.lo + (jb + 1) * BN > edge_hi || wg.lo + jb * BN < edge_lo; };
  uint32_t met_tiles = 0;  // edge tiles with such keys, by their number modulo 32
  auto store = [&](int buf, int jb) {
    if (is_edge(jb)) {
      bool met = false;
#pragma unroll
      for (int n = 0; n < NL; ++n) met |= scrub<T>(kr[n]);
      scrubbed[buf][wave] = __any(met);
    }
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const int slot = tid + n * NT, row = slot / PPR, piece = slot % PPR;
      if (row < BN) {
        TL::template store<BN>(ks[buf], row, piece, kr[n]);
        TL::template store<BN>(vs[buf], row, piece, vr[n]);
      }
    }
  };
  if (jb0 < jb1) {
    if (!kEarly) load(jb0);
    if constexpr (BUFS == 2) store(0, jb0);
  }
  for (int jb = jb0; jb < jb1; ++jb) {
    __syncthreads();
    if constexpr (BUFS == 1) {
      store(0, jb);
      __syncthreads();
    }
    if (jb + 1 < jb1) load(jb + 1);
    const int buf = BUFS == 2 ? (jb - jb0) & 1 : 0;
    int met = 0;
    if (is_edge(jb)) {
#pragma unroll
      for (int w = 0; w < WAVES; ++w) met |= scrubbed[buf][w];
      met = __builtin_amdgcn_readfirstlane(met);
      if (met) {
        met_tiles |= 1u << (jb & 31);
        for (int b = 0; b < BN / 32; ++b)  // (every wave writes the same)
          bad_keys[buf][b] = rows_not_finite(kbase, a.k_row, wg.lo + jb * BN + 32 * b, sp.nk, a.dim, lane);
      }
    }
    for (int b = 0; b < BN / 32; ++b) {
      const int j0 = wg.lo + jb * BN + 32 * b;
      if (!wave_on || j0 >= wv.hi) break;
      if (j0 + 32 <= wv.lo) continue;
      floatx16 s(0.f), dp(0.f);
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        s = mma_frag<T>(TL::template row_frag<BN>(ks[buf], 32 * b + (lane & 31), 2 * t + half), qf[t], s);
        dp = mma_frag<T>(TL::template row_frag<BN>(vs[buf], 32 * b + (lane & 31), 2 * t + half), gf[t], dp);
      }
      float ds[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) ds[i] = fast_exp2(__builtin_fmaf(s[i], c, -lse2)) * (dp[i] - dot);
      if (j0 + 32 > full_hi) {
        keep_branch();
        const int end = lane_hi - j0 - 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = c_row(i) < end ? ds[i] : 0.f;
      }
      if (j0 < full_lo) {
        keep_branch();
        const int first = lane_lo - j0 - 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = c_row(i) >= first ? ds[i] : 0.f;
      }
      if (met) {
        keep_branch();
        const uint32_t bad = bad_keys[buf][b] >> (4 * half);
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i] = (bad >> c_row(i) & 1) == 0 ? ds[i] : 0.f;
      }
      rescale<T, DB>(ds, factor, acc);
      mma_transposed<T, DP, DB, BN>(ks[buf], 32 * b, lane, ds, acc);
      settle();
    }
    if (BUFS == 2 && jb + 1 < jb1) store(buf ^ 1, jb + 1);
  }
  if (met_tiles != 0) {
    for (int jb = jb0; jb < jb1; ++jb) {
      if ((met_tiles >> (jb & 31) & 1) == 0 || !is_edge(jb)) continue;
      for (int j0 = wg.lo + jb * BN; j0 < wg.lo + (jb + 1) * BN; j0 += 32) {
        for (uint32_t bad = rows_not_finite(kbase, a.k_row, j0, sp.nk, a.dim, lane); bad != 0; bad &= bad - 1) {
          const int j = j0 + __builtin_ctz(bad);
          if (!has_row || j < lane_lo || j >= lane_hi) continue;
          const T* src = kbase + j * a.k_row;
#pragma unroll
          for (int db = 0; db < DB; ++db)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int d = db * 32 + 4 * half + c_row(i);
              const float x = d < a.dim ? to_f32(src[d]) : 0.f;
              // 0 times the value, or a NaN of the row's lse
              acc[db][i] += 0.f * x + 0.f * lse2;
            }
        }
      }
    }
  }

  const float mul = __is_same(T, _Float16) ? a.scale / factor * 6.103515625e-05f : a.scale;
  if (nsplit == 1)
    store_row<T, DB>(static_cast<T*>(a.grad_q) + static_cast<int64_t>(sp.q0 + tok) * a.gq_row + static_cast<int64_t>(head) * a.gq_head, acc, mul,
                     half, a.dim, has_row);
  else
    store_row<float, DB>(part + (static_cast<int64_t>(split) * a.total_q * a.heads + row_out) * a.dim, acc, mul, half, a.dim, has_row);
}

template <class T, int DP, int DQ, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 && DP <= 64 ? 2 : 1) void k_attention_dkv(AttentionArgs a, int slots, int run, int nsplit, const int32_t* order, const float2* stats,
                                                              float* part_k, float* part_v) {
  typedef Tile<T, DP> TL;
  constexpr int BN = kWalk<T, DP, WAVES>, BUFS = kBuffers<WAVES>, PPR = TL::PPR, DB = DP / 32, NT = 64 * WAVES;
  constexpr int BM = 32 * WAVES, KS = DQ / (2 * kPiece), NL = (BN * PPR + NT - 1) / NT;
  constexpr int NR = (BN + NT - 1) / NT;  // rows whose statistics each thread copies
  __shared__ uint4 qs[BUFS][kPlanes<T> * BN * PPR], gs[BUFS][kPlanes<T> * BN * PPR];
  __shared__ float4 row_lse[BUFS][BN / 4], row_delta[BUFS][BN / 4];  // lse in log2 units and shifted, D
  __shared__ int4 row_place[BUFS][BN / 4];

  const int split = static_cast<int>(blockIdx.x) & (nsplit - 1), id = static_cast<int>(blockIdx.x) >> __builtin_ctz(nsplit);
  const Place at_block = place_of(a, id, run);
  if (at_block.slot >= slots) return;
  const int kvh = at_block.kvh;
  const Span sp = find_span(a, true, 1, tile_shift(WAVES), order != nullptr ? order[at_block.slot] : at_block.slot, slots);
  if (!sp.any) return;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = sp.nq * a.group;
  const int shift = sp.nk - sp.nq;

  const int kw0 = sp.r0 + 32 * wave;
  const int key = kw0 + (lane & 31);
  const bool has_key = key < sp.nk;
  const int64_t krow = static_cast<int64_t>(sp.k0 + (has_key ? key : 0));
  Frag<T> kf[KS], vf[KS];
  {
    const T* src = static_cast<const T*>(a.k) + krow * a.k_row + static_cast<int64_t>(kvh) * a.k_head;
    const T* vsrc = static_cast<const T*>(a.v) + krow * a.v_row + static_cast<int64_t>(kvh) * a.v_head;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const int e = (2 * t + half) * kPiece;
      const bool ok = has_key && e < a.dim;
      kf[t] = to_frag<T>(load_piece(src + e, ok));
      vf[t] = to_frag<T>(load_piece(vsrc + e, ok));
    }
  }
  // Query rows that see a key of the workgroup: place - left <= key <= place + right.
  const int kt1 = min(sp.r0 + BM, sp.nk);
  const int i_lo = a.right >= 0 ? max(sp.r0 - a.right - shift, 0) : 0;
  const int i_hi = a.left >= 0 ? min(kt1 + a.left - shift, sp.nq) : sp.nq;
  const int f_lo = i_lo * a.group, f_hi = i_hi * a.group;
  const int blocks = f_hi > f_lo ? (f_hi - f_lo + BN - 1) / BN : 0;
  const Share mine = share_of(blocks, split, nsplit);
  const int rb0 = mine.first, rb1 = mine.end;
  const bool wave_on = kw0 < sp.nk;
  const int kw1 = min(kw0 + 32, sp.nk) - 1;  // last key of the wave

  Raw<T> qr[NL], gr[NL];
  float lse_r[NR], delta_r[NR];
  int place_r[NR];
  const T* qbase = static_cast<const T*>(a.q) + static_cast<int64_t>(sp.q0) * a.q_row + static_cast<int64_t>(kvh) * a.group * a.q_head;
  const T* gbase = static_cast<const T*>(a.grad_out) + static_cast<int64_t>(sp.q0) * a.go_row + static_cast<int64_t>(kvh) * a.group * a.go_head;
  const float2* sbase = stats + (static_cast<int64_t>(kvh) * a.total_q + sp.q0) * a.group;
  const uint32_t qb = static_cast<uint32_t>(a.q_row * sizeof(T)), gb = static_cast<uint32_t>(a.go_row * sizeof(T));
  auto load = [&](int rb) {
    const int r0 = f_lo + rb * BN;
    if (a.group == 1) {
      // flattened rows are rows: the offsets within a tile are the same for all
      const auto qbuf = rows_buffer(qbase + r0 * a.q_row, rows - r0, qb), gbuf = rows_buffer(gbase + r0 * a.go_row, rows - r0, gb);
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const int slot = tid + n * NT, row = slot / PPR, piece = slot % PPR;
        const bool on = row < BN && piece * kPiece < a.dim;
        qr[n] = load_piece<T>(qbuf, on ? row * qb + piece * kPieceBytes<T> : kNowhere);
        gr[n] = load_piece<T>(gbuf, on ? row * gb + piece * kPieceBytes<T> : kNowhere);
      }
    } else {
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const int slot = tid + n * NT, row = slot / PPR, piece = slot % PPR;
        const int r = r0 + row;
        const bool on = row < BN && r < rows && piece * kPiece < a.dim;
        const int tok = div_group(a, on ? r : 0), g = on ? r - tok * a.group : 0;
        qr[n] = load_piece(qbase + tok * a.q_row + g * a.q_head + piece * kPiece, on);
        gr[n] = load_piece(gbase + tok * a.go_row + g * a.go_head + piece * kPiece, on);
      }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int r = r0 + tid + n * NT;
      lse_r[n] = INFINITY;
      delta_r[n] = 0.f;
      place_r[n] = INT_MIN;
      if (tid + n * NT < BN && r < rows) {
        const float2 st = sbase[r];
        lse_r[n] = st.x;
        delta_r[n] = st.y;
        place_r[n] = div_group(a, r) + shift;
      }
    }
  };
  // Rows that do not see every key of the workgroup go into LDS with their
  // infinities and NaN as zeros: the keys that they do see get NaN from their
  // lse (q) or D (grad_out, through the lse too: see the statistics).
  auto store = [&](int buf, int rb) {
    const int r0 = f_lo + rb * BN;
    const int p0 = div_group(a, r0) + shift, p1 = div_group(a, min(r0 + BN, rows) - 1) + shift;
    if ((a.right >= 0 && kt1 - 1 > p0 + a.right) || (a.left >= 0 && sp.r0 < p1 - a.left)) {
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        scrub<T>(qr[n]);
        scrub<T>(gr[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const int slot = tid + n * NT, row = slot / PPR, piece = slot % PPR;
      if (row < BN) {
        TL::template store<BN>(qs[buf], row, piece, qr[n]);
        TL::template store<BN>(gs[buf], row, piece, gr[n]);
      }
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = tid + n * NT;
      if (row < BN) {
        reinterpret_cast<float*>(row_lse[buf])[row] = lse_r[n];
        reinterpret_cast<float*>(row_delta[buf])[row] = delta_r[n];
        reinterpret_cast<int*>(row_place[buf])[row] = place_r[n];
      }
    }
  };

  floatx16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) {
    dk[db] = floatx16(0.f);
    dv[db] = floatx16(0.f);
  }
  float factor = kFirstFactor;
  const float c = a.scale * kLog2e;

  if (rb0 < rb1) {
    load(rb0);
    if constexpr (BUFS == 2) store(0, rb0);
  }
  for (int rb = rb0; rb < rb1; ++rb) {
    __syncthreads();
    if constexpr (BUFS == 1) {
      store(0, rb);
      __syncthreads();
    }
    if (rb + 1 < rb1) load(rb + 1);
    const int buf = BUFS == 2 ? (rb - rb0) & 1 : 0;
    for (int b = 0; b < BN / 32; ++b) {
      const int r0 = f_lo + rb * BN + 32 * b;
      if (!wave_on || r0 >= rows) break;
      const int p0 = div_group(a, r0) + shift, p1 = div_group(a, min(r0 + 32, rows) - 1) + shift;  // places of the block
      if (a.right >= 0 && kw0 > p1 + a.right) continue;
      if (a.left >= 0 && kw1 < p0 - a.left) break;
      floatx16 s(0.f), dp(0.f);
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        s = mma_frag<T>(TL::template row_frag<BN>(qs[buf], 32 * b + (lane & 31), 2 * t + half), kf[t], s);
        dp = mma_frag<T>(TL::template row_frag<BN>(gs[buf], 32 * b + (lane & 31), 2 * t + half), vf[t], dp);
      }
      float p[16], ds[16];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 ls = row_lse[buf][8 * b + 2 * g + half], de = row_delta[buf][8 * b + 2 * g + half];
        const float lv[4] = {ls.x, ls.y, ls.z, ls.w}, dv4[4] = {de.x, de.y, de.z, de.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = 4 * g + u;
          p[i] = fast_exp2(__builtin_fmaf(s[i], c, -lv[u]));
          ds[i] = p[i] * (dp[i] - dv4[u]);
        }
      }
      const bool cut_hi = a.right >= 0 && kw1 > p0 + a.right, cut_lo = a.left >= 0 && kw0 < p1 - a.left;
      if (cut_hi || cut_lo || r0 + 32 > rows) {
        keep_branch();
        // places from first to last see the key; rows past the end stand below
        // all: their scores with a key that is not finite are NaN (of a
        // zero), which their lse of +inf does not take out
        const int first = cut_hi ? key - a.right : INT_MIN + 1, last = cut_lo ? key + a.left : INT_MAX;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int4 pl = row_place[buf][8 * b + 2 * g + half];
          const int pv[4] = {pl.x, pl.y, pl.z, pl.w};
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bool seen = pv[u] >= first && pv[u] <= last;
            p[4 * g + u] = seen ? p[4 * g + u] : 0.f;
            ds[4 * g + u] = seen ? ds[4 * g + u] : 0.f;
          }
        }
      }
      mma_transposed<T, DP, DB, BN>(gs[buf], 32 * b, lane, p, dv);
      rescale<T, DB>(ds, factor, dk);
      mma_transposed<T, DP, DB, BN>(qs[buf], 32 * b, lane, ds, dk);
      settle();
    }
    if (BUFS == 2 && rb + 1 < rb1) store(buf ^ 1, rb + 1);
  }

  constexpr float unshift = __is_same(T, _Float16) ? 6.103515625e-05f : 1.f;  // 2^-14
  const float mul = __is_same(T, _Float16) ? a.scale / factor * unshift : a.scale;
  if (nsplit == 1) {
    store_row<T, DB>(static_cast<T*>(a.grad_k) + krow * a.gk_row + static_cast<int64_t>(kvh) * a.gk_head, dk, mul, half, a.dim, has_key);
    store_row<T, DB>(static_cast<T*>(a.grad_v) + krow * a.gv_row + static_cast<int64_t>(kvh) * a.gv_head, dv, unshift, half, a.dim, has_key);
  } else {
    const int64_t at = (static_cast<int64_t>(split) * a.total_k * a.kv_heads + krow * a.kv_heads + kvh) * a.dim;
    store_row<float, DB>(part_k + at, dk, mul, half, a.dim, has_key);
    store_row<float, DB>(part_v + at, dv, unshift, half, a.dim, has_key);
  }
}

// One tensor's partial gradients: [nsplit][rows][heads][dim].
struct JoinJob {
  const float* part = nullptr;
  int nsplit = 0;  // 1: nothing to join
  int64_t rows = 0;
  int heads = 0;
  void* dst = nullptr;
  int64_t row_stride = 0, head_stride = 0;
  unsigned first_block = 0;
};
struct JoinJobs {
  JoinJob job[3];
};

// Adds the splits' partial gradients in order and rounds once, for all three
// tensors in one launch; four columns per thread.
template <class T>
__global__ __launch_bounds__(256) void k_attention_grad_join(JoinJobs jobs, int dim) {
  const int which = blockIdx.x >= jobs.job[2].first_block ? 2 : blockIdx.x >= jobs.job[1].first_block ? 1 : 0;
  const JoinJob& j = jobs.job[which];
  const int quads = dim / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x - j.first_block) * 256 + threadIdx.x;
  const int64_t rh = id / quads;
  if (rh >= j.rows * j.heads) return;
  const int quad = static_cast<int>(id - rh * quads);
  const int64_t row = rh / j.heads;
  const int head = static_cast<int>(rh - row * j.heads);
  float x = 0.f, y = 0.f, z = 0.f, w = 0.f;
  for (int s = 0; s < j.nsplit; ++s) {
    const float4 v = *reinterpret_cast<const float4*>(j.part + (s * j.rows * j.heads + rh) * dim + 4 * quad);
    x += v.x;
    y += v.y;
    z += v.z;
    w += v.w;
  }
  store4<T>(static_cast<T*>(j.dst) + row * j.row_stride + head * j.head_stride + 4 * quad, x, y, z, w);
}

// Launches the join of the jobs that have parts.
template <class T>
hipError_t launch_joins(JoinJobs jobs, int dim, hipStream_t stream) {
  unsigned blocks = 0;
  for (JoinJob& j : jobs.job) {
    j.first_block = blocks;
    if (j.nsplit > 1) blocks += static_cast<unsigned>((j.rows * j.heads * (dim / 4) + 255) / 256);
  }
  if (blocks == 0) return hipSuccess;
  k_attention_grad_join<T><<<blocks, 256, 0, stream>>>(jobs, dim);
  return hipGetLastError();
}

__global__ __launch_bounds__(1024) void k_attention_grad_order(AttentionArgs a, OrderJob q, OrderJob k) {
  order_slots(a, blockIdx.x == 0 ? q : k);
}

struct Plan {
  int q_waves, k_waves;
  int64_t q_slots, k_slots;
  int q_split, k_split;
  bool ordered;
};

Plan make_backward_plan(const AttentionArgs& a) {
  Plan p;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.group;
  const int64_t batch = std::max(a.batch, 1);
  const Cut q = cut_rows(a, rows / batch, rows, band_depth(a, a.total_k / batch, 1));
  const Cut k = cut_rows(a, a.total_k / batch, a.total_k, band_depth(a, a.total_q / batch, a.group));
  p.q_waves = q.waves;
  p.k_waves = k.waves;
  p.q_split = q.split;
  p.k_split = k.split;
  p.q_slots = span_slots(rows, a.batch, 32 * p.q_waves);
  p.k_slots = span_slots(a.total_k, a.batch, 32 * p.k_waves);
  p.ordered = order_pays(a, p.q_slots, p.q_split, 7) && order_pays(a, p.k_slots, p.k_split, 7);
  return p;
}

// Workgroups of the query gradient and of the key and value gradients.
int64_t q_groups(const AttentionArgs& a, const Plan& p) { return placed_slots(p.q_slots, p.ordered ? 0 : slot_run(a, p.q_slots)) * a.kv_heads * p.q_split; }
int64_t k_groups(const AttentionArgs& a, const Plan& p) { return placed_slots(p.k_slots, p.ordered ? 0 : slot_run(a, p.k_slots)) * a.kv_heads * p.k_split; }

struct Workspace {
  size_t stats, q, k, v, q_order, k_order, total;  // offsets in bytes
};
Workspace layout(const AttentionArgs& a, const Plan& p) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const size_t nq = static_cast<size_t>(a.total_q) * a.heads, nk = static_cast<size_t>(a.total_k) * a.kv_heads;
  Workspace w;
  w.stats = 0;
  w.q = up(nq * sizeof(float2));
  w.k = w.q + (p.q_split > 1 ? up(nq * a.dim * p.q_split * sizeof(float)) : 0);
  const size_t part = p.k_split > 1 ? up(nk * a.dim * p.k_split * sizeof(float)) : 0;
  w.v = w.k + part;
  w.q_order = w.v + part;
  w.k_order = w.q_order + (p.ordered ? up(static_cast<size_t>(p.q_slots) * sizeof(int32_t)) : 0);
  w.total = w.k_order + (p.ordered ? up(static_cast<size_t>(p.k_slots) * sizeof(int32_t)) : 0);
  return w;
}

}  // namespace

uint64_t attention_backward_work_items(const AttentionArgs& a) {
  const Plan p = make_backward_plan(a);
  uint64_t join = 0;
  if (p.q_split > 1) join += static_cast<uint64_t>(a.total_q) * a.heads * (a.dim / 4) + 255;
  if (p.k_split > 1) join += 2 * (static_cast<uint64_t>(a.total_k) * a.kv_heads * (a.dim / 4) + 255);
  return std::max({join, static_cast<uint64_t>(q_groups(a, p)) * 64 * p.q_waves, static_cast<uint64_t>(k_groups(a, p)) * 64 * p.k_waves});
}

size_t attention_backward_workspace_bytes(const AttentionArgs& a) { return layout(a, make_backward_plan(a)).total; }

hipError_t launch_attention_backward(const AttentionArgs& a, void* workspace, hipStream_t stream) {
  const Plan p = make_backward_plan(a);
  const Workspace w = layout(a, p);
  char* base = static_cast<char*>(workspace);
  float2* stats = reinterpret_cast<float2*>(base + w.stats);
  float* part_q = reinterpret_cast<float*>(base + w.q);
  float* part_k = reinterpret_cast<float*>(base + w.k);
  float* part_v = reinterpret_cast<float*>(base + w.v);
  int32_t* q_order = p.ordered ? reinterpret_cast<int32_t*>(base + w.q_order) : nullptr;
  int32_t* k_order = p.ordered ? reinterpret_cast<int32_t*>(base + w.k_order) : nullptr;
  if (p.ordered) {
    const OrderJob q = {q_order, false, a.group, tile_shift(p.q_waves), static_cast<int>(p.q_slots)};
    const OrderJob k = {k_order, true, 1, tile_shift(p.k_waves), static_cast<int>(p.k_slots)};
    k_attention_grad_order<<<2, 1024, 0, stream>>>(a, q, k);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return dispatch(a, [&](auto t, auto dp, auto dq) -> hipError_t {
    typedef decltype(t) T;
    constexpr int DP = decltype(dp)::value, DQ = decltype(dq)::value;
    if (a.total_q > 0) {
      const int run = p.ordered ? 0 : slot_run(a, p.q_slots);
      const dim3 grid(static_cast<unsigned>(q_groups(a, p)));
      if (p.q_waves == 1) k_attention_dq<T, DP, DQ, 1><<<grid, 64, 0, stream>>>(a, static_cast<int>(p.q_slots), run, p.q_split, q_order, stats, part_q);
      else if (p.q_waves == 2) k_attention_dq<T, DP, DQ, 2><<<grid, 128, 0, stream>>>(a, static_cast<int>(p.q_slots), run, p.q_split, q_order, stats, part_q);
      else k_attention_dq<T, DP, DQ, 4><<<grid, 256, 0, stream>>>(a, static_cast<int>(p.q_slots), run, p.q_split, q_order, stats, part_q);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (a.total_k > 0) {
      const int run = p.ordered ? 0 : slot_run(a, p.k_slots);
      const dim3 grid(static_cast<unsigned>(k_groups(a, p)));
      if (p.k_waves == 1) k_attention_dkv<T, DP, DQ, 1><<<grid, 64, 0, stream>>>(a, static_cast<int>(p.k_slots), run, p.k_split, k_order, stats, part_k, part_v);
      else if (p.k_waves == 2) k_attention_dkv<T, DP, DQ, 2><<<grid, 128, 0, stream>>>(a, static_cast<int>(p.k_slots), run, p.k_split, k_order, stats, part_k, part_v);
      else k_attention_dkv<T, DP, DQ, 4><<<grid, 256, 0, stream>>>(a, static_cast<int>(p.k_slots), run, p.k_split, k_order, stats, part_k, part_v);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const JoinJobs jobs = {{{part_q, p.q_split, a.total_q, a.heads, a.grad_q, a.gq_row, a.gq_head},
                            {part_k, p.k_split, a.total_k, a.kv_heads, a.grad_k, a.gk_row, a.gk_head},
                            {part_v, p.k_split, a.total_k, a.kv_heads, a.grad_v, a.gv_row, a.gv_head}}};
    return launch_joins<T>(jobs, a.dim, stream);
  });
}

}  // namespace spconv
