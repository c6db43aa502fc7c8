// Softmax attention over packed sequences, forward.
//
//   s_ij = scale q_i . k_j over the visible keys j of query i's sequence,
//   lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j;
//   a query without visible keys gets 0 and lse = -inf.
//
// One pass over the keys with the running maximum and sum of the softmax in
// fp32 registers.  Per 32 queries x 64 keys a wave issues about 160 vector
// instructions (scale and subtract, exponential, sum, maximum, conversion; the
// exponential takes two slots) beside DP / 4 matrix ones, so heads of 32 are
// bound by the vector unit and heads of 128 by how the two units overlap.
// Measured: 4 sequences of up to 8192 rows, 16 heads of 128 over 4 key heads,
// causal bf16, 0.90 TFLOP of visible pairs: 1004 us, 897 TFLOP/s (matrix unit
// 42% busy, vector unit 41%); 8 frames of up to 4000 rows, 8 heads of 32, f16:
// 140 us, 522 TFLOP/s (vector unit 83% busy).
//
// A query tile is 32 rows per wave, the wave's columns in every product: its
// softmax needs one exchange between the lane halves and no LDS.  Computing
// the next tile's scores beside this tile's exponentials in one wave was tried
// and is slower: the second set of scores does not fit the 256 registers that
// two waves per SIMD leave.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "attention_common.h"

namespace spconv {
namespace {

using namespace attn;

// Keys per LDS tile, and tiles of K and V in LDS (two: one read, one filled;
// a lone wave stages through one).  Tiles are as large as several workgroups
// per CU allow: a short sequence then needs one tile, and one barrier, in all.
template <class T, int DP, int WAVES>
constexpr int kKeys = sizeof(T) == 4 ? 32 : DP == 32 ? (WAVES == 4 ? 128 : 64) : WAVES == 4 || (WAVES == 2 && DP == 64) ? 64 : 32;
template <int WAVES>
constexpr int kBuffers = WAVES == 1 ? 1 : 2;

// How the keys of few rows are cut: sequences of at most 32 flattened rows
// (and some keys) go over chunks of 2^shift keys, one wave each, found by the
// same slots on the key side; the workgroups after them take the sequences
// that are left, a tile of rows at a time.  Balanced whatever the lengths.
struct Chunks {
  int slots = 0;  // 0: no chunks
  int shift = 0;
  int rows = 0;  // flattened rows that a sequence of these has at most
};
__device__ __forceinline__ bool chunked(int rows, int nk) { return rows <= 32 && nk > 0; }

// One workgroup: 32 flattened query rows per wave, one kv head, and the key
// tiles of one split or chunk.  Q stays in registers (operand B of
// S^T = K Q^T), K and V pass through LDS, loaded a tile ahead into registers.
template <class T, int DP, int DQ, int WAVES>
__global__ __launch_bounds__(64 * WAVES, sizeof(T) == 2 ? 2 : 1) void k_attention(AttentionArgs a, int slots, int run, int nsplit,
                                                                                 Chunks chunks, const int32_t* order, float* part_out,
                                                                                 float* part_lse) {
  typedef Tile<T, DP> TL;
  constexpr int BN = kKeys<T, DP, WAVES>, BUFS = kBuffers<WAVES>;
  constexpr int NB = BN >= 64 ? 2 : 1;  // blocks of 32 keys per softmax step
  constexpr int PPR = TL::PPR, DB = DP / 32, NT = 64 * WAVES;
  constexpr int BM = 32 * WAVES;                // flattened rows per workgroup
  constexpr int KS = DQ / (2 * kPiece);      // pieces per half of a row
  constexpr int NL = (BN * PPR + NT - 1) / NT;  // pieces each thread copies per tile
  __shared__ uint4 ks[BUFS][kPlanes<T> * BN * PPR], vs[BUFS][kPlanes<T> * BN * PPR];
  __shared__ uint32_t scrubbed[WAVES];  // edge tiles in whose values the wave found infinities or NaN, by their number modulo 32

  // a tile's splits follow one another (nsplit is a power of two)
  const int split = static_cast<int>(blockIdx.x) & (nsplit - 1), id = static_cast<int>(blockIdx.x) >> __builtin_ctz(nsplit);
  int kvh, chunk0 = 0, chunk1 = INT_MAX;
  int64_t part_row = -1;  // of the chunk's first row; -1: not a chunk
  Span sp;
  if (WAVES == 1 && chunks.slots > 0) {
    const int slot = fast_div(id, a.by_kv_heads);
    kvh = id - slot * a.kv_heads;
    if (slot < chunks.slots) {
      sp = find_span(a, true, 1, chunks.shift, slot, chunks.slots);
      if (!sp.any || sp.nq == 0 || !chunked(sp.nq * a.group, sp.nk)) return;
      chunk0 = sp.r0;
      chunk1 = sp.r0 + (1 << chunks.shift);
      sp.r0 = 0;
      part_row = (static_cast<int64_t>(slot) * a.kv_heads + kvh) * chunks.rows;
    } else {
      sp = find_span(a, false, a.group, tile_shift(WAVES), slot - chunks.slots, slots);
      if (!sp.any || chunked(sp.nq * a.group, sp.nk)) return;
    }
  } else {
    // The longest tiles first: by the order given, or under a causal mask the
    // last rows, which have the most keys.
    const Place at = place_of(a, id, run);
    if (at.slot >= slots) return;
    kvh = at.kvh;
    const int slot = order != nullptr ? order[at.slot] : a.right >= 0 ? slots - 1 - at.slot : at.slot;
    sp = find_span(a, false, a.group, tile_shift(WAVES), slot, slots);
    if (!sp.any) return;
  }
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int rows = sp.nq * a.group;
  const int shift = sp.nk - sp.nq;  // a query's place among the keys: its row + shift

  // This lane's query row.
  const int wr0 = sp.r0 + 32 * wave;
  const int r = wr0 + (lane & 31);
  const bool has_row = r < rows;
  const int tok = div_group(a, has_row ? r : 0);
  const int head = kvh * a.group + (has_row ? r - tok * a.group : 0);
  Frag<T> qf[KS];
  {
    const T* src = static_cast<const T*>(a.q) + static_cast<int64_t>(sp.q0 + tok) * a.q_row + static_cast<int64_t>(head) * a.q_head;
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      const int piece = 2 * t + half;
      qf[t] = to_frag<T>(load_piece(src + piece * kPiece, has_row && piece * kPiece < a.dim));
    }
  }
  const int place = tok + shift;
  const int lane_lo = a.left >= 0 ? place - a.left : 0;
  const int key_end = WAVES == 1 ? min(sp.nk, chunk1) : sp.nk;
  const int lane_hi = a.right >= 0 ? min(place + a.right + 1, key_end) : key_end;
  // Keys that the workgroup's rows, and this wave's, see.
  KeyRange wg = key_range(a, sp.nk, div_group(a, sp.r0) + shift, div_group(a, min(sp.r0 + BM, rows) - 1) + shift);
  if (WAVES == 1) {
    wg.lo = max(wg.lo, chunk0);
    wg.hi = min(wg.hi, chunk1);
  }
  const bool wave_on = wr0 < rows;
  const int wp0 = div_group(a, wave_on ? wr0 : 0) + shift, wp1 = div_group(a, wave_on ? min(wr0 + 32, rows) - 1 : 0) + shift;
  KeyRange wv = key_range(a, sp.nk, wp0, wp1);
  if (WAVES == 1) wv.hi = min(wv.hi, chunk1);
  const int full_lo = a.left >= 0 ? wp1 - a.left : 0;                        // keys from here on,
  const int full_hi = a.right >= 0 ? min(wp0 + a.right + 1, key_end) : key_end;  // and below here, every row of the wave sees

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
  // Edge tiles hold keys that some row of the workgroup does not see: their
  // values that are not finite go into LDS as zeros, and reach the rows that
  // see them after the loop.  What lies past the sequence's end is zero as
  // loaded, unless the rows repeat one.  In fp32 every tile is one: a
  // probability's lower planes are zeros too, and times an infinity NaN (32.8
  // against 31.8 us for 5 sequences of up to 2500 rows in a band of 200, 6
  // heads of 40).
  const int edge_end = key_end == sp.nk && a.v_row != 0 ? INT_MAX : key_end;
  const int edge_hi = a.right >= 0 ? min(div_group(a, sp.r0) + shift + a.right + 1, edge_end) : edge_end;
  const int edge_lo = a.left >= 0 ? div_group(a, min(sp.r0 + BM, rows) - 1) + shift - a.left : 0;
  auto is_edge = [&](int jb) { return sizeof(T) == 4 || wg.lo + (jb + 1) * BN > edge_hi || wg.lo + jb * BN < edge_lo; };
  auto store = [&](int buf, int jb) {
    if (is_edge(jb)) {
      bool met = false;
#pragma unroll
      for (int n = 0; n < NL; ++n) met |= scrub<T>(vr[n]);
      if (__any(met)) scrubbed[wave] |= 1u << (jb & 31);
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

  floatx16 acc[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) acc[db] = floatx16(0.f);
  float m = -INFINITY, l = 0.f;  // maximum (in log2 units, see below) and this half's sum
  const float c = a.scale * kLog2e;

  if (jb0 < jb1) {
    load(jb0);
    scrubbed[wave] = 0;
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
    for (int step = 0; step < BN / 32; step += NB) {
      const int j0 = wg.lo + jb * BN + 32 * step;
      if (!wave_on || j0 >= wv.hi) break;
      if (j0 + 32 * NB <= wv.lo) continue;
      floatx16 s[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        s[b] = floatx16(0.f);
#pragma unroll
        for (int t = 0; t < KS; ++t)
          s[b] = mma_frag<T>(TL::template row_frag<BN>(ks[buf], 32 * (step + b) + (lane & 31), 2 * t + half), qf[t], s[b]);
      }
      if (j0 + 32 * NB > full_hi) {
        keep_branch();
        const int end = lane_hi - j0 - 4 * half;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + c_row(i) < end ? s[b][i] : -INFINITY;
      }
      if (j0 < full_lo) {
        keep_branch();
        const int first = lane_lo - j0 - 4 * half;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[b][i] = 32 * b + c_row(i) >= first ? s[b][i] : -INFINITY;
      }
      float top = s[0][0];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
      const float m_new = fmaxf(m, halves_max(top) * c);
      // The sums are rescaled only when a row's maximum has grown by more than
      // 2^8: until then its terms stay below 2^8 times the largest.
      if (__any(m_new > m + 8.f)) {
        const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m - m_new);
        l *= alpha;
#pragma unroll
        for (int db = 0; db < DB; ++db)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[db][i] *= alpha;
        m = m_new;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          p[i] = fast_exp2(__builtin_fmaf(s[b][i], c, -base));
          l += p[i];
        }
        mma_transposed<T, DP, DB, BN>(vs[buf], 32 * (step + b), lane, p, acc);
      }
      settle();
    }
    if (BUFS == 2 && jb + 1 < jb1) store(buf ^ 1, jb + 1);
  }

  if (jb0 < jb1) {
    uint32_t met = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) met |= scrubbed[w];  // (a barrier has passed since the last was set)
    met = __builtin_amdgcn_readfirstlane(static_cast<int>(met));
    if (__builtin_expect(met != 0, 0)) {
      for (int jb = jb0; jb < jb1; ++jb) {
        if ((met >> (jb & 31) & 1) == 0 || !is_edge(jb)) continue;
#pragma unroll 1
        for (int j0 = wg.lo + jb * BN; j0 < wg.lo + (jb + 1) * BN; j0 += 32) {
          for (uint32_t bad = rows_not_finite(vbase, a.v_row, j0, sp.nk, a.dim, lane); bad != 0; bad &= bad - 1) {
            const int j = j0 + __builtin_ctz(bad);
            if (!has_row || j < lane_lo || j >= lane_hi) continue;
            const T* src = vbase + j * a.v_row;
#pragma unroll
            for (int db = 0; db < DB; ++db)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int d = db * 32 + 4 * half + c_row(i);
                const float x = d < a.dim ? to_f32(src[d]) : 0.f;
                acc[db][i] += fabsf(x) < INFINITY ? 0.f : x;
              }
          }
        }
      }
    }
  }
  const float sum = halves_sum(l);
  // Without a term: 0 for a row that sees no key; NaN for one whose scores are
  // all -inf, or whose largest is beyond fp32.  (A part of such scores counts
  // as -inf when it is joined.)  A NaN stays one.
  const bool none = max(lane_lo, WAVES == 1 ? chunk0 : 0) >= lane_hi;
  const float inv = sum > 0.f ? 1.f / sum : sum == 0.f && none ? 0.f : __builtin_nanf("");
  const float lse = sum == 0.f ? (m == INFINITY ? __builtin_nanf("") : -INFINITY) : ln_scaled(m, sum);
  const int64_t row_out = static_cast<int64_t>(sp.q0 + tok) * a.heads + head;
  if (nsplit == 1 && (WAVES > 1 || part_row < 0)) {
    if (has_row && half == 0) a.lse[row_out] = lse;
    store_row<T, DB>(static_cast<T*>(a.out) + row_out * a.dim, acc, inv, half, a.dim, has_row);
  } else {
    const int64_t at_out = WAVES == 1 && part_row >= 0 ? part_row + r : static_cast<int64_t>(split) * a.total_q * a.heads + row_out;
    if (has_row && half == 0) part_lse[at_out] = lse;
    store_row<float, DB>(part_out + at_out * a.dim, acc, inv, half, a.dim, has_row);
  }
}

// Joins parts of one output row: out = sum_p exp(lse_p - lse) out_p, for the
// rows first, first + step, ... of the parts.  A workgroup of 256: dim / 4
// lanes take 4 columns each, in 256 / (dim / 4) interleaved groups of parts,
// whose sums are added in a fixed order.
template <class T>
__device__ __forceinline__ void join_parts(const AttentionArgs& a, const float* part_out, const float* part_lse, int64_t first,
                                           int64_t step, int parts, int64_t row_out) {
  __shared__ float4 acc_s[256];
  __shared__ float top_s[256], sum_s[256], blank_s[256];
  const int quads = a.dim / 4, groups = 256 / quads, g = static_cast<int>(threadIdx.x) / quads, quad = static_cast<int>(threadIdx.x) - g * quads;
  float top = -INFINITY, sum = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  float blank = 0.f;  // NaN if the row sees a key in a part without a term
  constexpr int kBatch = 4;  // parts whose loads are issued together
  for (int p0 = g; g < groups && p0 < parts; p0 += kBatch * groups) {
    float ls[kBatch];
    float4 o[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t row = first + min(p0 + i * groups, parts - 1) * step;
      ls[i] = part_lse[row];
      o[i] = *reinterpret_cast<const float4*>(part_out + row * a.dim + 4 * quad);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (p0 + i * groups >= parts) continue;
      if (ls[i] == -INFINITY) {
        blank += o[i].x;
        continue;
      }
      const float now = fmaxf(top, ls[i]);
      const float keep = fast_exp2((top - now) * kLog2e), e = fast_exp2((ls[i] - now) * kLog2e);
      top = now;
      sum = sum * keep + e;
      x.x = x.x * keep + e * o[i].x;
      x.y = x.y * keep + e * o[i].y;
      x.z = x.z * keep + e * o[i].z;
      x.w = x.w * keep + e * o[i].w;
    }
  }
  acc_s[threadIdx.x] = x;
  top_s[threadIdx.x] = top;
  sum_s[threadIdx.x] = sum;
  blank_s[threadIdx.x] = blank;
  __syncthreads();
  if (g != 0) return;
  float all = -INFINITY;
  for (int q = 0; q < groups; ++q) all = fmaxf(all, top_s[q * quads + quad]);
  sum = 0.f;
  x = make_float4(0.f, 0.f, 0.f, 0.f);
  blank = 0.f;
  for (int q = 0; q < groups; ++q) {
    blank += blank_s[q * quads + quad];
    // A group without parts has a sum of 0.  (Its maximum does not tell: parts
    // whose lse is NaN leave that at -inf as well, and must reach the row.)
    if (sum_s[q * quads + quad] == 0.f) continue;
    const float e = fast_exp2((top_s[q * quads + quad] - all) * kLog2e);
    const float4 o = acc_s[q * quads + quad];
    sum += e * sum_s[q * quads + quad];
    x.x += e * o.x;
    x.y += e * o.y;
    x.z += e * o.z;
    x.w += e * o.w;
  }
  const float inv = sum == 0.f ? blank : 1.f / sum;
  store4<T>(static_cast<T*>(a.out) + row_out * a.dim + 4 * quad, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (quad == 0) a.lse[row_out] = sum == 0.f ? -INFINITY : all + ln_scaled(0.f, sum);
}

// Splits: part s of row r is at s x rows + r.  Few parts of many rows: four
// columns per thread.
template <class T>
__global__ __launch_bounds__(256) void k_attention_join(AttentionArgs a, int nsplit, const float* part_out,
                                                        const float* part_lse) {
  const int quads = a.dim / 4;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.heads;
  const int64_t row = id / quads;
  if (row >= rows) return;
  const int quad = static_cast<int>(id - row * quads);
  float top = -INFINITY;
  for (int s = 0; s < nsplit; ++s) top = fmaxf(top, part_lse[s * rows + row]);
  float sum = 0.f, blank = 0.f;  // blank: NaN if the row sees a key in a part without a term
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s = 0; s < nsplit; ++s) {
    const float ls = part_lse[s * rows + row];
    float4 o = *reinterpret_cast<const float4*>(part_out + (s * rows + row) * a.dim + 4 * quad);
    float e = fast_exp2((ls - top) * kLog2e);
    if (ls == -INFINITY) {
      blank += o.x;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      e = 0.f;
    }
    sum += e;
    x.x += e * o.x;
    x.y += e * o.y;
    x.z += e * o.z;
    x.w += e * o.w;
  }
  const float inv = sum == 0.f ? blank : 1.f / sum;
  store4<T>(static_cast<T*>(a.out) + row * a.dim + 4 * quad, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
  if (quad == 0) a.lse[row] = sum == 0.f ? -INFINITY : top + ln_scaled(0.f, sum);
}

// Chunks: one workgroup per query row and head.
template <class T>
__global__ __launch_bounds__(256) void k_attention_join_chunks(AttentionArgs a, Chunks chunks, const float* part_out,
                                                               const float* part_lse) {
  const int head = static_cast<int>(blockIdx.y);
  const Span sp = find_span(a, false, 1, 0, static_cast<int>(blockIdx.x), a.total_q + a.batch + 2);
  if (!sp.any || !chunked(sp.nq * a.group, sp.nk)) return;
  const int kvh = div_group(a, head), r = sp.r0 * a.group + head - kvh * a.group;
  const int slot0 = (sp.k0 >> chunks.shift) + sp.seq;
  const int parts = (sp.nk + (1 << chunks.shift) - 1) >> chunks.shift;
  join_parts<T>(a, part_out, part_lse, (static_cast<int64_t>(slot0) * a.kv_heads + kvh) * chunks.rows + r,
                static_cast<int64_t>(a.kv_heads) * chunks.rows, parts, static_cast<int64_t>(sp.q0 + sp.r0) * a.heads + head);
}

__global__ __launch_bounds__(1024) void k_attention_order(AttentionArgs a, OrderJob job) { order_slots(a, job); }

struct Plan {
  int waves;
  int64_t slots;
  int nsplit;
  Chunks chunks;
  int64_t parts;  // rows of the partial outputs
  bool ordered = false;
};

// Sequences of few rows over long keys (32 flattened rows in the mean, keys
// that fill a chunk) go by chunks: 24 single queries over up to 24000 keys,
// 16 heads of 128 over 2, bf16, 311 MB: 79 us with the join (4.0 TB/s),
// against 130 us when every sequence's keys are cut into the same number of
// parts.  Else the tiles of rows split the keys when they would leave SIMDs
// idle.
Plan make_forward_plan(const AttentionArgs& a) {
  Plan p;
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.group;
  const int64_t batch = std::max(a.batch, 1), mean = rows / batch, keys = a.total_k / batch;
  const Cut cut = cut_rows(a, mean, rows, band_depth(a, keys, 1));
  p.waves = cut.waves;
  p.nsplit = 1;
  p.parts = 0;
  if (p.waves == 1 && keys >= 256) {
    // about 4096 waves: two per SIMD, twice over
    const int64_t want = static_cast<int64_t>(a.total_k) * a.kv_heads / 4096;
    p.chunks.shift = 6;
    while (p.chunks.shift < 10 && (int64_t(1) << p.chunks.shift) < want) ++p.chunks.shift;
    p.chunks.slots = static_cast<int>(span_slots(a.total_k, a.batch, 1 << p.chunks.shift));
    p.slots = span_slots(rows, a.batch, 32);
    p.chunks.rows = static_cast<int>(std::min<int64_t>(rows, 32));
    p.parts = static_cast<int64_t>(p.chunks.slots) * a.kv_heads * p.chunks.rows;
    return p;
  }
  p.slots = span_slots(rows, a.batch, 32 * p.waves);
  p.nsplit = cut.split;
  if (p.nsplit > 1) p.parts = static_cast<int64_t>(p.nsplit) * a.total_q * a.heads;
  p.ordered = order_pays(a, p.slots, p.nsplit, 2);
  return p;
}

// Workgroups of the attention kernel.
int64_t forward_groups(const AttentionArgs& a, const Plan& p) {
  const int64_t placed = p.chunks.slots > 0 ? p.chunks.slots + p.slots : placed_slots(p.slots, p.ordered ? 0 : slot_run(a, p.slots));
  return placed * a.kv_heads * p.nsplit;
}

}  // namespace

uint64_t attention_work_items(const AttentionArgs& a) {
  const Plan p = make_forward_plan(a);
  const uint64_t groups = static_cast<uint64_t>(forward_groups(a, p)) * 64 * p.waves;
  const uint64_t rows = static_cast<uint64_t>(a.total_q) * a.heads;
  const uint64_t join = p.chunks.slots > 0 ? (static_cast<uint64_t>(a.total_q) + a.batch + 2) * 256 : p.nsplit > 1 ? rows * (a.dim / 4) + 255 : 0;
  return std::max(groups, join);
}

size_t attention_workspace_bytes(const AttentionArgs& a) {
  const Plan p = make_forward_plan(a);
  return static_cast<size_t>(p.parts) * (a.dim + 1) * sizeof(float) + (p.ordered ? static_cast<size_t>(p.slots) * sizeof(int32_t) : 0);
}

hipError_t launch_attention(const AttentionArgs& a, void* workspace, hipStream_t stream) {
  const Plan p = make_forward_plan(a);
  float* part_out = static_cast<float*>(workspace);
  float* part_lse = part_out + p.parts * a.dim;
  int32_t* order = p.ordered ? reinterpret_cast<int32_t*>(part_lse + p.parts) : nullptr;
  if (p.ordered) {
    const OrderJob job = {order, false, a.group, tile_shift(p.waves), static_cast<int>(p.slots)};
    k_attention_order<<<1, 1024, 0, stream>>>(a, job);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return dispatch(a, [&](auto t, auto dp, auto dq) -> hipError_t {
    typedef decltype(t) T;
    constexpr int DP = decltype(dp)::value, DQ = decltype(dq)::value;
    const int run = p.ordered ? 0 : slot_run(a, p.slots), slots = static_cast<int>(p.slots);
    const dim3 grid(static_cast<unsigned>(forward_groups(a, p)));
    if (p.waves == 1) k_attention<T, DP, DQ, 1><<<grid, 64, 0, stream>>>(a, slots, run, p.nsplit, p.chunks, order, part_out, part_lse);
    else if (p.waves == 2) k_attention<T, DP, DQ, 2><<<grid, 128, 0, stream>>>(a, slots, run, p.nsplit, p.chunks, order, part_out, part_lse);
    else k_attention<T, DP, DQ, 4><<<grid, 256, 0, stream>>>(a, slots, run, p.nsplit, p.chunks, order, part_out, part_lse);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.parts == 0) return e;
    if (p.chunks.slots > 0) {
      const dim3 rows(static_cast<unsigned>(a.total_q + a.batch + 2), static_cast<unsigned>(a.heads));
      k_attention_join_chunks<T><<<rows, 256, 0, stream>>>(a, p.chunks, part_out, part_lse);
    } else {
      const int64_t quads = static_cast<int64_t>(a.total_q) * a.heads * (a.dim / 4);
      k_attention_join<T><<<static_cast<unsigned>((quads + 255) / 256), 256, 0, stream>>>(a, p.nsplit, part_out, part_lse);
    }
    return hipGetLastError();
  });
}

}  // namespace spconv
