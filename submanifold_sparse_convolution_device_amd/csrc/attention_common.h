// Shared device code of the attention kernels (attention.hip,
// attention_backward.hip): MFMA operands, LDS tiles, and the cut of packed
// sequences into tiles of rows.
//
// Every product is a 32 x 32 MFMA tile C[m][n] = sum_k A[m][k] B[k][n], with
// C in 16 registers per lane: lane l holds column n = l mod 32 and rows
// m = 8 (i / 4) + 4 (l / 32) + i mod 4.  The contracted index may run in any
// order that A and B share, and the kernels choose it so that a C tile (of
// scores) is the B operand of the next product as it stands:
// step s, half h = l / 32, element j is row 16 s + 8 (j / 4) + 4 h + j mod 4,
// the C rows of registers 8 s + j.  So the products run transposed:
// S^T = K Q^T puts a query in each lane's column (its softmax needs one
// exchange, between the halves), and O^T = V^T P^T takes P^T from registers
// and V^T through the transposing LDS read.
//
// fp32 runs on the bf16 matrix unit, 16 times the rate of the fp32 one: a
// value splits exactly into three bf16 planes of 8 significant bits (each the
// nearest to what is left: x = hi + mid + lo, for x in [1, 2) |mid| <= 2^-8 and
// |lo| <= 2^-17), and a product is the six of the nine plane products
// that reach 2^-24 of it, summed in fp32:
//   hi hi + (hi mid + mid hi) + (hi lo + mid mid + lo hi);
// what is left out is at most 2 x 2^-8 x 2^-17 = 2^-24 of |a b|, half a unit
// of fp32's rounding, and of either sign.
// Against products on the fp32 matrix unit: a band of 200 rows over heads of
// 40 takes 30.5 us instead of 40, frames of 24 channels with gradients 104
// instead of 143.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"

namespace spconv {
namespace attn {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// What the two constants' roundings leave.
constexpr float kLog2eRest = static_cast<float>(1.4426950408889634 - static_cast<double>(kLog2e));
constexpr float kLn2Rest = static_cast<float>(0.6931471805599453 - static_cast<double>(kLn2));

// bf16 planes that hold one operand (fp32: three).
template <class T>
constexpr int kPlanes = sizeof(T) == 4 ? 3 : 1;
// A piece is 8 consecutive values: 16 bytes of each plane.
constexpr int kPiece = 8;

template <class T>
__device__ __forceinline__ float to_f32(T v) {
  return static_cast<float>(v);
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// ln(2^m x sum), rounded about once: the logarithm is taken of the mantissa
// and the parts are multiplied by ln 2 before they are added.  (m plus the
// unit's log2 of the whole sum, times ln 2, is too low by half of 2^-24 of the
// result in the mean, and so were all gradients too large by 2 to 3 x 10^-7:
// their error in fp32, over frames of 24 channels, is 4.2 x 10^-7 instead of
// 5.1.)  0 gives -inf, by the caller.
__device__ __forceinline__ float ln_scaled(float m, float sum) {
  const float mant = __builtin_amdgcn_logf(__builtin_amdgcn_frexp_mantf(sum)), e = static_cast<float>(__builtin_amdgcn_frexp_expf(sum));
  const float small = __builtin_fmaf(mant, kLn2, __builtin_fmaf(m + e, kLn2Rest, e * kLn2));
  return __builtin_fmaf(m, kLn2, small);
}
// x log2(e), rounded once.
__device__ __forceinline__ float log2_units(float x) { return __builtin_fmaf(x, kLog2e, x * kLog2eRest); }

// max / sum of a value over the two halves (lanes l and l xor 32).
struct HalfPair {
  float lo, hi;
};
__device__ __forceinline__ HalfPair halves(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t lo = r[0], hi = r[1];  // scalars first: a bit cast of a vector's element reads element 0
  return {__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)};
}
__device__ __forceinline__ float halves_max(float v) {
  const HalfPair p = halves(v);
  return fmaxf(p.lo, p.hi);
}
__device__ __forceinline__ float halves_sum(float v) {
  const HalfPair p = halves(v);
  return p.lo + p.hi;
}

// Reads of a tile's rows: a buffer over the rows that are left, so that rows
// past a sequence's end, and pieces past the head size (offset kNowhere),
// come back as zeros from the load's own bounds check.
constexpr uint32_t kBufferWord3 = 0x00020000;
constexpr uint32_t kNowhere = 0x80000000u;
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_buffer(const void* base, int rows_left, uint32_t row_bytes) {
  // rows that repeat one row (stride 0) have no end
  const uint64_t bytes = row_bytes == 0 ? 0x7fffffffull : static_cast<uint64_t>(max(rows_left, 0)) * row_bytes;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, static_cast<int>(min(bytes, static_cast<uint64_t>(0x7fffffff))),
                                           kBufferWord3);
}
// A piece as it lies in memory.
template <class T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
template <class T>
constexpr uint32_t kPieceBytes = kPiece * sizeof(T);

template <class T>
__device__ __forceinline__ Raw<T> load_piece(__amdgpu_buffer_rsrc_t rsrc, uint32_t offset) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    r.v[i] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, static_cast<int>(offset + 16 * i), 0, 0));
  return r;
}
template <class T>
__device__ __forceinline__ Raw<T> load_piece(const T* src, bool on) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    r.v[i] = on ? reinterpret_cast<const uint4*>(src)[i] : make_uint4(0, 0, 0, 0);
  return r;
}

// Sets the infinities and NaN of a piece to zero and returns whether there
// were any.  For rows that some of a tile's columns do not see: in a matrix
// product even a factor of zero would make NaN of them.
template <class T>
__device__ __forceinline__ bool scrub(Raw<T>& r) {
  constexpr uint32_t top = sizeof(T) == 4 ? 0x7f800000u : __is_same(T, _Float16) ? 0x7c007c00u : 0x7f807f80u;  // exponents
  constexpr uint32_t carry = sizeof(T) == 4 ? 0x00800000u : __is_same(T, _Float16) ? 0x04000400u : 0x00800080u;
  uint32_t any = 0;
  auto clean = [&](uint32_t w) {
    // an exponent of ones carries into the sign's place
    const uint32_t bad = ((w & top) + carry) & (sizeof(T) == 4 ? 0x80000000u : 0x80008000u);
    any |= bad;
    return w & ~(sizeof(T) == 4 ? static_cast<uint32_t>(static_cast<int32_t>(bad) >> 31) : (bad >> 15) * 0xffffu);
  };
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    r.v[i] = make_uint4(clean(r.v[i].x), clean(r.v[i].y), clean(r.v[i].z), clean(r.v[i].w));
  return any != 0;
}

// Which of the 32 rows row0 .. row0 + 31 (below `end`) of a tensor hold an
// infinity or NaN, as bits; for the rare tile that holds one somewhere.
template <class T>
__device__ __forceinline__ uint32_t rows_not_finite(const T* base, int64_t row_stride, int row0, int end, int dim, int lane) {
  asm volatile("" : "+v"(lane));  // keeps the addresses out of the registers of the loop around the rare call
  const int row = row0 + (lane & 31);
  bool bad = false;
  if (row < end) {
    for (int e = (lane >> 5) * kPiece; e < dim; e += 2 * kPiece) {
      Raw<T> r = load_piece(base + row * row_stride + e, true);
      bad |= scrub<T>(r);
    }
  }
  const uint64_t both = __ballot(bad);
  return static_cast<uint32_t>(both | both >> 32);
}

// A piece as an operand: one register quad per plane.
template <class T>
struct Frag {
  uint4 v[kPlanes<T>];
};

// The three planes of two fp32 values, two bf16 in a word each, rounded to
// nearest: what a plane leaves is at most half a unit of it, with a sign of
// its own (planes cut off towards zero leave twice as much in the first and
// the second, all of the value's sign, so that sums drift).  Values that
// round to a bf16 infinity keep the largest bf16 instead; an infinity or NaN
// has a NaN in its last plane, which makes NaN of all that it meets.
struct Split2 {
  uint32_t hi, mid, lo;
};
template <bool FINITE>
__device__ __forceinline__ Split2 split2(float x, float y) {
  typedef float floatx2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  constexpr float top = 3.3895313892515355e38f;  // the largest bf16
  auto pair = [](float f, float g) { return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{f, g}), bf16x2)); };
  auto first = [](uint32_t w) { return __builtin_bit_cast(float, w << 16); };
  auto second = [](uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); };
  Split2 r;
  r.hi = FINITE ? pair(x, y) : pair(__builtin_amdgcn_fmed3f(x, -top, top), __builtin_amdgcn_fmed3f(y, -top, top));
  const float rx = x - first(r.hi), ry = y - second(r.hi);  // exact
  r.mid = pair(rx, ry);
  r.lo = pair(rx - first(r.mid), ry - second(r.mid));  // exact
  return r;
}
template <bool FINITE>
__device__ __forceinline__ Frag<float> split8(const float (&x)[8]) {
  const Split2 a = split2<FINITE>(x[0], x[1]), b = split2<FINITE>(x[2], x[3]), c = split2<FINITE>(x[4], x[5]), d = split2<FINITE>(x[6], x[7]);
  Frag<float> f;
  f.v[0] = make_uint4(a.hi, b.hi, c.hi, d.hi);
  f.v[1] = make_uint4(a.mid, b.mid, c.mid, d.mid);
  f.v[2] = make_uint4(a.lo, b.lo, c.lo, d.lo);
  return f;
}
template <class T>
__device__ __forceinline__ Frag<T> to_frag(const Raw<T>& r) {
  if constexpr (sizeof(T) == 4) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 q = r.v[i / 4];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      x[i] = __builtin_bit_cast(float, w[i & 3]);
    }
    return split8<false>(x);
  } else {
    return {{r.v[0]}};
  }
}
// The operand of 8 values held in fp32 (rounded to T, or split).
template <class T>
__device__ __forceinline__ Frag<T> make_frag(const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    return split8<true>(x);
  } else {
    typedef T tx8 __attribute__((ext_vector_type(8)));
    tx8 b;
#pragma unroll
    for (int j = 0; j < 8; ++j) b[j] = static_cast<T>(x[j]);
    return {{__builtin_bit_cast(uint4, b)}};
  }
}

// C += A B over one piece per lane of each operand (half h's is piece
// 2 t + h of the row): 16 contracted values.
template <class T>
__device__ __forceinline__ floatx16 mma_frag(const Frag<T>& a, const Frag<T>& b, floatx16 c) {
  if constexpr (__is_same(T, _Float16)) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, a.v[0]), __builtin_bit_cast(half8, b.v[0]), c, 0, 0, 0);
  } else {
    auto term = [&](int i, int j) {
      c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.v[i]), __builtin_bit_cast(bf16x8, b.v[j]), c, 0, 0, 0);
    };
    if constexpr (sizeof(T) == 4) {
      term(2, 0);
      term(1, 1);
      term(0, 2);
      term(1, 0);
      term(0, 1);
    }
    term(0, 0);
    return c;
  }
}

// A tile of rows in LDS, DP elements each, in 16-byte pieces whose index is
// XOR-ed with a function of the row.  LDS serves 256 bytes (16 pieces) a
// clock to 16-byte reads and half of that to the transposing 8-byte ones: the
// swizzle puts one piece of 16 consecutive rows, 4 pieces of 4 rows and 2
// pieces of 8 rows (what a transposing read takes in 2 clocks) at 16
// different places modulo 256 bytes.  Measured per CU: 174 bytes a clock at
// 128 bf16 columns, against 16 for rows laid out plainly.
template <class T, int DP>
struct Tile {
  static constexpr int PPR = DP / kPiece;  // pieces per row
  static_assert(PPR % 4 == 0, "rows of whole 64-byte groups");
  __device__ static __forceinline__ int swz(int row) {
    if constexpr (PPR % 16 == 0) return (row & 3) << 2 | (row >> 2 & 1) << 1 | (row >> 3 & 1);
    if constexpr (PPR % 8 == 0) return (row >> 1 & 1) << 2 | (row >> 2 & 1) << 1 | (row >> 3 & 1);
    return (row >> 2 & 1) << 1 | (row >> 3 & 1);
  }
  __device__ static __forceinline__ int at(int row, int piece) { return row * PPR + (piece ^ swz(row)); }
  // A operand by rows: lane's row (m) and piece, of a tile of ROWS rows.
  template <int ROWS>
  __device__ static __forceinline__ Frag<T> row_frag(const uint4* lds, int row, int piece) {
    Frag<T> f;
#pragma unroll
    for (int p = 0; p < kPlanes<T>; ++p) f.v[p] = lds[p * ROWS * PPR + at(row, piece)];
    return f;
  }
  template <int ROWS>
  __device__ static __forceinline__ void store(uint4* lds, int row, int piece, const Raw<T>& r) {
    const Frag<T> f = to_frag<T>(r);
#pragma unroll
    for (int p = 0; p < kPlanes<T>; ++p) lds[p * ROWS * PPR + at(row, piece)] = f.v[p];
  }
};

// C tiles of one contraction over the 32 rows row0 .. row0 + 31 of a tile:
// acc[d][n] += sum_row tile[row][d] p[row][n] for DB blocks of 32 columns d;
// p in C layout.  16-bit types round p to T (an operand of the matrix
// instruction; the sums stay in fp32).
template <class T, int DP, int DB, int ROWS>
__device__ __forceinline__ void mma_transposed(const uint4* lds, int row0, int lane, const float (&p)[16],
                                               floatx16 (&acc)[DB]) {
  typedef Tile<T, DP> TL;
  const int g = lane & 15;
  // Lane g of a group of 16 addresses 4 columns of row g / 4; it receives
  // column g of the four rows.
  const int row = row0 + 4 * (lane >> 5) + (g >> 2);
  const int col = ((lane >> 4) & 1) * 16 + 4 * (g & 3);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = p[8 * s + j];
    const Frag<T> b = make_frag<T>(x);
#pragma unroll
    for (int db = 0; db < DB; ++db) {
      const int c = db * 32 + col;
      Frag<T> a;
#pragma unroll
      for (int q = 0; q < kPlanes<T>; ++q) {
        uint2 half[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const char* src = reinterpret_cast<const char*>(lds + q * ROWS * TL::PPR + TL::at(row + 16 * s + 8 * u, c / 8)) + (c & 4) * 2;
          half[u] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)src));
        }
        a.v[q] = make_uint4(half[0].x, half[0].y, half[1].x, half[1].y);
      }
      acc[db] = mma_frag<T>(a, b, acc[db]);
    }
  }
}

// Ends a step whose last instructions are matrix products: waits until their
// sums can be read.  The hardware does not hold back a vector instruction
// that reads an accumulator too early, and the compiler, which places the
// waits, has been seen to omit them where two paths of different length lead
// from the product to the read across blocks (the last accumulator register
// then held the value before the product).  8 passes need 12 states; with the
// wait in the product's own block no path is shorter.
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15");
  __builtin_amdgcn_sched_barrier(0);
}

__device__ __forceinline__ int div_group(const AttentionArgs& a, int row) { return fast_div(row, a.by_group); }

// One tile's sequence: its rows on both sides and the first (flattened) row
// of the tile in it.
struct Span {
  int q0, nq, k0, nk;  // first row and rows of the queries and of the keys
  int r0;              // first row of the tile within the sequence
  int seq, slot0;      // the sequence (as a bound's index) and its first slot
  bool any;            // the tile has rows
};

// The offsets bound the sequences: bound(0) = 0, bound(i) = cu[i - 1] and a
// last one of all rows, so rows before the first offset and after the last
// one form sequences without a counterpart (computed as rows without keys).
// Offsets are clamped to the rows there are: no access leaves the arrays
// whatever they hold.
__device__ __forceinline__ int bound(const int32_t* cu, int batch, int total, int i) {
  if (i <= 0) return 0;
  if (i > batch + 1) return total;
  const int v = cu[i - 1];
  return v < 0 ? 0 : v > total ? total : v;
}

// Sequence and tile of a slot, for tiles of 2^shift of the queries' flattened
// rows (mult = group), rows (mult = 1) or keys.  Sequence b starts at slot
// floor(bound(b) x mult / 2^shift) + b, which leaves every sequence at least
// ceil(rows x mult / 2^shift) slots and needs no pass over the lengths before.
// The wavefront finds b by probing 64 sequences at a time: first those around
// the place that equal lengths would give, which mostly ends the search in
// one round of loads, else in rounds that narrow 64-fold.
__device__ __forceinline__ Span find_span(const AttentionArgs& a, bool by_keys, int mult, int shift, int slot, int slots) {
  const int lane = threadIdx.x & 63;
  const int32_t* cu = by_keys ? a.cu_k : a.cu_q;
  const int total = by_keys ? a.total_k : a.total_q;
  const int last = a.batch + 2;  // bounds 0 .. last
  int lo = 0, hi = last, step = 1, v, c;
  auto probe = [&]() {
    const int at = lo + lane * step;
    v = bound(cu, a.batch, total, min(at, last));
    const int start = static_cast<int>((static_cast<int64_t>(v) * mult) >> shift) + at;
    return __builtin_popcountll(__ballot(at < hi && start <= slot));
  };
  bool found = false;
  if (last > 64) {
    const float guess = static_cast<float>(slot) * static_cast<float>(last) / static_cast<float>(slots);
    lo = min(max(static_cast<int>(guess) - 32, 0), last - 64);
    c = probe();
    found = c > 0 && (c < 64 || lo + 64 == last);
    if (!found) lo = 0;
  }
  while (!found) {
    step = (hi - lo + 63) >> 6;
    c = max(probe(), 1);
    if (step == 1) break;
    lo += (c - 1) * step;
    hi = min(lo + step, hi);
  }
  const int b = __builtin_amdgcn_readfirstlane(lo + c - 1);
  const int n = __builtin_amdgcn_readfirstlane(c);
  const int r0 = __builtin_amdgcn_readlane(v, n - 1);
  int r1 = n < 64 ? __builtin_amdgcn_readlane(v, n) : __builtin_amdgcn_readfirstlane(bound(cu, a.batch, total, b + 1));
  const int nr = max(r1 - r0, 0);
  int o0 = r0, no = nr;  // the other side
  if (a.cu_q != a.cu_k || a.total_q != a.total_k) {
    const int32_t* other = by_keys ? a.cu_q : a.cu_k;
    const int ototal = by_keys ? a.total_q : a.total_k;
    o0 = bound(other, a.batch, ototal, b);
    no = max(bound(other, a.batch, ototal, b + 1) - o0, 0);
    o0 = __builtin_amdgcn_readfirstlane(o0);
    no = __builtin_amdgcn_readfirstlane(no);
  }
  // a sequence before the first offset or after the last has no counterpart
  if (b == 0 || b == a.batch + 1) no = 0;
  Span s;
  s.q0 = by_keys ? o0 : r0;
  s.nq = by_keys ? no : nr;
  s.k0 = by_keys ? r0 : o0;
  s.nk = by_keys ? nr : no;
  const int64_t rows = static_cast<int64_t>(nr) * mult;
  s.slot0 = static_cast<int>((static_cast<int64_t>(r0) * mult) >> shift) + b;
  const int64_t t0 = (static_cast<int64_t>(slot) - s.slot0) * (int64_t(1) << shift);
  s.seq = b;
  s.any = t0 >= 0 && t0 < rows;
  s.r0 = s.any ? static_cast<int>(t0) : 0;
  return s;
}

// Slots that cover every tile of every sequence (find_span).
inline int64_t span_slots(int64_t rows, int batch, int tile) { return rows / tile + batch + 2; }

// Keys that the places p0 .. p1 see: [lo, hi).
struct KeyRange {
  int lo, hi;
};
__device__ __forceinline__ KeyRange key_range(const AttentionArgs& a, int nk, int p0, int p1) {
  KeyRange r;
  r.lo = a.left >= 0 ? max(p0 - a.left, 0) : 0;
  r.hi = a.right >= 0 ? min(p1 + a.right + 1, nk) : nk;
  return r;
}

// Keeps a rarely taken branch a branch: without it the compiler computes the
// masks of every tile and selects, 130 instructions a tile of 64 keys.
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }

// Slot and kv head of a workgroup.  Consecutive workgroups go to different
// XCDs, each with its own L2 (8 of them).
//   Heads first (run 0): an XCD sees few heads, whose keys and values fit its
//   L2 while the tiles of a long sequence walk them.
//   Runs of slots: an XCD takes `run` consecutive slots with all their heads.
//   Rows shorter than a 128-byte line share it with the next head, so that
//   heads on different XCDs would each fetch it: with 64-byte rows (1200
//   windows, 8 heads of 32) the gradients take 308 and 234 us instead of 331
//   and 264, and HBM reads fall to what there is to read.
struct Place {
  int slot, kvh;
};
constexpr int kXcds = 8;
__device__ __forceinline__ Place place_of(const AttentionArgs& a, int id, int run) {
  if (run == 0) {
    const int slot = fast_div(id, a.by_kv_heads);
    return {slot, id - slot * a.kv_heads};
  }
  const int j = id / kXcds, q = fast_div(j, a.by_kv_heads);
  return {(q / run * kXcds + id % kXcds) * run + q % run, j - q * a.kv_heads};
}
inline int slot_run(const AttentionArgs& a, int64_t slots) {
  const int bytes = a.dim * (a.dtype == 0 ? 4 : 2);
  return bytes < 128 && a.kv_heads > 1 && slots >= 128 ? 4 : 0;  // (fewer would leave XCDs without work)
}
inline int64_t placed_slots(int64_t slots, int run) {
  const int64_t unit = static_cast<int64_t>(run) * kXcds;
  return run == 0 ? slots : (slots + unit - 1) / unit * unit;
}

// Order of the slots by falling work (the other side's blocks of 32 that the
// slot's tile walks), for launches of few rounds of workgroups, where a long
// tile that starts late leaves the rest of the chip idle: a counting sort
// over 8 buckets per octave in one workgroup.  Slots of one bucket take any
// order, which no result depends on; slots without a tile go last.
struct OrderJob {
  int32_t* order = nullptr;  // NULL: none
  bool by_keys = false;
  int mult = 1, shift = 0, slots = 0;
};
constexpr int kOrderBuckets = 256, kOrderSlots = 2560;
__device__ __forceinline__ int order_bucket(int work) {
  if (work <= 0) return 0;
  const int top = 31 - __clz(work);
  const int frac = top >= 3 ? (work >> (top - 3)) & 7 : (work << (3 - top)) & 7;
  return min(1 + 8 * top + frac, kOrderBuckets - 1);
}
__device__ __forceinline__ void order_slots(const AttentionArgs& a, const OrderJob& job) {
  __shared__ __align__(16) int start[kOrderBuckets];
  __shared__ uint8_t bucket_of[kOrderSlots];
  const int tid = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);
  for (int i = tid; i < kOrderBuckets; i += nt) start[i] = 0;
  // slots that broken offsets leave to no sequence stay in the order
  for (int i = tid; i < job.slots; i += nt) bucket_of[i] = kOrderBuckets - 1;
  __syncthreads();
  const int32_t* cu = job.by_keys ? a.cu_k : a.cu_q;
  const int32_t* oc = job.by_keys ? a.cu_q : a.cu_k;
  const int total = job.by_keys ? a.total_k : a.total_q, ototal = job.by_keys ? a.total_q : a.total_k;
  // what the tile that starts at row r0 of n rows walks of the other side's m
  auto walk = [&](int r0, int n, int m) {
    const int rows = job.by_keys ? n : n * job.mult, r1 = min(r0 + (1 << job.shift), rows) - 1;
    if (job.by_keys) {
      const int to = n - m;  // a key's place among the queries: its row - to
      const int lo = a.right >= 0 ? max(r0 - a.right - to, 0) : 0, hi = a.left >= 0 ? min(r1 + a.left - to + 1, m) : m;
      return (max(hi - lo, 0) * a.group + 31) / 32;
    }
    const KeyRange k = key_range(a, m, div_group(a, r0) + m - n, div_group(a, r1) + m - n);
    return (max(k.hi - k.lo, 0) + 31) / 32;
  };
  for (int b = tid >> 5; b < a.batch + 2; b += nt >> 5) {
    const int r = bound(cu, a.batch, total, b), rn = bound(cu, a.batch, total, b + 1), n = max(rn - r, 0);
    const int o = bound(oc, a.batch, ototal, b), on = bound(oc, a.batch, ototal, b + 1);
    const int m = b == 0 || b == a.batch + 1 ? 0 : max(on - o, 0);
    const int slot0 = static_cast<int>((static_cast<int64_t>(r) * job.mult) >> job.shift) + b;
    const int next = b == a.batch + 1 ? job.slots : static_cast<int>((static_cast<int64_t>(rn) * job.mult) >> job.shift) + b + 1;
    for (int slot = slot0 + (tid & 31); slot < min(next, job.slots); slot += 32) {
      const int64_t r0 = static_cast<int64_t>(slot - slot0) << job.shift;
      const int w = r0 < static_cast<int64_t>(n) * job.mult ? 1 + walk(static_cast<int>(r0), n, m) : 0;
      const int bucket = kOrderBuckets - 1 - order_bucket(w);  // the most work first
      bucket_of[slot] = static_cast<uint8_t>(bucket);
      atomicAdd(&start[bucket], 1);
    }
  }
  __syncthreads();
  // exclusive prefix sum over the 256 buckets: 4 per lane of the first wave
  if (tid < 64) {
    const int4 c = reinterpret_cast<const int4*>(start)[tid];
    const int sum = c.x + c.y + c.z + c.w;
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int v = __shfl_up(incl, d);
      if (tid >= d) incl += v;
    }
    const int e = incl - sum;
    reinterpret_cast<int4*>(start)[tid] = make_int4(e, e + c.x, e + c.x + c.y, e + c.x + c.y + c.z);
  }
  __syncthreads();
  for (int slot = tid; slot < job.slots; slot += nt) {
    const int at = atomicAdd(&start[bucket_of[slot]], 1);
    if (at < job.slots) job.order[at] = slot;
  }
}
// Whether the sort, about 4 us, pays: few rounds of workgroups, and enough
// work (multiply-adds of one product, `products` of them) for them to last.
// What it gave over 1 to 16 sequences of 2000 to 32,000 rows in all, heads of
// 32, 64 and 128, bf16 and fp32, whole and causal (forward; gradients):
//   below 512 workgroups, which all run at once, -17 to 20%, mostly a loss;
//   -10 to 19%;
//   from 512 to 1000: -6 to 19%; -1 to 24%;
//   from 1000 to 2560: -6 to 45%; -1 to 49%;
//   at 4072: -1%; 1 to 16%.
// Below the two amounts of work its own time is a tenth of the forward's and
// more; what the gradients would gain there (up to 49%) the rule gives up.
// Causal sequences of up to 4096 rows with gradients: 173 and 124 us instead
// of 220 and 141; frames of 500 to 4000 rows, forward: 157 instead of 180.
inline bool order_pays(const AttentionArgs& a, int64_t slots, int split, double products) {
  const int64_t groups = slots * a.kv_heads * split;
  double work = static_cast<double>(a.total_q) * a.heads * (static_cast<double>(a.total_k) / std::max(a.batch, 1)) * a.dim * products;
  if (a.left >= 0 || a.right >= 0) work /= 2;
  return a.batch <= 1024 && slots <= kOrderSlots && groups >= 512 && groups <= 2560 && work >= (a.dtype == 0 ? 3e9 : 2.4e10);
}

// The blocks of one split: an even share of [0, blocks).
struct Share {
  int first, end;
};
__device__ __forceinline__ Share share_of(int blocks, int split, int nsplit) {
  if (nsplit == 1) return {0, blocks};
  // blocks < 2^26 (32 rows each) and nsplit <= 64
  const uint32_t b = static_cast<uint32_t>(blocks), n = static_cast<uint32_t>(nsplit), s = static_cast<uint32_t>(split);
  return {static_cast<int>(b * s / n), static_cast<int>(b * (s + 1) / n)};
}

// Row of register i of a C tile within its 32, without the half's 4.
__host__ __device__ constexpr int c_row(int i) { return 8 * (i / 4) + (i & 3); }

// log2 of a wavefront count's tile: 32 rows per wave.
constexpr int tile_shift(int waves) { return waves == 1 ? 5 : waves == 2 ? 6 : 7; }

// Stores 4 consecutive values as T.
template <class T>
__device__ __forceinline__ void store4(T* dst, float x, float y, float z, float w) {
  typedef T tx4 __attribute__((ext_vector_type(4)));
  tx4 v;
  v[0] = static_cast<T>(x);
  v[1] = static_cast<T>(y);
  v[2] = static_cast<T>(z);
  v[3] = static_cast<T>(w);
  *reinterpret_cast<tx4*>(dst) = v;
}

// Stores a lane's column of C tiles as a row of T, 8 consecutive values at a
// time: the halves exchange registers so that each holds whole pieces (half
// 0 those of columns 16 i, half 1 those of 16 i + 8), two for one of four.
template <class T, int DB>
__device__ __forceinline__ void store_row(T* dst, const floatx16 (&acc)[DB], float mul, int half, int dim, bool on) {
  typedef T tx4 __attribute__((ext_vector_type(4)));
  constexpr int W = sizeof(T);  // words of 4 values
  struct Words {
    uint32_t w[W];
  };
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      Words q[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        tx4 v;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = static_cast<T>(acc[db][8 * i + 4 * g + u] * mul);
        q[g] = __builtin_bit_cast(Words, v);
      }
      uint32_t piece[2 * W];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const auto r = __builtin_amdgcn_permlane32_swap(q[0].w[w], q[1].w[w], false, false);
        piece[w] = r[0];
        piece[W + w] = r[1];
      }
      const int d = db * 32 + 16 * i + 8 * half;
      if (on && d < dim) {
#pragma unroll
        for (int w = 0; w < 2 * W; w += 4)
          *reinterpret_cast<uint4*>(reinterpret_cast<char*>(dst + d) + 4 * w) = make_uint4(piece[w], piece[w + 1], piece[w + 2], piece[w + 3]);
      }
    }
}

// Calls f(type, DP, DQ): the head size rounded up to 32 (the blocks of the
// products that end in it) and to 16 (the steps of those over it).
template <class F>
hipError_t dispatch(const AttentionArgs& a, F&& f) {
  auto by_dim = [&](auto t) {
    typedef decltype(t) T;
#define SPCONV_DIM(q) \
  if (a.dim <= q) return f(T{}, std::integral_constant<int, (q + 31) / 32 * 32>{}, std::integral_constant<int, q>{});
    SPCONV_DIM(16)
    SPCONV_DIM(32)
    SPCONV_DIM(48)
    SPCONV_DIM(64)
    SPCONV_DIM(80)
    SPCONV_DIM(96)
    SPCONV_DIM(112)
#undef SPCONV_DIM
    return f(T{}, std::integral_constant<int, 128>{}, std::integral_constant<int, 128>{});
  };
  if (a.dtype == 0) return by_dim(float{});
  if (a.dtype == 1) return by_dim(static_cast<_Float16>(0));
  return by_dim(static_cast<__bf16>(0.f));
}

// How `rows` rows per kv head, `mean` in a sequence, that each walk `depth`
// rows of the other side, become workgroups: 32 rows per wave; the walk is
// split (into parts of at least 256, in fp32 128) until there are two waves
// per SIMD twice over; and where that leaves less than two workgroups per CU,
// two waves instead of four spread more evenly.
struct Cut {
  int waves, split;
};
inline Cut cut_rows(const AttentionArgs& a, int64_t mean, int64_t rows, int64_t depth) {
  Cut c;
  c.waves = mean <= 32 ? 1 : mean <= 64 ? 2 : 4;
  const int64_t tiles = std::max<int64_t>(rows / (32 * c.waves), std::max(a.batch, 1)) * a.kv_heads;
  const int64_t most = depth / (a.dtype == 0 ? 128 : 256), want = 4096 / (tiles * c.waves);
  c.split = 1;  // a power of two
  while (c.split < 16 && 2 * c.split <= std::min(most, want)) c.split *= 2;
  if (c.waves == 4 && tiles * c.split < 512) c.waves = 2;
  return c;
}
// Rows of the other side that a row's band reaches, of `rows` (times `group`).
inline int64_t band_depth(const AttentionArgs& a, int64_t rows, int64_t group) {
  if (a.left < 0 || a.right < 0) return rows * group;
  return std::min<int64_t>(rows, static_cast<int64_t>(a.left) + a.right + 1) * group;
}

}  // namespace attn
}  // namespace spconv
