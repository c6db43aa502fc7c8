// Products of packed rows with their epilogue, and their gradients: the plan
// of each call (tile shape, parts of the contraction, operands that have to be
// laid out first), the joins of the parts, and the activation's gradient.
//
//   forward:   out = act(x W + b) + residual            one product by rows
//   backward:  grad_x = grad W^T (x act'(before))       by rows, W transposed
//              grad_W = x^T grad, grad_b = sum of grad  over rows, one pass
//
// The products themselves are in linear_kernels.h.
#include <algorithm>
#include <type_traits>

#include "linear_common.h"

namespace spconv {
namespace {

using lin::Segment;

// ---- Laying out ----
// Rows of whole 16-byte pieces are read as they lie; other row lengths (or
// strides) are copied first, to rows padded with zeros.
template <class E>
__global__ __launch_bounds__(256) void k_lay_out(const E* src, int64_t src_row, int64_t rows, int cols, E* dst, int dst_cols) {
  constexpr int N = 16 / static_cast<int>(sizeof(E));
  typedef E vec __attribute__((ext_vector_type(N)));
  const int pieces = dst_cols / N;
  const int64_t total = rows * pieces;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / pieces;
    const int col = static_cast<int>(i - row * pieces) * N;
    vec v;
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = col + j < cols ? src[row * src_row + col + j] : static_cast<E>(0);
    *reinterpret_cast<vec*>(dst + row * dst_cols + col) = v;
  }
}

// ---- Joining ----
// By rows: the parts of k summed in their order, then the epilogue; 8 columns
// a thread.
template <class T, int FORM>
__global__ __launch_bounds__(256) void k_join_rows(ProductArgs a) {
  const int pieces = a.n_part / 8;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * pieces) return;
  const int64_t row = i / pieces;
  const int col = static_cast<int>(i - row * pieces) * 8, there = min(a.n - col, 8);
  int group = 0;
  if (a.cu != nullptr) {  // the segment: the last bound at or before the row
    int lo = 0, hi = a.groups + 2;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (attn::bound(a.cu, a.groups, a.rows, mid) <= row) lo = mid;
      else hi = mid;
    }
    group = lo == 0 || lo == a.groups + 1 ? -1 : lo - 1;
  }
  float v[8] = {}, bias[8] = {}, side[8] = {};
  if (group >= 0) {
    if (a.bias != nullptr) lin::load_some8<T>(static_cast<const T*>(a.bias) + static_cast<int64_t>(group) * a.n + col, there, a.whole, bias);
    if (a.side != nullptr) lin::load_some8<T>(lin::side_row<T>(a, row) + col, there, a.whole, side);
    const float* p = a.part + row * a.n_part + col;
    const int64_t step = static_cast<int64_t>(a.rows) * a.n_part;
#pragma unroll 4
    for (int s = 0; s < a.splits; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(p + s * step), y = *reinterpret_cast<const float4*>(p + s * step + 4);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] += bias[j];
  lin::finish<T, FORM, 8>(a, group >= 0, a.side != nullptr && group >= 0, [&](int j) { return side[j]; }, v,
                          [&](T* to, int64_t stride, const float (&x)[8]) { lin::store_some8<T>(to + row * stride + col, there, a.whole, x); });
}

// Over rows: the parts of each group summed in a fixed order; a group without
// rows gives zeros.  Row m of the sums is the column sums of b.  4 columns a
// thread, LANES threads for them that take the parts in turn and join in LDS:
// hundreds of parts of small sums would be a long chain of loads for one
// (512 parts of 64 x 64 in bf16: 22 us, with 16 lanes 5.7).
template <int LANES>
__global__ __launch_bounds__(256) void k_join_groups(ProductArgs a) {
  constexpr int QUADS = 256 / LANES;
  __shared__ float4 stage[LANES > 1 ? 256 : 1];
  const int group = blockIdx.y;
  const int pieces = a.n_part / 4;
  const int lane = threadIdx.x / QUADS;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * QUADS + threadIdx.x % QUADS;
  const bool there = i < static_cast<int64_t>(a.m + (a.sums != nullptr)) * pieces;
  const int m = there ? static_cast<int>(i / pieces) : 0, col = there ? static_cast<int>(i - static_cast<int64_t>(m) * pieces) * 4 : 0;
  int first = 0, rows = a.rows;
  if (a.cu != nullptr) {
    const int r0 = attn::bound(a.cu, a.groups, a.rows, group + 1), r1 = attn::bound(a.cu, a.groups, a.rows, group + 2);
    rows = max(r1 - r0, 0);
    first = lin::segment_start(a, group + 1);
  }
  const int parts = rows == 0 || !there ? 0 : fast_div(rows - 1, a.by_unit) + 1;
  const bool sums = m == a.m;
  const float* p = sums ? a.sums_part + static_cast<int64_t>(first) * a.n_part + col
                        : a.part + (static_cast<int64_t>(first) * a.m + m) * a.n_part + col;
  const int64_t step = sums ? a.n_part : static_cast<int64_t>(a.m) * a.n_part;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = lane; s < parts; s += LANES) {
    const float4 x = *reinterpret_cast<const float4*>(p + s * step);
    v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
  }
  if constexpr (LANES > 1) {
    stage[threadIdx.x] = v;
    __syncthreads();
    if (lane > 0) return;
#pragma unroll
    for (int q = 1; q < LANES; ++q) {
      const float4 x = stage[q * QUADS + threadIdx.x];
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
  }
  if (!there) return;
  float* dst = sums ? a.sums + static_cast<int64_t>(group) * a.n + col : static_cast<float*>(a.out) + (static_cast<int64_t>(group) * a.m + m) * a.n + col;
  if (a.whole && !sums) {
    *reinterpret_cast<float4*>(dst) = v;
  } else {
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < a.n) dst[j] = x[j];
  }
}

// ---- The activation's gradient ----
template <class T>
__global__ __launch_bounds__(256) void k_activation_backward(ActivationArgs a, int pieces, FastDiv by_pieces, bool whole) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * pieces) return;
  const int64_t row = i < (int64_t(1) << 31) ? fast_div(static_cast<int>(i), by_pieces) : i / pieces;
  const int col = static_cast<int>(i - row * pieces) * 8, there = min(a.cols - col, 8);
  float g[8], z[8];
  lin::load_some8<T>(static_cast<const T*>(a.grad) + row * a.grad_row + col, there, whole, g);
  lin::load_some8<T>(static_cast<const T*>(a.pre) + row * a.pre_row + col, there, whole, z);
  lin::times_slope<T, 8>(a.act, [&](int j) { return z[j]; }, g);
  lin::store_some8<T>(static_cast<T*>(a.out) + row * a.out_row + col, there, whole, g);
}

// ---- The plan ----
int64_t size_of(int dtype) { return dtype == 0 ? 4 : 2; }
bool whole_pieces(int64_t elements, int dtype) { return elements * size_of(dtype) % 16 == 0; }
int32_t padded(int32_t cols) { return (cols + 7) / 8 * 8; }
bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Takes pieces of a workspace one after another; without one it counts.
struct Carver {
  char* base;
  size_t at = 0;
  void* take(size_t bytes) {
    void* p = base == nullptr ? nullptr : base + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  }
};

// An operand and, where it has to be laid out first, its copy.
struct Operand {
  const void* p;
  int64_t row;
  int32_t cols;
  void* copy;
};
Operand operand(const void* p, int64_t row_stride, int64_t rows, int32_t cols, int dtype, Carver* w) {
  if (whole_pieces(cols, dtype) && whole_pieces(row_stride, dtype)) return {p, row_stride, cols, nullptr};
  const int32_t c = padded(cols);
  void* copy = w->take(static_cast<size_t>(rows) * c * size_of(dtype));
  return {copy, c, c, copy};
}
hipError_t lay_out(const Operand& o, const void* src, int64_t row_stride, int64_t rows, int32_t cols, int dtype, hipStream_t stream) {
  if (o.cols == cols && whole_pieces(row_stride, dtype)) return hipSuccess;
  const int64_t pieces = rows * (o.cols * size_of(dtype) / 16);
  if (pieces == 0) return hipSuccess;
  const unsigned blocks = static_cast<unsigned>(std::min<int64_t>((pieces + 255) / 256, 8192));
  if (dtype == 0) {
    k_lay_out<uint32_t><<<blocks, 256, 0, stream>>>(static_cast<const uint32_t*>(src), row_stride, rows, cols, static_cast<uint32_t*>(o.copy), o.cols);
  } else {
    k_lay_out<uint16_t><<<blocks, 256, 0, stream>>>(static_cast<const uint16_t*>(src), row_stride, rows, cols, static_cast<uint16_t*>(o.copy), o.cols);
  }
  return hipGetLastError();
}

struct ShapeSize {
  int bm, bn, bk, threads;
};
ShapeSize shape_size(int dtype, ProductForm form, ProductShape s) {
  const int few = dtype == 0 ? 32 : 64;  // contracted values of a wavefront's chunk
  if (s == kFewShape) return {32, 32, few * 8, 512};
  if (s == kFewWideShape) return {32, 64, few * 8, 512};
  if (s == kFewShortShape) return {32, form == kByRows ? 64 : 32, few * 4, 256};
  auto of = [](auto x) { return ShapeSize{decltype(x)::BM, decltype(x)::BN, decltype(x)::BK, decltype(x)::NT}; };
  auto by_shape = [&](auto shapes) {
    typedef decltype(shapes) S;
    return s == kNarrowShape ? of(typename S::Narrow{}) : s == kHalfShape ? of(typename S::Half{}) : s == kMediumShape ? of(typename S::Medium{}) : of(typename S::Large{});
  };
  return dtype == 0 ? by_shape(lin::Shapes<float>{}) : by_shape(lin::Shapes<_Float16>{});
}

int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Workgroups that fill the chip: two on each of 256 CUs.
constexpr int64_t kFill = 512;

struct Product {
  ProductArgs a;
  ProductForm form;
  ProductShape shape;
  int dtype;
  uint64_t items() const {
    return static_cast<uint64_t>(product_blocks(a, form)) * shape_size(dtype, form, shape).threads;
  }
};

// Sizes of a product by rows: rows x k times k x n of each group.
//
// Few rows of each group go by independent wavefronts (k_few), as tiles of 128
// rows would have few workgroups and a barrier a step (bf16: 5 rows 2048 ->
// 8192 13.3 us by tiles, 10.2; 100 rows 256 -> 4096 9.3 and 5.8; 64 rows 1024
// -> 1024 10.6 and 8.5).  Every 32 rows read the weights anew, from L2, so up
// to 32 rows of a group on average, or up to 128 in products small enough that
// the barriers cost more (bf16, groups of 1024 -> 1024: 8 of 80 rows 11.4 us
// by wavefronts, 17.5 by tiles; 32 of 40 rows 22.2 and 23.8, 32 of 120 29.9
// and 25.4, 128 of 120 114 and 108, transposed 133 and 101; one group: 120
// rows 2048 -> 2048 10.5 and 15.3, 40 rows 4096 -> 4096 19.4 and 17.6; f32,
// 256 -> 512: 32 groups of 80 rows 17.4 and 21.2, 128 groups 49 and 45).  32
// columns a workgroup while 64 would leave CUs without one; 4 wavefronts where the contraction gives 8 of them two chunks
// or fewer (32 groups of 64 rows 512 -> 1024: 10.4 us, with 8 13.6), 8 for
// the others (16 rows 512 -> 2048: 4.2, with 4 6.4).
//
// More rows go by tiles.  Narrow ones for up to 64 columns (f32, 80,000 rows
// 256 -> 64: 42 us by 128 columns, 31) and while tiles of 128 columns are
// fewer than CUs (bf16: 3,000 rows 1024 -> 1024 29.5 and 20.7).  In f32 those
// have 32 columns, or 64, whose rows are split into planes half as often,
// where these fill the CUs twice or the contraction is long enough for parts
// (69,924 rows 2448 -> 64 290 and 229 us, 2,500 rows 1024 -> 512 41 and 32;
// but 20,000 rows 256 -> 64 14.6 and 20.3).  The largest
// where they fill three quarters of their rounds of one workgroup a CU
// (8192 x 4096 x 4096: 250 us, by 128 x 128 322; 9,000 rows, half of the last
// round: 342 and 352; 6,000 rows: 224 and 236; 5,000 rows: 223 and 205), or
// five eighths of one where the contraction is long (5,700 rows 4096 -> 2048:
// 122 us by 128 x 128, 110; 10,000 rows 2048 -> 1024 65 and 62; 21,000 rows 768
// -> 512 31 and 32).
Product plan_by_rows(ProductForm form, int dtype, const int32_t* cu, int32_t rows, int32_t groups, int32_t k, int32_t n, Carver* w) {
  Product p;
  p.form = form;
  p.dtype = dtype;
  const int64_t each = rows / groups;
  const double products = static_cast<double>(rows) * k * n;
  const double most = dtype != 0 && cu == nullptr && k > 1024 ? 1 << 29 : 1 << 30;
  const bool few = each <= 32 || (each <= 128 && products <= most);
  if (few) {
    const int64_t wide = (rows / 32 + groups) * div_up(n, 64);  // workgroups of 64 columns
    p.shape = wide < 256 ? kFewShape : k <= 1024 ? kFewShortShape : kFewWideShape;
  } else {
    const int64_t medium = (rows / 128 + (cu == nullptr ? 1 : groups)) * div_up(n, 128);
    p.shape = n <= 64 || medium < 256 ? kNarrowShape : kMediumShape;
    const int64_t half = (rows / 128 + (cu == nullptr ? 1 : groups)) * div_up(n, 64);
    if (dtype == 0 && p.shape == kNarrowShape && n > 32 && (half >= 512 || k >= 1024)) p.shape = kHalfShape;
  }
  const int64_t large = div_up(rows, 256) * div_up(n, 256);
  const bool filled = 4 * large >= 3 * 256 * div_up(large, 256) || (large >= 160 && large <= 256 && k >= 2048);
  if (dtype != 0 && p.shape == kMediumShape && k >= 512 && n >= 192 && filled) p.shape = kLargeShape;
  const ShapeSize s = shape_size(dtype, p.form, p.shape);
  ProductArgs& a = p.a;
  a.cu = cu;
  a.groups = groups;
  a.rows = rows;
  a.n = n;
  a.k = k;
  a.by_unit = make_fast_div(s.bm);
  a.slots = static_cast<int32_t>(cu == nullptr ? div_up(rows, s.bm) : rows / s.bm + groups + 2);
  a.tiles = a.tiles_n = static_cast<int32_t>(div_up(n, s.bn));
  const int64_t steps = div_up(k, s.bk), blocks = std::max<int64_t>(1, static_cast<int64_t>(a.slots) * a.tiles);
  // Parts of the contraction, where the tiles alone leave CUs without work:
  // up to 256 workgroups of few rows (1 row in f32, 2048 -> 264: 9.4 us with
  // half as many, 8.7; grad_x of 5 rows 2048 -> 8192 16.9 and 13.6); up to two
  // on a CU of tiles, parts of four steps at least.  Never of the largest
  // tiles, of which one fills a CU (65,536 rows 1024 -> 256 in two parts 90
  // us, whole 44).
  int64_t splits = 1;
  if (few) {
    if (blocks * 2 <= 256) splits = std::max<int64_t>(1, std::min(256 / blocks, steps));
  } else if (p.shape != kLargeShape && blocks * 2 <= kFill && steps >= 8) {
    splits = std::min(kFill / blocks, steps / 4);
  }
  a.k_split = static_cast<int32_t>(div_up(steps, splits) * s.bk);
  a.splits = static_cast<int32_t>(div_up(k, a.k_split));
  a.n_part = padded(n);
  if (a.splits > 1) a.part = static_cast<float*>(w->take(static_cast<size_t>(a.splits) * rows * a.n_part * sizeof(float)));
  return p;
}

// Rows at the start of a dense product that go by whole rounds of the largest
// tiles, where all of them together would leave most of the last round's CUs
// without one (0: the product is one launch).  (bf16: 65,537 rows 1024 -> 256
// 60 us by smaller tiles, 55 in two launches; 4097 x 4096 x 4096 194 and 140.)
int32_t whole_rounds(int dtype, const int32_t* cu, int32_t rows, int32_t k, int32_t n) {
  const int64_t columns = div_up(n, 256), large = div_up(rows, 256) * columns;
  if (dtype == 0 || cu != nullptr || k < 512 || n < 192 || large <= 256 || 4 * large >= 3 * 256 * div_up(large, 256)) return 0;
  return static_cast<int32_t>(large / 256 * 256 / columns * 256);
}

// A product by rows: one launch, or the whole rounds and the rows after them.
struct ByRows {
  Product p, rest;
  int32_t head;
  uint64_t items() const { return head == 0 ? p.items() : std::max(p.items(), rest.items()); }
};
ByRows plan_all_rows(ProductForm form, int dtype, const int32_t* cu, int32_t rows, int32_t groups, int32_t k, int32_t n, Carver* w) {
  ByRows b;
  b.head = whole_rounds(dtype, cu, rows, k, n);
  const Carver before = *w;
  b.p = plan_by_rows(form, dtype, cu, b.head == 0 ? rows : b.head, groups, k, n, w);
  if (b.head != 0 && b.p.shape != kLargeShape) {
    // (many columns: whole rows of tiles are too little of a round for the
    // largest ones, and two launches would read all weights twice for nothing:
    // bf16, 300 rows 1024 -> 33,000 63 us, in one 49)
    b.head = 0;
    *w = before;
    b.p = plan_by_rows(form, dtype, cu, rows, groups, k, n, w);
  }
  if (b.head != 0) b.rest = plan_by_rows(form, dtype, cu, rows - b.head, groups, k, n, w);
  return b;
}

// Sizes of a product over the rows of each group: m x n sums.
//
// Narrow tiles for up to 64 columns, and while the sum is short: more tiles
// make for fewer parts to join (bf16, 256 x 256 sums: 100,000 rows 39 us by
// 128 columns, 33; 1024 x 1024: 2,500 rows 28.9 and 24.2, 20,000 rows 64 and
// 70; f32, 256 x 256: 2,500 rows 19.0 and 14.9, 20,000 rows 33 and 33, 80,000
// rows 73 and 109); 64 columns in f32 by tiles of as many for longer ones, as
// above (78,075 rows of 3176 x 40 335 and 251 us, 20,000 rows of 256 x 64 19.8
// and 20.6).  The largest for long sums (400,000 rows of 256 x 1024:
// 310 us by 128 x 128, 266; but 65,537 rows of 1024 x 256 60 and 66).
Product plan_over_rows(int dtype, const int32_t* cu, int32_t rows, int32_t groups, int32_t m, int32_t n, Carver* w) {
  Product p;
  p.form = kOverRows;
  p.dtype = dtype;
  const int64_t medium = div_up(m, 128) * div_up(n, 128);
  p.shape = n <= 64 || medium * rows < (dtype == 0 ? 1 << 16 : 1 << 19) ? kNarrowShape : kMediumShape;
  if (dtype == 0 && n > 32 && n <= 64 && medium * rows >= 1 << 17) p.shape = kHalfShape;
  if (dtype != 0 && p.shape == kMediumShape && m > 128 && n > 128 && div_up(m, 256) * div_up(n, 256) * (rows / 64) >= 32 * 256) p.shape = kLargeShape;
  const ShapeSize s = shape_size(dtype, p.form, p.shape);
  ProductArgs& a = p.a;
  a.cu = cu;
  a.groups = groups;
  a.rows = rows;
  a.m = m;
  a.n = n;
  a.tiles_n = static_cast<int32_t>(div_up(n, s.bn));
  a.tiles = static_cast<int32_t>(div_up(m, s.bm) * a.tiles_n);
  a.n_part = padded(n);
  // Parts of 128 rows at least (f32, 20,011 rows of 128 x 192: 28.2 us, with
  // 256 31.4).  A group may end in a part of few rows: room for one each, that
  // all parts run in one round (16 groups of 12,500 rows of 512 x 512: 162 us,
  // without it 223).
  const int64_t fill = (p.shape == kLargeShape ? 256 : kFill) / a.tiles;
  const int64_t parts = std::min<int64_t>(cu != nullptr && 4 * groups <= fill ? fill - groups : fill, rows / 128);
  if (parts <= 1 || parts <= groups) {  // every group is one part
    a.by_unit = make_fast_div(1 << 30);
    a.slots = cu == nullptr ? 1 : groups + 2;
    a.by_tiles = a.tiles >= 8;  // (16 groups of 3600 x 1304, the last with a fifth of 18,540 rows: 630 us in eighths, 327)
  } else {
    const int64_t unit = div_up(div_up(rows, parts), s.bk) * s.bk;
    a.by_unit = make_fast_div(static_cast<int32_t>(unit));
    a.slots = static_cast<int32_t>(cu == nullptr ? div_up(rows, unit) : rows / unit + groups + 2);
    // (a part's tiles share rows: spread only where many do.  8 groups of 2,500
    // rows of 512 x 1024: 61 us by parts, 49 by tiles; 4 groups of 25,000 rows
    // of 512 x 512: 79 and 106)
    a.by_tiles = a.tiles >= 32;
    a.part = static_cast<float*>(w->take(static_cast<size_t>(a.slots) * m * a.n_part * sizeof(float)));
    a.sums_part = static_cast<float*>(w->take(static_cast<size_t>(a.slots) * a.n_part * sizeof(float)));
  }
  return p;
}

// The join over rows: 4 columns a thread, and the lanes that share the parts
// of one group (their number on average).
int64_t join_pieces(const ProductArgs& a) { return static_cast<int64_t>(a.m + 1) * (a.n_part / 4); }
int join_lanes(const ProductArgs& a) {
  const int parts = a.slots / a.groups;
  return parts >= 32 ? 16 : parts >= 8 ? 4 : 1;
}

hipError_t run_product(const Product& p, hipStream_t stream) {
  if (p.dtype == 0) return launch_product_f32(p.a, p.form, p.shape, stream);
  if (p.dtype == 1) return launch_product_f16(p.a, p.form, p.shape, stream);
  return launch_product_bf16(p.a, p.form, p.shape, stream);
}

// Whether a product keeps its weights in registers: the contraction fits them,
// and the columns fill a workgroup's (bf16, against tiles: 400,000 rows 256 ->
// 1024 293 us and 562, 128 -> 128 36 and 52, 64 -> 64 21 and 28; f32, 100,000
// rows 128 -> 256 46 and 68).
bool streams(const Product& p) {
  const ProductArgs& a = p.a;
  if (!a.whole || a.splits > 1 || p.shape == kFewShape || p.shape == kFewWideShape || p.shape == kFewShortShape) return false;
  return p.dtype == 0 ? a.k <= 128 && a.n > 64 : a.k <= 256 && a.n >= 64;
}

hipError_t run_by_rows(Product& p, hipStream_t stream) {
  if (p.a.rows == 0) return hipSuccess;
  if (streams(p)) p.shape = kStreamShape;
  const hipError_t e = run_product(p, stream);
  if (e != hipSuccess || p.a.splits == 1) return e;
  const unsigned blocks = static_cast<unsigned>(div_up(static_cast<int64_t>(p.a.rows) * (p.a.n_part / 8), 256));
  auto join = [&](auto t) {
    typedef decltype(t) T;
    if (p.form == kByRows) k_join_rows<T, kByRows><<<blocks, 256, 0, stream>>>(p.a);
    else k_join_rows<T, kByRowsT><<<blocks, 256, 0, stream>>>(p.a);
  };
  if (p.dtype == 0) join(0.f);
  else if (p.dtype == 1) join(static_cast<_Float16>(0));
  else join(static_cast<__bf16>(0.f));
  return hipGetLastError();
}

// Whether rows of `cols` values take 16-byte accesses, 8 values at a time (NULL: nothing is accessed).
bool whole_rows(const void* p, int64_t row_stride, int64_t cols, int dtype) {
  return p == nullptr || (aligned(p) && whole_pieces(row_stride, dtype) && cols % 8 == 0);
}

// (b.p.a holds the operands and the epilogue of all rows)
hipError_t run_all_rows(ByRows& b, hipStream_t stream) {
  const hipError_t e = run_by_rows(b.p, stream);
  if (e != hipSuccess || b.head == 0) return e;
  const ProductArgs& all = b.p.a;
  ProductArgs& a = b.rest.a;
  const int64_t size = size_of(b.p.dtype);
  auto after = [&](const void* p, int64_t row) { return p == nullptr ? nullptr : static_cast<const char*>(p) + b.head * row * size; };
  auto out_after = [&](void* p, int64_t row) { return p == nullptr ? nullptr : static_cast<char*>(p) + b.head * row * size; };
  a.a = after(all.a, all.a_row);
  a.a_row = all.a_row;
  a.a_cols = all.a_cols;
  a.b = all.b;
  a.b_row = all.b_row;
  a.b_cols = all.b_cols;
  a.b_group = all.b_group;
  a.bias = all.bias;
  a.side = after(all.side, all.side_row);
  a.side_row = all.side_row;
  a.pre = out_after(all.pre, all.pre_row);
  a.pre_row = all.pre_row;
  a.out = out_after(all.out, all.out_row);
  a.out_row = all.out_row;
  a.act = all.act;
  a.whole = all.whole;
  return run_by_rows(b.rest, stream);
}

struct Forward {
  Operand x, w;
  ByRows p;
  size_t bytes;
};
Forward plan_forward(const LinearArgs& a, void* workspace) {
  Forward f;
  Carver c{static_cast<char*>(workspace)};
  f.x = operand(a.x, a.x_row, a.rows, a.c_in, a.dtype, &c);
  f.w = operand(a.weight, a.c_out, static_cast<int64_t>(a.groups) * a.c_in, a.c_out, a.dtype, &c);
  f.p = plan_all_rows(kByRows, a.dtype, a.cu, a.rows, a.groups, a.c_in, a.c_out, &c);
  f.bytes = c.at;
  return f;
}

struct Backward {
  Operand x, w, g;
  ByRows gx;
  Product gw;
  size_t bytes;
};
Backward plan_backward(const LinearArgs& a, void* workspace) {
  Backward b;
  Carver c{static_cast<char*>(workspace)};
  b.x = operand(a.x, a.x_row, a.rows, a.c_in, a.dtype, &c);
  b.g = operand(a.grad_out, a.grad_out_row, a.rows, a.c_out, a.dtype, &c);
  b.w = operand(a.weight, a.c_out, static_cast<int64_t>(a.groups) * a.c_in, a.c_out, a.dtype, &c);
  // (the two products run one after the other: their parts may share a place)
  Carver c1 = c, c2 = c;
  b.gx = plan_all_rows(kByRowsT, a.dtype, a.cu, a.rows, a.groups, a.c_out, a.c_in, &c1);
  b.gw = plan_over_rows(a.dtype, a.cu, a.rows, a.groups, a.c_in, a.c_out, &c2);
  b.bytes = std::max(c1.at, c2.at);
  return b;
}

}  // namespace

uint64_t linear_work_items(const LinearArgs& a, bool backward) {
  if (!backward) return plan_forward(a, nullptr).p.items();
  const Backward b = plan_backward(a, nullptr);
  const ProductArgs& p = b.gw.a;
  const bool joined = p.by_unit.d != (1 << 30);
  const uint64_t join = joined ? static_cast<uint64_t>(div_up(join_pieces(p), 256 / join_lanes(p))) * 256 * a.groups : 0;
  return std::max({b.gx.items(), b.gw.items(), join});
}

size_t linear_workspace_bytes(const LinearArgs& a) { return plan_forward(a, nullptr).bytes; }
size_t linear_backward_workspace_bytes(const LinearArgs& a) { return plan_backward(a, nullptr).bytes; }

hipError_t launch_linear(const LinearArgs& a, void* workspace, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  Forward f = plan_forward(a, workspace);
  hipError_t e = lay_out(f.x, a.x, a.x_row, a.rows, a.c_in, a.dtype, stream);
  if (e == hipSuccess) e = lay_out(f.w, a.weight, a.c_out, static_cast<int64_t>(a.groups) * a.c_in, a.c_out, a.dtype, stream);
  if (e != hipSuccess) return e;
  ProductArgs& p = f.p.p.a;
  p.a = f.x.p;
  p.a_row = f.x.row;
  p.a_cols = f.x.cols;
  p.b = f.w.p;
  p.b_row = f.w.row;
  p.b_cols = f.w.cols;
  p.b_group = static_cast<int64_t>(a.c_in) * f.w.row;
  p.bias = a.bias;
  p.side = a.residual;
  p.side_row = a.residual_row;
  p.pre = a.pre;
  p.pre_row = a.pre_row;
  p.out = a.out;
  p.out_row = a.out_row;
  p.act = a.act;
  p.whole = whole_rows(a.out, a.out_row, a.c_out, a.dtype) && whole_rows(a.pre, a.pre_row, a.c_out, a.dtype) &&
            whole_rows(a.residual, a.residual_row, a.c_out, a.dtype) && whole_rows(a.bias, a.c_out, a.c_out, a.dtype);
  return run_all_rows(f.p, stream);
}

hipError_t launch_linear_backward(const LinearArgs& a, void* workspace, hipStream_t stream) {
  Backward b = plan_backward(a, workspace);
  hipError_t e = lay_out(b.g, a.grad_out, a.grad_out_row, a.rows, a.c_out, a.dtype, stream);
  if (e == hipSuccess && a.grad_weight != nullptr) e = lay_out(b.x, a.x, a.x_row, a.rows, a.c_in, a.dtype, stream);
  if (e == hipSuccess && a.grad_x != nullptr) e = lay_out(b.w, a.weight, a.c_out, static_cast<int64_t>(a.groups) * a.c_in, a.c_out, a.dtype, stream);
  if (e != hipSuccess) return e;
  if (a.grad_x != nullptr) {
    ProductArgs& p = b.gx.p.a;
    p.a = b.g.p;
    p.a_row = b.g.row;
    p.a_cols = b.g.cols;
    p.b = b.w.p;
    p.b_row = b.w.row;
    p.b_cols = b.w.cols;
    p.b_group = static_cast<int64_t>(a.c_in) * b.w.row;
    p.side = a.before;
    p.side_row = a.before_row;
    p.act = a.act;
    p.out = a.grad_x;
    p.out_row = a.grad_x_row;
    p.whole = whole_rows(a.grad_x, a.grad_x_row, a.c_in, a.dtype) && whole_rows(a.before, a.before_row, a.c_in, a.dtype);
    e = run_all_rows(b.gx, stream);
    if (e != hipSuccess) return e;
  }
  if (a.grad_weight != nullptr) {
    ProductArgs& p = b.gw.a;
    p.a = b.x.p;
    p.a_row = b.x.row;
    p.a_cols = b.x.cols;
    p.b = b.g.p;
    p.b_row = b.g.row;
    p.b_cols = b.g.cols;
    p.out = a.grad_weight;
    p.sums = a.grad_bias;
    if (a.grad_bias == nullptr) p.sums_part = nullptr;
    p.whole = whole_rows(a.grad_weight, a.c_out, a.c_out, 0);
    e = run_product(b.gw, stream);
    if (e != hipSuccess || p.part == nullptr) return e;
    auto join = [&](auto lanes) {
      constexpr int LANES = decltype(lanes)::value;
      k_join_groups<LANES><<<dim3(static_cast<unsigned>(div_up(join_pieces(p), 256 / LANES)), static_cast<unsigned>(p.groups)), 256, 0, stream>>>(p);
    };
    switch (join_lanes(p)) {
      case 1: join(std::integral_constant<int, 1>{}); break;
      case 4: join(std::integral_constant<int, 4>{}); break;
      default: join(std::integral_constant<int, 16>{}); break;
    }
    return hipGetLastError();
  }
  return hipSuccess;
}

hipError_t launch_activation_backward(const ActivationArgs& a, hipStream_t stream) {
  const int pieces = (a.cols + 7) / 8;
  const int64_t total = static_cast<int64_t>(a.rows) * pieces;
  if (total == 0) return hipSuccess;
  const bool w = whole_rows(a.grad, a.grad_row, a.cols, a.dtype) && whole_rows(a.pre, a.pre_row, a.cols, a.dtype) &&
                 whole_rows(a.out, a.out_row, a.cols, a.dtype);
  const unsigned blocks = static_cast<unsigned>(div_up(total, 256));
  const FastDiv by = make_fast_div(pieces);
  if (a.dtype == 0) k_activation_backward<float><<<blocks, 256, 0, stream>>>(a, pieces, by, w);
  else if (a.dtype == 1) k_activation_backward<_Float16><<<blocks, 256, 0, stream>>>(a, pieces, by, w);
  else k_activation_backward<__bf16><<<blocks, 256, 0, stream>>>(a, pieces, by, w);
  return hipGetLastError();
}

}  // namespace spconv
