// Host side of the C ABI declared in include/spconv.h: argument validation,
// stream-ordered memory, the single read-back of the map build, and kernel
// launches.  No compute happens here.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <new>
#include <string>
#include <utility>
#include <vector>

#include "../../include/spconv.h"
#include "internal.h"

namespace {

// Pinned host slot that receives one build's summary (written by the build's
// last kernel), with the event that marks its arrival.  Slots are reused; a
// slot released while its build may still be running is reclaimed only once
// its event has completed.
struct SummarySlot {
  long long* host = nullptr;
  long long* device = nullptr;  // the same memory, as the device addresses it
  hipEvent_t done = nullptr;
};

}  // namespace

struct spconv_map {
  int device = 0;
  hipStream_t stream = nullptr;
  int32_t K = 0;
  int32_t KV = 0;
  int64_t n = 0;      // output rows (the forward's rows and tiles)
  int64_t n_in = 0;   // input rows (n for a submanifold map)
  int32_t centre = 0;  // offset whose list is the identity, -1 for none
  int32_t stride = 1;
  int32_t kind = 0;    // SPCONV_MAP_SUBMANIFOLD, _STRIDED or _TRANSPOSED
  int32_t* out_coords = nullptr;  // [n][4] (strided and transposed maps; in the block)
  int32_t* in_coords = nullptr;   // [n_in][4] copy (strided and transposed maps; in the block)
  int64_t tiles = 0;
  void* block = nullptr;  // one pool allocation holding the MapBuffers
  size_t block_bytes = 0;
  spconv::MapBuffers buf;
  // Filled when the build's summary has been read (see finish_build).
  SummarySlot* slot = nullptr;   // non-null while the summary is not yet read
  spconv_status status = SPCONV_OK;
  std::string error;             // detail of a device-detected error
  int64_t total = 0;
  std::vector<int64_t> counts;   // KV
  std::vector<int64_t> offsets;  // KV + 1
};

// A copy of one layer's weights made for repeated forwards: the raw
// [K^3][C_in][C_out] copy and, for the shapes the wide and tiled paths take,
// the same weights in MFMA operand order with the zero row after them.
struct spconv_weights {
  int device = 0;
  int32_t KV = 0, c_in = 0, c_out = 0;
  spconv_dtype dtype = SPCONV_F32;
  void* raw = nullptr;
  void* prepared = nullptr;  // NULL for shapes that never use it
};

namespace {

thread_local std::string g_last_error;

spconv_status fail(spconv_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

spconv_status hip_fail(hipError_t e, const char* what) {
  const spconv_status st =
      (e == hipErrorOutOfMemory || e == hipErrorMemoryAllocation) ? SPCONV_ERR_OUT_OF_MEMORY
                                                                   : SPCONV_ERR_DEVICE;
  return fail(st, "%s: %s (%d)", what, hipGetErrorString(e), static_cast<int>(e));
}

#define SPCONV_HIP(call, what)                 \
  do {                                         \
    const hipError_t e_ = (call);              \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

// One stream-ordered pool per device, kept warm (no release at sync points),
// so per-build workspace and map buffers cost no driver allocation once the
// pool has grown.
std::mutex g_pool_mu;
std::vector<hipMemPool_t> g_pools;

spconv_status pool_for(int device, hipMemPool_t* out) {
  std::lock_guard<std::mutex> lock(g_pool_mu);
  if (static_cast<int>(g_pools.size()) <= device) g_pools.resize(device + 1, nullptr);
  if (g_pools[device] == nullptr) {
    hipMemPoolProps props;
    std::memset(&props, 0, sizeof(props));
    props.allocType = hipMemAllocationTypePinned;
    props.location.type = hipMemLocationTypeDevice;
    props.location.id = device;
    hipMemPool_t pool = nullptr;
    SPCONV_HIP(hipMemPoolCreate(&pool, &props), "hipMemPoolCreate");
    uint64_t keep = ~0ull;
    SPCONV_HIP(hipMemPoolSetAttribute(pool, hipMemPoolAttrReleaseThreshold, &keep),
               "hipMemPoolSetAttribute");
    g_pools[device] = pool;
  }
  *out = g_pools[device];
  return SPCONV_OK;
}

// Device buffers kept per (device, stream) between calls.  Work on one stream
// runs in order, so a buffer that earlier work on a stream has released can
// be handed to later work on the same stream with no allocator call (the
// pool's asynchronous malloc and free cost several microseconds of host time
// each, on every build and forward otherwise).  Buffers leave a stream only
// through the pool's stream-ordered free.
struct StreamCache {
  int device = 0;
  hipStream_t stream = nullptr;
  void* scratch = nullptr;  // map build workspace
  size_t scratch_bytes = 0;
  // Table slots of the last build launched on the scratch, whose table and
  // occupancy map it leaves clear (0: not known clear).
  int64_t clear_slots = 0;
  void* fwd = nullptr;  // forward workspace
  size_t fwd_bytes = 0;
  std::vector<std::pair<void*, size_t>> blocks;  // map blocks released on this stream
};
constexpr size_t kCachedBlocks = 4;
std::mutex g_cache_mu;
std::vector<StreamCache*> g_caches;

StreamCache* cache_for(int device, hipStream_t stream) {
  for (StreamCache* c : g_caches)
    if (c->device == device && c->stream == stream) return c;
  StreamCache* c = new StreamCache;
  c->device = device;
  c->stream = stream;
  g_caches.push_back(c);
  return c;
}

// Makes `buf` hold at least `need` bytes (grown with 25% headroom).
spconv_status grow_buffer(void*& buf, size_t& have, size_t need, hipMemPool_t pool, hipStream_t stream,
                          const char* what) {
  if (have >= need && buf != nullptr) return SPCONV_OK;
  if (buf != nullptr) (void)hipFreeAsync(buf, stream);
  buf = nullptr;
  have = 0;
  const size_t want = need + need / 4;
  SPCONV_HIP(hipMallocFromPoolAsync(&buf, want, pool, stream), what);
  have = want;
  return SPCONV_OK;
}

// A released map block of at least `need` bytes (and at most twice that),
// else a new one.
spconv_status take_block(StreamCache* c, size_t need, hipMemPool_t pool, void** out, size_t* bytes) {
  size_t best = c->blocks.size();
  for (size_t i = 0; i < c->blocks.size(); ++i) {
    const size_t b = c->blocks[i].second;
    if (b >= need && b <= 2 * need && (best == c->blocks.size() || b < c->blocks[best].second)) best = i;
  }
  if (best < c->blocks.size()) {
    *out = c->blocks[best].first;
    *bytes = c->blocks[best].second;
    c->blocks.erase(c->blocks.begin() + static_cast<std::ptrdiff_t>(best));
    return SPCONV_OK;
  }
  SPCONV_HIP(hipMallocFromPoolAsync(out, need, pool, c->stream), "map allocation");
  *bytes = need;
  return SPCONV_OK;
}

void release_block(int device, hipStream_t stream, void* block, size_t bytes) {
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(device, stream);
  if (c->blocks.size() < kCachedBlocks) {
    c->blocks.emplace_back(block, bytes);
  } else {
    (void)hipFreeAsync(block, stream);
  }
}

// Summary slots, one free list per device.  A slot holds enough for the
// largest kernel (K = 7).
constexpr size_t kSlotBytes = sizeof(long long) * (spconv::kSummaryHead + 343);
constexpr int kSlotsPerBatch = 16;

struct SlotPool {
  std::vector<SummarySlot*> free;
  std::vector<SummarySlot*> pending;  // released while their build may still write them
};
std::mutex g_slot_mu;
std::vector<SlotPool> g_slots;

spconv_status acquire_slot(int device, SummarySlot** out) {
  std::lock_guard<std::mutex> lock(g_slot_mu);
  if (static_cast<int>(g_slots.size()) <= device) g_slots.resize(device + 1);
  SlotPool& pool = g_slots[device];
  for (size_t i = 0; i < pool.pending.size();) {
    if (hipEventQuery(pool.pending[i]->done) == hipSuccess) {
      pool.free.push_back(pool.pending[i]);
      pool.pending[i] = pool.pending.back();
      pool.pending.pop_back();
    } else {
      ++i;
    }
  }
  if (pool.free.empty()) {
    void* p = nullptr;
    SPCONV_HIP(hipHostMalloc(&p, kSlotBytes * kSlotsPerBatch,
                             hipHostMallocPortable | hipHostMallocMapped | hipHostMallocCoherent),
               "hipHostMalloc");
    for (int i = 0; i < kSlotsPerBatch; ++i) {
      SummarySlot* slot = new (std::nothrow) SummarySlot;
      if (slot == nullptr) return fail(SPCONV_ERR_OUT_OF_MEMORY, "host allocation");
      slot->host = reinterpret_cast<long long*>(static_cast<char*>(p) + kSlotBytes * i);
      void* dp = nullptr;
      SPCONV_HIP(hipHostGetDevicePointer(&dp, slot->host, 0), "hipHostGetDevicePointer");
      slot->device = static_cast<long long*>(dp);
      SPCONV_HIP(hipEventCreateWithFlags(&slot->done, hipEventDisableTiming), "hipEventCreateWithFlags");
      pool.free.push_back(slot);
    }
  }
  *out = pool.free.back();
  pool.free.pop_back();
  return SPCONV_OK;
}

void release_slot(int device, SummarySlot* slot) {
  std::lock_guard<std::mutex> lock(g_slot_mu);
  g_slots[device].pending.push_back(slot);
}

// Waits for the build's summary (once) and records the counts or the device
// error it reports.
spconv_status finish_build(spconv_map* m) {
  if (m->slot != nullptr) {
    hipError_t e;
    // Spinning keeps the wake-up latency of a blocking wait off the critical path.
    while ((e = hipEventQuery(m->slot->done)) == hipErrorNotReady) {
    }
    const long long* sum = m->slot->host;
    if (e != hipSuccess) {
      m->status = hip_fail(e, "map build");
      m->error = g_last_error;
    } else {
      const unsigned long long flags = static_cast<unsigned long long>(sum[0]);
      if (flags & spconv::kFlagRange) {
        m->status = SPCONV_ERR_COORD_RANGE;
        m->error = "a coordinate is outside b in [0, 2^15), z, y, x in [0, 2^16)";
      } else if (flags & spconv::kFlagDuplicate) {
        m->status = SPCONV_ERR_DUPLICATE_COORD;
        m->error = "two rows share one (b, z, y, x) coordinate";
      } else if (flags & spconv::kFlagTableFull) {
        m->status = SPCONV_ERR_DEVICE;
        m->error = "internal: hash table probe exceeded its bound";
      } else {
        m->counts.assign(sum + spconv::kSummaryHead, sum + spconv::kSummaryHead + m->KV);
        m->offsets.resize(m->KV + 1);
        m->offsets[0] = 0;
        for (int k = 0; k < m->KV; ++k) m->offsets[k + 1] = m->offsets[k] + m->counts[k];
        m->total = m->offsets[m->KV];
      }
    }
    release_slot(m->device, m->slot);
    m->slot = nullptr;
  }
  if (m->status != SPCONV_OK) return fail(m->status, "%s", m->error.c_str());
  return SPCONV_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Fixed scratch of spconv_forward_noalloc: one array per device, held until
// the process ends, for the forward workspace (weights in MFMA operand order,
// the zero row and any fp32 partial outputs).  Host code never uses the
// array's name as an address: each device's address comes from
// hipGetSymbolAddress, taken once with that device current.
constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
static __device__ __align__(256) unsigned char scratch[kNoAllocScratchBytes];
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

spconv_status noalloc_scratch(int device, void** out) {
  if (device < 0 || device >= kMaxDevices) {
    return fail(SPCONV_ERR_UNSUPPORTED, "device %d beyond the %d the fixed scratch covers", device, kMaxDevices);
  }
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[device] == nullptr) {
    void* ptr = nullptr;
    SPCONV_HIP(hipGetSymbolAddress(&ptr, HIP_SYMBOL(scratch)), "hipGetSymbolAddress(scratch)");
    if (ptr == nullptr) return fail(SPCONV_ERR_DEVICE, "hipGetSymbolAddress(scratch) returned NULL");
    g_scratch_ptr[device] = ptr;
  }
  *out = g_scratch_ptr[device];
  return SPCONV_OK;
}

// Validates a forward call and fills its launch arguments.
spconv_status forward_args(const void* d_feats, const void* d_weights, const spconv_map* map, int32_t c_in,
                           int32_t c_out, spconv_dtype dtype, void* d_out, spconv::ForwardArgs* out) {
  // Checks that need no map first, then those that read it.
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if (d_weights == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "NULL weight pointer");
  if (!aligned16(d_feats) || !aligned16(d_weights) || !aligned16(d_out)) {
    return fail(SPCONV_ERR_INVALID_ARG, "feature, weight and output buffers must be 16-byte aligned");
  }
  if (dtype != SPCONV_F32 && dtype != SPCONV_F16 && dtype != SPCONV_BF16) {
    return fail(SPCONV_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  }
  const int32_t cmax = (dtype == SPCONV_F32) ? 512 : 1024;
  if (c_in < 1 || c_out < 1 || c_in > cmax || c_out > cmax) {
    return fail(SPCONV_ERR_INVALID_ARG, "c_in = %d, c_out = %d must lie in [1, %d]", c_in, c_out, cmax);
  }
  const int32_t mult = (dtype == SPCONV_F32) ? 4 : 8;
  if (c_in % mult != 0 || c_out % mult != 0) {
    return fail(SPCONV_ERR_UNSUPPORTED, "c_in = %d and c_out = %d must be multiples of %d", c_in,
                c_out, mult);
  }
  // A side with no rows (a strided map without outputs, or its transpose)
  // may be NULL: nothing of it is read or written.
  if ((d_feats == nullptr && map->n_in > 0) || (d_out == nullptr && map->n > 0)) {
    return fail(SPCONV_ERR_INVALID_ARG, "NULL feature or output pointer");
  }
  {
    // The output is written while other workgroups still read input rows and
    // weights: it must not share a byte with either.
    const uint64_t es = (dtype == SPCONV_F32) ? 4u : 2u;
    const uint64_t out_b = static_cast<uint64_t>(map->n) * c_out * es;
    const uint64_t in_b = static_cast<uint64_t>(map->n_in) * c_in * es;
    const uint64_t w_b = static_cast<uint64_t>(map->KV) * c_in * c_out * es;
    auto overlap = [](const void* p, uint64_t np, const void* q, uint64_t nq) {
      const uint64_t a0 = reinterpret_cast<uintptr_t>(p), b0 = reinterpret_cast<uintptr_t>(q);
      return a0 < b0 + nq && b0 < a0 + np;
    };
    if (overlap(d_out, out_b, d_feats, in_b) || overlap(d_out, out_b, d_weights, w_b)) {
      return fail(SPCONV_ERR_INVALID_ARG, "d_out overlaps the features or the weights");
    }
  }
  spconv::ForwardArgs& a = *out;
  a.feats = d_feats;
  a.weights = d_weights;
  a.out = d_out;
  a.in_idx = map->buf.in_idx;
  a.out_idx = map->buf.out_idx;
  a.tile_off = map->buf.tile_off;
  a.tile_mask = map->buf.tile_mask;
  a.tile_rows = map->buf.tile_rows;
  a.perm = map->buf.perm;
  a.n = map->n;
  a.tiles = map->tiles;
  a.KV = map->KV;
  a.cin = c_in;
  a.cout = c_out;
  a.dtype = static_cast<int32_t>(dtype);
  a.centre = map->centre;
  a.n_in = map->n_in;
  return SPCONV_OK;
}

// A map known to hold no entries (a strided map with no outputs, or its
// transpose): the forward writes zeros and launches no kernel.
bool known_empty(const spconv_map* map) { return map->slot == nullptr && map->total == 0; }

spconv_status zero_output(void* d_out, int64_t rows, int32_t c_out, spconv_dtype dtype, hipStream_t stream) {
  const size_t es = (dtype == SPCONV_F32) ? 4u : 2u;
  if (rows > 0) SPCONV_HIP(hipMemsetAsync(d_out, 0, static_cast<size_t>(rows) * c_out * es, stream), "hipMemsetAsync");
  return SPCONV_OK;
}

// Orders `stream` after the map's build when it is another stream than the
// build's and the build is not yet known complete.
spconv_status order_after_build(const spconv_map* map, hipStream_t stream) {
  if (stream != map->stream && map->slot != nullptr) {
    const hipError_t ew = hipStreamWaitEvent(stream, map->slot->done, 0);
    if (ew != hipSuccess) return hip_fail(ew, "hipStreamWaitEvent");
  }
  return SPCONV_OK;
}

enum class ForwardPath { kSmall, kWide, kTiled, kGeneric };

ForwardPath forward_path(const spconv::ForwardArgs& a) {
  if (spconv::small_supported(a)) return ForwardPath::kSmall;
  if (spconv::wide_supported(a)) return ForwardPath::kWide;
  if (spconv::tiled_supported(a)) return ForwardPath::kTiled;
  return ForwardPath::kGeneric;
}

size_t forward_workspace_bytes(ForwardPath path, const spconv::ForwardArgs& a) {
  if (path == ForwardPath::kWide) return spconv::wide_workspace_bytes(a);
  if (path == ForwardPath::kTiled) return a.prepared != nullptr ? 0 : spconv::tiled_workspace_bytes(a);
  return 0;
}

// Launches the forward's kernels; `ws` holds forward_workspace_bytes(path, a)
// bytes (unused by the small and generic paths).
spconv_status launch_forward_path(ForwardPath path, const spconv::ForwardArgs& a, void* ws, hipStream_t stream) {
  hipError_t e;
  switch (path) {
    case ForwardPath::kWide:
      e = a.prepared != nullptr ? hipSuccess : spconv::launch_prep_weights(a, ws, stream);
      if (e == hipSuccess) e = spconv::launch_forward_wide(a, ws, stream);
      break;
    case ForwardPath::kTiled:
      e = spconv::launch_forward_tiled(a, ws, stream);
      break;
    default:
      e = spconv::launch_forward(a, stream);
      break;
  }
  if (e != hipSuccess) return hip_fail(e, "forward launch");
  return SPCONV_OK;
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Block layout of a strided or transposed map: the lists (cap entries), tile
// offsets, masks and slot table over `tiles` output tiles, then the output
// and input coordinates.
struct GeneralLayout {
  size_t list_b, tile_off_b, mask_b, rows_b, out_c_b, in_c_b;
};
GeneralLayout general_layout(int64_t tiles, int32_t KV, int64_t cap, int64_t n_out, int64_t n_in, size_t* total) {
  GeneralLayout l;
  const size_t t = static_cast<size_t>(KV) * tiles;
  l.list_b = align256(static_cast<size_t>(cap) * sizeof(int32_t));
  l.tile_off_b = align256((t + 1) * sizeof(int32_t));
  l.mask_b = align256(std::max<size_t>(t, 1) * sizeof(unsigned long long));
  l.rows_b = align256(std::max<size_t>(static_cast<size_t>(tiles), 1) * spconv::kTileSlots * sizeof(int32_t));
  l.out_c_b = align256(std::max<size_t>(static_cast<size_t>(n_out), 1) * 4 * sizeof(int32_t));
  l.in_c_b = align256(std::max<size_t>(static_cast<size_t>(n_in), 1) * 4 * sizeof(int32_t));
  *total = 2 * l.list_b + l.tile_off_b + l.mask_b + l.rows_b + l.out_c_b + l.in_c_b;
  return l;
}
void carve_general(const GeneralLayout& l, spconv_map* m) {
  char* c = static_cast<char*>(m->block);
  m->buf.in_idx = reinterpret_cast<int32_t*>(c);
  c += l.list_b;
  m->buf.out_idx = reinterpret_cast<int32_t*>(c);
  c += l.list_b;
  m->buf.tile_off = reinterpret_cast<int32_t*>(c);
  c += l.tile_off_b;
  m->buf.tile_mask = reinterpret_cast<unsigned long long*>(c);
  c += l.mask_b;
  m->buf.tile_rows = reinterpret_cast<int32_t*>(c);
  c += l.rows_b;
  m->buf.perm = nullptr;
  m->out_coords = reinterpret_cast<int32_t*>(c);
  c += l.out_c_b;
  m->in_coords = reinterpret_cast<int32_t*>(c);
}

// A map with no entries: complete at once (no summary to wait for).
void mark_empty(spconv_map* m) {
  if (m->slot != nullptr) {
    release_slot(m->device, m->slot);
    m->slot = nullptr;
  }
  m->counts.assign(static_cast<size_t>(m->KV), 0);
  m->offsets.assign(static_cast<size_t>(m->KV) + 1, 0);
  m->total = 0;
}


// ---- grouped (weight-stationary) forward ----

spconv_status check_plan_args(double epsilon, double S) {
  if (!(epsilon >= 0.0) || !(S >= 0.0)) {
    return fail(SPCONV_ERR_INVALID_ARG, "epsilon = %g and S = %g must be >= 0 (S may be +inf)", epsilon, S);
  }
  return SPCONV_OK;
}

// Launches the grouped forward of `a` with `plan` from the stream's cached
// forward workspace.
spconv_status launch_grouped(const spconv_map* map, const spconv::ForwardArgs& a, const spconv::GroupPlan& plan,
                             hipStream_t stream) {
  hipMemPool_t pool = nullptr;
  spconv_status st = pool_for(map->device, &pool);
  if (st != SPCONV_OK) return st;
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(map->device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, spconv::grouped_workspace_bytes(a, plan), pool, stream,
                   "forward workspace allocation");
  if (st != SPCONV_OK) return st;
  const hipError_t e = spconv::launch_forward_grouped(a, plan, c->fwd, stream);
  if (e != hipSuccess) return hip_fail(e, "grouped forward launch");
  return SPCONV_OK;
}

// The fused forward (the path spconv_forward takes) from the stream's cache.
spconv_status launch_fused(const spconv_map* map, const spconv::ForwardArgs& a, hipStream_t stream) {
  const ForwardPath path = forward_path(a);
  const size_t ws_bytes = forward_workspace_bytes(path, a);
  if (ws_bytes == 0) return launch_forward_path(path, a, nullptr, stream);
  hipMemPool_t pool = nullptr;
  spconv_status st = pool_for(map->device, &pool);
  if (st != SPCONV_OK) return st;
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(map->device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, ws_bytes, pool, stream, "forward workspace allocation");
  if (st != SPCONV_OK) return st;
  return launch_forward_path(path, a, c->fwd, stream);
}

bool same_plan(const spconv::GroupPlan& x, const spconv::GroupPlan& y) {
  return x.entries == y.entries && x.entry_group == y.entry_group;
}

// ---- Attention, head norm and rotation ----

// Bytes that a [rows][heads][dim] tensor with these strides spans (0 when it
// has no values).
uint64_t span_bytes(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t dim, uint64_t es) {
  if (rows <= 0 || heads <= 0) return 0;
  return (static_cast<uint64_t>(rows - 1) * row_stride + static_cast<uint64_t>(heads - 1) * head_stride + dim) * es;
}

bool ranges_overlap(const void* p, uint64_t np, const void* q, uint64_t nq) {
  const uint64_t a0 = reinterpret_cast<uintptr_t>(p), b0 = reinterpret_cast<uintptr_t>(q);
  return np != 0 && nq != 0 && a0 < b0 + nq && b0 < a0 + np;
}

// A tensor argument of these operators.
struct Strided {
  const char* name;
  const void* p;
  int64_t rows, row_stride, heads, head_stride, dim;
  uint64_t es;
  uint64_t bytes() const { return span_bytes(rows, row_stride, heads, head_stride, dim, es); }
};

// A tile's rows are read with 32-bit offsets from its first one.
constexpr int64_t kMaxRowBytes = int64_t(1) << 24;

// Alignment, strides and size of a tensor; a written one must keep its rows
// and heads apart.
spconv_status check_strided(const Strided& t, bool written) {
  if (t.rows == 0 || t.heads == 0) return SPCONV_OK;  // nothing of it is read or written
  if (t.p == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "%s is NULL", t.name);
  if (!aligned16(t.p)) return fail(SPCONV_ERR_INVALID_ARG, "%s is not 16-byte aligned", t.name);
  const int64_t piece = static_cast<int64_t>(16 / t.es);
  if (t.row_stride < 0 || t.head_stride < 0 || t.row_stride % piece != 0 || t.head_stride % piece != 0 ||
      t.row_stride * static_cast<int64_t>(t.es) > kMaxRowBytes || t.head_stride > (int64_t(1) << 40) ||
      (t.row_stride != 0 && t.row_stride < t.dim)) {
    return fail(SPCONV_ERR_INVALID_ARG, "%s: row stride %lld (0, or head_dim and more, at most 2^24 bytes) and head stride %lld (at most 2^40) must be multiples of %lld elements, not negative",
                t.name, (long long)t.row_stride, (long long)t.head_stride, (long long)piece);
  }
  if (written) {
    // rows of heads, or heads of rows
    const bool by_rows = t.head_stride >= t.dim && t.row_stride >= (t.heads - 1) * t.head_stride + t.dim;
    const bool by_heads = t.row_stride >= t.dim && t.head_stride >= (t.rows - 1) * t.row_stride + t.dim;
    const bool one_row = t.rows == 1 && (t.heads == 1 || t.head_stride >= t.dim);
    const bool one_head = t.heads == 1 && t.row_stride >= t.dim;
    if (!by_rows && !by_heads && !one_row && !one_head) {
      return fail(SPCONV_ERR_INVALID_ARG, "%s: row stride %lld and head stride %lld let values overlap", t.name,
                  (long long)t.row_stride, (long long)t.head_stride);
    }
  }
  return SPCONV_OK;
}

spconv_status check_apart(const Strided& out, const Strided& in) {
  if (!ranges_overlap(out.p, out.bytes(), in.p, in.bytes())) return SPCONV_OK;
  // Slices of one buffer interleave without sharing a byte: both walk rows by
  // the same stride, and within a row they keep apart.
  const uint64_t row = static_cast<uint64_t>(out.row_stride) * out.es;
  if (out.row_stride == in.row_stride && out.es == in.es && row > 0) {
    const uint64_t a = reinterpret_cast<uintptr_t>(out.p), b = reinterpret_cast<uintptr_t>(in.p);
    const uint64_t wa = span_bytes(1, 0, out.heads, out.head_stride, out.dim, out.es);
    const uint64_t wb = span_bytes(1, 0, in.heads, in.head_stride, in.dim, in.es);
    const uint64_t gap = b >= a ? (b - a) % row : (row - (a - b) % row) % row;  // from out's row to in's next start
    if (gap >= wa && row - gap >= wb) return SPCONV_OK;
  }
  return fail(SPCONV_ERR_INVALID_ARG, "%s overlaps %s", out.name, in.name);
}

bool same_place(const Strided& a, const Strided& b) {
  return a.p == b.p && a.row_stride == b.row_stride && a.head_stride == b.head_stride;
}

spconv_status check_head_dim(int32_t dtype, int32_t dim) {
  if (dtype != SPCONV_F32 && dtype != SPCONV_F16 && dtype != SPCONV_BF16) {
    return fail(SPCONV_ERR_UNSUPPORTED, "dtype %d not supported", dtype);
  }
  if (dim < 8 || dim > 128 || dim % 8 != 0) {
    return fail(SPCONV_ERR_UNSUPPORTED, "head_dim = %d must be a multiple of 8 in [8, 128]", dim);
  }
  return SPCONV_OK;
}

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;

struct AttentionTensors {
  Strided q, k, v, out, lse;
};

// Validates the sizes of an attention call and fills them in: all that its
// launches, and so its workspace, depend on.
spconv_status attention_sizes(const spconv_attention* x, spconv::AttentionArgs* a) {
  if (x == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "args is NULL");
  const spconv_status st = check_head_dim(x->dtype, x->head_dim);
  if (st != SPCONV_OK) return st;
  if (x->batch < 0 || x->batch > (1 << 24)) return fail(SPCONV_ERR_INVALID_ARG, "batch = %d must lie in [0, 2^24]", x->batch);
  if (x->heads < 1 || x->kv_heads < 1 || x->heads % x->kv_heads != 0 || x->heads > 65535) {
    return fail(SPCONV_ERR_INVALID_ARG, "heads = %d (at most 65535) must be a positive multiple of kv_heads = %d", x->heads, x->kv_heads);
  }
  if (static_cast<int64_t>(x->batch + 2) * x->kv_heads > (int64_t(1) << 30)) {
    return fail(SPCONV_ERR_INVALID_ARG, "batch = %d x kv_heads = %d must stay below 2^30", x->batch, x->kv_heads);
  }
  if (x->total_q < 0 || x->total_k < 0 || x->total_q > kMaxRows / x->heads || x->total_k > kMaxRows / x->kv_heads ||
      x->total_q > (int64_t(1) << 30) || x->total_k > (int64_t(1) << 30)) {
    return fail(SPCONV_ERR_INVALID_ARG, "total_q = %lld, total_k = %lld: rows x heads must stay below 2^31 and rows below 2^30",
                (long long)x->total_q, (long long)x->total_k);
  }
  a->batch = x->batch;
  a->total_q = static_cast<int32_t>(x->total_q);
  a->total_k = static_cast<int32_t>(x->total_k);
  a->heads = x->heads;
  a->kv_heads = x->kv_heads;
  a->group = x->heads / x->kv_heads;
  a->dim = x->head_dim;
  a->by_group = spconv::make_fast_div(a->group);
  a->by_kv_heads = spconv::make_fast_div(a->kv_heads);
  // a bound past every row is none
  a->left = x->left < 0 || x->left >= (1 << 30) ? -1 : x->left;
  a->right = x->right < 0 || x->right >= (1 << 30) ? -1 : x->right;
  a->dtype = x->dtype;
  return SPCONV_OK;
}

// A call whose launches are larger than a dispatch can be.
spconv_status check_work_items(uint64_t items) {
  if (items <= spconv::kMaxWorkItems) return SPCONV_OK;
  return fail(SPCONV_ERR_INVALID_ARG, "the call takes %llu work items in one launch, of at most 2^32 - 1: split it", (unsigned long long)items);
}

// Validates an attention call and fills its launch arguments.
spconv_status attention_args(const spconv_attention* x, const void* d_out, const float* d_lse,
                             spconv::AttentionArgs* a, AttentionTensors* t) {
  const spconv_status st = attention_sizes(x, a);
  if (st != SPCONV_OK) return st;
  if (!(x->scale > 0.f) || !std::isfinite(x->scale)) return fail(SPCONV_ERR_INVALID_ARG, "scale = %g must be positive and finite", x->scale);
  if (x->cu_q == nullptr || x->cu_k == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "cu_q or cu_k is NULL");
  if ((reinterpret_cast<uintptr_t>(x->cu_q) | reinterpret_cast<uintptr_t>(x->cu_k) | reinterpret_cast<uintptr_t>(d_lse)) & 3u) {
    return fail(SPCONV_ERR_INVALID_ARG, "cu_q, cu_k and lse must be 4-byte aligned");
  }
  const uint64_t es = x->dtype == SPCONV_F32 ? 4u : 2u;
  const int64_t hd = static_cast<int64_t>(x->heads) * x->head_dim;
  t->q = {"q", x->q, x->total_q, x->q_row_stride, x->heads, x->q_head_stride, x->head_dim, es};
  t->k = {"k", x->k, x->total_k, x->k_row_stride, x->kv_heads, x->k_head_stride, x->head_dim, es};
  t->v = {"v", x->v, x->total_k, x->v_row_stride, x->kv_heads, x->v_head_stride, x->head_dim, es};
  t->out = {"out", d_out, x->total_q, hd, x->heads, x->head_dim, x->head_dim, es};
  t->lse = {"lse", d_lse, x->total_q, x->heads, 1, 0, x->heads, 4};
  for (const Strided* s : {&t->q, &t->k, &t->v, &t->out}) {
    const spconv_status e = check_strided(*s, false);
    if (e != SPCONV_OK) return e;
  }
  if (x->total_q > 0 && d_lse == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "lse is NULL");
  a->q = x->q;
  a->k = x->k;
  a->v = x->v;
  a->q_row = x->q_row_stride;
  a->q_head = x->q_head_stride;
  a->k_row = x->k_row_stride;
  a->k_head = x->k_head_stride;
  a->v_row = x->v_row_stride;
  a->v_head = x->v_head_stride;
  a->cu_q = x->cu_q;
  a->cu_k = x->cu_k;
  a->scale = x->scale;
  a->out = const_cast<void*>(d_out);
  a->lse = const_cast<float*>(d_lse);
  return SPCONV_OK;
}

// A workspace that the caller gives.
struct CallerWorkspace {
  void* p;
  uint64_t bytes;
};

// `launch` with a workspace of `need` bytes (NULL when none is needed): the
// caller's, which must keep apart from `tensors`, or else the stream's, held
// for this stream until the launches are enqueued.  A captured call must
// bring its own: the graph would keep the address of a buffer that the
// stream's later calls replace, and an allocation under capture would belong
// to the graph while the cache hands it to calls outside.
template <class F>
spconv_status with_workspace(size_t need, const CallerWorkspace* own, std::initializer_list<const Strided*> tensors, hipStream_t stream,
                             const char* what, F&& launch) {
  if (need == 0) {
    const hipError_t e = launch(static_cast<void*>(nullptr));
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, what);
  }
  if (own != nullptr) {
    if (own->p == nullptr || own->bytes < need) {
      return fail(SPCONV_ERR_INVALID_ARG, "the call needs %zu bytes of workspace, %llu given", need,
                  (unsigned long long)(own->p == nullptr ? 0 : own->bytes));
    }
    if (!aligned16(own->p)) return fail(SPCONV_ERR_INVALID_ARG, "the workspace is not 16-byte aligned");
    for (const Strided* t : tensors) {
      if (ranges_overlap(own->p, need, t->p, t->bytes())) return fail(SPCONV_ERR_INVALID_ARG, "the workspace overlaps %s", t->name);
    }
    const hipError_t e = launch(own->p);
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, what);
  }
  if (stream != nullptr) {  // (the null stream cannot be captured)
    hipStreamCaptureStatus capture = hipStreamCaptureStatusNone;
    SPCONV_HIP(hipStreamIsCapturing(stream, &capture), "hipStreamIsCapturing");
    if (capture != hipStreamCaptureStatusNone) {
      return fail(SPCONV_ERR_INVALID_ARG, "under graph capture this call needs a workspace of %zu bytes of the caller's (the _noalloc entry points)", need);
    }
  }
  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  hipMemPool_t pool = nullptr;
  spconv_status st = pool_for(device, &pool);
  if (st != SPCONV_OK) return st;
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, need, pool, stream, "workspace allocation");
  if (st != SPCONV_OK) return st;
  const hipError_t e = launch(c->fwd);
  return e == hipSuccess ? SPCONV_OK : hip_fail(e, what);
}

// Validates a norm and rotation call and fills its launch arguments.
spconv_status norm_rotary_args(const spconv_norm_rotary* x, spconv::NormRotaryArgs* a, Strided (&in)[2]) {
  if (x == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "args is NULL");
  const spconv_status st = check_head_dim(x->dtype, x->head_dim);
  if (st != SPCONV_OK) return st;
  if (x->q_heads < 0 || x->k_heads < 0 || x->rows < 0 || x->rows > (int64_t(1) << 30) ||
      (x->q_heads > 0 && x->rows > kMaxRows / x->q_heads) || (x->k_heads > 0 && x->rows > kMaxRows / x->k_heads)) {
    return fail(SPCONV_ERR_INVALID_ARG, "rows = %lld, q_heads = %d, k_heads = %d: rows x heads must stay below 2^31 and rows below 2^30",
                (long long)x->rows, x->q_heads, x->k_heads);
  }
  if (!(x->eps >= 0.f) || !std::isfinite(x->eps)) return fail(SPCONV_ERR_INVALID_ARG, "eps = %g must be finite and not negative", x->eps);
  if (x->interleaved != 0 && x->interleaved != 1) return fail(SPCONV_ERR_INVALID_ARG, "interleaved = %d must be 0 or 1", x->interleaved);
  if (x->rotary_dim < 0 || x->rotary_dim > x->head_dim) {
    return fail(SPCONV_ERR_INVALID_ARG, "rotary_dim = %d must lie in [0, head_dim = %d]", x->rotary_dim, x->head_dim);
  }
  if (x->rotary_dim > 0) {
    if (x->axes < 1 || x->axes > 4) return fail(SPCONV_ERR_INVALID_ARG, "axes = %d must lie in [1, 4]", x->axes);
    if (x->rotary_dim % (2 * x->axes) != 0) {
      return fail(SPCONV_ERR_UNSUPPORTED, "rotary_dim = %d must be a multiple of 2 axes = %d", x->rotary_dim, 2 * x->axes);
    }
    if (x->extent < 1 || x->extent > (1 << 24)) return fail(SPCONV_ERR_INVALID_ARG, "extent = %d must lie in [1, 2^24]", x->extent);
    if (x->rows > 0 && (x->table == nullptr || x->positions == nullptr)) return fail(SPCONV_ERR_INVALID_ARG, "table or positions is NULL");
    if ((reinterpret_cast<uintptr_t>(x->table) & 7u) || (reinterpret_cast<uintptr_t>(x->positions) & 3u)) {
      return fail(SPCONV_ERR_INVALID_ARG, "table must be 8-byte and positions 4-byte aligned");
    }
    if (x->position_row_stride < 0 || x->position_row_stride > (int64_t(1) << 31)) {
      return fail(SPCONV_ERR_INVALID_ARG, "position_row_stride = %lld must lie in [0, 2^31]", (long long)x->position_row_stride);
    }
  }
  if (!aligned16(x->q_weight) || !aligned16(x->k_weight)) return fail(SPCONV_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
  const uint64_t es = x->dtype == SPCONV_F32 ? 4u : 2u;
  in[0] = {"q", x->q, x->rows, x->q_row_stride, x->q_heads, x->q_head_stride, x->head_dim, es};
  in[1] = {"k", x->k, x->rows, x->k_row_stride, x->k_heads, x->k_head_stride, x->head_dim, es};
  for (int i = 0; i < 2; ++i) {
    const spconv_status e = check_strided(in[i], false);
    if (e != SPCONV_OK) return e;
    a->t[i].x = in[i].p;
    a->t[i].x_row = in[i].row_stride;
    a->t[i].x_head = in[i].head_stride;
    a->t[i].heads = static_cast<int32_t>(in[i].heads);
    if (in[i].heads > 0) a->t[i].by_heads = spconv::make_fast_div(a->t[i].heads);
  }
  a->t[0].weight = x->q_weight;
  a->t[1].weight = x->k_weight;
  a->rows = static_cast<int32_t>(x->rows);
  a->dim = x->head_dim;
  a->rotary = x->rotary_dim;
  a->axes = x->rotary_dim > 0 ? x->axes : 1;
  a->interleaved = x->interleaved;
  a->dtype = x->dtype;
  a->eps = x->eps;
  a->table = x->table;
  a->extent = x->extent;
  a->positions = x->positions;
  a->pos_row = x->position_row_stride;
  return SPCONV_OK;
}

spconv_status attention_forward(const spconv_attention* args, void* d_out, float* d_lse, const CallerWorkspace* own, void* hip_stream) {
  g_last_error.clear();
  spconv::AttentionArgs a;
  AttentionTensors t;
  spconv_status st = attention_args(args, d_out, d_lse, &a, &t);
  if (st != SPCONV_OK) return st;
  for (const Strided* out : {&t.out, &t.lse}) {
    for (const Strided* in : {&t.q, &t.k, &t.v}) {
      st = check_apart(*out, *in);
      if (st != SPCONV_OK) return st;
    }
  }
  st = check_apart(t.out, t.lse);
  if (st == SPCONV_OK) st = check_work_items(spconv::attention_work_items(a));
  if (st != SPCONV_OK) return st;
  if (a.total_q == 0) return SPCONV_OK;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::attention_workspace_bytes(a), own, {&t.q, &t.k, &t.v, &t.out, &t.lse}, stream, "attention launch",
                        [&](void* ws) { return spconv::launch_attention(a, ws, stream); });
}

spconv_status attention_backward(const spconv_attention* args, const void* d_out, const float* d_lse,
                                 const spconv_attention_gradients* grads, const CallerWorkspace* own, void* hip_stream) {
  g_last_error.clear();
  spconv::AttentionArgs a;
  AttentionTensors t;
  spconv_status st = attention_args(args, d_out, d_lse, &a, &t);
  if (st != SPCONV_OK) return st;
  if (grads == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "grads is NULL");
  const uint64_t es = t.q.es;
  const Strided go = {"grad_out", grads->grad_out, a.total_q, grads->grad_out_row_stride, a.heads, grads->grad_out_head_stride, a.dim, es};
  const Strided gq = {"grad_q", grads->grad_q, a.total_q, grads->grad_q_row_stride, a.heads, grads->grad_q_head_stride, a.dim, es};
  const Strided gk = {"grad_k", grads->grad_k, a.total_k, grads->grad_k_row_stride, a.kv_heads, grads->grad_k_head_stride, a.dim, es};
  const Strided gv = {"grad_v", grads->grad_v, a.total_k, grads->grad_v_row_stride, a.kv_heads, grads->grad_v_head_stride, a.dim, es};
  st = check_strided(go, false);
  if (st != SPCONV_OK) return st;
  for (const Strided* out : {&gq, &gk, &gv}) {
    st = check_strided(*out, true);
    if (st != SPCONV_OK) return st;
    for (const Strided& in : {t.q, t.k, t.v, t.out, t.lse, go}) {
      st = check_apart(*out, in);
      if (st != SPCONV_OK) return st;
    }
  }
  for (const auto& pair : {std::make_pair(&gq, &gk), std::make_pair(&gq, &gv), std::make_pair(&gk, &gv)}) {
    st = check_apart(*pair.first, *pair.second);
    if (st != SPCONV_OK) return st;
  }
  a.grad_out = go.p;
  a.go_row = go.row_stride;
  a.go_head = go.head_stride;
  a.grad_q = grads->grad_q;
  a.gq_row = gq.row_stride;
  a.gq_head = gq.head_stride;
  a.grad_k = grads->grad_k;
  a.gk_row = gk.row_stride;
  a.gk_head = gk.head_stride;
  a.grad_v = grads->grad_v;
  a.gv_row = gv.row_stride;
  a.gv_head = gv.head_stride;
  st = check_work_items(spconv::attention_backward_work_items(a));
  if (st != SPCONV_OK) return st;
  if (a.total_q == 0 && a.total_k == 0) return SPCONV_OK;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::attention_backward_workspace_bytes(a), own, {&t.q, &t.k, &t.v, &t.out, &t.lse, &go, &gq, &gk, &gv}, stream,
                        "attention backward launch",
                        [&](void* ws) { return spconv::launch_attention_backward(a, ws, stream); });
}

spconv_status norm_rotary_backward(const spconv_norm_rotary* args, const spconv_norm_rotary_gradients* grads, const CallerWorkspace* own,
                                   void* hip_stream) {
  g_last_error.clear();
  spconv::NormRotaryArgs a;
  Strided in[2];
  spconv_status st = norm_rotary_args(args, &a, in);
  if (st != SPCONV_OK) return st;
  if (grads == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "grads is NULL");
  if ((reinterpret_cast<uintptr_t>(grads->grad_q_weight) | reinterpret_cast<uintptr_t>(grads->grad_k_weight)) & 3u) {
    return fail(SPCONV_ERR_INVALID_ARG, "the weight gradients must be 4-byte aligned");
  }
  const Strided g[2] = {
      {"grad_q_out", grads->grad_q_out, a.rows, grads->grad_q_out_row_stride, a.t[0].heads, grads->grad_q_out_head_stride, a.dim, in[0].es},
      {"grad_k_out", grads->grad_k_out, a.rows, grads->grad_k_out_row_stride, a.t[1].heads, grads->grad_k_out_head_stride, a.dim, in[0].es}};
  const Strided gx[2] = {
      {"grad_q", grads->grad_q, a.rows, grads->grad_q_row_stride, a.t[0].heads, grads->grad_q_head_stride, a.dim, in[0].es},
      {"grad_k", grads->grad_k, a.rows, grads->grad_k_row_stride, a.t[1].heads, grads->grad_k_head_stride, a.dim, in[0].es}};
  for (int i = 0; i < 2; ++i) {
    st = check_strided(g[i], false);
    if (st == SPCONV_OK) st = check_strided(gx[i], true);
    for (int j = 0; j < 2 && st == SPCONV_OK; ++j) {
      st = check_apart(gx[i], in[j]);
      if (st == SPCONV_OK && (i != j || !same_place(gx[i], g[j]))) st = check_apart(gx[i], g[j]);
    }
    if (st != SPCONV_OK) return st;
    a.t[i].grad = g[i].p;
    a.t[i].g_row = g[i].row_stride;
    a.t[i].g_head = g[i].head_stride;
    a.t[i].grad_x = const_cast<void*>(gx[i].p);
    a.t[i].gx_row = gx[i].row_stride;
    a.t[i].gx_head = gx[i].head_stride;
  }
  st = check_apart(gx[0], gx[1]);
  if (st != SPCONV_OK) return st;
  a.t[0].grad_weight = grads->grad_q_weight;
  a.t[1].grad_weight = grads->grad_k_weight;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::norm_rotary_backward_workspace_bytes(a), own, {&in[0], &in[1], &g[0], &g[1], &gx[0], &gx[1]}, stream,
                        "norm and rotation backward launch",
                        [&](void* ws) { return spconv::launch_norm_rotary_backward(a, ws, stream); });
}

// ---- Row norm with the residual's addition, products of rows ----

spconv_status check_dtype(int32_t dtype) {
  if (dtype == SPCONV_F32 || dtype == SPCONV_F16 || dtype == SPCONV_BF16) return SPCONV_OK;
  return fail(SPCONV_ERR_UNSUPPORTED, "dtype %d not supported", dtype);
}

// A tensor [rows][dim] with a row stride of at least dim.  `piece`: addresses
// and strides are multiples of that many bytes.
Strided row_tensor(const char* name, const void* p, int64_t rows, int64_t row_stride, int64_t dim, uint64_t es) {
  return {name, p, rows, row_stride, 1, 0, dim, es};
}
spconv_status check_rows(const Strided& t, uint64_t base_piece, uint64_t stride_piece, int64_t most_bytes) {
  if (t.rows == 0) return SPCONV_OK;
  if (t.p == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "%s is NULL", t.name);
  if (reinterpret_cast<uintptr_t>(t.p) % base_piece != 0) return fail(SPCONV_ERR_INVALID_ARG, "%s is not %llu-byte aligned", t.name, (unsigned long long)base_piece);
  if (t.row_stride < t.dim || t.row_stride > most_bytes / static_cast<int64_t>(t.es) || static_cast<uint64_t>(t.row_stride) * t.es % stride_piece != 0) {
    return fail(SPCONV_ERR_INVALID_ARG, "%s: row stride %lld must be at least %lld, at most %lld bytes and a multiple of %llu bytes", t.name,
                (long long)t.row_stride, (long long)t.dim, (long long)most_bytes, (unsigned long long)stride_piece);
  }
  return SPCONV_OK;
}
// `out` keeps apart from `in`, or (in_place) is it.
spconv_status check_apart_or_same(const Strided& out, const Strided& in, bool in_place) {
  if (in_place && out.p == in.p && out.row_stride == in.row_stride) return SPCONV_OK;
  return check_apart(out, in);
}

spconv_status add_norm_args(const spconv_add_norm* x, spconv::AddNormArgs* a) {
  if (x == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "args is NULL");
  const spconv_status st = check_dtype(x->dtype);
  if (st != SPCONV_OK) return st;
  const int64_t es = x->dtype == SPCONV_F32 ? 4 : 2;
  if (x->channels < 8 || x->channels % 8 != 0 || x->channels > 32768 / es) {
    return fail(SPCONV_ERR_UNSUPPORTED, "channels = %d must be a multiple of 8 in [8, %lld]", x->channels, (long long)(32768 / es));
  }
  if (x->rows < 0 || x->rows > (int64_t(1) << 30)) return fail(SPCONV_ERR_INVALID_ARG, "rows = %lld must lie in [0, 2^30]", (long long)x->rows);
  if (!(x->eps >= 0.f) || !std::isfinite(x->eps)) return fail(SPCONV_ERR_INVALID_ARG, "eps = %g must be finite and not negative", x->eps);
  if (x->weight == nullptr || !aligned16(x->weight)) return fail(SPCONV_ERR_INVALID_ARG, "weight is NULL or not 16-byte aligned");
  a->weight = x->weight;
  a->rows = static_cast<int32_t>(x->rows);
  a->channels = x->channels;
  a->dtype = x->dtype;
  a->eps = x->eps;
  return check_work_items(spconv::add_norm_work_items(*a));
}

spconv_status add_norm_forward(const spconv_add_norm* args, void* d_h, int64_t h_row_stride, void* d_y, int64_t y_row_stride, void* hip_stream) {
  g_last_error.clear();
  spconv::AddNormArgs a;
  spconv_status st = add_norm_args(args, &a);
  if (st != SPCONV_OK) return st;
  const uint64_t es = a.dtype == SPCONV_F32 ? 4u : 2u;
  const bool add = args->residual != nullptr;
  const int64_t sum_rows = add ? a.rows : 0;  // (tensors of no rows are not looked at)
  const Strided x = row_tensor("x", args->x, a.rows, args->x_row_stride, a.channels, es);
  const Strided residual = row_tensor("residual", args->residual, sum_rows, args->residual_row_stride, a.channels, es);
  const Strided h = row_tensor("h", d_h, sum_rows, h_row_stride, a.channels, es);
  const Strided y = row_tensor("y", d_y, a.rows, y_row_stride, a.channels, es);
  const Strided weight = row_tensor("weight", a.weight, 1, a.channels, a.channels, es);
  if (!add && a.rows > 0 && d_h != nullptr) return fail(SPCONV_ERR_INVALID_ARG, "h is given without a residual");
  for (const Strided* t : {&x, &residual, &h, &y}) {
    st = check_rows(*t, 16, 16, kMaxRowBytes);
    if (st != SPCONV_OK) return st;
  }
  for (const Strided* out : {&h, &y}) {
    for (const Strided* in : {&x, &residual}) {
      st = check_apart_or_same(*out, *in, true);
      if (st != SPCONV_OK) return st;
    }
    st = check_apart(*out, weight);
    if (st != SPCONV_OK) return st;
  }
  st = check_apart(h, y);
  if (st != SPCONV_OK) return st;
  a.x = x.p;
  a.x_row = x.row_stride;
  a.residual = residual.p;
  a.residual_row = residual.row_stride;
  a.h = d_h;
  a.h_row = h_row_stride;
  a.y = d_y;
  a.y_row = y_row_stride;
  const hipError_t e = spconv::launch_add_norm(a, static_cast<hipStream_t>(hip_stream));
  return e == hipSuccess ? SPCONV_OK : hip_fail(e, "add and norm launch");
}

spconv_status add_norm_backward(const spconv_add_norm* args, const spconv_add_norm_gradients* grads, const CallerWorkspace* own, void* hip_stream) {
  g_last_error.clear();
  spconv::AddNormArgs a;
  spconv_status st = add_norm_args(args, &a);
  if (st != SPCONV_OK) return st;
  if (grads == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "grads is NULL");
  if (reinterpret_cast<uintptr_t>(grads->grad_weight) & 3u) return fail(SPCONV_ERR_INVALID_ARG, "grad_weight must be 4-byte aligned");
  const uint64_t es = a.dtype == SPCONV_F32 ? 4u : 2u;
  const Strided h = row_tensor("x (the sum h)", args->x, a.rows, args->x_row_stride, a.channels, es);
  const Strided gh = row_tensor("grad_h", grads->grad_h, grads->grad_h == nullptr ? 0 : a.rows, grads->grad_h_row_stride, a.channels, es);
  const Strided gy = row_tensor("grad_y", grads->grad_y, a.rows, grads->grad_y_row_stride, a.channels, es);
  const Strided grad = row_tensor("grad", grads->grad, a.rows, grads->grad_row_stride, a.channels, es);
  const Strided weight = row_tensor("weight", a.weight, 1, a.channels, a.channels, es);
  const Strided gw = row_tensor("grad_weight", grads->grad_weight, grads->grad_weight == nullptr ? 0 : 1, a.channels, a.channels, 4);
  for (const Strided* t : {&h, &gh, &gy, &grad}) {
    st = check_rows(*t, 16, 16, kMaxRowBytes);
    if (st != SPCONV_OK) return st;
  }
  st = check_apart(grad, h);
  if (st == SPCONV_OK) st = check_apart_or_same(grad, gh, true);
  if (st == SPCONV_OK) st = check_apart_or_same(grad, gy, true);
  if (st == SPCONV_OK) st = check_apart(grad, weight);
  for (const Strided* t : {&h, &gh, &gy, &grad, &weight})
    if (st == SPCONV_OK) st = check_apart(gw, *t);
  if (st != SPCONV_OK) return st;
  a.h = const_cast<void*>(h.p);
  a.h_row = h.row_stride;
  a.grad_h = gh.p;
  a.grad_h_row = gh.row_stride;
  a.grad_y = gy.p;
  a.grad_y_row = gy.row_stride;
  a.grad = grads->grad;
  a.grad_row = grad.row_stride;
  a.grad_weight = grads->grad_weight;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::add_norm_backward_workspace_bytes(a), own, {&h, &gh, &gy, &grad, &weight, &gw}, stream, "add and norm backward launch",
                        [&](void* ws) { return spconv::launch_add_norm_backward(a, ws, stream); });
}

constexpr int64_t kMaxLinearRowBytes = int64_t(1) << 22;

// The sizes of a product, all that its workspace depends on.
spconv_status linear_sizes(const spconv_linear* x, spconv::LinearArgs* a) {
  if (x == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "args is NULL");
  const spconv_status st = check_dtype(x->dtype);
  if (st != SPCONV_OK) return st;
  if (x->c_in < 1 || x->c_out < 1 || x->c_in > (1 << 18) || x->c_out > (1 << 18)) {
    return fail(SPCONV_ERR_INVALID_ARG, "c_in = %d and c_out = %d must lie in [1, 2^18]", x->c_in, x->c_out);
  }
  if (x->rows < 0 || x->rows > (int64_t(1) << 30)) return fail(SPCONV_ERR_INVALID_ARG, "rows = %lld must lie in [0, 2^30]", (long long)x->rows);
  if (x->groups < 1 || x->groups > 65535) return fail(SPCONV_ERR_INVALID_ARG, "groups = %d must lie in [1, 65535]", x->groups);
  if (x->cu == nullptr && x->groups != 1) return fail(SPCONV_ERR_INVALID_ARG, "groups = %d need their row offsets", x->groups);
  if (x->activation < SPCONV_ACT_NONE || x->activation > SPCONV_ACT_GELU) return fail(SPCONV_ERR_INVALID_ARG, "activation = %d is none", x->activation);
  const int64_t es = x->dtype == SPCONV_F32 ? 4 : 2;
  if (x->rows > 0 && (x->x_row_stride < x->c_in || x->x_row_stride > kMaxLinearRowBytes / es)) {
    return fail(SPCONV_ERR_INVALID_ARG, "x: row stride %lld must be at least %d and at most 2^22 bytes", (long long)x->x_row_stride, x->c_in);
  }
  a->x_row = x->x_row_stride;
  a->cu = x->cu;
  a->rows = static_cast<int32_t>(x->rows);
  a->groups = x->groups;
  a->c_in = x->c_in;
  a->c_out = x->c_out;
  a->act = x->activation;
  a->dtype = x->dtype;
  a->grad_out_row = x->c_out;  // (or any whole number of pieces, which needs no more workspace)
  return SPCONV_OK;
}

struct LinearTensors {
  Strided x, weight, cu;
};
spconv_status linear_args(const spconv_linear* x, spconv::LinearArgs* a, LinearTensors* t) {
  const spconv_status st = linear_sizes(x, a);
  if (st != SPCONV_OK) return st;
  const uint64_t es = a->dtype == SPCONV_F32 ? 4u : 2u;
  t->x = row_tensor("x", x->x, a->rows, x->x_row_stride, a->c_in, es);
  t->weight = row_tensor("weight", x->weight, static_cast<int64_t>(a->groups) * a->c_in, a->c_out, a->c_out, es);
  t->cu = row_tensor("cu", x->cu, x->cu == nullptr ? 0 : 1, a->groups + 1, a->groups + 1, 4);
  spconv_status e = check_rows(t->x, 16, es, kMaxLinearRowBytes);
  if (e == SPCONV_OK) e = check_rows(t->weight, 16, es, kMaxLinearRowBytes);
  if (e == SPCONV_OK) e = check_rows(t->cu, 4, 4, int64_t(1) << 40);
  a->x = x->x;
  a->weight = x->weight;
  return e;
}

spconv_status linear_forward(const spconv_linear* args, const spconv_linear_epilogue* epilogue, const CallerWorkspace* own, void* hip_stream) {
  g_last_error.clear();
  spconv::LinearArgs a;
  LinearTensors t;
  spconv_status st = linear_args(args, &a, &t);
  if (st != SPCONV_OK) return st;
  if (epilogue == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "epilogue is NULL");
  const uint64_t es = t.x.es;
  const spconv_linear_epilogue& p = *epilogue;
  const Strided bias = row_tensor("bias", p.bias, p.bias == nullptr ? 0 : a.groups, a.c_out, a.c_out, es);
  const Strided residual = row_tensor("residual", p.residual, p.residual == nullptr ? 0 : a.rows, p.residual_row_stride, a.c_out, es);
  const Strided pre = row_tensor("pre", p.pre, p.pre == nullptr ? 0 : a.rows, p.pre_row_stride, a.c_out, es);
  const Strided out = row_tensor("out", p.out, a.rows, p.out_row_stride, a.c_out, es);
  for (const Strided* s : {&bias, &residual, &pre, &out}) {
    st = check_rows(*s, es, es, kMaxLinearRowBytes);
    if (st != SPCONV_OK) return st;
  }
  for (const Strided* o : {&out, &pre}) {
    for (const Strided& in : {t.x, t.weight, t.cu, bias}) {
      st = check_apart(*o, in);
      if (st != SPCONV_OK) return st;
    }
    st = check_apart_or_same(*o, residual, o == &out);
    if (st != SPCONV_OK) return st;
  }
  st = check_apart(out, pre);
  if (st == SPCONV_OK) st = check_work_items(spconv::linear_work_items(a, false));
  if (st != SPCONV_OK) return st;
  if (a.rows == 0) return SPCONV_OK;
  a.bias = p.bias;
  a.residual = p.residual;
  a.residual_row = p.residual_row_stride;
  a.pre = p.pre;
  a.pre_row = p.pre_row_stride;
  a.out = p.out;
  a.out_row = p.out_row_stride;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::linear_workspace_bytes(a), own, {&t.x, &t.weight, &t.cu, &bias, &residual, &pre, &out}, stream, "linear launch",
                        [&](void* ws) { return spconv::launch_linear(a, ws, stream); });
}

spconv_status linear_backward(const spconv_linear* args, const spconv_linear_gradients* grads, const CallerWorkspace* own, void* hip_stream) {
  g_last_error.clear();
  spconv::LinearArgs a;
  LinearTensors t;
  spconv_status st = linear_args(args, &a, &t);
  if (st != SPCONV_OK) return st;
  if (grads == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "grads is NULL");
  const uint64_t es = t.x.es;
  const spconv_linear_gradients& g = *grads;
  if (g.before != nullptr && a.act == SPCONV_ACT_NONE) return fail(SPCONV_ERR_INVALID_ARG, "before needs its activation");
  if (g.grad_bias != nullptr && g.grad_weight == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "grad_bias needs grad_weight");
  const Strided go = row_tensor("grad_out", g.grad_out, a.rows, g.grad_out_row_stride, a.c_out, es);
  const Strided before = row_tensor("before", g.before, g.before == nullptr ? 0 : a.rows, g.before_row_stride, a.c_in, es);
  const Strided gx = row_tensor("grad_x", g.grad_x, g.grad_x == nullptr ? 0 : a.rows, g.grad_x_row_stride, a.c_in, es);
  const Strided gw = row_tensor("grad_weight", g.grad_weight, g.grad_weight == nullptr ? 0 : static_cast<int64_t>(a.groups) * a.c_in, a.c_out, a.c_out, 4);
  const Strided gb = row_tensor("grad_bias", g.grad_bias, g.grad_bias == nullptr ? 0 : a.groups, a.c_out, a.c_out, 4);
  st = check_rows(go, 16, a.c_out * es % 16 == 0 ? 16 : es, kMaxLinearRowBytes);
  for (const Strided* s : {&before, &gx})
    if (st == SPCONV_OK) st = check_rows(*s, es, es, kMaxLinearRowBytes);
  for (const Strided* s : {&gw, &gb})
    if (st == SPCONV_OK) st = check_rows(*s, 4, 4, kMaxLinearRowBytes);
  for (const Strided* o : {&gx, &gw, &gb})
    for (const Strided& in : {t.x, t.weight, t.cu, go, before})
      if (st == SPCONV_OK) st = check_apart(*o, in);
  if (st == SPCONV_OK) st = check_apart(gx, gw);
  if (st == SPCONV_OK) st = check_apart(gx, gb);
  if (st == SPCONV_OK) st = check_apart(gw, gb);
  if (st != SPCONV_OK) return st;
  a.grad_out = g.grad_out;
  if (a.rows > 0) a.grad_out_row = g.grad_out_row_stride;
  a.before = g.before;
  a.before_row = g.before_row_stride;
  a.grad_x = g.grad_x;
  a.grad_x_row = g.grad_x_row_stride;
  a.grad_weight = g.grad_weight;
  a.grad_bias = g.grad_bias;
  st = check_work_items(spconv::linear_work_items(a, true));
  if (st != SPCONV_OK) return st;
  if (a.grad_weight == nullptr && (a.rows == 0 || a.grad_x == nullptr)) return SPCONV_OK;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  return with_workspace(spconv::linear_backward_workspace_bytes(a), own, {&t.x, &t.weight, &t.cu, &go, &before, &gx, &gw, &gb}, stream,
                        "linear backward launch", [&](void* ws) { return spconv::launch_linear_backward(a, ws, stream); });
}

spconv_status activation_backward(const void* d_grad_out, int64_t grad_out_row_stride, const void* d_pre, int64_t pre_row_stride, void* d_grad_pre,
                                  int64_t grad_pre_row_stride, int64_t rows, int32_t channels, int32_t activation, int32_t dtype, void* hip_stream) {
  g_last_error.clear();
  spconv_status st = check_dtype(dtype);
  if (st != SPCONV_OK) return st;
  if (rows < 0 || rows > (int64_t(1) << 30) || channels < 1 || channels > (1 << 18)) {
    return fail(SPCONV_ERR_INVALID_ARG, "rows = %lld must lie in [0, 2^30] and channels = %d in [1, 2^18]", (long long)rows, channels);
  }
  if (activation < SPCONV_ACT_NONE || activation > SPCONV_ACT_GELU) return fail(SPCONV_ERR_INVALID_ARG, "activation = %d is none", activation);
  const uint64_t es = dtype == SPCONV_F32 ? 4u : 2u;
  const Strided g = row_tensor("grad_out", d_grad_out, rows, grad_out_row_stride, channels, es);
  const Strided pre = row_tensor("pre", d_pre, rows, pre_row_stride, channels, es);
  const Strided out = row_tensor("grad_pre", d_grad_pre, rows, grad_pre_row_stride, channels, es);
  for (const Strided* t : {&g, &pre, &out}) {
    st = check_rows(*t, es, es, kMaxLinearRowBytes);
    if (st != SPCONV_OK) return st;
  }
  st = check_apart_or_same(out, g, true);
  if (st == SPCONV_OK) st = check_apart(out, pre);
  if (st == SPCONV_OK) st = check_work_items(static_cast<uint64_t>(rows) * ((channels + 7) / 8) + 256);
  if (st != SPCONV_OK) return st;
  spconv::ActivationArgs a;
  a.grad = d_grad_out;
  a.pre = d_pre;
  a.out = d_grad_pre;
  a.grad_row = grad_out_row_stride;
  a.pre_row = pre_row_stride;
  a.out_row = grad_pre_row_stride;
  a.rows = static_cast<int32_t>(rows);
  a.cols = channels;
  a.act = activation;
  a.dtype = dtype;
  const hipError_t e = spconv::launch_activation_backward(a, static_cast<hipStream_t>(hip_stream));
  return e == hipSuccess ? SPCONV_OK : hip_fail(e, "activation backward launch");
}

// Nothing throws across the ABI: a host allocation that fails becomes a status.
template <class F>
spconv_status guarded(F&& f) {
  try {
    return f();
  } catch (const std::bad_alloc&) {
    return SPCONV_ERR_OUT_OF_MEMORY;
  } catch (...) {
    return SPCONV_ERR_DEVICE;
  }
}
}  // namespace

extern "C" {

int32_t spconv_abi_version(void) { return 5; }

const char* spconv_status_string(spconv_status s) {
  switch (s) {
    case SPCONV_OK: return "SPCONV_OK";
    case SPCONV_ERR_INVALID_ARG: return "SPCONV_ERR_INVALID_ARG";
    case SPCONV_ERR_DUPLICATE_COORD: return "SPCONV_ERR_DUPLICATE_COORD";
    case SPCONV_ERR_COORD_RANGE: return "SPCONV_ERR_COORD_RANGE";
    case SPCONV_ERR_UNSUPPORTED: return "SPCONV_ERR_UNSUPPORTED";
    case SPCONV_ERR_OUT_OF_MEMORY: return "SPCONV_ERR_OUT_OF_MEMORY";
    case SPCONV_ERR_DEVICE: return "SPCONV_ERR_DEVICE";
  }
  return "SPCONV_ERR_UNKNOWN";
}

const char* spconv_last_error(void) { return g_last_error.c_str(); }

spconv_status spconv_build_map_async(const int32_t* d_coords, int64_t n, int32_t kernel_size,
                                     void* hip_stream, spconv_map** out_map) {
  g_last_error.clear();
  if (out_map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "out_map is NULL");
  *out_map = nullptr;
  if (d_coords == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "d_coords is NULL");
  if (!aligned16(d_coords)) return fail(SPCONV_ERR_INVALID_ARG, "d_coords is not 16-byte aligned");
  if (n <= 0) return fail(SPCONV_ERR_INVALID_ARG, "n = %lld must be positive", (long long)n);
  if (kernel_size != 1 && kernel_size != 3 && kernel_size != 5 && kernel_size != 7) {
    return fail(SPCONV_ERR_UNSUPPORTED, "kernel_size = %d not in {1, 3, 5, 7}", kernel_size);
  }
  const int32_t KV = kernel_size * kernel_size * kernel_size;
  if (n >= (int64_t(1) << 31) / KV) {
    return fail(SPCONV_ERR_INVALID_ARG, "n x K^3 = %lld x %d must stay below 2^31",
                (long long)n, KV);
  }
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);

  const spconv::BuildPlan p = spconv::make_plan(n, kernel_size);

  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  hipMemPool_t pool = nullptr;
  spconv_status st = pool_for(device, &pool);
  if (st != SPCONV_OK) return st;

  spconv_map* m = new (std::nothrow) spconv_map;
  if (m == nullptr) return fail(SPCONV_ERR_OUT_OF_MEMORY, "host allocation");
  st = acquire_slot(device, &m->slot);
  if (st != SPCONV_OK) {
    delete m;
    return st;
  }
  // The stream's build workspace and a map block (both reused across builds
  // on this stream); the cache lock also serialises enqueueing on a stream.
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(device, stream);
  void* const scratch_before = c->scratch;
  st = grow_buffer(c->scratch, c->scratch_bytes, spconv::build_scratch_bytes(p), pool, stream,
                   "workspace allocation");
  if (c->scratch != scratch_before) c->clear_slots = 0;  // new memory
  if (st == SPCONV_OK) st = take_block(c, spconv::map_buffer_bytes(p), pool, &m->block, &m->block_bytes);
  if (st != SPCONV_OK) {
    release_slot(device, m->slot);
    delete m;
    return st;
  }
  spconv::BuildScratch s;
  spconv::carve_build_scratch(p, c->scratch, &s);
  spconv::carve_map_buffers(p, m->block, &m->buf);
  auto discard = [&](spconv_status st) {
    (void)hipFreeAsync(m->block, stream);
    release_slot(device, m->slot);
    delete m;
    return st;
  };

  // The table sits at the start of the scratch, so a clear table of the same
  // size is this build's table.  Until the launches succeed it is not known
  // clear.
  const bool table_clear = c->clear_slots == p.table_slots;
  c->clear_slots = 0;
  hipError_t e = spconv::launch_build(p, d_coords, s, m->buf, m->slot->device, table_clear, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "map build launch"));
  c->clear_slots = p.ordered ? 0 : p.table_slots;  // k_compact leaves an unordered map's table clear
  e = hipEventRecord(m->slot->done, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "hipEventRecord"));

  m->device = device;
  m->stream = stream;
  m->K = kernel_size;
  m->KV = KV;
  m->n = n;
  m->n_in = n;
  m->centre = (KV - 1) / 2;
  m->tiles = p.tiles;
  *out_map = m;
  return SPCONV_OK;
}

spconv_status spconv_build_map(const int32_t* d_coords, int64_t n, int32_t kernel_size,
                               void* hip_stream, spconv_map** out_map) {
  spconv_status st = spconv_build_map_async(d_coords, n, kernel_size, hip_stream, out_map);
  if (st != SPCONV_OK) return st;
  st = finish_build(*out_map);
  if (st != SPCONV_OK) {
    spconv_map_free(*out_map);
    *out_map = nullptr;
  }
  return st;
}

spconv_status spconv_map_wait(spconv_map* map) {
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  return finish_build(map);
}

spconv_status spconv_map_info(spconv_map* map, int32_t* kernel_size, int64_t* n,
                              int64_t* total_entries) {
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if (kernel_size) *kernel_size = map->K;
  if (n) *n = map->n;
  if (total_entries) {
    const spconv_status st = finish_build(map);
    if (st != SPCONV_OK) return st;
    *total_entries = map->total;
  }
  return SPCONV_OK;
}

spconv_status spconv_map_counts(spconv_map* map, int64_t* h_counts, int64_t* h_offsets) {
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  const spconv_status st = finish_build(map);
  if (st != SPCONV_OK) return st;
  if (h_counts) std::memcpy(h_counts, map->counts.data(), sizeof(int64_t) * map->KV);
  if (h_offsets) std::memcpy(h_offsets, map->offsets.data(), sizeof(int64_t) * (map->KV + 1));
  return SPCONV_OK;
}

spconv_status spconv_map_lists(const spconv_map* map, const int32_t** d_in_idx,
                               const int32_t** d_out_idx) {
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if (d_in_idx) *d_in_idx = map->buf.in_idx;
  if (d_out_idx) *d_out_idx = map->buf.out_idx;
  return SPCONV_OK;
}

spconv_status spconv_forward(const void* d_feats, const void* d_weights, const spconv_map* map,
                             int32_t c_in, int32_t c_out, spconv_dtype dtype, void* d_out,
                             void* hip_stream) {
  g_last_error.clear();
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_feats, d_weights, map, c_in, c_out, dtype, d_out, &a);
  if (st != SPCONV_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  if (known_empty(map)) return zero_output(d_out, map->n, c_out, dtype, stream);
  const ForwardPath path = forward_path(a);
  const size_t ws_bytes = forward_workspace_bytes(path, a);
  if (ws_bytes == 0) return launch_forward_path(path, a, nullptr, stream);
  hipMemPool_t pool = nullptr;
  st = pool_for(map->device, &pool);
  if (st != SPCONV_OK) return st;
  // The stream's forward workspace (prepared weights, zero row, partials),
  // reused by later forwards on the stream.
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(map->device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, ws_bytes, pool, stream, "forward workspace allocation");
  if (st != SPCONV_OK) return st;
  return launch_forward_path(path, a, c->fwd, stream);
}

spconv_status spconv_forward_noalloc(const void* d_feats, const void* d_weights, const spconv_map* map,
                                     int32_t c_in, int32_t c_out, spconv_dtype dtype, void* d_out,
                                     void* hip_stream) {
  g_last_error.clear();
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_feats, d_weights, map, c_in, c_out, dtype, d_out, &a);
  if (st != SPCONV_OK) return st;
  const ForwardPath path = forward_path(a);
  const size_t ws_bytes = forward_workspace_bytes(path, a);
  if (ws_bytes > kNoAllocScratchBytes) {
    return fail(SPCONV_ERR_UNSUPPORTED,
                "this forward needs %zu bytes of workspace; the fixed scratch of spconv_forward_noalloc holds %zu",
                ws_bytes, kNoAllocScratchBytes);
  }
  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  if (device != map->device) {
    return fail(SPCONV_ERR_INVALID_ARG, "the current device (%d) is not the map's (%d)", device, map->device);
  }
  void* ws = nullptr;
  if (ws_bytes > 0) {
    st = noalloc_scratch(device, &ws);
    if (st != SPCONV_OK) return st;
  }
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  if (known_empty(map)) return zero_output(d_out, map->n, c_out, dtype, stream);
  return launch_forward_path(path, a, ws, stream);
}

spconv_status spconv_weights_prepare(const void* d_weights, int32_t kernel_volume, int32_t c_in, int32_t c_out,
                                     spconv_dtype dtype, void* hip_stream, spconv_weights** out) {
  g_last_error.clear();
  if (out == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (d_weights == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "NULL weight pointer");
  if (!aligned16(d_weights)) return fail(SPCONV_ERR_INVALID_ARG, "the weights must be 16-byte aligned");
  if (dtype != SPCONV_F32 && dtype != SPCONV_F16 && dtype != SPCONV_BF16) {
    return fail(SPCONV_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  }
  if (kernel_volume < 1 || kernel_volume > 343) {
    return fail(SPCONV_ERR_INVALID_ARG, "kernel_volume = %d must lie in [1, 343]", kernel_volume);
  }
  const int32_t cmax = (dtype == SPCONV_F32) ? 512 : 1024;
  if (c_in < 1 || c_out < 1 || c_in > cmax || c_out > cmax) {
    return fail(SPCONV_ERR_INVALID_ARG, "c_in = %d, c_out = %d must lie in [1, %d]", c_in, c_out, cmax);
  }
  const int32_t mult = (dtype == SPCONV_F32) ? 4 : 8;
  if (c_in % mult != 0 || c_out % mult != 0) {
    return fail(SPCONV_ERR_UNSUPPORTED, "c_in = %d and c_out = %d must be multiples of %d", c_in, c_out, mult);
  }
  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  auto* w = new (std::nothrow) spconv_weights;
  if (w == nullptr) return fail(SPCONV_ERR_OUT_OF_MEMORY, "host allocation of the weight handle");
  w->device = device;
  w->KV = kernel_volume;
  w->c_in = c_in;
  w->c_out = c_out;
  w->dtype = dtype;
  const size_t raw_b = static_cast<size_t>(kernel_volume) * c_in * c_out * (dtype == SPCONV_F32 ? 4 : 2);
  // The operand-order copy exists for the shapes of the wide and tiled paths
  // (F16/BF16, C_in in {32, 64, 128, 256}, C_out a multiple of 16, K^3 <= 128).
  spconv::ForwardArgs a;
  a.weights = d_weights;
  a.KV = kernel_volume;
  a.cin = c_in;
  a.cout = c_out;
  a.dtype = static_cast<int32_t>(dtype);
  const bool with_prepared = dtype != SPCONV_F32 && kernel_volume <= 128 && c_out % 16 == 0 &&
                             (c_in == 32 || c_in == 64 || c_in == 128 || c_in == 256);
  hipError_t e = hipMalloc(&w->raw, raw_b);
  if (e == hipSuccess && with_prepared) e = hipMalloc(&w->prepared, spconv::tiled_workspace_bytes(a));
  if (e != hipSuccess) {
    spconv_weights_free(w);
    return e == hipErrorOutOfMemory ? fail(SPCONV_ERR_OUT_OF_MEMORY, "weight copy allocation")
                                    : hip_fail(e, "weight copy allocation");
  }
  e = hipMemcpyAsync(w->raw, d_weights, raw_b, hipMemcpyDeviceToDevice, stream);
  if (e == hipSuccess && with_prepared) e = spconv::launch_prep_weights(a, w->prepared, stream);
  if (e != hipSuccess) {
    spconv_weights_free(w);
    return hip_fail(e, "weight preparation");
  }
  *out = w;
  return SPCONV_OK;
}

spconv_status spconv_forward_prepared(const void* d_feats, const spconv_weights* weights, const spconv_map* map,
                                      void* d_out, void* hip_stream) {
  g_last_error.clear();
  if (weights == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "weights is NULL");
  if (map != nullptr && map->KV != weights->KV) {
    return fail(SPCONV_ERR_INVALID_ARG, "the map has %d offsets, the weights %d", map->KV, weights->KV);
  }
  if (map != nullptr && map->device != weights->device) {
    return fail(SPCONV_ERR_INVALID_ARG, "the map is on device %d, the weights on %d", map->device, weights->device);
  }
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_feats, weights->raw, map, weights->c_in, weights->c_out, weights->dtype, d_out,
                                  &a);
  if (st != SPCONV_OK) return st;
  a.prepared = weights->prepared;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  if (known_empty(map)) return zero_output(d_out, map->n, weights->c_out, weights->dtype, stream);
  return launch_fused(map, a, stream);
}

void spconv_weights_free(spconv_weights* weights) {
  if (weights == nullptr) return;
  // hipFree waits for the device's work in flight, which may still read them.
  if (weights->raw != nullptr) (void)hipFree(weights->raw);
  if (weights->prepared != nullptr) (void)hipFree(weights->prepared);
  delete weights;
}

spconv_status spconv_backward_data(const void* d_grad_out, const void* d_weights, const spconv_map* map,
                                   int32_t c_in, int32_t c_out, spconv_dtype dtype, void* d_grad_in,
                                   void* hip_stream) {
  g_last_error.clear();
  if (map != nullptr && map->kind != SPCONV_MAP_SUBMANIFOLD) {
    return fail(SPCONV_ERR_UNSUPPORTED,
                "the data gradient of a strided or transposed map is the forward over its transpose "
                "(spconv_map_transpose) with the weights W[k]^T");
  }
  // The data gradient is the forward of grad_out over the same map with the
  // mirrored, transposed weights: C_out channels in, C_in out.
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_grad_out, d_weights, map, c_out, c_in, dtype, d_grad_in, &a);
  if (st != SPCONV_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  const size_t mirror_bytes = spconv::mirror_workspace_bytes(map->KV, c_in, c_out, static_cast<int>(dtype));
  const ForwardPath path = forward_path(a);
  const size_t ws_bytes = mirror_bytes + forward_workspace_bytes(path, a);
  hipMemPool_t pool = nullptr;
  st = pool_for(map->device, &pool);
  if (st != SPCONV_OK) return st;
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(map->device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, ws_bytes, pool, stream, "backward workspace allocation");
  if (st != SPCONV_OK) return st;
  const hipError_t e = spconv::launch_mirror_transpose(d_weights, c->fwd, map->KV, c_in, c_out,
                                                       static_cast<int>(dtype), stream);
  if (e != hipSuccess) return hip_fail(e, "weight mirror launch");
  a.weights = c->fwd;
  return launch_forward_path(path, a, static_cast<char*>(c->fwd) + mirror_bytes, stream);
}

spconv_status spconv_backward_weights(const void* d_feats, const void* d_grad_out, const spconv_map* map,
                                      int32_t c_in, int32_t c_out, spconv_dtype dtype, float* d_grad_w,
                                      void* hip_stream) {
  g_last_error.clear();
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if ((d_feats == nullptr && map->n_in > 0) || (d_grad_out == nullptr && map->n > 0) || d_grad_w == nullptr) {
    return fail(SPCONV_ERR_INVALID_ARG, "NULL feature, gradient or weight-gradient pointer");
  }
  if (!aligned16(d_feats) || !aligned16(d_grad_out) || !aligned16(d_grad_w)) {
    return fail(SPCONV_ERR_INVALID_ARG, "feature and gradient buffers must be 16-byte aligned");
  }
  if (dtype != SPCONV_F32 && dtype != SPCONV_F16 && dtype != SPCONV_BF16) {
    return fail(SPCONV_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  }
  const int32_t cmax = (dtype == SPCONV_F32) ? 512 : 1024;
  if (c_in < 1 || c_out < 1 || c_in > cmax || c_out > cmax) {
    return fail(SPCONV_ERR_INVALID_ARG, "c_in = %d, c_out = %d must lie in [1, %d]", c_in, c_out, cmax);
  }
  const int32_t mult = (dtype == SPCONV_F32) ? 4 : 8;
  if (c_in % mult != 0 || c_out % mult != 0) {
    return fail(SPCONV_ERR_UNSUPPORTED, "c_in = %d and c_out = %d must be multiples of %d", c_in, c_out, mult);
  }
  {
    const uint64_t es = (dtype == SPCONV_F32) ? 4u : 2u;
    const uint64_t gw_b = static_cast<uint64_t>(map->KV) * c_in * c_out * sizeof(float);
    auto overlap = [](const void* p, uint64_t np, const void* q, uint64_t nq) {
      const uint64_t a0 = reinterpret_cast<uintptr_t>(p), b0 = reinterpret_cast<uintptr_t>(q);
      return a0 < b0 + nq && b0 < a0 + np;
    };
    if (overlap(d_grad_w, gw_b, d_feats, static_cast<uint64_t>(map->n_in) * c_in * es) ||
        overlap(d_grad_w, gw_b, d_grad_out, static_cast<uint64_t>(map->n) * c_out * es)) {
      return fail(SPCONV_ERR_INVALID_ARG, "d_grad_w overlaps the features or the output gradient");
    }
  }
  spconv::WgradArgs a;
  a.feats = d_feats;
  a.grad_out = d_grad_out;
  a.grad_w = d_grad_w;
  a.in_idx = map->buf.in_idx;
  a.out_idx = map->buf.out_idx;
  a.tile_off = map->buf.tile_off;
  a.n = map->n;
  a.n_in = map->n_in;
  a.tiles = map->tiles;
  a.KV = map->KV;
  a.cin = c_in;
  a.cout = c_out;
  a.dtype = static_cast<int32_t>(dtype);
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  spconv_status st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  if (known_empty(map)) {
    SPCONV_HIP(hipMemsetAsync(d_grad_w, 0, static_cast<size_t>(map->KV) * c_in * c_out * sizeof(float), stream),
               "hipMemsetAsync");
    return SPCONV_OK;
  }
  hipMemPool_t pool = nullptr;
  st = pool_for(map->device, &pool);
  if (st != SPCONV_OK) return st;
  std::lock_guard<std::mutex> lock(g_cache_mu);
  StreamCache* c = cache_for(map->device, stream);
  st = grow_buffer(c->fwd, c->fwd_bytes, spconv::wgrad_workspace_bytes(a), pool, stream,
                   "weight-gradient workspace allocation");
  if (st != SPCONV_OK) return st;
  const hipError_t e = spconv::launch_wgrad(a, c->fwd, stream);
  if (e != hipSuccess) return hip_fail(e, "weight-gradient launch");
  return SPCONV_OK;
}

spconv_status spconv_build_map_strided(const int32_t* d_coords, int64_t n_in, int32_t kernel_size, int32_t stride,
                                       void* hip_stream, spconv_map** out_map) {
  g_last_error.clear();
  if (out_map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "out_map is NULL");
  *out_map = nullptr;
  if (d_coords == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "d_coords is NULL");
  if (!aligned16(d_coords)) return fail(SPCONV_ERR_INVALID_ARG, "d_coords is not 16-byte aligned");
  if (n_in <= 0) return fail(SPCONV_ERR_INVALID_ARG, "n_in = %lld must be positive", (long long)n_in);
  if (kernel_size < 1 || kernel_size > 5) {
    return fail(SPCONV_ERR_UNSUPPORTED, "kernel_size = %d not in [1, 5] for a strided map", kernel_size);
  }
  if (stride < 1 || stride > 16) return fail(SPCONV_ERR_UNSUPPORTED, "stride = %d not in [1, 16]", stride);
  const spconv::OutCoordPlan op = spconv::out_coord_plan(n_in, kernel_size, stride);
  if (op.m >= (int64_t(1) << 31)) {
    return fail(SPCONV_ERR_INVALID_ARG, "n_in x ceil(K / stride)^3 = %lld must stay below 2^31", (long long)op.m);
  }
  const int32_t KV = kernel_size * kernel_size * kernel_size;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  hipMemPool_t pool = nullptr;
  spconv_status st = pool_for(device, &pool);
  if (st != SPCONV_OK) return st;
  spconv_map* m = new (std::nothrow) spconv_map;
  if (m == nullptr) return fail(SPCONV_ERR_OUT_OF_MEMORY, "host allocation");
  m->device = device;
  m->stream = stream;
  m->K = kernel_size;
  m->KV = KV;
  m->n_in = n_in;
  m->centre = -1;
  m->stride = stride;
  m->kind = SPCONV_MAP_STRIDED;
  st = acquire_slot(device, &m->slot);
  if (st != SPCONV_OK) {
    delete m;
    return st;
  }
  // Phase 1: the input table, the outputs' keys sorted and counted; the host
  // reads the flags and the number of outputs (the map's size depends on it).
  const int64_t slots = spconv::table_slots_for(n_in);
  const size_t table_b = align256(static_cast<size_t>(slots) * sizeof(ulonglong2));
  const size_t occ_b = align256(static_cast<size_t>(slots / 4) * sizeof(uint4));
  const size_t sum_b = align256(static_cast<size_t>(spconv::kSummaryHead + KV) * sizeof(long long));
  const size_t a_bytes = table_b + occ_b + sum_b + spconv::out_coord_scratch_bytes(op);
  void* a_buf = nullptr;
  void* b_buf = nullptr;
  auto discard = [&](spconv_status s2) {
    if (m->block != nullptr) (void)hipFreeAsync(m->block, stream);
    if (a_buf != nullptr) (void)hipFreeAsync(a_buf, stream);
    if (b_buf != nullptr) (void)hipFreeAsync(b_buf, stream);
    if (m->slot != nullptr) release_slot(device, m->slot);
    delete m;
    return s2;
  };
  hipError_t e = hipMallocFromPoolAsync(&a_buf, a_bytes, pool, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "strided map workspace allocation"));
  char* ac = static_cast<char*>(a_buf);
  ulonglong2* table = reinterpret_cast<ulonglong2*>(ac);
  uint4* occ = reinterpret_cast<uint4*>(ac + table_b);
  long long* summary = reinterpret_cast<long long*>(ac + table_b + occ_b);
  void* sort_scratch = ac + table_b + occ_b + sum_b;
  e = spconv::launch_table_build(d_coords, n_in, table, slots, occ, summary, spconv::kSummaryHead + KV, stream);
  if (e == hipSuccess) e = spconv::launch_out_coords_count(op, d_coords, sort_scratch, summary + 1, stream);
  if (e == hipSuccess) {
    e = hipMemcpyAsync(m->slot->host, summary, 2 * sizeof(long long), hipMemcpyDeviceToHost, stream);
  }
  if (e == hipSuccess) e = hipEventRecord(m->slot->done, stream);
  if (e == hipSuccess) e = hipEventSynchronize(m->slot->done);
  if (e != hipSuccess) return discard(hip_fail(e, "strided map build"));
  const unsigned long long flags = static_cast<unsigned long long>(m->slot->host[0]);
  if (flags & spconv::kFlagRange) {
    return discard(fail(SPCONV_ERR_COORD_RANGE, "a coordinate is outside b in [0, 2^15), z, y, x in [0, 2^16)"));
  }
  if (flags & spconv::kFlagDuplicate) {
    return discard(fail(SPCONV_ERR_DUPLICATE_COORD, "two rows share one (b, z, y, x) coordinate"));
  }
  if (flags & spconv::kFlagTableFull) return discard(fail(SPCONV_ERR_DEVICE, "internal: hash table probe exceeded its bound"));
  const int64_t n_out = m->slot->host[1];
  if (n_out * KV >= (int64_t(1) << 31)) {
    return discard(fail(SPCONV_ERR_INVALID_ARG, "n_out x K^3 = %lld x %d must stay below 2^31", (long long)n_out, KV));
  }
  // Phase 2: the map over the n_out outputs.
  const int64_t cap = std::max<int64_t>(64, std::min<int64_t>(static_cast<int64_t>(KV) * n_out, op.m));
  m->n = n_out;
  m->tiles = (n_out + spconv::kTileRows - 1) / spconv::kTileRows;
  size_t block_bytes = 0;
  const GeneralLayout lay = general_layout(m->tiles, KV, cap, n_out, n_in, &block_bytes);
  e = hipMallocFromPoolAsync(&m->block, block_bytes, pool, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "map allocation"));
  m->block_bytes = block_bytes;
  carve_general(lay, m);
  if (n_out > 0) {
    e = hipMallocFromPoolAsync(&b_buf, spconv::general_scratch_bytes(n_out, kernel_size), pool, stream);
    if (e != hipSuccess) return discard(hip_fail(e, "strided map workspace allocation"));
  }
  e = spconv::launch_out_coords_write(op, sort_scratch, m->out_coords, stream);
  if (e == hipSuccess) {
    e = hipMemcpyAsync(m->in_coords, d_coords, static_cast<size_t>(n_in) * 4 * sizeof(int32_t),
                       hipMemcpyDeviceToDevice, stream);
  }
  if (e == hipSuccess && n_out > 0) {
    spconv::GeneralMapArgs g;
    g.qcoords = m->out_coords;
    g.nq = n_out;
    g.table = table;
    g.table_slots = slots;
    g.K = kernel_size;
    g.lo = -((kernel_size - 1) / 2);
    g.stride = stride;
    g.mode = 0;
    spconv::carve_general_scratch(n_out, kernel_size, b_buf, &g);
    g.summary = summary;
    g.host_summary = m->slot->device;
    g.map = m->buf;
    e = spconv::launch_general_map(g, stream);
  }
  if (e != hipSuccess) return discard(hip_fail(e, "strided map launch"));
  if (n_out == 0) {
    mark_empty(m);
  } else {
    e = hipEventRecord(m->slot->done, stream);
    if (e != hipSuccess) return discard(hip_fail(e, "hipEventRecord"));
  }
  (void)hipFreeAsync(a_buf, stream);
  if (b_buf != nullptr) (void)hipFreeAsync(b_buf, stream);
  a_buf = b_buf = nullptr;
  st = finish_build(m);
  if (st != SPCONV_OK) {
    spconv_map_free(m);
    return st;
  }
  *out_map = m;
  return SPCONV_OK;
}

spconv_status spconv_map_transpose(spconv_map* map, void* hip_stream, spconv_map** out_map) {
  g_last_error.clear();
  if (out_map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "out_map is NULL");
  *out_map = nullptr;
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if (map->kind != SPCONV_MAP_STRIDED) {
    return fail(SPCONV_ERR_UNSUPPORTED, "only a strided map has a transpose here (a submanifold map is its own, "
                                        "with mirrored weights)");
  }
  spconv_status st = finish_build(map);
  if (st != SPCONV_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  int device = 0;
  SPCONV_HIP(hipGetDevice(&device), "hipGetDevice");
  if (device != map->device) {
    return fail(SPCONV_ERR_INVALID_ARG, "the current device (%d) is not the map's (%d)", device, map->device);
  }
  st = order_after_build(map, stream);
  if (st != SPCONV_OK) return st;
  hipMemPool_t pool = nullptr;
  st = pool_for(device, &pool);
  if (st != SPCONV_OK) return st;
  spconv_map* t = new (std::nothrow) spconv_map;
  if (t == nullptr) return fail(SPCONV_ERR_OUT_OF_MEMORY, "host allocation");
  t->device = device;
  t->stream = stream;
  t->K = map->K;
  t->KV = map->KV;
  t->n = map->n_in;
  t->n_in = map->n;
  t->centre = -1;
  t->stride = map->stride;
  t->kind = SPCONV_MAP_TRANSPOSED;
  t->tiles = (t->n + spconv::kTileRows - 1) / spconv::kTileRows;
  void* a_buf = nullptr;
  auto discard = [&](spconv_status s2) {
    if (t->block != nullptr) (void)hipFreeAsync(t->block, stream);
    if (a_buf != nullptr) (void)hipFreeAsync(a_buf, stream);
    if (t->slot != nullptr) release_slot(device, t->slot);
    delete t;
    return s2;
  };
  st = acquire_slot(device, &t->slot);
  if (st != SPCONV_OK) {
    delete t;
    return st;
  }
  const int64_t cap = std::max<int64_t>(64, map->total);
  size_t block_bytes = 0;
  const GeneralLayout lay = general_layout(t->tiles, t->KV, cap, t->n, t->n_in, &block_bytes);
  hipError_t e = hipMallocFromPoolAsync(&t->block, block_bytes, pool, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "map allocation"));
  t->block_bytes = block_bytes;
  carve_general(lay, t);
  e = hipMemcpyAsync(t->out_coords, map->in_coords, static_cast<size_t>(t->n) * 4 * sizeof(int32_t),
                     hipMemcpyDeviceToDevice, stream);
  if (e == hipSuccess && t->n_in > 0) {
    e = hipMemcpyAsync(t->in_coords, map->out_coords, static_cast<size_t>(t->n_in) * 4 * sizeof(int32_t),
                       hipMemcpyDeviceToDevice, stream);
  }
  if (e != hipSuccess) return discard(hip_fail(e, "hipMemcpyAsync"));
  if (map->total == 0) {
    mark_empty(t);
    *out_map = t;
    return SPCONV_OK;
  }
  // The strided map's outputs in a table; each of its inputs probes the
  // outputs q' with stride x q' + d = p.
  const int64_t slots = spconv::table_slots_for(t->n_in);
  const size_t table_b = align256(static_cast<size_t>(slots) * sizeof(ulonglong2));
  const size_t occ_b = align256(static_cast<size_t>(slots / 4) * sizeof(uint4));
  const size_t sum_b = align256(static_cast<size_t>(spconv::kSummaryHead + t->KV) * sizeof(long long));
  e = hipMallocFromPoolAsync(&a_buf, table_b + occ_b + sum_b + spconv::general_scratch_bytes(t->n, t->K), pool,
                             stream);
  if (e != hipSuccess) return discard(hip_fail(e, "transpose workspace allocation"));
  char* ac = static_cast<char*>(a_buf);
  ulonglong2* table = reinterpret_cast<ulonglong2*>(ac);
  uint4* occ = reinterpret_cast<uint4*>(ac + table_b);
  long long* summary = reinterpret_cast<long long*>(ac + table_b + occ_b);
  e = spconv::launch_table_build(map->out_coords, t->n_in, table, slots, occ, summary, spconv::kSummaryHead + t->KV,
                                 stream);
  if (e == hipSuccess) {
    spconv::GeneralMapArgs g;
    g.qcoords = t->out_coords;
    g.nq = t->n;
    g.table = table;
    g.table_slots = slots;
    g.K = t->K;
    g.lo = -((t->K - 1) / 2);
    g.stride = t->stride;
    g.mode = 1;
    spconv::carve_general_scratch(t->n, t->K, ac + table_b + occ_b + sum_b, &g);
    g.summary = summary;
    g.host_summary = t->slot->device;
    g.map = t->buf;
    e = spconv::launch_general_map(g, stream);
  }
  if (e == hipSuccess) e = hipEventRecord(t->slot->done, stream);
  if (e != hipSuccess) return discard(hip_fail(e, "transpose launch"));
  (void)hipFreeAsync(a_buf, stream);
  a_buf = nullptr;
  st = finish_build(t);
  if (st == SPCONV_OK && t->total != map->total) {
    st = fail(SPCONV_ERR_DEVICE, "internal: the transpose holds %lld entries, the map %lld", (long long)t->total,
              (long long)map->total);
  }
  if (st != SPCONV_OK) {
    spconv_map_free(t);
    return st;
  }
  *out_map = t;
  return SPCONV_OK;
}

spconv_status spconv_map_geometry(const spconv_map* map, int64_t* n_in, int64_t* n_out, int32_t* stride,
                                  int32_t* kind) {
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  if (n_in) *n_in = map->n_in;
  if (n_out) *n_out = map->n;
  if (stride) *stride = map->stride;
  if (kind) *kind = map->kind;
  return SPCONV_OK;
}

spconv_status spconv_map_out_coords(const spconv_map* map, const int32_t** d_out_coords) {
  if (map == nullptr || d_out_coords == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "NULL argument");
  if (map->kind == SPCONV_MAP_SUBMANIFOLD) {
    return fail(SPCONV_ERR_UNSUPPORTED, "a submanifold map's outputs are its inputs (the caller's coordinates)");
  }
  *d_out_coords = map->out_coords;
  return SPCONV_OK;
}

spconv_status spconv_group_plan_counts(const int64_t* h_counts, int32_t kernel_volume, int32_t centre,
                                       double epsilon, double S, int32_t capacity, int32_t* h_offsets,
                                       int32_t* h_groups, int32_t* n_entries, int32_t* n_groups,
                                       int64_t* padded_rows) {
  g_last_error.clear();
  if (h_counts == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "h_counts is NULL");
  if (kernel_volume < 1 || kernel_volume > spconv::kMaxGroupEntries) {
    return fail(SPCONV_ERR_INVALID_ARG, "kernel_volume = %d not in [1, %d]", kernel_volume,
                spconv::kMaxGroupEntries);
  }
  if (centre < -1 || centre >= kernel_volume) {
    return fail(SPCONV_ERR_INVALID_ARG, "centre = %d not in [-1, %d)", centre, kernel_volume);
  }
  for (int32_t k = 0; k < kernel_volume; ++k) {
    if (h_counts[k] < 0 || h_counts[k] >= (int64_t(1) << 40)) {
      return fail(SPCONV_ERR_INVALID_ARG, "count %lld of offset %d not in [0, 2^40)", (long long)h_counts[k], k);
    }
  }
  spconv_status st = check_plan_args(epsilon, S);
  if (st != SPCONV_OK) return st;
  const spconv::GroupPlan plan = spconv::make_group_plan(h_counts, kernel_volume, centre, epsilon, S);
  const int32_t n = static_cast<int32_t>(plan.entries.size());
  if ((h_offsets != nullptr || h_groups != nullptr) && capacity < n) {
    return fail(SPCONV_ERR_INVALID_ARG, "capacity %d below the plan's %d entries", capacity, n);
  }
  for (int32_t i = 0; i < n; ++i) {
    if (h_offsets) h_offsets[i] = plan.entries[i];
    if (h_groups) h_groups[i] = plan.entry_group[i];
  }
  if (n_entries) *n_entries = n;
  if (n_groups) *n_groups = plan.groups;
  if (padded_rows) *padded_rows = plan.padded_rows;
  return SPCONV_OK;
}

spconv_status spconv_group_plan(spconv_map* map, double epsilon, double S, int32_t capacity, int32_t* h_offsets,
                                int32_t* h_groups, int32_t* n_entries, int32_t* n_groups, int64_t* padded_rows) {
  g_last_error.clear();
  if (map == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "map is NULL");
  spconv_status st = check_plan_args(epsilon, S);
  if (st != SPCONV_OK) return st;
  st = finish_build(map);
  if (st != SPCONV_OK) return st;
  return spconv_group_plan_counts(map->counts.data(), map->KV, map->centre, epsilon, S, capacity, h_offsets,
                                  h_groups, n_entries, n_groups, padded_rows);
}

spconv_status spconv_forward_grouped(const void* d_feats, const void* d_weights, spconv_map* map, int32_t c_in,
                                     int32_t c_out, spconv_dtype dtype, double epsilon, double S, void* d_out,
                                     void* hip_stream) {
  g_last_error.clear();
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_feats, d_weights, map, c_in, c_out, dtype, d_out, &a);
  if (st != SPCONV_OK) return st;
  st = check_plan_args(epsilon, S);
  if (st != SPCONV_OK) return st;
  if (!spconv::grouped_supported(a)) {
    return fail(SPCONV_ERR_UNSUPPORTED, "the grouped forward needs f16 or bf16, c_in %% 32 == 0 and c_out %% 16 == 0");
  }
  st = finish_build(map);
  if (st != SPCONV_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  if (map->total == 0) return zero_output(d_out, map->n, c_out, dtype, stream);
  const spconv::GroupPlan plan = spconv::make_group_plan(map->counts.data(), map->KV, map->centre, epsilon, S);
  return launch_grouped(map, a, plan, stream);
}

spconv_status spconv_select_dataflow(const void* d_feats, const void* d_weights, spconv_map* map, int32_t c_in,
                                     int32_t c_out, spconv_dtype dtype, const double* epsilons, int32_t n_epsilons,
                                     const double* thresholds, int32_t n_thresholds, int32_t reps, void* d_out,
                                     void* hip_stream, spconv_dataflow* best) {
  g_last_error.clear();
  if (best == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "best is NULL");
  spconv::ForwardArgs a;
  spconv_status st = forward_args(d_feats, d_weights, map, c_in, c_out, dtype, d_out, &a);
  if (st != SPCONV_OK) return st;
  if (reps < 1 || reps > 1000) return fail(SPCONV_ERR_INVALID_ARG, "reps = %d not in [1, 1000]", reps);
  static const double kEps[] = {0.0, 0.1, 0.2, 0.3, 0.5, 1.0};
  static const double kS[] = {HUGE_VAL, 65536.0, 16384.0, 0.0};
  if (epsilons == nullptr) {
    epsilons = kEps;
    n_epsilons = static_cast<int32_t>(sizeof(kEps) / sizeof(kEps[0]));
  }
  if (thresholds == nullptr) {
    thresholds = kS;
    n_thresholds = static_cast<int32_t>(sizeof(kS) / sizeof(kS[0]));
  }
  if (n_epsilons < 0 || n_thresholds < 0 || n_epsilons > 64 || n_thresholds > 64) {
    return fail(SPCONV_ERR_INVALID_ARG, "grids of %d and %d values (at most 64 each)", n_epsilons, n_thresholds);
  }
  for (int32_t i = 0; i < n_epsilons; ++i) {
    st = check_plan_args(epsilons[i], 0.0);
    if (st != SPCONV_OK) return st;
  }
  for (int32_t i = 0; i < n_thresholds; ++i) {
    st = check_plan_args(0.0, thresholds[i]);
    if (st != SPCONV_OK) return st;
  }
  st = finish_build(map);
  if (st != SPCONV_OK) return st;
  hipStream_t stream = static_cast<hipStream_t>(hip_stream);
  std::memset(best, 0, sizeof(*best));
  best->kind = SPCONV_DATAFLOW_FUSED;
  if (map->total == 0) {
    best->candidates = 1;
    return zero_output(d_out, map->n, c_out, dtype, stream);
  }
  // Candidates: the fused forward, then each distinct plan of the grid.
  struct Candidate {
    bool grouped;
    double epsilon, S;
    spconv::GroupPlan plan;
  };
  std::vector<Candidate> cands;
  cands.push_back({false, 0.0, 0.0, {}});
  if (spconv::grouped_supported(a)) {
    for (int32_t j = 0; j < n_thresholds; ++j) {
      for (int32_t i = 0; i < n_epsilons; ++i) {
        spconv::GroupPlan p =
            spconv::make_group_plan(map->counts.data(), map->KV, map->centre, epsilons[i], thresholds[j]);
        bool seen = false;
        for (size_t c = 1; c < cands.size() && !seen; ++c) seen = same_plan(cands[c].plan, p);
        if (!seen) cands.push_back({true, epsilons[i], thresholds[j], std::move(p)});
      }
    }
  }
  auto run = [&](const Candidate& c) {
    return c.grouped ? launch_grouped(map, a, c.plan, stream) : launch_fused(map, a, stream);
  };
  hipEvent_t t0 = nullptr, t1 = nullptr;
  SPCONV_HIP(hipEventCreate(&t0), "hipEventCreate");
  hipError_t ec = hipEventCreate(&t1);
  if (ec != hipSuccess) {
    (void)hipEventDestroy(t0);
    return hip_fail(ec, "hipEventCreate");
  }
  size_t win = 0;
  float win_ms = 0.f;
  for (size_t c = 0; c < cands.size() && st == SPCONV_OK; ++c) {
    st = run(cands[c]);  // warm-up (workspace growth, first-touch)
    if (st != SPCONV_OK) break;
    ec = hipEventRecord(t0, stream);
    for (int32_t r = 0; r < reps && st == SPCONV_OK && ec == hipSuccess; ++r) st = run(cands[c]);
    if (st != SPCONV_OK) break;
    if (ec == hipSuccess) ec = hipEventRecord(t1, stream);
    if (ec == hipSuccess) ec = hipEventSynchronize(t1);
    float ms = 0.f;
    if (ec == hipSuccess) ec = hipEventElapsedTime(&ms, t0, t1);
    if (ec != hipSuccess) {
      st = hip_fail(ec, "dataflow timing");
      break;
    }
    ms /= static_cast<float>(reps);
    if (c == 0) best->fused_ms = ms;
    if (c == 0 || ms < win_ms) {
      win = c;
      win_ms = ms;
    }
  }
  (void)hipEventDestroy(t0);
  (void)hipEventDestroy(t1);
  if (st != SPCONV_OK) return st;
  // Leave the winner's result in d_out.
  st = run(cands[win]);
  if (st != SPCONV_OK) return st;
  best->kind = cands[win].grouped ? SPCONV_DATAFLOW_GROUPED : SPCONV_DATAFLOW_FUSED;
  best->groups = cands[win].grouped ? cands[win].plan.groups : 0;
  best->epsilon = cands[win].epsilon;
  best->S = cands[win].S;
  best->ms = win_ms;
  best->candidates = static_cast<int32_t>(cands.size());
  return SPCONV_OK;
}

spconv_status spconv_attention_forward(const spconv_attention* args, void* d_out, float* d_lse, void* hip_stream) {
  return guarded([&] { return attention_forward(args, d_out, d_lse, nullptr, hip_stream); });
}

spconv_status spconv_attention_forward_noalloc(const spconv_attention* args, void* d_out, float* d_lse, void* d_workspace,
                                               uint64_t workspace_bytes, void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return attention_forward(args, d_out, d_lse, &own, hip_stream); });
}

spconv_status spconv_attention_backward(const spconv_attention* args, const void* d_out, const float* d_lse,
                                        const spconv_attention_gradients* grads, void* hip_stream) {
  return guarded([&] { return attention_backward(args, d_out, d_lse, grads, nullptr, hip_stream); });
}

spconv_status spconv_attention_backward_noalloc(const spconv_attention* args, const void* d_out, const float* d_lse,
                                                const spconv_attention_gradients* grads, void* d_workspace, uint64_t workspace_bytes,
                                                void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return attention_backward(args, d_out, d_lse, grads, &own, hip_stream); });
}

spconv_status spconv_attention_workspace(const spconv_attention* args, uint64_t* forward_bytes, uint64_t* backward_bytes) {
  return guarded([&]() -> spconv_status {
    g_last_error.clear();
    spconv::AttentionArgs a;
    const spconv_status st = attention_sizes(args, &a);
    if (st != SPCONV_OK) return st;
    if (forward_bytes != nullptr) *forward_bytes = a.total_q == 0 ? 0 : spconv::attention_workspace_bytes(a);
    if (backward_bytes != nullptr) *backward_bytes = a.total_q == 0 && a.total_k == 0 ? 0 : spconv::attention_backward_workspace_bytes(a);
    return SPCONV_OK;
  });
}

spconv_status spconv_norm_rotary_forward(const spconv_norm_rotary* args, void* d_q_out, int64_t q_out_row_stride,
                                         int64_t q_out_head_stride, void* d_k_out, int64_t k_out_row_stride,
                                         int64_t k_out_head_stride, void* hip_stream) {
  return guarded([&]() -> spconv_status {
    g_last_error.clear();
    spconv::NormRotaryArgs a;
    Strided in[2];
    spconv_status st = norm_rotary_args(args, &a, in);
    if (st != SPCONV_OK) return st;
    Strided out[2] = {{"q_out", d_q_out, a.rows, q_out_row_stride, a.t[0].heads, q_out_head_stride, a.dim, in[0].es},
                      {"k_out", d_k_out, a.rows, k_out_row_stride, a.t[1].heads, k_out_head_stride, a.dim, in[0].es}};
    for (int i = 0; i < 2; ++i) {
      st = check_strided(out[i], true);
      for (int j = 0; j < 2 && st == SPCONV_OK; ++j)
        if (i != j || !same_place(out[i], in[j])) st = check_apart(out[i], in[j]);
      if (st != SPCONV_OK) return st;
      a.t[i].y = const_cast<void*>(out[i].p);
      a.t[i].y_row = out[i].row_stride;
      a.t[i].y_head = out[i].head_stride;
    }
    st = check_apart(out[0], out[1]);
    if (st == SPCONV_OK) st = check_work_items(spconv::norm_rotary_work_items(a));
    if (st != SPCONV_OK) return st;
    const hipError_t e = spconv::launch_norm_rotary(a, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? SPCONV_OK : hip_fail(e, "norm and rotation launch");
  });
}

spconv_status spconv_norm_rotary_backward(const spconv_norm_rotary* args, const spconv_norm_rotary_gradients* grads,
                                          void* hip_stream) {
  return guarded([&] { return norm_rotary_backward(args, grads, nullptr, hip_stream); });
}

spconv_status spconv_norm_rotary_backward_noalloc(const spconv_norm_rotary* args, const spconv_norm_rotary_gradients* grads,
                                                  void* d_workspace, uint64_t workspace_bytes, void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return norm_rotary_backward(args, grads, &own, hip_stream); });
}

spconv_status spconv_norm_rotary_workspace(int32_t head_dim, uint64_t* backward_bytes) {
  g_last_error.clear();
  const spconv_status st = check_head_dim(SPCONV_F32, head_dim);
  if (st != SPCONV_OK) return st;
  if (backward_bytes == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "backward_bytes is NULL");
  spconv::NormRotaryArgs a;
  a.dim = head_dim;
  *backward_bytes = spconv::norm_rotary_backward_workspace_bytes(a);
  return SPCONV_OK;
}

spconv_status spconv_rotary_table(float* d_table, int32_t extent, int32_t pairs, double base, double position_scale,
                                  void* hip_stream) {
  g_last_error.clear();
  if (d_table == nullptr || (reinterpret_cast<uintptr_t>(d_table) & 7u)) {
    return fail(SPCONV_ERR_INVALID_ARG, "table is NULL or not 8-byte aligned");
  }
  if (extent < 1 || extent > (1 << 24) || pairs < 1 || pairs > (1 << 24)) {
    return fail(SPCONV_ERR_INVALID_ARG, "extent = %d and pairs = %d must lie in [1, 2^24]", extent, pairs);
  }
  if (!(base > 0.0) || !std::isfinite(base) || !std::isfinite(position_scale)) {
    return fail(SPCONV_ERR_INVALID_ARG, "base = %g must be positive and finite, position_scale = %g finite", base, position_scale);
  }
  const spconv_status st = check_work_items((static_cast<uint64_t>(extent) * pairs + 255) / 256 * 256);
  if (st != SPCONV_OK) return st;
  const hipError_t e = spconv::launch_rotary_table(d_table, extent, pairs, base, position_scale, static_cast<hipStream_t>(hip_stream));
  return e == hipSuccess ? SPCONV_OK : hip_fail(e, "rotary table launch");
}

void spconv_map_free(spconv_map* map) {
  if (map == nullptr) return;
  if (map->block != nullptr) release_block(map->device, map->stream, map->block, map->block_bytes);
  if (map->slot != nullptr) release_slot(map->device, map->slot);
  delete map;
}

spconv_status spconv_add_norm_forward(const spconv_add_norm* args, void* d_h, int64_t h_row_stride, void* d_y, int64_t y_row_stride,
                                      void* hip_stream) {
  return guarded([&] { return add_norm_forward(args, d_h, h_row_stride, d_y, y_row_stride, hip_stream); });
}

spconv_status spconv_add_norm_backward(const spconv_add_norm* args, const spconv_add_norm_gradients* grads, void* hip_stream) {
  return guarded([&] { return add_norm_backward(args, grads, nullptr, hip_stream); });
}

spconv_status spconv_add_norm_backward_noalloc(const spconv_add_norm* args, const spconv_add_norm_gradients* grads, void* d_workspace,
                                               uint64_t workspace_bytes, void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return add_norm_backward(args, grads, &own, hip_stream); });
}

spconv_status spconv_add_norm_workspace(int32_t channels, uint64_t* backward_bytes) {
  return guarded([&]() -> spconv_status {
    g_last_error.clear();
    if (backward_bytes == nullptr) return fail(SPCONV_ERR_INVALID_ARG, "backward_bytes is NULL");
    if (channels < 8 || channels % 8 != 0 || channels > 16384) {
      return fail(SPCONV_ERR_UNSUPPORTED, "channels = %d must be a multiple of 8 in [8, 16384]", channels);
    }
    spconv::AddNormArgs a;
    a.channels = channels;
    *backward_bytes = spconv::add_norm_backward_workspace_bytes(a);
    return SPCONV_OK;
  });
}

spconv_status spconv_linear_forward(const spconv_linear* args, const spconv_linear_epilogue* epilogue, void* hip_stream) {
  return guarded([&] { return linear_forward(args, epilogue, nullptr, hip_stream); });
}

spconv_status spconv_linear_forward_noalloc(const spconv_linear* args, const spconv_linear_epilogue* epilogue, void* d_workspace,
                                            uint64_t workspace_bytes, void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return linear_forward(args, epilogue, &own, hip_stream); });
}

spconv_status spconv_linear_backward(const spconv_linear* args, const spconv_linear_gradients* grads, void* hip_stream) {
  return guarded([&] { return linear_backward(args, grads, nullptr, hip_stream); });
}

spconv_status spconv_linear_backward_noalloc(const spconv_linear* args, const spconv_linear_gradients* grads, void* d_workspace,
                                             uint64_t workspace_bytes, void* hip_stream) {
  const CallerWorkspace own = {d_workspace, workspace_bytes};
  return guarded([&] { return linear_backward(args, grads, &own, hip_stream); });
}

spconv_status spconv_linear_workspace(const spconv_linear* args, uint64_t* forward_bytes, uint64_t* backward_bytes) {
  return guarded([&]() -> spconv_status {
    g_last_error.clear();
    spconv::LinearArgs a;
    const spconv_status st = linear_sizes(args, &a);
    if (st != SPCONV_OK) return st;
    if (forward_bytes != nullptr) *forward_bytes = a.rows == 0 ? 0 : spconv::linear_workspace_bytes(a);
    if (backward_bytes != nullptr) *backward_bytes = spconv::linear_backward_workspace_bytes(a);
    return SPCONV_OK;
  });
}

spconv_status spconv_activation_backward(const void* d_grad_out, int64_t grad_out_row_stride, const void* d_pre, int64_t pre_row_stride,
                                         void* d_grad_pre, int64_t grad_pre_row_stride, int64_t rows, int32_t channels, int32_t activation,
                                         spconv_dtype dtype, void* hip_stream) {
  return guarded([&] {
    return activation_backward(d_grad_out, grad_out_row_stride, d_pre, pre_row_stride, d_grad_pre, grad_pre_row_stride, rows, channels,
                               activation, static_cast<int32_t>(dtype), hip_stream);
  });
}

}  // extern "C"
