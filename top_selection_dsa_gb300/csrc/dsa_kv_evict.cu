// dsa_kv_evict.cu -- eviction from a paged cache by accumulated attention
// weight: which tokens a budget keeps, and moving their rows together.
//
//   keep[b] = the first `sink` positions, the `budget - sink - recent` of the
//             middle with the largest weight (ties to the lower position) and
//             the last `recent`, ascending
//
// Few requests of up to kSmallCtx positions: one CTA each does all of it, its
// weights in registers (evict_small_kernel).  Else the middle's selection is the
// library's masked top-k on the weights, and two small kernels make its row
// ranges and put the three parts together.
// Compaction then moves row keep[b][i] of every cache to position i: to fresh
// pages, or in place.  Because keep ascends, keep[i] >= i: in place, a CTA
// that owns one request's slice of bytes goes through the rows in chunks and
// reads a chunk before anything at or above its first position is written.
#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

__device__ __forceinline__ int clamp_len(int L, int cap) { return L < 0 ? 0 : (L > cap ? cap : L); }

__global__ void __launch_bounds__(256)
    evict_ranges_kernel(const int32_t* __restrict__ lens, int B, int max_ctx, int sink, int recent,
                        int32_t* __restrict__ starts, int32_t* __restrict__ ends, uint32_t* err) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= B) return;
  const int raw = lens[b];
  if (raw < 0 || raw > max_ctx) record_error(err, kErrBadIndex);
  const int L = clamp_len(raw, max_ctx);
  const int lo = min(sink, L);
  starts[b] = lo;
  ends[b] = max(lo, L - recent);
}

__global__ void __launch_bounds__(256)
    evict_keep_kernel(const int32_t* __restrict__ lens, const int32_t* __restrict__ starts,
                      const int32_t* __restrict__ ends, const int32_t* __restrict__ mid, int B,
                      int max_ctx, int room, int budget, int32_t* __restrict__ keep,
                      int32_t* __restrict__ new_lens) {
  const int b = blockIdx.y;
  const int L = clamp_len(lens[b], max_ctx);
  const int lo = starts[b], hi = ends[b];
  const int32_t* m = mid + static_cast<int64_t>(b) * room;
  // Entries of the selection before its -1 padding (it ascends): as many as
  // fit, unless some weights could not be chosen; then the end is searched.
  int n = min(room, hi - lo);
  if (n > 0 && m[n - 1] < 0) {
    int most = n, step = 1;
    n = 0;
    while (step <= most) step <<= 1;
    for (step >>= 1; step > 0; step >>= 1)
      if (n + step <= most && m[n + step - 1] >= 0) n += step;
  }
  const int total = lo + n + (L - hi);
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i == 0) new_lens[b] = total;
  if (i >= budget) return;
  int pos = -1;
  if (i < lo) pos = i;
  else if (i < lo + n) pos = m[i - lo];
  else if (i < total) pos = hi + (i - lo - n);
  keep[static_cast<int64_t>(b) * budget + i] = pos;
}

// ------------------------------------------------- selection, short contexts

constexpr int kSmallThreads = 1024;
constexpr int kSmallKeys = 32;  // weights a thread holds
constexpr int kSmallCtx = kSmallThreads * kSmallKeys;

// Order of a weight as an unsigned number: 0 for NaN and -inf, which are never
// chosen; -0 as +0.
__device__ __forceinline__ uint32_t weight_order(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return w > -INFINITY ? o : 0u;
}

__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* slots) {
  const uint32_t w = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = w;
  __syncthreads();
  return __reduce_add_sync(0xffffffffu, slots[threadIdx.x & 31]);
}

// Sum over the threads before this one, and of all.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* slots, uint32_t* total) {
  const int lane = threadIdx.x & 31;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) slots[threadIdx.x >> 5] = incl;
  __syncthreads();
  uint32_t warps = slots[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, warps, o);
    if (lane >= o) warps += y;
  }
  *total = __shfl_sync(0xffffffffu, warps, 31);
  const int w = threadIdx.x >> 5;
  const uint32_t before = __shfl_sync(0xffffffffu, warps, w > 0 ? w - 1 : 0);
  return incl - v + (w > 0 ? before : 0u);
}

// The `room`-th largest order of the middle is found bit by bit, from the
// highest in which the weights differ: a bit stays if at least `room` weights
// are at or above the number so far (until exactly `room` are).  Every step
// counts all weights, two instructions each, and sums over the CTA: 20 steps of
// about 0.55 us.  What lies above it is kept, of its ties the lowest; the kept
// positions are counted off over bitmaps of 32 neighbouring positions a thread.
__global__ void __launch_bounds__(kSmallThreads)
    evict_small_kernel(const float* __restrict__ weights, int64_t ldw,
                       const int32_t* __restrict__ lens, int max_ctx, int budget, int sink,
                       int recent, int32_t* __restrict__ keep, int32_t* __restrict__ new_lens,
                       uint32_t* err) {
  __shared__ uint32_t slots[2][32];  // by turns, so that one barrier a sum is enough
  __shared__ uint32_t above[kSmallThreads], ties[kSmallThreads];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int raw = lens[b];
  if (tid == 0 && (raw < 0 || raw > max_ctx)) record_error(err, kErrBadIndex);
  const int L = clamp_len(raw, max_ctx);
  const int lo = min(sink, L), hi = max(lo, L - recent);
  const uint32_t room = budget - sink - recent;
  const float* w = weights + static_cast<int64_t>(b) * ldw + lo;
  const int n = hi - lo;
  uint32_t key[kSmallKeys];  // position lo + 1024 i + tid
#pragma unroll
  for (int i = 0; i < kSmallKeys; ++i) {
    const int at = i * kSmallThreads + tid;
    key[i] = at < n ? weight_order(__ldg(w + at)) : 0u;
  }
  uint32_t any = 0, all = 0xFFFFFFFFu, valid = 0;
#pragma unroll
  for (int i = 0; i < kSmallKeys; ++i)
    if (key[i] != 0) any |= key[i], all &= key[i], ++valid;
  int turn = 0;
  valid = block_sum(valid, slots[turn]);
  uint32_t bound = 1, taken = valid;  // at or above `bound`: `taken` weights
  if (valid > room) {
    any = __reduce_or_sync(0xffffffffu, any);
    all = __reduce_and_sync(0xffffffffu, all);
    if (lane == 0) ties[warp] = any, above[warp] = all;
    __syncthreads();
    any = __reduce_or_sync(0xffffffffu, ties[lane]);
    all = __reduce_and_sync(0xffffffffu, above[lane]);
    const uint32_t differ = any & ~all;
    const int top = differ ? 31 - __clz(differ) : -1;
    bound = top >= 0 ? any & ~((2u << top) - 1u) : any;
    for (int bit = top; bit >= 0 && taken != room; --bit) {
      const uint32_t t = bound | (1u << bit);
      uint32_t c = 0;
#pragma unroll
      for (int i = 0; i < kSmallKeys; ++i) c += key[i] >= t;
      turn ^= 1;
      c = block_sum(c, slots[turn]);
      if (c >= room) bound = t, taken = c;
    }
  }
  __syncthreads();
  // More than room at or above: the lowest of those equal to the bound go in.
#pragma unroll
  for (int i = 0; i < kSmallKeys; ++i) {
    const bool exact = taken > room && key[i] == bound;
    const uint32_t g = __ballot_sync(0xffffffffu, key[i] >= bound && !exact);
    const uint32_t e = __ballot_sync(0xffffffffu, exact);
    if (lane == 0) above[i * 32 + warp] = g, ties[i * 32 + warp] = e;
  }
  __syncthreads();
  uint32_t mask = above[tid], tie = ties[tid];
  uint32_t total, sum;
  turn ^= 1;
  const uint32_t ties_before = block_scan(__popc(tie), slots[turn], &sum);
  const uint32_t wanted = taken > room ? sum - (taken - room) : 0;
  if (ties_before < wanted) {
    uint32_t take = min(wanted - ties_before, static_cast<uint32_t>(__popc(tie)));
    for (; take > 0; --take) {
      mask |= tie & (0u - tie);
      tie &= tie - 1;
    }
  }
  turn ^= 1;
  uint32_t out = block_scan(__popc(mask), slots[turn], &total);
  int32_t* row = keep + static_cast<int64_t>(b) * budget;
  for (; mask; mask &= mask - 1) row[lo + out++] = lo + tid * 32 + __ffs(mask) - 1;
  const int kept = lo + static_cast<int>(total) + (L - hi);
  for (int i = tid; i < lo; i += kSmallThreads) row[i] = i;
  for (int i = lo + total + tid; i < budget; i += kSmallThreads)
    row[i] = i < kept ? hi + (i - lo - static_cast<int>(total)) : -1;
  if (tid == 0) new_lens[b] = kept;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;  // rows a thread holds per chunk
constexpr int kSlice = 128;     // bytes of a row one CTA moves in place
constexpr int kPartRows = 32;   // rows a CTA moves to fresh pages
constexpr int kCopyUnroll = 4;  // copies a thread has in flight there

// Rows a request keeps: new_lens, within the lists of `keep` and the `places`
// its pages have; more are recorded, and left out.
__device__ __forceinline__ int rows_to_keep(const CompactParams& p, int b, int places,
                                            bool report) {
  const int n = __ldg(p.new_lens + b), most = min(p.budget, places);
  if (report && threadIdx.x == 0 && (n < 0 || n > most)) record_error(p.err, kErrBadIndex);
  return n < 0 ? 0 : min(n, most);
}

// To fresh pages: a CTA takes kPartRows rows of a request in every cache.
// Where they are is looked up once; after that the copies are independent of
// one another and cost two additions of an address each.  Bound by the
// latency of reading single rows.  Selection and move of 64 requests that keep
// 4096 positions each, 8 heads of 128 and an indexer's keys: 185 us, 4.0 TB/s
// (four copies in flight a thread, six CTAs an SM); eight and four 205 us, and
// with the rows' numbers turned into addresses copy by copy 225 us.
struct RowMove {
  const uint8_t* from;  // in plane 0; null: not moved
  uint8_t* to;
};

template <typename V>
__device__ __forceinline__ void copy_rows(const CompactParams::Cache& c, const RowMove* rows,
                                          int n, int log_bs) {
  const int vecs = c.row_bytes / static_cast<int>(sizeof(V));  // of a row
  const int lanes = min(vecs, kMoveThreads), step = kMoveThreads / lanes;
  if (static_cast<int>(threadIdx.x) >= lanes * step) return;
  const int64_t stride = static_cast<int64_t>(c.row_bytes) << log_bs;  // between planes
  // Rows of all planes in one sequence, `step` apart.
  const int by_plane = step / n, by_row = step - by_plane * n;
  const int first = threadIdx.x / lanes;
  for (int v = threadIdx.x % lanes; v < vecs; v += lanes) {
    int plane = first / n, row = first - plane * n;
    while (plane < c.planes) {
      V buf[kCopyUnroll];
      uint32_t has = 0;
      const int row0 = row, plane0 = plane;
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u) {
        if (plane < c.planes) {
          const uint8_t* from = rows[row].from;
          if (from) {
            buf[u] = __ldcs(reinterpret_cast<const V*>(from + plane * stride) + v);
            has |= 1u << u;
          }
        }
        row += by_row, plane += by_plane;
        if (row >= n) row -= n, ++plane;
      }
      int r = row0, pl = plane0;
#pragma unroll
      for (int u = 0; u < kCopyUnroll; ++u) {
        if ((has >> u) & 1) *(reinterpret_cast<V*>(rows[r].to + pl * stride) + v) = buf[u];
        r += by_row, pl += by_plane;
        if (r >= n) r -= n, ++pl;
      }
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads, 6)
    kv_move_kernel(const __grid_constant__ CompactParams p) {
  __shared__ RowMove moves[kMaxCompact][kPartRows];
  const int b = blockIdx.y, part = blockIdx.x;
  const int cap = p.max_blocks << p.log_bs;
  const int old_len = clamp_len(__ldg(p.old_lens + b), cap);
  const int n = rows_to_keep(p, b, min(cap, p.new_max_blocks << p.log_bs), part == 0);
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.budget;
  const int i0 = part * kPartRows;
  if (p.weights) {
    // The weights: one value a position, and zeros after the last kept one.
    // Rewritten where they lie, they are one CTA's work.
    const float* w = p.weights + static_cast<int64_t>(b) * p.ldw;
    float* out = p.weights_out + static_cast<int64_t>(b) * p.ldw;
    const bool alone = p.weights_out == p.weights;
    if (!alone || part == 0) {
      const int w0 = alone ? 0 : i0, w1 = alone ? n : min(n, i0 + kPartRows);
      for (int base = w0; base < w1; base += kMoveThreads) {
        const int i = base + threadIdx.x;
        float v = 0.f;
        if (i < w1) {
          const int pos = __ldg(keep + i);
          if (pos >= 0 && pos < old_len) v = w[pos];
        }
        __syncthreads();
        if (i < w1) out[i] = v;
      }
      __syncthreads();
      const int parts = alone ? 1 : static_cast<int>(gridDim.x);
      const int64_t share = (cap - n + parts - 1) / parts;
      const int z0 = static_cast<int>(min(static_cast<int64_t>(cap), n + share * part));
      const int z1 = static_cast<int>(min(static_cast<int64_t>(cap), z0 + share));
      for (int i = z0 + threadIdx.x; i < z1; i += kMoveThreads) out[i] = 0.f;
    }
  }
  const int rows = min(n - i0, kPartRows);
  if (rows <= 0 || p.ncaches == 0) return;
  if (threadIdx.x < rows) {
    const int i = i0 + threadIdx.x;
    const int pos = __ldg(keep + i);
    const int mask = (1 << p.log_bs) - 1;
    int from = -1, to = -1;
    if (pos >= 0 && pos < old_len) {
      from = __ldg(p.block_table + static_cast<int64_t>(b) * p.max_blocks + (pos >> p.log_bs));
      to = __ldg(p.new_block_table + static_cast<int64_t>(b) * p.new_max_blocks + (i >> p.log_bs));
    }
    const bool bad = from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks;
    if (bad) record_error(p.err, kErrBadIndex);
    for (int c = 0; c < p.ncaches; ++c) {
      const CompactParams::Cache& cache = p.cache[c];
      const int64_t page = static_cast<int64_t>(cache.planes) << p.log_bs;
      RowMove m;
      m.from = bad ? nullptr : cache.base + (from * page + (pos & mask)) * cache.row_bytes;
      m.to = bad ? nullptr : cache.base + (to * page + (i & mask)) * cache.row_bytes;
      moves[c][threadIdx.x] = m;
    }
  }
  __syncthreads();
  for (int c = 0; c < p.ncaches; ++c) {
    const CompactParams::Cache cache = p.cache[c];
    if (cache.row_bytes % 16 == 0) copy_rows<uint4>(cache, moves[c], rows, p.log_bs);
    else if (cache.row_bytes % 8 == 0) copy_rows<uint2>(cache, moves[c], rows, p.log_bs);
    else copy_rows<uint32_t>(cache, moves[c], rows, p.log_bs);
  }
}

// In place: rows [0, i1) of one slice (plane, byte range) of a cache.
template <typename V>
__device__ __forceinline__ void move_rows(const CompactParams& p, const CompactParams::Cache& c,
                                          int plane, int at, int width, int b, int old_len,
                                          int i1) {
  const int lanes = width / static_cast<int>(sizeof(V));
  const int sub = threadIdx.x % lanes;
  const int row_in = threadIdx.x / lanes;
  const int rows = kMoveThreads / lanes;  // per unroll step
  const bool live = row_in < rows;
  const int chunk = rows * kMoveUnroll;
  const int mask = (1 << p.log_bs) - 1;
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.budget;
  const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_blocks;
  auto address = [&](const int32_t* tab, int pos) -> uint8_t* {
    const int block = __ldg(tab + (pos >> p.log_bs));
    if (block < 0 || block >= p.num_blocks) {
      record_error(p.err, kErrBadIndex);
      return nullptr;
    }
    const int64_t row = ((static_cast<int64_t>(block) * c.planes + plane) << p.log_bs) + (pos & mask);
    return c.base + row * c.row_bytes + at + sub * static_cast<int>(sizeof(V));
  };
  V buf[2][kMoveUnroll];
  uint32_t got[2] = {0u, 0u};
  auto load = [&](V (&v)[kMoveUnroll], uint32_t& ok, int base) {
    ok = 0;
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const int i = base + u * rows + row_in;
      if (!live || i >= i1) continue;
      const int pos = __ldg(keep + i);
      if (pos < 0 || pos >= old_len) {
        record_error(p.err, kErrBadIndex);
        continue;
      }
      if (pos == i) continue;
      const uint8_t* src = address(table, pos);
      if (!src) continue;
      v[u] = *reinterpret_cast<const V*>(src);
      ok |= 1u << u;
    }
  };
  auto store = [&](const V (&v)[kMoveUnroll], uint32_t ok, int base) {
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      if (!((ok >> u) & 1)) continue;
      uint8_t* dst = address(table, base + u * rows + row_in);
      if (dst) *reinterpret_cast<V*>(dst) = v[u];
    }
  };
  load(buf[0], got[0], 0);
  for (int base = 0; base < i1; base += 2 * chunk) {
    // The next chunk's rows lie at or above its own first position, so
    // reading them does not wait for this chunk's stores; this chunk's stores
    // wait for every thread's reads of this chunk.
    load(buf[1], got[1], base + chunk);
    __syncthreads();
    store(buf[0], got[0], base);
    load(buf[0], got[0], base + 2 * chunk);
    __syncthreads();
    store(buf[1], got[1], base + chunk);
  }
}

__global__ void __launch_bounds__(kMoveThreads)
    kv_compact_kernel(const __grid_constant__ CompactParams p) {
  const int b = blockIdx.y, unit = blockIdx.x;
  const int cap = p.max_blocks << p.log_bs;
  const int old_len = clamp_len(__ldg(p.old_lens + b), cap);
  const int n = rows_to_keep(p, b, cap, unit == 0);
  if (unit < p.units) {
    int c = 0;
    while (unit >= p.first_unit[c + 1]) ++c;
    const CompactParams::Cache cache = p.cache[c];
    const int slices = (cache.row_bytes + kSlice - 1) / kSlice;
    const int u = unit - p.first_unit[c];
    const int plane = u / slices, at = (u % slices) * kSlice;
    const int width = min(kSlice, cache.row_bytes - at);
    if (width % 16 == 0 && cache.row_bytes % 16 == 0)
      move_rows<uint4>(p, cache, plane, at, width, b, old_len, n);
    else if (width % 8 == 0 && cache.row_bytes % 8 == 0)
      move_rows<uint2>(p, cache, plane, at, width, b, old_len, n);
    else
      move_rows<uint32_t>(p, cache, plane, at, width, b, old_len, n);
    return;
  }
  // The weights: one value a position, and zeros after the last kept one.
  const float* w = p.weights + static_cast<int64_t>(b) * p.ldw;
  float* out = p.weights_out + static_cast<int64_t>(b) * p.ldw;
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.budget;
  for (int base = 0; base < n; base += kMoveThreads) {
    const int i = base + threadIdx.x;
    float v = 0.f;
    if (i < n) {
      const int pos = __ldg(keep + i);
      if (pos >= 0 && pos < old_len) v = w[pos];
    }
    __syncthreads();
    if (i < n) out[i] = v;
  }
  __syncthreads();
  for (int i = n + threadIdx.x; i < cap; i += kMoveThreads) out[i] = 0.f;
}

}  // namespace

// Short contexts, and no more requests than there are SMs, for one fills one:
// selecting and moving 1024 of up to 32768 positions takes, with the one kernel
// and with the general path, 53 and 68 us (1 request), 49 and 69 (8), 70 and 70
// (64), 104 and 105 (128), but 154 and 145 (192) and 190 and 182 (256).
bool evict_small(int B, int max_ctx) {
  return max_ctx <= kSmallCtx && B <= device_sm_count();
}

cudaError_t launch_evict_small(const float* weights, int64_t ldw, const int32_t* lens, int B,
                               int max_ctx, int budget, int sink, int recent, int32_t* keep,
                               int32_t* new_lens, uint32_t* err, cudaStream_t s) {
  evict_small_kernel<<<B, kSmallThreads, 0, s>>>(weights, ldw, lens, max_ctx, budget, sink, recent,
                                                 keep, new_lens, err);
  return cudaGetLastError();
}

cudaError_t launch_evict_ranges(const int32_t* lens, int B, int max_ctx, int sink, int recent,
                                int32_t* starts, int32_t* ends, uint32_t* err, cudaStream_t s) {
  evict_ranges_kernel<<<(B + 255) / 256, 256, 0, s>>>(lens, B, max_ctx, sink, recent, starts, ends,
                                                      err);
  return cudaGetLastError();
}

cudaError_t launch_evict_keep(const int32_t* lens, const int32_t* starts, const int32_t* ends,
                              const int32_t* mid, int B, int max_ctx, int room, int budget,
                              int32_t* keep, int32_t* new_lens, cudaStream_t s) {
  const dim3 grid((budget + 255) / 256, B);
  evict_keep_kernel<<<grid, 256, 0, s>>>(lens, starts, ends, mid, B, max_ctx, room, budget, keep,
                                         new_lens);
  return cudaGetLastError();
}

int64_t compact_units(const CompactParams::Cache& c) {
  const int64_t slices = (static_cast<int64_t>(c.row_bytes) + kSlice - 1) / kSlice;
  return c.planes * slices;
}

cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t s) {
  const int units = p.units + (p.weights ? 1 : 0);
  if (units == 0 || p.B == 0) return cudaSuccess;
  if (p.new_block_table)
    kv_move_kernel<<<dim3((p.budget + kPartRows - 1) / kPartRows, p.B), kMoveThreads, 0, s>>>(p);
  else
    kv_compact_kernel<<<dim3(units, p.B), kMoveThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
