// dsa_kv_evict.cu -- eviction from a paged cache by accumulated attention
// weight: which tokens a budget keeps, and moving their rows together.
//
//   keep[b] = the first `sink` positions, the `budget - sink - recent` of the
//             middle with the largest weight (ties to the lower position) and
//             the last `recent`, ascending
//
// The middle's selection is the library's masked top-k on the weights; the two
// small kernels here make its row ranges and put the three parts together.
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
  // Entries of the selection before its -1 padding (it ascends).
  int n = 0, step = 1;
  while (step <= room) step <<= 1;
  for (step >>= 1; step > 0; step >>= 1)
    if (n + step <= room && m[n + step - 1] >= 0) n += step;
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

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;  // rows a thread holds per chunk
constexpr int kSlice = 128;     // bytes of a row one CTA moves
constexpr int kPartRows = 1024; // rows a CTA moves when pages are fresh

// Rows [i0, i1) of one slice (plane, byte range) of a cache.
template <typename V, bool kInPlace>
__device__ __forceinline__ void move_rows(const CompactParams& p, const CompactParams::Cache& c,
                                          int plane, int at, int width, int b, int old_len, int i0,
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
  const int32_t* dst_table =
      kInPlace ? table : p.new_block_table + static_cast<int64_t>(b) * p.new_max_blocks;
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
      if (kInPlace && pos == i) continue;
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
      uint8_t* dst = address(dst_table, base + u * rows + row_in);
      if (dst) *reinterpret_cast<V*>(dst) = v[u];
    }
  };
  load(buf[0], got[0], i0);
  for (int base = i0; base < i1; base += 2 * chunk) {
    // The next chunk's rows lie at or above its own first position, so
    // reading them does not wait for this chunk's stores; this chunk's stores
    // wait for every thread's reads of this chunk.
    load(buf[1], got[1], base + chunk);
    if (kInPlace) __syncthreads();
    store(buf[0], got[0], base);
    load(buf[0], got[0], base + 2 * chunk);
    if (kInPlace) __syncthreads();
    store(buf[1], got[1], base + chunk);
  }
}

template <bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads)
    kv_compact_kernel(const __grid_constant__ CompactParams p) {
  const int b = blockIdx.z, unit = blockIdx.x, part = blockIdx.y;
  const int cap = p.max_blocks << p.log_bs;
  const int old_len = clamp_len(__ldg(p.old_lens + b), cap);
  int n = __ldg(p.new_lens + b);
  if (n < 0 || n > p.budget) {
    if (threadIdx.x == 0) record_error(p.err, kErrBadIndex);
    n = n < 0 ? 0 : p.budget;
  }
  if (!kInPlace) n = min(n, p.new_max_blocks << p.log_bs);
  else n = min(n, cap);
  if (unit < p.units) {
    const int i0 = kInPlace ? 0 : part * kPartRows;
    const int i1 = kInPlace ? n : min(n, i0 + kPartRows);
    if (i0 >= i1) return;
    int c = 0;
    while (unit >= p.first_unit[c + 1]) ++c;
    const CompactParams::Cache cache = p.cache[c];
    const int slices = (cache.row_bytes + kSlice - 1) / kSlice;
    const int u = unit - p.first_unit[c];
    const int plane = u / slices, at = (u % slices) * kSlice;
    const int width = min(kSlice, cache.row_bytes - at);
    if (width % 16 == 0 && cache.row_bytes % 16 == 0)
      move_rows<uint4, kInPlace>(p, cache, plane, at, width, b, old_len, i0, i1);
    else if (width % 8 == 0 && cache.row_bytes % 8 == 0)
      move_rows<uint2, kInPlace>(p, cache, plane, at, width, b, old_len, i0, i1);
    else
      move_rows<uint32_t, kInPlace>(p, cache, plane, at, width, b, old_len, i0, i1);
    return;
  }
  // The weights: one value a position, and zeros after the last kept one.
  const float* w = p.weights + static_cast<int64_t>(b) * p.ldw;
  float* out = p.weights_out + static_cast<int64_t>(b) * p.ldw;
  // Rewritten where they lie, they are one CTA's work whatever the pages do.
  const bool alone = p.weights_out == p.weights;
  if (alone && part > 0) return;
  const int i0 = alone ? 0 : part * kPartRows, i1 = alone ? n : min(n, i0 + kPartRows);
  const int32_t* keep = p.keep + static_cast<int64_t>(b) * p.budget;
  for (int base = i0; base < i1; base += kMoveThreads) {
    const int i = base + threadIdx.x;
    float v = 0.f;
    if (i < i1) {
      const int pos = __ldg(keep + i);
      if (pos >= 0 && pos < old_len) v = w[pos];
    }
    __syncthreads();
    if (i < i1) out[i] = v;
  }
  __syncthreads();
  const int parts = alone ? 1 : gridDim.y;
  const int64_t rest = cap - n;
  const int64_t z0 = n + rest * part / parts, z1 = n + rest * (part + 1) / parts;
  for (int64_t i = z0 + threadIdx.x; i < z1; i += kMoveThreads) out[i] = 0.f;
}

}  // namespace

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

int compact_units(const CompactParams::Cache& c) {
  return c.planes * ((c.row_bytes + kSlice - 1) / kSlice);
}

cudaError_t launch_kv_compact(const CompactParams& p, cudaStream_t s) {
  const int units = p.units + (p.weights ? 1 : 0);
  if (units == 0 || p.B == 0) return cudaSuccess;
  if (p.new_block_table) {
    const dim3 grid(units, (p.budget + kPartRows - 1) / kPartRows, p.B);
    kv_compact_kernel<false><<<grid, kMoveThreads, 0, s>>>(p);
  } else {
    kv_compact_kernel<true><<<dim3(units, 1, p.B), kMoveThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace dsa
