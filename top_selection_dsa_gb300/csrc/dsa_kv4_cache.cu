// dsa_kv4_cache.cu -- writing bf16 keys and values into the paged 4-bit cache
// and reading them back as bf16.
//
// Quantisation, per block of 32 elements of a head's row: s = 2^e with e the
// smallest exponent, no less than -126, for which max|x| <= 6 * 2^e (e = 0 for
// a block of zeros), codes = x / s rounded to the nearest E2M1 value, ties to
// the even code (nothing saturates).  A block that holds a NaN or an infinity
// is written as scale code 255 (NaN) with zero codes: all of it reads back as
// NaN.  Reading back is exact in bf16 (two significant bits times a power of
// two).
//
// Both are memory-bound: one lane moves eight elements (16 bytes of bf16), a
// record takes D/4 lanes (the key's, then the value's), and a lane has
// kRecords records in flight.  A lane's eight value codes belong to two rows of
// the record four bytes apart; it exchanges half of them with the lane of the
// neighbouring block, so that a record is one 4-byte access a lane.
#include "dsa_internal.h"
#include "dsa_kv4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kRecords = 4;

struct CacheParams {
  const uint16_t* k;  // insert: [T, Hkv, D], rows k_stride / v_stride elements apart
  const uint16_t* v;
  int64_t k_stride, v_stride;
  uint16_t* k_out;    // gather: [T, Hkv, D], dense
  uint16_t* v_out;
  const int64_t* slots;
  uint32_t items;     // T * Hkv
  int Hkv, log_bs;
  uint32_t div_mul;   // item / Hkv = (item * div_mul) >> div_shift, for items < 2^30
  int div_shift;
  int64_t capacity;
  uint8_t* cache;
  uint8_t* scales;
  uint32_t* err;
};

__device__ __forceinline__ uint32_t token_of(const CacheParams& p, uint32_t item) {
  return static_cast<uint32_t>((static_cast<uint64_t>(item) * p.div_mul) >> p.div_shift);
}

// Record number of (slot, head), a slot of the cache: ((slot / bs) * Hkv +
// head) * bs + slot % bs, below 2^32 as all record numbers are.
__device__ __forceinline__ uint32_t record_of(const CacheParams& p, uint32_t slot, uint32_t head) {
  const uint32_t block = slot >> p.log_bs;
  return ((block * p.Hkv + head) << p.log_bs) + (slot & ((1u << p.log_bs) - 1u));
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Where lane `sub` of a record's D/4 lanes keeps its codes.
template <int D>
struct Lane {
  static constexpr int G = D / kMxBlock;
  bool is_v;
  int e8, g, t;   // its eight elements 8 e8 .., their block and place in it
  int word;       // its 4-byte word of the record
  __device__ explicit Lane(int sub) {
    is_v = sub >= D / 8;
    e8 = sub % (D / 8);
    g = e8 / 4, t = e8 % 4;
    // Value: units 2t (even blocks) or 2t + 1 (odd) of its block and the
    // neighbouring one.
    word = is_v ? D / 8 + ((2 * t + g % 2) * G + (g & ~1)) / 2 : t * G + g;
  }
  // A lane's eight codes <-> the word it accesses (the exchange is its own
  // inverse; executed by whole warps).
  __device__ uint32_t exchange(uint32_t w) const {
    const bool odd = g % 2;
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? w : w >> 16, 4);
    const uint32_t mixed = odd ? (got & 0xFFFFu) | (w & 0xFFFF0000u) : (w & 0xFFFFu) | (got << 16);
    return is_v ? mixed : w;
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_insert_kernel(const __grid_constant__ CacheParams p) {
  constexpr int G = D / kMxBlock;
  constexpr int kLanes = D / 4;  // D/8 for the key row, D/8 for the value row
  constexpr uint32_t kPerCta = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const Lane<D> lane(sub);
  const uint16_t* const src = lane.is_v ? p.v : p.k;
  const int64_t src_stride = lane.is_v ? p.v_stride : p.k_stride;
  const uint32_t step = gridDim.x * kPerCta;
  const uint32_t first = blockIdx.x * kPerCta;
  for (uint32_t base = first; base < p.items; base += step * kRecords) {
    uint4 raw[kRecords];
    uint32_t rec[kRecords], ok = 0;
#pragma unroll
    for (int i = 0; i < kRecords; ++i) {
      const uint32_t item = base + threadIdx.x / kLanes + i * step;
      rec[i] = 0;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (item < p.items) {
        const uint32_t tok = token_of(p, item);
        const uint32_t head = item - tok * p.Hkv;
        const int64_t slot = __ldg(p.slots + tok);
        raw[i] = __ldg(reinterpret_cast<const uint4*>(src + tok * src_stride + head * D) + lane.e8);
        if (slot >= p.capacity) {
          if (sub == 0 && head == 0) record_error(p.err, kErrBadIndex);
        } else if (slot >= 0) {
          rec[i] = record_of(p, static_cast<uint32_t>(slot), head);
          ok |= 1u << i;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRecords; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      // The largest magnitude as bits: a NaN's or an infinity's are above
      // every finite value's, so one integer maximum finds either.
      uint32_t mag = max_u16x2(max_u16x2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                               max_u16x2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
      mag = max_u16x2(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
      mag = max_u16x2(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
      const uint32_t amax = max(mag & 0xFFFFu, mag >> 16);  // bf16 bits
      // 6 * 2^e = 1.5 * 2^(e+2): compare the mantissa with 1.5.
      int e = static_cast<int>(amax >> 7) - 127 - 2 + ((amax & 0x7Fu) > 0x40u ? 1 : 0);
      e = amax == 0 ? 0 : max(e, -126);
      const bool bad = amax >= 0x7F80u;
      // x / 2^e: exact where it matters (what it rounds, below 2^-126, is
      // far below half of the smallest code).
      const uint32_t inv = static_cast<uint32_t>(127 - e) << 7;
      uint32_t codes = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = mul_bf16x2(w[j], inv | (inv << 16));
        codes |= f32x2_to_e2m1x2(bf16_lo(y), bf16_hi(y)) << (8 * j);
      }
      codes = lane.exchange(bad ? 0u : codes);
      if (!((ok >> i) & 1)) continue;
      *(reinterpret_cast<uint32_t*>(p.cache + static_cast<uint64_t>(rec[i]) * D) + lane.word) =
          codes;
      if (lane.t == 0)
        p.scales[static_cast<uint64_t>(rec[i]) * (D / 16) + (lane.is_v ? G : 0) + lane.g] =
            bad ? 255 : static_cast<uint8_t>(e + 127);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const __grid_constant__ CacheParams p) {
  constexpr int G = D / kMxBlock;
  constexpr int kLanes = D / 4;
  constexpr uint32_t kPerCta = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const Lane<D> lane(sub);
  uint16_t* const out = lane.is_v ? p.v_out : p.k_out;
  const uint32_t step = gridDim.x * kPerCta;
  const uint32_t first = blockIdx.x * kPerCta;
  for (uint32_t base = first; base < p.items; base += step * kRecords) {
    uint32_t codes[kRecords];
    uint32_t sc[kRecords];
#pragma unroll
    for (int i = 0; i < kRecords; ++i) {
      const uint32_t item = base + threadIdx.x / kLanes + i * step;
      codes[i] = 0;
      sc[i] = 127;
      if (item < p.items) {
        const uint32_t tok = token_of(p, item);
        const uint32_t head = item - tok * p.Hkv;
        const int64_t slot = __ldg(p.slots + tok);
        if (slot >= p.capacity) {
          if (sub == 0 && head == 0) record_error(p.err, kErrBadIndex);
        } else if (slot >= 0) {
          const uint64_t rec = record_of(p, static_cast<uint32_t>(slot), head);
          codes[i] = *(reinterpret_cast<const uint32_t*>(p.cache + rec * D) + lane.word);
          sc[i] = p.scales[rec * (D / 16) + (lane.is_v ? G : 0) + lane.g];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kRecords; ++i) {
      const uint32_t item = base + threadIdx.x / kLanes + i * step;
      const uint32_t c = lane.exchange(codes[i]);
      if (item >= p.items) continue;
      const float s = __uint_as_float(sc[i] == 255 ? 0x7FC00000u : sc[i] << 23);
      const uint32_t h[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c), e2m1x2_to_f16x2<2>(c),
                             e2m1x2_to_f16x2<3>(c)};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        o[j] = pack_bf16(f.x * s, f.y * s);
      }
      *(reinterpret_cast<uint4*>(out + static_cast<int64_t>(item) * D) + lane.e8) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int cache_grid(int64_t items, int D) {
  const int64_t per = static_cast<int64_t>(kThreads / (D / 4)) * kRecords;
  const int64_t need = (items + per - 1) / per;
  const int64_t cap = static_cast<int64_t>(device_sm_count() > 0 ? device_sm_count() : 1) * 16;
  return static_cast<int>(need < cap ? need : cap);
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

// Division by Hkv of numbers below 2^30, by a multiplication: with l the
// exponent of the power of two at or above Hkv, floor(2^(30+l) / Hkv) + 1 is
// close enough to 2^(30+l) / Hkv.
void set_division(CacheParams* p) {
  const int l = log2_of(p->Hkv);
  p->div_shift = 30 + l;
  p->div_mul = static_cast<uint32_t>((uint64_t(1) << (30 + l)) / p->Hkv + 1);
}

}  // namespace

cudaError_t launch_kv4_insert(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                              const int64_t* slots, int T, int Hkv, int D, void* cache,
                              void* scales, int num_blocks, int block_size, uint32_t* err,
                              cudaStream_t s) {
  CacheParams p = {};
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.items = static_cast<uint32_t>(T) * static_cast<uint32_t>(Hkv);
  p.Hkv = Hkv;
  set_division(&p);
  p.log_bs = log2_of(block_size);
  p.capacity = static_cast<int64_t>(num_blocks) * block_size;
  p.cache = static_cast<uint8_t*>(cache);
  p.scales = static_cast<uint8_t*>(scales);
  p.err = err;
  if (p.items == 0) return cudaSuccess;
  if (D == 128)
    kv4_insert_kernel<128><<<cache_grid(p.items, D), kThreads, 0, s>>>(p);
  else
    kv4_insert_kernel<64><<<cache_grid(p.items, D), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const void* cache, const void* scales, const int64_t* slots, int T,
                              int Hkv, int D, int num_blocks, int block_size, void* k, void* v,
                              uint32_t* err, cudaStream_t s) {
  CacheParams p = {};
  p.k_out = static_cast<uint16_t*>(k);
  p.v_out = static_cast<uint16_t*>(v);
  p.slots = slots;
  p.items = static_cast<uint32_t>(T) * static_cast<uint32_t>(Hkv);
  p.Hkv = Hkv;
  set_division(&p);
  p.log_bs = log2_of(block_size);
  p.capacity = static_cast<int64_t>(num_blocks) * block_size;
  p.cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  p.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  p.err = err;
  if (p.items == 0) return cudaSuccess;
  if (D == 128)
    kv4_gather_kernel<128><<<cache_grid(p.items, D), kThreads, 0, s>>>(p);
  else
    kv4_gather_kernel<64><<<cache_grid(p.items, D), kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace dsa
