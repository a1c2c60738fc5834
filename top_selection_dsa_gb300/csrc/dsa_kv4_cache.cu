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
// A lane moves sixteen elements: the same eighth-of-32 of two neighbouring scale
// blocks (two 16-byte pieces of bf16).  Their key codes are 8 contiguous bytes
// of the record; their value codes are two units in each of two rows of units
// (with two blocks a record these are contiguous; with four, the lanes of the
// two pairs exchange half of them).  A record takes D/8 lanes (the key's, then
// the value's).
// Memory-bound next to its instructions: 32768 tokens of 8 heads of 128 written
// and read back in 66 us, 5.1 TB/s, 100000 in 182 us, 5.7 TB/s.  More records in
// flight a lane were slower (two 69 us, four 73 us), and so was one 16-byte
// piece a lane, which pays for addresses, maxima and exchanges twice as often
// (90 us).
#include "dsa_internal.h"
#include "dsa_kv4.cuh"

namespace dsa {
namespace {

constexpr int kThreads = 256;

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

// Where lane `sub` of a record's D/8 lanes keeps its codes.
template <int D>
struct Lane {
  static constexpr int G = D / kMxBlock;
  bool is_v;
  int g, t;   // its blocks, g and g + 1, and place in them
  int word;   // its two 4-byte words of the record: the first
  __device__ explicit Lane(int sub) {
    is_v = sub >= D / 16;
    g = 2 * (sub % (D / 16) / 4), t = sub % 4;
    // Value: rows 2t and 2t + 1 of units, G/2 words each; with four blocks the
    // first pair's lane keeps the one and the second's the other.
    word = !is_v ? t * G + g : D / 8 + (G == 2 ? 2 * t : 4 * t + g);
  }
  __device__ int e16(int b) const { return 4 * (g + b) + t; }  // its 16-byte pieces of a row
  // Codes of its eight elements of either block -> the words it stores (whole
  // warps).
  __device__ uint2 pack(uint2 c) const {
    const uint2 v = make_uint2(__byte_perm(c.x, c.y, 0x5410), __byte_perm(c.x, c.y, 0x7632));
    const uint2 x = G == 4 ? swap(v) : v;
    return is_v ? x : c;
  }
  // The words it loaded -> codes of its elements (whole warps).
  __device__ uint2 unpack(uint2 w) const {
    uint2 v = G == 4 ? swap(w) : w;
    v = make_uint2(__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632));
    return is_v ? v : w;
  }

 private:
  // Of a 2 x 2 block of words in two lanes, the transpose.
  __device__ uint2 swap(uint2 v) const {
    const uint32_t got = __shfl_xor_sync(0xffffffffu, g ? v.x : v.y, 4);
    return g ? make_uint2(got, v.y) : make_uint2(v.x, got);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_insert_kernel(const __grid_constant__ CacheParams p) {
  constexpr int G = D / kMxBlock;
  constexpr int kLanes = D / 8;  // D/16 for the key row, D/16 for the value row
  constexpr uint32_t kPerCta = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const Lane<D> lane(sub);
  const uint16_t* const src = lane.is_v ? p.v : p.k;
  const int64_t src_stride = lane.is_v ? p.v_stride : p.k_stride;
  for (uint32_t base = blockIdx.x * kPerCta; base < p.items; base += gridDim.x * kPerCta) {
    const uint32_t item = base + threadIdx.x / kLanes;
    uint4 raw[2];
    raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
    uint32_t rec = 0;
    bool ok = false;
    if (item < p.items) {
      const uint32_t tok = token_of(p, item);
      const uint32_t head = item - tok * p.Hkv;
      const int64_t slot = __ldg(p.slots + tok);
      const uint4* row = reinterpret_cast<const uint4*>(src + tok * src_stride + head * D);
      raw[0] = __ldg(row + lane.e16(0));
      raw[1] = __ldg(row + lane.e16(1));
      ok = slot >= 0 && slot < p.capacity;
      if (ok) rec = record_of(p, static_cast<uint32_t>(slot), head);
      else if (slot >= 0 && sub == 0 && head == 0) record_error(p.err, kErrBadIndex);
    }
    // The largest magnitudes as bits: a NaN's or an infinity's are above every
    // finite value's, so one integer maximum finds either.  The two blocks'
    // share a word.
    uint32_t m[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
      m[b] = max_u16x2(max_u16x2(raw[b].x & 0x7FFF7FFFu, raw[b].y & 0x7FFF7FFFu),
                       max_u16x2(raw[b].z & 0x7FFF7FFFu, raw[b].w & 0x7FFF7FFFu));
    uint32_t mag = max_u16x2(__byte_perm(m[0], m[1], 0x5410), __byte_perm(m[0], m[1], 0x7632));
    mag = max_u16x2(mag, __shfl_xor_sync(0xffffffffu, mag, 1));
    mag = max_u16x2(mag, __shfl_xor_sync(0xffffffffu, mag, 2));
    uint32_t codes[2], scale[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
      const uint32_t amax = b == 0 ? mag & 0xFFFFu : mag >> 16;  // bf16 bits
      // 6 * 2^e = 1.5 * 2^(e+2): biased, the exponent of amax less two, and one
      // more for a mantissa above 1.5 (whose addition carries).
      int e = static_cast<int>((amax + 0x3Fu) >> 7) - 2;
      e = amax == 0 ? 127 : max(e, 1);
      const bool bad = amax >= 0x7F80u;
      // x / 2^(e - 127): exact where it matters (what it rounds, below 2^-126,
      // is far below half of the smallest code).
      const uint32_t inv = static_cast<uint32_t>(254 - e) * 0x00800080u;
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = mul_bf16x2(w[j], inv);
        c |= f32x2_to_e2m1x2(bf16_lo(y), bf16_hi(y)) << (8 * j);
      }
      codes[b] = bad ? 0u : c;
      scale[b] = bad ? 255u : static_cast<uint32_t>(e);
    }
    const uint2 out = lane.pack(make_uint2(codes[0], codes[1]));
    if (!ok) continue;
    *reinterpret_cast<uint2*>(p.cache + static_cast<uint64_t>(rec) * D + lane.word * 4) = out;
    if (lane.t == 0)
      *reinterpret_cast<uint16_t*>(p.scales + static_cast<uint64_t>(rec) * (D / 16) +
                                   (lane.is_v ? G : 0) + lane.g) =
          static_cast<uint16_t>(scale[0] | (scale[1] << 8));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_gather_kernel(const __grid_constant__ CacheParams p) {
  constexpr int G = D / kMxBlock;
  constexpr int kLanes = D / 8;
  constexpr uint32_t kPerCta = kThreads / kLanes;
  const int sub = threadIdx.x % kLanes;
  const Lane<D> lane(sub);
  uint16_t* const out = lane.is_v ? p.v_out : p.k_out;
  for (uint32_t base = blockIdx.x * kPerCta; base < p.items; base += gridDim.x * kPerCta) {
    const uint32_t item = base + threadIdx.x / kLanes;
    uint2 codes = make_uint2(0u, 0u);
    uint32_t scales = 0x7F7Fu;
    if (item < p.items) {
      const uint32_t tok = token_of(p, item);
      const uint32_t head = item - tok * p.Hkv;
      const int64_t slot = __ldg(p.slots + tok);
      if (slot >= p.capacity) {
        if (sub == 0 && head == 0) record_error(p.err, kErrBadIndex);
      } else if (slot >= 0) {
        const uint64_t rec = record_of(p, static_cast<uint32_t>(slot), head);
        codes = *reinterpret_cast<const uint2*>(p.cache + rec * D + lane.word * 4);
        scales = *reinterpret_cast<const uint16_t*>(p.scales + rec * (D / 16) +
                                                    (lane.is_v ? G : 0) + lane.g);
      }
    }
    codes = lane.unpack(codes);
    if (item >= p.items) continue;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t c = b == 0 ? codes.x : codes.y;
      const uint32_t e = b == 0 ? scales & 0xFFu : scales >> 8;
      const float s = __uint_as_float(e == 255 ? 0x7FC00000u : e << 23);
      const uint32_t h[4] = {e2m1x2_to_f16x2<0>(c), e2m1x2_to_f16x2<1>(c),
                             e2m1x2_to_f16x2<2>(c), e2m1x2_to_f16x2<3>(c)};
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
        o[j] = pack_bf16(f.x * s, f.y * s);
      }
      *(reinterpret_cast<uint4*>(out + static_cast<int64_t>(item) * D) + lane.e16(b)) =
          make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

int cache_grid(int64_t items, int D) {
  const int64_t per = kThreads / (D / 8);
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
