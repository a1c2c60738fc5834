// dsa_kv4_attn.cu -- decode attention over the paged 4-bit key/value cache
// (layout in dsa_kv4.cuh), over every key of a request or over the columns an
// indexer selected.
//
//   S[n,c] = scale * q[n] . K[c]       for the columns c that row n sees
//   lse[n] = log sum_c exp S[n,c]      out[n] = sum_c exp(S[n,c] - lse[n]) V[c]
//
// The query rows of a key/value head (its group's heads, of all tokens of the
// request, or of one token on a selection) share one reading of its records;
// two kernels take them:
//
// Up to 16 rows: kv4_attn_kernel.  One warp walks tiles of 64 columns: TMA
// (dense) or cp.async (selected) brings the tile's records and scales into the
// warp's own two-stage ring, and everything after that stays in registers.
//   S     mma m16n8k16.  Up to 8 rows the keys are the 16-row operand, S^T =
//         K q^T; from 9 on the query rows are, S = q K^T, with q's fragments
//         in shared memory.  The keys' fp16 elements are the E2M1 codes'
//         values themselves (exact); the blocks of 32 elements accumulate
//         apart and are summed in fp32 with their power-of-two scales.  q is
//         divided by a power of two per row so that its largest element is in
//         [1, 2): bf16's eight bits fit fp16 exactly, and elements below 2^-24
//         of the row's largest vanish.
//   softmax  one pass: running maximum m and sum l per row (base 2, in fp32);
//         m lags by up to a slack, so that the accumulated output is rescaled
//         seldom.
//   O     += V^T P (O += P V): V's elements again the codes' values, and the
//         value scales multiplied into P (fp16), by block of 32 channels
//         relative to the largest scale met so far, 2^x, which lags behind by up
//         to kValueMost; terms below 2^-24 of 2^x in units of 2^-kRoom vanish.
//         A request's new tokens do not all see one another: a later one's
//         larger scale is met in a window of columns of its own, after those
//         that every row sees, and rows that do not see it keep their 2^x.
// More rows: kv4_attn_tc_kernel, the same on the tensor cores' tcgen05 form
// (further down).
//
// Times of one GB300 (copy bandwidth 6.68 TB/s), calls with their joins:
//   64 requests of 4096 to 131072 keys, 8 key/value heads of 128 (2.55 GB):
//     8 rows a head    412 us, 6.2 TB/s: bound by memory
//     16 rows          597 us, 4.3 TB/s: bound by issue and latency (53 % of
//                      the issue slots, ALU and tensor pipes 45 % each, three
//                      warps a scheduler is what the registers leave)
//   one request of 131071 keys, 8 rows   40 us, 3.5 TB/s: start and join
//   2048 selected of each of 128 rows    80 us: single records of 128 bytes and
//     scales of 8 from all over 2.5 GB (a plain gather of those took 71 us;
//     DRAM is read by 64 bytes, which makes it 400 MB); 105 us with weights
// Tried and slower: tiles of 32 columns in three stages; 8 warps with 254
// registers for 16 rows (637 to 716 us); tcgen05 for 16 rows (856); TMA gathers
// of selected records (103.5 against cp.async's 98.4).
// Rounding P to fp16 costs up to 2^-11 of each term (the output's bf16 rounding
// up to 2^-8); l sums the unrounded weights.  A reference by block and windows
// instead of one reference for all columns and channels: 8 rows 405 -> 412 us, 16
// rows 590 -> 597.
//
// Rows of the m16 operand are permuted within each group of eight (odd rows
// exchange halves, row i holds key i ^ 4): with the records' 16-byte chunks
// XOR-swizzled by the key's index in its group of eight, the 16-byte key
// loads and the 8-byte value loads are then both free of bank conflicts.
//
// The work is cut into equal shares, one per resident CTA, whatever the
// requests' lengths (Walk below); a CTA that has all of a row's columns writes
// the result, otherwise partial sums that a second kernel joins.
#include <math.h>

#include <atomic>

#include "dsa_internal.h"
#include "dsa_kv4.cuh"
#include "dsa_kv4_span.h"

namespace dsa {
namespace {

constexpr int kTile = 64;       // columns a warp takes at a time
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
// A weight's largest value is 2^(kSlack + kRoom), a value scale's over its
// reference kValueMost; fp16 holds their product.  What is below 2^-24 of 1
// vanishes: the room keeps the sum of many small weights beside a large one.
constexpr float kSlack = 8.f;
constexpr float kRoom = 5.f;
constexpr float kValueMost = 4.f;
// Three fill an SM's registers (168 a thread) and shared memory.  On a selection
// that leaves the L1, through which the gathers of single records go, 28 KB, and
// two CTAs' fewer copies in flight are faster: 128 rows of 2048 selected keys, 8
// heads, 82 us against 97 (with weights 108 against 131), 4 requests' 18
// against 22; but two CTAs of three stages, which fill the shared memory again,
// 107.  Dense copies do not pass through it: 64 requests 404 us with three CTAs,
// 456 with two.
constexpr int ctas_per_sm(bool sel) { return sel ? 2 : 3; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 pol;\n\tcreatepolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
      "cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, pol;\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes)
      : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The low nibbles of a's bytes with the high nibbles of b's: one three-input
// logic operation.
__device__ __forceinline__ uint32_t low_nibbles_of(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, 0x0F0F0F0F, 0xE4;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
// The two low bytes of w as bf16 numbers 2^(byte - 127).
__device__ __forceinline__ uint32_t e8m0x2_to_bf16x2(uint32_t w) {
  return ((w & 0xFFu) << 7) | ((w & 0xFF00u) << 15);
}

// Non-zero when a byte of w is 255.
__device__ __forceinline__ uint32_t has_ff(uint32_t w) {
  return (~w - 0x01010101u) & w & 0x80808080u;
}

// Shared memory of a CTA: all warps' rings of tiles first (1024-byte aligned,
// the swizzle is a function of the address; there is no static shared memory,
// so the block begins so aligned), then by warp the tiles' scales, what the
// tile in work needs of them -- 2^e of every key's blocks (fp32), and the
// value factors as fp16 pairs in the order of P's fragments -- the ring's
// barriers, and the value scales' references.
template <int D, int NT>
struct Layout {
  static constexpr int G = D / kMxBlock;        // scale blocks of a row
  static constexpr int kChunks = D / 16;        // 16-byte chunks of a record
  static constexpr int kSc = D / 16;            // scale bytes of a record
  static constexpr int kTileBytes = kTile * D;
  static constexpr int kScaleBytes = kTile * kSc;
  static constexpr int kWarpTiles = kStages * kTileBytes;
  // Per warp, after all warps' tiles:
  static constexpr int kScales = 0;
  static constexpr int kKeyScales = kScales + kStages * kScaleBytes;
  static constexpr int kFactors = kKeyScales + (NT > 1 ? 0 : kTile * G * 4);
  static constexpr int kBarriers = kFactors + kTile * G * 2;
  static constexpr int kInvUnit = kBarriers + 8 * kStages;    // 2^-x by block
  static constexpr int kRowUnits = kInvUnit + 16;             // every row's x, E8M0 by block
  static constexpr int kNext = kRowUnits + NT * 8 * 4;        // where the tile's next window begins
  static constexpr int kWarpRest = kNext + 16;
  static_assert(kInvUnit % 16 == 0 && kWarpRest % 16 == 0, "");
  // Then, with two row tiles, the query fragments and their factors.
  static constexpr int kQueries = kWarps * (kWarpTiles + kWarpRest);
  static constexpr int kFactorF = kQueries + (NT > 1 ? NT * G * 32 * 16 : 0);
  static constexpr int kLimits = kFactorF + (NT > 1 ? NT * 8 * 4 : 0);
  static constexpr int kWalk = kLimits + NT * 8 * 4;
  static constexpr int kBytes = kWalk + 128;
  // Byte address of chunk c of key `row` of a tile: the 128- (64-) byte
  // swizzle of a tensor map whose rows are the records.
  __device__ static __forceinline__ uint32_t chunk_at(int row, int c) {
    const int f = D == 128 ? (row & 7) : ((row >> 1) & 3);
    return row * D + ((c ^ f) << 4);
  }
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t x) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(x) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

// Byte g of w as the fp32 number 2^(byte - 127) (0 for byte 0).
template <int kByte>
__device__ __forceinline__ uint32_t e8m0_bits(uint32_t w) {
  return (kByte == 3 ? w >> 1 : w << (23 - 8 * kByte)) & 0x7F800000u;
}

// The group (request, or selected row) a CTA works for.
struct Group {
  int b;       // request
  int L;       // tokens in its cache
  int cols;    // columns: cached tokens, or entries of the selection
  int limit;   // selected row: columns it may see
};

__device__ __forceinline__ int context_len(const Kv4AttnParams& p, int b, bool report = false) {
  const int cap = p.max_blocks << p.log_bs;
  const int raw = __ldg(p.context_lens + b);
  if (report && (raw < 0 || raw > cap)) record_error(p.err, kErrBadIndex);
  return raw < 0 ? 0 : (raw > cap ? cap : raw);
}

template <bool kSel>
__device__ __forceinline__ Group group_of(const Kv4AttnParams& p, int g) {
  Group r;
  r.b = kSel ? g / p.next_n : g;
  r.L = context_len(p, r.b);
  r.cols = kSel ? p.sel_k : r.L;
  r.limit = kSel ? max(r.L - p.next_n + (g - r.b * p.next_n) + 1, 0) : r.L;
  return r;
}

// The work of a call is a list of units of kUnit columns, by group, then head
// and row tile, then column (a group without columns has one empty unit); CTA
// i of P takes T / P of the T there are (the first T % P CTAs one more),
// whatever the requests' lengths.  A run of units of one group, head and row tile is a
// span; a CTA's spans are whole, but for its first and its last, which may be
// shared with its neighbours.
// The walk lives in shared memory (its state would cost every thread a dozen
// registers): warp 0 begins it, thread 0 takes the next span.
struct Span {
  int g, ht;       // group (-1: no more); head and row tile
  int u0, u1;      // units of it
  int units;       // that there are
  int first;       // of the CTA
  Group gr;
  __device__ bool whole() const { return u0 == 0 && u1 == units; }
};

template <bool kSel, int kUnit>
struct Walk {
  uint32_t t, t1;        // units left: [t, t1)
  uint32_t each, more;   // every CTA has `each` units, the first `more` one more
  uint32_t base;         // units before group g
  int g;
  bool first;
  Span span;             // the one in work

  __device__ static int units_of(int cols) { return cols > 0 ? (cols + kUnit - 1) / kUnit : 1; }

  __device__ Walk() {}
  // Executed by whole warps.
  __device__ __forceinline__ explicit Walk(const Kv4AttnParams& p) {
    const int per = p.Hkv * p.row_tiles;
    const int lane = threadIdx.x & 31;
    first = true;
    if constexpr (kSel) {
      const uint32_t upg = static_cast<uint32_t>(units_of(p.sel_k)) * per;
      share(upg * p.groups);
      g = static_cast<int>(t / upg);
      base = g * upg;
      if (blockIdx.x == 0)
        for (int b = lane; b < p.groups / p.next_n; b += 32) context_len(p, b, true);
    } else {
      const bool report = blockIdx.x == 0;
      uint32_t mine = 0;
      for (int b = lane; b < p.groups; b += 32)
        mine += units_of(context_len(p, b, report));
      share(__reduce_add_sync(0xffffffffu, mine) * per);
      base = 0;
      g = 0;
      for (int b0 = 0; b0 < p.groups; b0 += 32) {
        const uint32_t v =
            b0 + lane < p.groups
                ? static_cast<uint32_t>(units_of(context_len(p, b0 + lane))) * per : 0;
        uint32_t incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, t < base + incl);
        if (past) {
          const int src = __ffs(past) - 1;
          g = b0 + src;
          base += __shfl_sync(0xffffffffu, incl - v, src);
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  __device__ __forceinline__ void share(uint32_t total) {
    each = total / gridDim.x;
    more = total - each * gridDim.x;
    t = blockIdx.x * each + min(blockIdx.x, more);
    t1 = t + each + (blockIdx.x < more ? 1 : 0);
  }
  // Thread 0: the next span.  Where its group, head and row tile begin is noted
  // for the join: .x this CTA; .y how many CTAs share them; .z which of this
  // CTA's two partial results is theirs (the others' are their first).
  __device__ __forceinline__ void next(const Kv4AttnParams& p) {
    if (t >= t1) {
      span.g = -1;
      return;
    }
    Span s;
    s.gr = group_of<kSel>(p, g);
    s.g = g;
    s.units = units_of(s.gr.cols);
    s.ht = static_cast<int>((t - base) / s.units);
    s.u0 = static_cast<int>(t - base) - s.ht * s.units;
    s.u1 = min(s.u0 + static_cast<int>(t1 - t), s.units);
    s.first = first;
    first = false;
    t += s.u1 - s.u0;
    if (s.u0 == 0 && p.spans)
      p.spans[static_cast<int64_t>(s.g) * p.Hkv * p.row_tiles + s.ht] =
          make_int4(blockIdx.x, cta_of(t + s.units - s.u1 - 1) - blockIdx.x + 1, s.first ? 0 : 1, 0);
    if (s.u1 == s.units && s.ht == p.Hkv * p.row_tiles - 1) {
      ++g;
      base = t;
    }
    span = s;
  }
  // The CTA that takes unit x.
  __device__ __forceinline__ int cta_of(uint32_t x) const {
    const uint32_t ahead = more * (each + 1);
    return static_cast<int>(x < ahead ? x / (each + 1) : more + (x - ahead) / each);
  }
};

// Warp 0 of a CTA: begins the walk.
template <class W>
__device__ __forceinline__ void begin_walk(W* walk, const Kv4AttnParams& p) {
  const W w(p);
  if (threadIdx.x == 0) *walk = w;
}

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Where query row n (of a group's rows for one key/value head) lies: the row
// of q, out and lse as [rows, Hq].
template <bool kSel>
__device__ __forceinline__ int64_t head_row(const Kv4AttnParams& p, int g, int head, int n) {
  const int j = kSel ? 0 : n / p.heads;
  const int64_t row = kSel ? g : static_cast<int64_t>(g) * p.next_n + j;
  return row * p.Hq + head * p.heads + (n - j * p.heads);
}

// What an accumulator of a query row that was divided by 2^E counts in its
// base-2 logit.  Never 0, which a masked column's -inf would make NaN.
__device__ __forceinline__ float row_factor(const Kv4AttnParams& p, int E) {
  if (p.scale_log2e == 0.f) return 1.f;
  return fmaxf(ldexpf(fabsf(p.scale_log2e), E), 1.4012985e-45f);
}

// Which kernel takes a CTA's rows (padded to 8, 16, 32 or 64).  Measured, us,
// mma.sync in tiles of 16 rows against tcgen05, D = 128:
//   64 requests of 4096 to 131072 keys
//     16 rows (4 key/value heads)  303 against 542 (in tiles of 32 rows); as two
//                                  tiles of 8 rows 406
//     32 rows (2 heads; 1)         303; 162 against 301; 161
//     64 rows (2 heads; 1)         588; 303 against 357; 192
//   2048 selected keys of 128 rows, 8 heads, 32 and 64 rows: 185, 350 against
//     165, 230
//   64 requests of 1024 to 16384 keys, 32 and 64 rows on one head: 41, 69 against
//     45, 55 (D = 64: 30, 48 against 37, 46)
//   one request of 131071 keys, 32 and 64 rows on one head: 34, 38 against 42, 46
// So mma.sync is faster still with few columns for every CTA, and with weights,
// where the logits' writes count (64 rows: 90 against 97 for 16 requests of up
// to 32768 keys, 547 against 506 for the 64 above, 270 against 285 on 64
// selections); but whether the weights are asked for does not change the output.
constexpr bool uses_tc(int rows) { return rows > 16; }

// One over a sum of weights, 0 for that of no columns.  Weighted values are
// divided by it before they leave the units of their scales: the mean of the
// values is finite where their sum may not be.
__device__ __forceinline__ float inverse_sum(float l) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(l));  // within 2^-23
  return l == 0.f ? 0.f : r;
}

// One row's four channels d .. d + 3: the result, when the columns summed are
// all of the row's, else the partial result `part` (M: reference of the weights,
// base 2; L: their sum; a: the values' mean under them).
template <int D, int kRows, bool kSel, bool kScores>
__device__ __forceinline__ void write_row(const Kv4AttnParams& p, int grp, int ht, int row0,
                                          int nrows, int row, int d, bool whole, int64_t part,
                                          float M, float L, float4 a) {
  const int per_split = p.Hkv * p.row_tiles;
  const int head = ht / p.row_tiles;
  const int n = row0 + row;
  if (whole) {
    const float lse2 = M + log2f(L);
    if (n < nrows) {
      const int64_t hr = head_row<kSel>(p, grp, head, n);
      *reinterpret_cast<uint2*>(p.out + hr * D + d) =
          make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
      if (d == 0 && p.lse) p.lse[hr] = L == 0.f ? -INFINITY : lse2 * 0.69314718055994531f;
    }
    if (kScores && d == 0)
      p.lse2[(static_cast<int64_t>(grp) * per_split + ht) * kRows + row] =
          n >= nrows || L == 0.f ? INFINITY : lse2;
  } else {
    *reinterpret_cast<float4*>(p.part_o + (part * kRows + row) * D + d) = a;
    if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (part * kRows + row) * 2) = make_float2(M, L);
  }
}

template <int D, int NT, bool kSel, bool kScores>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(kSel))
    kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  using Lay = Layout<D, NT>;
  constexpr int G = Lay::G;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;

  uint8_t* const tiles_p = smem + warp * Lay::kWarpTiles;
  uint8_t* const rest_p = smem + kWarps * Lay::kWarpTiles + warp * Lay::kWarpRest;
  const uint32_t ring = smem_u32(tiles_p), rest = smem_u32(rest_p);
  uint64_t* const bar = reinterpret_cast<uint64_t*>(rest_p + Lay::kBarriers);
  if (!kSel) {
    if (lane == 0) {
#pragma unroll
      for (int s = 0; s < kStages; ++s) mbar_init(&bar[s], 1);
      fence_barrier_init();
    }
    __syncwarp();
  }
  const int per_split = p.Hkv * p.row_tiles;
  const int nrows = kSel ? p.heads : p.heads * p.next_n;
  // The products' fragments.  One row tile: S^T = K q^T and O^T = V^T P, keys
  // and channels as the 16 rows, query rows as the 8 columns: this lane has
  // query rows 2t and 2t + 1, S in two tiles of 16 keys a half tile, O in two
  // of 16 channels a scale block.  Two row tiles: S = q K^T and O = P V, the
  // query rows as the 16 rows: this lane has rows r and r + 8, S in four tiles
  // of 8 keys, O in four of 8 channels a block.
  constexpr int kOut = 2 * NT * G, kPerBlock = 2 * NT;
  auto row_of = [&](int i) { return NT == 1 ? 2 * t + i : r + 8 * i; };
  auto row_ix = [](int j) { return NT == 1 ? j & 1 : j >> 1; };  // of a fragment's element j
  auto* const walk = reinterpret_cast<Walk<kSel, kTile * kWarps>*>(smem + Lay::kWalk);
  if (warp == 0) begin_walk(walk, p);
  launch_dependents();
  int s = 0;           // stage and phase of this warp's next tile
  uint32_t phase = 0;
  bool ok = true;
  for (;;) {
  if (threadIdx.x == 0) walk->next(p);
  if (!__syncthreads_and(ok)) break;  // and the last span's shared memory is free
  const Span span = walk->span;
  if (span.g < 0) break;
  const Group& gr = span.gr;
  const int grp = span.g, ht = span.ht;
  const int head = ht / p.row_tiles;
  const int row0 = (ht % p.row_tiles) * kRows;
  const int c0 = span.u0 * (kTile * kWarps);
  const int c1 = min(gr.cols, span.u1 * (kTile * kWarps));

  // The query rows: one row tile's every warp reads, and before the tiles'
  // copies, behind which it would wait; two tiles' warps 0 and 1 read, later
  // (their other warps' registers are not theirs to fill).
  const bool has_q = NT == 1 || warp < NT;
  const int q_row = row0 + (NT == 1 ? 0 : warp * 8) + r;
  uint4 raw[G];
  auto read_queries = [&]() {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      raw[g] = make_uint4(0u, 0u, 0u, 0u);
      if (q_row < nrows)
        raw[g] = __ldg(reinterpret_cast<const uint4*>(
            p.q + head_row<kSel>(p, grp, head, q_row) * D + g * 32 + t * 8));
    }
  };
  if (NT == 1) read_queries();

  // ------------------------------------------------------------------ loads
  // Tiles of this warp: columns c0 + 64 (warp + 4 i), in stage i % kStages.
  const int tiles = (c1 - c0 + kTile - 1) / kTile;
  const int bs_mask = (1 << p.log_bs) - 1;
  const int32_t* table = p.block_table + static_cast<int64_t>(gr.b) * p.max_blocks;
  // Records of a page and head: result << log_bs ..
  auto page_of = [&](int block) {
    if (block < 0 || block >= p.num_blocks) {
      record_error(p.err, kErrBadIndex);
      block = 0;
    }
    return static_cast<uint32_t>(block) * p.Hkv + head;
  };
  // What a tile's loads need is read ahead of them, and looked at only when
  // they are issued.  Dense: lane i < 64 / rows reads the page of the tile's
  // i-th run of `rows` tokens.  Selected: a lane has the columns `lane` and
  // `lane + 32`, their positions read one tile before their pages.
  const int rows = min(1 << p.log_bs, kTile);
  constexpr int kMine = kSel ? 2 : 1;  // columns (runs) of a tile a lane looks after
  int pos[kMine], next_pos[kMine], block[kMine];
  auto read_columns = [&](int tile, int (&to)[kMine]) {  // selected: positions of `tile`
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int col = c0 + tile * kTile + lane + 32 * i;
      to[i] = col < c1 ? __ldg(p.sel + static_cast<int64_t>(grp) * p.sel_k + col) : -1;
    }
  };
  auto read_pages = [&](int tile, int (&at)[kMine], int (&page)[kMine]) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if constexpr (kSel) {
        if (at[i] < -1 || at[i] >= gr.limit) {
          record_error(p.err, kErrBadIndex);
          at[i] = -1;
        }
      } else {
        at[i] = c0 + tile * kTile + lane * rows;
        if (lane * rows >= kTile || at[i] >= c1) at[i] = -1;
      }
      page[i] = at[i] >= 0 ? __ldg(table + (at[i] >> p.log_bs)) : 0;
    }
  };
  auto locate = [&](int tile) {
    if constexpr (kSel)
#pragma unroll
      for (int i = 0; i < kMine; ++i) pos[i] = next_pos[i];
    read_pages(tile, pos, block);
    if constexpr (kSel) read_columns(tile + kWarps, next_pos);
  };
  // Starts the copies of the located tile into stage s; returns which columns
  // of a selected tile there are (.x: columns 0 .. 31).
  auto fetch = [&](int s, int tile) {
    uint2 cols = make_uint2(0u, 0u);
    const uint32_t base = ring + s * Lay::kTileBytes;
    const uint32_t sbase = rest + Lay::kScales + s * Lay::kScaleBytes;
    if constexpr (kSel) {
      cols.x = __ballot_sync(0xffffffffu, pos[0] >= 0);
      cols.y = __ballot_sync(0xffffffffu, pos[1] >= 0);
      if (cols.x | cols.y) {  // absent columns become zeros
        uint32_t rec[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rec[i] = pos[i] >= 0 ? (page_of(block[i]) << p.log_bs) + (pos[i] & bs_mask) : 0u;
        constexpr int kPer = 32 / Lay::kChunks;  // records per instruction
        const int c = lane % Lay::kChunks;
#pragma unroll
        for (int i = 0; i < kTile / kPer; ++i) {
          const int row = i * kPer + lane / Lay::kChunks;
          const bool upper = i >= kTile / kPer / 2;
          const uint32_t rc = __shfl_sync(0xffffffffu, upper ? rec[1] : rec[0], row & 31);
          cp_async16(base + Lay::chunk_at(row, c), p.cache + static_cast<int64_t>(rc) * D + c * 16,
                     ((upper ? cols.y : cols.x) >> (row & 31)) & 1 ? 16u : 0u);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
          cp_async_small<Lay::kSc>(sbase + (lane + 32 * i) * Lay::kSc,
                                   p.scales + static_cast<int64_t>(rec[i]) * Lay::kSc,
                                   pos[i] >= 0 ? Lay::kSc : 0);
      }
      cp_async_commit();
    } else if (tile < tiles) {
      // Whole runs of a page: what lies past the last column is masked.
      const int n = __popc(__ballot_sync(0xffffffffu, pos[0] >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&bar[s], n * rows * (D + Lay::kSc));
      __syncwarp();
      if (pos[0] >= 0) {
        const uint32_t page = page_of(block[0]);
        const int at = pos[0] & bs_mask;
        tma_load_3d(tiles_p + s * Lay::kTileBytes + lane * rows * D, &p.tmap, &bar[s], 0, at,
                    static_cast<int>(page));
        bulk_load(sbase + lane * rows * Lay::kSc,
                  p.scales + ((static_cast<int64_t>(page) << p.log_bs) + at) * Lay::kSc,
                  rows * Lay::kSc, &bar[s]);
      }
    }
    return cols;
  };

  uint2 cols[kStages];  // oldest first
  {
    // The first tiles' positions, and their pages, read at once.
    int at[kStages][kMine], page[kStages][kMine];
    if constexpr (kSel) {
#pragma unroll
      for (int i = 0; i < kStages; ++i) read_columns(warp + i * kWarps, at[i]);
      read_columns(warp + kStages * kWarps, next_pos);
    }
#pragma unroll
    for (int i = 0; i < kStages; ++i) read_pages(warp + i * kWarps, at[i], page[i]);
#pragma unroll
    for (int i = 0; i < kStages; ++i) {
#pragma unroll
      for (int j = 0; j < kMine; ++j) pos[j] = at[i][j], block[j] = page[i][j];
      cols[i] = fetch((s + i) % kStages, warp + i * kWarps);
    }
  }

  // ---------------------------------------------------------------- queries
  // Lane (r, t) has row r's elements 32 g + 8 t .. + 7, times the softmax
  // scale's sign.  One row tile: the lane's B fragments, which every warp keeps
  // in registers.  Two: the A fragments' rows r and r + 8, prepared by warps 0
  // and 1, which all read from shared memory.
  uint32_t qf[NT == 1 ? G : 1][4];
  float f[2];        // base-2 logit = f * accumulator (f > 0), of this lane's rows
  const bool zero = p.scale_log2e == 0.f;
  const float sign = zero ? 0.f : (p.scale_log2e < 0.f ? -1.f : 1.f);
  const uint32_t q_at = smem_u32(smem) + Lay::kQueries + lane * 16;
  int* const limit_s = reinterpret_cast<int*>(smem + Lay::kLimits);
  if (threadIdx.x < kRows)
    limit_s[threadIdx.x] =
        kSel ? gr.cols
             : gr.L - p.next_n +
                   min((row0 + static_cast<int>(threadIdx.x)) / p.heads, p.next_n - 1) + 1;
  float* const f_s = reinterpret_cast<float*>(smem + Lay::kFactorF);
  if (has_q) {
    if (NT > 1) read_queries();
    const int nt = NT == 1 ? 0 : warp;
    uint32_t amax = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        amax = max(amax, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
    }
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // Exponent of the largest element; rows with none (all zero, or an
    // infinity or NaN somewhere) keep their values.
    const int E = amax == 0 || amax >= 0x7F800000u ? 0
                                                   : max(static_cast<int>(amax >> 23), 1) - 127;
    const float down = ldexpf(sign, -E);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t w[4] = {raw[g].x, raw[g].y, raw[g].z, raw[g].w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = pack_f16(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
      if constexpr (NT == 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) qf[g][i] = h[i];
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = q_at + (g * 2 + i) * 512 + nt * 4;
          sts32(at, h[2 * i]);
          sts32(at + 8, h[2 * i + 1]);
        }
      }
    }
    const float fr = row_factor(p, E);
    if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) f[i] = __shfl_sync(0xffffffffu, fr, (2 * t + i) * 4);
    } else if (t == 0) {
      f_s[nt * 8 + r] = fr;
    }
  }
  __syncthreads();
  if constexpr (NT > 1) {
    f[0] = f_s[r], f[1] = f_s[r + 8];
  }
  // Columns that this lane's row i sees (asked for in the tiles where some row
  // does not see all of them).
  auto limit = [&](int i) { return limit_s[row_of(i)]; };
  const int all_see = kSel ? gr.cols : gr.L - p.next_n + 1;  // columns every row sees

  float o[kOut][4];
#pragma unroll
  for (int x = 0; x < kOut; ++x)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[x][j] = 0.f;
  // m: reference of a row's accumulators, weight = 2^(f (accumulator - m)).  It
  // is raised to the running maximum only when a logit passes it by kSlack
  // (base 2), that is when an accumulator passes thr, so most tiles need no
  // maximum across lanes and no rescaling; weights are then at most 2^kSlack,
  // which fp16 and fp32 hold as well as 1, times 2^kRoom.  thr = -inf: the row
  // has seen no column.
  float thr[2], m[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) thr[i] = -INFINITY, m[i] = l[i] = 0.f;
  // o is in units of its block's largest value scale so far.
  const uint32_t inv_at = rest + Lay::kInvUnit, row_units_at = rest + Lay::kRowUnits;
  if (lane < 4) sts32(inv_at + lane * 4, 0x7E800000u);  // 2^126
  if (lane < kRows) sts32(row_units_at + lane * 4, 0x01010101u);
  const uint32_t next_at = rest + Lay::kNext;  // 0: the tile has no other window
  if (lane == 0) sts32(next_at, 0u);
  __syncwarp();

  // Lane addresses that do not change from tile to tile: the key chunk of
  // rows pi(r) (+ 8, + 16 ..), the value units of rows 2t and (2t+1)^4.
  const int prow = r ^ ((r & 1) << 2);
  const uint32_t k_at =
      D == 128 ? Lay::chunk_at(prow, t) : Lay::chunk_at(prow, t >> 1) + (t & 1) * 8;
  const int v_row[2] = {2 * t, (2 * t + 1) ^ 4};
  uint32_t v_at[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    v_at[i] = D == 128 ? Lay::chunk_at(v_row[i], 4 + (r >> 1)) + (r & 1) * 8
                       : Lay::chunk_at(v_row[i], 2 + (r >> 2)) + (r & 3) * 4;
  const uint32_t ks_at = rest + Lay::kKeyScales, fac_at = rest + Lay::kFactors;

  for (int tile = warp; tile < tiles;) {
    locate(tile + kStages * kWarps);  // what it reads returns under this tile's work
    const int col0 = c0 + tile * kTile;
    const bool tail = !kSel && col0 + kTile > all_see;  // not every row sees all of it
    const int first = tail ? static_cast<int>(lds32(next_at)) : 0;  // of the window
    uint2 live;  // columns of this tile, and window
    if constexpr (kSel) {
      cp_async_wait<kStages - 1>();
      __syncwarp();
      live = cols[0];
    } else {
      ok = mbar_wait_bounded(&bar[s], phase, nullptr);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      const int n = c1 - col0;
      live.x = n >= 32 ? 0xffffffffu : (1u << n) - 1u;
      live.y = n >= 64 ? 0xffffffffu : (n > 32 ? (1u << (n - 32)) - 1u : 0u);
      if (first > 0) {
        live.x &= first >= 32 ? 0u : ~0u << first;
        live.y &= first > 32 ? ~0u << (first - 32) : ~0u;
        __syncwarp();
        if (lane == 0) sts32(next_at, 0u);
      }
    }
    const uint32_t base = ring + s * Lay::kTileBytes;
    const uint32_t sbase = rest + Lay::kScales + s * Lay::kScaleBytes;
    if (live.x | live.y) {
      uint2 nan = make_uint2(0u, 0u);  // keys with a NaN scale
      // ---------------------------------------------------------------- scales
      // Lane 4 q8 + t takes the keys of rows 2t and 2t + 1 of the q8-th group
      // of eight: one fragment pair.
      {
        uint32_t kw[2], vw[2];
        float inv[G], vs[2][G];  // references' inverses; value scales over their references
        int key[2];
        if constexpr (D == 128) {
          const uint4 u = lds128(inv_at);
          inv[0] = __uint_as_float(u.x), inv[1] = __uint_as_float(u.y);
          inv[2] = __uint_as_float(u.z), inv[3] = __uint_as_float(u.w);
        } else {
          const uint2 u = lds64(inv_at);
          inv[0] = __uint_as_float(u.x), inv[1] = __uint_as_float(u.y);
        }
        auto value_scales = [&](uint32_t w, float (&f)[G]) {
          f[0] = __uint_as_float(e8m0_bits<0>(w)), f[1] = __uint_as_float(e8m0_bits<1>(w));
          if constexpr (D == 128)
            f[2] = __uint_as_float(e8m0_bits<2>(w)), f[3] = __uint_as_float(e8m0_bits<3>(w));
        };
        bool rare = false;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          key[i] = r * 8 + v_row[i];
          if constexpr (D == 128) {
            const uint2 u = lds64(sbase + key[i] * 8);
            kw[i] = u.x, vw[i] = u.y;
          } else {
            const uint32_t u = lds32(sbase + key[i] * 4);
            kw[i] = u & 0xFFFFu, vw[i] = u >> 16;
          }
          if constexpr (NT > 1 && !kSel) {
            // A later window: the words made way for the first one's factors.
            if (first > 0 && col0 + key[i] < c1) {
              const int col = col0 + key[i];
              const uint8_t* at = p.scales +
                                  ((static_cast<int64_t>(page_of(__ldg(table + (col >> p.log_bs))))
                                    << p.log_bs) + (col & bs_mask)) * Lay::kSc;
              if constexpr (D == 128) {
                const uint2 u = *reinterpret_cast<const uint2*>(at);
                kw[i] = u.x, vw[i] = u.y;
              } else {
                const uint32_t u = *reinterpret_cast<const uint32_t*>(at);
                kw[i] = u & 0xFFFFu, vw[i] = u >> 16;
              }
            }
          }
          if (!(((r >= 4 ? live.y : live.x) >> (key[i] & 31)) & 1)) kw[i] = vw[i] = 0u;
          rare |= has_ff(kw[i]) != 0;
          value_scales(vw[i], vs[i]);
          float most = 0.f;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            vs[i][g] *= inv[g];
            most = fmaxf(most, vs[i][g]);
          }
          rare |= most > kValueMost;
        }
        if (__any_sync(0xffffffffu, rare)) {
          if (__any_sync(0xffffffffu, has_ff(kw[0]) | has_ff(kw[1]) | has_ff(vw[0]) |
                                          has_ff(vw[1]))) {
            // NaN scales (code 255).  A key's makes its logits NaN below; a
            // value's makes its 32 channels of every row that sees the column
            // NaN, here, and takes no part in the products.
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t from = __ballot_sync(0xffffffffu, has_ff(kw[i]) != 0);
              while (from) {
                const int src = __ffs(from) - 1;
                from &= from - 1;
                const int k = __shfl_sync(0xffffffffu, key[i], src);
                if (k < 32) nan.x |= 1u << k;
                else nan.y |= 1u << (k - 32);
              }
              from = __ballot_sync(0xffffffffu, has_ff(vw[i]) != 0);
              while (from) {
                const int src = __ffs(from) - 1;
                from &= from - 1;
                const uint32_t word = __shfl_sync(0xffffffffu, vw[i], src);
                const int col = col0 + __shfl_sync(0xffffffffu, key[i], src);
                const bool sees[2] = {col < limit(0), col < limit(1)};
#pragma unroll
                for (int g = 0; g < G; ++g)
                  if (((word >> (8 * g)) & 255u) == 255u)
#pragma unroll
                    for (int x = 0; x < kPerBlock; ++x)
#pragma unroll
                      for (int j = 0; j < 4; ++j)
                        if (sees[row_ix(j)]) o[kPerBlock * g + x][j] = __uint_as_float(0x7FC00000u);
              }
#pragma unroll
              for (int g = 0; g < G; ++g)
                if (((vw[i] >> (8 * g)) & 255u) == 255u) vw[i] &= ~(255u << (8 * g));
            }
          }
          // New references: the largest scales of the columns before w0, which
          // the same rows see.  The first column from w0 on whose scale is above
          // them ends the window.
          const int w0 = tail ? max(all_see - col0, first + 1) : kTile;
          float up[G];
          value_scales(vw[0], vs[0]), value_scales(vw[1], vs[1]);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t top = __reduce_max_sync(
                0xffffffffu, max(key[0] < w0 ? __float_as_uint(vs[0][g]) : 0u,
                                 key[1] < w0 ? __float_as_uint(vs[1][g]) : 0u));
            up[g] = fminf(inv[g], __uint_as_float(max(0x7F000000u - top, 0x00800000u)));
          }
          if (tail) {
            int past = kTile;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int g = 0; g < G; ++g)
                if (key[i] >= w0 && vs[i][g] * up[g] > kValueMost) past = min(past, key[i]);
            past = __reduce_min_sync(0xffffffffu, past);
            if (past < kTile) {
              if (lane == 0) sts32(next_at, past);
              live.x &= past >= 32 ? ~0u : (1u << past) - 1u;
              live.y &= past > 32 ? (1u << (past - 32)) - 1u : 0u;
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (key[i] >= past) {
                  kw[i] = 0u;
#pragma unroll
                  for (int g = 0; g < G; ++g) vs[i][g] = 0.f;
                }
            }
          }
          const bool sees[2] = {kSel || limit(0) > col0 + first, kSel || limit(1) > col0 + first};
          uint32_t units = 0;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const float down = up[g] * __uint_as_float(0x7F000000u - __float_as_uint(inv[g]));
            units |= (254u - (__float_as_uint(up[g]) >> 23)) << (8 * g);
            vs[0][g] *= up[g], vs[1][g] *= up[g];
#pragma unroll
            for (int x = 0; x < kPerBlock; ++x)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (sees[row_ix(j)]) o[kPerBlock * g + x][j] *= down;
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (sees[i] && (NT == 1 ? r == 0 : t == 0)) sts32(row_units_at + row_of(i) * 4, units);
          if (lane == 0)
#pragma unroll
            for (int g = 0; g < G; ++g) sts32(inv_at + g * 4, __float_as_uint(up[g]));
        }
        if constexpr (NT == 1) {
          // The key scales as fp32, where rows r of a group of eight find
          // them side by side.
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = ks_at + (r * 8 + 2 * t + i) * (4 * G);
            if constexpr (D == 128)
              sts128(at, e8m0_bits<0>(kw[i]), e8m0_bits<1>(kw[i]), e8m0_bits<2>(kw[i]),
                     e8m0_bits<3>(kw[i]));
            else
              sts64(at, e8m0_bits<0>(kw[i]), e8m0_bits<1>(kw[i]));
          }
        } else {
          // The pair's key scales as bf16, in the place of the scale words
          // (read above): a lane's two keys of an eight-key tile side by side.
          if constexpr (D == 128)
            sts128(sbase + lane * 16, e8m0x2_to_bf16x2(kw[0]), e8m0x2_to_bf16x2(kw[0] >> 16),
                   e8m0x2_to_bf16x2(kw[1]), e8m0x2_to_bf16x2(kw[1] >> 16));
          else
            sts64(sbase + lane * 8, e8m0x2_to_bf16x2(kw[0]), e8m0x2_to_bf16x2(kw[1]));
        }
        uint32_t fac[G];
#pragma unroll
        for (int g = 0; g < G; ++g)
          fac[g] = pack_f16(vs[0][g], vs[1][g]);
        if constexpr (D == 128) sts128(fac_at + lane * 16, fac[0], fac[1], fac[2], fac[3]);
        else sts64(fac_at + lane * 8, fac[0], fac[1]);
        __syncwarp();
      }
      const bool clean =
          (nan.x | nan.y) == 0 && (kSel ? (live.x & live.y) == 0xffffffffu
                                        : col0 + kTile <= min(c1, all_see));
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t hbase = base + half * 32 * D;
        // ------------------------------------------------------------- S = q K^T
        float sacc[2 * NT][4];
        if constexpr (NT == 1) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            uint32_t kw[2][G];
            float ks[2][G];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = hbase + (mt * 16 + h * 8) * D + k_at;
              const uint32_t sat = ks_at + (half * 32 + mt * 16 + h * 8 + r) * (4 * G);
              if constexpr (D == 128) {
                const uint4 u = lds128(at), v = lds128(sat);
                kw[h][0] = u.x, kw[h][1] = u.y, kw[h][2] = u.z, kw[h][3] = u.w;
                ks[h][0] = __uint_as_float(v.x), ks[h][1] = __uint_as_float(v.y);
                ks[h][2] = __uint_as_float(v.z), ks[h][3] = __uint_as_float(v.w);
              } else {
                const uint2 u = lds64(at), v = lds64(sat);
                kw[h][0] = u.x, kw[h][1] = u.y;
                ks[h][0] = __uint_as_float(v.x), ks[h][1] = __uint_as_float(v.y);
              }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t a0 = e2m1x2_to_f16x2<0>(kw[0][g]), a1 = e2m1x2_to_f16x2<0>(kw[1][g]);
              const uint32_t a2 = e2m1x2_to_f16x2<1>(kw[0][g]), a3 = e2m1x2_to_f16x2<1>(kw[1][g]);
              const uint32_t b0 = e2m1x2_to_f16x2<2>(kw[0][g]), b1 = e2m1x2_to_f16x2<2>(kw[1][g]);
              const uint32_t b2 = e2m1x2_to_f16x2<3>(kw[0][g]), b3 = e2m1x2_to_f16x2<3>(kw[1][g]);
              float c[4];
              mma16816_zero(c, a0, a1, a2, a3, qf[g][0], qf[g][1]);
              mma16816(c, b0, b1, b2, b3, qf[g][2], qf[g][3]);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sacc[mt][j] = g == 0 ? c[j] * ks[j >> 1][g] : fmaf(c[j], ks[j >> 1][g], sacc[mt][j]);
            }
          }
        } else {
#pragma unroll
          for (int np = 0; np < 2; ++np) {  // pairs of eight-key tiles share the query fragments
            uint32_t kw[2][G], ks[2][G];    // ks: key a's scales by two blocks, then key b's
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t at = hbase + (np * 16 + h * 8) * D + k_at;
              const uint32_t sat = sbase + ((half * 4 + np * 2 + h) * 4 + t) * (4 * G);
              if constexpr (D == 128) {
                const uint4 u = lds128(at), v = lds128(sat);
                kw[h][0] = u.x, kw[h][1] = u.y, kw[h][2] = u.z, kw[h][3] = u.w;
                ks[h][0] = v.x, ks[h][1] = v.y, ks[h][2] = v.z, ks[h][3] = v.w;
              } else {
                const uint2 u = lds64(at), v = lds64(sat);
                kw[h][0] = u.x, kw[h][1] = u.y, ks[h][0] = v.x, ks[h][1] = v.y;
              }
            }
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint4 qa = lds128(q_at + (g * 2) * 512), qb = lds128(q_at + (g * 2 + 1) * 512);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float c[4];
                mma16816_zero(c, qa.x, qa.y, qa.z, qa.w, e2m1x2_to_f16x2<0>(kw[h][g]),
                              e2m1x2_to_f16x2<1>(kw[h][g]));
                mma16816(c, qb.x, qb.y, qb.z, qb.w, e2m1x2_to_f16x2<2>(kw[h][g]),
                         e2m1x2_to_f16x2<3>(kw[h][g]));
                const uint32_t wa = ks[h][g / 2], wb = ks[h][G / 2 + g / 2];
                const float sc[2] = {__uint_as_float(g % 2 ? wa & 0xFFFF0000u : wa << 16),
                                     __uint_as_float(g % 2 ? wb & 0xFFFF0000u : wb << 16)};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  sacc[np * 2 + h][j] =
                      g == 0 ? c[j] * sc[j & 1] : fmaf(c[j], sc[j & 1], sacc[np * 2 + h][j]);
              }
            }
          }
        }
        // ------------------------------------------------------------- softmax
        // Key of element j of S tile x, within the half.
        auto key_of = [&](int x, int j) {
          return NT == 1 ? x * 16 + (j >> 1) * 8 + prow : x * 8 + v_row[j & 1];
        };
        if (!clean) {
          const uint32_t hlive = half ? live.y : live.x, hnan = half ? nan.y : nan.x;
          const int sees[2] = {limit(0) - col0 - half * 32, limit(1) - col0 - half * 32};
#pragma unroll
          for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key_of(x, j);
              if ((hnan >> key) & 1) sacc[x][j] = __uint_as_float(0x7FC00000u);
              if (!((hlive >> key) & 1) || (!kSel && key >= sees[row_ix(j)]))
                sacc[x][j] = -INFINITY;
            }
        }
        if constexpr (kScores) {
          float* dst =
              p.scores + (static_cast<int64_t>(grp) * per_split + ht) * p.cols * p.score_rows;
#pragma unroll
          for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
            for (int j = 0; j < 4; j += NT == 1 ? 2 : 1) {
              const int col = col0 + half * 32 + key_of(x, j);
              if ((((half ? live.y : live.x) >> key_of(x, j)) & 1) &&
                  row_of(row_ix(j)) < p.score_rows) {
                float* at = dst + static_cast<int64_t>(col) * p.score_rows + row_of(row_ix(j));
                if constexpr (NT == 1)
                  *reinterpret_cast<float2*>(at) =
                      make_float2(sacc[x][j] * f[0], sacc[x][j + 1] * f[1]);
                else
                  *at = sacc[x][j] * f[row_ix(j)];
              }
            }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x)
#pragma unroll
          for (int j = 0; j < 4; ++j) top[row_ix(j)] = fmaxf(top[row_ix(j)], sacc[x][j]);
        if (__any_sync(0xffffffffu, top[0] > thr[0] || top[1] > thr[1])) {
          float a[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = top[i];
#pragma unroll
            for (int x = NT == 1 ? 4 : 1; x < (NT == 1 ? 32 : 4); x <<= 1)
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, x));
            a[i] = 1.f;
            if (v > thr[i]) {
              a[i] = thr[i] == -INFINITY ? 0.f : ex2((m[i] - v) * f[i]);
              m[i] = v;
              thr[i] = v + kSlack / f[i];
              l[i] *= a[i];
            }
          }
#pragma unroll
          for (int x = 0; x < kOut; ++x)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[x][j] *= a[row_ix(j)];
        }
        // P: one row tile, B fragments (row r, keys 2t, 2t+1, then + 8); two, A
        // fragments (rows r and r + 8, those keys).  Of 16 keys each.
        uint32_t pf[2][2 * NT];
#pragma unroll
        for (int x = 0; x < 2 * NT; ++x) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[j] = ex2(fmaf(sacc[x][j] - m[row_ix(j)], f[row_ix(j)], kRoom));
            l[row_ix(j)] += e[j];
          }
          if constexpr (NT == 1) {
            pf[x][0] = transpose8x8(pack_f16(e[0], e[1]));
            pf[x][1] = transpose8x8(pack_f16(e[2], e[3]));
          } else {
            pf[x / 2][(x % 2) * 2] = pack_f16(e[0], e[1]);
            pf[x / 2][(x % 2) * 2 + 1] = pack_f16(e[2], e[3]);
          }
        }
        // --------------------------------------------------------------- O += P V
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          // lo/hi: the even/odd codes of this lane's units for the key pairs
          // (2t, 2t+1) and (2t+8, 2t+9), one pair per byte.
          uint32_t lo[2][G / 2], hi[2][G / 2];
          uint32_t fac[2][G];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t va[G / 2], vb[G / 2];
            const uint32_t at = hbase + (mt * 16 + h * 8) * D;
            const uint32_t fat = fac_at + ((half * 4 + mt * 2 + h) * 4 + t) * (4 * G);
            if constexpr (D == 128) {
              const uint2 ua = lds64(at + v_at[0]), ub = lds64(at + v_at[1]);
              va[0] = ua.x, va[1] = ua.y, vb[0] = ub.x, vb[1] = ub.y;
              const uint4 u = lds128(fat);
              fac[h][0] = u.x, fac[h][1] = u.y, fac[h][2] = u.z, fac[h][3] = u.w;
            } else {
              va[0] = lds32(at + v_at[0]), vb[0] = lds32(at + v_at[1]);
              const uint2 u = lds64(fat);
              fac[h][0] = u.x, fac[h][1] = u.y;
            }
#pragma unroll
            for (int i = 0; i < G / 2; ++i) {
              lo[h][i] = low_nibbles_of(va[i], vb[i] << 4);
              hi[h][i] = low_nibbles_of(va[i] >> 4, vb[i]);
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            // v[i][h]: channel 32 g + 4 r + i of the keys 2t, 2t+1 (+ 8 h).
            uint32_t v[4][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t wl = lo[h][g / 2], wh = hi[h][g / 2];
              if (g % 2 == 0) {
                v[0][h] = e2m1x2_to_f16x2<0>(wl), v[1][h] = e2m1x2_to_f16x2<0>(wh);
                v[2][h] = e2m1x2_to_f16x2<1>(wl), v[3][h] = e2m1x2_to_f16x2<1>(wh);
              } else {
                v[0][h] = e2m1x2_to_f16x2<2>(wl), v[1][h] = e2m1x2_to_f16x2<2>(wh);
                v[2][h] = e2m1x2_to_f16x2<3>(wl), v[3][h] = e2m1x2_to_f16x2<3>(wh);
              }
            }
            if constexpr (NT == 1) {
              const uint32_t b0 = mul_f16x2(pf[mt][0], fac[0][g]);
              const uint32_t b1 = mul_f16x2(pf[mt][1], fac[1][g]);
              mma16816(o[2 * g], v[0][0], v[1][0], v[0][1], v[1][1], b0, b1);
              mma16816(o[2 * g + 1], v[2][0], v[3][0], v[2][1], v[3][1], b0, b1);
            } else {
              const uint32_t a0 = mul_f16x2(pf[mt][0], fac[0][g]);
              const uint32_t a1 = mul_f16x2(pf[mt][1], fac[0][g]);
              const uint32_t a2 = mul_f16x2(pf[mt][2], fac[1][g]);
              const uint32_t a3 = mul_f16x2(pf[mt][3], fac[1][g]);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                mma16816(o[4 * g + i], a0, a1, a2, a3, v[i][0], v[i][1]);
            }
          }
        }
      }
    }
    if (tail && lds32(next_at) > 0) {  // the tile's next window
      __syncwarp();
      continue;
    }
    if (NT == 2 && !kSel)  // the key scales written above make way for a copy
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    const uint2 c = fetch(s, tile + kStages * kWarps);
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) cols[i] = cols[i + 1];
    cols[kStages - 1] = c;
    s = s + 1 == kStages ? 0 : s + 1;
    phase ^= s == 0;
    tile += kWarps;
  }
  if (!kSel && !ok) {
    // A copy never came: report, and give the others their time to land.
    if (lane == 0) record_error(p.err, kErrTimeout);
    for (int i = 0; i < kStages; ++i) mbar_wait_bounded(&bar[i], i < s ? phase ^ 1u : phase, nullptr);
  }

  // ------------------------------------------- join the four warps, write out
  cp_async_wait<0>();
  __syncthreads();
  const uint32_t row_units_of[2] = {lds32(row_units_at + row_of(0) * 4),
                                    lds32(row_units_at + row_of(1) * 4)};
  float* so = reinterpret_cast<float*>(smem);              // [warp][row][D]
  float* sml = so + kWarps * kRows * D;                    // [warp][row][2]
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float sum = l[i];
#pragma unroll
    for (int x = NT == 1 ? 4 : 1; x < (NT == 1 ? 32 : 4); x <<= 1)
      sum += __shfl_xor_sync(0xffffffffu, sum, x);
    const int row = row_of(i);
    if (NT == 1 ? r == 0 : t == 0) {
      sml[(warp * kRows + row) * 2] = thr[i] == -INFINITY ? -INFINITY : m[i] * f[i] - kRoom;
      sml[(warp * kRows + row) * 2 + 1] = sum;
    }
    float* dst = so + (warp * kRows + row) * D;
    const float inv = inverse_sum(sum);
    float units[G];
    {
      const uint32_t w = row_units_of[i];
      units[0] = __uint_as_float(e8m0_bits<0>(w)), units[1] = __uint_as_float(e8m0_bits<1>(w));
      if constexpr (D == 128)
        units[2] = __uint_as_float(e8m0_bits<2>(w)), units[3] = __uint_as_float(e8m0_bits<3>(w));
    }
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float unit = units[g];
      if constexpr (NT == 1) {
        *reinterpret_cast<float4*>(dst + 32 * g + 4 * r) =
            make_float4(o[2 * g][i] * inv * unit, o[2 * g][2 + i] * inv * unit,
                        o[2 * g + 1][i] * inv * unit, o[2 * g + 1][2 + i] * inv * unit);
      } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)  // columns 2t and 2t + 1 of the four tiles
          *reinterpret_cast<float4*>(dst + 32 * g + 8 * t + 4 * c) =
              make_float4(o[4 * g][2 * i + c] * inv * unit, o[4 * g + 1][2 * i + c] * inv * unit,
                          o[4 * g + 2][2 * i + c] * inv * unit,
                          o[4 * g + 3][2 * i + c] * inv * unit);
      }
    }
  }
  __syncthreads();
  const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + (span.first ? 0 : 1);
  for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[(w * kRows + row) * 2]);
    const float z0 = M == -INFINITY ? 0.f : M;
    float share[kWarps], L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      share[w] = sml[(w * kRows + row) * 2 + 1] * ex2(sml[(w * kRows + row) * 2] - z0);
      L += share[w];
    }
    const float inv = inverse_sum(L);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = share[w] * inv;
      const float4 x = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + d);
      a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y);
      a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
    }
    write_row<D, kRows, kSel, kScores>(p, grp, ht, row0, nrows, row, d, span.whole(), part, M, L,
                                       a);
  }
  // The next span's copies overwrite what was read and written here.
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
}

// --------------------------------------------- more than 16 rows: tcgen05.mma
//
// Tiles of 128 columns by N = 32 or 64 query rows, two products a tile:
//   S [128 x N]  = K' q^T    K' = K / 2^k in TMEM, a key a lane: warps 0-3, one
//                            key a thread
//   O^T [D x N] += V'^T P    V' = V 2^-ref and P in shared memory, one row per
//                            column: warps 4-7 make V', both kinds P, half of
//                            the query rows each
// A key is scaled by itself: 2^k is its largest block's scale less kKeyRoom, so
// that fp16 holds its blocks exactly down to 2^-35 of that, and every key's
// thread multiplies its logits by 2^k.  The values have a reference for each
// block of 32 channels: the largest scale is 2^kTcValueRoom of it when it is set,
// V' exact down to 2^-28 of that scale, and it is raised when a scale passes
// kTcValueMost.  References of the weights likewise lag behind the rows' maxima.
// Raising any is rare and costs one more round of the tile.  As above, a later
// token's scale that would raise the values' is met in a window of its own, and
// rows that do not see it keep theirs (64 rows of 2 heads of the 64 requests
// above 341 -> 358 us; a key scaled by itself instead of by a reference made
// attend_shared_head of perf/operators.py 53 -> 51).
// 64 requests of up to 16384 keys, 64 rows on one head: 55 us for 50 MB (0.9
// TB/s), 119 us with every key's weight.  Bound by the chain of a tile's steps
// (decode, product, softmax, product) with two CTAs an SM to overlap them, which
// shared memory and TMEM allow: issue 35 %, tensor pipe 12 %, and the stalls
// spread over copies, barriers and the chain itself.
constexpr int kTcTile = 128;    // columns of a tile: one TMEM lane each
constexpr int kTcThreads = 256; // warps 0-3: keys; warps 4-7: values; both: softmax
constexpr int kTcStages = 2;
constexpr int kTcCtas = 2;      // an SM holds
constexpr int kKeyRoom = 12;    // a key's largest elements are up to 6 * 2^kKeyRoom in fp16
constexpr float kTcRoom = 7.f;    // as kRoom: the values' scales are not in the weights here
constexpr int kTcValueRoom = 5;   // V' at a new reference
constexpr float kTcValueMost = 8192.f;  // a scale over its reference: 2^(kTcValueRoom + 8)
// Reference of a row that has seen no column.  Its factor F is 1 until then, so
// that any logit is far above it.
constexpr float kUnseen = -3e38f;

// Shared memory of a CTA (1024-byte aligned).
template <int D, int N>
struct TcLayout {
  static_assert(N == 32 || N == 64, "");
  static constexpr int G = D / kMxBlock;
  static constexpr int kTileBytes = kTcTile * D;
  static constexpr int kSc = D / 16;
  static constexpr int kTiles = 0;
  static constexpr int kValues = kTiles + kTcStages * kTileBytes;  // fp16 [key][D], and at the end
  static constexpr int kValueBytes = kTcTile * D * 2;              // fp32 [row][D]
  static constexpr int kQ = kValues + kValueBytes;                 // fp16 [row][D]
  static constexpr int kP = kQ + N * D * 2;                        // fp16 [key][row]
  static constexpr int kScales = kP + kTcTile * N * 2;
  // float2 [row]: F and m, weight = 2^(F (accumulator - m))
  static constexpr int kFz = kScales + kTcStages * kTcTile * kSc;
  static constexpr int kRowF = kFz + N * 8;
  static constexpr int kLimit = kRowF + N * 4;
  static constexpr int kAlpha = kLimit + N * 4;
  static constexpr int kNan = kAlpha + N * 4;
  static constexpr int kPart = kNan + N * 4;       // [4][row] of a reduction over warps
  static constexpr int kRowUnits = kPart + 4 * N * 4;  // [row]: O's units, E8M0 by block
  static constexpr int kInvUnit = kRowUnits + N * 4;   // [4]: 1 / the values' references
  // Maxima by block of the value warps; O's factors and the new references'
  // inverses by block; a window's end.
  static constexpr int kRed = kInvUnit + 16;
  static constexpr int kBars = kRed + 25 * 4 + 4;
  static constexpr int kSlot = kBars + 8 * (kTcStages + 2);
  static constexpr int kWalk = kSlot + 16;
  static constexpr int kBytes = kWalk + 128;
  static constexpr int kTmemK = 0;                 // columns: K', S, O
  static constexpr int kTmemS = D / 2;
  static constexpr int kTmemO = kTmemS + N;
  static constexpr int kTmemCols = kTmemO + N <= 128 ? 128 : 256;
  static_assert(kTmemO + N <= kTmemCols && kTmemCols * kTcCtas <= 512, "");
};

__device__ __forceinline__ void tmem_store8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D (+)= A B^T with A [128 x 16] fp16 in TMEM, B from shared memory.
__device__ __forceinline__ void mma_ts_f16(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Shared-memory descriptor of an operand stored M- (or N-) major: rows of 2^s
// bytes along M, one row per k, swizzled over the row (mode 2: 128 bytes, 4:
// 64); `lead` bytes between row-wide blocks along M, eight k rows `row8`
// bytes apart.
__device__ __forceinline__ uint64_t mn_major_desc(uint32_t saddr, uint32_t lead, uint32_t row8,
                                                  uint32_t mode) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lead >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((row8 >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(mode) << 61;
  return d;
}

// K-major, rows of 2^s bytes (128 or 64: the swizzle), eight rows `row8` apart.
__device__ __forceinline__ uint64_t k_major_desc(uint32_t saddr, uint32_t row8, uint32_t mode) {
  return mn_major_desc(saddr, 16, row8, mode);
}

__device__ __forceinline__ uint32_t order_f32(float x) {  // order of floats as unsigned
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unorder_f32(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}

// mbar_wait_bounded for waits that are long as a rule: every try suspends the
// thread for up to a microsecond, so that a waiting warp takes no issue slots.
__device__ __forceinline__ bool mbar_wait_long(uint64_t* bar, uint32_t parity,
                                               volatile uint32_t* abort,
                                               uint64_t timeout_ns = kWaitTimeoutNs) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(1000u)
        : "memory");
    if (ok) return true;
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    if ((abort && *abort) || now - t0 > timeout_ns) return false;
  }
}

// Barrier of the four warps of one kind.
__device__ __forceinline__ void kind_barrier(int id) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(id) : "memory");
}

template <int D, int N, bool kSel, bool kScores>
__global__ void __launch_bounds__(kTcThreads, kTcCtas)
    kv4_attn_tc_kernel(const __grid_constant__ Kv4AttnParams p) {
  using Lay = TcLayout<D, N>;
  constexpr int G = Lay::G;
  constexpr int kChunks = D / 16;
  constexpr int kHalf = N / 2;  // rows of a warp's share of the softmax
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool is_v = warp >= 4;   // value warps
  const int key = tid & 127;     // of a tile: this thread's, and its TMEM lane

  const int per_split = p.Hkv * p.row_tiles;
  const int nrows = kSel ? p.heads : p.heads * p.next_n;
  const uint32_t sb = smem_u32(smem);
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + Lay::kBars);
  uint64_t* const s_done = full + kTcStages;
  uint64_t* const o_done = s_done + 1;
  volatile uint32_t* const slot = reinterpret_cast<volatile uint32_t*>(smem + Lay::kSlot);
  volatile uint32_t* const abort_flag = slot + 1;
  float2* const fz = reinterpret_cast<float2*>(smem + Lay::kFz);
  float* const row_f = reinterpret_cast<float*>(smem + Lay::kRowF);
  int* const limit = reinterpret_cast<int*>(smem + Lay::kLimit);
  float* const alpha = reinterpret_cast<float*>(smem + Lay::kAlpha);
  uint32_t* const nan_rows = reinterpret_cast<uint32_t*>(smem + Lay::kNan);
  uint32_t* const part = reinterpret_cast<uint32_t*>(smem + Lay::kPart);
  uint32_t* const row_units = reinterpret_cast<uint32_t*>(smem + Lay::kRowUnits);
  float* const inv_unit = reinterpret_cast<float*>(smem + Lay::kInvUnit);
  uint32_t* const red = reinterpret_cast<uint32_t*>(smem + Lay::kRed);
  float* const down = reinterpret_cast<float*>(red + 16);
  float* const new_inv = down + 4;
  int* const window_end = reinterpret_cast<int*>(red + 24);

  if (tid == 0) {
    for (int s = 0; s < kTcStages; ++s) mbar_init(&full[s], 1);
    mbar_init(s_done, 1);
    mbar_init(o_done, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  auto* const walk = reinterpret_cast<Walk<kSel, kTcTile>*>(smem + Lay::kWalk);
  if (warp == 0) begin_walk(walk, p);
  if (warp == 1) tmem_alloc(const_cast<uint32_t*>(slot), Lay::kTmemCols);
  launch_dependents();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *slot;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(warp & 3) << 21);  // this warp's 32 lanes
  uint32_t done = 0;   // tiles so far: their stages and phases
  uint32_t prods = 0;  // pairs of products so far: their phases
  bool ok = true;
  for (;;) {
  if (tid == 0) walk->next(p);
  if (!__syncthreads_and(ok)) break;
  const Span span = walk->span;
  if (span.g < 0) break;
  const Group& gr = span.gr;
  const int grp = span.g, ht = span.ht;
  const int head = ht / p.row_tiles;
  const int row0 = (ht % p.row_tiles) * N;
  const int c0 = span.u0 * kTcTile;
  const int c1 = min(gr.cols, span.u1 * kTcTile);
  const int tiles = (c1 - c0 + kTcTile - 1) / kTcTile;

  // ------------------------------------------------------------------ loads
  const int bs_mask = (1 << p.log_bs) - 1;
  const int32_t* table = p.block_table + static_cast<int64_t>(gr.b) * p.max_blocks;
  auto page_of = [&](int block) {
    if (block < 0 || block >= p.num_blocks) {
      record_error(p.err, kErrBadIndex);
      block = 0;
    }
    return static_cast<uint32_t>(block) * p.Hkv + head;
  };
  // Dense: lane i of warp 0 reads the page of the tile's i-th run of `rows`
  // tokens.  Selected: thread i of either kind has column i, read a tile
  // before its page; the key warps copy the keys' half of the record and its
  // scales, the value warps the values' half.
  const int rows = min(1 << p.log_bs, kTcTile);
  int pos = -1, next_pos = -1, block = 0;
  auto read_column = [&](int tile) {
    const int col = c0 + tile * kTcTile + key;
    next_pos = col < c1 ? __ldg(p.sel + static_cast<int64_t>(grp) * p.sel_k + col) : -1;
  };
  auto locate = [&](int tile) {
    if constexpr (kSel) {
      pos = next_pos;
      if (pos < -1 || pos >= gr.limit) {
        record_error(p.err, kErrBadIndex);
        pos = -1;
      }
      if (pos >= 0) block = __ldg(table + (pos >> p.log_bs));
      read_column(tile + 1);
    } else if (warp == 0) {
      pos = c0 + tile * kTcTile + lane * rows;
      if (lane * rows >= kTcTile || pos >= c1) pos = -1;
      else block = __ldg(table + (pos >> p.log_bs));
    }
  };
  // Starts the copies of the located tile into stage s; returns whether this
  // thread's column (selected) is there.  Warp w copies columns 32 (w % 4) ..,
  // what its own threads read.
  auto fetch = [&](int s, int tile) {
    bool here = false;
    if constexpr (kSel) {
      here = pos >= 0;
      const uint32_t cols = __ballot_sync(0xffffffffu, here);
      const uint32_t rec = here ? (page_of(block) << p.log_bs) + (pos & bs_mask) : 0u;
      const uint32_t base = sb + Lay::kTiles + s * Lay::kTileBytes;
      constexpr int kPer = 64 / kChunks;  // records per instruction, half of each
      const int c = lane % (kChunks / 2) + (is_v ? kChunks / 2 : 0);
      if (cols) {
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
          const int row = i * kPer + lane / (kChunks / 2);
          const uint32_t rc = __shfl_sync(0xffffffffu, rec, row);
          cp_async16(base + Layout<D, 1>::chunk_at((warp & 3) * 32 + row, c),
                     p.cache + static_cast<int64_t>(rc) * D + c * 16,
                     (cols >> row) & 1 ? 16u : 0u);
        }
        if (!is_v)
          cp_async_small<Lay::kSc>(sb + Lay::kScales + (s * kTcTile + key) * Lay::kSc,
                                   p.scales + static_cast<int64_t>(rec) * Lay::kSc,
                                   here ? Lay::kSc : 0);
      }
      cp_async_commit();
    } else if (warp == 0 && tile < tiles) {
      const int n = __popc(__ballot_sync(0xffffffffu, pos >= 0));
      if (lane == 0) mbar_arrive_expect_tx(&full[s], n * rows * (D + Lay::kSc));
      __syncwarp();
      if (pos >= 0) {
        const uint32_t page = page_of(block);
        const int at = pos & bs_mask;
        tma_load_3d(smem + Lay::kTiles + s * Lay::kTileBytes + lane * rows * D, &p.tmap, &full[s],
                    0, at, static_cast<int>(page));
        bulk_load(sb + Lay::kScales + (s * kTcTile + lane * rows) * Lay::kSc,
                  p.scales + ((static_cast<int64_t>(page) << p.log_bs) + at) * Lay::kSc,
                  rows * Lay::kSc, &full[s]);
      }
    }
    return here;
  };
  bool here[kTcStages];
  if (kSel) read_column(0);
#pragma unroll
  for (int i = 0; i < kTcStages; ++i) {
    locate(i);
    here[i] = fetch((done + i) % kTcStages, i);
  }

  // ---------------------------------------------------------------- queries
  // Row n as fp16 in the keys' order of codes, K-major, swizzled over 128
  // bytes (64 elements); D/16 threads a row, 16 elements each.
  const bool zero = p.scale_log2e == 0.f;
  const float sign = zero ? 0.f : (p.scale_log2e < 0.f ? -1.f : 1.f);
  {
    constexpr int kPer = D / 16;
    const int sub = tid % kPer;
#pragma unroll 2
    for (int n = tid / kPer; n < N; n += kTcThreads / kPer) {  // whole warps
      uint4 raw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (row0 + n < nrows) {
        const uint4* src = reinterpret_cast<const uint4*>(
            p.q + head_row<kSel>(p, grp, head, row0 + n) * D + sub * 16);
        raw[0] = __ldg(src), raw[1] = __ldg(src + 1);
      }
      uint32_t amax = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          amax = max(amax, max((w[i] << 16) & 0x7FFF0000u, w[i] & 0x7FFF0000u));
      }
#pragma unroll
      for (int x = 1; x < kPer; x <<= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, x));
      const int E = amax == 0 || amax >= 0x7F800000u
                        ? 0
                        : max(static_cast<int>(amax >> 23), 1) - 127;
      const float down = ldexpf(sign, -E);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        const int lc = sub * 2 + j;                       // elements 8 lc ..: block lc / 4
        const int kc = (lc % 4) * G + lc / 4;             // their place in a record
        const uint32_t at = sb + Lay::kQ + (kc / 8) * (N * 128) + n * 128 +
                            (((kc % 8) ^ (n & 7)) << 4);
        sts128(at, pack_f16(bf16_lo(w[0]) * down, bf16_hi(w[0]) * down),
               pack_f16(bf16_lo(w[1]) * down, bf16_hi(w[1]) * down),
               pack_f16(bf16_lo(w[2]) * down, bf16_hi(w[2]) * down),
               pack_f16(bf16_lo(w[3]) * down, bf16_hi(w[3]) * down));
      }
      if (sub == 0) {
        row_f[n] = row_factor(p, E);
        fz[n] = make_float2(1.f, kUnseen);
        limit[n] = kSel ? gr.cols
                        : gr.L - p.next_n + min((row0 + n) / p.heads, p.next_n - 1) + 1;
        nan_rows[n] = 0;
        row_units[n] = 0x01010101u;
      }
    }
    if (tid < 4) inv_unit[tid] = __uint_as_float(0x7E800000u);  // 2^126
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  const int all_see = kSel ? gr.cols : gr.L - p.next_n + 1;

  // This thread's rows of the softmax: n0 .. n0 + kHalf - 1, of its key lane.
  const int n0 = is_v ? kHalf : 0;
  float l[kHalf];  // the key lane's share of their sums
#pragma unroll
  for (int n = 0; n < kHalf; ++n) l[n] = 0.f;
  bool started = false;  // there are products of this span
  constexpr uint32_t kIdescS = mma_idesc(0, 128, N);
  constexpr uint32_t kIdescO = mma_idesc(0, 128, N) | (1u << 15) | (1u << 16);
  constexpr uint32_t kModeP = N == 32 ? 4 : 2;
  for (int tile = 0; tile < tiles; ++tile, ++done) {
    const int s = done % kTcStages;
    locate(tile + kTcStages);
    const int col0 = c0 + tile * kTcTile, col = col0 + key;
    bool there, fail = false;  // fail: a wait gave up (votes carry it to every thread)
    if constexpr (kSel) {
      cp_async_wait<kTcStages - 1>();
      // The value warps read scales that the key warps copied.
      __syncthreads();
      there = here[0];
    } else {
      if (!mbar_wait_long(&full[s], (done / kTcStages) & 1, abort_flag)) fail = true;
      there = col < c1;
    }
    // Windows of the tile's columns: one, but where a later token's value scale
    // ends it.
    for (int lo = 0;;) {
    // The last tile's logits were read, for the weights, after its last barrier:
    // what follows writes over them (S) and what they were read with (fz).
    if constexpr (kScores && !kSel) __syncthreads();
    const uint32_t base = sb + Lay::kTiles + s * Lay::kTileBytes;
    // ---------------------------------------------------------------- scales
    uint32_t kw, vw;  // of the key, and of the value
    {
      const uint32_t at = sb + Lay::kScales + (s * kTcTile + key) * Lay::kSc;
      if constexpr (D == 128) {
        const uint2 u = lds64(at);
        kw = u.x, vw = u.y;
      } else {
        const uint32_t u = lds32(at);
        kw = u & 0xFFFFu, vw = u >> 16;
      }
      if (!there || key < lo) kw = vw = 0u;
    }
    // A logit is ks times the product.  NaN scales (rare) take no part in the
    // products: a key's makes its logits NaN, a value's makes its 32 channels of
    // every row that sees the column NaN at the end.
    const bool k_nan = has_ff(kw);
    auto bits_of = [](uint32_t w, uint32_t (&f)[G]) {
      f[0] = e8m0_bits<0>(w), f[1] = e8m0_bits<1>(w);
      if constexpr (D == 128) f[2] = e8m0_bits<2>(w), f[3] = e8m0_bits<3>(w);
      if (has_ff(w))
#pragma unroll
        for (int g = 0; g < G; ++g)
          if (f[g] == 0x7F800000u) f[g] = 0u;
    };
    auto top_of = [](const uint32_t (&f)[G]) {
      uint32_t t = f[0];
#pragma unroll
      for (int g = 1; g < G; ++g) t = max(t, f[g]);
      return t;
    };
    uint32_t sf[G];
    bits_of(kw, sf);
    // 2^kKeyRoom / its inverse and it are normal numbers from here on.
    const uint32_t k_top = max(top_of(sf), static_cast<uint32_t>(kKeyRoom + 1) << 23);
    const float ks = __uint_as_float(k_top - (static_cast<uint32_t>(kKeyRoom) << 23));
    if (is_v) {
      bits_of(vw, sf);
      if (has_ff(vw))
        for (int g = 0; g < G; ++g)
          if (((vw >> (8 * g)) & 255u) == 255u)
            for (int n = 0; n < N; ++n)
              if (col < limit[n]) atomicOr(&nan_rows[n], 1u << g);
    }
    auto references = [&](float (&inv)[G]) {
#pragma unroll
      for (int g = 0; g < G; ++g) inv[g] = inv_unit[g];
    };
    // Value warps: the largest scales of the keys for which `of`, as the warps
    // put them in `red`; and the references (inverses) that go with them.
    auto put_tops = [&](bool of) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t t = __reduce_max_sync(0xffffffffu, of ? sf[g] : 0u);
        if (lane == 0) red[4 * g + (warp & 3)] = t;
      }
    };
    auto top_in = [&](int g) {
      return max(max(red[4 * g], red[4 * g + 1]), max(red[4 * g + 2], red[4 * g + 3]));
    };
    auto raised = [&](float inv, uint32_t t) {
      constexpr uint32_t kRoom = static_cast<uint32_t>(kTcValueRoom) << 23;
      return fminf(inv, __uint_as_float(0x7F000000u + kRoom - max(t, kRoom + 0x00800000u)));
    };
    // Columns that not every row sees begin new windows: those of [lo, w0) are
    // seen by the same rows, and raise references; the first one from w0 on that
    // would ends the window.
    int hi = kTcTile, w0 = kTcTile;
    if (!kSel && min(c1, col0 + kTcTile) > all_see) {
      w0 = max(all_see - col0, lo + 1);
      if (is_v) put_tops(key < w0);
      if (tid == 0) *window_end = kTcTile;
      __syncthreads();
      if (is_v) {
        float inv[G];
        references(inv);
        bool passes = false, ends = false;
#pragma unroll
        for (int g = 0; g < G; ++g)
          passes |= __uint_as_float(top_in(g)) * inv[g] > kTcValueMost;
#pragma unroll
        for (int g = 0; g < G; ++g)
          ends |= __uint_as_float(sf[g]) * (passes ? raised(inv[g], top_in(g)) : inv[g]) >
                  kTcValueMost;
        if (key >= w0 && ends) atomicMin(window_end, key);
      }
      __syncthreads();
      hi = *window_end;
      if (is_v && key >= hi)
#pragma unroll
        for (int g = 0; g < G; ++g) sf[g] = 0u;
    }
    const bool valid = there && key >= lo && key < hi;
    // V' = V over the references, one channel-major row per key.
    auto put_values = [&](const float (&inv)[G]) {
      uint32_t fac[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float x = __uint_as_float(sf[g]) * inv[g];
        fac[g] = pack_f16(x, x);
      }
#pragma unroll
      for (int c = 0; c < kChunks / 2; ++c) {
        const uint4 u = lds128(base + Layout<D, 1>::chunk_at(key, kChunks / 2 + c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int g = (2 * i) % G;  // blocks of the word's two units
          const int m8 = c * 4 + i;   // its eight channels' place
          sts128(sb + Lay::kValues + (m8 / 8) * (kTcTile * 128) + key * 128 +
                     (((m8 % 8) ^ (key & 7)) << 4),
                 mul_f16x2(e2m1x2_to_f16x2<0>(w[i]), fac[g]),
                 mul_f16x2(e2m1x2_to_f16x2<1>(w[i]), fac[g]),
                 mul_f16x2(e2m1x2_to_f16x2<2>(w[i]), fac[g + 1]),
                 mul_f16x2(e2m1x2_to_f16x2<3>(w[i]), fac[g + 1]));
        }
      }
    };
    bool again = false;  // the values' reference is too low: they are written once more
    if (!is_v) {
      // ------------------------------------------- K' = K / 2^k to TMEM, S = K' q^T
      const float inv =
          __uint_as_float(0x7F000000u + (static_cast<uint32_t>(kKeyRoom) << 23) - k_top);
      uint32_t fac[G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float x = __uint_as_float(sf[g]) * inv;
        fac[g] = k_nan ? 0x7E007E00u : pack_f16(x, x);
      }
#pragma unroll
      for (int c = 0; c < kChunks / 2; ++c) {
        const uint4 u = lds128(base + Layout<D, 1>::chunk_at(key, c));
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
        uint32_t r[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int g = i % G;
          r[4 * i] = mul_f16x2(e2m1x2_to_f16x2<0>(w[i]), fac[g]);
          r[4 * i + 1] = mul_f16x2(e2m1x2_to_f16x2<1>(w[i]), fac[g]);
          r[4 * i + 2] = mul_f16x2(e2m1x2_to_f16x2<2>(w[i]), fac[g]);
          r[4 * i + 3] = mul_f16x2(e2m1x2_to_f16x2<3>(w[i]), fac[g]);
        }
        tmem_store16(lanes + Lay::kTmemK + c * 16, r);
      }
      tmem_wait_st();
      tc_fence_before_sync();
      kind_barrier(1);
      if (tid == 0) {
        tc_fence_after_sync();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts_f16(tmem + Lay::kTmemS, tmem + Lay::kTmemK + k * 8,
                     k_major_desc(sb + Lay::kQ + (k / 4) * (N * 128) + (k % 4) * 32, 1024, 2),
                     kIdescS, k > 0);
        mma_commit(s_done);
      }
      __syncwarp();
      // P's buffer is free once the last tile's products are done.
      if (started && !mbar_wait_long(o_done, (prods - 1) & 1, abort_flag)) fail = true;
    } else {
      if (started && !mbar_wait_long(o_done, (prods - 1) & 1, abort_flag)) fail = true;
      float inv[G];
      references(inv);
#pragma unroll
      for (int g = 0; g < G; ++g)
        again |= key < w0 && __uint_as_float(sf[g]) * inv[g] > kTcValueMost;
      put_values(inv);
    }
    if (!mbar_wait_long(s_done, prods & 1, abort_flag)) fail = true;
    tc_fence_after_sync();
    // ---------------------------------------------------------------- softmax
    const bool clean = col0 + kTcTile <= min(c1, all_see) && (!kSel || valid);
    if (__any_sync(0xffffffffu, !clean)) {
      // Columns that are not there, or that a row does not see: -inf, written
      // back (their weight is zero whatever the reference).
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 8) {
        float x[8];
        tmem_load8(lanes + Lay::kTmemS + n0 + c, x);
        uint32_t r[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          r[j] = !valid || (!kSel && col >= limit[n0 + c + j]) ? 0xFF800000u : __float_as_uint(x[j]);
        tmem_store8(lanes + Lay::kTmemS + n0 + c, r);
      }
      tmem_wait_st();
    }
    float pr[kHalf];
    // Once, but for the rare cases below, which need one round more.
    for (int round = 0;; ++round) {
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < kHalf; c += 8) {
        float x[8];
        tmem_load8(lanes + Lay::kTmemS + n0 + c, x);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 f = *reinterpret_cast<const float4*>(&fz[n0 + c + j]);
          const float e0 = fmaf(fmaf(x[j], ks, -f.y), f.x, kTcRoom);
          const float e1 = fmaf(fmaf(x[j + 1], ks, -f.w), f.z, kTcRoom);
          mx = fmaxf(mx, fmaxf(e0, e1));
          pr[c + j] = ex2(e0), pr[c + j + 1] = ex2(e1);
        }
        const int ch = (n0 + c) / 8;
        const int fl = N == 32 ? (key >> 1) & 3 : key & 7;
        sts128(sb + Lay::kP + key * (2 * N) + ((ch ^ fl) << 4), pack_f16(pr[c], pr[c + 1]),
               pack_f16(pr[c + 2], pr[c + 3]), pack_f16(pr[c + 4], pr[c + 5]),
               pack_f16(pr[c + 6], pr[c + 7]));
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      tc_fence_before_sync();
      if (fail) *abort_flag = 1;
      if (!__syncthreads_or(mx > kSlack + kTcRoom || again || fail) || round == 3) break;
      // Rare.  A larger value scale than the reference allows for: a new
      // reference, the values once more, O in the new unit.  A logit far above
      // its row's reference: rows' maxima over the tile, new references, sums
      // and O by what that takes off.
      if (*abort_flag) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      if (is_v) {
        put_tops(key < w0);
        kind_barrier(2);
        float inv[G];
        references(inv);
        bool moved = false;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float up = raised(inv[g], top_in(g));
          if (tid == 128) down[g] = up / inv[g], new_inv[g] = up;
          moved |= up != inv[g];
          inv[g] = up;
        }
        if (moved) put_values(inv);
      }
      again = false;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 8) {
        float x[8];
        tmem_load8(lanes + Lay::kTmemS + n0 + c, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = n0 + c + j;
          // A NaN stays one without a reference.
          const float v = x[j] == x[j] ? x[j] * ks : -INFINITY;
          const uint32_t w = __reduce_max_sync(0xffffffffu, order_f32(v));
          if (lane == 0) part[(warp & 3) * N + n] = w;
        }
      }
      __syncthreads();
      if (tid >= 128 && tid < 128 + G) inv_unit[tid - 128] = new_inv[tid - 128];
      if (tid < N) {
        const float2 f = fz[tid];
        const float m = unorder_f32(max(max(part[tid], part[N + tid]),
                                        max(part[2 * N + tid], part[3 * N + tid])));
        float a = 1.f;
        if (m > f.y && (f.y == kUnseen || (m - f.y) * f.x > kSlack)) {
          a = f.y == kUnseen ? 0.f : ex2((f.y - m) * f.x);
          fz[tid] = make_float2(row_f[tid], m);
        }
        alpha[tid] = a;
      }
      __syncthreads();
      if (tid < N && limit[tid] > col0 + lo) {
        uint32_t units = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
          units |= (254u - (__float_as_uint(inv_unit[g]) >> 23)) << (8 * g);
        row_units[tid] = units;
      }
#pragma unroll
      for (int n = 0; n < kHalf; ++n) l[n] *= alpha[n0 + n];
      if (started) {
        const float by = down[(key / 4) % G];  // of this lane's channel
#pragma unroll 1
        for (int c = 0; c < kHalf; c += 8) {
          float o[8];
          tmem_load8(lanes + Lay::kTmemO + n0 + c, o);
          uint32_t r[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int n = n0 + c + j;
            r[j] = __float_as_uint(o[j] * alpha[n] * (limit[n] > col0 + lo ? by : 1.f));
          }
          tmem_store8(lanes + Lay::kTmemO + n0 + c, r);
        }
        tmem_wait_st();
      }
    }
    if (!ok) break;
    if constexpr (kScores) {
      float* dst =
          p.scores + ((static_cast<int64_t>(grp) * per_split + ht) * p.cols + col) * p.score_rows;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += 8) {
        float v[8];
        tmem_load8(lanes + Lay::kTmemS + n0 + c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[j] = v[j] * ks * fz[n0 + c + j].x;
        const int n = n0 + c;
        if ((kSel ? col < c1 : valid) && n < p.score_rows)
          *reinterpret_cast<float4*>(dst + n) = make_float4(v[0], v[1], v[2], v[3]);
        if ((kSel ? col < c1 : valid) && n + 4 < p.score_rows)
          *reinterpret_cast<float4*>(dst + n + 4) = make_float4(v[4], v[5], v[6], v[7]);
        __syncwarp();
      }
      tc_fence_before_sync();
    }
#pragma unroll
    for (int n = 0; n < kHalf; ++n) l[n] += pr[n];
    // --------------------------------------------------------------- O += V'^T P
    if (tid == 0) {
      tc_fence_after_sync();
#pragma unroll
      for (int k = 0; k < kTcTile / 16; ++k)
        mma_ss<false>(tmem + Lay::kTmemO,
                      mn_major_desc(sb + Lay::kValues + k * 2048, D == 128 ? kTcTile * 128 : 0,
                                    1024, 2),
                      mn_major_desc(sb + Lay::kP + k * (32 * N), 16, 16 * N, kModeP), kIdescO,
                      started || k > 0);
      mma_commit(o_done);
    }
    __syncwarp();
    started = true;
    ++prods;
    if (kSel || hi == kTcTile) break;
    lo = hi;
    }
    if (!ok) break;
    const bool h = fetch(s, tile + kTcStages);
#pragma unroll
    for (int i = 0; i + 1 < kTcStages; ++i) here[i] = here[i + 1];
    here[kTcStages - 1] = h;
  }
  if (ok && tiles > 0) {
    if (!mbar_wait_long(o_done, (prods - 1) & 1, abort_flag)) {
      record_error(p.err, kErrTimeout);
      ok = false;
    }
  } else if (!ok) {
    // A copy or a product never came: report, and give what is in flight its
    // time.
    if (tid == 0) record_error(p.err, kErrTimeout);
    if (!kSel)
      for (int i = 0; i < kTcStages; ++i)
        mbar_wait_long(&full[(done + i) % kTcStages], ((done + i) / kTcStages) & 1, nullptr);
    mbar_wait_long(s_done, prods & 1, nullptr, 1000000);
    mbar_wait_long(o_done, prods & 1, nullptr, 1000000);
  }
  cp_async_wait<0>();
  tc_fence_after_sync();

  // -------------------------------------------------------------- write out
  // O^T's lane m holds channel 32 g + 4 r + i, m = (r G + g) 4 + i.
  float* const so = reinterpret_cast<float*>(smem + Lay::kValues);  // [row][D]
  float* const lp = reinterpret_cast<float*>(part);
  if (tiles > 0) {
    // Sums over the warp's lanes: halves of the rows change sides until a lane
    // has one row (or lanes share it).
#pragma unroll
    for (int x = 1, w = kHalf / 2; x < 32; x <<= 1, w >>= 1) {
      if (w > 0) {
        const bool high = lane & x;
#pragma unroll
        for (int n = 0; n < w; ++n) {
          const float give = high ? l[n] : l[n + w], keep = high ? l[n + w] : l[n];
          l[n] = keep + __shfl_xor_sync(0xffffffffu, give, x);
        }
      } else {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], x);
      }
    }
    // Lane bit b chose between halves of width kHalf >> (b + 1).
    int mine = 0;
#pragma unroll
    for (int x = 1, w = kHalf / 2; w > 0; x <<= 1, w >>= 1) mine += lane & x ? w : 0;
    if (lane < kHalf) lp[(warp & 3) * N + n0 + mine] = l[0];
  }
  __syncthreads();
  if (tiles > 0) {
    // Every row's sum, in the place of the first part, and its inverse.
    if (tid < N) {
      lp[tid] = (lp[tid] + lp[N + tid]) + (lp[2 * N + tid] + lp[3 * N + tid]);
      alpha[tid] = inverse_sum(lp[tid]);
    }
    __syncthreads();
    const int g = (key / 4) % G, r = key / (4 * G), d = 32 * g + 4 * r + key % 4;
#pragma unroll 1
    for (int c = 0; c < kHalf; c += 8) {
      float o[8];
      tmem_load8(lanes + Lay::kTmemO + n0 + c, o);
      if (key < D) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int n = n0 + c + j;
          so[n * D + d] =
              o[j] * alpha[n] * __uint_as_float(((row_units[n] >> (8 * g)) & 255u) << 23);
        }
      }
      __syncwarp();
    }
    tc_fence_before_sync();
  }
  __syncthreads();
  const int64_t pt = static_cast<int64_t>(blockIdx.x) * 2 + (span.first ? 0 : 1);
  for (int e = tid; e < N * D / 4; e += kTcThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float L = 0.f, M = -INFINITY;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (tiles > 0) {
      L = lp[row];
      a = *reinterpret_cast<const float4*>(so + row * D + d);
      if (fz[row].y != kUnseen) M = fz[row].y * fz[row].x - kTcRoom;
      if ((nan_rows[row] >> (d / 32)) & 1)
        a.x = a.y = a.z = a.w = __uint_as_float(0x7FC00000u);
    }
    write_row<D, N, kSel, kScores>(p, grp, ht, row0, nrows, row, d, span.whole(), pt, M, L, a);
  }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Lay::kTmemCols);
  }
}

// Joins the partial results of a group, head and row tile that CTAs share: one
// CTA per kPer rows of each.  First a row's largest reference and sum, then its
// channels, four a lane, all results' loads independent of one another.  A row
// is one warp's (kPer = 8), or eight warps take every eighth result of it
// (kPer = 1): that is for so many results a row that one warp would wait for
// its loads several times over (a request of 131071 columns, 57 results: 10 ->
// 6 us).
constexpr int kJoinThreads = 256;
constexpr int kJoinMany = 16;  // results a row, on average, from which on
// (whole calls, one warp a row against eight: 131071 columns 49 and 40 us, 32768
// columns 32 and 24, 8192 columns 19.7 and 16.9; but for 512 items of 1 to 3
// results 405 and 411, 22.1 and 23.8).

template <int D, int kRows, int kPer, bool kSel, bool kScores>
__global__ void __launch_bounds__(kJoinThreads)
    kv4_join_kernel(const __grid_constant__ Kv4AttnParams p) {
  __shared__ float4 sums[kPer == 1 ? 8 : 1][D / 4];
  grid_dependency_wait();
  constexpr int kSets = kRows / kPer;
  const int item = blockIdx.x / kSets, per_split = p.Hkv * p.row_tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = kPer == 1 ? blockIdx.x % kSets : (blockIdx.x % kSets) * 8 + warp;
  const int4 sp = p.spans[item];
  const int cta = sp.x, n = sp.y;
  if (!span_noted(cta, n, sp.z, p.ctas)) return;  // a wait gave up, and that is recorded
  if (n == 1) return;                             // written by the CTA that had all of it
  const int grp = item / per_split, ht = item % per_split;
  const int row0 = (ht % p.row_tiles) * kRows;
  const int nrows = kSel ? p.heads : p.heads * p.next_n;
  if (!kScores && row0 + row >= nrows) return;
  auto part_of = [&](int i) {
    return (static_cast<int64_t>(cta + i) * 2 + (i == 0 ? sp.z : 0)) * kRows + row;
  };
  auto ml_of = [&](int i) { return *reinterpret_cast<const float2*>(p.part_ml + part_of(i) * 2); };
  float M = -INFINITY;
  for (int i = lane; i < n; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float z = M == -INFINITY ? 0.f : M;
  float L = 0.f;
  for (int i = lane; i < n; i += 32) {
    const float2 ml = ml_of(i);
    L = fmaf(ml.y, ex2(ml.x - z), L);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  const float inv = inverse_sum(L);
  constexpr int kQuads = D / 4, kHalves = 32 / kQuads, kDeal = (kPer == 1 ? 8 : 1) * kHalves;
  const int q = lane % kQuads;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = (kPer == 1 ? warp * kHalves : 0) + lane / kQuads; i < n; i += kDeal) {
    const float4 x = *reinterpret_cast<const float4*>(p.part_o + part_of(i) * D + q * 4);
    const float2 ml = ml_of(i);
    const float f = ml.y * ex2(ml.x - z) * inv;
    a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y);
    a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
  }
  if constexpr (kHalves == 2) {
    a.x += __shfl_xor_sync(0xffffffffu, a.x, 16), a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, 16), a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
  }
  if constexpr (kPer == 1) {
    if (lane < kQuads) sums[warp][q] = a;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 x = sums[w][q];
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
  }
  if (lane < kQuads)
    write_row<D, kRows, kSel, kScores>(p, grp, ht, row0, nrows, row, q * 4, true, 0, M, L, a);
}

// A column's attention weight, summed over heads and rows in one fixed order:
// w = sum exp2(S - lse).  Dense: added to key_weights.  Selected: written to
// sel_weights, and (one token a request) added to key_weights at the column's
// position.  One read of the logits, which lie in L2 where they fit: 11 us for
// 16 requests of up to 32768 columns and 32 heads, 15 us for 128 rows of 2048
// selected columns and 64 heads (67 MB, 4.5 TB/s).
template <int NT, bool kSel>
__global__ void __launch_bounds__(256) kv4_weight_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int kRows = 8 * NT;
  const int per_split = p.Hkv * p.row_tiles;
  const int per_grp = (p.cols + 255) / 256;
  const int grp = static_cast<int>(blockIdx.x / per_grp);
  const int col = static_cast<int>(blockIdx.x % per_grp) * 256 + threadIdx.x;
  const Group gr = group_of<kSel>(p, grp);
  if (static_cast<int>(blockIdx.x % per_grp) * 256 >= gr.cols) return;
  extern __shared__ float lse_s[];
  for (int i = threadIdx.x; i < per_split * kRows; i += 256)
    lse_s[i] = p.lse2[static_cast<int64_t>(grp) * per_split * kRows + i];
  __syncthreads();
  if (col >= gr.cols) return;
  float w = 0.f;
  int pos = col;
  if (kSel) {
    pos = __ldg(p.sel + static_cast<int64_t>(grp) * p.sel_k + col);
    if (pos < 0 || pos >= gr.limit) pos = -1;
  }
  if (pos >= 0) {
#pragma unroll 4
    for (int ht = 0; ht < per_split; ++ht) {
      const float4* src = reinterpret_cast<const float4*>(
          p.scores + ((static_cast<int64_t>(grp) * per_split + ht) * p.cols + col) * p.score_rows);
      const float4* z = reinterpret_cast<const float4*>(lse_s + ht * kRows);
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
        if (4 * i >= p.score_rows) break;
        const float4 x = __ldg(src + i), y = z[i];
        w += ex2(x.x - y.x) + ex2(x.y - y.y) + ex2(x.z - y.z) + ex2(x.w - y.w);
      }
    }
  }
  if (kSel) {
    if (p.sel_weights) p.sel_weights[static_cast<int64_t>(grp) * p.sel_k + col] = w;
    if (p.key_weights && p.next_n == 1 && pos >= 0)
      atomicAdd(p.key_weights + static_cast<int64_t>(gr.b) * p.ldw + pos, w);
  } else {
    p.key_weights[static_cast<int64_t>(gr.b) * p.ldw + col] += w;
  }
}

// Several tokens a request: their rows may select the same column, so one CTA
// per request adds row after row (a row's columns are distinct, so the sums
// do not depend on the order the threads run in).
__global__ void __launch_bounds__(1024)
    kv4_weight_scatter_kernel(const __grid_constant__ Kv4AttnParams p) {
  const int b = blockIdx.x;
  for (int j = 0; j < p.next_n; ++j) {
    const int64_t row = static_cast<int64_t>(b) * p.next_n + j;
    const Group gr = group_of<true>(p, static_cast<int>(row));
    for (int c = threadIdx.x; c < p.sel_k; c += blockDim.x) {
      const int pos = __ldg(p.sel + row * p.sel_k + c);
      if (pos >= 0 && pos < gr.limit)
        atomicAdd(p.key_weights + static_cast<int64_t>(b) * p.ldw + pos,
                  p.sel_weights[row * p.sel_k + c]);
    }
    __syncthreads();
  }
}

// Rows of a CTA (padded), its kernel and what that takes.
template <int D, int kRows, bool kSel, bool kScores>
cudaError_t launch_rows(const Kv4AttnParams& p, cudaStream_t s) {
  cudaError_t e;
  auto launch = [&](auto* fn, int threads, int smem) {
    static std::atomic<uint64_t> ready{0};  // devices this kernel's limit is set on
    int dev = 0;
    cudaError_t r = cudaGetDevice(&dev);
    if (r != cudaSuccess) return r;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
      r = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (r != cudaSuccess) return r;
      ready.fetch_or(bit, std::memory_order_relaxed);
    }
    fn<<<p.ctas, threads, smem, s>>>(p);
    return cudaGetLastError();
  };
  if constexpr (!uses_tc(kRows)) {
    using Lay = Layout<D, kRows / 8>;
    constexpr int kJoin = kWarps * kRows * (D + 2) * 4;
    static_assert(kJoin <= Lay::kWalk && sizeof(Walk<kSel, kTile * kWarps>) <= 128, "");
    e = launch(kv4_attn_kernel<D, kRows / 8, kSel, kScores>, kThreads, Lay::kBytes);
  } else {
    e = launch(kv4_attn_tc_kernel<D, kRows, kSel, kScores>, kTcThreads,
               TcLayout<D, kRows>::kBytes);
  }
  if (e == cudaSuccess && p.spans) {
    const int64_t items = static_cast<int64_t>(p.groups) * p.Hkv * p.row_tiles;
    const bool many = p.ctas >= items * kJoinMany;
    const unsigned grid = static_cast<unsigned>(items * (many ? kRows : kRows / 8));
    // Launched while the attention kernel still runs (it waits inside).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = many ? cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, kRows, 1, kSel, kScores>, p)
             : cudaLaunchKernelEx(&cfg, kv4_join_kernel<D, kRows, 8, kSel, kScores>, p);
  }
  if (e == cudaSuccess && kScores) {
    const int64_t grid = static_cast<int64_t>(p.groups) * ((p.cols + 255) / 256);
    const size_t sm = static_cast<size_t>(p.Hkv) * p.row_tiles * kRows * sizeof(float);
    kv4_weight_kernel<kRows / 8, kSel><<<static_cast<unsigned>(grid), 256, sm, s>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess && kSel && p.key_weights && p.next_n > 1) {
      kv4_weight_scatter_kernel<<<static_cast<unsigned>(p.groups / p.next_n), 1024, 0, s>>>(p);
      e = cudaGetLastError();
    }
  }
  return e;
}

template <int D, int kRows>
cudaError_t launch_kind(const Kv4AttnParams& p, bool scores, cudaStream_t s) {
  if (p.sel)
    return scores ? launch_rows<D, kRows, true, true>(p, s) : launch_rows<D, kRows, true, false>(p, s);
  return scores ? launch_rows<D, kRows, false, true>(p, s) : launch_rows<D, kRows, false, false>(p, s);
}

template <int D>
cudaError_t launch_d(const Kv4AttnParams& p, int rows, bool scores, cudaStream_t s) {
  switch (rows) {
    case 8: return launch_kind<D, 8>(p, scores, s);
    case 16: return launch_kind<D, 16>(p, scores, s);
    case 32: return launch_kind<D, 32>(p, scores, s);
    default: return launch_kind<D, 64>(p, scores, s);
  }
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

Kv4AttnPlan kv4_attn_plan(int B, int next_n, int Hq, int Hkv, int D, int64_t cols, bool selected,
                          bool weights) {
  Kv4AttnPlan pl = {};
  pl.heads = Hq / Hkv;
  pl.groups = selected ? static_cast<int64_t>(B) * next_n : B;
  const int rows = selected ? pl.heads : pl.heads * next_n;
  pl.rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : (rows <= 32 ? 32 : 64));
  pl.row_tiles = (rows + pl.rows - 1) / pl.rows;
  pl.tile = uses_tc(pl.rows) ? kTcTile : kTile;
  // As many CTAs as the device holds, or as there can be units of work.
  const int64_t unit = pl.unit = uses_tc(pl.rows) ? kTcTile : kTile * kWarps;
  const int64_t units = cols > 0 ? (cols + unit - 1) / unit : 1;
  const int64_t lanes = pl.groups * Hkv * pl.row_tiles;
  const int64_t places = static_cast<int64_t>(device_sm_count() > 0 ? device_sm_count() : 152) *
                         (uses_tc(pl.rows) ? kTcCtas : ctas_per_sm(selected));
  pl.ctas = static_cast<int>(units * lanes < places ? units * lanes : places);
  pl.split = units > 1;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += up256(bytes);
    return at;
  };
  const int64_t parts = pl.split ? static_cast<int64_t>(pl.ctas) * 2 * pl.rows : 0;
  pl.part_o = take(parts * D * 4);
  pl.part_ml = take(parts * 8);
  pl.spans = take(pl.split ? lanes * 16 : 0);
  // Logits kept for the weights: of the rows there are, by fours.
  pl.score_rows = pl.row_tiles > 1 ? pl.rows : (rows + 3) / 4 * 4;
  pl.scores = take(weights ? lanes * cols * pl.score_rows * 4 : 0);
  pl.lse2 = take(weights ? lanes * pl.rows * 4 : 0);
  pl.sel_weights = take(weights && selected && next_n > 1 ? pl.groups * cols * 4 : 0);
  pl.bytes = off;
  return pl;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int D, int rows, bool scores,
                                 cudaStream_t s) {
  return D == 128 ? launch_d<128>(p, rows, scores, s) : launch_d<64>(p, rows, scores, s);
}

}  // namespace dsa
