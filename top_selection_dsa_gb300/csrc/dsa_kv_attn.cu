// dsa_kv_attn.cu -- attention of chunks of new tokens over the 16-bit paged
// key/value cache (sm_103a).
//
// Request b's n tokens stand at the end of its context of L; the one at
// position p sees the keys c <= p, with a window W only c > p - W or c < sink:
//   S = scale q . k,  lse = log sum exp S,  out = sum exp(S - lse) v
//
// Rows.  The query heads of one key/value head share their keys, so a row of
// the products is a (token, head of the group) pair: 128 rows hold
// tpt = floor(128 / G) whole tokens.  Two such row tiles, A and B, run at a
// time, each with a warpgroup of its own for the softmax (a thread a row):
// while one is exponentiated, the tensor cores work on the other.
//   tall  more than tpt tokens: A and B are neighbouring rows on the same keys
//   short no more: A takes the even key tiles and B the odd ones of the same
//         rows, and their results are joined at the end, so that a single
//         token's long axis keeps both halves busy too
//
// Work.  A unit is one tile of 128 keys (tall) or two (short).  The units of
// all heads, requests and row tiles, in that order, and what each tile costs
// besides, are cut into equal runs, one for each CTA; a tile that a cut goes
// through leaves its parts (reference, sum, unscaled output, all fp32) in the
// workspace, and a second kernel joins them in their fixed order.  Lengths are
// read on the device, so a captured graph serves every step, and one long
// request fills the GPU as evenly as many short ones.
//
// Roles: warps 0-3 softmax of A, 4-7 of B, 8 TMA (queries, then a ring of key
// and value tiles fetched page by page), 9 and 10 tcgen05.mma of A and of B, 11
// watches the ring.  S = Q K^T goes to TMEM; P overwrites it as bf16 and is the A
// operand of O += P V straight from TMEM.  Weights are relative to a reference
// that is a row's maximum at first and only moves, with O rescaled, when a tile's
// weights add to more than 2^16: no tile but the first needs a maximum, and fp32
// sums lose nothing by it.  P is rounded to bf16, 2^-8 relative each (the error of
// the output's own rounding over again: 0.0017 becomes 0.0023 of its size); all
// else is fp32.
//
// What bounds it (times at 64 query heads on 8 of 128, measured copy bandwidth
// 6672 GB/s, bf16 products 1964 TFLOP/s, 1735 sustained):
//   single tokens   memory: 64 contexts of 4096 to 131072 keys, 9.6 GB, 1.31 ms,
//                   7.3 TB/s; one of 131071 90 us, 5.9 TB/s with its start and join
//   prompts         a row tile's chain of product, softmax and product, about 2900
//                   cycles a unit where the products alone take 2060 (S reads
//                   both operands from shared memory at its full rate): 8192
//                   tokens 0.77 to 0.84 ms, 1.31 to 1.42 PFLOP/s; 2048 in 65536
//                   2.9 to 3.3 ms, 1.32 to 1.5, where power caps the clock
//   in between      what starts and ends a tile, about 9000 cycles
//
// Values that a row does not see never reach it, whatever they hold: in tiles
// that are not wholly seen, infinities and NaN among the values are replaced
// by zeros before the product (0 * inf would be NaN), and rows that do see
// them have them added at the end.  A piece's first and last such key are kept, so
// that values behind a context cost no search: NaN there, 64 requests of one token
// over 1000 to 4843 keys 142 us, without 124.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kTile = 128;    // keys of a tile, rows of a row tile
constexpr int kThreads = 384;
constexpr int kTallLog = 1;   // log2 of a tall unit's cost: starts and ends count halves
// Warps: 0-7 softmax, then these (an issuer for A, one for B).
constexpr int kProducer = 8, kIssuer = 9, kWatch = 11;
constexpr int kMaxStages = 12;
// A row's weights of one tile add to no more than this, or its reference moves.
constexpr float kMostSum = 65536.f;
// A reference (times the scale) from here on is no number, and so are its row's
// results: fp32 holds it to 16 only, and at 2^31 weights relative to it, which are all
// off by the same factor then, would leave fp32's range.  (Taking the difference from
// the maximum ahead of the scale has no such bound: a prompt 806 us against 774.)
constexpr float kMostRef = 0x1p28f;
// Registers a thread: 168 at launch, shifted to the softmax (8 warps at 208 and
// 4 at 88 are the block's 64512).
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split");

__device__ __forceinline__ void launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A wait for the phase of `bar` with the given parity that gives up after
// timeout_ns or once another role did.  mbar_wait_bounded reads the clock at its
// first failure, which takes longer than most waits here.
constexpr uint64_t kDrainNs = 100000000ull;
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity,
                                             volatile uint32_t* abort,
                                             uint64_t timeout_ns = kWaitTimeoutNs) {
  uint64_t t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (__builtin_expect(mbar_try_wait(bar, parity), 1)) return true;
    if ((it & 255u) == 0) {
      if (abort && *abort) return false;
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > timeout_ns) return false;
    }
  }
}

__device__ __forceinline__ void tma_load_box3(void* dst, const CUtensorMap* map, uint64_t* bar,
                                              int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Descriptor of a [keys, 64-element columns] tile read along its elements
// (N-major B operand): 8-key atoms 1024 bytes apart, columns `column` bytes.
__device__ __forceinline__ uint64_t sw128_nmajor_desc(uint32_t saddr, uint32_t column) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(column >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// D[tmem] (+)= A[tmem] * B[smem], one elected thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
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

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// ------------------------------------------------------------------- the work

// One request: its first token, tokens and context, all inside the buffers.
struct Req {
  int b, s0, n, L;
};

__device__ __forceinline__ Req req_of(const KvAttnParams& p, int b, uint32_t* err = nullptr) {
  const int a = __ldg(p.starts + b), e = __ldg(p.starts + b + 1), L = __ldg(p.context_lens + b);
  const int cap = p.max_blocks << p.log_bs;
  Req r;
  r.b = b;
  r.s0 = min(max(a, 0), p.T);
  r.n = min(max(e, r.s0), p.T) - r.s0;
  r.L = min(max(L, 0), cap);
  if (err && (a < 0 || e < a || e > p.T || L < 0 || L > cap)) record_error(err, kErrBadIndex);
  return r;
}

__device__ __forceinline__ int tiles_of(const KvAttnParams& p, const Req& r) {
  return (r.n + 2 * p.tpt - 1) / (2 * p.tpt);
}

// One tile of rows: its tokens, their positions, and the key tiles that any of
// them sees: the first `nsink`, then those from `first` on, `keys` in all (one
// when none is seen, so that the rows' empty results are written).
struct Tile {
  int tok0, ntok, p0, nsink, first, keys, units;
  int start, log;  // cost of its start and end, and of a unit (2^log)
  bool tall;
  __device__ int last() const { return p0 + ntok - 1; }
  __device__ int cost() const { return start + (units << log); }
};

__device__ __forceinline__ Tile tile_of(const KvAttnParams& p, const Req& r, int qt) {
  Tile t;
  const int at = qt * 2 * p.tpt;
  t.ntok = min(2 * p.tpt, r.n - at);
  t.tall = t.ntok > p.tpt;
  t.tok0 = r.s0 + at;
  t.p0 = r.L - r.n + at;
  const int end = max(t.last() + 1, 0);
  t.first = p.window > 0 ? max(t.p0 - p.window + 1, 0) / kTile : 0;
  t.nsink = min((min(p.sink, end) + kTile - 1) / kTile, t.first);
  t.keys = max(t.nsink + (end + kTile - 1) / kTile - t.first, 1);
  t.units = t.tall ? t.keys : (t.keys + 1) / 2;
  t.log = t.tall ? kTallLog : p.short_log;
  t.start = t.tall ? p.tall_start : p.short_start;
  return t;
}

// What a CTA does next of a tile: `take` of its units from j on.  The producer
// writes it to shared memory, every other role reads it there.
struct Piece {
  int tok0, ntok, p0, last, nsink, first, keys, tall;  // of the tile; last: its last position
  int j, take;   // take 0: no more pieces
  int a, b;      // key tiles that A and B take
  int h, req;
  int whole;     // the piece is the whole tile
  int more;      // CTAs that go on with the tile (where the piece starts it)
  // Key tiles that every row sees whole: those below `seen`, of these in a
  // window the ones from `behind` on and the first `kept`.
  int seen, behind, kept;
  __device__ bool all_seen(int kt) const { return kt < seen && (kt >= behind || kt < kept); }
  // Whether any row sees the key.
  __device__ bool sees(const KvAttnParams& p, int key) const {
    return key <= last && (p.window == 0 || key > p0 - p.window || key < p.sink);
  }
  // The i-th key tile of group g.
  __device__ int key_of(int i, int g) const {
    const int k = tall ? j + i : 2 * (j + i) + g;
    return k < nsink ? k : first + (k - nsink);
  }
};
constexpr int kPieces = 4;    // published ahead

// A CTA's run of the work and where it stands.
struct Walk {
  Req r;
  int h, qt, at;        // at: how much of the tile's cost lies behind
  int64_t left, total;  // cost to go, and of the whole call
  __device__ void next(const KvAttnParams& p, int taken) {
    left -= taken;
    at = 0;
    if (left <= 0) return;
    if (++qt < tiles_of(p, r)) return;
    qt = 0;
    do {
      if (r.b + 1 < p.B) {
        r = req_of(p, r.b + 1);
      } else {
        ++h;
        r = req_of(p, 0);
      }
    } while (r.n == 0);
  }
};

// a * b / c, rounded down: 32-bit arithmetic where it serves (a 64-bit
// division takes some 400 cycles).
__device__ __forceinline__ int64_t muldiv(int64_t a, int64_t b, int64_t c) {
  const uint64_t ab = static_cast<uint64_t>(a * b);
  if ((ab | static_cast<uint64_t>(c)) >> 32 == 0)
    return static_cast<uint32_t>(ab) / static_cast<uint32_t>(c);
  return static_cast<int64_t>(ab / static_cast<uint64_t>(c));
}

// CTAs that share the work: each has the cost of a short tile's unit at least, so
// that none between a tile's first and last is without a unit of it.
__device__ __forceinline__ int64_t ctas_of(const KvAttnParams& p, int64_t total) {
  return min(static_cast<int64_t>(gridDim.x), total >> p.short_log);
}

// This CTA's run, for the producer's warp.  Called by all threads; `pfx` is
// B + 1 ints of scratch.
__device__ Walk find_run(const KvAttnParams& p, int* pfx) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Requests of few row tiles are summed by a thread each, others by a warp.
  constexpr int kFew = 4;
  uint32_t* err = blockIdx.x == 0 ? p.err : nullptr;
  int descends = 0;
#pragma unroll 1
  for (int b = tid; b < p.B; b += kThreads) {
    const Req r = req_of(p, b, err);
    descends |= __ldg(p.starts + b + 1) < __ldg(p.starts + b);
    const int nt = tiles_of(p, r);
    int u = -1;
    if (nt <= kFew) {
      u = 0;
#pragma unroll 1
      for (int qt = 0; qt < nt; ++qt) u += tile_of(p, r, qt).cost();
    }
    pfx[b + 1] = u;
  }
  descends = __syncthreads_or(descends);
#pragma unroll 1
  for (int b = warp; b < p.B; b += kThreads / 32) {
    if (pfx[b + 1] >= 0) continue;
    const Req r = req_of(p, b);
    const int nt = tiles_of(p, r);
    int u = 0;
#pragma unroll 1
    for (int qt = lane; qt < nt; qt += 32) u += tile_of(p, r, qt).cost();
    u = __reduce_add_sync(0xffffffffu, u);
    __syncwarp();
    if (lane == 0) pfx[b + 1] = u;
  }
  __syncthreads();
  if (warp == 0) {
    int carry = 0;
    if (lane == 0) pfx[0] = 0;
#pragma unroll 1
    for (int at = 0; at < p.B; at += 32) {
      int v = at + lane < p.B ? pfx[at + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      if (at + lane < p.B) pfx[at + lane + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  }
  __syncthreads();
  int U = pfx[p.B];
  if (descends) {
    // Requests that overlap can be more work than 32 bits count: none then.
    int64_t tokens = 0;
#pragma unroll 1
    for (int b = 0; b < p.B; ++b) tokens += req_of(p, b).n;
    if (tokens > p.T) U = 0;
  }
  const int64_t total = static_cast<int64_t>(U) * p.Hkv;
  const int64_t ctas = ctas_of(p, total);
  Walk w = {};
  w.total = total;
  if (warp == kProducer && static_cast<int64_t>(blockIdx.x) < ctas) {
    const int64_t u0 = muldiv(blockIdx.x, total, ctas);
    w.left = muldiv(blockIdx.x + 1, total, ctas) - u0;
    w.h = static_cast<int>(muldiv(u0, 1, U));
    int at = static_cast<int>(u0 - static_cast<int64_t>(w.h) * U);
    int lo = 0, hi = p.B;  // the request: pfx[lo] <= at < pfx[lo + 1]
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pfx[mid] <= at) lo = mid; else hi = mid;
    }
    at -= pfx[lo];
    w.r = req_of(p, lo);
    const int nt = tiles_of(p, w.r);
#pragma unroll 1
    for (int base = 0; base < nt; base += 32) {
      const int u = base + lane < nt ? tile_of(p, w.r, base + lane).cost() : 0;
      int incl = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, incl > at);
      if (past) {
        const int k = __ffs(past) - 1;
        w.qt = base + k;
        w.at = at - __shfl_sync(0xffffffffu, incl - u, k);
        break;
      }
      at -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // The scratch is the ring that TMA writes next.
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  return w;
}

// Two bf16 values, infinities and NaN as zeros.
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x) {
  if ((x & 0x7F80u) == 0x7F80u) x &= 0xFFFF0000u;
  if ((x & 0x7F800000u) == 0x7F800000u) x &= 0xFFFFu;
  return x;
}

// Where a role stands in the ring of stages.
template <int N>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ void step() {
    if (++st == N) {
      st = 0;
      ph ^= 1u;
    }
  }
};

// Zeroes the infinities and NaN of tile kt in shared memory (one warp).  Of those
// at keys that some row of the piece sees, *found holds the first and last key.
// (The second loop is not unrolled: by 2 its code beside the other roles' made a
// prompt of 8192 tokens 787 us instead of 766.)
template <int BYTES>
__device__ __forceinline__ void clear_nonfinite(const KvAttnParams& p, const Piece& t, int kt,
                                                uint8_t* tile, int me, int2* found) {
  constexpr int kPerHalf = kTile * 8;  // 16-byte parts of a column of 64 elements
  uint4* v = reinterpret_cast<uint4*>(tile);
  uint32_t top = 0;
#pragma unroll 8
  for (int k = me; k < BYTES / 16; k += 32) {
    const uint4 x = v[k];
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                 __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
  }
  if ((top & 0xFFFFu) < 0x7F80u && (top >> 16) < 0x7F80u) return;
  int first = 0x7FFFFFFF, last = -1;
#pragma unroll 1
  for (int k = me; k < BYTES / 16; k += 32) {
    const uint4 x = v[k];
    const uint4 y = {finite_or_zero(x.x), finite_or_zero(x.y), finite_or_zero(x.z),
                     finite_or_zero(x.w)};
    v[k] = y;
    const int key = kt * kTile + k % kPerHalf / 8;
    if (((x.x ^ y.x) | (x.y ^ y.y) | (x.z ^ y.z) | (x.w ^ y.w)) != 0 && t.sees(p, key)) {
      first = min(first, key);
      last = max(last, key);
    }
  }
  if (last >= 0) {
    atomicMin(&found->x, first);
    atomicMax(&found->y, last);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Bits below x of a 32-bit word.
__device__ __forceinline__ uint32_t below(int x) {
  return x <= 0 ? 0u : x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u;
}

// What a row sees, relative to a key tile: columns <= hi that are >= lo or < sk.
struct Sight {
  int hi, lo, sk;
  __device__ bool all() const { return hi >= kTile - 1 && (lo <= 0 || sk >= kTile); }
  __device__ uint32_t word(int k) const {
    return below(hi + 1 - 32 * k) & (~below(lo - 32 * k) | below(sk - 32 * k));
  }
  __device__ bool sees(int c) const { return c <= hi && (c >= lo || c < sk); }
};

__device__ __forceinline__ Sight sight_of(const KvAttnParams& p, int pos, int c0) {
  return {pos - c0, p.window > 0 ? pos - p.window + 1 - c0 : 0, p.sink - c0};
}

// A request's row of the block table and the pages of it that some row of a piece
// sees: up to `last`, from `first` on or below `kept`.
struct Pages {
  const int32_t* row;
  int first, last, kept;
  // The entry of page k.  One that no row sees is not looked up, as the caller may
  // have given it away: the last row's page stands in for it.
  __device__ int entry(int k) const {
    k = min(k, last);
    if (k < first && k >= kept) k = last;
    return k < 0 ? 0 : __ldg(row + k);
  }
};

__device__ __forceinline__ Pages pages_of(const KvAttnParams& p, const Piece& t) {
  return {p.block_table + static_cast<int64_t>(t.req) * p.max_blocks,
          p.window > 0 ? max(t.p0 - p.window + 1, 0) >> p.log_bs : 0, t.last >> p.log_bs,
          (p.sink + (1 << p.log_bs) - 1) >> p.log_bs};
}

// The page that an entry stands for.
__device__ __forceinline__ int page_of(const KvAttnParams& p, int entry) {
  if (static_cast<uint32_t>(entry) < static_cast<uint32_t>(p.num_blocks)) return entry;
  record_error(p.err, kErrBadIndex);
  return 0;
}

// Infinities and NaN among the values that a row sees in tiles that are not
// wholly seen, which the products left out, added to `n` elements from d0 on of
// its output as this thread stored it: bf16 at `out`, or fp32 at `part`.  They
// are at keys from `found.x` to `found.y`.
template <int D>
__device__ __noinline__ void add_nonfinite(const KvAttnParams& p, const Piece& t, int2 found,
                                           int pos, int d0, int n, uint16_t* out, float* part) {
  const Pages pages = pages_of(p, t);
#pragma unroll 1
  for (int i = 0; i < t.a + (t.tall ? 0 : t.b); ++i) {
    const int kt = t.tall ? t.key_of(i, 0) : t.key_of(i / 2, i % 2);
    if (t.all_seen(kt)) continue;
    const Sight s = sight_of(p, pos, kt * kTile);
    const int c1 = min(found.y - kt * kTile, kTile - 1);
#pragma unroll 1
    for (int c = max(found.x - kt * kTile, 0); c <= c1; ++c) {
      if (!s.sees(c)) continue;
      const int key = kt * kTile + c;
      const int64_t page = page_of(p, pages.entry(key >> p.log_bs));
      const int64_t row = ((page * p.Hkv + t.h) << p.log_bs) + (key & ((1 << p.log_bs) - 1));
#pragma unroll 1
      for (int d = d0; d < d0 + n; d += 8) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.v + row * D + d));
        auto add = [&](uint32_t pair, int at) {
          if (pair == finite_or_zero(pair)) return;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float v = __uint_as_float(k ? pair & 0xFFFF0000u : pair << 16);
            if (isfinite(v)) continue;
            if (part)
              part[at + k] += v;
            else
              out[at + k] = __bfloat16_as_ushort(__float2bfloat16_rn(
                  __uint_as_float(static_cast<uint32_t>(out[at + k]) << 16) + v));
          }
        };
        add(x.x, d);
        add(x.y, d + 2);
        add(x.z, d + 4);
        add(x.w, d + 6);
      }
    }
  }
}

// 32 bytes to one row.  A warp's lanes write 32 rows, so that a store costs the
// same whatever its width: half as many of these as of 16 bytes.
__device__ __forceinline__ void store32(void* to, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// N elements of an output row times f: bf16 to `out` (16-byte aligned, `wide`: 32),
// or fp32 to a part.
template <int N>
__device__ __forceinline__ void store_out(uint16_t* out, const float (&o)[N], float f, bool wide) {
#pragma unroll
  for (int i = 0; i < N; i += 16) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(o[i + 2 * k] * f, o[i + 2 * k + 1] * f);
      v[k] = *reinterpret_cast<const uint32_t*>(&x);
    }
    if (wide) {
      store32(out + i, v);
    } else {
      *reinterpret_cast<uint4*>(out + i) = make_uint4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<uint4*>(out + i + 8) = make_uint4(v[4], v[5], v[6], v[7]);
    }
  }
}
template <int N>
__device__ __forceinline__ void store_part(float* out, const float (&o)[N], float f) {
#pragma unroll
  for (int i = 0; i < N; i += 8) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[i + k] * f);
    store32(out + i, v);
  }
}

__device__ __forceinline__ float lse_of(float m2, float l) {
  return l == 0.f ? -INFINITY : (m2 + log2f(l)) * 0.69314718055994531f;
}

// ----------------------------------------------------------------- the kernel

template <int D>
struct AttnCfg {
  static constexpr int HALVES = D / 64;               // 128-byte columns of a row
  static constexpr int HALF_BYTES = kTile * 128;      // one column of a tile
  static constexpr int TILE_BYTES = HALVES * HALF_BYTES;
  static constexpr int NST = D == 128 ? 5 : 12;       // what shared memory has room for
  static constexpr int RING = 2 * TILE_BYTES;
  static constexpr int MISC = RING + NST * TILE_BYTES;
  static constexpr int XML = 0;                       // float2[2][128]
  static constexpr int BARS = 2048;
  static constexpr int SLOT = BARS + 8 * (2 * kMaxStages + 16 + 2 * kPieces);
  static constexpr int FOUND = SLOT + 8;
  static constexpr int PIECES = FOUND + 8 * kPieces;
  static constexpr int END = PIECES + kPieces * static_cast<int>(sizeof(Piece));
  static constexpr int SMEM = MISC + (END + 127) / 128 * 128;
  static constexpr uint32_t S_COL = 0, O_COL = 256;   // TMEM: S/P of A, of B; O of A, of B
  static constexpr uint32_t IDESC_S = mma_idesc(1u, 128, 128);
  static constexpr uint32_t IDESC_O = mma_idesc(1u, 128, D) | (1u << 16);  // V: N-major
  static_assert(SMEM <= 232448, "shared memory");
  static_assert((kMaxPagedRequests + 1) * 4 <= NST * TILE_BYTES, "prefix sums in the ring");
};

// kSmall: pages of 8 or 16 keys, whose copies one lane issues (in a kernel of
// their own: that code beside the other roles' slowed these by a tenth).
template <int D, bool kSmall>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attn_kernel(const __grid_constant__ KvAttnParams p) {
  using C = AttnCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + C::RING;
  uint8_t* misc = smem + C::MISC;
  float2* xml = reinterpret_cast<float2*>(misc + C::XML);
  uint64_t* full = reinterpret_cast<uint64_t*>(misc + C::BARS);
  uint64_t* empty = full + kMaxStages;
  uint64_t* qfull = empty + kMaxStages;
  uint64_t* qempty = qfull + 1;
  uint64_t* sfull = qempty + 1;  // [2] S is in TMEM
  uint64_t* pfull = sfull + 2;   // [2] P is in TMEM, O rescaled; the stages arrived, its turn
  uint64_t* kfirst = pfull + 2;  // [2] the first keys of a piece have arrived
  uint64_t* ofull = kfirst + 2;   // [2][2] a piece's last product is done: tall, short ones
  uint64_t* xbar = ofull + 4;    // [2] short pieces: sums exchanged; both outputs read
  uint64_t* drained = xbar + 2;
  uint64_t* told = drained + 1;       // [kPieces] a piece is published
  uint64_t* done = told + kPieces;    // [kPieces] and read by all
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + C::SLOT);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  // [kPieces] first and last key with a value that is no number (of those that
  // clear_nonfinite looked at, and some row sees): none where the first is past the last.
  int2* found = reinterpret_cast<int2*>(misc + C::FOUND);
  Piece* pieces = reinterpret_cast<Piece*>(misc + C::PIECES);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 3);  // both issuers' products, and the watcher
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 2);
    mbar_init(drained, 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 6);  // four warps' weights, the watcher, the turn
      mbar_init(&kfirst[i], 1);
      mbar_init(&ofull[i], 1);
      mbar_init(&ofull[2 + i], 1);
      mbar_init(&xbar[i], 256);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(&told[i], 1);
      mbar_init(&done[i], 11);  // every warp but the producer's
    }
    tmem_slot[1] = 0;
    fence_barrier_init();
    p.notes[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  if (warp == kIssuer) tmem_alloc(tmem_slot, 512);
  if (warp == kProducer && lane == 0) {
    tma_prefetch_desc(&p.tmap_q);
    tma_prefetch_desc(&p.tmap_k);
    tma_prefetch_desc(&p.tmap_v);
  }
  tc_fence_before_sync();
  Walk w = find_run(p, reinterpret_cast<int*>(ring));
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  bool ok = true;
  // Waits of a whole warp; after one that gave up the others pass at once.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag) ? 1 : 0);
  };
  // The next piece, and its return once nothing of it is read any more.
  Ring<kPieces> next;
  auto piece = [&]() -> const Piece& {
    wait(&told[next.st], next.ph);
    return pieces[next.st];
  };
  auto piece_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&done[next.st]);
    next.step();
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kProducer) {
      // ------------------------------------------------------------- producer
      Ring<C::NST> at;
      int queries = 0, loads = 0;
      const int per_tile = kTile >> p.log_bs;
      const int lane_tile = lane >> 3;  // which of four tiles a lane copies pages of
      // The entries of this lane's pages (lane & 7, and 8 more) of the tiles of
      // step i: the values of A's tile i, the keys of its tile i + 1, the same
      // of B (tall: A alone).  Returns whether there is such a tile.
      auto entries = [&](const Piece& t, const Pages& pages, int i, int (&e)[2]) {
        const int g = lane_tile >> 1, k = i + (lane_tile & 1);
        const bool here = k >= 0 && k < (g ? (t.tall ? 0 : t.b) : t.a) &&
                          (i >= 0 || (lane_tile & 1));
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int page = (lane & 7) + 8 * q;
          e[q] = here && page < per_tile
                     ? pages.entry((t.key_of(k, g) * kTile >> p.log_bs) + page)
                     : 0;
        }
        return here;
      };
#pragma unroll 1
      while (true) {
        wait(&done[next.st], next.ph ^ 1u);
        if (!ok) break;
        Piece t = {};
        int taken = 0;
        while (w.left > 0) {
          const Tile tile = tile_of(p, w.r, w.qt);
          const int cost = tile.cost();
          taken = static_cast<int>(min(static_cast<int64_t>(cost - w.at), w.left));
          t.j = max(w.at - tile.start, 0) >> tile.log;
          t.take = (max(w.at + taken - tile.start, 0) >> tile.log) - t.j;
          if (t.take == 0) {  // a cut in what starts the tile: the next CTA's
            w.next(p, taken);
            continue;
          }
          t.tok0 = tile.tok0;
          t.ntok = tile.ntok;
          t.p0 = tile.p0;
          t.last = tile.last();
          t.nsink = tile.nsink;
          t.first = tile.first;
          t.keys = tile.keys;
          t.tall = tile.tall;
          t.seen = max(t.p0 + 1, 0) / kTile;
          t.behind = p.window > 0 ? max(t.last - p.window + kTile, 0) / kTile : 0;
          t.kept = p.sink / kTile;
          t.a = t.take;
          t.b = t.tall || 2 * (t.j + t.take) <= t.keys ? t.take : t.take - 1;
          t.h = w.h;
          t.req = w.r.b;
          t.whole = t.j == 0 && t.take == tile.units;
          if (t.j == 0 && !t.whole) {
            // CTA c has the cost from floor(c total / ctas) on: who has the tile's end.
            const int64_t ctas = ctas_of(p, w.total);
            const int64_t end = muldiv(blockIdx.x + 1, w.total, ctas) - w.left - w.at + cost;
            t.more = static_cast<int>(muldiv(end * ctas - 1, 1, w.total)) -
                     static_cast<int>(blockIdx.x);
          }
          break;
        }
        if (lane == 0) {
          pieces[next.st] = t;
          found[next.st] = make_int2(0x7FFFFFFF, -1);
          mbar_arrive(&told[next.st]);
        }
        __syncwarp();
        next.step();
        if (t.take == 0) break;
        const bool two = !t.tall;  // A and B have key tiles of their own
        int e[2];
        const Pages pages = pages_of(p, t);
        bool here = entries(t, pages, -1, e);
        wait(qempty, (static_cast<uint32_t>(queries) & 1u) ^ 1u);
        if (!ok) break;
        if (lane == 0) {
          const int nq = two ? 1 : 2;
          mbar_arrive_expect_tx(qfull, nq * C::HALVES * p.tpt * p.G * 128);
          for (int q = 0; q < nq; ++q)
#pragma unroll
            for (int a = 0; a < C::HALVES; ++a)
              tma_load_box3(smem + q * C::TILE_BYTES + a * C::HALF_BYTES, &p.tmap_q, qfull, a * 64,
                            t.h * p.G, t.tok0 + q * p.tpt);
        }
        __syncwarp();
        ++queries;
#pragma unroll 1
        for (int i = -1; ok && i < t.a; ++i) {
          const uint32_t tiles = __ballot_sync(0xffffffffu, here);
          int row[2];
#pragma unroll
          for (int q = 0; q < 2; ++q)
            row[q] = here ? (page_of(p, e[q]) * p.Hkv + t.h) << p.log_bs : 0;
          here = entries(t, pages, i + 1, e);  // read a step ahead
          // Small pages of tile q of the step: the whole warp walks them and one
          // lane issues eight at a time.  With a lane for each page the warp took
          // 80 cycles a copy: decode over pages of 8 and 16 612 and 416 us (2.3 GB,
          // heads of 128) against 352 and 340, an 8192-token prompt over pages of
          // 16 1002 against 828.
          auto copy_small = [&](int q, int st) {
            const CUtensorMap* map = q & 1 ? &p.tmap_k : &p.tmap_v;
#pragma unroll 1
            for (int box = 0; box < per_tile; box += 8) {
              int from[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                from[k] = __shfl_sync(0xffffffffu, box ? row[1] : row[0], 8 * q + k);
              if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                  for (int a = 0; a < C::HALVES; ++a)
                    tma_load_2d(ring + st * C::TILE_BYTES + a * C::HALF_BYTES +
                                    (((box + k) * 128) << p.log_bs),
                                map, &full[st], a * 64, from[k]);
              }
              __syncwarp();
            }
          };
          // This lane's pages of its tile, a box of 64 elements each.
          auto copy = [&](int st) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const int box = (lane & 7) + 8 * q;
              if (box >= per_tile) break;
#pragma unroll
              for (int a = 0; a < C::HALVES; ++a)
                tma_load_2d(ring + st * C::TILE_BYTES + a * C::HALF_BYTES +
                                ((box * 128) << p.log_bs),
                            (lane_tile & 1) ? &p.tmap_k : &p.tmap_v, &full[st], a * 64, row[q]);
            }
          };
          if constexpr (D == 128) {
            // Tile by tile, each as soon as its stage is free.
#pragma unroll 1
            for (int q = 0; ok && q < 4; ++q) {
              if (!(tiles >> 8 * q & 1u)) continue;
              wait(&empty[at.st], at.ph ^ 1u);
              if (!ok) break;
              const int st = at.st;
              if (lane == 0) mbar_arrive_expect_tx(&full[st], C::TILE_BYTES);
              __syncwarp();
              if constexpr (kSmall)
                copy_small(q, __shfl_sync(0xffffffffu, st, 0));
              else if (lane_tile == q)
                copy(st);
              __syncwarp();
              at.step();
              ++loads;
            }
          } else {
            // Half the bytes a tile, and stages enough: a step's four tiles at
            // once, eight lanes a tile (353 us against 428 for 32 single tokens
            // of 2.3 GB, pages of 128).
            const int before = __popc(tiles & ((1u << (lane & 24)) - 1u)) >> 3;
            const bool mine = tiles >> lane & 1u;
            int st = at.st + before;
            uint32_t ph = at.ph;
            if (st >= C::NST) {
              st -= C::NST;
              ph ^= 1u;
            }
            const bool got = !mine || wait_bounded(&empty[st], ph ^ 1u, abort_flag);
            ok = __all_sync(0xffffffffu, got ? 1 : 0) != 0;
            if (!ok) break;
            if (mine && (lane & 7) == 0) mbar_arrive_expect_tx(&full[st], C::TILE_BYTES);
            __syncwarp();
            if (!kSmall && mine) copy(st);
            __syncwarp();
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              if (!(tiles >> 8 * q & 1u)) continue;
              if constexpr (kSmall) copy_small(q, __shfl_sync(0xffffffffu, at.st, 0));
              at.step();
              ++loads;
            }
          }
        }
        w.next(p, taken);
      }
      if (!ok && lane == 0) {
        // Let the copies already in flight land before the CTA retires.
        for (int i = loads > C::NST ? loads - C::NST : 0; i < loads; ++i)
          wait_bounded(&full[i % C::NST], static_cast<uint32_t>(i / C::NST) & 1u, nullptr,
                            kDrainNs);
        if (queries > 0)
          wait_bounded(qfull, static_cast<uint32_t>(queries - 1) & 1u, nullptr, kDrainNs);
      }
      __syncwarp();
    } else if (warp < kWatch) {
      // --------------------------------------------------- MMA issuers, one a group
      // The products read shared memory at its full rate, and a look at a
      // barrier then takes some 250 cycles, as long as the products still in
      // the tensor core's queue.  So there is one look a step -- pfull counts
      // the weights, the stages (from the watcher) and the turn (from the other
      // issuer) -- and it is taken while the other group's products run.  Turns
      // keep the groups half a step apart: the products of one beside the
      // softmax of the other.  The whole warp walks, so that descriptors are
      // uniform values, and one lane issues: with one lane's own values each
      // instruction waited for its operands' way into uniform registers, 107
      // cycles a product of 64.
      const int g = warp - kIssuer;
      Ring<C::NST> at;
      uint32_t pn = 0, qn = 0, kn = 0;  // parities of pfull, qfull and kfirst
      uint32_t an = 0;                  // B: of A's pfull
      bool any = false;                 // B: whether that had a phase
      const uint32_t q_addr = smem_u32(smem), r_addr = smem_u32(ring);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t st = tm + C::S_COL + g * 128, ot = tm + C::O_COL + g * D;
      auto take_stage = [&]() {
        const int k = at.st;
        at.step();
        return __shfl_sync(0xffffffffu, k, 0);
      };
#pragma unroll 1
      while (true) {
        const Piece t = piece();
        if (!ok || t.take == 0) break;
        const bool tall = t.tall;
        const int n = g ? t.b : t.a, other = g ? t.a : t.b;  // key tiles of both groups
        const uint32_t qa = q_addr + (tall ? g : 0) * C::TILE_BYTES;
        wait(qfull, qn);
        qn ^= 1u;
        // Step i: the product with the values of the group's tile i, then S of
        // its next tile; before the first only S.  The stages of the other
        // group's steps are passed by (tall: both use the same).
#pragma unroll 1
        for (int i = n > 0 ? -1 : 0; ok && i < n; ++i) {
          const bool more = i + 1 < n;
          int vs = 0, ks = 0;
          if (tall || g == 0) {
            if (i >= 0) vs = take_stage();
            if (more) ks = take_stage();
            if (!tall && i < other) {
              if (i >= 0) at.step();
              if (i + 1 < other) at.step();
            }
          } else {
            if (i >= 0) at.step();
            if (i + 1 < other) at.step();
            if (i >= 0) vs = take_stage();
            if (more) ks = take_stage();
          }
          if (i < 0) {
            wait(&kfirst[g], kn);
            kn ^= 1u;
          } else {
            wait(&pfull[g], pn);
            pn ^= 1u;
          }
          if (!ok) break;
          tc_fence_after_sync();
          const uint32_t va = r_addr + vs * C::TILE_BYTES, ka = r_addr + ks * C::TILE_BYTES;
          // S overwrites P: the tensor core takes one thread's products in
          // their order.
          auto s_mma = [&](int from, int to) {
#pragma unroll
            for (int k = from; k < to; ++k) {
              const uint32_t off = (k / 4) * C::HALF_BYTES + (k % 4) * 32;
              mma_ss<false>(st, sw128_kmajor_desc(qa + off), sw128_kmajor_desc(ka + off),
                            C::IDESC_S, k > 0 ? 1u : 0u);
            }
          };
          if (elect_one()) {
            if (i >= 0) {
#pragma unroll
              for (int k = 0; k < kTile / 16; ++k)
                mma_ts(ot, st + k * 8, sw128_nmajor_desc(va + k * 2048, C::HALF_BYTES), C::IDESC_O,
                       k > 0 || i > 0 ? 1u : 0u);
              mma_commit(&empty[vs]);
              if (!tall) mma_commit(&empty[vs]);  // for the other issuer
              if (!more) mma_commit(&ofull[tall ? g : 2 + g]);
            }
            if (more) s_mma(0, D / 32);
            // The turn of B's same step, or of A's next.
            if (g == 0 && i >= 0 && i < other) mbar_arrive(&pfull[1]);
            if (g == 1 && i >= 0 && i + 1 < other) mbar_arrive(&pfull[0]);
            if (more) {
              s_mma(D / 32, D / 16);
              mma_commit(&sfull[g]);
              mma_commit(&empty[ks]);
              if (!tall) mma_commit(&empty[ks]);
              if (i + 2 == n) mma_commit(qempty);  // the queries' last use
            }
          }
          __syncwarp();
          if (g == 1 && i < 0) {
            // A's first turn; its last step of the piece before is awaited, that
            // this is not counted there.
            if (any) wait(&pfull[0], an ^ 1u);
            if (ok && elect_one()) mbar_arrive(&pfull[0]);
            __syncwarp();
          }
        }
        if (!ok) break;
        if (g == 1) {
          if (n == 0) {
            // No step of its own: the stages passed by, the queries given back,
            // A's one turn.
            at.step();
            at.step();
            if (any) wait(&pfull[0], an ^ 1u);
            if (ok && elect_one()) {
              mbar_arrive(qempty);
              mbar_arrive(&pfull[0]);
            }
            __syncwarp();
          } else if (!tall && n < other) {
            at.step();  // A's last values
          }
          any = true;
          an ^= other & 1u;
        }
        piece_done();
      }
      // All products of this CTA are done before its TMEM is given back.
      if (elect_one()) mma_commit(drained);
      __syncwarp();
      wait_bounded(drained, 0, nullptr, kDrainNs);
      __syncwarp();
    } else {
      // -------------------------------------------------------------- watcher
      // It sees every stage arrive, clears what some row must not see of the
      // values in it, and tells the issuers when a step has its stages.
      Ring<C::NST> at;
      uint32_t pn = 0, any = 0;  // a bit a group: parity of pfull's phase to come, was there one
      // A stage is given back beside the products' own return.
      auto pass = [&](const Piece& t, int kt, bool look) {
        wait(&full[at.st], at.ph);
        if (ok && look)
          clear_nonfinite<C::TILE_BYTES>(p, t, kt, ring + at.st * C::TILE_BYTES, lane,
                                         &found[next.st]);
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(&empty[at.st]);
        at.step();
      };
#pragma unroll 1
      while (true) {
        const Piece t = piece();
        if (!ok || t.take == 0) break;
        const bool tall = t.tall;
#pragma unroll 1
        for (int s = -2; ok && s < 2 * t.a; ++s) {
          const int i = s >> 1, g = s & 1, n = g ? t.b : t.a;
          if (i >= n) continue;
          if (!tall || g == 0) {
            const int kt = i >= 0 ? t.key_of(i, g) : 0;
            if (i >= 0) pass(t, kt, !t.all_seen(kt));
            if (i + 1 < n) pass(t, 0, false);
          }
          // An arrival ahead of the step before would be counted with it.
          if (any >> g & 1u) wait(&pfull[g], (pn >> g & 1u) ^ 1u);
          if (i < 0) {
            if (ok && n > 0 && lane == 0) mbar_arrive(&kfirst[g]);
            continue;
          }
          if (ok && lane == 0) mbar_arrive(&pfull[g]);
          any |= 1u << g;
          pn ^= 1u << g;
        }
        piece_done();
      }
    }
  } else {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int g = warp >> 2, row = tid & 127;
    const int row_tok = row / p.G, row_head = row - row_tok * p.G;
    const uint32_t quarter = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes, << 16
    const uint32_t s_addr = tmem + quarter + C::S_COL + g * 128;
    const uint32_t o_addr = tmem + quarter + C::O_COL;
    const float sc = p.scale_log2e;
    uint32_t sn = 0, xn = 0, on = 0;  // parities of the phases waited for (ofull: a bit each)
#pragma unroll 1
    while (true) {
      const Piece& t = piece();
      if (!ok || t.take == 0) break;
      const int tok = row_tok + (t.tall ? g * p.tpt : 0);
      const bool mine = row_tok < p.tpt && tok < t.ntok;
      const bool busy = __any_sync(0xffffffffu, mine);
      const int pos = t.p0 + tok;
      float m = -INFINITY, l = 0.f;
      const int steps = g ? t.b : t.a;
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        const Sight see = sight_of(p, pos, t.key_of(i, g) * kTile);
        const bool masked = __any_sync(0xffffffffu, mine && !see.all());
        wait(&sfull[g], sn);
        sn ^= 1u;
        if (!ok) break;
        if (busy) {
          tc_fence_after_sync();
          // Weights by the present reference.  S stays in TMEM until they serve,
          // so that registers hold it only up to its exponential: kept beside
          // them for a second try, it took the exponentials their overlap (1250
          // cycles a tile, against 720).
          uint32_t pk[4][16];
          float add = 0.f;
          bool fresh = i == 0;
#pragma unroll 1
          while (true) {
            uint32_t s[4][32];
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_ld32_async(s_addr + 32 * k, s[k]);
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_wait_ld(s[k]);
            if (__builtin_expect(masked, 0)) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t word = see.word(k);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  if (!(word >> c & 1u)) s[k][c] = 0xFF800000u;
              }
            }
            if (__builtin_expect(fresh, 0)) {
              float mx[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                mx[k] = __uint_as_float(s[k / 2][k % 2 * 16]);
#pragma unroll
                for (int c = 1; c < 16; ++c)
                  mx[k] = fmaxf(mx[k], __uint_as_float(s[k / 2][k % 2 * 16 + c]));
              }
              const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                                      fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7])));
              const float mn = fmaxf(m, top);
              const float f = m == -INFINITY ? 0.f : ex2((m - mn) * sc);
              m = fabsf(mn * sc) < kMostRef || mn == -INFINITY ? mn : NAN;
              l *= f;
              if (i > 0) {
#pragma unroll 1
                for (int d = 0; d < D; d += 16) {
                  float o[16];
                  tmem_load16(o_addr + g * D + d, o);
                  uint32_t r[16];
#pragma unroll
                  for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(o[k] * f);
                  tmem_st16(o_addr + g * D + d, r);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : -m * sc;
            const float2 ref2 = make_float2(ref, ref), sc2 = make_float2(sc, sc);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                const float2 x = __ffma2_rn(
                    make_float2(__uint_as_float(s[k][c]), __uint_as_float(s[k][c + 1])), sc2, ref2);
                const float2 e = make_float2(ex2(x.x), ex2(x.y));
                sum[c >> 1 & 1] = __fadd2_rn(sum[c >> 1 & 1], e);
                const __nv_bfloat162 y = __floats2bfloat162_rn(e.x, e.y);
                pk[k][c >> 1] = *reinterpret_cast<const uint32_t*>(&y);
              }
            }
            const float2 both = __fadd2_rn(sum[0], sum[1]);
            add = both.x + both.y;
            // A new reference: the first tile, rows that have seen nothing yet,
            // and where the old one lets the weights grow (or they are NaN).
            if (fresh ||
                !__any_sync(0xffffffffu, mine && (m == -INFINITY || !(add <= kMostSum))))
              break;
            fresh = true;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_st16(s_addr + 16 * k, pk[k]);
          l += add;
          tmem_wait_st();
          tc_fence_before_sync();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[g]);
      }
      // The piece's outputs.
      // Tall pieces have barriers of their own, one group waiting on each, so
      // that A need not wait for B's end and no phase goes unseen.
      auto wait_o = [&](int k) {
        wait(&ofull[k], on >> k & 1u);
        on ^= 1u << k;
      };
      if (t.tall) {
        wait_o(g);
      } else {
        wait_o(2);
        if (t.b > 0) wait_o(3);
      }
      if (!ok) break;
      tc_fence_after_sync();
      const bool whole = t.whole;
      const int64_t at = static_cast<int64_t>(t.tok0 + tok) * p.Hq + t.h * p.G + row_head;
      // Slot 1 starts a tile, slot 0 goes on with one that an earlier CTA started.
      const int64_t part = static_cast<int64_t>(2 * blockIdx.x + (t.j == 0 ? 1 : 0)) * p.slot_rows +
                           (t.tall ? g * kTile : 0) + row;
      // Tall: this group's rows.  Short: A and B hold two halves of the same
      // rows' keys, and each group joins one half of the elements.
      float top = m * sc, sum = l, fa = 1.f, fb = 0.f;
      int d0 = 0, d1 = D;
      uint32_t from = o_addr + g * D;
      if (!t.tall) {
        xml[g * 128 + row] = make_float2(top, l);
        mbar_arrive(&xbar[0]);
        wait(&xbar[0], xn);
        if (!ok) break;
        const float2 a = xml[row], b = t.b > 0 ? xml[128 + row] : make_float2(-INFINITY, 0.f);
        top = fmaxf(a.x, b.x);
        fa = a.x == -INFINITY ? 0.f : ex2(a.x - top);
        fb = b.x == -INFINITY ? 0.f : ex2(b.x - top);
        sum = a.y * fa + b.y * fb;
        d0 = g * (D / 2);
        d1 = d0 + D / 2;
        from = o_addr;
      }
      const float f = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
      const bool second = !t.tall && t.b > 0;
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
      if (busy) {
#pragma unroll 1
        for (int d = d0; d < d1; d += 32) {
          float o[32];
          tmem_load32(from + d, o);
          if (second) {
            float o2[32];
            tmem_load32(o_addr + D + d, o2);
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = fmaf(o2[k], fb, o[k] * fa);
          }
          if (mine) {
            if (whole)
              store_out(p.out + at * D + d, o, second ? f : f * fa, wide);
            else
              store_part(p.part_o + part * D + d, o, second ? 1.f : fa);
          }
          __syncwarp();
        }
      }
      if (mine) {
        const int2 keys = found[next.st];
        if (__builtin_expect(keys.x <= keys.y, 0))
          add_nonfinite<D>(p, t, keys, pos, d0, d1 - d0, p.out + at * D,
                           whole ? nullptr : p.part_o + part * D);
        if (d0 == 0) {
          if (!whole)
            p.part_ml[part] = make_float2(top, sum);
          else if (p.lse)
            p.lse[at] = lse_of(top, sum);
        }
      }
      __syncwarp();
      if (!whole && t.j == 0 && tid == 0)
        p.notes[blockIdx.x] = make_int4(t.tok0, t.ntok, t.h, t.more);
      if (!t.tall) {
        tc_fence_before_sync();
        mbar_arrive(&xbar[1]);
        wait(&xbar[1], xn);
        xn ^= 1u;
        tc_fence_after_sync();
      }
      if (!ok) break;
      piece_done();
    }
  }
  if (!ok) {
    *abort_flag = 1;
    record_error(p.err, kErrTimeout);
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kIssuer) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------- the join

constexpr int kJoinWarps = 8;

// A part's value times its weight: what is not finite shows where fp32 holds the
// weight as zero too, as it does where a tile is not cut.
__device__ __forceinline__ float weighted(float v, float f) {
  return f != 0.f ? v * f : isfinite(v) ? 0.f : v;
}

// The parts of each cut tile, a warp a row.  CTA blockIdx.x started the tile
// (its slot 1), the next ones went on with it (their slots 0).
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv_join_kernel(
    const __grid_constant__ KvAttnParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cta = blockIdx.x;
  const int4 note = p.notes[cta];  // first token, tokens, head, CTAs that went on
  const int rows = note.y * p.G, more = note.w;
  constexpr int N = D / 32;
  for (int i = blockIdx.y * kJoinWarps + warp; i < rows; i += gridDim.y * kJoinWarps) {
    const int tok = i / p.G, g = i - tok * p.G;
    const int row = tok / p.tpt * kTile + (tok % p.tpt) * p.G + g;
    auto part = [&](int k) {
      return static_cast<int64_t>(k == 0 ? 2 * cta + 1 : 2 * (cta + k)) * p.slot_rows + row;
    };
    // Parts k0 .. k0 + K - 1, one running maximum: their sums and values are
    // read together.
    float top = -INFINITY, sum = 0.f, acc[N] = {};
    auto add = [&](auto count, int k0) {
      constexpr int K = decltype(count)::value;
      float2 ml[K];
      float v[K][N];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int q = 0; q < N; ++q) v[k][q] = 0.f;
        if (K > 2 && k0 + k > more) continue;
        const int64_t at = part(k0 + k);
        ml[k] = p.part_ml[at];
        if constexpr (N == 4) {
          const float4 x = reinterpret_cast<const float4*>(p.part_o + at * D)[lane];
          v[k][0] = x.x; v[k][1] = x.y; v[k][2] = x.z; v[k][3] = x.w;
        } else {
          const float2 x = reinterpret_cast<const float2*>(p.part_o + at * D)[lane];
          v[k][0] = x.x; v[k][1] = x.y;
        }
      }
      const float was = top;
#pragma unroll
      for (int k = 0; k < K; ++k) top = fmaxf(top, ml[k].x);
      const float keep = was == -INFINITY ? 0.f : ex2(was - top);
      sum *= keep;
#pragma unroll
      for (int q = 0; q < N; ++q) acc[q] = weighted(acc[q], keep);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float f = ml[k].x == -INFINITY ? 0.f : ex2(ml[k].x - top);
        sum = fmaf(ml[k].y, f, sum);
#pragma unroll
        for (int q = 0; q < N; ++q)
          acc[q] = f == 0.f ? acc[q] + weighted(v[k][q], f) : fmaf(v[k][q], f, acc[q]);
      }
    };
    if (more == 1) {  // most rows of prompts
      add(std::integral_constant<int, 2>(), 0);
    } else {
#pragma unroll 1
      for (int k0 = 0; k0 <= more; k0 += 4) add(std::integral_constant<int, 4>(), k0);
    }
    const float f = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t at = static_cast<int64_t>(note.x + tok) * p.Hq + note.z * p.G + g;
    uint32_t v[N / 2];
#pragma unroll
    for (int q = 0; q < N / 2; ++q) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[2 * q] * f, acc[2 * q + 1] * f);
      v[q] = *reinterpret_cast<const uint32_t*>(&x);
    }
    if constexpr (N == 4)
      reinterpret_cast<uint2*>(p.out + at * D)[lane] = make_uint2(v[0], v[1]);
    else
      reinterpret_cast<uint32_t*>(p.out + at * D)[lane] = v[0];
    if (lane == 0 && p.lse) p.lse[at] = lse_of(top, sum);
  }
}

template <int D, bool kSmall>
cudaError_t launch_d(const KvAttnParams& p, cudaStream_t s) {
  using C = AttnCfg<D>;
  // The attribute is set once a device (devices past 64: every time).
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv_attn_kernel<D, kSmall>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  kv_attn_kernel<D, kSmall><<<p.ctas, kThreads, C::SMEM, s>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // A tile of one unit is never cut.
  const int64_t keys = ((static_cast<int64_t>(p.max_blocks) << p.log_bs) + kTile - 1) / kTile;
  if ((p.slot_rows > kTile ? keys : (keys + 1) / 2) <= 1) return cudaSuccess;
  // Launched while the attention kernel still runs (it waits inside).
  const int64_t rows = static_cast<int64_t>(p.T) * p.G;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.ctas, ((rows < p.slot_rows ? static_cast<int>(rows) : p.slot_rows) +
                              kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D>, p);
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

KvAttnPlan kv_attn_plan(int T, int G, int D) {
  KvAttnPlan pl = {};
  pl.tpt = kTile / G;
  pl.ctas = device_sm_count() > 0 ? device_sm_count() : 1;
  pl.slot_rows = T > pl.tpt ? 2 * kTile : kTile;
  const int64_t rows = static_cast<int64_t>(pl.ctas) * 2 * pl.slot_rows;
  pl.part_ml = up256(static_cast<int64_t>(pl.ctas) * 16);
  pl.part_o = pl.part_ml + up256(rows * 8);
  pl.bytes = pl.part_o + up256(rows * D * 4);
  return pl;
}

int64_t kv_attn_units(int T, int B, int G, int64_t max_ctx) {
  // (the cost of a row tile is at most twice its tiles of keys and 5)
  return (static_cast<int64_t>(T) / (2 * (kTile / G)) + B) *
         (((max_ctx + kTile - 1) / kTile + 3) << kTallLog);
}

cudaError_t launch_kv_attention(const KvAttnParams& p, int D, cudaStream_t s) {
  if (p.log_bs < 5) return D == 64 ? launch_d<64, true>(p, s) : launch_d<128, true>(p, s);
  return D == 64 ? launch_d<64, false>(p, s) : launch_d<128, false>(p, s);
}

}  // namespace dsa
