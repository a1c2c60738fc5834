// dsa_kv4_attn.cu -- decode attention over the paged 4-bit key/value cache
// (layout in dsa_kv4.cuh), over every key of a request or over the columns an
// indexer selected.
//
//   S[n,c] = scale * q[n] . K[c]       for the columns c that row n sees
//   lse[n] = log sum_c exp S[n,c]      out[n] = sum_c exp(S[n,c] - lse[n]) V[c]
//
// One warp walks tiles of 64 columns of one key/value head for up to 16 query
// rows (the rows of the head's group, all tokens of the request): cp.async
// brings the tile's records and scales into the warp's own two-stage ring,
// and everything after that stays in registers.
//   S^T = K q^T   mma m16n8k16 with the keys as the 16-row operand: its fp16
//                 elements are the E2M1 codes' values themselves (exact); the
//                 four blocks of 32 elements accumulate apart and are summed
//                 in fp32 with their power-of-two scales.  q is divided by a
//                 power of two per row so that its largest element is in
//                 [1, 2): bf16's eight bits fit fp16 exactly, and elements
//                 below 2^-24 of the row's largest vanish.
//   softmax       one pass: running maximum m and sum l per row (base 2, in
//                 fp32), the accumulated output rescaled when m rises.
//   O^T += V^T P  keys as the contraction: V's elements again the codes'
//                 values, one 16-row tile per half block of channels, and the
//                 value scales multiplied into P (fp16) once per block of 32
//                 channels, relative to the largest scale met so far, 2^x:
//                 P 2^(e - x) <= 1, and terms below 2^-24 of that vanish.
// Rounding P to fp16 costs 2^-12 of each term (the output's bf16 rounding is
// 2^-9); l sums the unrounded weights.
//
// Rows of the m16 operand are permuted within each group of eight (odd rows
// exchange halves, row i holds key i ^ 4): with the records' 16-byte chunks
// XOR-swizzled by the key's index in its group of eight, the 16-byte key
// loads and the 8-byte value loads are then both free of bank conflicts.
//
// The columns of a request are cut into chunks, one CTA (four warps, tiles
// dealt round) per chunk, head and 16 rows; a CTA that covers all of a row's
// columns writes the result, otherwise partial sums that a second kernel
// joins.
#include <math.h>

#include "dsa_internal.h"
#include "dsa_kv4.cuh"

namespace dsa {
namespace {

constexpr int kTile = kKv4Tile;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kCtasPerSm = 3;   // registers (168 a thread) and shared memory

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
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
// Non-zero when a byte of w is 255.
__device__ __forceinline__ uint32_t has_ff(uint32_t w) {
  return (~w - 0x01010101u) & w & 0x80808080u;
}

// Shared memory of a CTA: all warps' rings of tiles first (1024-byte aligned,
// the swizzle is a function of the address; there is no static shared memory,
// so the block begins so aligned), then by warp the tiles' scales, what the
// tile in work needs of them -- 2^e of every key's blocks (fp32), and the
// value factors as fp16 pairs in the order of P's fragments -- and the ring's
// barriers.
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
  static constexpr int kWarpRest = (kBarriers + 8 * kStages + 15) / 16 * 16;
  // Then, with two row tiles, the query fragments and their factors.
  static constexpr int kQueries = kWarps * (kWarpTiles + kWarpRest);
  static constexpr int kFactorF = kQueries + (NT > 1 ? NT * G * 32 * 16 : 0);
  static constexpr int kBytes = kFactorF + (NT > 1 ? NT * 8 * 4 : 0);
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

template <bool kSel>
__device__ __forceinline__ Group group_of(const Kv4AttnParams& p, int g, bool report) {
  Group r;
  r.b = kSel ? g / p.next_n : g;
  const int cap = p.max_blocks << p.log_bs;
  const int raw = __ldg(p.context_lens + r.b);
  if (report && (raw < 0 || raw > cap)) record_error(p.err, kErrBadIndex);
  r.L = raw < 0 ? 0 : (raw > cap ? cap : raw);
  r.cols = kSel ? p.sel_k : r.L;
  r.limit = kSel ? max(r.L - p.next_n + (g - r.b * p.next_n) + 1, 0) : r.L;
  return r;
}

// Where query row n (of a group's rows for one key/value head) lies: the row
// of q, out and lse as [rows, Hq].
template <bool kSel>
__device__ __forceinline__ int64_t head_row(const Kv4AttnParams& p, int g, int head, int n) {
  const int j = kSel ? 0 : n / p.heads;
  const int64_t row = kSel ? g : static_cast<int64_t>(g) * p.next_n + j;
  return row * p.Hq + head * p.heads + (n - j * p.heads);
}

template <int D, int NT, bool kSel, bool kScores>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    kv4_attn_kernel(const __grid_constant__ Kv4AttnParams p) {
  using Lay = Layout<D, NT>;
  constexpr int G = Lay::G;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane >> 2, t = lane & 3;

  // head and row tile fastest: neighbouring CTAs read neighbouring heads of
  // the same pages.
  const int per_split = p.Hkv * p.row_tiles;
  int64_t id = blockIdx.x;
  const int ht = static_cast<int>(id % per_split);
  id /= per_split;
  const int split = static_cast<int>(id % p.nsplit);
  const int grp = static_cast<int>(id / p.nsplit);
  const int head = ht / p.row_tiles;
  const int row0 = (ht % p.row_tiles) * kRows;
  const int nrows = kSel ? p.heads : p.heads * p.next_n;

  const Group gr = group_of<kSel>(p, grp, split == 0 && ht == 0 && threadIdx.x == 0);
  const int c0 = split * p.chunk;
  if (c0 >= gr.cols && split > 0) return;
  const int c1 = min(gr.cols, c0 + p.chunk);
  const bool whole = gr.cols <= p.chunk;

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
  int pos[2] = {-1, -1}, next_pos[2] = {-1, -1}, block[2] = {0, 0};
  auto read_columns = [&](int tile) {  // selected: this lane's positions of `tile`
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = c0 + tile * kTile + lane + 32 * i;
      next_pos[i] = col < c1 ? __ldg(p.sel + static_cast<int64_t>(grp) * p.sel_k + col) : -1;
    }
  };
  auto locate = [&](int tile) {
    if constexpr (kSel) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pos[i] = next_pos[i];
        if (pos[i] < -1 || pos[i] >= gr.limit) {
          record_error(p.err, kErrBadIndex);
          pos[i] = -1;
        }
        if (pos[i] >= 0) block[i] = __ldg(table + (pos[i] >> p.log_bs));
      }
      read_columns(tile + kWarps);
    } else {
      pos[0] = c0 + tile * kTile + lane * rows;
      if (lane * rows >= kTile || pos[0] >= c1) pos[0] = -1;
      else block[0] = __ldg(table + (pos[0] >> p.log_bs));
    }
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
  if (kSel) read_columns(warp);
#pragma unroll
  for (int s = 0; s < kStages; ++s) {
    locate(warp + s * kWarps);
    cols[s] = fetch(s, warp + s * kWarps);
  }

  // ---------------------------------------------------------------- queries
  // B fragments: lane (r, t) holds row r's elements 32 g + 8 t .. + 7, times
  // the softmax scale's sign.
  // One row tile: every warp keeps the fragments in registers.  Two: warps 0
  // and 1 prepare one each, and all read them from shared memory.
  uint32_t qf[NT == 1 ? G : 1][4];
  float f[NT][2];    // base-2 logit = f * accumulator (f > 0), rows 2t and 2t + 1
  const bool zero = p.scale_log2e == 0.f;
  const float sign = zero ? 0.f : (p.scale_log2e < 0.f ? -1.f : 1.f);
  const uint32_t q_at = smem_u32(smem) + Lay::kQueries + lane * 16;
  float* const f_s = reinterpret_cast<float*>(smem + Lay::kFactorF);
  if (NT == 1 || warp < NT) {
    const int nt = NT == 1 ? 0 : warp;
    const int n = row0 + nt * 8 + r;
    uint4 raw[G];
    uint32_t amax = 0;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      raw[g] = make_uint4(0u, 0u, 0u, 0u);
      if (n < nrows)
        raw[g] = __ldg(reinterpret_cast<const uint4*>(
            p.q + head_row<kSel>(p, grp, head, n) * D + g * 32 + t * 8));
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
        sts128(q_at + (nt * G + g) * 512, h[0], h[1], h[2], h[3]);
      }
    }
    const float fr = zero ? 1.f : ldexpf(fabsf(p.scale_log2e), E);
    if constexpr (NT == 1) {
#pragma unroll
      for (int i = 0; i < 2; ++i) f[0][i] = __shfl_sync(0xffffffffu, fr, (2 * t + i) * 4);
    } else if (t == 0) {
      f_s[nt * 8 + r] = fr;
    }
  }
  if constexpr (NT > 1) {
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) f[nt][i] = f_s[nt * 8 + 2 * t + i];
  }
  // Columns that query row 2t + i of row tile nt sees (asked for in the tiles
  // where some row does not see all of them).
  auto limit = [&](int nt, int i) {
    if (kSel) return gr.cols;
    const int j = (row0 + nt * 8 + 2 * t + i) / p.heads;
    return gr.L - p.next_n + min(j, p.next_n - 1) + 1;
  };
  const int all_see = kSel ? gr.cols : gr.L - p.next_n + 1;  // columns every row sees

  float o[NT][2 * G][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2 * G; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
  // z: reference of a row's exponents (base 2).  It is raised to the running
  // maximum only when a logit passes it by kSlack, that is when an accumulator
  // passes thr, so most tiles need no maximum across lanes and no rescaling;
  // weights are then at most 2^kSlack, which fp16 and fp32 hold as well as 1.
  // thr = -inf: the row has seen no column.
  constexpr float kSlack = 8.f;
  float thr[NT][2], z[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) thr[nt][i] = -INFINITY, z[nt][i] = l[nt][i] = 0.f;
  float unit = 0.f, inv_unit = 0.f;  // o is in units of the largest value scale so far

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

  int s = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int tile = warp; tile < tiles; tile += kWarps) {
    locate(tile + kStages * kWarps);  // what it reads returns under this tile's work
    const int col0 = c0 + tile * kTile;
    uint2 live;  // columns of this tile
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
    }
    const uint32_t base = ring + s * Lay::kTileBytes;
    const uint32_t sbase = rest + Lay::kScales + s * Lay::kScaleBytes;
    if (live.x | live.y) {
      uint2 nan = make_uint2(0u, 0u);  // keys with a NaN scale
      // ---------------------------------------------------------------- scales
      // Lane 4 q8 + t takes the keys of rows 2t and 2t + 1 of the q8-th group
      // of eight: one fragment pair.
      {
        uint32_t kw[2], vw[2], vf[2][G];
        int key[2];
        uint32_t top = 0;  // scales order as their bits
        bool bad = false;
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
          if (!(((r >= 4 ? live.y : live.x) >> (key[i] & 31)) & 1)) kw[i] = vw[i] = 0u;
          bad |= has_ff(kw[i]) != 0;
          vf[i][0] = e8m0_bits<0>(vw[i]), vf[i][1] = e8m0_bits<1>(vw[i]);
          if constexpr (D == 128) vf[i][2] = e8m0_bits<2>(vw[i]), vf[i][3] = e8m0_bits<3>(vw[i]);
#pragma unroll
          for (int g = 0; g < G; ++g) top = max(top, vf[i][g]);
        }
        if (__any_sync(0xffffffffu, bad || top == 0x7F800000u)) {
          // NaN scales (code 255; rare).  A key's makes its logits NaN below;
          // a value's makes its 32 channels of every row that sees the column
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
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                  for (int g = 0; g < G; ++g)
                    if (((word >> (8 * g)) & 255u) == 255u && col < limit(nt, h)) {
                      o[nt][2 * g][h] = o[nt][2 * g][2 + h] = __uint_as_float(0x7FC00000u);
                      o[nt][2 * g + 1][h] = o[nt][2 * g + 1][2 + h] = __uint_as_float(0x7FC00000u);
                    }
            }
          }
          top = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              if (vf[i][g] == 0x7F800000u) vf[i][g] = 0u;
              top = max(top, vf[i][g]);
            }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (top > __float_as_uint(unit)) {
          const float up = __uint_as_float(top);
          const float down = unit == 0.f ? 0.f : unit / up;
          unit = up;
          inv_unit = 1.f / up;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2 * G; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) o[nt][i][j] *= down;
        }
        if constexpr (NT == 1) {
          // The key scales as fp32, where rows r of a group of eight find
          // them side by side.  (With two row tiles there is no room for
          // them: the scale words are unpacked where they are used.)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t at = ks_at + (r * 8 + 2 * t + i) * (4 * G);
            if constexpr (D == 128)
              sts128(at, e8m0_bits<0>(kw[i]), e8m0_bits<1>(kw[i]), e8m0_bits<2>(kw[i]),
                     e8m0_bits<3>(kw[i]));
            else
              sts64(at, e8m0_bits<0>(kw[i]), e8m0_bits<1>(kw[i]));
          }
        }
        uint32_t fac[G];
#pragma unroll
        for (int g = 0; g < G; ++g)
          fac[g] = pack_f16(__uint_as_float(vf[0][g]) * inv_unit,
                            __uint_as_float(vf[1][g]) * inv_unit);
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
        // ---------------------------------------------------------- S^T = K q^T
        float sacc[2][NT][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          uint32_t kw[2][G];
          float ks[2][G];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t at = hbase + (mt * 16 + h * 8) * D + k_at;
            if constexpr (D == 128) {
              const uint4 u = lds128(at);
              kw[h][0] = u.x, kw[h][1] = u.y, kw[h][2] = u.z, kw[h][3] = u.w;
            } else {
              const uint2 u = lds64(at);
              kw[h][0] = u.x, kw[h][1] = u.y;
            }
            if constexpr (NT == 1) {
              const uint32_t sat = ks_at + (half * 32 + mt * 16 + h * 8 + r) * (4 * G);
              if constexpr (D == 128) {
                const uint4 v = lds128(sat);
                ks[h][0] = __uint_as_float(v.x), ks[h][1] = __uint_as_float(v.y);
                ks[h][2] = __uint_as_float(v.z), ks[h][3] = __uint_as_float(v.w);
              } else {
                const uint2 v = lds64(sat);
                ks[h][0] = __uint_as_float(v.x), ks[h][1] = __uint_as_float(v.y);
              }
            } else {
              const uint32_t w = lds32(sbase + (half * 32 + mt * 16 + h * 8 + prow) * Lay::kSc);
              ks[h][0] = __uint_as_float(e8m0_bits<0>(w));
              ks[h][1] = __uint_as_float(e8m0_bits<1>(w));
              if constexpr (D == 128) {
                ks[h][2] = __uint_as_float(e8m0_bits<2>(w));
                ks[h][3] = __uint_as_float(e8m0_bits<3>(w));
              }
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            const uint32_t a0 = e2m1x2_to_f16x2<0>(kw[0][g]), a1 = e2m1x2_to_f16x2<0>(kw[1][g]);
            const uint32_t a2 = e2m1x2_to_f16x2<1>(kw[0][g]), a3 = e2m1x2_to_f16x2<1>(kw[1][g]);
            const uint32_t b0 = e2m1x2_to_f16x2<2>(kw[0][g]), b1 = e2m1x2_to_f16x2<2>(kw[1][g]);
            const uint32_t b2 = e2m1x2_to_f16x2<3>(kw[0][g]), b3 = e2m1x2_to_f16x2<3>(kw[1][g]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float c[4];
              uint4 q;
              if constexpr (NT == 1) q = make_uint4(qf[g][0], qf[g][1], qf[g][2], qf[g][3]);
              else q = lds128(q_at + (nt * G + g) * 512);
              mma16816_zero(c, a0, a1, a2, a3, q.x, q.y);
              mma16816(c, b0, b1, b2, b3, q.z, q.w);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sacc[mt][nt][j] =
                    g == 0 ? c[j] * ks[j >> 1][g] : fmaf(c[j], ks[j >> 1][g], sacc[mt][nt][j]);
            }
          }
        }
        // ------------------------------------------------------------- softmax
        if (!clean) {
          const uint32_t hlive = half ? live.y : live.x, hnan = half ? nan.y : nan.x;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = mt * 16 + h * 8 + prow;
              const bool here = (hlive >> key) & 1, bad = (hnan >> key) & 1;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  if (bad) sacc[mt][nt][2 * h + i] = __uint_as_float(0x7FC00000u);
                  if (!here || (!kSel && col0 + half * 32 + key >= limit(nt, i)))
                    sacc[mt][nt][2 * h + i] = -INFINITY;
                }
            }
        }
        if constexpr (kScores) {
          float* dst = p.scores + (static_cast<int64_t>(grp) * per_split + ht) * p.cols * kRows;
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int col = col0 + half * 32 + mt * 16 + h * 8 + prow;
              if (col < c1) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  *reinterpret_cast<float2*>(dst + static_cast<int64_t>(col) * kRows + nt * 8 +
                                             2 * t) =
                      make_float2(sacc[mt][nt][2 * h] * f[nt][0],
                                  sacc[mt][nt][2 * h + 1] * f[nt][1]);
              }
            }
        }
        float x[NT][2];
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            x[nt][i] = fmaxf(fmaxf(sacc[0][nt][i], sacc[0][nt][2 + i]),
                             fmaxf(sacc[1][nt][i], sacc[1][nt][2 + i]));
            up |= x[nt][i] > thr[nt][i];
          }
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float v = fmaxf(x[nt][i], __shfl_xor_sync(0xffffffffu, x[nt][i], 4));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
              v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
              if (v > thr[nt][i]) {
                const float zn = v * f[nt][i];
                const float a = thr[nt][i] == -INFINITY ? 0.f : ex2(z[nt][i] - zn);
                z[nt][i] = zn;
                thr[nt][i] = v + kSlack / f[nt][i];
                l[nt][i] *= a;
#pragma unroll
                for (int j = 0; j < 2 * G; ++j) o[nt][j][i] *= a, o[nt][j][2 + i] *= a;
              }
            }
        }
        uint32_t pf[2][NT][2];  // P as B fragments: row r, keys 2t, 2t+1 (+ 8)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const float p0 = ex2(fmaf(sacc[mt][nt][0], f[nt][0], -z[nt][0]));
            const float p1 = ex2(fmaf(sacc[mt][nt][1], f[nt][1], -z[nt][1]));
            const float p2 = ex2(fmaf(sacc[mt][nt][2], f[nt][0], -z[nt][0]));
            const float p3 = ex2(fmaf(sacc[mt][nt][3], f[nt][1], -z[nt][1]));
            l[nt][0] += p0 + p2;
            l[nt][1] += p1 + p3;
            pf[mt][nt][0] = transpose8x8(pack_f16(p0, p1));
            pf[mt][nt][1] = transpose8x8(pack_f16(p2, p3));
          }
        // ---------------------------------------------------------- O^T += V^T P
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
              lo[h][i] = (va[i] & 0x0F0F0F0Fu) | ((vb[i] << 4) & 0xF0F0F0F0u);
              hi[h][i] = ((va[i] >> 4) & 0x0F0F0F0Fu) | (vb[i] & 0xF0F0F0F0u);
            }
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            // Channels 32 g + 4 r + {0, 1} (first tile) and + {2, 3} (second).
            const uint32_t l0 = lo[0][g / 2], h0 = hi[0][g / 2];
            const uint32_t l1 = lo[1][g / 2], h1 = hi[1][g / 2];
            uint32_t a[2][4];
            if (g % 2 == 0) {
              a[0][0] = e2m1x2_to_f16x2<0>(l0), a[0][1] = e2m1x2_to_f16x2<0>(h0);
              a[0][2] = e2m1x2_to_f16x2<0>(l1), a[0][3] = e2m1x2_to_f16x2<0>(h1);
              a[1][0] = e2m1x2_to_f16x2<1>(l0), a[1][1] = e2m1x2_to_f16x2<1>(h0);
              a[1][2] = e2m1x2_to_f16x2<1>(l1), a[1][3] = e2m1x2_to_f16x2<1>(h1);
            } else {
              a[0][0] = e2m1x2_to_f16x2<2>(l0), a[0][1] = e2m1x2_to_f16x2<2>(h0);
              a[0][2] = e2m1x2_to_f16x2<2>(l1), a[0][3] = e2m1x2_to_f16x2<2>(h1);
              a[1][0] = e2m1x2_to_f16x2<3>(l0), a[1][1] = e2m1x2_to_f16x2<3>(h0);
              a[1][2] = e2m1x2_to_f16x2<3>(l1), a[1][3] = e2m1x2_to_f16x2<3>(h1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t b0 = mul_f16x2(pf[mt][nt][0], fac[0][g]);
              const uint32_t b1 = mul_f16x2(pf[mt][nt][1], fac[1][g]);
              mma16816(o[nt][2 * g], a[0][0], a[0][1], a[0][2], a[0][3], b0, b1);
              mma16816(o[nt][2 * g + 1], a[1][0], a[1][1], a[1][2], a[1][3], b0, b1);
            }
          }
        }
      }
    }
    __syncwarp();
    const uint2 c = fetch(s, tile + kStages * kWarps);
#pragma unroll
    for (int i = 0; i + 1 < kStages; ++i) cols[i] = cols[i + 1];
    cols[kStages - 1] = c;
    s = s + 1 == kStages ? 0 : s + 1;
    phase ^= s == 0;
  }
  if (!kSel && !ok) {
    // A copy never came: report, and give the others their time to land.
    if (lane == 0) record_error(p.err, kErrTimeout);
    for (int i = 0; i < kStages; ++i) mbar_wait_bounded(&bar[i], i < s ? phase ^ 1u : phase, nullptr);
  }

  // ------------------------------------------- join the four warps, write out
  cp_async_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);              // [warp][row][D]
  float* sml = so + kWarps * kRows * D;                    // [warp][row][2]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x = l[nt][i];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int row = nt * 8 + 2 * t + i;
      if (r == 0) {
        sml[(warp * kRows + row) * 2] = thr[nt][i] == -INFINITY ? -INFINITY : z[nt][i];
        sml[(warp * kRows + row) * 2 + 1] = x;
      }
      float* dst = so + (warp * kRows + row) * D;
#pragma unroll
      for (int g = 0; g < G; ++g)
        *reinterpret_cast<float4*>(dst + 32 * g + 4 * r) =
            make_float4(o[nt][2 * g][i] * unit, o[nt][2 * g][2 + i] * unit,
                        o[nt][2 * g + 1][i] * unit, o[nt][2 * g + 1][2 + i] * unit);
    }
  __syncthreads();
  const int64_t part = (static_cast<int64_t>(grp) * p.nsplit + split) * per_split + ht;
  for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[(w * kRows + row) * 2]);
    const float z0 = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sml[(w * kRows + row) * 2] - z0);
      L = fmaf(sml[(w * kRows + row) * 2 + 1], f, L);
      const float4 x = *reinterpret_cast<const float4*>(so + (w * kRows + row) * D + d);
      a.x = fmaf(x.x, f, a.x), a.y = fmaf(x.y, f, a.y);
      a.z = fmaf(x.z, f, a.z), a.w = fmaf(x.w, f, a.w);
    }
    const int n = row0 + row;
    if (whole) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      const float lse2 = M + log2f(L);
      if (n < nrows) {
        const int64_t hr = head_row<kSel>(p, grp, head, n);
        *reinterpret_cast<uint2*>(p.out + hr * D + d) =
            make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        if (d == 0 && p.lse) p.lse[hr] = L == 0.f ? -INFINITY : lse2 * 0.69314718055994531f;
      }
      if (kScores && d == 0)
        p.lse2[(static_cast<int64_t>(grp) * per_split + ht) * kRows + row] =
            n >= nrows || L == 0.f ? INFINITY : lse2;
    } else {
      *reinterpret_cast<float4*>(p.part_o + (part * kRows + row) * D + d) = a;
      if (d == 0)
        *reinterpret_cast<float2*>(p.part_ml + (part * kRows + row) * 2) = make_float2(M, L);
    }
  }
}

// Joins the partial sums of a group's chunks: one CTA per group, head and row
// tile, D/4 threads a row.
template <int D, int NT, bool kSel, bool kScores>
__global__ void __launch_bounds__(kThreads)
    kv4_join_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int kRows = 8 * NT;
  const int per_split = p.Hkv * p.row_tiles;
  const int ht = static_cast<int>(blockIdx.x % per_split);
  const int grp = static_cast<int>(blockIdx.x / per_split);
  const int head = ht / p.row_tiles;
  const int row0 = (ht % p.row_tiles) * kRows;
  const int nrows = kSel ? p.heads : p.heads * p.next_n;
  const Group gr = group_of<kSel>(p, grp, false);
  if (gr.cols <= p.chunk) return;
  const int ns = (gr.cols + p.chunk - 1) / p.chunk;
  for (int e = threadIdx.x; e < kRows * D / 4; e += kThreads) {
    const int row = e / (D / 4), d = (e % (D / 4)) * 4;
    float M = -INFINITY, L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int sp = 0; sp < ns; ++sp) {
      const int64_t part = (static_cast<int64_t>(grp) * p.nsplit + sp) * per_split + ht;
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + (part * kRows + row) * 2);
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + (part * kRows + row) * D + d);
      const float Mn = fmaxf(M, ml.x);
      const float z = Mn == -INFINITY ? 0.f : Mn;
      const float fo = ex2(M - z), fn = ex2(ml.x - z);
      M = Mn;
      L = L * fo + ml.y * fn;
      a.x = a.x * fo + x.x * fn, a.y = a.y * fo + x.y * fn;
      a.z = a.z * fo + x.z * fn, a.w = a.w * fo + x.w * fn;
    }
    const int n = row0 + row;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const float lse2 = M + log2f(L);
    if (n < nrows) {
      const int64_t hr = head_row<kSel>(p, grp, head, n);
      *reinterpret_cast<uint2*>(p.out + hr * D + d) =
          make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
      if (d == 0 && p.lse) p.lse[hr] = L == 0.f ? -INFINITY : lse2 * 0.69314718055994531f;
    }
    if (kScores && d == 0)
      p.lse2[(static_cast<int64_t>(grp) * per_split + ht) * kRows + row] =
          n >= nrows || L == 0.f ? INFINITY : lse2;
  }
}

// A column's attention weight, summed over heads and rows in one fixed order:
// w = sum exp2(S - lse).  Dense: added to key_weights.  Selected: written to
// sel_weights, and (one token a request) added to key_weights at the column's
// position.
template <int NT, bool kSel>
__global__ void __launch_bounds__(256) kv4_weight_kernel(const __grid_constant__ Kv4AttnParams p) {
  constexpr int kRows = 8 * NT;
  const int per_split = p.Hkv * p.row_tiles;
  const int per_grp = (p.cols + 255) / 256;
  const int grp = static_cast<int>(blockIdx.x / per_grp);
  const int col = static_cast<int>(blockIdx.x % per_grp) * 256 + threadIdx.x;
  const Group gr = group_of<kSel>(p, grp, false);
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
    for (int ht = 0; ht < per_split; ++ht) {
      const float4* src = reinterpret_cast<const float4*>(
          p.scores + ((static_cast<int64_t>(grp) * per_split + ht) * p.cols + col) * kRows);
      const float4* z = reinterpret_cast<const float4*>(lse_s + ht * kRows);
#pragma unroll
      for (int i = 0; i < kRows / 4; ++i) {
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
    const Group gr = group_of<true>(p, static_cast<int>(row), false);
    for (int c = threadIdx.x; c < p.sel_k; c += blockDim.x) {
      const int pos = __ldg(p.sel + row * p.sel_k + c);
      if (pos >= 0 && pos < gr.limit)
        atomicAdd(p.key_weights + static_cast<int64_t>(b) * p.ldw + pos,
                  p.sel_weights[row * p.sel_k + c]);
    }
    __syncthreads();
  }
}

template <int D, int NT, bool kSel, bool kScores>
cudaError_t launch_one(const Kv4AttnParams& p, cudaStream_t s) {
  using Lay = Layout<D, NT>;
  constexpr int kRing = Lay::kBytes;
  constexpr int kJoin = kWarps * 8 * NT * (D + 2) * 4;
  constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
  auto* fn = kv4_attn_kernel<D, NT, kSel, kScores>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles = static_cast<int64_t>(p.groups) * p.Hkv * p.row_tiles;
  fn<<<static_cast<unsigned>(tiles * p.nsplit), kThreads, kSmem, s>>>(p);
  e = cudaGetLastError();
  if (e == cudaSuccess && p.nsplit > 1) {
    kv4_join_kernel<D, NT, kSel, kScores><<<static_cast<unsigned>(tiles), kThreads, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && kScores) {
    const int64_t grid = static_cast<int64_t>(p.groups) * ((p.cols + 255) / 256);
    const size_t sm = static_cast<size_t>(p.Hkv) * p.row_tiles * 8 * NT * sizeof(float);
    kv4_weight_kernel<NT, kSel><<<static_cast<unsigned>(grid), 256, sm, s>>>(p);
    e = cudaGetLastError();
    if (e == cudaSuccess && kSel && p.key_weights && p.next_n > 1) {
      kv4_weight_scatter_kernel<<<static_cast<unsigned>(p.groups / p.next_n), 1024, 0, s>>>(p);
      e = cudaGetLastError();
    }
  }
  return e;
}

template <int D, int NT>
cudaError_t launch_nt(const Kv4AttnParams& p, bool scores, cudaStream_t s) {
  if (p.sel) return scores ? launch_one<D, NT, true, true>(p, s) : launch_one<D, NT, true, false>(p, s);
  return scores ? launch_one<D, NT, false, true>(p, s) : launch_one<D, NT, false, false>(p, s);
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

Kv4AttnPlan kv4_attn_plan(int B, int next_n, int Hq, int Hkv, int D, int64_t cols, bool selected,
                          bool weights) {
  Kv4AttnPlan pl = {};
  pl.heads = Hq / Hkv;
  pl.groups = selected ? static_cast<int64_t>(B) * next_n : B;
  const int rows = selected ? pl.heads : pl.heads * next_n;
  pl.nt = rows <= 8 ? 1 : 2;
  pl.row_tiles = (rows + 8 * pl.nt - 1) / (8 * pl.nt);
  // Chunks: enough CTAs for every SM's three places, at least one tile a
  // warp, and no more than 64 tiles so that requests of unequal length spread.
  const int64_t tiles = (cols + kTile - 1) / kTile;
  const int64_t lanes = pl.groups * Hkv * pl.row_tiles;
  const int64_t places =
      static_cast<int64_t>(device_sm_count() > 0 ? device_sm_count() : 152) * kCtasPerSm;
  int64_t per = (tiles * lanes + places - 1) / (places > 0 ? places : 1);
  per = per < kWarps ? kWarps : (per > 64 ? 64 : per);
  per = (per + kWarps - 1) / kWarps * kWarps;
  pl.chunk = static_cast<int>(per) * kTile;
  pl.nsplit = static_cast<int>((cols + pl.chunk - 1) / pl.chunk);
  if (pl.nsplit < 1) pl.nsplit = 1;
  const int64_t parts = lanes * pl.nsplit * 8 * pl.nt;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += up256(bytes);
    return at;
  };
  pl.part_o = take(pl.nsplit > 1 ? parts * D * 4 : 0);
  pl.part_ml = take(pl.nsplit > 1 ? parts * 8 : 0);
  pl.scores = take(weights ? lanes * cols * 8 * pl.nt * 4 : 0);
  pl.lse2 = take(weights ? lanes * 8 * pl.nt * 4 : 0);
  pl.sel_weights = take(weights && selected && next_n > 1 ? pl.groups * cols * 4 : 0);
  pl.bytes = off;
  return pl;
}

cudaError_t launch_kv4_attention(const Kv4AttnParams& p, int D, int nt, bool scores,
                                 cudaStream_t s) {
  if (D == 128) return nt == 1 ? launch_nt<128, 1>(p, scores, s) : launch_nt<128, 2>(p, scores, s);
  return nt == 1 ? launch_nt<64, 1>(p, scores, s) : launch_nt<64, 2>(p, scores, s);
}

}  // namespace dsa
