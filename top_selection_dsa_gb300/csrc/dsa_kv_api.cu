// dsa_kv_api.cu -- C-ABI entry points of the 4-bit key/value cache: argument
// checks, workspace layout and launches on the caller's stream.  Like the
// indexer's entry points they allocate nothing and report what the host can
// see before anything is launched.
#include <math.h>

#include "dsa_abi.h"
#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

// Shape of a cache: head dimension, page size, and records countable in 32 bits.
dsa_status_t check_cache(const void* cache, const void* scales, int num_blocks, int block_size,
                         int Hkv, int D) {
  if (!cache || !scales || num_blocks < 1 || block_size < 1 || Hkv < 1 || D < 1)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(scales, 16)) return DSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
  if (!pow2(block_size) || block_size < 8 || block_size > 128) return DSA_ERR_UNSUPPORTED;
  if (static_cast<uint64_t>(num_blocks) * static_cast<uint64_t>(block_size) >
      0xFFFFFFFFull / static_cast<uint64_t>(Hkv))
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

struct AttnArgs {
  const void* q;
  const void* cache;
  const uint8_t* scales;
  int num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* context_lens;
  int B, next_n, block_size, Hq, Hkv, D;
  float softmax_scale;
  const int32_t* sel;
  int sel_k;
  void* out;
  float* lse;
  float* sel_weights;
  float* key_weights;
  int64_t ldw;
  void* workspace;
  size_t ws_bytes;
};

dsa_status_t run_attention(const AttnArgs& a, bool selected, dsa_stream_t stream) {
  if (!a.q || !a.block_table || !a.context_lens || !a.out || (selected && !a.sel))
    return DSA_ERR_INVALID_ARG;
  if (a.B < 0 || a.next_n < 1 || a.max_blocks < 1 || a.Hq < 1 || (selected && a.sel_k < 1) ||
      !isfinite(a.softmax_scale))
    return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_cache(a.cache, a.scales, a.num_blocks, a.block_size, a.Hkv, a.D);
  if (st != DSA_OK) return st;
  if (a.Hq % a.Hkv != 0) return DSA_ERR_INVALID_ARG;
  if (!aligned(a.q, 16) || !aligned(a.out, 8) || !aligned(a.block_table, 4) ||
      !aligned(a.context_lens, 4) || !aligned(a.sel, 4) || !aligned(a.lse, 4) ||
      !aligned(a.sel_weights, 4) || !aligned(a.key_weights, 4))
    return DSA_ERR_INVALID_ARG;
  const int64_t max_ctx = static_cast<int64_t>(a.max_blocks) * a.block_size;
  if (a.key_weights && a.ldw < max_ctx) return DSA_ERR_INVALID_ARG;
  if (max_ctx >= (int64_t(1) << 30) || a.B > 65535 ||
      static_cast<int64_t>(a.B) * a.next_n * a.Hq >= (int64_t(1) << 31))
    return DSA_ERR_UNSUPPORTED;
  const bool weights = a.key_weights || a.sel_weights;
  const int64_t cols = selected ? a.sel_k : max_ctx;
  if (a.B == 0) return DSA_OK;
  const Kv4AttnPlan pl =
      kv4_attn_plan(a.B, a.next_n, a.Hq, a.Hkv, a.D, cols, selected, weights);
  const int64_t lanes = static_cast<int64_t>(a.Hkv) * pl.row_tiles;
  // Units of work are counted in 32 bits.
  const int64_t units = cols / pl.unit + 1;
  if (pl.groups * lanes >= (int64_t(1) << 31) / (units > pl.rows ? units : pl.rows) ||
      pl.groups * ((cols + 255) / 256) >= (int64_t(1) << 31) ||
      (weights && lanes * pl.rows * 4 > 48 * 1024))
    return DSA_ERR_UNSUPPORTED;
  if (pl.bytes > 0 && (!a.workspace || !aligned(a.workspace, 256) ||
                       a.ws_bytes < static_cast<size_t>(pl.bytes)))
    return DSA_ERR_INVALID_ARG;
  Kv4AttnParams p = {};
  if (!selected && !encode_rows_map(&p.tmap, a.cache, a.D, a.block_size,
                                    a.block_size < pl.tile ? a.block_size : pl.tile,
                                    static_cast<int64_t>(a.num_blocks) * a.Hkv))
    return DSA_ERR_CUDA;
  p.q = static_cast<const uint16_t*>(a.q);
  p.cache = static_cast<const uint8_t*>(a.cache);
  p.scales = a.scales;
  p.block_table = a.block_table;
  p.context_lens = a.context_lens;
  p.sel = selected ? a.sel : nullptr;
  p.sel_k = a.sel_k;
  p.groups = static_cast<int>(pl.groups);
  p.next_n = a.next_n;
  p.heads = pl.heads;
  p.Hkv = a.Hkv;
  p.Hq = a.Hq;
  p.row_tiles = pl.row_tiles;
  p.max_blocks = a.max_blocks;
  p.num_blocks = a.num_blocks;
  p.log_bs = log2_of(a.block_size);
  p.scale_log2e = static_cast<float>(static_cast<double>(a.softmax_scale) * 1.4426950408889634);
  p.ctas = pl.ctas;
  p.cols = static_cast<int>(cols);
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  char* ws = static_cast<char*>(a.workspace);
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.part_ml = reinterpret_cast<float*>(ws + pl.part_ml);
  p.spans = pl.split ? reinterpret_cast<int4*>(ws + pl.spans) : nullptr;
  p.scores = reinterpret_cast<float*>(ws + pl.scores);
  p.score_rows = pl.score_rows;
  p.lse2 = reinterpret_cast<float*>(ws + pl.lse2);
  // Several tokens a request: the scatter reads the rows' weights, so they
  // are written out even when the caller does not ask for them.
  p.sel_weights = a.sel_weights ? a.sel_weights
                  : selected && a.key_weights && a.next_n > 1
                      ? reinterpret_cast<float*>(ws + pl.sel_weights)
                      : nullptr;
  p.key_weights = a.key_weights;
  p.ldw = a.ldw;
  p.err = error_word();
  if (!p.err) return DSA_ERR_CUDA;
  return from_cuda(launch_kv4_attention(p, a.D, pl.rows, weights, as_stream(stream)));
}

// Workspace of the eviction: row ranges, the middle's selection, and the
// top-k's scratch for few long rows.
struct EvictPlan {
  int64_t starts, ends, mid, split, bytes;
};
EvictPlan evict_plan(int64_t B, int64_t max_ctx, int64_t room) {
  EvictPlan pl = {};
  int64_t off = 0;
  auto take = [&](int64_t n) {
    const int64_t at = off;
    off += up256(n);
    return at;
  };
  pl.starts = take(B * 4);
  pl.ends = take(B * 4);
  pl.mid = take(B * room * 4);
  pl.split = take(topk_split_rows(B, max_ctx) ? B * topk_split_words(max_ctx) * 4 : 0);
  pl.bytes = off;
  return pl;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status_t dsa_kv4_insert(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const int64_t* slot_mapping, int T, int Hkv, int D, void* cache,
                            uint8_t* scales, int num_blocks, int block_size,
                            dsa_stream_t stream) {
  const CallRange range("dsa_kv4_insert");
  if (!k || !v || !slot_mapping || T < 0) return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_cache(cache, scales, num_blocks, block_size, Hkv, D);
  if (st != DSA_OK) return st;
  const int64_t row = static_cast<int64_t>(Hkv) * D;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_mapping, 8) || k_stride % 8 != 0 ||
      v_stride % 8 != 0 || (T > 1 && (k_stride < row || v_stride < row)))
    return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * Hkv >= (int64_t(1) << 30)) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  uint32_t* err = error_word();
  if (!err) return DSA_ERR_CUDA;
  return from_cuda(launch_kv4_insert(k, k_stride, v, v_stride, slot_mapping, T, Hkv, D, cache,
                                     scales, num_blocks, block_size, err, as_stream(stream)));
}

dsa_status_t dsa_kv4_gather(const void* cache, const uint8_t* scales, int num_blocks,
                            int block_size, const int64_t* slots, int T, int Hkv, int D, void* k,
                            void* v, dsa_stream_t stream) {
  const CallRange range("dsa_kv4_gather");
  if (!slots || !k || !v || T < 0) return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_cache(cache, scales, num_blocks, block_size, Hkv, D);
  if (st != DSA_OK) return st;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return DSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * Hkv >= (int64_t(1) << 30)) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  uint32_t* err = error_word();
  if (!err) return DSA_ERR_CUDA;
  return from_cuda(launch_kv4_gather(cache, scales, slots, T, Hkv, D, num_blocks, block_size, k, v,
                                     err, as_stream(stream)));
}

size_t dsa_kv4_attention_workspace_bytes(int B, int next_n, int Hq, int Hkv, int D, int64_t cols,
                                         int selected, int weights) {
  if (B < 0 || next_n < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 1 || cols < 0)
    return static_cast<size_t>(-1);
  if (B == 0) return 0;
  return static_cast<size_t>(
      kv4_attn_plan(B, next_n, Hq, Hkv, D, cols, selected != 0, weights != 0).bytes);
}

dsa_status_t dsa_kv4_attention(const void* q, const void* cache, const uint8_t* scales,
                               int num_blocks, const int32_t* block_table, int max_blocks,
                               const int32_t* context_lens, int B, int next_n, int block_size,
                               int Hq, int Hkv, int D, float softmax_scale, void* out, float* lse,
                               float* key_weights, int64_t ldw, void* workspace, size_t ws_bytes,
                               dsa_stream_t stream) {
  const CallRange range("dsa_kv4_attention");
  const AttnArgs a = {q,       cache,   scales, num_blocks, block_table, max_blocks,
                      context_lens, B, next_n, block_size, Hq, Hkv, D, softmax_scale,
                      nullptr, 0,       out,    lse,        nullptr,     key_weights,
                      ldw,     workspace, ws_bytes};
  return run_attention(a, false, stream);
}

dsa_status_t dsa_kv4_attention_topk(const void* q, const void* cache, const uint8_t* scales,
                                    int num_blocks, const int32_t* block_table, int max_blocks,
                                    const int32_t* context_lens, const int32_t* topk, int k, int B,
                                    int next_n, int block_size, int Hq, int Hkv, int D,
                                    float softmax_scale, void* out, float* lse,
                                    float* topk_weights, float* key_weights, int64_t ldw,
                                    void* workspace, size_t ws_bytes, dsa_stream_t stream) {
  const CallRange range("dsa_kv4_attention_topk");
  const AttnArgs a = {q,    cache, scales, num_blocks, block_table,  max_blocks,
                      context_lens, B, next_n, block_size, Hq, Hkv, D, softmax_scale,
                      topk, k,     out,    lse,        topk_weights, key_weights,
                      ldw,  workspace, ws_bytes};
  return run_attention(a, true, stream);
}

size_t dsa_kv_evict_workspace_bytes(int B, int64_t max_ctx, int budget) {
  if (B < 0 || max_ctx < 0 || budget < 1) return static_cast<size_t>(-1);
  return static_cast<size_t>(evict_plan(B, max_ctx, budget).bytes);
}

dsa_status_t dsa_kv_evict_select(const float* key_weights, int64_t ldw,
                                 const int32_t* context_lens, int B, int max_ctx, int budget,
                                 int sink, int recent, int32_t* keep, int32_t* new_lens,
                                 void* workspace, size_t ws_bytes, dsa_stream_t stream) {
  const CallRange range("dsa_kv_evict_select");
  if (!key_weights || !context_lens || !keep || !new_lens) return DSA_ERR_INVALID_ARG;
  if (B < 0 || max_ctx < 1 || ldw < max_ctx || budget < 1 || sink < 0 || recent < 0 ||
      static_cast<int64_t>(sink) + recent > budget)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(key_weights, 4) || !aligned(context_lens, 4) || !aligned(keep, 4) ||
      !aligned(new_lens, 4))
    return DSA_ERR_INVALID_ARG;
  if (!topk_supported(max_ctx) || B > 65535) return DSA_ERR_UNSUPPORTED;
  if (B == 0) return DSA_OK;
  const EvictPlan pl = evict_plan(B, max_ctx, budget);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < static_cast<size_t>(pl.bytes))
    return DSA_ERR_INVALID_ARG;
  char* ws = static_cast<char*>(workspace);
  int32_t* starts = reinterpret_cast<int32_t*>(ws + pl.starts);
  int32_t* ends = reinterpret_cast<int32_t*>(ws + pl.ends);
  int32_t* mid = reinterpret_cast<int32_t*>(ws + pl.mid);
  const int room = budget - sink - recent;
  cudaStream_t st = as_stream(stream);
  uint32_t* err = error_word();
  if (!err) return DSA_ERR_CUDA;
  if (evict_small(B, max_ctx))
    return from_cuda(launch_evict_small(key_weights, ldw, context_lens, B, max_ctx, budget, sink,
                                        recent, keep, new_lens, err, st));
  cudaError_t e =
      launch_evict_ranges(context_lens, B, max_ctx, sink, recent, starts, ends, err, st);
  if (e == cudaSuccess && room > 0) {
    TopkParams p = {};
    p.logits = key_weights;
    p.ld = ldw;
    p.row_starts = starts;
    p.row_ends = ends;
    p.next_n = 1;
    p.R = B;
    p.S = max_ctx;
    p.k = room;
    p.bitmap_words = topk_bitmap_words(max_ctx);
    p.out = mid;
    if (topk_split_rows(B, max_ctx)) {
      p.split = reinterpret_cast<uint32_t*>(ws + pl.split);
      p.split_words = topk_split_words(max_ctx);
    }
    e = launch_topk(p, st);
  }
  if (e == cudaSuccess)
    e = launch_evict_keep(context_lens, starts, ends, mid, B, max_ctx, room, budget, keep,
                          new_lens, st);
  return from_cuda(e);
}

dsa_status_t dsa_kv_compact(const dsa_paged_rows_t* caches, int n_caches, int num_blocks,
                            int block_size, const int32_t* block_table, int max_blocks,
                            const int32_t* new_block_table, int new_max_blocks,
                            const int32_t* context_lens, const int32_t* keep,
                            const int32_t* new_lens, int B, int budget, const float* key_weights,
                            float* key_weights_out, int64_t ldw, dsa_stream_t stream) {
  const CallRange range("dsa_kv_compact");
  if ((n_caches > 0 && !caches) || !block_table || !context_lens || !keep || !new_lens)
    return DSA_ERR_INVALID_ARG;
  if (n_caches < 0 || num_blocks < 1 || block_size < 1 || max_blocks < 1 || B < 0 || budget < 1 ||
      (new_block_table && new_max_blocks < 1))
    return DSA_ERR_INVALID_ARG;
  if ((key_weights != nullptr) != (key_weights_out != nullptr)) return DSA_ERR_INVALID_ARG;
  const int64_t max_ctx = static_cast<int64_t>(max_blocks) * block_size;
  if (key_weights && ldw < max_ctx) return DSA_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(new_block_table, 4) || !aligned(context_lens, 4) ||
      !aligned(keep, 4) || !aligned(new_lens, 4) || !aligned(key_weights, 4) ||
      !aligned(key_weights_out, 4))
    return DSA_ERR_INVALID_ARG;
  for (int i = 0; i < n_caches; ++i)
    if (!caches[i].base || !aligned(caches[i].base, 16) || caches[i].planes < 1 ||
        caches[i].row_bytes < 4 || caches[i].row_bytes % 4 != 0)
      return DSA_ERR_INVALID_ARG;
  if (n_caches > kMaxCompact || !pow2(block_size) || B > 65535 ||
      max_ctx >= (int64_t(1) << 30) ||
      static_cast<int64_t>(new_max_blocks) * block_size >= (int64_t(1) << 30) ||
      budget > 65535 * 1024)
    return DSA_ERR_UNSUPPORTED;
  CompactParams p = {};
  int64_t units = 0;
  for (int i = 0; i < n_caches; ++i) {
    p.cache[i].base = static_cast<uint8_t*>(caches[i].base);
    p.cache[i].planes = caches[i].planes;
    p.cache[i].row_bytes = caches[i].row_bytes;
    p.first_unit[i] = static_cast<int>(units);
    units += compact_units(p.cache[i]);
    if (units > (1 << 30)) return DSA_ERR_UNSUPPORTED;
    p.first_unit[i + 1] = static_cast<int>(units);
  }
  p.ncaches = n_caches;
  p.units = static_cast<int>(units);
  if (B == 0) return DSA_OK;
  p.keep = keep;
  p.new_lens = new_lens;
  p.block_table = block_table;
  p.new_block_table = new_block_table;
  p.B = B;
  p.budget = budget;
  p.max_blocks = max_blocks;
  p.new_max_blocks = new_block_table ? new_max_blocks : 0;
  p.num_blocks = num_blocks;
  p.log_bs = log2_of(block_size);
  p.weights = key_weights;
  p.weights_out = key_weights_out;
  p.ldw = ldw;
  p.old_lens = context_lens;
  p.err = error_word();
  if (!p.err) return DSA_ERR_CUDA;
  return from_cuda(launch_kv_compact(p, as_stream(stream)));
}

}  // extern "C"
