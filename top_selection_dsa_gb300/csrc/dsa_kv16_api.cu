// dsa_kv16_api.cu -- C-ABI entry points of the 16-bit key/value cache: argument
// checks, workspace layout and launches on the caller's stream.  Like the
// other entry points they allocate nothing and report what the host can see
// before anything is launched.
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

// Shape of a cache: head dimension, page size, and rows countable in 31 bits
// (the coordinate of a TMA box).
dsa_status_t check_pages(const void* k_cache, const void* v_cache, int num_blocks, int block_size,
                         int Hkv, int D) {
  if (!k_cache || !v_cache || num_blocks < 1 || block_size < 1 || Hkv < 1 || D < 1)
    return DSA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return DSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
  if (!pow2(block_size) || block_size < 8 || block_size > 128) return DSA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_blocks) * block_size > 0x7FFFFFFFll / Hkv)
    return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

bool bad_rows(const void* x, int64_t stride, int T, int H, int D) {
  return !aligned(x, 16) || stride % 8 != 0 ||
         (T > 1 && stride < static_cast<int64_t>(H) * D);
}

// The rotation's arguments, common to both calls.
dsa_status_t check_rotation(const int32_t* positions, const uint64_t* turns, int rotary,
                            float rope_scale, const float* q_weight, const float* k_weight,
                            float eps, int D) {
  if (rotary < 0 || rotary > D || rotary % 2 != 0) return DSA_ERR_INVALID_ARG;
  if (rotary % 16 != 0) return DSA_ERR_UNSUPPORTED;
  if (rotary > 0 && (!positions || !turns || !isfinite(rope_scale))) return DSA_ERR_INVALID_ARG;
  if ((q_weight || k_weight) && !(isfinite(eps) && eps >= 0.f)) return DSA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(turns, 8) || !aligned(q_weight, 4) ||
      !aligned(k_weight, 4))
    return DSA_ERR_INVALID_ARG;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

dsa_status_t dsa_qk_norm_rope(const void* q, int64_t q_stride, int Hq, const void* k,
                              int64_t k_stride, int Hk, int T, int D, const int32_t* positions,
                              const uint64_t* turns, int rotary, int interleaved,
                              float rope_scale, const float* q_weight, const float* k_weight,
                              float eps, void* q_out, void* k_out, dsa_stream_t stream) {
  const CallRange range("dsa_qk_norm_rope");
  if (!q || !q_out || T < 0 || Hq < 1 || D < 1) return DSA_ERR_INVALID_ARG;
  if (k ? (!k_out || Hk < 1) : (k_out || Hk != 0)) return DSA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return DSA_ERR_UNSUPPORTED;
  if (bad_rows(q, q_stride, T, Hq, D) || !aligned(q_out, 16)) return DSA_ERR_INVALID_ARG;
  if (k && (bad_rows(k, k_stride, T, Hk, D) || !aligned(k_out, 16))) return DSA_ERR_INVALID_ARG;
  dsa_status_t st =
      check_rotation(positions, turns, rotary, rope_scale, q_weight, k_weight, eps, D);
  if (st != DSA_OK) return st;
  if (Hq > 4096 || Hk > 4096 || T >= (1 << 30)) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  RopeParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.T = T;
  p.Hq = Hq;
  p.Hk = Hk;
  p.positions = positions;
  p.turns = turns;
  p.rotary = rotary;
  p.rope_scale = rope_scale;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  return from_cuda(launch_rope(p, D, interleaved != 0, as_stream(stream)));
}

dsa_status_t dsa_kv_append(const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int64_t* slot_mapping, int T, int Hkv, int D,
                           const int32_t* positions, const uint64_t* turns, int rotary,
                           int interleaved, float rope_scale, const float* k_weight, float eps,
                           void* k_cache, void* v_cache, int num_blocks, int block_size,
                           const void* q, int64_t q_stride, int Hq, const float* q_weight,
                           void* q_out, dsa_stream_t stream) {
  const CallRange range("dsa_kv_append");
  if (!k || !v || !slot_mapping || T < 0) return DSA_ERR_INVALID_ARG;
  if (q ? (!q_out || Hq < 1) : (q_out || q_weight || Hq != 0)) return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_pages(k_cache, v_cache, num_blocks, block_size, Hkv, D);
  if (st != DSA_OK) return st;
  if (bad_rows(k, k_stride, T, Hkv, D) || bad_rows(v, v_stride, T, Hkv, D) ||
      !aligned(slot_mapping, 8))
    return DSA_ERR_INVALID_ARG;
  if (q && (bad_rows(q, q_stride, T, Hq, D) || !aligned(q_out, 16))) return DSA_ERR_INVALID_ARG;
  st = check_rotation(positions, turns, rotary, rope_scale, q_weight, k_weight, eps, D);
  if (st != DSA_OK) return st;
  if (Hq > 4096 || Hkv > 4096 || T >= (1 << 30)) return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  RopeParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.T = T;
  p.Hq = Hq;
  p.Hk = p.Hv = Hkv;
  p.positions = positions;
  p.turns = turns;
  p.rotary = rotary;
  p.rope_scale = rope_scale;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.eps = eps;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_cache);
  p.v_out = static_cast<uint16_t*>(v_cache);
  p.slots = slot_mapping;
  p.capacity = static_cast<int64_t>(num_blocks) * block_size;
  p.log_bs = log2_of(block_size);
  p.err = error_word();
  if (!p.err) return DSA_ERR_CUDA;
  return from_cuda(launch_rope(p, D, interleaved != 0, as_stream(stream)));
}

size_t dsa_kv_attention_workspace_bytes(int T, int Hq, int Hkv, int D) {
  if (T < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Hq / Hkv > 128 || (D != 64 && D != 128))
    return static_cast<size_t>(-1);
  return static_cast<size_t>(kv_attn_plan(T, Hq / Hkv, D).bytes);
}

dsa_status_t dsa_kv_attention(const void* q, int64_t q_stride, const void* k_cache,
                              const void* v_cache, int num_blocks, const int32_t* block_table,
                              int max_blocks, const int32_t* context_lens,
                              const int32_t* query_starts, int T, int B, int block_size, int Hq,
                              int Hkv, int D, float softmax_scale, int window, int sink, void* out,
                              float* lse, void* workspace, size_t ws_bytes, dsa_stream_t stream) {
  const CallRange range("dsa_kv_attention");
  if (!q || !block_table || !context_lens || !query_starts || !out) return DSA_ERR_INVALID_ARG;
  // (Where the scaled logits leave the range that the weights serve, rows are NaN.)
  if (T < 0 || B < 0 || max_blocks < 1 || Hq < 1 || window < 0 || sink < 0 ||
      !(softmax_scale >= 0x1p-64f && softmax_scale <= 0x1p64f))
    return DSA_ERR_INVALID_ARG;
  dsa_status_t st = check_pages(k_cache, v_cache, num_blocks, block_size, Hkv, D);
  if (st != DSA_OK) return st;
  if (Hq % Hkv != 0) return DSA_ERR_INVALID_ARG;
  if (bad_rows(q, q_stride, T, Hq, D) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(context_lens, 4) || !aligned(query_starts, 4) || !aligned(lse, 4))
    return DSA_ERR_INVALID_ARG;
  const int64_t max_ctx = static_cast<int64_t>(max_blocks) * block_size;
  const int G = Hq / Hkv;
  if (G > 128 || B > kMaxPagedRequests || max_ctx >= (int64_t(1) << 30) || T >= (1 << 30) ||
      q_stride >= (int64_t(1) << 38) || kv_attn_units(T, B, G, max_ctx) >= (int64_t(1) << 31))
    return DSA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return DSA_OK;
  const KvAttnPlan pl = kv_attn_plan(T, G, D);
  if (!workspace || !aligned(workspace, 256) || ws_bytes < static_cast<size_t>(pl.bytes))
    return DSA_ERR_INVALID_ARG;
  KvAttnParams p = {};
  const uint64_t qd[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(Hq),
                          static_cast<uint64_t>(T)};
  // One token: its stride is not used, and need not be one.
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  const uint64_t qs[2] = {row, T > 1 ? static_cast<uint64_t>(q_stride) * 2 : row * Hq};
  const uint32_t qb[3] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(pl.tpt)};
  const uint64_t kd[2] = {static_cast<uint64_t>(D),
                          static_cast<uint64_t>(num_blocks) * Hkv * block_size};
  const uint64_t ks[1] = {row};
  const uint32_t kb[2] = {64, static_cast<uint32_t>(block_size)};
  if (!encode_bf16_boxes(&p.tmap_q, q, 3, qd, qs, qb) ||
      !encode_bf16_boxes(&p.tmap_k, k_cache, 2, kd, ks, kb) ||
      !encode_bf16_boxes(&p.tmap_v, v_cache, 2, kd, ks, kb))
    return DSA_ERR_CUDA;
  p.v = static_cast<const uint16_t*>(v_cache);
  p.block_table = block_table;
  p.context_lens = context_lens;
  p.starts = query_starts;
  p.T = T;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.tpt = pl.tpt;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  p.log_bs = log2_of(block_size);
  // A window or sink past every context changes nothing more.
  p.window = window < max_ctx ? window : 0;
  p.sink = static_cast<int>(sink < max_ctx ? sink : max_ctx);
  // Cost, in halves of a tall unit (some 3000 cycles), as fitted to the SMs' times
  // of 40 batches: D = 128, where a short unit's twice the keys are bound by
  // memory, 4 a short unit, 5 and 2 a tile's start and end; D = 64 2, 4 and 3.
  // (Starts of 6 and 4, 6 and 2 instead: 0.9 and 2.5 % slower over all.)
  p.short_log = D == 128 ? 2 : 1;
  p.tall_start = D == 128 ? 5 : 4;
  p.short_start = D == 128 ? 2 : 3;
  p.scale_log2e = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.ctas = pl.ctas;
  p.slot_rows = pl.slot_rows;
  char* ws = static_cast<char*>(workspace);
  p.notes = reinterpret_cast<int4*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + pl.part_ml);
  p.part_o = reinterpret_cast<float*>(ws + pl.part_o);
  p.err = error_word();
  if (!p.err) return DSA_ERR_CUDA;
  return from_cuda(launch_kv_attention(p, D, as_stream(stream)));
}

}  // extern "C"
