// dsa_rope.cu -- a norm of each query and key head and its rotation by
// position, in one pass, and the append of the results to the 16-bit paged
// cache (sm_103a).
//
// A head's row x of D elements at position p:
//   y = x / sqrt(mean(x^2) + eps) * weight             (with a weight)
//   the first R = 2 F elements in pairs (y_i, y_{i+F}), or interleaved
//   (y_{2i}, y_{2i+1}), by the angle p f_i:
//     m (a cos - b sin),  m (a sin + b cos)
// all in fp32, rounded to bf16 once.
//
// Angles.  f_i comes as `turns`, f_i / (2 pi) in units of 2^-64 turns: p times
// it, modulo 2^64, is the angle's fraction of a turn exactly (integers wrap at
// whole turns), whatever the position: no table over positions, no 64-bit
// floating point.  Its distance from the nearest quarter turn is rounded to fp32,
// 2^-28 turns at most; the table's own rounding times the position is 2^-34 at most.
//
// A CTA writes the cosines and sines of its tokens to shared memory once; D / 8
// lanes take a row, each the elements of whole pairs (two groups of four that
// lie F apart, or eight neighbours), so nothing but the norm's sum crosses
// lanes.  A warp's task is some rows of one token and kind, all loaded at once,
// and the products of weights, cosines and sines are made once for it.
//
// The pass is memory-bound: 16384 tokens of 64 + 8 heads of 128 with norms 99 us,
// 6.1 TB/s (92 % of the measured copy bandwidth, 71 % of the issue slots); index
// queries and key, 8191 tokens of 64 + 1 heads, half of them rotated, 45 us, 6.0;
// 32768 tokens appended, 48 us, 5.6.  With pairs across lanes and heads stepped
// one by one (194 instructions a warp's row instead of some 90) it was bound by
// issue: 159 us for the first.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 32;  // of a CTA
constexpr int kAhead = 4;       // rows whose loads a lane has in flight

// A CTA takes `tasks` of the tasks of each of `tokens` tokens (blockIdx.y says
// which); a task is up to kAhead rows a lane group of one token's queries, keys
// or values, and goes to one warp.
struct RopeShape {
  int tokens, tasks;
};

__device__ __forceinline__ float2 unpack2(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t pack2(const float2 v) {
  const __nv_bfloat162 o = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&o);
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeParams p, const RopeShape sh) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = 32 / kLanes;      // rows of a warp at a time
  constexpr int kRows = kGroups * kAhead;   // of a task
  // Cosine and sine of every pair, by token; pairs four by four, cosines first.
  __shared__ float4 turn[kMaxTokens][D / 4];
  const int tid = threadIdx.x, warp = tid >> 5, sub = tid % kLanes, group = tid % 32 / kLanes;
  const int t0 = blockIdx.x * sh.tokens;
  const int nt = min(sh.tokens, p.T - t0);
  const int nq = (p.Hq + kRows - 1) / kRows, nk = (p.Hk + kRows - 1) / kRows,
            nv = (p.Hv + kRows - 1) / kRows;
  const int first = blockIdx.y * sh.tasks;
  const int per = min(sh.tasks, nq + nk + nv - first);  // of one token here
  const int F = p.rotary / 2;
  // This lane's elements: four from e0, four from e1.  Half layout: pairs
  // (e0 + i, e1 + i) for the first F / 4 lanes, eight neighbours for the rest.
  const bool turned = kInterleaved ? 8 * sub < p.rotary : 4 * sub < F;
  const int e0 = kInterleaved ? 8 * sub : turned ? 4 * sub : 2 * F + 8 * (sub - F / 4);
  const int e1 = !kInterleaved && turned ? e0 + F : e0 + 4;
  const int first_pair = kInterleaved ? e0 / 2 : e0;  // of four

  for (int i = tid; i < nt * F; i += kThreads) {
    const int tt = i / F, f = i - tt * F;
    const int64_t pos = __ldg(p.positions + t0 + tt);
    const uint64_t angle = __ldg(p.turns + f) * static_cast<uint64_t>(pos);
    // The nearest quarter turn, and what is left of an eighth turn at most, which fp32
    // holds to 2^-28 turns (half turns for sincospif).
    const uint64_t quarter = (angle + (uint64_t(1) << 61)) >> 62;
    const float rest = __ll2float_rn(static_cast<int64_t>(angle - (quarter << 62))) * 0x1p-63f;
    float s0, c0;
    sincospif(rest, &s0, &c0);
    const float s1 = quarter & 1 ? c0 : s0, c1 = quarter & 1 ? s0 : c0;
    const float sn = quarter & 2 ? -s1 : s1;
    const float cs = (quarter + 1) & 2 ? -c1 : c1;
    float* to = reinterpret_cast<float*>(&turn[tt][f / 4 * 2]) + f % 4;
    to[0] = cs * p.rope_scale;
    to[4] = sn * p.rope_scale;
  }
  bool ready = false;  // the table: waited for with the first rows' loads in flight

  for (int task = warp; task < nt * per || !ready; task += kWarps) {
    const bool none = task >= nt * per;
    const int tt = none ? 0 : task / per;
    const int c = first + (none ? 0 : task - tt * per);
    const int64_t t = t0 + tt;
    // What the task takes: kind 0 queries, 1 keys, 2 values.
    const int kind = c < nq ? 0 : c < nq + nk ? 1 : 2;
    const int h0 = (kind == 0 ? c : kind == 1 ? c - nq : c - nq - nk) * kRows + group;
    const int H = none ? 0 : kind == 0 ? p.Hq : kind == 1 ? p.Hk : p.Hv;
    const uint16_t* src = (kind == 0   ? p.q + t * p.q_stride
                           : kind == 1 ? p.k + t * p.k_stride
                                       : p.v + t * p.v_stride) + h0 * D;
    uint4 raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h0 + i * kGroups < H) {
        if constexpr (kInterleaved) {
          raw[i] = *reinterpret_cast<const uint4*>(src + i * kGroups * D + e0);
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(src + i * kGroups * D + e0);
          const uint2 b = *reinterpret_cast<const uint2*>(src + i * kGroups * D + e1);
          raw[i] = make_uint4(a.x, a.y, b.x, b.y);
        }
      }
    }
    // Where it goes: rows `pitch` elements apart.
    uint16_t* dst = kind == 0 ? p.q_out : kind == 1 ? p.k_out : p.v_out;
    int64_t pitch = D;
    bool skip = none;
    if (kind > 0 && p.slots) {
      const int64_t slot = __ldg(p.slots + t);
      const bool past = slot >= p.capacity;
      if (past && (tid & 31) == 0 && !none) record_error(p.err, kErrBadIndex);
      skip = skip || slot < 0 || past;
      dst += (((slot >> p.log_bs) * H << p.log_bs) + (slot & ((1 << p.log_bs) - 1))) * D;
      pitch = static_cast<int64_t>(D) << p.log_bs;
    } else {
      dst += t * H * D;
    }
    dst += h0 * pitch;
    if (!ready) {
      __syncthreads();
      ready = true;
    }
    if (skip) continue;
    auto store = [&](int i, const uint4 u) {
      uint16_t* to = dst + i * kGroups * pitch;
      if constexpr (kInterleaved) {
        *reinterpret_cast<uint4*>(to + e0) = u;
      } else {
        *reinterpret_cast<uint2*>(to + e0) = make_uint2(u.x, u.y);
        *reinterpret_cast<uint2*>(to + e1) = make_uint2(u.z, u.w);
      }
    };
    if (kind == 2) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h0 + i * kGroups < H) store(i, raw[i]);
      continue;
    }
    // out = rstd (x A + partner B), in pairs of neighbouring elements.
    const float* weight = kind == 0 ? p.q_weight : p.k_weight;
    float2 A[4], B[4];
    {
      float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
      if (turned) {
        cs = turn[tt][first_pair / 2];
        sn = turn[tt][first_pair / 2 + 1];
      }
      float4 w0 = make_float4(1.f, 1.f, 1.f, 1.f), w1 = w0;
      if (weight) {  // aligned to 4 bytes only
        w0 = make_float4(__ldg(weight + e0), __ldg(weight + e0 + 1), __ldg(weight + e0 + 2),
                         __ldg(weight + e0 + 3));
        w1 = make_float4(__ldg(weight + e1), __ldg(weight + e1 + 1), __ldg(weight + e1 + 2),
                         __ldg(weight + e1 + 3));
      }
      if constexpr (kInterleaved) {  // pairs (x, y) of a float2
        A[0] = make_float2(w0.x * cs.x, w0.y * cs.x);
        A[1] = make_float2(w0.z * cs.y, w0.w * cs.y);
        A[2] = make_float2(w1.x * cs.z, w1.y * cs.z);
        A[3] = make_float2(w1.z * cs.w, w1.w * cs.w);
        B[0] = make_float2(-w0.y * sn.x, w0.x * sn.x);
        B[1] = make_float2(-w0.w * sn.y, w0.z * sn.y);
        B[2] = make_float2(-w1.y * sn.z, w1.x * sn.z);
        B[3] = make_float2(-w1.w * sn.w, w1.z * sn.w);
      } else {  // pairs (x[q], x[q + 2])
        A[0] = make_float2(w0.x * cs.x, w0.y * cs.y);
        A[1] = make_float2(w0.z * cs.z, w0.w * cs.w);
        A[2] = make_float2(w1.x * cs.x, w1.y * cs.y);
        A[3] = make_float2(w1.z * cs.z, w1.w * cs.w);
        B[0] = make_float2(-w1.x * sn.x, -w1.y * sn.y);
        B[1] = make_float2(-w1.z * sn.z, -w1.w * sn.w);
        B[2] = make_float2(w0.x * sn.x, w0.y * sn.y);
        B[3] = make_float2(w0.z * sn.z, w0.w * sn.w);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h0 - group + i * kGroups >= H) break;  // the whole warp
      float2 x[4] = {unpack2(raw[i].x), unpack2(raw[i].y), unpack2(raw[i].z), unpack2(raw[i].w)};
      float2 y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        y[q] = __fmul2_rn(x[q], A[q]);
        if (turned)
          y[q] = __ffma2_rn(kInterleaved ? make_float2(x[q].y, x[q].x) : x[q ^ 2], B[q], y[q]);
      }
      if (weight) {
        float2 ss = __fmul2_rn(x[0], x[0]);
#pragma unroll
        for (int q = 1; q < 4; ++q) ss = __ffma2_rn(x[q], x[q], ss);
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float rstd = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = __fmul2_rn(y[q], make_float2(rstd, rstd));
      }
      if (h0 + i * kGroups < H)
        store(i, make_uint4(pack2(y[0]), pack2(y[1]), pack2(y[2]), pack2(y[3])));
    }
  }
}

template <int D>
cudaError_t launch_d(const RopeParams& p, bool interleaved, cudaStream_t s) {
  constexpr int kRows = 32 / (D / 8) * kAhead;
  if (p.T <= 0) return cudaSuccess;
  const int per = (p.Hq + kRows - 1) / kRows + (p.Hk + kRows - 1) / kRows +
                  (p.Hv + kRows - 1) / kRows;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
  // A CTA takes up to eight tasks a warp: several tokens, or a share of one
  // token's tasks; fewer where that leaves SMs without work.
  RopeShape sh;
  int target = 8 * kWarps;
  while (target > kWarps / 2 &&
         static_cast<int64_t>(p.T) * per < static_cast<int64_t>(8) * sms * target)
    target /= 2;
  const int chunks = (per + target - 1) / target;
  sh.tasks = (per + chunks - 1) / chunks;
  sh.tokens = target / sh.tasks;
  if (sh.tokens < 1) sh.tokens = 1;
  if (sh.tokens > kMaxTokens) sh.tokens = kMaxTokens;
  const dim3 grid((p.T + sh.tokens - 1) / sh.tokens, (per + sh.tasks - 1) / sh.tasks);
  if (interleaved)
    rope_kernel<D, true><<<grid, kThreads, 0, s>>>(p, sh);
  else
    rope_kernel<D, false><<<grid, kThreads, 0, s>>>(p, sh);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int D, bool interleaved, cudaStream_t s) {
  return D == 64 ? launch_d<64>(p, interleaved, s) : launch_d<128>(p, interleaved, s);
}

}  // namespace dsa
