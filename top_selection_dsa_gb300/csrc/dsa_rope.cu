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
// floating point, and an error below 2^-31 turns at every position of 32 bits.
//
// Every element needs only its own and its partner's input:
//   out_i = rstd (x_i A_i + x_partner B_i),  A = w_i m cos,  B = +-w_partner m sin
// so a CTA writes A and B of its tokens to shared memory once and applies them
// to all heads.  D / 8 lanes take a row, 16 bytes each; the partner's elements
// come by shuffles.  The pass is memory-bound.
#include <cuda_bf16.h>

#include "dsa_common.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // of a CTA
constexpr int kAhead = 4;      // rows whose loads a lane has in flight

struct RopeShape {
  int tokens;  // of a CTA
  int rows;    // of one token that a CTA takes (blockIdx.y: which)
};

__device__ __forceinline__ void unpack8(const uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

template <int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p, const RopeShape sh) {
  constexpr int kLanes = D / 8;
  constexpr int kGroups = kThreads / kLanes;
  // A and B of every element, for queries and for keys of each token.
  __shared__ float2 ab[kMaxTokens][2][D];
  const int tid = threadIdx.x, sub = tid % kLanes, group = tid / kLanes;
  const int heads = p.Hq + p.Hk + p.Hv;
  const int h0 = blockIdx.y * sh.rows;
  const int hn = min(sh.rows, heads - h0);  // rows of one token here
  const int t0 = blockIdx.x * sh.tokens;
  const int nt = min(sh.tokens, p.T - t0);
  const int rows = nt * hn;

  // Row `i` of this CTA: what it is, and where it comes from.
  struct Row {
    int t, h, kind;  // kind 0 query, 1 key, 2 value
  };
  auto row_of = [&](int i) {
    Row r;
    const int tt = i / hn;
    const int h = h0 + (i - tt * hn);
    r.t = t0 + tt;
    r.kind = h < p.Hq ? 0 : h < p.Hq + p.Hk ? 1 : 2;
    r.h = r.kind == 0 ? h : r.kind == 1 ? h - p.Hq : h - p.Hq - p.Hk;
    return r;
  };
  auto fetch = [&](int i) {
    if (i >= rows) return make_uint4(0u, 0u, 0u, 0u);
    const Row r = row_of(i);
    const uint16_t* src = r.kind == 0   ? p.q + r.t * p.q_stride
                          : r.kind == 1 ? p.k + r.t * p.k_stride
                                        : p.v + r.t * p.v_stride;
    return *(reinterpret_cast<const uint4*>(src + r.h * D) + sub);
  };
  uint4 raw[kAhead];
#pragma unroll
  for (int a = 0; a < kAhead; ++a) raw[a] = fetch(group + a * kGroups);

  const int F = p.rotary / 2;
  for (int i = tid; i < nt * 2 * D; i += kThreads) {
    const int e = i % D, which = i / D & 1, tt = i / (2 * D);
    if ((which == 0 ? p.Hq : p.Hk) == 0) continue;
    const float* weight = which == 0 ? p.q_weight : p.k_weight;
    float2 c = make_float2(weight ? __ldg(weight + e) : 1.f, 0.f);
    if (e < p.rotary) {
      const int f = kInterleaved ? e >> 1 : e < F ? e : e - F;
      const bool second = kInterleaved ? (e & 1) != 0 : e >= F;
      const int partner = kInterleaved ? e ^ 1 : second ? e - F : e + F;
      const uint64_t angle =
          __ldg(p.turns + f) * static_cast<uint64_t>(static_cast<int64_t>(__ldg(p.positions + t0 + tt)));
      float sn, cs;
      // Half turns in [-1, 1).
      sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &sn, &cs);
      c.x *= cs * p.rope_scale;
      c.y = (weight ? __ldg(weight + partner) : 1.f) * (sn * p.rope_scale);
      if (!second) c.y = -c.y;
    }
    ab[tt][which][e] = c;
  }
  __syncthreads();

  const bool turned = sub * 8 < p.rotary;  // whole lanes: rotary is a multiple of 16
  const int other = kInterleaved ? sub : sub * 8 < F ? sub + F / 8 : sub - F / 8;
  for (int base = group; base - group < rows; base += kAhead * kGroups) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = base + a * kGroups;
      if (i - group >= rows) break;  // the same for every group
      const uint4 u = raw[a];
      raw[a] = fetch(i + kAhead * kGroups);
      uint4 pu = u;
      if constexpr (!kInterleaved) {
        pu.x = __shfl_sync(0xffffffffu, u.x, other, kLanes);
        pu.y = __shfl_sync(0xffffffffu, u.y, other, kLanes);
        pu.z = __shfl_sync(0xffffffffu, u.z, other, kLanes);
        pu.w = __shfl_sync(0xffffffffu, u.w, other, kLanes);
      }
      float x[8], y[8];
      unpack8(u, x);
      unpack8(pu, y);
      float ss = 0.f;
#pragma unroll
      for (int q = 0; q < 8; ++q) ss = fmaf(x[q], x[q], ss);
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (i >= rows) continue;
      const Row r = row_of(i);
      uint16_t* dst;
      if (r.kind == 0) {
        dst = p.q_out + (static_cast<int64_t>(r.t) * p.Hq + r.h) * D;
      } else {
        const int H = r.kind == 1 ? p.Hk : p.Hv;
        uint16_t* out = r.kind == 1 ? p.k_out : p.v_out;
        if (p.slots) {
          const int64_t slot = __ldg(p.slots + r.t);
          if (slot < 0) continue;
          if (slot >= p.capacity) {
            if (sub == 0) record_error(p.err, kErrBadIndex);
            continue;
          }
          dst = out + ((((slot >> p.log_bs) * H + r.h) << p.log_bs) +
                       (slot & ((1 << p.log_bs) - 1))) * D;
        } else {
          dst = out + (static_cast<int64_t>(r.t) * H + r.h) * D;
        }
      }
      if (r.kind == 2) {
        *(reinterpret_cast<uint4*>(dst) + sub) = u;
        continue;
      }
      const float4* c4 = reinterpret_cast<const float4*>(&ab[r.t - t0][r.kind][8 * sub]);
      const bool norm = (r.kind == 0 ? p.q_weight : p.k_weight) != nullptr;
      const float rstd = norm ? rsqrtf(ss * (1.f / D) + p.eps) : 1.f;
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 c = c4[q];  // A, B of elements 2q and 2q + 1
        const float pa = kInterleaved ? x[2 * q + 1] : y[2 * q];
        const float pb = kInterleaved ? x[2 * q] : y[2 * q + 1];
        float oa = x[2 * q] * c.x, ob = x[2 * q + 1] * c.z;
        if (turned) {
          oa = fmaf(pa, c.y, oa);
          ob = fmaf(pb, c.w, ob);
        }
        const __nv_bfloat162 o = __floats2bfloat162_rn(oa * rstd, ob * rstd);
        w[q] = *reinterpret_cast<const uint32_t*>(&o);
      }
      *(reinterpret_cast<uint4*>(dst) + sub) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

template <int D>
cudaError_t launch_d(const RopeParams& p, bool interleaved, cudaStream_t s) {
  const int heads = p.Hq + p.Hk + p.Hv;
  if (p.T <= 0 || heads <= 0) return cudaSuccess;
  const int sms = device_sm_count() > 0 ? device_sm_count() : 1;
  constexpr int kGroups = kThreads / (D / 8);
  // A CTA takes about kAhead rows a lane group, all of them in flight at once:
  // several tokens of few heads, or a share of one token's heads; fewer rows
  // where that leaves SMs without work.
  RopeShape sh;
  int target = kAhead * kGroups;
  while (target > kGroups &&
         static_cast<int64_t>(p.T) * heads < static_cast<int64_t>(2) * sms * target)
    target /= 2;
  const int chunks = (heads + target - 1) / target;
  sh.rows = (heads + chunks - 1) / chunks;
  sh.tokens = target / sh.rows;
  if (sh.tokens < 1) sh.tokens = 1;
  if (sh.tokens > kMaxTokens) sh.tokens = kMaxTokens;
  const dim3 grid((p.T + sh.tokens - 1) / sh.tokens, (heads + sh.rows - 1) / sh.rows);
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
