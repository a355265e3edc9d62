// Norms of queries and keys for each head with the position rotation, in one pass.
//
//   y = x r w, r = 1 / sqrt(mean(x^2) + eps) over a head's D elements (or y = x);
//   pair i of the first `rot` elements turns by a = position[axis(i)] inv_freq[i]:
//   (u, v) -> (u cos a - v sin a, v cos a + u sin a).
//
// GB300 mapping: a head is 8 to 32 lanes' with two runs of four elements a lane, the
// two that turn against each other where pairs are split over halves: a head stays in
// registers from one load to one store, pairs need no exchange, and a warp has two
// heads' (or pairs of heads') loads on the way. HBM bounds many tokens, launch and one
// trip of loads a few. The sines of a token are formed once for all of its heads, by a thread a pair
// and for up to eight tokens at once, into one of two tables in shared memory (one
// barrier a round).
//
// Angles: a / 2 pi counts whole turns, so the fraction of a turn that a position
// adds is kept as a 64-bit fixed-point number per thread and multiplied by the
// position modulo 2^64: off by 2^-52 of the turns made (the rounding of
// inv_freq / 2 pi), with no 64-bit floating-point instruction per token (GB300
// issues two of those a cycle and SM).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kUnroll = 2, kCtas = 4;

// four consecutive elements as loaded
template <bool F32>
struct Quad {
  uint32_t w[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* p) {
    if (F32) {
      const uint4 v = *static_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[F32 ? 2 : 0] = v.z, w[F32 ? 3 : 1] = v.w;
    } else {
      const uint2 v = *static_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
  }
  __device__ __forceinline__ void values(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = __uint_as_float(F32 ? w[F32 ? j : 0] : j % 2 ? w[j / 2] & 0xFFFF0000u : w[j / 2] << 16);
  }
};

// L: lanes of a head, each with two of its quads of elements; F32: the type of x
template <bool F32, int L>
__global__ void __launch_bounds__(kThreads, kCtas) qk_rope_kernel(RopeArgs a, int lead, int lead_log) {
  constexpr int HW = 32 / L;              // heads of a warp's load
  constexpr int kSize = F32 ? 4 : 2;      // bytes of an element
  __shared__ float2 turn[2][kThreads];    // (cos, sin) of the pairs of a round's tokens
  __shared__ __align__(16) float weight[2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ql = lane % L, half = a.rot / 2;
  // A lane's quads begin at e[0] and e[1]: where halves turn against each other the elements of a pair are the same
  // ones of its two quads; else, and past the turning elements, its quads are neighbours.
  const bool split = !a.interleaved && 4 * ql < half;
  const int e[2] = {split ? 4 * ql : 8 * ql, split ? 4 * ql + half : 8 * ql + 4};
  const bool in = e[0] < a.D, turns = e[0] < a.rot;
  pdl_wait();
  pdl_launch_dependents();

  // A round is kThreads / lead tokens; a thread forms the sines of one pair of one of them. The fraction of a turn per
  // position, times 2^64:
  const int pair = threadIdx.x & (lead - 1), my_token = threadIdx.x >> lead_log, tokens = kThreads >> lead_log;
  unsigned long long step = 0;
  const int32_t* my_pos = a.pos;
  if (pair < half) {
    const double t = a.inv_freq[pair] * 0.15915494309189533577;  // 1 / (2 pi)
    step = 2ull * (unsigned long long)__double2ll_rn((t - rint(t)) * 9223372036854775808.0);
    my_pos += (long long)(a.axis_bits[pair >> 4] >> (2 * (pair & 15)) & 3u) * a.T;
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < 2 * a.D; i += kThreads) {
    const int k = i >= a.D, e = i - k * a.D;
    const void* w = k ? a.k_w : a.q_w;
    weight[k][e] = !w ? 1.f : a.w_f32 ? static_cast<const float*>(w)[e] : bf16_bits_to_f32(static_cast<const uint16_t*>(w)[e]);
  }
  const int heads = a.Hq + a.Hkv, units = (heads + HW - 1) / HW;
  // a token's units go to kWarps / tokens warps (one round's tokens at most kWarps) of gridDim.y CTAs
  const int t_of = warp & (tokens - 1), per = kWarps / tokens;
  const int u0 = blockIdx.y * per + warp / tokens, du = gridDim.y * per;
  const float inv_d = 1.f / (float)a.D;
  const bool normed = a.q_w || a.k_w;

  int b = 0;
#pragma unroll 1
  for (int t0 = blockIdx.x * tokens; t0 < a.T; t0 += gridDim.x * tokens, b ^= 1) {
    const int t = t0 + t_of;
    const bool live = t < a.T && a.pos[min(t, a.T - 1)] >= 0;  // (the same for a warp)
    // rows of the token; the keys' so that they too are indexed by the head's number among all
    const char* q_in = static_cast<const char*>(a.q) + t * a.q_stride * kSize;
    const char* k_in = static_cast<const char*>(a.k) + (t * a.k_stride - a.Hq * a.D) * kSize;
    Quad<F32> raw[kUnroll][2];
    auto fetch = [&](int u) {
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        const int h = (u + n * du) * HW + lane / L;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int j = 0; j < kSize; ++j) raw[n][c].w[j] = 0u;
        }
        if (live && h < heads && in) {
          const char* src = h < a.Hq ? q_in : k_in;
#pragma unroll
          for (int c = 0; c < 2; ++c) raw[n][c].load(src + (h * a.D + e[c]) * kSize);
        }
      }
    };
    fetch(u0);  // on the way while the sines are formed
    if (pair < half && t0 + my_token < a.T) {
      const long long p = my_pos[t0 + my_token];
      const float half_turns = (float)(long long)(step * (unsigned long long)p) * 0x1p-63f;  // in [-1, 1]
      float s, c;
      sincospif(half_turns, &s, &c);
      turn[b][threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();  // (a table is written again two rounds later, past the next round's barrier)
    if (!live) continue;
    // split halves: four pairs (x[0][j], x[1][j]); else pairs (x[c][j], x[c][j + 1]), j even
    float cs[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = !turns ? 0 : split ? e[0] + j : e[0] / 2 + j;
      const float2 x = turn[b][t_of * lead + at];
      cs[j] = turns ? x.x : 1.f, sn[j] = turns ? x.y : 0.f;
    }
#pragma unroll 1
    for (int u = u0; u < units; u += kUnroll * du) {
      if (u != u0) fetch(u);
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        if (u + n * du >= units) break;
        const int h = (u + n * du) * HW + lane / L;
        const bool is_q = h < a.Hq;
        float x[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) raw[n][c].values(x + 4 * c);
        if (normed) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
          if (in && (is_q ? a.q_w != nullptr : a.k_w != nullptr)) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float4 g = *reinterpret_cast<const float4*>(weight[is_q ? 0 : 1] + e[c]);
              x[4 * c] = x[4 * c] * r * g.x, x[4 * c + 1] = x[4 * c + 1] * r * g.y;
              x[4 * c + 2] = x[4 * c + 2] * r * g.z, x[4 * c + 3] = x[4 * c + 3] * r * g.w;
            }
          }
        }
        if (turns) {
          if (split) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v = x[j], w = x[4 + j];
              x[j] = fmaf(v, cs[j], -w * sn[j]), x[4 + j] = fmaf(w, cs[j], v * sn[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v = x[2 * j], w = x[2 * j + 1];
              x[2 * j] = fmaf(v, cs[j], -w * sn[j]), x[2 * j + 1] = fmaf(w, cs[j], v * sn[j]);
            }
          }
        }
        if (h < heads && in) {
          const long long row = is_q ? (long long)t * a.Hq + h : (long long)t * a.Hkv + h - a.Hq;
          if (!is_q && a.k_out_f32) {
            float* dst = static_cast<float*>(a.k_out) + row * a.D;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<float4*>(dst + e[c]) = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
          } else {
            uint16_t* dst = (is_q ? a.q_out : static_cast<uint16_t*>(a.k_out)) + row * a.D;
#pragma unroll
            for (int c = 0; c < 2; ++c)
              *reinterpret_cast<uint2*>(dst + e[c]) =
                  make_uint2(f32_to_bf16x2(x[4 * c], x[4 * c + 1]), f32_to_bf16x2(x[4 * c + 2], x[4 * c + 3]));
          }
        }
      }
    }
  }
}

template <bool F32, int L>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream, bool pdl) {
  const int sms = device_sm_count(), units = (a.Hq + a.Hkv + 32 / L - 1) / (32 / L);
  // Threads per token of a round: its pairs, filled up to a power of two. A round takes as many tokens as keep the SMs
  // busy, eight at most (a warp each); few tokens: one a round, its heads over several CTAs, one to a warp.
  int lead_log = 5;
  while (1 << lead_log < a.rot / 2) ++lead_log;
  while (lead_log < 8 && (a.T + (kThreads >> lead_log) - 1) / (kThreads >> lead_log) < kCtas * sms) ++lead_log;
  const int tokens = kThreads >> lead_log, rounds = (a.T + tokens - 1) / tokens;
  const int parts = tokens > 1 ? 1 : std::min((units + kWarps - 1) / kWarps, std::max(1, 2 * sms / rounds));
  auto k = qk_rope_kernel<F32, L>;
  return launch_kernel(k, dim3(std::min(rounds, kCtas * sms), parts), dim3(kThreads), 0, stream, pdl, a, 1 << lead_log,
                       lead_log);
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs& a, cudaStream_t stream, bool pdl) {
  if (a.D <= 64) return a.x_f32 ? launch<true, 8>(a, stream, pdl) : launch<false, 8>(a, stream, pdl);
  if (a.D <= 128) return a.x_f32 ? launch<true, 16>(a, stream, pdl) : launch<false, 16>(a, stream, pdl);
  return a.x_f32 ? launch<true, 32>(a, stream, pdl) : launch<false, 32>(a, stream, pdl);
}

}  // namespace qg
