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
// inv_freq / 2 pi) and by 2^-64 turns a position (that of the fixed point: 2^-33
// turns at the farthest), with no 64-bit floating-point instruction per token
// (GB300 issues two of those a cycle and SM).
//
// Measured (32/8 heads of 128): 16384 tokens of bf16 rows 66 us for 336 MB (5.1 TB/s; the bytes' floor is 50): 54 M warp
// instructions, an issue in 70 % of the cycles, two thirds of them conversions, products and the rounding of elements.
// 4093 fp32 tokens of 16/8 heads with three axes 20.4 us (84 MB), one token 4.2. Three CTAs an SM of 80 registers; the
// next heads' loads are issued before the present ones are worked on (77 us without).
#include <cuda_runtime.h>

#include <algorithm>

#include "kv8.cuh"
#include "qg_common.cuh"
#include "qg_internal.h"

namespace qg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kUnroll = 2, kCtas = 3;

// four consecutive elements as loaded
template <bool F32>
struct Quad {
  uint32_t w[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* p, bool there) {
    if (!there) return;  // (the values are not used)
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
  const int units_q = (a.Hq + HW - 1) / HW, units_k = (a.Hkv + HW - 1) / HW;
  // a token's units go to kWarps / tokens warps (one round's tokens at most kWarps) of gridDim.y CTAs, the queries' first
  const int t_of = warp & (tokens - 1), per = kWarps / tokens;
  const int w0 = blockIdx.y * per + warp / tokens, du = gridDim.y * per;
  const int k0 = (w0 - units_q % du + du) % du;
  const float inv_d = 1.f / (float)a.D;
  const int at0 = (lane / L) * a.D + e[0], gap = e[1] - e[0], step_u = du * HW * a.D;

  int b = 0;
#pragma unroll 1
  for (int t0 = blockIdx.x * tokens; t0 < a.T; t0 += gridDim.x * tokens, b ^= 1) {
    const int t = t0 + t_of;
    const bool live = t < a.T && a.pos[min(t, a.T - 1)] >= 0;  // (the same for a warp)
    const char* q_in = static_cast<const char*>(a.q) + t * a.q_stride * kSize;
    const char* k_in = static_cast<const char*>(a.k) + t * a.k_stride * kSize;
    Quad<F32> next[kUnroll][2];  // the loads on the way: a group of units ahead of what is worked on
    // the warp's unit u of H heads and the kUnroll - 1 after it; a lane that has no head there reads the first one's
    auto fetch = [&](const char* src, int u, int H) {
#pragma unroll
      for (int n = 0; n < kUnroll; ++n) {
        const bool there = live && in && (u + n * du) * HW + lane / L < H;
        const int at = there ? u * HW * a.D + n * step_u + at0 : 0;
        next[n][0].load(src + at * kSize, live);
        next[n][1].load(src + (there ? at + gap : 0) * kSize, live);
      }
    };
    const bool no_q = w0 >= units_q;
    fetch(no_q ? k_in : q_in, no_q ? k0 : w0, no_q ? a.Hkv : a.Hq);  // on the way while the sines are formed
    if (pair < half && t0 + my_token < a.T) {
      const long long p = my_pos[t0 + my_token];
      const float half_turns = (float)(long long)(step * (unsigned long long)p) * 0x1p-63f;  // in [-1, 1]
      float s, c;
      sincospif(half_turns, &s, &c);
      turn[b][threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();  // (a table is written again two rounds later, past the next round's barrier)
    if (!live) continue;
    // Pair j of the lane's four is (x[0][j], x[1][j]) where halves are split, else x[j / 2][j % 2 * 2] and the next one:
    // (u, v) -> (u a - v b, v c + u d), with the weights in the factors.
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int H = side ? a.Hkv : a.Hq, units = side ? units_k : units_q, first = side ? k0 : w0;
      const bool normed = side ? a.k_w != nullptr : a.q_w != nullptr;
      const char* src = side ? k_in : q_in;
      if (first >= units) continue;
      float ca[4], cb[4], cc[4], cd[4];
      {
        const float4 w0_ = *reinterpret_cast<const float4*>(weight[side] + (in ? e[0] : 0)),
                     w1_ = *reinterpret_cast<const float4*>(weight[side] + (in ? e[1] : 0));
        const float w[8] = {w0_.x, w0_.y, w0_.z, w0_.w, w1_.x, w1_.y, w1_.z, w1_.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int at = !turns ? 0 : split ? e[0] + j : e[0] / 2 + j;
          const float2 x = turn[b][t_of * lead + at];
          const float c = turns ? x.x : 1.f, s = turns ? x.y : 0.f, wu = split ? w[j] : w[2 * j], wv = split ? w[4 + j] : w[2 * j + 1];
          ca[j] = c * wu, cb[j] = s * wv, cc[j] = c * wv, cd[j] = s * wu;
        }
      }
      const long long row = (long long)t * H * a.D;
      uint16_t* out16 = (side ? static_cast<uint16_t*>(a.k_out) : a.q_out) + row;
      float* out32 = static_cast<float*>(a.k_out) + row;
      const bool wide = side && a.k_out_f32;
#pragma unroll 1
      for (int u = first; u < units; u += kUnroll * du) {
        Quad<F32> raw[kUnroll][2];
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) raw[n][0] = next[n][0], raw[n][1] = next[n][1];
        if (u + kUnroll * du < units)
          fetch(src, u + kUnroll * du, H);
        else if (side == 0 && k0 < units_k)
          fetch(k_in, k0, a.Hkv);
#pragma unroll
        for (int n = 0; n < kUnroll; ++n) {
          if (u + n * du >= units) break;
          float x[8];
          raw[n][0].values(x);
          raw[n][1].values(x + 4);
          float r = 1.f;
          if (normed) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            ss = in ? ss : 0.f;
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            r = rsqrtf(fmaf(ss, inv_d, a.eps));
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= r;
          float y[8];
          if (split) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[j] = fmaf(x[j], ca[j], -x[4 + j] * cb[j]);
              y[4 + j] = fmaf(x[4 + j], cc[j], x[j] * cd[j]);
            }
          } else if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              y[2 * j] = fmaf(x[2 * j], ca[j], -x[2 * j + 1] * cb[j]);
              y[2 * j + 1] = fmaf(x[2 * j + 1], cc[j], x[2 * j] * cd[j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[2 * j] = x[2 * j] * ca[j], y[2 * j + 1] = x[2 * j + 1] * cc[j];
          }
          if (in && (u + n * du) * HW + lane / L < H) {
            const int at = u * HW * a.D + n * step_u + at0;
            if (wide) {
              *reinterpret_cast<float4*>(out32 + at) = make_float4(y[0], y[1], y[2], y[3]);
              *reinterpret_cast<float4*>(out32 + at + gap) = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              *reinterpret_cast<uint2*>(out16 + at) = make_uint2(f32_to_bf16x2(y[0], y[1]), f32_to_bf16x2(y[2], y[3]));
              *reinterpret_cast<uint2*>(out16 + at + gap) = make_uint2(f32_to_bf16x2(y[4], y[5]), f32_to_bf16x2(y[6], y[7]));
            }
          }
        }
      }
    }
  }
}

template <bool F32, int L>
cudaError_t launch(const RopeArgs& a, cudaStream_t stream, bool pdl) {
  const int sms = device_sm_count(), units = (a.Hq + 32 / L - 1) / (32 / L) + (a.Hkv + 32 / L - 1) / (32 / L);
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
